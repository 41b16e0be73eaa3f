// kv4.cuh — how the 4-bit decode cuts its work, shared with the kernels that
// merge the parts.
//
// The work is a line of 32-key chunks, head after head (u = b * h_kv + g; a
// head of sequence b has ceil(L_b / 32) of them).  Warp w of `parts` takes
// chunks [floor(w T / parts), floor((w + 1) T / parts)) of the T in all, and
// writes its part of head u to partial w + u: heads and warps both only go up
// along the line, so no two parts share a number.
#pragma once

#include <stdint.h>

namespace da {

constexpr int kKv4ChunkKeys = 32;
constexpr int kKv4MaxGrid = 256;   // CTAs at most (one per SM)
constexpr int kKv4MaxWarps = 16;   // of each

// Parts of a line of `total` chunks for `warps` warps: a chunk each while half
// of the warps are enough for that (one sequence of 1000 keys and 8 KV heads, in
// a cache too long for blocks of its own, takes 10.8 us so, 11.7 us with two
// each), else at least two (8 of them: 12.9 and 11.6 us: below it the parts cost
// more to merge than they save).
__host__ __device__ inline int64_t kv4_parts(int64_t total, int64_t warps) {
  const int64_t most = total <= warps / 2 ? total : (total + 1) / 2;
  return most < warps ? most : warps;
}

// The numbers of a head's first and last partial, left by the warps that take
// its first and its last chunk (a head without chunks has no entry).
struct Kv4Parts {
  int first, last;
};

}  // namespace da
