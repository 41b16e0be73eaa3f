// kv4.cuh — how the 4-bit decode cuts its work, shared with the kernels that
// merge the parts.
//
// The work is a line of 32-key chunks, head after head (u = b * h_kv + g; a
// head of sequence b has ceil(L_b / 32) of them).  CTA c of `parts` takes
// chunks [floor(c T / parts), floor((c + 1) T / parts)) of the T in all, and
// writes its part of head u to partial c + u: heads and CTAs both only go up
// along the line, so no two parts share a number.
#pragma once

#include <stdint.h>

namespace da {

constexpr int kKv4ChunkKeys = 32;
// A CTA takes at least this many chunks: below it the parts cost more to
// merge than they save.
constexpr int kKv4MinPart = 8;
// CTAs at most (one per SM), and so partials of one head.
constexpr int kKv4MaxGrid = 512;

__host__ __device__ inline int64_t kv4_parts(int64_t total, int64_t grid) {
  const int64_t most = (total + kKv4MinPart - 1) / kKv4MinPart;
  return most < grid ? most : grid;
}

// The numbers of a head's first and last partial, left by the CTAs that take
// its first and its last chunk (a head without chunks has no entry).
struct Kv4Parts {
  int first, last;
};

}  // namespace da
