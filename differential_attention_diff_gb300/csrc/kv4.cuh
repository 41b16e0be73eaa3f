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

__host__ __device__ inline int64_t kv4_parts(int64_t total, int64_t grid) {
  const int64_t most = (total + kKv4MinPart - 1) / kKv4MinPart;
  return most < grid ? most : grid;
}

// The partials of head (b, g): numbers first .. first + count - 1.
struct Kv4Parts {
  int64_t first;
  int count;
};
__device__ inline Kv4Parts kv4_head_parts(const int64_t* prefix, int B, int h_kv, int b, int g, int grid) {
  const int64_t total = prefix[B] * h_kv, n = prefix[b + 1] - prefix[b];
  if (n == 0) return {0, 0};
  const int64_t parts = kv4_parts(total, grid);
  const int64_t from = prefix[b] * h_kv + g * n;
  // chunk x is in the last part that starts at or before it
  const int64_t c0 = ((from + 1) * parts - 1) / total, c1 = ((from + n) * parts - 1) / total;
  return {c0 + static_cast<int64_t>(b) * h_kv + g, static_cast<int>(c1 - c0 + 1)};
}

}  // namespace da
