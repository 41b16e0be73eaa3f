// paged_merge.cu — joins the parts of the items that a share's end has cut
// (paged.cuh): the softmax rule over each part's maximum and sum, then even -
// gate * odd.
//
// Block c of the grid's rows looks after the item that CTA c of the attention
// began and did not end, if there is one: its parts are slot 2c + 1 and then the
// slots 2c', c' = c + 1, ..., up to the CTA that ends it.  The item's pairs are
// dealt to the blocks (c, y); a block's threads are the head's features times
// ways that share the parts, and the ways are added in their order.
#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 1024;  // of an item: CTAs of a grid

template <int D>
__global__ void __launch_bounds__(kThreads)
paged_merge_kernel(PagedArgs a) {
  constexpr int kWays = kThreads / D;
  __shared__ float weight[2][kMaxParts];
  __shared__ float inv[2];
  __shared__ float sums[kWays][2][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  cudaGridDependencySynchronize();  // the parts (and, behind them, the gate)
  const PagedDesc d = a.desc[c];
  if (!(d.flags & kPagedOpen)) return;
  int parts = 1;  // and those of the CTAs that follow, up to the one that ends it
  for (int x = c + 1; x < a.grid; ++x) {
    ++parts;
    if (a.desc[x].flags & kPagedEnds) break;
  }
  const int t0 = a.cache.cu_seqlens[d.b], n = a.cache.cu_seqlens[d.b + 1] - t0;
  const int tokens = min(a.tq, n - d.i * a.tq), half = a.G / 2;
  const int col = tid % D, way = tid / D;
  for (int pair = blockIdx.y; pair < tokens * half; pair += gridDim.y) {
    const int tok = pair / half, p = pair % half;
    const int row = tok / a.tq1 * 128 + tok % a.tq1 * a.G + 2 * p;
    auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.rows + row; };
    // the parts' weights: warp e takes head e of the pair
    if (warp < 2) {
      float m = -INFINITY;
      for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.part_ml[(slot(i) + warp) * 2]);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f;
      for (int i = lane; i < parts; i += 32) {
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (slot(i) + warp) * 2);
        const float f = exp2f(ml.x - base);
        weight[warp][i] = f;
        l = fmaf(ml.y, f, l);
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) inv[warp] = 1.f / l;
    }
    __syncthreads();
    float o0 = 0.f, o1 = 0.f;
#pragma unroll 4
    for (int i = way; i < parts; i += kWays) {
      const float* o = a.part_o + slot(i) * D + col;
      o0 = fmaf(o[0], weight[0][i], o0);
      o1 = fmaf(o[D], weight[1][i], o1);
    }
    sums[way][0][col] = o0;
    sums[way][1][col] = o1;
    __syncthreads();
    if (way == 0) {
      for (int w = 1; w < kWays; ++w) {
        o0 += sums[w][0][col];
        o1 += sums[w][1][col];
      }
      const int64_t t = t0 + d.i * a.tq + tok;
      const int head = d.g * half + p;
      // the products rounded apart, so that equal heads cancel with gate 1
      const float y = __fsub_rn(__fmul_rn(o0, inv[0]), __fmul_rn(o1, inv[1] * a.gate[t * a.h + head]));
      static_cast<__nv_bfloat16*>(a.out.ptr)[t * a.out.st + head * a.out.sh + col] = __float2bfloat16_rn(y);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t s) {
  if (a.grid > kMaxParts) return cudaErrorInvalidValue;
  if (a.grid < 2) return cudaSuccess;  // one CTA cuts nothing
  const int pairs = a.tq * a.G / 2;
  const dim3 grid(a.grid - 1, pairs < 16 ? pairs : 16);
  if (a.cache.d == 128) return launch_ahead(paged_merge_kernel<128>, grid, dim3(kThreads), 0, s, true, a);
  return launch_ahead(paged_merge_kernel<64>, grid, dim3(kThreads), 0, s, true, a);
}

}  // namespace da
