// paged_merge.cu — joins the parts of the items that a share's end has cut
// (paged.cuh): the softmax rule over each part's maximum and sum, then even -
// gate * odd.
//
// Share c of the attention describes the item that it began and did not end, if
// there is one: the item's parts are slot 2c + 1 and then the slots 2c', c' = c + 1,
// ..., up to the share that ends it.  Every block reads all descriptions, and the
// items' pairs are dealt to the blocks; no more of them than run at once, since a
// block that finds nothing to do costs as much as one that does (32 sequences of
// 4096, d 64, 4 tokens: 7 us for 152 x 16 blocks, 3 for these).  An item of a
// prompt has many pairs and few parts (of many key tiles each): a warp takes a
// pair, d / 32 features of both heads to a lane, and nothing is shared.  One of a
// decode step has few pairs and may have many parts: the block takes a pair, its
// threads are the features times ways that share the parts, added in their order.
#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 2;
constexpr int kMaxShares = 1024;
constexpr int kFew = 8;          // parts that a warp joins by itself

template <int D>
struct Merge {
  const PagedArgs& a;
  PagedDesc d;
  int c, parts;
  __device__ __forceinline__ int64_t slot(int i, int row) const {
    return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.rows + row;
  }
  __device__ __forceinline__ int row(int pair) const {
    const int half = a.G / 2, tok = pair / half;
    return tok / a.tq1 * 128 + tok % a.tq1 * a.G + 2 * (pair % half);
  }
  __device__ __forceinline__ const float* part(int i, int row, int col) const {
    return a.part_o + slot(i, 0) * D + static_cast<int64_t>(row) * a.part_row + (col >> 2) * a.part_group + (col & 3);
  }
  // of the pair, the output's token row and head
  __device__ __forceinline__ int64_t token(int pair) const { return d.token + pair / (a.G / 2); }
  __device__ __forceinline__ int head(int pair) const { return d.g * (a.G / 2) + pair % (a.G / 2); }
  __device__ __forceinline__ __nv_bfloat16* out(int pair, int col) const {
    return static_cast<__nv_bfloat16*>(a.out.ptr) + token(pair) * a.out.st + head(pair) * a.out.sh + col;
  }
};

// The weight of part `lane` of a head's row (lanes from `parts` on: 0), and 1 / sum.
__device__ __forceinline__ float part_weight(const float* part_ml, int64_t slot, bool there, float* inv) {
  const float2 ml = there ? *reinterpret_cast<const float2*>(part_ml + slot * 2) : make_float2(-INFINITY, 0.f);
  float m = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float f = exp2f(ml.x - (m == -INFINITY ? 0.f : m));
  float l = ml.y * f;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
  *inv = 1.f / l;
  return f;
}

template <int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
paged_merge_kernel(PagedArgs a) {
  constexpr int kWays = kThreads / D;
  __shared__ float weight[2][kMaxShares];
  __shared__ float inv[2];
  __shared__ float sums[kWays][2][D];
  __shared__ uint8_t flags[kMaxShares];
  __shared__ int16_t open[kMaxShares];  // the shares that left an item open, in order
  __shared__ int counts[kWarps];
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int shares = a.grid * a.turns;
  cudaGridDependencySynchronize();  // the parts (and, behind them, the gate)
  int n_open = 0;
  for (int c0 = 0; c0 < shares; c0 += kThreads) {
    const int c = c0 + tid, f = c < shares ? a.desc[c].flags : 0;
    if (c < shares) flags[c] = static_cast<uint8_t>(f);
    const uint32_t mask = __ballot_sync(0xffffffffu, f & kPagedOpen);
    if (lane == 0) counts[warp] = __popc(mask);
    __syncthreads();
    int before = n_open;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += counts[w];
      n_open += counts[w];
    }
    if (f & kPagedOpen) open[before + __popc(mask & ((1u << lane) - 1))] = static_cast<int16_t>(c);
    __syncthreads();
  }
  // a unit of work: the block's eight warps' pairs, or one pair where that fills fewer blocks
  const int most = a.tq * (a.G / 2), per = n_open * most <= static_cast<int>(gridDim.x) ? 1 : kWarps;
  const int groups = (most + per - 1) / per;
  for (int unit = blockIdx.x; unit < n_open * groups; unit += gridDim.x) {
    const int c = open[unit / groups], first = unit % groups * per;
    if (tid == 0) last = shares - 1;
    __syncthreads();
    // the share that ends the item: the first of those that follow that ends one
    for (int x = c + 1 + tid; x < shares; x += kThreads)
      if (flags[x] & kPagedEnds) {
        atomicMin(&last, x);
        break;
      }
    Merge<D> mg{a, a.desc[c], c, 0};
    const int pairs = min(mg.d.tokens * (a.G / 2), first + per);
    __syncthreads();
    const int parts = mg.parts = last - c + 1;
    __syncthreads();
    if (parts <= kFew) {
      constexpr int kPer = D / 32;
      if (const int pair = first + warp; pair < pairs) {
        const int row = mg.row(pair);
        const float g = a.gate[mg.token(pair) * a.h + mg.head(pair)];
        float x[2][kFew][kPer], o[2][kPer], iv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i = 0; i < kFew; ++i) {
            const float* po = mg.part(i, row + e, lane * kPer);
            if constexpr (kPer == 4)
              *reinterpret_cast<float4*>(x[e][i]) = i < parts ? *reinterpret_cast<const float4*>(po) : make_float4(0, 0, 0, 0);
            else
              *reinterpret_cast<float2*>(x[e][i]) = i < parts ? *reinterpret_cast<const float2*>(po) : make_float2(0, 0);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = part_weight(a.part_ml, mg.slot(lane < parts ? lane : 0, row + e), lane < parts, &iv[e]);
#pragma unroll
          for (int q = 0; q < kPer; ++q) o[e][q] = 0.f;
#pragma unroll
          for (int i = 0; i < kFew; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
            for (int q = 0; q < kPer; ++q) o[e][q] = i < parts ? fmaf(x[e][i][q], w, o[e][q]) : o[e][q];
          }
        }
        uint32_t y[kPer / 2];
        const float c0 = iv[0], c1 = iv[1] * g;
#pragma unroll
        for (int q = 0; q < kPer / 2; ++q)  // the products rounded apart, so that equal heads cancel with gate 1
          y[q] = pack_bf16x2(__fsub_rn(__fmul_rn(o[0][2 * q], c0), __fmul_rn(o[1][2 * q], c1)),
                             __fsub_rn(__fmul_rn(o[0][2 * q + 1], c0), __fmul_rn(o[1][2 * q + 1], c1)));
        uint32_t* dst = reinterpret_cast<uint32_t*>(mg.out(pair, lane * kPer));
#pragma unroll
        for (int q = 0; q < kPer / 2; ++q) dst[q] = y[q];
      }
      continue;
    }
    const int col = tid % D, way = tid / D;
    for (int pair = first; pair < pairs; ++pair) {
      const int row = mg.row(pair);
      // the parts' weights: warp e takes head e of the pair
      if (warp < 2) {
        float m = -INFINITY;
        for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.part_ml[mg.slot(i, row + warp) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        for (int i = lane; i < parts; i += 32) {
          const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + mg.slot(i, row + warp) * 2);
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
        const float* o = mg.part(i, row, col);
        o0 = fmaf(o[0], weight[0][i], o0);
        o1 = fmaf(o[a.part_row], weight[1][i], o1);
      }
      sums[way][0][col] = o0;
      sums[way][1][col] = o1;
      __syncthreads();
      if (way == 0) {
        for (int w = 1; w < kWays; ++w) {
          o0 += sums[w][0][col];
          o1 += sums[w][1][col];
        }
        const float g = a.gate[mg.token(pair) * a.h + mg.head(pair)];
        *mg.out(pair, col) = __float2bfloat16_rn(__fsub_rn(__fmul_rn(o0, inv[0]), __fmul_rn(o1, inv[1] * g)));
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t s) {
  if (a.grid * a.turns > kMaxShares) return cudaErrorInvalidValue;
  if (a.grid * a.turns < 2) return cudaSuccess;  // one share cuts nothing
  const dim3 grid(a.grid * kBlocksPerSm);
  if (a.cache.d == 128) return launch_ahead(paged_merge_kernel<128>, grid, dim3(kThreads), 0, s, true, a);
  return launch_ahead(paged_merge_kernel<64>, grid, dim3(kThreads), 0, s, true, a);
}

}  // namespace da
