// paged_merge.cu — joins the parts of the items that a share's end has cut
// (paged.cuh): the softmax rule over each part's maximum and sum, then even -
// gate * odd.
//
// Share c of the attention describes the item that it began and did not end, if
// there is one: the item's parts are slot 2c + 1 and then the slots 2c', c' = c + 1,
// ..., up to the share that ends it.  Every block reads all descriptions, and the
// items' pairs are dealt out; there are no more blocks than run at once, since one
// that finds nothing to do costs as much as one that does (32 sequences of 4096,
// d 64, 4 tokens: 7 us for 152 x 16 blocks, 3 for these).  An item of a prompt has
// many pairs and few parts (of many key tiles each): its pairs go to the warps, two
// at a time, d / 32 features of both heads to a lane, and nothing is shared.  One of
// a decode step has few pairs and may have many parts: a block takes a pair, its
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

// A pair (heads 2p and 2p + 1 of a token) of an item that is to be joined.
struct Pair {
  int c, parts;       // the share that began the item
  int row;            // of the even head in the parts
  int64_t token;
  int head;           // of the output
  __device__ __forceinline__ Pair() : c(0), parts(0) {}
  __device__ __forceinline__ Pair(const PagedArgs& a, const PagedDesc& d, int c_, int parts_, int pair) : c(c_), parts(parts_) {
    const int half = a.G / 2, tok = pair / half, p = pair - tok * half, tile = tok / a.tq1;
    row = tile * 128 + (tok - tile * a.tq1) * a.G + 2 * p;
    token = d.token + tok;
    head = d.g * half + p;
  }
  __device__ __forceinline__ int64_t slot(const PagedArgs& a, int i) const {
    return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.rows;
  }
  template <int D>
  __device__ __forceinline__ const float* part(const PagedArgs& a, int i, int e, int col) const {
    return a.part_o + slot(a, i) * D + static_cast<int64_t>(row + e) * a.part_row + (col >> 2) * a.part_group + (col & 3);
  }
  __device__ __forceinline__ float2 ml(const PagedArgs& a, int i, int e) const {
    return *reinterpret_cast<const float2*>(a.part_ml + (slot(a, i) + row + e) * 2);
  }
  __device__ __forceinline__ float gate(const PagedArgs& a) const { return a.gate[token * a.h + head]; }
  __device__ __forceinline__ __nv_bfloat16* out(const PagedArgs& a, int col) const {
    return static_cast<__nv_bfloat16*>(a.out.ptr) + token * a.out.st + head * a.out.sh + col;
  }
};

// A warp's join of a pair of up to kN parts: what it loads, and the rest.
template <int D, int kN>
struct Join {
  static constexpr int kPer = D / 32;
  float x[2][kN][kPer];
  float2 ml[2][kN];
  float g;
  __device__ __forceinline__ void load(const PagedArgs& a, const Pair& p, int lane) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const bool there = i < p.parts;
        const float* o = p.part<D>(a, there ? i : 0, e, lane * kPer);
        if constexpr (kPer == 4)
          *reinterpret_cast<float4*>(x[e][i]) = *reinterpret_cast<const float4*>(o);
        else
          *reinterpret_cast<float2*>(x[e][i]) = *reinterpret_cast<const float2*>(o);
        ml[e][i] = p.ml(a, there ? i : 0, e);
        if (!there) ml[e][i] = make_float2(-INFINITY, 0.f);
      }
    }
    g = p.gate(a);
  }
  __device__ __forceinline__ void finish(const PagedArgs& a, const Pair& p, int lane) const {
    float o[2][kPer];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = ml[e][0].x;
#pragma unroll
      for (int i = 1; i < kN; ++i) m = fmaxf(m, ml[e][i].x);
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) o[e][q] = 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float w = exp2f(ml[e][i].x - base);
        l = fmaf(ml[e][i].y, w, l);
#pragma unroll
        for (int q = 0; q < kPer; ++q) o[e][q] = i == 0 || i < p.parts ? fmaf(x[e][i][q], w, o[e][q]) : o[e][q];
      }
      const float scale = (e ? g : 1.f) / l;
#pragma unroll
      for (int q = 0; q < kPer; ++q) o[e][q] = __fmul_rn(o[e][q], scale);
    }
    uint32_t y[kPer / 2];
#pragma unroll
    for (int q = 0; q < kPer / 2; ++q)  // the products rounded apart, so that equal heads cancel with gate 1
      y[q] = pack_bf16x2(__fsub_rn(o[0][2 * q], o[1][2 * q]), __fsub_rn(o[0][2 * q + 1], o[1][2 * q + 1]));
    __nv_bfloat16* dst = p.out(a, lane * kPer);
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = y[0];
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
paged_merge_kernel(PagedArgs a) {
  constexpr int kWays = kThreads / D;
  __shared__ float weight[2][kMaxShares];
  __shared__ float inv[2];
  __shared__ float sums[kWays][2][D];
  __shared__ uint8_t flags[kMaxShares];
  __shared__ int16_t open[kMaxShares], parts[kMaxShares];  // the shares that left an item open, in order; its parts
  __shared__ int counts[kWarps];
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
  bool long_ones = false;
  for (int o = tid; o < n_open; o += kThreads) {
    int x = open[o] + 1;  // the share that ends the item: the first of those that follow that ends one
    while (x < shares - 1 && !(flags[x] & kPagedEnds)) ++x;
    const int n = x - open[o] + 1;
    parts[o] = static_cast<int16_t>(n);
    long_ones |= n > kFew;
  }
  long_ones = __syncthreads_or(long_ones);
  const int most = a.tq * (a.G / 2), all = n_open * most;
  // items of few parts: a warp takes two pairs at a time
  const int stride = static_cast<int>(gridDim.x) * kWarps;
  auto pair_at = [&](int w) {
    if (w >= all) return Pair();
    const int o = w / most, pair = w - o * most;
    const PagedDesc d = a.desc[open[o]];
    return parts[o] <= kFew && pair < d.tokens * (a.G / 2) ? Pair(a, d, open[o], parts[o], pair) : Pair();
  };
  for (int w = warp * gridDim.x + blockIdx.x; w < all; w += 2 * stride) {
    const Pair p0 = pair_at(w), p1 = pair_at(w + stride);
    if (p0.parts && p1.parts && max(p0.parts, p1.parts) <= 2) {
      Join<D, 2> j0, j1;
      j0.load(a, p0, lane);
      j1.load(a, p1, lane);
      j0.finish(a, p0, lane);
      j1.finish(a, p1, lane);
    } else {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const Pair p = k ? p1 : p0;
        if (!p.parts) continue;
        Join<D, kFew> j;
        j.load(a, p, lane);
        j.finish(a, p, lane);
      }
    }
  }
  if (!long_ones) return;
  const int col = tid % D, way = tid / D;
  for (int w = blockIdx.x; w < all; w += gridDim.x) {
    const int o = w / most, pair = w - o * most, n = parts[o];
    const PagedDesc d = a.desc[open[o]];
    if (n <= kFew || pair >= d.tokens * (a.G / 2)) continue;
    const Pair p(a, d, open[o], n, pair);
    // the parts' weights: warp e takes head e of the pair
    if (warp < 2) {
      float m = -INFINITY;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, p.ml(a, i, warp).x);
#pragma unroll
      for (int h = 16; h > 0; h /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, h));
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float2 ml = p.ml(a, i, warp);
        const float f = exp2f(ml.x - base);
        weight[warp][i] = f;
        l = fmaf(ml.y, f, l);
      }
#pragma unroll
      for (int h = 16; h > 0; h /= 2) l += __shfl_xor_sync(0xffffffffu, l, h);
      if (lane == 0) inv[warp] = 1.f / l;
    }
    __syncthreads();
    float o0 = 0.f, o1 = 0.f;
#pragma unroll 4
    for (int i = way; i < n; i += kWays) {
      const float* x = p.part<D>(a, i, 0, col);
      o0 = fmaf(x[0], weight[0][i], o0);
      o1 = fmaf(x[a.part_row], weight[1][i], o1);
    }
    sums[way][0][col] = o0;
    sums[way][1][col] = o1;
    __syncthreads();
    if (way == 0) {
      for (int v = 1; v < kWays; ++v) {
        o0 += sums[v][0][col];
        o1 += sums[v][1][col];
      }
      *p.out(a, col) = __float2bfloat16_rn(__fsub_rn(__fmul_rn(o0, inv[0]), __fmul_rn(o1, inv[1] * p.gate(a))));
    }
    __syncthreads();
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
