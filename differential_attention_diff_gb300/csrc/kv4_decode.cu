// kv4_decode.cu — V2 decode over a 4-bit KV cache (records of kv4.cu).
//
// Split-KV as in decode.cu: grid (splits, h_kv, B), partial (max, sum, O) per
// split and query head, then the same merge.  Each warp takes every eighth
// key of the split: its lanes hold D/32 features of the record's two rows,
// scores are reduced by shuffles, and the online softmax runs per warp.
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxG = 16;

__device__ __forceinline__ float bf16_at(uint2 par, int i) {
  const uint32_t w = i < 2 ? par.x : par.y;
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv4_split_kernel(Kv4DecodeArgs a) {
  constexpr int F = D / 32;  // features per lane, contiguous
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H2 = 2 * a.h, G = H2 / a.h_kv, qh0 = g * G;
  int L = a.seqlens ? a.seqlens[b] : a.L_max;
  if (L < 1 || L > a.L_max) {
    if (threadIdx.x == 0) record_status(a.status, DA_ERR_BOUNDS, 0x4B02);
    L = 0;
  }
  const int chunk = (L + a.num_splits - 1) / a.num_splits;
  const int k0 = min(L, split * chunk), k1 = min(L, k0 + chunk);

  float q[kMaxG][F], o[kMaxG][F], m[kMaxG], l[kMaxG];
#pragma unroll
  for (int r = 0; r < kMaxG; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      o[r][f] = 0.f;
      q[r][f] = r < G ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[(static_cast<int64_t>(b) * H2 + qh0 + r) * D +
                                                                                lane * F + f])
                      : 0.f;
    }
  }
  const uint8_t* base = static_cast<const uint8_t*>(a.cache.ptr) + b * a.cache.sb + g * a.cache.sh;
  for (int key = k0 + warp; key < k1; key += kWarps) {
    const uint8_t* rec = base + key * a.cache.sn;
    float kv[2][F];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint2 par = *reinterpret_cast<const uint2*>(rec + D + 8 * w);
      const float s = bf16_at(par, lane >> 4), mn = bf16_at(par, 2 + (lane >> 4));
#pragma unroll
      for (int f = 0; f < F; f += 2) {
        const uint32_t c = rec[w * (D / 2) + (lane * F + f) / 2];
        kv[w][f] = fmaf(s, static_cast<float>(c & 15u), mn);
        kv[w][f + 1] = fmaf(s, static_cast<float>(c >> 4), mn);
      }
    }
#pragma unroll
    for (int r = 0; r < kMaxG; ++r) {
      if (r >= G) break;
      float t = 0.f;
#pragma unroll
      for (int f = 0; f < F; ++f) t = fmaf(q[r][f], kv[0][f], t);
#pragma unroll
      for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
      t *= a.scale_log2;
      if (a.scores && lane == 0)
        a.scores[((static_cast<int64_t>(b) * a.h_kv + g) * a.L_max + key) * G + r] = t;
      const float mn = fmaxf(m[r], t);
      const float base_m = mn == -INFINITY ? 0.f : mn;
      const float al = exp2f(m[r] - base_m), p = exp2f(t - base_m);
      m[r] = mn;
      l[r] = l[r] * al + p;
#pragma unroll
      for (int f = 0; f < F; ++f) o[r][f] = fmaf(p, kv[1][f], o[r][f] * al);
    }
  }
  __shared__ float so[kWarps][kMaxG][D];
  __shared__ float sm[kWarps][kMaxG], sl[kWarps][kMaxG];
#pragma unroll
  for (int r = 0; r < kMaxG; ++r) {
    if (r >= G) break;
#pragma unroll
    for (int f = 0; f < F; ++f) so[warp][r][lane * F + f] = o[r][f];
    if (lane == 0) sm[warp][r] = m[r], sl[warp][r] = l[r];
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < G * D; idx += kWarps * 32) {
    const int r = idx / D, f = idx % D;
    float mt = -INFINITY, lt = 0.f, ot = 0.f;
    for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm[w][r]);
    const float base_m = mt == -INFINITY ? 0.f : mt;
    for (int w = 0; w < kWarps; ++w) {
      const float e = exp2f(sm[w][r] - base_m);
      lt += sl[w][r] * e;
      ot += so[w][r][f] * e;
    }
    const int64_t at = (static_cast<int64_t>(split) * a.B + b) * H2 + qh0 + r;
    a.part_o[at * D + f] = ot;
    if (f == 0) a.part_ml[at * 2] = mt, a.part_ml[at * 2 + 1] = lt;
  }
}

// One output head's splits merged, even - gate * odd.
__global__ void __launch_bounds__(128) kv4_merge_kernel(Kv4DecodeArgs a) {
  const int p = blockIdx.x, b = blockIdx.y, f = threadIdx.x, H2 = 2 * a.h;
  float res[2];
  for (int e = 0; e < 2; ++e) {
    float mt = -INFINITY, lt = 0.f, ot = 0.f;
    for (int s = 0; s < a.num_splits; ++s)
      mt = fmaxf(mt, a.part_ml[((static_cast<int64_t>(s) * a.B + b) * H2 + 2 * p + e) * 2]);
    const float base_m = mt == -INFINITY ? 0.f : mt;
    for (int s = 0; s < a.num_splits; ++s) {
      const int64_t at = (static_cast<int64_t>(s) * a.B + b) * H2 + 2 * p + e;
      const float c = exp2f(a.part_ml[at * 2] - base_m);
      lt += a.part_ml[at * 2 + 1] * c;
      ot += a.part_o[at * a.d + f] * c;
    }
    // a sum of 0 is an empty sequence or keys that are all -inf: zeros, as in decode.cu; NaN stays
    res[e] = lt == 0.f ? 0.f : ot / lt;
  }
  const int64_t at = static_cast<int64_t>(b) * a.h + p;
  static_cast<__nv_bfloat16*>(a.out)[at * a.d + f] =
      __float2bfloat16_rn(__fsub_rn(res[0], __fmul_rn(a.gate[at], res[1])));
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s) {
  const dim3 grid(a.num_splits, a.h_kv, a.B);
  if (a.d == 128)
    kv4_split_kernel<128><<<grid, kWarps * 32, 0, s>>>(a);
  else
    kv4_split_kernel<64><<<grid, kWarps * 32, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kv4_merge_kernel<<<dim3(a.h, a.B), a.d, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.weights_out == nullptr) return e;
  const KeyWeightsArgs w{a.B, a.h, a.h_kv, a.L_max, a.num_splits, a.seqlens, a.gate, a.part_ml, a.scores,
                         a.weights_in, a.weights_out};
  return launch_key_weights(w, s);
}

}  // namespace da
