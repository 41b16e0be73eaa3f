// key_weights.cu — the weight that each cached key gathers in a V2 decode
// step: w[j] = sum over the KV head's pairs p of |A_2p[j] - gate_p A_2p+1[j]|.
//
// A key's weight needs both maps' normalisers, which exist only after the
// whole sequence was read.  The decode's split kernel therefore stores its
// scaled scores t (log2 units, fp32); this kernel merges the partials' maxima
// and sums and takes A = exp2(t - max) / sum from them.  Scores in fewer bits
// would not do: an error e in t is an error of 0.7 e in the weight.  4 G bytes
// of scores per key are fewer than its K row's 2 d of bf16, so keeping them
// beats a second pass over K.
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 4;  // per thread, all loaded before the first is used

// P pairs of heads; block (1024 keys, KV head, sequence).
template <int P>
__global__ void __launch_bounds__(kThreads) key_weights_kernel(KeyWeightsArgs a) {
  constexpr int G = 2 * P;
  __shared__ float sm[G], sc[G];
  cudaGridDependencySynchronize();  // scores and partials
  const int g = blockIdx.y, b = blockIdx.z;
  const int L = a.seqlens ? a.seqlens[b] : a.L_max;
  if (L < 1 || L > a.L_max) return;  // recorded by the split kernel
  const int key0 = blockIdx.x * (kThreads * kKeys);
  if (key0 >= L) return;
  const int64_t unit = static_cast<int64_t>(b) * a.h_kv + g;
  const int64_t base = unit * a.L_max;
  // loads first: they do not wait for the normalisers
  float2 t[kKeys][P];
  float w[kKeys];
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int key = key0 + k * kThreads + threadIdx.x;
    if (key < L) {
      const float* s = a.scores + (base + key) * G;
      if constexpr (P % 2 == 0) {
#pragma unroll
        for (int p = 0; p < P; p += 2) {
          const float4 v = reinterpret_cast<const float4*>(s)[p / 2];
          t[k][p] = make_float2(v.x, v.y);
          t[k][p + 1] = make_float2(v.z, v.w);
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) t[k][p] = reinterpret_cast<const float2*>(s)[p];
      }
      w[k] = a.weights_in ? a.weights_in[base + key] : 0.f;
    }
  }
  // a warp per head, a lane per partial
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < G; r += kThreads / 32) {
    const int64_t head = static_cast<int64_t>(b) * 2 * a.h + g * G + r;
    if (a.norm) {
      if (lane == 0) {
        const float2 n = a.norm[head];
        sm[r] = n.x;
        sc[r] = (r & 1) ? n.y * a.gate[head / 2] : n.y;
      }
      continue;
    }
    float mt = -INFINITY, lt = 0.f;
    for (int i = lane; i < a.splits; i += 32) {
      const float2 ml = reinterpret_cast<const float2*>(a.part_ml)[i * static_cast<int64_t>(a.B) * 2 * a.h + head];
      const float top = fmaxf(mt, ml.x), nb = top == -INFINITY ? 0.f : top;
      lt = lt * exp2f(mt - nb) + ml.y * exp2f(ml.x - nb);
      mt = top;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, mt, o), l2 = __shfl_xor_sync(0xffffffffu, lt, o);
      const float top = fmaxf(mt, m2), nb = top == -INFINITY ? 0.f : top;
      lt = lt * exp2f(mt - nb) + l2 * exp2f(m2 - nb);
      mt = top;
    }
    if (lane == 0) {
      float c = lt == 0.f ? 0.f : 1.f / lt;
      if (r & 1) c *= a.gate[head / 2];
      sm[r] = mt == -INFINITY ? 0.f : mt;
      sc[r] = c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int key = key0 + k * kThreads + threadIdx.x;
    if (key >= L) continue;
    // products rounded before they are subtracted: equal maps cancel to zero
#pragma unroll
    for (int p = 0; p < P; ++p)
      w[k] += fabsf(__fsub_rn(__fmul_rn(exp2f(t[k][p].x - sm[2 * p]), sc[2 * p]),
                              __fmul_rn(exp2f(t[k][p].y - sm[2 * p + 1]), sc[2 * p + 1])));
    a.weights_out[base + key] = w[k];
  }
}

template <int P>
cudaError_t launch_pairs(const KeyWeightsArgs& a, cudaStream_t s) {
  const dim3 grid((a.L_max + kThreads * kKeys - 1) / (kThreads * kKeys), a.h_kv, a.B);
  return launch_ahead(key_weights_kernel<P>, grid, dim3(kThreads), 0, s, true, a);
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsArgs& a, cudaStream_t s) {
  switch (a.h / a.h_kv) {  // pairs per KV head
    case 1: return launch_pairs<1>(a, s);
    case 2: return launch_pairs<2>(a, s);
    case 3: return launch_pairs<3>(a, s);
    case 4: return launch_pairs<4>(a, s);
    case 5: return launch_pairs<5>(a, s);
    case 6: return launch_pairs<6>(a, s);
    case 7: return launch_pairs<7>(a, s);
    case 8: return launch_pairs<8>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace da
