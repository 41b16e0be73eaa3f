// key_weights.cu — the weight that each cached key gathers in a V2 decode
// step: w[j] = sum over the KV head's pairs p of |A_2p[j] - gate_p A_2p+1[j]|.
//
// A key's weight needs both maps' normalisers, which exist only after the
// whole sequence was read.  The decode's split kernel therefore stores its
// scaled scores t (log2 units, fp32); this kernel merges the splits' maxima
// and sums and takes A = exp2(t - max) / sum from them.  Scores in fewer bits
// would not do: an error e in t is an error of 0.7 e in the weight.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxG = 16;

__global__ void __launch_bounds__(kThreads) key_weights_kernel(KeyWeightsArgs a) {
  const int g = blockIdx.y, b = blockIdx.z;
  const int H2 = 2 * a.h, G = H2 / a.h_kv;
  const int L = a.seqlens ? a.seqlens[b] : a.L_max;
  if (L < 1 || L > a.L_max) return;  // recorded by the split kernel
  if (static_cast<int64_t>(blockIdx.x) * kThreads >= L) return;
  __shared__ float sm[kMaxG], sc[kMaxG];
  if (threadIdx.x < G) {
    const int j = g * G + threadIdx.x;
    // this head's partials: one per split, or the parts of a line of chunks
    int64_t first = static_cast<int64_t>(b) * a.h_kv + g, step = static_cast<int64_t>(a.B) * a.h_kv;
    int count = a.splits;
    if (a.prefix) {
      const Kv4Parts s = kv4_head_parts(a.prefix, a.B, a.h_kv, b, g, a.splits);
      first = s.first;
      count = s.count;
      step = 1;
    }
    float mt = -INFINITY, lt = 0.f;
    for (int i = 0; i < count; ++i) mt = fmaxf(mt, a.part_ml[((first + i * step) * G + threadIdx.x) * 2]);
    const float base = mt == -INFINITY ? 0.f : mt;
    for (int i = 0; i < count; ++i) {
      const float* ml = a.part_ml + ((first + i * step) * G + threadIdx.x) * 2;
      lt += ml[1] * exp2f(ml[0] - base);
    }
    float c = lt == 0.f ? 0.f : 1.f / lt;
    if (threadIdx.x & 1) c *= a.gate[static_cast<int64_t>(b) * a.h + j / 2];
    sm[threadIdx.x] = base;
    sc[threadIdx.x] = c;
  }
  __syncthreads();
  const int key = blockIdx.x * kThreads + threadIdx.x;
  if (key >= L) return;
  const int64_t at = (static_cast<int64_t>(b) * a.h_kv + g) * a.L_max + key;
  const float* t = a.scores + at * G;
  float w = a.weights_in ? a.weights_in[at] : 0.f;
  // products rounded before they are subtracted: equal maps cancel to zero
  for (int r = 0; r < G; r += 2)
    w += fabsf(__fsub_rn(__fmul_rn(exp2f(t[r] - sm[r]), sc[r]), __fmul_rn(exp2f(t[r + 1] - sm[r + 1]), sc[r + 1])));
  a.weights_out[at] = w;
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsArgs& a, cudaStream_t s) {
  const dim3 grid((a.L_max + kThreads - 1) / kThreads, a.h_kv, a.B);
  key_weights_kernel<<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace da
