// key_weights.cu — the end of a V2 decode step that gathers the keys' weights,
//   w[j] = sum over the KV head's pairs p of |A_2p[j] - gate_p A_2p+1[j]|.
//
// A key's weight needs both maps' normalisers, which exist only after the
// whole sequence was read.  The decode's split kernel therefore stores its
// scaled scores t (log2 units, fp32); this kernel takes A = exp2(t - max) / sum
// from them.  Scores in fewer bits would not do: an error e in t is an error
// of 0.7 e in the weight.  Stored and read, that is 8 G bytes per key.  A second
// pass over K instead would read its row's 2 d of bf16 and compute the scores
// again, which is fewer bytes nowhere (G up to 16; equal at d 64); over a 4-bit
// cache it would read d/2 + 8, which is fewer from G = 10 on at d 128 and from
// G = 6 at d 64 (not built).
//
// Over a bf16 cache the same launch merges the splits, in its first blocks: in
// two launches that cost 22 us for 8 ragged sequences up to 4096 keys, in one
// 19.4.  Over a 4-bit cache the merge has left the normalisers.  Bound by the
// scores' traffic: 32 x 16384 keys of 8 heads, 168 MB, 31 us under the profiler.
#include "common.cuh"
#include "decode_merge.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 4;  // per thread, all loaded before the first is used
constexpr int kBlockKeys = kThreads * kKeys;

// A head's maximum and 1 / sum: from the table, or over the splits by a warp.  A
// sum of 0 is keys that are all -inf: zero weights; NaN stays.
__device__ __forceinline__ float2 head_norm(const FinishArgs& a, int64_t head) {
  if (a.norm) return a.norm[head];
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + head;
  const int64_t step = static_cast<int64_t>(a.B) * 2 * a.h;
  const int lane = threadIdx.x & 31;
  float mt = -INFINITY, lt = 0.f;
  for (int i = lane; i < a.splits; i += 32) mt = fmaxf(mt, ml[i * step].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
  mt = mt == -INFINITY ? 0.f : mt;
  for (int i = lane; i < a.splits; i += 32) lt += ml[i * step].y * exp2f(ml[i * step].x - mt);
#pragma unroll
  for (int o = 16; o; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
  return make_float2(mt, lt == 0.f ? 0.f : 1.f / lt);
}

// P pairs of heads per KV head.  Blocks: the merge's, then (1024 keys, KV
// head, sequence).
template <int P>
__global__ void __launch_bounds__(kThreads) decode_finish_kernel(FinishArgs a, int merge_blocks) {
  constexpr int G = 2 * P;
  // Scores and partials.  Over a 4-bit cache they were there before the merge
  // that runs ahead of this kernel let it start; only the normalisers are
  // waited for, below.
  if (!a.norm) cudaGridDependencySynchronize();
  const int tid = threadIdx.x;
  if (blockIdx.x < static_cast<unsigned>(merge_blocks)) {
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * (kThreads / a.d) + tid / a.d;
    if (pair >= static_cast<int64_t>(a.B) * a.h) return;
    const int b = static_cast<int>(pair / a.h), p = static_cast<int>(pair % a.h), col = tid % a.d;
    float res[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      res[e] = merged_head(a.part_o, a.part_ml, a.splits, a.B, 2 * a.h, a.d, b, 2 * p + e, col);
    store_pair(a.out, a.gate, pair, a.d, col, res[0], res[1]);
    return;
  }
  __shared__ float sm[G], sc[G];
  const unsigned block = blockIdx.x - merge_blocks, per = (a.L_max + kBlockKeys - 1) / kBlockKeys;
  const int64_t unit = block / per;
  const int b = static_cast<int>(unit / a.h_kv);
  const int key0 = static_cast<int>(block % per) * kBlockKeys;
  const int L = a.seqlens ? a.seqlens[b] : a.L_max;
  if (L < 1 || L > a.L_max || key0 >= L) {  // a bad length is recorded by the split kernel
    if (a.norm) cudaGridDependencySynchronize();
    return;
  }
  const int64_t base = unit * a.L_max;
  // loads first: they do not wait for the normalisers (and go to L2, as nothing
  // has been waited for yet that would say what L1 holds)
  float2 t[kKeys][P];
  float w[kKeys];
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int key = key0 + k * kThreads + tid;
    if (key < L) {
      const float* s = a.scores + (base + key) * G;
      if constexpr (P % 2 == 0) {
#pragma unroll
        for (int p = 0; p < P; p += 2) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + p / 2);
          t[k][p] = make_float2(v.x, v.y);
          t[k][p + 1] = make_float2(v.z, v.w);
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) t[k][p] = __ldcg(reinterpret_cast<const float2*>(s) + p);
      }
      w[k] = a.weights_in ? __ldcg(a.weights_in + base + key) : 0.f;
    }
  }
  if (a.norm) cudaGridDependencySynchronize();
  for (int r = tid >> 5; r < G; r += kWarps) {
    const float2 n = head_norm(a, unit * G + r);
    if ((tid & 31) == 0) {
      sm[r] = n.x;
      sc[r] = (r & 1) ? n.y * a.gate[unit * P + r / 2] : n.y;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int key = key0 + k * kThreads + tid;
    if (key >= L) continue;
    // products rounded before they are subtracted: equal maps cancel to zero
#pragma unroll
    for (int p = 0; p < P; ++p)
      w[k] += fabsf(__fsub_rn(__fmul_rn(exp2f(t[k][p].x - sm[2 * p]), sc[2 * p]),
                              __fmul_rn(exp2f(t[k][p].y - sm[2 * p + 1]), sc[2 * p + 1])));
    a.weights_out[base + key] = w[k];
  }
}

}  // namespace

cudaError_t launch_decode_finish(const FinishArgs& a, cudaStream_t s) {
  const int64_t pairs = static_cast<int64_t>(a.B) * a.h, per = kThreads / a.d;
  const int64_t merge = a.out ? (pairs + per - 1) / per : 0;
  const int64_t blocks = merge + static_cast<int64_t>(a.B) * a.h_kv * ((a.L_max + kBlockKeys - 1) / kBlockKeys);
  if (blocks > 2147483647) return cudaErrorInvalidValue;
  const int m = static_cast<int>(merge);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  switch (a.h / a.h_kv) {  // pairs per KV head
    case 1: return launch_ahead(decode_finish_kernel<1>, grid, block, 0, s, true, a, m);
    case 2: return launch_ahead(decode_finish_kernel<2>, grid, block, 0, s, true, a, m);
    case 3: return launch_ahead(decode_finish_kernel<3>, grid, block, 0, s, true, a, m);
    case 4: return launch_ahead(decode_finish_kernel<4>, grid, block, 0, s, true, a, m);
    case 5: return launch_ahead(decode_finish_kernel<5>, grid, block, 0, s, true, a, m);
    case 6: return launch_ahead(decode_finish_kernel<6>, grid, block, 0, s, true, a, m);
    case 7: return launch_ahead(decode_finish_kernel<7>, grid, block, 0, s, true, a, m);
    case 8: return launch_ahead(decode_finish_kernel<8>, grid, block, 0, s, true, a, m);
  }
  return cudaErrorInvalidValue;
}

}  // namespace da
