// decode_merge.cuh — one head's key-range splits merged, shared by the V2
// decode's merge and by the kernel that also gathers the keys' weights, so
// that both give the same bits.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace da {

// Feature `col` of query head j of sequence b, over the splits in their order.
// A sum of 0 is an empty sequence or keys that are all -inf: zeros; NaN stays.
__device__ __forceinline__ float merged_head(const float* part_o, const float* part_ml, int num_splits, int B, int H2,
                                             int d, int b, int j, int col) {
  float mt = -INFINITY;
  for (int s = 0; s < num_splits; ++s)
    mt = fmaxf(mt, part_ml[((static_cast<int64_t>(s) * B + b) * H2 + j) * 2]);
  const float base = mt == -INFINITY ? 0.f : mt;
  float lt = 0.f, ot = 0.f;
  for (int s = 0; s < num_splits; ++s) {
    const int64_t pidx = (static_cast<int64_t>(s) * B + b) * H2 + j;
    const float f = exp2f(part_ml[pidx * 2] - base);
    lt += part_ml[pidx * 2 + 1] * f;
    ot += part_o[pidx * d + col] * f;
  }
  return lt == 0.f ? 0.f : ot / lt;
}

// Even - gate * odd, the two products rounded apart so that equal heads cancel.
__device__ __forceinline__ void store_pair(void* out, const float* gate, int64_t pair, int d, int col, float even, float odd) {
  static_cast<__nv_bfloat16*>(out)[pair * d + col] = __float2bfloat16_rn(__fsub_rn(even, __fmul_rn(gate[pair], odd)));
}

}  // namespace da
