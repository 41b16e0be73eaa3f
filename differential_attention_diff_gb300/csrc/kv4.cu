// kv4.cu — rows of a 4-bit KV cache: quantise bf16 key and value rows into
// records, and read records back as bf16 rows.
//
// A record (layout in diffattn.h) holds a key and a value row; each row has
// two groups of d/2 features with value = s * code + m, m the group's
// minimum and s = bf16(range / 15).  Both kernels give a row to d/8 lanes of
// 8 features each: one 16-byte access on the bf16 side and one 4-byte word of
// codes on the other, so a warp touches whole contiguous rows.  A group's
// minimum and maximum come from shuffles over its d/16 lanes.
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The rows that a sequence's start and count name; false (recorded once) if
// they leave the cache.
__device__ __forceinline__ bool sequence_rows(const Kv4RowsArgs& a, int b, bool report, int& start, int& count) {
  start = a.start ? a.start[b] : 0;
  count = a.counts ? a.counts[b] : a.N;
  if (start >= 0 && count >= 0 && count <= a.N && start <= a.L_max - count) return true;
  if (report) record_status(a.status, DA_ERR_BOUNDS, 0x4B01);
  return false;
}

// Row index r = (((b * N + i) * h_kv + g) * 2 + is_value); D / 8 lanes each.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(Kv4RowsArgs a) {
  constexpr int kLanes = D / 8;        // of a row
  constexpr int kGroupLanes = D / 16;  // of a group
  const int64_t rows = static_cast<int64_t>(a.B) * a.N * a.h_kv * 2;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = t / kLanes;
  const int l = threadIdx.x % kLanes;
  if (r >= rows) return;  // whole rows leave: the shuffles below stay inside a row
  const bool is_v = r & 1;
  int64_t u = r >> 1;
  const int g = static_cast<int>(u % a.h_kv);
  u /= a.h_kv;
  const int i = static_cast<int>(u % a.N), b = static_cast<int>(u / a.N);
  int start, count;
  if (!sequence_rows(a, b, i == 0 && g == 0 && l == 0, start, count) || i >= count) return;

  const da_t4& src = is_v ? a.v : a.k;
  const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(src.ptr) + b * src.sb + i * src.sn + g * src.sh;
  const uint4 w = *reinterpret_cast<const uint4*>(row + l * 8);
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_lo(ws[e]);
    x[2 * e + 1] = bf16_hi(ws[e]);
  }
  float lo = x[0], hi = x[0];
  bool nan = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    nan |= x[e] != x[e];
  }
  // a NaN is ignored by fminf / fmaxf: carry it as an infinite maximum
  if (nan) hi = INFINITY;
#pragma unroll
  for (int o = 1; o < kGroupLanes; o <<= 1) {
    const unsigned m = ((1ull << kGroupLanes) - 1) << ((threadIdx.x & 31) / kGroupLanes * kGroupLanes);
    lo = fminf(lo, __shfl_xor_sync(m, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(m, hi, o));
  }
  float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
  const bool bad = !(fabsf(s) < INFINITY);
  uint32_t codes = 0;
  if (!bad && s > 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float n = fminf(rintf(__fdiv_rn(__fsub_rn(x[e], lo), s)), 15.f);
      codes |= static_cast<uint32_t>(n) << (4 * e);
    }
  }
  if (bad) s = lo = NAN;

  uint8_t* rec = static_cast<uint8_t*>(a.cache.ptr) + b * a.cache.sb + (static_cast<int64_t>(start) + i) * a.cache.sn +
                 g * a.cache.sh;
  *reinterpret_cast<uint32_t*>(rec + (is_v ? D / 2 : 0) + l * 4) = codes;
  if (l % kGroupLanes == 0) {
    __nv_bfloat16* par = reinterpret_cast<__nv_bfloat16*>(rec + D + (is_v ? 8 : 0)) + l / kGroupLanes;
    par[0] = __float2bfloat16_rn(s);
    par[2] = __float2bfloat16_rn(lo);
  }
  if (!is_v && l == 0) {
    const int64_t at = (static_cast<int64_t>(b) * a.h_kv + g) * a.L_max + start + i;
    if (a.key_weights) a.key_weights[at] = 0.f;
    if (a.positions) a.positions[at] = (a.first_position ? a.first_position[b] : start) + i;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(Kv4RowsArgs a) {
  constexpr int kLanes = D / 8;
  const int64_t rows = static_cast<int64_t>(a.B) * a.N * a.h_kv * 2;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = t / kLanes;
  const int l = threadIdx.x % kLanes;
  if (r >= rows) return;
  const bool is_v = r & 1;
  int64_t u = r >> 1;
  const int g = static_cast<int>(u % a.h_kv);
  u /= a.h_kv;
  const int i = static_cast<int>(u % a.N), b = static_cast<int>(u / a.N);
  int start, count;
  if (!sequence_rows(a, b, i == 0 && g == 0 && l == 0, start, count) || i >= count) return;

  const uint8_t* rec = static_cast<const uint8_t*>(a.cache.ptr) + b * a.cache.sb +
                       (static_cast<int64_t>(start) + i) * a.cache.sn + g * a.cache.sh;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(rec + (is_v ? D / 2 : 0) + l * 4);
  const uint2 par = *reinterpret_cast<const uint2*>(rec + D + (is_v ? 8 : 0));
  const bool second = l >= kLanes / 2;
  const float s = second ? bf16_hi(par.x) : bf16_lo(par.x);
  const float m = second ? bf16_hi(par.y) : bf16_lo(par.y);
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    out[e] = pack_bf16x2(fmaf(s, static_cast<float>((codes >> (8 * e)) & 15u), m),
                         fmaf(s, static_cast<float>((codes >> (8 * e + 4)) & 15u), m));
  const da_t4& dst = is_v ? a.v : a.k;
  __nv_bfloat16* row = static_cast<__nv_bfloat16*>(dst.ptr) + b * dst.sb + i * dst.sn + g * dst.sh;
  *reinterpret_cast<uint4*>(row + l * 8) = make_uint4(out[0], out[1], out[2], out[3]);
}

unsigned blocks_for(const Kv4RowsArgs& a) {
  const int64_t threads = static_cast<int64_t>(a.B) * a.N * a.h_kv * 2 * (a.d / 8);
  return static_cast<unsigned>((threads + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s) {
  if (a.d == 128)
    kv4_append_kernel<128><<<blocks_for(a), kThreads, 0, s>>>(a);
  else
    kv4_append_kernel<64><<<blocks_for(a), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s) {
  if (a.d == 128)
    kv4_read_kernel<128><<<blocks_for(a), kThreads, 0, s>>>(a);
  else
    kv4_read_kernel<64><<<blocks_for(a), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace da
