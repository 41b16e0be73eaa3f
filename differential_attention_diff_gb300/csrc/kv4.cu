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

// A block's rows: kRows passes of kThreads / (D/8) rows each, out of the
// sequence's N * h_kv * 2 (row = (i * h_kv + g) * 2 + is_value).  Loading
// kRows rows before the first is used keeps enough bytes in flight.
constexpr int kRows = 4;

struct RowAt {
  bool live;
  bool is_v;
  int i, g;
};
__device__ __forceinline__ RowAt row_at(const Kv4RowsArgs& a, unsigned r, unsigned rows) {
  RowAt x;
  const unsigned u = r >> 1;
  x.is_v = r & 1;
  x.i = static_cast<int>(u / static_cast<unsigned>(a.h_kv));
  x.g = static_cast<int>(u % static_cast<unsigned>(a.h_kv));
  x.live = r < rows;
  return x;
}

// Quantisation needs the exactly rounded quotient only where it is near a tie
// between two codes; elsewhere a product with the reciprocal, off by at most
// 2^-21 of 15, rounds to the same code.
__device__ __forceinline__ uint32_t code_of(float t, float s, float inv) {
  float q = t * inv, n = rintf(q);
  if (!(fabsf(q - n) < 0.4999f)) n = rintf(__fdiv_rn(t, s));  // also where inv overflowed
  return static_cast<uint32_t>(fminf(n, 15.f));
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(Kv4RowsArgs a) {
  constexpr int kLanes = D / 8;        // of a row
  constexpr int kGroupLanes = D / 16;  // of a group
  constexpr int kPass = kThreads / kLanes;
  const int l = threadIdx.x % kLanes;
  const unsigned r0 = blockIdx.x * (kRows * kPass) + threadIdx.x / kLanes;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    int start, count;
    if (!sequence_rows(a, b, blockIdx.x == 0 && threadIdx.x == 0, start, count)) continue;
    const unsigned rows = static_cast<unsigned>(count) * a.h_kv * 2;
    if (blockIdx.x * (kRows * kPass) >= rows) continue;
    uint4 in[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const RowAt x = row_at(a, r0 + j * kPass, rows);
      const da_t4& src = x.is_v ? a.v : a.k;
      in[j] = make_uint4(0, 0, 0, 0);
      if (x.live)
        in[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src.ptr) + b * src.sb +
                                                      x.i * src.sn + x.g * src.sh + l * 8));
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const RowAt r = row_at(a, r0 + j * kPass, rows);
      const uint32_t ws[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
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
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
      const bool bad = !(fabsf(s) < INFINITY);
      uint32_t codes = 0;
      if (!bad && s > 0.f) {
        const float inv = __frcp_rn(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) codes |= code_of(__fsub_rn(x[e], lo), s, inv) << (4 * e);
      }
      if (bad) s = lo = NAN;
      // both groups' parameters at the row's first lane
      const uint32_t mine = pack_bf16x2(s, lo);
      const uint32_t other = __shfl_down_sync(0xffffffffu, mine, kGroupLanes);
      if (!r.live) continue;
      uint8_t* rec = static_cast<uint8_t*>(a.cache.ptr) + b * a.cache.sb +
                     (static_cast<int64_t>(start) + r.i) * a.cache.sn + r.g * a.cache.sh;
      *reinterpret_cast<uint32_t*>(rec + (r.is_v ? D / 2 : 0) + l * 4) = codes;
      if (l == 0) {
        *reinterpret_cast<uint2*>(rec + D + (r.is_v ? 8 : 0)) =
            make_uint2(__byte_perm(mine, other, 0x5410), __byte_perm(mine, other, 0x7632));
        if (!r.is_v) {
          const int64_t at = (static_cast<int64_t>(b) * a.h_kv + r.g) * a.L_max + start + r.i;
          if (a.key_weights) a.key_weights[at] = 0.f;
          if (a.positions) a.positions[at] = (a.first_position ? a.first_position[b] : start) + r.i;
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(Kv4RowsArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kPass = kThreads / kLanes;
  const int l = threadIdx.x % kLanes;
  const unsigned r0 = blockIdx.x * (kRows * kPass) + threadIdx.x / kLanes;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    int start, count;
    if (!sequence_rows(a, b, blockIdx.x == 0 && threadIdx.x == 0, start, count)) continue;
    const unsigned rows = static_cast<unsigned>(count) * a.h_kv * 2;
    if (blockIdx.x * (kRows * kPass) >= rows) continue;
    uint32_t codes[kRows];
    uint2 par[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const RowAt r = row_at(a, r0 + j * kPass, rows);
      codes[j] = 0;
      par[j] = make_uint2(0, 0);
      if (!r.live) continue;
      const uint8_t* rec = static_cast<const uint8_t*>(a.cache.ptr) + b * a.cache.sb +
                           (static_cast<int64_t>(start) + r.i) * a.cache.sn + r.g * a.cache.sh;
      codes[j] = *reinterpret_cast<const uint32_t*>(rec + (r.is_v ? D / 2 : 0) + l * 4);
      par[j] = *reinterpret_cast<const uint2*>(rec + D + (r.is_v ? 8 : 0));
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const RowAt r = row_at(a, r0 + j * kPass, rows);
      if (!r.live) continue;
      const bool second = l >= kLanes / 2;
      const float s = second ? bf16_hi(par[j].x) : bf16_lo(par[j].x);
      const float m = second ? bf16_hi(par[j].y) : bf16_lo(par[j].y);
      uint32_t out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[e] = pack_bf16x2(fmaf(s, static_cast<float>((codes[j] >> (8 * e)) & 15u), m),
                             fmaf(s, static_cast<float>((codes[j] >> (8 * e + 4)) & 15u), m));
      const da_t4& dst = r.is_v ? a.v : a.k;
      __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst.ptr) + b * dst.sb + r.i * dst.sn +
                                      r.g * dst.sh + l * 8),
             make_uint4(out[0], out[1], out[2], out[3]));
    }
  }
}

// Blocks of rows of one sequence along x, sequences along y.
dim3 grid_for(const Kv4RowsArgs& a) {
  const unsigned rows = static_cast<unsigned>(a.N) * a.h_kv * 2, per = kRows * kThreads / (a.d / 8);
  return dim3((rows + per - 1) / per, a.B < 65535 ? a.B : 65535);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s) {
  if (a.d == 128)
    kv4_append_kernel<128><<<grid_for(a), kThreads, 0, s>>>(a);
  else
    kv4_append_kernel<64><<<grid_for(a), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s) {
  if (a.d == 128)
    kv4_read_kernel<128><<<grid_for(a), kThreads, 0, s>>>(a);
  else
    kv4_read_kernel<64><<<grid_for(a), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace da
