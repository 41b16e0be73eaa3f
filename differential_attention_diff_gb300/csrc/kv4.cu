// kv4.cu — rows of a 4-bit KV cache: quantise bf16 key and value rows into
// records, and read records back as bf16 rows.
//
// A record (layout in diffattn.h) holds a key and a value row; each row has
// two groups of d/2 features with value = s * code + m, m the group's
// minimum and s = bf16(range / 15).  Both kernels give a row to d/16 lanes of
// 16 features each: two 16-byte accesses on the bf16 side and 8 bytes of codes
// on the other, so a warp touches whole contiguous rows.  Neither is bound by
// memory alone: with 656 bytes moved per record, an SM has about 28 cycles for
// one, so the instructions per feature count too.  Measured, 16 x 4096 x 8
// rows of d 128: append 72.4 us, 4.75 TB/s, with no unit full (issue slots 67 %
// busy, the ALU pipe 57 %, 45 % of the warps at 62 registers); read 55.4 us, 6.2
// TB/s, 0.91 of a copy.
#include "common.cuh"
#include "fp32_pair.cuh"
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

// A block's rows: kBatches x kRows passes of kThreads / (D/16) rows each, out
// of the sequence's N * h_kv * 2 (row = (i * h_kv + g) * 2 + is_value; a pass
// is an even number of rows, so a thread has keys only or values only).
// Loading kRows rows before the first is used keeps enough bytes in flight;
// the batches spread the set-up.
constexpr int kRows = 2;
constexpr int kBatches = 4;  // 1 where the rows are too few to fill the GPU with that many each

// Byte offset of a thread's row in a [N, h_kv] array, and its token and head,
// walked from pass to pass with additions only: 64-bit products per row would
// be half of the kernels' instructions.
struct RowWalk {
  int64_t at;
  int i, g;
  __device__ RowWalk(unsigned r, int h_kv, int64_t sn, int64_t sh) {
    const unsigned u = r >> 1, h = static_cast<unsigned>(h_kv);
    i = static_cast<int>(u / h);
    g = static_cast<int>(u - i * h);
    at = i * sn + g * sh;
  }
  __device__ __forceinline__ void next(const Kv4RowsArgs& a, int64_t step, int64_t wrap) {
    i += a.step_i;
    g += a.step_g;
    at += step;
    if (g >= a.h_kv) {
      g -= a.h_kv;
      ++i;
      at += wrap;
    }
  }
};

// x / 15, rounded once, as a quotient corrected by its residual (Markstein's
// correction); NaN and infinity stay something that is not finite.
__device__ __forceinline__ float fifteenth(float x) {
  if (x > 0.f && x < 0x1p-90f) return __fdiv_rn(x, 15.f);  // the residual may not be a normal number
  const float q = x * (1.f / 15.f);
  return fmaf(fmaf(q, -15.f, x), 1.f / 15.f, q);
}
__device__ __forceinline__ float reciprocal(float x) {  // within an ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight codes of bf16 pairs w: rint(t / s) for t = x - lo in [0, 15.03 s],
// exactly, without a division (Markstein's correction again).  q = t inv is off by an ulp or two; its residual
// t - q s fits fp32, and q + residual inv is rounded once, from a value within
// 2^-21 ulp of t / s: the rounded quotient, but where t / s lies that close to
// the middle between two numbers.  The rounding to a code could still go wrong
// where t / s lies within half an ulp of a tie k + 1/2 without being one; but
// (k + 1/2) s has 13 bits and t 24, so that they differ by more than that (by
// 2^-24 t (1 + 2^-13) at least, half an ulp of the tie being 2^-24 of it at
// most), and a true tie comes out exactly.  The code stays in the low bits of
// 1.5 2^23 + q and is summed with those bits; what the eight constants add to
// is taken off.
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[4], float lo, float s, float inv) {
  constexpr float kMagic = 12582912.f;  // 0x4b400000
  const F2 inv2(inv, inv), s2(-s, -s), lo2(-lo, -lo), magic(kMagic, kMagic);
  uint32_t sum = 0;
#pragma unroll
  for (int e = 3; e >= 0; --e) {
    const F2 t = add2(F2(bf16_lo(w[e]), bf16_hi(w[e])), lo2);
    const F2 q = mul2(t, inv2);
    const uint2 code = add2(fma2(fma2(q, s2, t), inv2, q), magic).bits();
    sum = (sum * 16u + code.y) * 16u + code.x;
  }
  return sum - 0x4b400000u * 0x11111111u;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(Kv4RowsArgs a, int batches) {
  constexpr int kLanes = D / 16;       // of a row
  constexpr int kGroupLanes = D / 32;  // of a group
  constexpr int kPass = kThreads / kLanes;
  const int l = threadIdx.x % kLanes;
  const unsigned r0 = blockIdx.x * (batches * kRows * kPass) + threadIdx.x / kLanes;
  const bool is_v = r0 & 1;
  const int64_t sn = 2 * (is_v ? a.v.sn : a.k.sn), sh = 2 * (is_v ? a.v.sh : a.k.sh), sb = 2 * (is_v ? a.v.sb : a.k.sb);
  const int64_t step = a.step_i * sn + a.step_g * sh, wrap = sn - a.h_kv * sh;
  const int64_t step_c = a.step_i * a.cache.sn + a.step_g * a.cache.sh, wrap_c = a.cache.sn - a.h_kv * a.cache.sh;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    int start, count;
    if (!sequence_rows(a, b, blockIdx.x == 0 && threadIdx.x == 0, start, count)) continue;
    const unsigned rows = static_cast<unsigned>(count) * a.h_kv * 2;
    if (blockIdx.x * (batches * kRows * kPass) >= rows) continue;
    const uint8_t* from = static_cast<const uint8_t*>(is_v ? a.v.ptr : a.k.ptr) + b * sb + l * 32;
    uint8_t* to = static_cast<uint8_t*>(a.cache.ptr) + b * a.cache.sb + start * a.cache.sn;
    RowWalk wi(r0, a.h_kv, sn, sh), wo(r0, a.h_kv, a.cache.sn, a.cache.sh);
    unsigned r = r0;
#pragma unroll 1
    for (int batch = 0; batch < batches; ++batch) {
      if (r - threadIdx.x / kLanes >= rows) break;  // the whole block's
      uint4 in[kRows][2];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        in[j][0] = in[j][1] = make_uint4(0, 0, 0, 0);
        if (r + j * kPass < rows) {
          in[j][0] = __ldcs(reinterpret_cast<const uint4*>(from + wi.at));
          in[j][1] = __ldcs(reinterpret_cast<const uint4*>(from + wi.at) + 1);
        }
        wi.next(a, step, wrap);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const uint32_t w0[4] = {in[j][0].x, in[j][0].y, in[j][0].z, in[j][0].w};
        const uint32_t w1[4] = {in[j][1].x, in[j][1].y, in[j][1].z, in[j][1].w};
        const __nv_bfloat162 *x0 = reinterpret_cast<const __nv_bfloat162*>(w0), *x1 = reinterpret_cast<const __nv_bfloat162*>(w1);
        // both halves' minimum and maximum at once; NaN stays
        __nv_bfloat162 lo2 = __hmin2_nan(x0[0], x1[0]), hi2 = __hmax2_nan(x0[0], x1[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          lo2 = __hmin2_nan(lo2, __hmin2_nan(x0[e], x1[e]));
          hi2 = __hmax2_nan(hi2, __hmax2_nan(x0[e], x1[e]));
        }
#pragma unroll
        for (int o = 1; o < kGroupLanes; o <<= 1) {
          lo2 = __hmin2_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
          hi2 = __hmax2_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
        }
        float lo = __bfloat162float(__hmin_nan(lo2.x, lo2.y));
        const float hi = __bfloat162float(__hmax_nan(hi2.x, hi2.y));
        float s = __bfloat162float(__float2bfloat16_rn(fifteenth(__fsub_rn(hi, lo))));
        const bool bad = !(fabsf(s) < INFINITY);
        uint2 codes = make_uint2(0, 0);
        if (s >= 0x1p-100f && !bad) {
          const float inv = reciprocal(s);
          codes = make_uint2(codes_of(w0, lo, s, inv), codes_of(w1, lo, s, inv));
        } else if (s > 0.f && !bad) {  // the reciprocal or the residual may not be normal numbers
          for (int e = 0; e < 16; ++e) {
            const uint32_t w = (e & 8) ? w1[(e & 7) >> 1] : w0[e >> 1];
            const float x = (e & 1) ? bf16_hi(w) : bf16_lo(w);
            const uint32_t n = static_cast<uint32_t>(fminf(rintf(__fdiv_rn(__fsub_rn(x, lo), s)), 15.f));
            if (e & 8)
              codes.y |= n << (4 * (e & 7));
            else
              codes.x |= n << (4 * e);
          }
        }
        if (bad) s = lo = NAN;
        // both groups' parameters at the row's first lane
        const uint32_t mine = pack_bf16x2(s, lo);
        const uint32_t other = __shfl_down_sync(0xffffffffu, mine, kGroupLanes);
        if (r + j * kPass < rows) {
          uint8_t* rec = to + wo.at;
          *reinterpret_cast<uint2*>(rec + (is_v ? D / 2 : 0) + l * 8) = codes;
          if (l == 0) {
            *reinterpret_cast<uint2*>(rec + D + (is_v ? 8 : 0)) =
                make_uint2(__byte_perm(mine, other, 0x5410), __byte_perm(mine, other, 0x7632));
            if (!is_v && (a.key_weights || a.positions)) {
              const int64_t at = (static_cast<int64_t>(b) * a.h_kv + wo.g) * a.L_max + start + wo.i;
              if (a.key_weights) a.key_weights[at] = 0.f;
              if (a.positions) a.positions[at] = (a.first_position ? a.first_position[b] : start) + wo.i;
            }
          }
        }
        wo.next(a, step_c, wrap_c);
      }
      r += kRows * kPass;
    }
  }
}

// Four output words of eight codes.  A code byte times 0x1001 has its lower
// code at bit 0 and its upper one at bit 16; set into the mantissa of bf16 128
// each is 128 plus the code, and the fused multiply-add of s, code and m, all
// exact in bf16, rounds once.
__device__ __forceinline__ uint4 values_of(uint32_t codes, uint32_t s_twice, uint32_t m_twice) {
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s_twice);
  const __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&m_twice);
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t y = __byte_perm(codes, 0u, 0x4440u + e) * 0x1001u;
    const uint32_t n = (y & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hfma2(s, __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&n), __nv_bfloat162(128.f, 128.f)), m);
    out[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A read holds less per row than an append does: twice the rows at once.
constexpr int kReadRows = 2 * kRows;

template <int D>
__global__ void __launch_bounds__(kThreads, 6) kv4_read_kernel(Kv4RowsArgs a, int batches) {
  constexpr int kLanes = D / 16;
  constexpr int kPass = kThreads / kLanes;
  const int l = threadIdx.x % kLanes;
  const unsigned r0 = blockIdx.x * (batches * kReadRows * kPass) + threadIdx.x / kLanes;
  const bool is_v = r0 & 1;
  const int64_t sn = 2 * (is_v ? a.v.sn : a.k.sn), sh = 2 * (is_v ? a.v.sh : a.k.sh), sb = 2 * (is_v ? a.v.sb : a.k.sb);
  const int64_t step = a.step_i * sn + a.step_g * sh, wrap = sn - a.h_kv * sh;
  const int64_t step_c = a.step_i * a.cache.sn + a.step_g * a.cache.sh, wrap_c = a.cache.sn - a.h_kv * a.cache.sh;
  // a lane takes 8 features of each group, so that the lanes' stores lie side by side
  const int code_at = (is_v ? D / 2 : 0) + l * 4, par_at = D + (is_v ? 8 : 0);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    int start, count;
    if (!sequence_rows(a, b, blockIdx.x == 0 && threadIdx.x == 0, start, count)) continue;
    const unsigned rows = static_cast<unsigned>(count) * a.h_kv * 2;
    if (blockIdx.x * (batches * kReadRows * kPass) >= rows) continue;
    const uint8_t* from = static_cast<const uint8_t*>(a.cache.ptr) + b * a.cache.sb + start * a.cache.sn;
    uint8_t* to = static_cast<uint8_t*>(is_v ? a.v.ptr : a.k.ptr) + b * sb + l * 16;
    RowWalk wi(r0, a.h_kv, a.cache.sn, a.cache.sh), wo(r0, a.h_kv, sn, sh);
    unsigned r = r0;
#pragma unroll 1
    for (int batch = 0; batch < batches; ++batch) {
      if (r - threadIdx.x / kLanes >= rows) break;  // the whole block's
      uint2 codes[kReadRows], par[kReadRows];
#pragma unroll
      for (int j = 0; j < kReadRows; ++j) {
        codes[j] = par[j] = make_uint2(0, 0);
        if (r + j * kPass < rows) {
          codes[j].x = *reinterpret_cast<const uint32_t*>(from + wi.at + code_at);
          codes[j].y = *reinterpret_cast<const uint32_t*>(from + wi.at + code_at + D / 4);
          par[j] = *reinterpret_cast<const uint2*>(from + wi.at + par_at);
        }
        wi.next(a, step_c, wrap_c);
      }
#pragma unroll
      for (int j = 0; j < kReadRows; ++j) {
        if (r + j * kPass < rows) {
          const uint32_t s0 = __byte_perm(par[j].x, 0u, 0x1010), m0 = __byte_perm(par[j].y, 0u, 0x1010);
          const uint32_t s1 = __byte_perm(par[j].x, 0u, 0x3232), m1 = __byte_perm(par[j].y, 0u, 0x3232);
          __stcs(reinterpret_cast<uint4*>(to + wo.at), values_of(codes[j].x, s0, m0));
          __stcs(reinterpret_cast<uint4*>(to + wo.at + D), values_of(codes[j].y, s1, m1));
        }
        wo.next(a, step, wrap);
      }
      r += kReadRows * kPass;
    }
  }
}

// Blocks of rows of one sequence along x, sequences along y.
template <class F>
cudaError_t launch_rows(F kernel, Kv4RowsArgs a, int rows_at_once, cudaStream_t s) {
  const int pass = kThreads / (a.d / 16);  // rows
  a.step_i = pass / 2 / a.h_kv;
  a.step_g = pass / 2 % a.h_kv;
  const unsigned rows = static_cast<unsigned>(a.N) * a.h_kv * 2, per = rows_at_once * pass;
  const unsigned y = a.B < 65535 ? a.B : 65535;
  const int most = kBatches * kRows / rows_at_once;
  const int batches = static_cast<int64_t>(rows) * y / (static_cast<int64_t>(per) * most) >= 1024 ? most : 1;
  kernel<<<dim3((rows + per * batches - 1) / (per * batches), y), kThreads, 0, s>>>(a, batches);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s) {
  return a.d == 128 ? launch_rows(kv4_append_kernel<128>, a, kRows, s) : launch_rows(kv4_append_kernel<64>, a, kRows, s);
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s) {
  return a.d == 128 ? launch_rows(kv4_read_kernel<128>, a, kReadRows, s) : launch_rows(kv4_read_kernel<64>, a, kReadRows, s);
}

}  // namespace da
