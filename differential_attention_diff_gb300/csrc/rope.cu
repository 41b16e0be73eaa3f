// rope.cu — queries and keys normed (per-head RMSNorm) and rotated by their
// positions: forward, backward, and the append of new tokens to a paged cache
// with both applied on the way.
//
// Definitions in diffattn.h.  All three stream rows of d features once and are
// bound by memory; what they must not do is compute angles per row.  A warp
// takes a token (or a share of its heads, where there are few tokens), computes
// the token's cosines and sines once, and passes over its rows: d / 8 lanes to a
// row, each with four pairs of features, so a row's sums take log2(d / 8)
// shuffles and the rotation none.
//
// The angle: position * inv_freq in turns, as a 64-bit fixed-point fraction that
// wraps by itself (position times 2^64 inv_freq / 2 pi, modulo 2^64).  It is off
// by 2^-64 turns a position at most, so far positions keep the accuracy of near
// ones, and the quarter of the turn comes out of its top bits exactly; what goes
// to sincospi is at most an eighth of a turn either way.
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// 2^64 inv_freq / 2 pi modulo 2^64.  1 / 2 pi in two doubles (the first is it
// rounded, the second the rest): their product with a 24-bit number is good to
// 2^-77 of itself.
__device__ __forceinline__ uint64_t turns(float inv_freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double f = inv_freq;
  const double hi = f * kHi;
  const double lo = fma(f, kHi, -hi) + f * kLo;
  const double frac = hi - floor(hi);
  return __double2ull_rn(frac * 18446744073709551616.0) + static_cast<uint64_t>(__double2ll_rn(lo * 18446744073709551616.0));
}

__device__ __forceinline__ void sincos_turns(uint64_t t, float scale, float& s, float& c) {
  const uint32_t quarter = static_cast<uint32_t>((t + (1ull << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(t - (static_cast<uint64_t>(quarter) << 62));  // within 2^61 either way
  float s0, c0;
  sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &s0, &c0);  // 2^-63: half turns
  const float a = (quarter & 1) ? c0 : s0, b = (quarter & 1) ? s0 : c0;
  s = (quarter & 2) ? -a * scale : a * scale;
  c = ((quarter + 1) & 2) ? -b * scale : b * scale;
}

// Four neighbouring features, as they are stored.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float* x) { v = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); }
};
template <>
struct Four<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ __forceinline__ void get(float* x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  __device__ __forceinline__ void set(const float* x) { v = make_float4(x[0], x[1], x[2], x[3]); }
};

// The features of lane l of a row: four at `a` and four at `b`.  Half layout:
// features 4l .. and their partners rot / 2 further on; interleaved, or behind
// rot: eight in a row.  x[i] and x[4 + i], or x[2i] and x[2i + 1], are pair i.
template <bool kInter>
struct Lane {
  bool rotated;
  int a, b;
  __device__ __forceinline__ Lane(int l, int rot) {
    rotated = 8 * l < rot;
    const bool split = !kInter && rotated;
    a = split ? 4 * l : 8 * l;
    b = split ? 4 * l + rot / 2 : 8 * l + 4;
  }
  __device__ static __forceinline__ constexpr int u(int i) { return kInter ? 2 * i : i; }
  __device__ static __forceinline__ constexpr int v(int i) { return kInter ? 2 * i + 1 : 4 + i; }
};

template <bool kInter>
__device__ __forceinline__ void rotate(float* x, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p = x[Lane<kInter>::u(i)], q = x[Lane<kInter>::v(i)];
    x[Lane<kInter>::u(i)] = p * c[i] - q * s[i];
    x[Lane<kInter>::v(i)] = q * c[i] + p * s[i];
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void load_weight(const float* w, int a, int b, float* out) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.f;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = __ldg(w + a + i), out[4 + i] = __ldg(w + b + i);
}

template <typename T>
__device__ __forceinline__ T* at(const da_t4& t, int64_t b, int64_t n) {
  return static_cast<T*>(t.ptr) + b * t.sb + n * t.sn;
}

// Where a packed token belongs: its sequence (the last that starts at or before
// it) by a 32-way search, a lane a probe.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t, int lane) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool before = i < n && cu[lo + i] <= t;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, before) | 1u);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// Whether a sequence's rows and length are within bounds (diffattn.h).
__device__ __forceinline__ bool sequence_ok(const da_paged_cache& c, int t0, int t1, int L) {
  return t0 >= 0 && t0 <= t1 && t1 <= c.T && L >= t1 - t0 && L <= static_cast<int64_t>(c.max_pages) * c.page_size;
}

template <typename T, int D, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kThreads)
rope_rows_kernel(RopeArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes to a row, rows to a warp's pass
  constexpr int kUnroll = 4;
  __shared__ uint64_t freq[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) freq[i] = turns(a.inv_freq[i]);
  if constexpr (kPaged) {
    const da_paged_cache& c = a.cache;
    for (int b = threadIdx.x; blockIdx.x == 0 && b < c.B; b += kThreads)
      if (!sequence_ok(c, c.cu_seqlens[b], c.cu_seqlens[b + 1], c.seqlens[b])) record_status(a.status, DA_ERR_BOUNDS, 0x0E01);
  }
  __syncthreads();
  const int l = lane % kLanes, sub = lane / kLanes;
  const Lane<kInter> f(l, a.rot);
  const int passes[3] = {(a.h_q + kRows - 1) / kRows, (a.h_k + kRows - 1) / kRows, (a.h_v + kRows - 1) / kRows};
  const int heads[3] = {a.h_q, a.h_k, a.h_v};
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp; unit < a.units;
       unit += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(unit / a.chunks), chunk = static_cast<int>(unit % a.chunks);
    int64_t sb = 0, sn = t, db = 0, dn = t;  // the rows' place in the sources and in q_out
    int64_t page = 0, slot = 0;
    bool paged_ok = true;
    int pos;
    if constexpr (kPaged) {
      const da_paged_cache& c = a.cache;
      const int b = sequence_of(c.cu_seqlens, c.B, t, lane);
      const int t0 = c.cu_seqlens[b], t1 = c.cu_seqlens[b + 1], L = c.seqlens[b];
      // padding, or a sequence that is out of bounds
      if (t < t0 || t >= t1 || !sequence_ok(c, t0, t1, L)) continue;
      const int j = L - t1 + t;
      const int id = c.block_table[static_cast<int64_t>(b) * c.max_pages + j / c.page_size];
      paged_ok = id >= 0 && id < c.n_pages;
      if (!paged_ok && lane == 0) record_status(a.status, DA_ERR_BOUNDS, 0x0E02);
      page = id;
      slot = j % c.page_size;
      pos = a.positions ? a.positions[t] : j;
    } else {
      sb = db = t / a.N;
      sn = dn = t % a.N;
      pos = a.positions ? a.positions[t] : static_cast<int>(sn);
    }
    float co[4], si[4];
    if (f.rotated) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sincos_turns(static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq[4 * l + i], a.rope_scale, si[i], co[i]);
    }
    const int p0 = chunk * a.chunk_passes, p1 = p0 + a.chunk_passes;
    int base = 0;
#pragma unroll
    for (int kind = 0; kind < (kPaged ? 3 : 2); ++kind) {
      const int lo = max(p0, base), hi = min(p1, base + passes[kind]);
      if (lo < hi && (kind == 0 || paged_ok)) {
        const da_t4& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const da_t4& dst = kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out;
        const T* from = at<T>(src, sb, sn);
        T* to = kPaged && kind > 0 ? at<T>(dst, page, slot) : at<T>(dst, db, dn);
        float w[8];
        if (a.norm && kind < 2) load_weight(kind == 0 ? a.q_weight : a.k_weight, f.a, f.b, w);
        for (int p = lo; p < hi; p += kUnroll) {
          Four<T> xa[kUnroll], xb[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int h = (p + u - base) * kRows + sub;
            if (p + u < hi && h < heads[kind]) {
              xa[u].load(from + h * src.sh + f.a);
              xb[u].load(from + h * src.sh + f.b);
            } else {
              xa[u].v = {};
              xb[u].v = {};
            }
          }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            if (p + u >= hi) break;
            const int h = (p + u - base) * kRows + sub;
            if (kind < 2) {
              float x[8];
              xa[u].get(x);
              xb[u].get(x + 4);
              if (a.norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + a.norm_eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
              }
              if (f.rotated) rotate<kInter>(x, co, si);
              xa[u].set(x);
              xb[u].set(x + 4);
            }
            if (h < heads[kind]) {
              xa[u].store(to + h * dst.sh + f.a);
              xb[u].store(to + h * dst.sh + f.b);
            }
          }
        }
      }
      base += passes[kind];
    }
  }
}

// The gradients.  The weights' are summed by each lane over its rows in fp32
// (some hundred to a few thousand of them), over a block's lanes and warps in a
// fixed order, and over the blocks by the kernel below in fp64.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads)
rope_bwd_kernel(RopeBwdArgs g) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  constexpr int kUnroll = 2;
  const RopeArgs& a = g.a;
  __shared__ uint64_t freq[D / 2];
  __shared__ float sums[kWarps][2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) freq[i] = turns(a.inv_freq[i]);
  __syncthreads();
  const int l = lane % kLanes, sub = lane / kLanes;
  const Lane<kInter> f(l, a.rot);
  const int passes[2] = {(a.h_q + kRows - 1) / kRows, (a.h_k + kRows - 1) / kRows};
  const int heads[2] = {a.h_q, a.h_k};
  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp; unit < a.units;
       unit += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(unit / a.chunks), chunk = static_cast<int>(unit % a.chunks);
    const int b = t / a.N, n = t % a.N;
    const int pos = a.positions ? a.positions[t] : n;
    float co[4], si[4];
    if (f.rotated) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sincos_turns(static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq[4 * l + i], a.rope_scale, si[i], co[i]);
        si[i] = -si[i];
      }
    }
    const int p0 = chunk * a.chunk_passes, p1 = p0 + a.chunk_passes;
    int base = 0;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int lo = max(p0, base), hi = min(p1, base + passes[kind]);
      if (lo < hi) {
        const da_t4& x_ = kind == 0 ? a.q : a.k;
        const da_t4& dy_ = kind == 0 ? g.dq_out : g.dk_out;
        const da_t4& dx_ = kind == 0 ? g.dq : g.dk;
        const T* xp = a.norm ? at<T>(x_, b, n) : nullptr;
        const T* dyp = at<T>(dy_, b, n);
        T* dxp = at<T>(dx_, b, n);
        float w[8];
        if (a.norm) load_weight(kind == 0 ? a.q_weight : a.k_weight, f.a, f.b, w);
        for (int p = lo; p < hi; p += kUnroll) {
          Four<T> xa[kUnroll], xb[kUnroll], ya[kUnroll], yb[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int h = (p + u - base) * kRows + sub;
            xa[u].v = xb[u].v = ya[u].v = yb[u].v = {};
            if (p + u < hi && h < heads[kind]) {
              ya[u].load(dyp + h * dy_.sh + f.a);
              yb[u].load(dyp + h * dy_.sh + f.b);
              if (a.norm) {
                xa[u].load(xp + h * x_.sh + f.a);
                xb[u].load(xp + h * x_.sh + f.b);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            if (p + u >= hi) break;
            const int h = (p + u - base) * kRows + sub;
            float dz[8];
            ya[u].get(dz);
            yb[u].get(dz + 4);
            if (f.rotated) rotate<kInter>(dz, co, si);
            if (a.norm) {
              float x[8];
              xa[u].get(x);
              xb[u].get(x + 4);
              float ss = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
              const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + a.norm_eps);
              float m = 0.f;
              const bool row = h < heads[kind];  // a row that is not there is zeros; with norm_eps 0 its r is infinite
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                x[i] *= r;
                if (row) acc[kind][i] = fmaf(dz[i], x[i], acc[kind][i]);
                dz[i] *= w[i];
                m = fmaf(dz[i], x[i], m);
              }
              m = row_sum<kLanes>(m) * (1.f / D);
#pragma unroll
              for (int i = 0; i < 8; ++i) dz[i] = r * (dz[i] - x[i] * m);
            }
            if (h < heads[kind]) {
              xa[u].set(dz);
              xb[u].set(dz + 4);
              xa[u].store(dxp + h * dx_.sh + f.a);
              xb[u].store(dxp + h * dx_.sh + f.b);
            }
          }
        }
      }
      base += passes[kind];
    }
  }
  if (g.part == nullptr) return;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = acc[kind][i];
#pragma unroll
      for (int o = kLanes; o < 32; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (sub == 0) sums[warp][kind][(i < 4 ? f.a : f.b) + (i & 3)] = x;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += sums[w][i / D][i % D];
    g.part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = x;
  }
}

// dq_weight and dk_weight [d] from the blocks' sums [blocks, 2, d]: a block per 32
// features, its eight warps a share of the blocks each.
__global__ void __launch_bounds__(256) rope_dw_kernel(const float* part, int blocks, int d, float* dq_weight, float* dk_weight) {
  __shared__ double sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 32 + lane;
  double x = 0.0;
  cudaGridDependencySynchronize();
#pragma unroll 4
  for (int b = warp; b < blocks; b += 8) x += static_cast<double>(part[static_cast<int64_t>(b) * 2 * d + i]);
  sums[warp][lane] = x;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < 8; ++w) x += sums[w][lane];
    float* out = i < d ? dq_weight : dk_weight;
    if (out) out[i < d ? i : i - d] = static_cast<float>(x);
  }
}

// The warps' shares: a token each where there are enough of them to fill the
// SMs' warps, else some passes of a token's heads (at least one).
void share(RopeArgs& a, int d, int warps) {
  const int rows = 256 / d;
  const int64_t passes = (a.h_q + rows - 1) / rows + (a.h_k + rows - 1) / rows + (a.h_v + rows - 1) / rows;
  int64_t each = a.tokens * passes / warps;
  each = each < 1 ? 1 : each > passes ? passes : each;
  a.chunk_passes = static_cast<int>(each);
  a.chunks = static_cast<int>((passes + each - 1) / each);
  a.units = a.tokens * a.chunks;
}

template <bool kPaged, typename T, int D>
cudaError_t launch_rows(RopeArgs a, int sms, cudaStream_t s) {
  share(a, D, sms * 32);
  const int64_t blocks = (a.units + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * 4;
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  if (a.interleaved)
    rope_rows_kernel<T, D, true, kPaged><<<grid, kThreads, 0, s>>>(a);
  else
    rope_rows_kernel<T, D, false, kPaged><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd(RopeBwdArgs g, int sms, cudaStream_t s) {
  share(g.a, D, sms * 32);
  const unsigned grid = static_cast<unsigned>(rope_bwd_blocks(g.a.units, sms));
  if (g.a.interleaved)
    rope_bwd_kernel<T, D, true><<<grid, kThreads, 0, s>>>(g);
  else
    rope_bwd_kernel<T, D, false><<<grid, kThreads, 0, s>>>(g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || g.part == nullptr) return e;
  return launch_ahead(rope_dw_kernel, dim3(2 * D / 32), dim3(256), 0, s, true, static_cast<const float*>(g.part),
                      static_cast<int>(grid), D, g.dq_weight, g.dk_weight);
}

}  // namespace

int64_t rope_bwd_blocks(int64_t units, int sms) {
  const int64_t blocks = (units + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * kRopeBwdBlocksPerSm;
  return blocks < most ? blocks : most;
}

cudaError_t launch_rope_fwd(const RopeArgs& a, int d, bool f32, int sms, cudaStream_t s) {
  switch (d) {
    case 16: return f32 ? launch_rows<false, float, 16>(a, sms, s) : launch_rows<false, __nv_bfloat16, 16>(a, sms, s);
    case 32: return f32 ? launch_rows<false, float, 32>(a, sms, s) : launch_rows<false, __nv_bfloat16, 32>(a, sms, s);
    case 64: return f32 ? launch_rows<false, float, 64>(a, sms, s) : launch_rows<false, __nv_bfloat16, 64>(a, sms, s);
    case 128: return f32 ? launch_rows<false, float, 128>(a, sms, s) : launch_rows<false, __nv_bfloat16, 128>(a, sms, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope_bwd(const RopeBwdArgs& g, int d, bool f32, int sms, cudaStream_t s) {
  switch (d) {
    case 16: return f32 ? launch_bwd<float, 16>(g, sms, s) : launch_bwd<__nv_bfloat16, 16>(g, sms, s);
    case 32: return f32 ? launch_bwd<float, 32>(g, sms, s) : launch_bwd<__nv_bfloat16, 32>(g, sms, s);
    case 64: return f32 ? launch_bwd<float, 64>(g, sms, s) : launch_bwd<__nv_bfloat16, 64>(g, sms, s);
    case 128: return f32 ? launch_bwd<float, 128>(g, sms, s) : launch_bwd<__nv_bfloat16, 128>(g, sms, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_append(const RopeArgs& a, int d, int sms, cudaStream_t s) {
  if (d == 128) return launch_rows<true, __nv_bfloat16, 128>(a, sms, s);
  if (d == 64) return launch_rows<true, __nv_bfloat16, 64>(a, sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace da
