// rope.cu — queries and keys normed (per-head RMSNorm) and rotated by their
// positions: forward, backward, and the append of new tokens to a paged cache
// with both applied on the way.
//
// Definitions in diffattn.h.  All three stream rows of d features once and are
// bound by memory, as long as little else is done per row and enough of them are
// on their way.  A warp takes a token's rows of one kind (queries, keys, or values
// to copy), or a share of them where there are few tokens, computes the token's
// cosines and sines once, a frequency to a lane, and passes over its rows; all of
// its queries come first, then its keys, so weights, and the sums of the weights'
// gradients, stay in registers.  d / F lanes have a row, F = 16 features each (8 where
// they are fp32, or where rot_dim is no multiple of 16): two pieces of 16 bytes
// that hold whole pairs, so a row's sums take log2(d / F) shuffles and the
// rotation none, and two features go through an instruction.  The pieces come by
// asynchronous copies, each lane its own, kStages groups of rows ahead and across
// the warp's tokens: 128 KB per SM in flight (192 in the backward).  With rows in
// registers instead, the backward of 2 x 8192 tokens of 64 + 8 heads, d 128, norm,
// took 165 us on a GB300 (150 now, 6.1 TB/s; the forward 106, 5.7 TB/s).
//
// The angle: position * inv_freq in turns, as a 64-bit fixed-point fraction that
// wraps by itself (position times 2^64 inv_freq / 2 pi, modulo 2^64).  It is off
// by 2^-63 turns a position at most, so far positions keep the accuracy of near
// ones, and the quarter of the turn comes out of its top bits exactly.
#include "common.cuh"
#include "fp32_pair.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace da {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

constexpr int kUnroll = 2;      // passes (of 32 / lanes rows) that are a group
constexpr int kStagesFwd = 4, kStagesBwd = 3;
// The passes of a share of work, 1 KB of rows each, where there is plenty.  Fewer
// compute more angles, more spread what the GPU reads at a time; beyond that times
// go up and down with the shape, and no number is best for all.  Forward, us, for 3,
// 4, 5, 6, 8 (norm unless said otherwise, bf16, all of the head rotated):
//   2 x 8192 tokens, 64 + 8 heads, d 128     123, 105, 117, 100, 111
//   the same without norm                    113,  98, 106, 110, 111
//   the same, half of the head rotated       121, 106, 115,  97, 108
//   the same in fp32, 2 x 4096               109,  94, 106, 112, 109
//   4 x 4096, 32 + 8                          70,  64,  66,  69,  63
//   1 x 16384, 40 + 10, interleaved           97,  80,  76,  76,  83
//   4 x 8192, 24 + 2                         102, 106, 115,  88,  88
//   8 x 2048, 16 + 16, d 64                   33,  33,  33,  33,  33
//   six prompts appended, 64 + 8 and values  142, 119, 133, 111, 124
//   the same without norm                    131, 111, 121, 125, 128
// 4 and 6 have the lowest sums, 1 % apart, and each is up to 20 % behind the other
// somewhere.  The backward of the first takes 156, 150, 153, 168 with 4, 6, 8, 16
// (103, 99, 112, 112 without norm).
constexpr int kSharePasses = 4, kSharePassesBwd = 6;

// 2^64 inv_freq / 2 pi modulo 2^64, to an even number, for frequencies below 2^32;
// 1 for any other, an infinity or a NaN.  1 / 2 pi in two doubles (the first is it
// rounded, the second the rest): their product with a 24-bit number is good to
// 2^-105 of itself, and below 2^32 to 2^-75.
__device__ __forceinline__ uint64_t turns(float inv_freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double f = inv_freq;
  const double hi = f * kHi;
  const double lo = fma(f, kHi, -hi) + f * kLo;
  const double frac = hi - floor(hi);
  constexpr double k64 = 18446744073709551616.0;  // 2^64
  const uint64_t t = __double2ull_rn(frac * k64) + static_cast<uint64_t>(__double2ll_rn(lo * k64));
  return fabsf(inv_freq) < 4294967296.0f ? t & ~1ull : 1;
}

// Sine and cosine of t / 2^64 turns, times scale.  What is left of the nearest
// quarter, at most an eighth of a turn, is taken to 2^-34 of a turn; Taylor's
// series up to x^9 and x^10 are off by 2^-29 and 2^-33 there.
__device__ __forceinline__ void sincos_turns(uint64_t t, float scale, float& s, float& c) {
  const uint32_t quarter = static_cast<uint32_t>((t + (1ull << 61)) >> 62);
  const int rest = static_cast<int>(static_cast<int64_t>(t - (static_cast<uint64_t>(quarter) << 62)) >> 30);  // 2^-34 turns
  const float x = static_cast<float>(rest) * 3.6572951982e-10f;                                               // 2 pi 2^-34
  const float x2 = x * x;
  float p = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  p = fmaf(x2, p, 1.f / 120.f);
  p = fmaf(x2, p, -1.f / 6.f);
  const float s0 = fmaf(x * x2, p, x);
  p = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
  p = fmaf(x2, p, -1.f / 720.f);
  p = fmaf(x2, p, 1.f / 24.f);
  p = fmaf(x2, p, -0.5f);
  const float c0 = fmaf(x2, p, 1.f);
  const float a = (quarter & 1) ? c0 : s0, b = (quarter & 1) ? s0 : c0;
  s = (quarter & 2) ? -a * scale : a * scale;
  c = ((quarter + 1) & 2) ? -b * scale : b * scale;
}

// The features of a lane of a row, F of them: F / 2 at `a` and F / 2 at `b`, half
// of the rotated features (or of those behind them) further on, so that a row's
// lanes read on end; as stored, and as F / 4 pairs (fp32) of first and of second
// features of rotation pairs.  Half layout: a holds first features, b their
// partners; interleaved: each holds whole pairs.
template <typename T, int D, int F, bool kInter>
struct Lane {
  static constexpr int kHalf = F / 2;                              // features of a piece
  static constexpr int kWords = kHalf * static_cast<int>(sizeof(T)) / 4;  // 2 or 4
  static constexpr int kPiece = 4 * kWords;                        // bytes of one
  static constexpr int kSlot = 64 * kPiece;                        // of a warp's pass: two pieces a lane
  bool rotated;
  int a, b;
  // this lane's pieces of row p, to its place in a slot
  __device__ __forceinline__ void fetch(uint32_t slot, const T* p) const {
    if constexpr (kPiece == 16) {
      cp_async_16(slot, p + a, 16);
      cp_async_16(slot + 32 * kPiece, p + b, 16);
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(slot), "l"(p + a));
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(slot + 32 * kPiece), "l"(p + b));
    }
  }
  __device__ __forceinline__ Lane(int l, int rot) {
    rotated = F * l < rot;
    a = rotated ? kHalf * l : rot + kHalf * (l - rot / F);
    b = a + (rotated ? rot : D - rot) / 2;
  }
  struct Raw {
    uint32_t w[2][kWords];
    // from a slot of two pieces per lane (`fetch`)
    __device__ __forceinline__ void load(const uint8_t* slot) {
      if constexpr (kWords == 4) {
        *reinterpret_cast<uint4*>(w[0]) = *reinterpret_cast<const uint4*>(slot);
        *reinterpret_cast<uint4*>(w[1]) = *reinterpret_cast<const uint4*>(slot + 32 * kPiece);
      } else {
        *reinterpret_cast<uint2*>(w[0]) = *reinterpret_cast<const uint2*>(slot);
        *reinterpret_cast<uint2*>(w[1]) = *reinterpret_cast<const uint2*>(slot + 32 * kPiece);
      }
    }
    __device__ __forceinline__ void store(T* p, const Lane& f) const {
      if constexpr (kWords == 4) {
        *reinterpret_cast<uint4*>(p + f.a) = *reinterpret_cast<const uint4*>(w[0]);
        *reinterpret_cast<uint4*>(p + f.b) = *reinterpret_cast<const uint4*>(w[1]);
      } else {
        *reinterpret_cast<uint2*>(p + f.a) = *reinterpret_cast<const uint2*>(w[0]);
        *reinterpret_cast<uint2*>(p + f.b) = *reinterpret_cast<const uint2*>(w[1]);
      }
    }
    // feature i of the lane's F, from a's first to b's last
    __device__ __forceinline__ float at(int i) const {
      if constexpr (sizeof(T) == 4) {
        return __uint_as_float(w[i / kHalf][i % kHalf]);
      } else {
        const uint32_t x = w[i / kHalf][i % kHalf / 2];
        return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
      }
    }
    __device__ __forceinline__ void put(int i, float lo, float hi) {  // features i and i + 1 (i even)
      if constexpr (sizeof(T) == 4) {
        w[i / kHalf][i % kHalf] = __float_as_uint(lo);
        w[i / kHalf][i % kHalf + 1] = __float_as_uint(hi);
      } else {
        w[i / kHalf][i % kHalf / 2] = pack_bf16x2(lo, hi);
      }
    }
  };
  // the lane's index of the first / second feature of its rotation pair i
  __device__ static __forceinline__ constexpr int u(int i) { return kInter ? 2 * i : i; }
  __device__ static __forceinline__ constexpr int v(int i) { return kInter ? 2 * i + 1 : kHalf + i; }
  __device__ static __forceinline__ void get(const Raw& r, F2Pair (&x)[F / 2]) {
#pragma unroll
    for (int i = 0; i < F / 4; ++i) {
      x[i] = {r.at(u(2 * i)), r.at(u(2 * i + 1))};
      x[F / 4 + i] = {r.at(v(2 * i)), r.at(v(2 * i + 1))};
    }
  }
  __device__ static __forceinline__ void put(Raw& r, const F2Pair (&x)[F / 2]) {
#pragma unroll
    for (int i = 0; i < F / 4; ++i) {
      if constexpr (kInter) {
        r.put(4 * i, x[i].lo(), x[F / 4 + i].lo());
        r.put(4 * i + 2, x[i].hi(), x[F / 4 + i].hi());
      } else {
        r.put(2 * i, x[i].lo(), x[i].hi());
        r.put(kHalf + 2 * i, x[F / 4 + i].lo(), x[F / 4 + i].hi());
      }
    }
  }
  // where pair-array entry e, half h is among the row's features
  __device__ __forceinline__ int feature(int e, int h) const {
    const int i = e < F / 4 ? u(2 * e + h) : v(2 * (e - F / 4) + h);
    return i < kHalf ? a + i : b + i - kHalf;
  }
};

// The rotation of a lane's pairs, with what its features are multiplied by before
// (w) and which way: u' = u uc + v us, v' = v vc + u vs.
template <int P>
struct Turn {
  F2Pair uc[P], us[P], vc[P], vs[P];
  // no rotation
  __device__ __forceinline__ void set(const F2Pair (&w)[2 * P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      uc[i] = w[i];
      vc[i] = w[P + i];
      us[i] = vs[i] = {0.f, 0.f};
    }
  }
  __device__ __forceinline__ void set(const F2Pair (&w)[2 * P], const F2Pair (&c)[P], const F2Pair (&s)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      uc[i] = w[i] * c[i];
      us[i] = -(w[P + i] * s[i]);
      vc[i] = w[P + i] * c[i];
      vs[i] = w[i] * s[i];
    }
  }
  __device__ __forceinline__ void apply(F2Pair (&x)[2 * P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const F2Pair u = x[i], v = x[P + i];
      x[i] = fma2(v, us[i], u * uc[i]);
      x[P + i] = fma2(u, vs[i], v * vc[i]);
    }
  }
  // what `apply` is without rotation, where it may not multiply by 0
  __device__ __forceinline__ void scale(F2Pair (&x)[2 * P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = x[i] * uc[i];
      x[P + i] = x[P + i] * vc[i];
    }
  }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int P>
__device__ __forceinline__ float square_sum(const F2Pair (&x)[P]) {
  F2Pair s = x[0] * x[0];
#pragma unroll
  for (int i = 1; i < P; ++i) s = fma2(x[i], x[i], s);
  return s.lo() + s.hi();
}

// A token's cosines and sines, a frequency to a lane, left in shared memory for
// the lanes that have its pairs; NaN for a frequency that is none.
__device__ __forceinline__ void token_angles(const RopeArgs& a, const uint64_t* freq, int pos, float* cs, int stride, int lane) {
  __syncwarp();
  for (int i = lane; i < a.rot / 2; i += 32) {
    float s, c;
    const uint64_t f = freq[i], t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * f;
    sincos_turns(t, f & 1 ? __int_as_float(0x7fffffff) : a.rope_scale, s, c);
    cs[i] = c;
    cs[stride + i] = s;
  }
  __syncwarp();
}

// The lane's: of its pairs 0 .. 2P - 1, half layout on end from 2P l; interleaved
// the first P from P l, the others rot / 4 further on.
template <int P, bool kInter>
__device__ __forceinline__ void load_angles(const float* cs, int stride, int l, int rot, F2Pair (&c)[P], F2Pair (&s)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = kInter ? P * l + 2 * i + (2 * i >= P ? rot / 4 - P : 0) : 2 * P * l + 2 * i;
    const float2 x = *reinterpret_cast<const float2*>(cs + at);
    const float2 y = *reinterpret_cast<const float2*>(cs + stride + at);
    c[i] = {x.x, x.y};
    s[i] = {y.x, y.y};
  }
}

template <int F, class L>
__device__ __forceinline__ void load_weight(const float* w, const L& f, F2Pair (&out)[F / 2]) {
#pragma unroll
  for (int e = 0; e < F / 2; ++e)
    out[e] = w == nullptr ? F2Pair{1.f, 1.f} : F2Pair{__ldg(w + f.feature(e, 0)), __ldg(w + f.feature(e, 1))};
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

// A warp's way through its shares of tokens (units), those of the queries, then
// the keys', then the values', a group of kUnroll passes at a time.  One runs
// ahead to fetch, one follows.
struct Way {
  const RopeArgs* args;
  uint32_t unit;
  int which;       // kind of rows
  int t, p, p1;    // token, first pass of the group, end of the share
  bool fresh;      // the group is a share's first
  __device__ __forceinline__ Way(const RopeArgs& a_, int warp) : args(&a_), unit(blockIdx.x * kWarps + warp) { share(); }
  __device__ __forceinline__ bool more() const { return unit < args->units; }
  __device__ __forceinline__ const RopeKind& kind() const { return args->kind[which]; }
  __device__ __forceinline__ void share() {
    which = unit < args->kind[1].unit0 ? 0 : unit < args->kind[2].unit0 ? 1 : 2;
    const RopeKind& k = kind();
    const uint32_t u = unit - k.unit0;
    t = static_cast<int>(k.chunks <= 1 ? u : u / k.chunks);
    p = k.chunks <= 1 ? 0 : static_cast<int>(u - t * k.chunks) * k.chunk_passes;
    p1 = min(k.passes, p + k.chunk_passes);
    fresh = true;
  }
  __device__ __forceinline__ void step() {  // to the next share
    unit += gridDim.x * kWarps;
    if (more()) share();
  }
  __device__ __forceinline__ void next() {
    p += kUnroll;
    fresh = false;
    if (p >= p1) step();
  }
  // whether pass u of the group has a row of this lane, and its head
  template <int kRows>
  __device__ __forceinline__ bool row(int u, int sub, int* h) const {
    *h = (p + u) * kRows + sub;
    return p + u < p1 && *h < kind().heads;
  }
};

// A token's place: its rotation's position and where its rows go, as far as they
// are loaded and not looked at (a share ahead of their use).
struct Place {
  int pos;      // the rotation's
  int page, j;  // paged: the entry of the block table (keys and values), the position in the sequence
  bool ok;      // the rows are written
};
template <bool kPaged>
__device__ __forceinline__ Place place_of(const RopeArgs& a, int which, int t, int lane) {
  Place r{0, 0, 0, true};
  if constexpr (kPaged) {
    const da_paged_cache& c = a.cache;
    const int b = sequence_of(c.cu_seqlens, c.B, t, lane);
    const int t0 = c.cu_seqlens[b], t1 = c.cu_seqlens[b + 1], len = c.seqlens[b];
    // else padding, or a sequence that is out of bounds
    r.ok = t >= t0 && t < t1 && paged_sequence_ok(c, t0, t1, len);
    if (r.ok) {
      r.j = len - t1 + t;
      r.pos = a.positions ? a.positions[t] : r.j;
      if (which > 0) r.page = c.block_table[static_cast<int64_t>(b) * c.max_pages + r.j / c.page_size];
    }
  } else {
    r.pos = a.positions ? a.positions[t] : t % a.N;
  }
  return r;
}

// kRest: rows with a norm of which not all features are rotated (an instance of
// its own, since its check would cost the others 2 %).
template <typename T, int D, int F, bool kInter, bool kPaged, bool kRest>
__global__ void __launch_bounds__(kThreads, kRopeBlocksPerSm)
rope_rows_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / F, kRows = 32 / kLanes;  // lanes to a row, rows to a warp's pass
  using L = Lane<T, D, F, kInter>;
  extern __shared__ __align__(16) uint8_t ring[];     // [warp][stage][pass][two pieces of every lane]
  __shared__ uint64_t freq[D / 2];
  __shared__ __align__(16) float angles[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes;
  const L f(l, a.rot);
  uint8_t* mine = ring + warp * kStagesFwd * kUnroll * L::kSlot + lane * L::kPiece;
  const uint32_t mine_s = smem_u32(mine);
  Way ahead(a, warp);
  const T* from = nullptr;
  auto fetch = [&](int st) {
    if (ahead.more()) {
      const da_t4& src = ahead.kind().src;
      if (ahead.fresh) from = kPaged ? at<T>(src, 0, ahead.t) : at<T>(src, ahead.t / a.N, ahead.t % a.N);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        int h;
        if (ahead.row<kRows>(u, sub, &h)) f.fetch(mine_s + (st * kUnroll + u) * L::kSlot, from + h * src.sh);
      }
      ahead.next();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int st = 0; st < kStagesFwd - 1; ++st) fetch(st);
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) freq[i] = turns(a.inv_freq[i]);
  if constexpr (kPaged) {
    const da_paged_cache& c = a.cache;
    for (int b = threadIdx.x; blockIdx.x == 0 && b < c.B; b += kThreads)
      if (!paged_sequence_ok(c, c.cu_seqlens[b], c.cu_seqlens[b + 1], c.seqlens[b])) record_status(a.status, DA_ERR_BOUNDS, 0x0E01);
  }
  __syncthreads();
  F2Pair w[F / 2];
  Turn<F / 4> turn;
  int st = 0, kind = -1;
  Way way(a, warp);
  Place next{};
  if (way.more()) next = place_of<kPaged>(a, way.which, way.t, lane);
  while (way.more()) {
    // a share: where its rows go, and what turns them
    Place place = next;
    Way after = way;
    after.step();
    if (after.more()) next = place_of<kPaged>(a, after.which, after.t, lane);  // looked up a share ahead
    const RopeKind& kd = way.kind();
    if (way.which != kind) {
      kind = way.which;
      load_weight<F>(a.norm ? kd.weight : nullptr, f, w);
    }
    const bool turned = kind < 2 && (a.norm || a.rot), norm = kind < 2 && a.norm;
    T* to;
    if constexpr (kPaged) {
      if (place.ok && kind > 0 && (place.page < 0 || place.page >= a.cache.n_pages)) {
        if (lane == 0) record_status(a.status, DA_ERR_BOUNDS, 0x0E02);
        place.ok = false;
      }
      to = kind > 0 ? at<T>(kd.dst, place.page, place.j % a.cache.page_size) : at<T>(kd.dst, 0, way.t);
    } else {
      to = at<T>(kd.dst, way.t / a.N, way.t % a.N);
    }
    if (turned) {
      if (a.rot) token_angles(a, freq, place.pos, angles[warp], D / 2, lane);
      if (f.rotated) {
        F2Pair co[F / 4], si[F / 4];
        load_angles<F / 4, kInter>(angles[warp], D / 2, l, a.rot, co, si);
        turn.set(w, co, si);
      } else {
        turn.set(w);
      }
    }
    for (int p = way.p; p < way.p1; p += kUnroll, st = st + 1 == kStagesFwd ? 0 : st + 1) {
      fetch(st == 0 ? kStagesFwd - 1 : st - 1);
      cp_async_wait<kStagesFwd - 1>();
      [[maybe_unused]] float squares = 0.f;  // of the group's rows
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p + u >= way.p1) break;
        const int h = (p + u) * kRows + sub;
        typename L::Raw x;
        x.load(mine + (st * kUnroll + u) * L::kSlot);
        if (turned) {
          F2Pair y[F / 2];
          L::get(x, y);
          if (norm) {
            const float sum = row_sum<kLanes>(square_sum(y));
            const float r = rsqrtf(sum * (1.f / D) + a.norm_eps);
            if (kRest && h < kd.heads) squares += sum;
            turn.apply(y);
#pragma unroll
            for (int e = 0; e < F / 2; ++e) y[e] = y[e] * F2Pair{r, r};
          } else if (f.rotated) {
            turn.apply(y);
          }
          L::put(x, y);
        }
        if (h < kd.heads && place.ok) x.store(to + h * kd.dst.sh, f);
      }
      if constexpr (kRest) {
        // 0 times an infinity is NaN, which its partner is not where they are not
        // rotated: such rows' rest again
        if (__any_sync(0xffffffffu, norm && !(squares < INFINITY))) {
#pragma unroll 1
          for (int u = 0; u < kUnroll && p + u < way.p1; ++u) {
            const int h = (p + u) * kRows + sub;
            typename L::Raw x;
            x.load(mine + (st * kUnroll + u) * L::kSlot);
            F2Pair y[F / 2];
            L::get(x, y);
            const float r = rsqrtf(row_sum<kLanes>(square_sum(y)) * (1.f / D) + a.norm_eps);
            turn.scale(y);
#pragma unroll
            for (int e = 0; e < F / 2; ++e) y[e] = y[e] * F2Pair{r, r};
            L::put(x, y);
            if (!f.rotated && h < kd.heads && place.ok) x.store(to + h * kd.dst.sh, f);
          }
        }
      }
    }
    way = after;
  }
  cp_async_wait<0>();
}

// The gradients.  The weights' are summed by each lane over its rows in fp32
// (some hundred to a few thousand of them), over a block's lanes and warps in a
// fixed order, and over the blocks by the kernel below in fp64.
template <typename T, int D, int F, bool kInter>
__global__ void __launch_bounds__(kThreads, kRopeBlocksPerSm)
rope_bwd_kernel(const __grid_constant__ RopeBwdArgs g) {
  constexpr int kLanes = D / F, kRows = 32 / kLanes;
  using L = Lane<T, D, F, kInter>;
  const RopeArgs& a = g.a;
  extern __shared__ __align__(16) uint8_t ring[];     // [warp][stage][pass][x, dy][two pieces of every lane]
  __shared__ uint64_t freq[D / 2];
  __shared__ __align__(16) float angles[kWarps][D];
  __shared__ float sums[kWarps][2][D];                // the warps' sums of the weights' gradients
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes;
  const L f(l, a.rot);
  uint8_t* mine = ring + warp * kStagesBwd * kUnroll * 2 * L::kSlot + lane * L::kPiece;
  const uint32_t mine_s = smem_u32(mine);
  Way ahead(a, warp);
  const T *xp = nullptr, *yp = nullptr;
  auto fetch = [&](int st) {
    if (ahead.more()) {
      const da_t4 &src = ahead.kind().src, &gy = ahead.which == 0 ? g.dq_out : g.dk_out;
      if (ahead.fresh) {
        const int b = ahead.t / a.N, n = ahead.t - b * a.N;
        xp = at<T>(src, b, n);
        yp = at<T>(gy, b, n);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        int h;
        if (ahead.row<kRows>(u, sub, &h)) {
          const uint32_t slot = mine_s + (st * kUnroll + u) * 2 * L::kSlot;
          f.fetch(slot + L::kSlot, yp + h * gy.sh);
          if (a.norm) f.fetch(slot, xp + h * src.sh);
        }
      }
      ahead.next();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int st = 0; st < kStagesBwd - 1; ++st) fetch(st);
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) freq[i] = turns(a.inv_freq[i]);
  for (int i = lane; i < 2 * D; i += 32) (&sums[warp][0][0])[i] = 0.f;
  __syncthreads();
  F2Pair w[F / 2], acc[F / 2];
  F2Pair co[F / 4], si[F / 4];
  auto clear = [&]() {
#pragma unroll
    for (int e = 0; e < F / 2; ++e) acc[e] = {0.f, 0.f};
  };
  // the warp's sums of a kind, once: its rows of that kind come on end
  auto keep = [&](int kind) {
#pragma unroll
    for (int e = 0; e < F / 2; ++e) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x = half ? acc[e].hi() : acc[e].lo();
#pragma unroll
        for (int o = kLanes; o < 32; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (sub == 0) sums[warp][kind][f.feature(e, half)] = x;
      }
    }
  };
  clear();
  int st = 0, kind = -1;
  Way way(a, warp);
  Place next{};
  if (way.more()) next = place_of<false>(a, way.which, way.t, lane);
  while (way.more()) {
    const Place place = next;
    Way after = way;
    after.step();
    if (after.more()) next = place_of<false>(a, after.which, after.t, lane);
    const RopeKind& kd = way.kind();  // (kd.dst: dq or dk)
    if (way.which != kind) {
      if (kind >= 0 && g.part) {
        keep(kind);
        clear();
      }
      kind = way.which;
      if (a.norm) load_weight<F>(kd.weight, f, w);
    }
    T* to = at<T>(kd.dst, way.t / a.N, way.t % a.N);
    if (a.rot) {
      token_angles(a, freq, place.pos, angles[warp], D / 2, lane);
      if (f.rotated) load_angles<F / 4, kInter>(angles[warp], D / 2, l, a.rot, co, si);
    }
    for (int p = way.p; p < way.p1; p += kUnroll, st = st + 1 == kStagesBwd ? 0 : st + 1) {
      fetch(st == 0 ? kStagesBwd - 1 : st - 1);
      cp_async_wait<kStagesBwd - 1>();
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p + u >= way.p1) break;
        const int h = (p + u) * kRows + sub;
        const bool row = h < kd.heads;
        const uint8_t* slot = mine + (st * kUnroll + u) * 2 * L::kSlot;
        typename L::Raw x;
        x.load(slot + L::kSlot);
        F2Pair dz[F / 2];
        L::get(x, dz);
        if (f.rotated) {  // the other way: u c + v s, v c - u s
#pragma unroll
          for (int i = 0; i < F / 4; ++i) {
            const F2Pair du = dz[i], dv = dz[F / 4 + i];
            dz[i] = fma2(dv, si[i], du * co[i]);
            dz[F / 4 + i] = fma2(-du, si[i], dv * co[i]);
          }
        }
        if (a.norm) {
          F2Pair xh[F / 2];
          x.load(slot);
          L::get(x, xh);
          const float r = rsqrtf(row_sum<kLanes>(square_sum(xh)) * (1.f / D) + a.norm_eps);
          F2Pair m{0.f, 0.f};
#pragma unroll
          for (int e = 0; e < F / 2; ++e) {
            xh[e] = xh[e] * F2Pair{r, r};
            if (row) acc[e] = fma2(dz[e], xh[e], acc[e]);  // where there is none the slot holds anything
            dz[e] = dz[e] * w[e];
            m = fma2(dz[e], xh[e], m);
          }
          const float mean = row_sum<kLanes>(m.lo() + m.hi()) * (-1.f / D);
#pragma unroll
          for (int e = 0; e < F / 2; ++e) dz[e] = fma2(xh[e], F2Pair{mean, mean}, dz[e]) * F2Pair{r, r};
        }
        if (row) {
          L::put(x, dz);
          x.store(to + h * kd.dst.sh, f);
        }
      }
    }
    way = after;
  }
  cp_async_wait<0>();
  if (g.part == nullptr) return;
  if (kind >= 0) keep(kind);
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float x = 0.f;
    for (int v = 0; v < kWarps; ++v) x += sums[v][i / D][i % D];
    g.part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = x;
  }
}

// dq_weight and dk_weight [d] from the blocks' sums [blocks, 2, d]: a block per 8
// features of one of them, an 8-lane group per share of the blocks, the groups
// added in their order.
__global__ void __launch_bounds__(256) rope_dw_kernel(const float* part, int blocks, int d, float* dq_weight, float* dk_weight) {
  __shared__ double sums[32][8];
  const int group = threadIdx.x / 8, k = threadIdx.x % 8;
  const int i = blockIdx.x * 8 + k;
  double x = 0.0;
  cudaGridDependencySynchronize();
#pragma unroll 4
  for (int b = group; b < blocks; b += 32) x += static_cast<double>(part[static_cast<int64_t>(b) * 2 * d + i]);
  sums[group][k] = x;
  __syncthreads();
  if (group == 0) {
    for (int v = 1; v < 32; ++v) x += sums[v][k];
    float* out = i < d ? dq_weight : dk_weight;
    if (out) out[i < d ? i : i - d] = static_cast<float>(x);
  }
}

// The warps' shares: up to most_passes passes over a token's rows of a kind where
// there are enough of them to fill the SMs' warps, else fewer (at least one).
// They are dealt to the warps in one row: what the GPU reads at a time lies close
// together, and the kinds need not cost the same.  Returns the grid.
unsigned share(RopeArgs& a, int rows, int sms, int most_passes) {
  const int64_t warps = static_cast<int64_t>(sms) * kRopeBlocksPerSm * kWarps;
  int64_t passes = 0, units = 0;
  for (RopeKind& k : a.kind) {
    k.passes = (k.heads + rows - 1) / rows;
    passes += k.passes;
  }
  int64_t each = a.tokens * passes / warps;  // passes to a warp
  if (each > most_passes && a.tokens < (1 << 20)) each = most_passes;  // (units are counted in 32 bits)
  if (each < 1) each = 1;
  for (RopeKind& k : a.kind) {
    k.unit0 = static_cast<uint32_t>(units);
    k.chunk_passes = static_cast<int>(each < k.passes ? each : k.passes);
    k.chunks = k.passes ? (k.passes + k.chunk_passes - 1) / k.chunk_passes : 0;
    units += a.tokens * k.chunks;
  }
  a.units = static_cast<uint32_t>(units);
  const int64_t want = (units + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * kRopeBlocksPerSm;
  return static_cast<unsigned>(want < most ? want : most);
}

template <class A>
cudaError_t launch(void (*kernel)(A), OncePerDevice& once, const A& a, unsigned grid, int smem, cudaStream_t s) {
  const cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <bool kPaged, typename T, int D, int F>
cudaError_t launch_rows_f(RopeArgs a, int sms, cudaStream_t s) {
  constexpr int kSmem = kWarps * kStagesFwd * kUnroll * Lane<T, D, F, false>::kSlot;
  static OncePerDevice once[4];
  const unsigned grid = share(a, 32 * F / D, sms, kSharePasses);
  if (a.norm && a.rot < D)
    return a.interleaved ? launch(rope_rows_kernel<T, D, F, true, kPaged, true>, once[3], a, grid, kSmem, s)
                         : launch(rope_rows_kernel<T, D, F, false, kPaged, true>, once[2], a, grid, kSmem, s);
  return a.interleaved ? launch(rope_rows_kernel<T, D, F, true, kPaged, false>, once[1], a, grid, kSmem, s)
                       : launch(rope_rows_kernel<T, D, F, false, kPaged, false>, once[0], a, grid, kSmem, s);
}

template <typename T, int D, int F>
cudaError_t launch_bwd_f(RopeBwdArgs g, int sms, cudaStream_t s) {
  constexpr int kSmem = kWarps * kStagesBwd * kUnroll * 2 * Lane<T, D, F, false>::kSlot;
  static OncePerDevice once[2];
  const unsigned grid = share(g.a, 32 * F / D, sms, kSharePassesBwd);
  const cudaError_t e = g.a.interleaved ? launch(rope_bwd_kernel<T, D, F, true>, once[1], g, grid, kSmem, s)
                                        : launch(rope_bwd_kernel<T, D, F, false>, once[0], g, grid, kSmem, s);
  if (e != cudaSuccess || g.part == nullptr) return e;
  return launch_ahead(rope_dw_kernel, dim3(2 * D / 8), dim3(256), 0, s, true, static_cast<const float*>(g.part),
                      static_cast<int>(grid), D, g.dq_weight, g.dk_weight);
}

// Features of a lane: what two 16-byte pieces hold, if whole lanes are rotated.
template <bool kPaged, typename T, int D>
cudaError_t launch_rows(const RopeArgs& a, int sms, cudaStream_t s) {
  if (sizeof(T) == 2 && a.rot % 16 == 0) return launch_rows_f<kPaged, T, D, sizeof(T) == 2 ? 16 : 8>(a, sms, s);
  return launch_rows_f<kPaged, T, D, 8>(a, sms, s);
}

template <typename T, int D>
cudaError_t launch_bwd(const RopeBwdArgs& g, int sms, cudaStream_t s) {
  if (sizeof(T) == 2 && g.a.rot % 16 == 0) return launch_bwd_f<T, D, sizeof(T) == 2 ? 16 : 8>(g, sms, s);
  return launch_bwd_f<T, D, 8>(g, sms, s);
}

}  // namespace

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
