// paged_decode.cu — V2 differential attention over a paged cache for few new
// tokens per sequence (decode steps, drafted tokens to verify), bound by reading
// the cache once.
//
// The keys are the MMA's 128 rows and the queries its columns: S = K Q^T is 128
// keys x C columns, C = 8, 16 or 32 of (token, query head of the KV head), so
// that the products cost what the queries need and not 128 rows of them, a
// thread of the softmax holds the C scores of one key, and the output
// O = V^T P^T (D features x C columns) adds up in its registers.
//
//   P goes to the value product as two bf16 numbers, P = hi + lo, side by side as
//   2C columns of one MMA: 16 bits of the weights for a product that is not what
//   bounds the kernel (bf16 alone: 0.0026 of the output's norm off, with lo 0.0017,
//   the output's own rounding, 64 sequences of 32768).
//   The first tile of a part gives each column's maximum m; later tiles only
//   check that no weight passes 2^24, and the rare one that does raises m.
//   Every tile's product starts from zero and is added in fp32.
//
//   a warpgroup or, for C = 32, two with half of the columns each: softmax, sums,
//     epilogue (thread = key of the tile, then feature)
//   a warp, with pages of 16 and D = 64 two: TMA producer (queries; K and V page by
//     page, paged.cuh)
//   a warp (one lane): MMA issuer; S of the next tile, the next item's first
//     among them, goes ahead of the product of this one
//   Shared memory: K and V rings (3 stages of 64 KB for D = 128, 6 of 32 KB for
//   64: what HBM's latency needs in flight), two query tiles, the P buffers.
//   TMEM: two S buffers of max(C, 16) columns, two O buffers of 2C.
//
// A CTA's share of the work is a run of key tiles (paged.cuh); copies of its next
// items run while it ends one.  64 sequences of 32768 with 8 KV heads, d 128: 1192
// us, 7.2 TB/s, every byte of the cache read once (ncu: 537 MB for 537 of 16 x
// 8192); 16 x 8192: 90 us, of which 6 are the shares and the first tile's way from
// memory, 4 the joining of cut items; 1 x 1000: 12 us, all of it latency.
#include <type_traits>

#include "paged.cuh"
#include "softmax.cuh"
#include "tma.cuh"

namespace da {
namespace {

// barrier indices (8 bytes each); up to 6 stages
enum { B_QFULL = 0, B_QEMPTY = 2, B_SFULL = 4, B_PFULL = 6, B_OFULL = 8, B_KFULL = 10, B_KEMPTY = 16, B_VFULL = 22, B_VEMPTY = 28,
       B_COUNT = 34 };
constexpr int kBarBytes = 320;
static_assert(B_COUNT * 8 <= kBarBytes, "barrier area");

template <int D, int C, int P>  // P: producer warps
struct Cfg {
  using Tile = KeyTile<D>;
  static constexpr int kStages = D == 128 ? 3 : 6;
  // 32 columns take a warpgroup longer than the memory takes a tile of D = 64
  // (32 sequences of 4096, 4 tokens x 8 heads: 55 us, 43 with two)
  static constexpr int kGroups = C == 32 ? 2 : 1;
  static constexpr int kCols = C / kGroups;              // of a warpgroup
  static constexpr int kThreads = kGroups * 128 + P * 32 + 32;
  static constexpr int kCq = C < 16 ? 16 : C;            // an MMA has 16 columns at least
  static constexpr int kQBytes = Tile::kNB * kCq * 128;  // boxes of 64 features x kCq rows
  static constexpr int kPBox = 2 * C * 128;              // 64 keys x (C columns hi, C lo)
  static constexpr int kPBytes = 2 * kPBox;
  static constexpr int kPBufs = C == 32 ? 1 : 2;         // as many as fit beside the rings
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kStages * Tile::kBytes;
  static constexpr int kOffQ = 2 * kStages * Tile::kBytes;
  static constexpr int kOffP = kOffQ + 2 * kQBytes;
  static constexpr int kOffBar = kOffP + kPBufs * kPBytes;
  // barriers, reduction buffers [4 warps][C] x 2, slack for alignment
  static constexpr int kSmem = kOffBar + kBarBytes + 2 * 4 * C * 4 + 1024;
  static constexpr int kTmemO = 2 * kCq;
  static constexpr int kTmem = 2 * kCq + 4 * C <= 64 ? 64 : 2 * kCq + 4 * C <= 128 ? 128 : 256;
  static_assert(kSmem <= 232448 - 256, "shared memory of a block, some of it static");
};

__host__ __device__ constexpr uint32_t idesc_t(int N, int a_mn_major) {  // M = 128, B K-major
  return idesc_bf16(128, N, 0) | (static_cast<uint32_t>(a_mn_major) << 15);
}

__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ bool wait_bar(volatile int* abort_flag, uint32_t bar, uint32_t parity, uint32_t* status, uint32_t site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer() - t0 > 2000000000ull) {
      record_status(status, DA_ERR_TIMEOUT, site);
      *abort_flag = 1;
      return false;
    }
  }
}

// A named barrier (1 and up) over a warpgroup; the second also says whether any passed `pred`.
__device__ __forceinline__ void sync_128(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool any_128(int id, bool pred) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(pred)), "r"(id)
               : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// N consecutive TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  } else {
    static_assert(N == 8, "8 or 16 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  }
}

template <int D, int C, int P>
__global__ void __launch_bounds__(Cfg<D, C, P>::kThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, PagedArgs a) {
  using F = Cfg<D, C, P>;
  using Tile = typename F::Tile;
  constexpr int kS = F::kStages;
  constexpr int kProducer = F::kGroups * 4, kIssuer = kProducer + P;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PagedShares<1> share;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + F::kOffBar + 8 * i; };
  float* red = reinterpret_cast<float*>(gen + F::kOffBar + kBarBytes);  // [2][4][C]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  PagedSequence mine;
  if (threadIdx.x < a.cache.B) mine.load(a.cache, threadIdx.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_QEMPTY + i), 1);
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_PFULL + i), F::kGroups * 128);
      mbar_init(bar(B_OFULL + i), 1);
    }
    for (int i = 0; i < kS; ++i) {
      mbar_init(bar(B_KFULL + i), 1);
      mbar_init(bar(B_KEMPTY + i), 1);
      mbar_init(bar(B_VFULL + i), 1);
      mbar_init(bar(B_VEMPTY + i), 1);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(&tmem_slot), F::kTmem);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  paged_share<F::kThreads>(a, mine, &share);
  if (share.bad) paged_out_of_bounds(a, &share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // A producer warp's copies of the queries and keys, of the values, or of all.
  auto produce = [&](auto keys, auto values) {
    constexpr bool kKeys = decltype(keys)::value, kValues = decltype(values)::value;
    const PageCopies copies(a, lane);
    auto wait_warp = [&](uint32_t b, uint32_t parity, uint32_t site) {
      return __all_sync(0xffffffffu, wait_bar(&abort_flag, b, parity, a.status, site)) != 0;
    };
    int it = 0, st = 0;
    uint32_t round = 0;  // of the rings
    bool ok = true;
    for (PagedWalk<1> w(a, share); w.more() && ok; w.next(), ++it) {
      int entry = copies.entry(w.b, w.L, w.j);
      if (kKeys && it > 1) ok = wait_warp(bar(B_QEMPTY + (it & 1)), ((it >> 1) - 1) & 1, 0x9001);
      if (!ok) break;
      if (kKeys && lane == 0) {
        mbar_arrive_expect_tx(bar(B_QFULL + (it & 1)), Tile::kNB * a.G * a.tq * 128);
        for (int box = 0; box < Tile::kNB; ++box)
          tma_load_3d(base + F::kOffQ + (it & 1) * F::kQBytes + box * F::kCq * 128, &tm_q, bar(B_QFULL + (it & 1)), box * 64,
                      w.g * a.G, w.t0 + w.i * a.tq);
      }
      for (int j = w.j; j < w.j1; ++j) {
        const int page = copies.page(entry, w.L, j), group = copies.group(j);
        if (j + 1 < w.j1) entry = copies.entry(w.b, w.L, j + 1);  // looked up a tile ahead
        const uint32_t to = st * Tile::kBytes + Tile::row(copies.row0);
        if constexpr (kKeys) {
          if (round > 0) ok = wait_warp(bar(B_KEMPTY + st), (round - 1) & 1, 0x9002);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(B_KFULL + st), Tile::kBytes);
          __syncwarp();
          if (copies.mine)
            tma_load_5d(base + F::kOffK + to, &tm_k, bar(B_KFULL + st), 0, 0, w.g * copies.k_block, group, page);
        }
        if constexpr (kValues) {
          if (round > 0) ok = wait_warp(bar(B_VEMPTY + st), (round - 1) & 1, 0x9003);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(B_VFULL + st), Tile::kBytes);
          __syncwarp();
          if (copies.mine)
            tma_load_5d(base + F::kOffV + to, &tm_v, bar(B_VFULL + st), 0, 0, w.g * copies.v_block, group, page);
        }
        if (++st == kS) st = 0, ++round;
      }
    }
    if (!ok) {
      // give the copies already issued (bounded) time to land
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 100000000ull) {
      }
    }
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;

  if (warp == kProducer) {
    // ------------------------------------------------------ TMA producer --
    if constexpr (P > 1)
      produce(yes, no);
    else
      produce(yes, yes);
  } else if (P > 1 && warp == kProducer + 1) {
    produce(no, yes);
  } else if (warp == kIssuer) {
    // ------------------------------------------------------- MMA issuer ---
    if (lane == 0) {
      constexpr uint32_t kTile = Tile::kBytes >> 4;
      const uint32_t q0 = sdesc_lo(base + F::kOffQ, 16), k0 = sdesc_lo(base + F::kOffK, 16);
      // with D = 64 rows 64 to 127 of V^T are the next rows' features: no one looks at what they give
      const uint32_t v0 = sdesc_lo(base + F::kOffV, 1024), p0 = sdesc_lo(base + F::kOffP, 16);
      auto wait = [&](uint32_t b, uint32_t parity, uint32_t site) { return wait_bar(&abort_flag, b, parity, a.status, site); };
      // S of tile x (of the CTA's share) for the item that a walk of its own is at
      PagedWalk<1> ahead(a, share);
      int it = 0, j = ahead.j, ks = 0;
      uint32_t k_round = 0;
      auto start = [&](int x) {
        if (j == ahead.j && !wait(bar(B_QFULL + (it & 1)), (it >> 1) & 1, 0x9101)) return false;
        if (!wait(bar(B_KFULL + ks), k_round & 1, 0x9102)) return false;
        tc_fence_after();
        const uint32_t q = q0 + (it & 1) * (F::kQBytes >> 4), k = k0 + ks * kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_lo(tmem + (x & 1) * F::kCq, k + Tile::feature_step(kk), Tile::kHi,
                       q + (((kk >> 2) * F::kCq * 128 + (kk & 3) * 32) >> 4), sdesc_hi(1024), idesc_t(F::kCq, 0), kk > 0);
        tc_commit(bar(B_SFULL + (x & 1)));
        tc_commit(bar(B_KEMPTY + ks));
        if (++ks == kS) ks = 0, ++k_round;
        if (++j == ahead.j1) {
          tc_commit(bar(B_QEMPTY + (it & 1)));
          ++it;
          ahead.next();
          j = ahead.j;
        }
        return true;
      };
      int vs = 0;
      uint32_t v_round = 0;
      bool more = ahead.more() && start(0);
      for (int x = 0; more; ++x) {
        more = ahead.more();
        if (more && !start(x + 1)) break;
        if (!wait(bar(B_VFULL + vs), v_round & 1, 0x9103) || !wait(bar(B_PFULL + (x & 1)), (x >> 1) & 1, 0x9104)) break;
        tc_fence_after();
        const uint32_t v = v0 + vs * kTile, p = p0 + (x & (F::kPBufs - 1)) * (F::kPBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kPagedTile / 16; ++kk)
          tc_mma_ss_lo(tmem + F::kTmemO + (x & 1) * 2 * C, v + Tile::key_step(kk), Tile::kHi,
                       p + (((kk >> 2) * F::kPBox + (kk & 3) * 32) >> 4), sdesc_hi(1024), idesc_t(2 * C, 1), kk > 0);
        tc_commit(bar(B_OFULL + (x & 1)));
        tc_commit(bar(B_VEMPTY + vs));
        if (++vs == kS) vs = 0, ++v_round;
      }
    }
  } else {
    // --------------------------------------------- softmax + epilogue -----
    // The four warps of a warpgroup reach its named barrier in the same order: it
    // depends on the part, the tile and barrier reductions only, and a failed wait
    // leaves at the end of a part, for all of them.
    constexpr int kC = F::kCols;
    const int wg = F::kGroups > 1 ? warp >> 2 : 0, q4 = warp & 3, id = 1 + wg;
    const int n0 = wg * kC;              // the warpgroup's first column
    const int r = threadIdx.x & 127;     // key of the tile; TMEM lane; feature of the output
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const float sl2 = a.scale_log2;
    // this key's place in a P row: 64 keys to a box, 16-byte pieces swizzled by the row
    uint8_t* p_key = gen + F::kOffP + (r >> 6) * F::kPBox + (r & 7) * 2 + n0 * 128;
    const int piece = (r & 63) >> 3;
    red += wg * 8 * kC;                  // [2][4][kC]
    int x = 0, flags = 0, vs = 0;
    uint32_t v_round = 0;
    PagedDesc desc{0, 0, 0, 0};
    bool ok = true, synced = !a.after_gate;
    for (PagedWalk<1> w(a, share); w.more(); w.next()) {
      const int cols = w.tokens * a.G - n0;  // the item's columns, from n0 on
      const bool whole = w.begins() && w.ends();
      const int64_t part = static_cast<int64_t>(2 * w.number() + (w.begins() ? 1 : 0)) * a.rows;
      // what thread n's column n is scaled by: 1 (even heads) or the gate
      auto gate_of = [&]() {
        const int tok = (n0 + r) / a.G;
        return (r & 1) && r < cols && r < kC
                   ? a.gate[(w.t0 + static_cast<int64_t>(w.i) * a.tq + tok) * a.h + w.g * (a.G / 2) + (n0 + r - tok * a.G) / 2]
                   : 1.f;
      };
      float gate = whole && synced ? gate_of() : 1.f;
      float m[kC], l[kC], o[kC];
#pragma unroll
      for (int n = 0; n < kC; ++n) m[n] = l[n] = o[n] = 0.f;
      // the product of the tile before: O += hi part + lo part
      auto add_product = [&]() {
        if (!wait_bar(&abort_flag, bar(B_OFULL + ((x - 1) & 1)), ((x - 1) >> 1) & 1, a.status, 0x9202)) ok = false;
        tc_fence_after();
        uint32_t hi[kC], lo[kC];
        const uint32_t t = tmem + lane_off + F::kTmemO + ((x - 1) & 1) * 2 * C + n0;
        tmem_ld<kC>(t, hi);
        tmem_ld<kC>(t + C, lo);
        tmem_ld_wait();
#pragma unroll
        for (int n = 0; n < kC; ++n) o[n] += __uint_as_float(hi[n]) + __uint_as_float(lo[n]);
        tc_fence_before();
      };
      for (int j = w.j; j < w.j1; ++j, ++x) {
        const int key = j * kPagedTile + r;
        const bool masked = j * kPagedTile + kPagedTile - 1 > w.first_position();
        if (!wait_bar(&abort_flag, bar(B_SFULL + (x & 1)), (x >> 1) & 1, a.status, 0x9201)) ok = false;
        tc_fence_after();
        uint32_t s[kC];
        tmem_ld<kC>(tmem + lane_off + (x & 1) * F::kCq + n0, s);
        tmem_ld_wait();
        float p[kC];
#pragma unroll
        for (int n = 0; n < kC; ++n) p[n] = __uint_as_float(s[n]) * sl2;
        if (masked) {
          // column n is token n / G, which sees the keys up to its position
          const int from = max(0, key - w.first_position()) * a.G - n0;  // columns from here on see the key
#pragma unroll
          for (int n = 0; n < kC; ++n)
            if (n < from) p[n] = -INFINITY;
        }
        // the maximum of every column over the tile's keys (between two of these
        // there is always another barrier, so `red` has been read)
        auto tile_max = [&](float (&mx)[kC]) {
#pragma unroll
          for (int n = 0; n < kC; ++n) {
            const float v = warp_max(p[n]);
            if (lane == (n & 31)) red[q4 * kC + n] = v;
          }
          sync_128(id);
#pragma unroll
          for (int n = 0; n < kC; ++n) {
            mx[n] = fmaxf(fmaxf(red[n], red[kC + n]), fmaxf(red[2 * kC + n], red[3 * kC + n]));
          }
        };
        float e[kC], scale[kC];
        bool raised = false;
        if (j == w.j) {
          tile_max(m);
#pragma unroll
          for (int n = 0; n < kC; ++n)
            if (m[n] == -INFINITY) m[n] = 0.f;  // a column that sees none of these keys sees none behind them
        } else {
          bool over = false;
#pragma unroll
          for (int n = 0; n < kC; ++n) over |= n < cols && !(p[n] - m[n] <= static_cast<float>(kRaise));
          if (any_128(id, over)) {
            float mx[kC];
            tile_max(mx);
            raised = true;
#pragma unroll
            for (int n = 0; n < kC; ++n) {
              const float mn = fmaxf(m[n], mx[n]);
              scale[n] = exp2f(m[n] - mn);
              m[n] = mn;
              l[n] *= scale[n];
            }
          }
        }
#pragma unroll
        for (int n = 0; n < kC; ++n) {
          e[n] = fast_exp2(p[n] - m[n]);
          l[n] += e[n];
        }
        if (key >= w.L && wg == 0) {
          // a value behind the sequence's end may be a NaN, and 0 times it is not 0
          if (!wait_bar(&abort_flag, bar(B_VFULL + vs), v_round & 1, a.status, 0x9203)) ok = false;
          uint8_t* v = gen + F::kOffV + vs * Tile::kBytes + Tile::row(r);
#pragma unroll
          for (int c = 0; c < 8 * Tile::kNB; ++c)
            *reinterpret_cast<uint4*>(v + c / 8 * 1024 + c % 8 * 16) = make_uint4(0, 0, 0, 0);
        }
        if (F::kPBufs == 1 && x > 0 && j > w.j) add_product();  // the P buffer is free once its product is there
        uint8_t* pk = p_key + (x & (F::kPBufs - 1)) * F::kPBytes;
#pragma unroll
        for (int n = 0; n < kC; ++n) {
          const __nv_bfloat16 hi = __float2bfloat16_rn(e[n]);
          const __nv_bfloat16 lo = __float2bfloat16_rn(e[n] - __bfloat162float(hi));
          *reinterpret_cast<__nv_bfloat16*>(pk + n * 128 + ((piece ^ (n & 7)) << 4)) = hi;
          *reinterpret_cast<__nv_bfloat16*>(pk + (C + n) * 128 + ((piece ^ (n & 7)) << 4)) = lo;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(B_PFULL + (x & 1)));
        if (F::kPBufs > 1 && j > w.j) add_product();
        if (raised) {
#pragma unroll
          for (int n = 0; n < kC; ++n) o[n] *= scale[n];
        }
        if (++vs == kS) vs = 0, ++v_round;
      }
      // ----------------------------------------------------- epilogue ----
      add_product();
      // each column's sum over the warp's keys: the columns are halved with every
      // exchange, until a lane has one
      int col = 0, off = 16;
#pragma unroll
      for (int half = kC / 2; half > 0; half /= 2, off /= 2) {
        const bool upper = lane & off;
#pragma unroll
        for (int n = 0; n < half; ++n) {
          const float send = upper ? l[n] : l[n + half];
          l[n] = (upper ? l[n + half] : l[n]) + __shfl_xor_sync(0xffffffffu, send, off);
        }
        col += upper ? half : 0;
      }
      float lw = l[0];
      for (; off > 0; off /= 2) lw += __shfl_xor_sync(0xffffffffu, lw, off);
      if ((lane & (32 / kC - 1)) == 0) red[(4 + q4) * kC + col] = lw;
      if (whole && !synced) {
        cudaGridDependencySynchronize();  // the gate
        synced = true;
        gate = gate_of();
      }
      if (any_128(id, !ok || abort_flag)) {
        ok = false;
        break;
      }
      if (r < kC) {  // thread n has column n's sum
        const float sum = (red[4 * kC + r] + red[5 * kC + r]) + (red[6 * kC + r] + red[7 * kC + r]);
        if (whole) {
          red[4 * kC + r] = gate / sum;
        } else if (r < cols) {
          float mr = m[0];
#pragma unroll
          for (int n = 1; n < kC; ++n) mr = r == n ? m[n] : mr;
          *reinterpret_cast<float2*>(a.part_ml + (part + n0 + r) * 2) = make_float2(sum == 0.f ? -INFINITY : mr, sum);
        }
      }
      if (whole) {
        sync_128(id);
        const int half = a.G / 2;
        int tok = n0 / a.G, p = (n0 - tok * a.G) / 2;
#pragma unroll
        for (int n = 0; n < kC; n += 2) {
          if (n < cols && r < D) {
            const int64_t t = w.t0 + static_cast<int64_t>(w.i) * a.tq + tok;
            // the products rounded apart, so that equal heads cancel with gate 1
            const float y = __fsub_rn(__fmul_rn(o[n], red[4 * kC + n]), __fmul_rn(o[n + 1], red[4 * kC + n + 1]));
            static_cast<__nv_bfloat16*>(a.out.ptr)[t * a.out.st + (w.g * half + p) * a.out.sh + r] = __float2bfloat16_rn(y);
          }
          if (++p == half) p = 0, ++tok;
        }
      } else {
#pragma unroll
        for (int n = 0; n < kC; ++n)
          if (n < cols && r < D) a.part_o[(part + n0 + n) * D + r] = o[n];
        if (!w.begins() && w.ends()) flags |= kPagedEnds;
        if (w.begins()) desc = PagedDesc{kPagedOpen, w.t0 + w.i * a.tq, w.tokens, w.g};
      }
    }
    if (threadIdx.x == 0) {
      desc.flags = ok ? desc.flags | flags : 0;
      a.desc[blockIdx.x] = desc;
    }
    if (!synced) cudaGridDependencySynchronize();  // the merge counts on the gate's end
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, F::kTmem);
}

template <int D, int C, int P>
cudaError_t launch_p(const PagedArgs& a, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  const da_paged_cache& c = a.cache;
  if (!encode_queries(&tq, a, a.tq) || !encode_pages(&tk, c.k_pages, c, a.box) || !encode_pages(&tv, c.v_pages, c, a.box))
    return cudaErrorInvalidValue;
  static OncePerDevice once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(paged_decode_kernel<D, C, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, C, P>::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_ahead(paged_decode_kernel<D, C, P>, dim3(a.grid), dim3(Cfg<D, C, P>::kThreads), Cfg<D, C, P>::kSmem, s,
                      a.after_gate, tq, tk, tv, a);
}

// A warp issues its lanes' copies one after the other: with 16 to a tile of 32 KB the
// values' are a second warp's (pages of 16, d 64, 24 ragged sequences up to 20000: 131
// us with one warp, 109 with two; with fewer or longer copies two warps are 2 to 4 %
// slower, pages of 64: 112 and 114).
template <int D, int C>
cudaError_t launch_c(const PagedArgs& a, cudaStream_t s) {
  if constexpr (D == 64) {
    if (a.box == 16) return launch_p<D, C, 2>(a, s);
  }
  return launch_p<D, C, 1>(a, s);
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, cudaStream_t s) {
  switch (a.rows) {
    case 8: return launch_c<D, 8>(a, s);
    case 16: return launch_c<D, 16>(a, s);
    case 32: return launch_c<D, 32>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t s) {
  const cudaError_t e = a.cache.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
  return e == cudaSuccess ? launch_paged_merge(a, s) : e;
}

}  // namespace da
