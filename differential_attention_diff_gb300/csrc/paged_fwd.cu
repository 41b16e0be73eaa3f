// paged_fwd.cu — V2 differential attention of new tokens over a paged cache, for
// chunks of a prompt, on the 5th-generation tensor cores (tcgen05, TMEM, TMA).
//
// Token i of a sequence's n new ones sees keys 0 .. L - n + i of its L cached
// ones (its own among them); out = O_2p - gate O_2p+1 (diffattn.h).
//
// A CTA's share of the work is a run of key tiles of a run of items (paged.cuh).
// The MMA's 128 rows are 128 / G tokens times the G query heads of a KV head, in
// the order in which q holds them, so that one TMA copy fills a Q tile and heads
// 2p and 2p + 1 are neighbouring rows (lanes); every K and V tile is read for all
// heads of the group.  An item has two such Q tiles, A and B, whose softmax and
// MMAs take turns: one's products run under the other's exponentials.  An item
// with the rows of one Q tile only keeps both turns busy by giving them its even
// and its odd key tiles, joined at its end.
//
//   TMEM (512 columns x 128 lanes, lane = row):
//     [0, 128) S_A (fp32 scores) / P_A (bf16)    [128, 256) S_B / P_B
//     [256, 384) O_A    [384, 512) O_B            (the first D columns of each)
//   Shared memory: Q_A, Q_B in 128-byte-swizzled 64-column boxes of 128 rows, K
//   and V rings of two stages of tiles of pages (paged.cuh), each filled by copies
//   of `box` rows, the largest power of two that divides the page (at most 128);
//   the lanes of the producer warp look up and issue one of K and one of V each.
//
//   warp 8: TMA producer; warp 9 (one lane): MMA issuer; warps 0-7: softmax and
//   epilogue, each warpgroup half of a tile's keys (softmax.cuh).
//
// P is rounded to bf16 for its product, as in the V2 forward: with the differences
// that the gate makes, outputs are 0.0026 of their norm off where their own
// rounding is 0.0017.  A second bf16 for the rest of P would make half as many
// products again, which are what bounds the kernel: a tile pair (256 rows x 128
// keys, d 128) takes 1.55 us where cuBLAS's rate is 1.32, and an item about 4 us
// beside its tiles.  64 query and 8 KV heads, d 128: 2048 tokens of 32768 in 1307 us
// (1.63 PFLOP/s, 0.84 of measured), 8192 of 8192 in 722 us (1.52), 2048 of 8192 in
// 325 us (1.48), the joining of parts among them; tensor pipe 65 % active.
//
// A tile that reaches past the sequence's end holds what the page holds there:
// the scores are masked, and the values' rows are zeroed in shared memory before
// the product, since 0 times a NaN would not be 0.
#include "paged.cuh"
#include "softmax.cuh"
#include "tma.cuh"

namespace da {
namespace {

constexpr int kThreads = 320;
constexpr int kBox = 128 * 128;            // bytes of one 64-column box of 128 rows
constexpr int kOffBar = 12 * kBox;
constexpr int kSmemBytes = kOffBar + 8192 + 1024;  // + barriers and exchange, + alignment slack

enum {
  B_QFULL = 0, B_QEMPTY = 1, B_KFULL = 2, B_VFULL = 4, B_KEMPTY = 6, B_VEMPTY = 8, B_SFULL = 10, B_PFULL = 12,
  B_ORDY = 14, B_COUNT = 15
};
constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0);  // Q (K-major) x K (K-major)

struct Shared {
  uint32_t base;  // 1024-aligned shared address of the tile region
  uint8_t* gen;   // the same, as a pointer
  __device__ uint32_t bar(int i) const { return base + kOffBar + 8 * i; }
  __device__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(gen + kOffBar + 128); }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(gen + kOffBar + 192); }
  // rows' partial sums [turn][half][128] and half maxima [turn][half][128]
  __device__ float* lx() const { return reinterpret_cast<float*>(gen + kOffBar + 256); }
  __device__ float* xm() const { return reinterpret_cast<float*>(gen + kOffBar + 256 + 2048); }
};

__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Bounded wait that also gives up when another role raised the abort flag.
__device__ __forceinline__ bool wait_bar(const Shared& sh, uint32_t bar, uint32_t parity, uint32_t* status, uint32_t site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*sh.abort_flag()) return false;
    if (globaltimer() - t0 > 2000000000ull) {
      record_status(status, DA_ERR_TIMEOUT, site);
      *sh.abort_flag() = 1;
      return false;
    }
  }
}

template <int D, int kTurns>
__global__ void __launch_bounds__(kThreads, 1)
paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PagedShares<kTurns> share;
  Shared sh;
  {
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t aligned = (raw + 1023u) & ~1023u;
    sh.base = aligned;
    sh.gen = smem_raw + (aligned - raw);
  }
  using Tile = KeyTile<D>;
  constexpr int kNB = D / 64;  // 64-column boxes per Q tile
  constexpr int kOffQ = 0, kOffK = 2 * kNB * kBox, kOffV = kOffK + 2 * Tile::kBytes;
  constexpr uint32_t kIdescPV = idesc_bf16(128, D, 1);  // P (TMEM) x V (MN-major)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  PagedSequence mine;
  if (threadIdx.x < a.cache.B) mine.load(a.cache, threadIdx.x);

  if (threadIdx.x == 0) {
    mbar_init(sh.bar(B_QFULL), 1);
    mbar_init(sh.bar(B_QEMPTY), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(sh.bar(B_KFULL + s), 1);
      mbar_init(sh.bar(B_VFULL + s), 1);
      mbar_init(sh.bar(B_KEMPTY + s), 1);
      mbar_init(sh.bar(B_VEMPTY + s), 1);
      mbar_init(sh.bar(B_SFULL + s), 1);
      mbar_init(sh.bar(B_PFULL + s), 256);
    }
    mbar_init(sh.bar(B_ORDY), 1);
    *sh.abort_flag() = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(sh.tmem_slot()), 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  paged_share<kThreads>(a, mine, &share);
  if (share.bad) paged_out_of_bounds(a, &share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh.tmem_slot();
  // the item's tokens have two Q tiles (A and B over the same key tiles), or one
  // (A and B over every other key tile)
  auto two = [&](const PagedWalk<kTurns>& w) { return w.tokens > a.tq1; };

  if (warp == 8) {
    // ------------------------------------------------------ TMA producer --
    const PageCopies copies(a, lane);
    // all lanes wait, and all go on or none
    auto wait_warp = [&](uint32_t bar, uint32_t parity, uint32_t site) {
      return __all_sync(0xffffffffu, wait_bar(sh, bar, parity, a.status, site)) != 0;
    };
    int kv_it = 0, it = 0;
    bool ok = true;
    for (PagedWalk<kTurns> w(a, share); w.more() && ok; w.next(), ++it) {
      int entry = copies.entry(w.b, w.L, w.j);
      if (it > 0) ok = wait_warp(sh.bar(B_QEMPTY), (it - 1) & 1, 0x8001);
      if (ok && lane == 0) {
        const int tiles = two(w) ? 2 : 1;
        mbar_arrive_expect_tx(sh.bar(B_QFULL), tiles * kNB * a.G * a.tq1 * 128);
        for (int s = 0; s < tiles; ++s)
          for (int box = 0; box < kNB; ++box)
            tma_load_3d(sh.base + kOffQ + (s * kNB + box) * kBox, &tm_q, sh.bar(B_QFULL), box * 64, w.g * a.G,
                        w.t0 + w.i * a.tq + s * a.tq1);
      }
      for (int j = w.j; j < w.j1 && ok; ++j, ++kv_it) {
        const int st = kv_it & 1, use = kv_it >> 1;
        const int page = copies.page(entry, w.L, j), group = copies.group(j);
        if (j + 1 < w.j1) entry = copies.entry(w.b, w.L, j + 1);  // looked up a tile ahead
        const uint32_t to = st * Tile::kBytes + Tile::row(copies.row0);
        if (use > 0) ok = wait_warp(sh.bar(B_KEMPTY + st), (use - 1) & 1, 0x8002);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(sh.bar(B_KFULL + st), Tile::kBytes);
        __syncwarp();
        if (copies.mine)
          tma_load_5d(sh.base + kOffK + to, &tm_k, sh.bar(B_KFULL + st), 0, 0, w.g * copies.k_block, group, page);
        if (use > 0) ok = wait_warp(sh.bar(B_VEMPTY + st), (use - 1) & 1, 0x8003);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(sh.bar(B_VFULL + st), Tile::kBytes);
        __syncwarp();
        if (copies.mine)
          tma_load_5d(sh.base + kOffV + to, &tm_v, sh.bar(B_VFULL + st), 0, 0, w.g * copies.v_block, group, page);
      }
    }
    if (!ok) {
      // give the copies already issued (bounded) time to land
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 100000000ull) {
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------- MMA issuer ---
    // One thread, whose instructions between two MMAs are what bounds the loop
    // when there are many: descriptors are sums of a base and constants, and
    // turns are told apart by unrolling.
    if (lane == 0) {
      int kv_it = 0, it = 0;
      uint32_t pc[2] = {0, 0};
      bool ok = true;
      const uint32_t q0 = sdesc_lo(sh.base + kOffQ, 16), k0 = sdesc_lo(sh.base + kOffK, 16), v0 = sdesc_lo(sh.base + kOffV, 1024);
      constexpr uint32_t kTile = Tile::kBytes >> 4;  // descriptor units (16 bytes) from one tile (Q, K or V) to the next
      auto issue_s = [&](int s, uint32_t q, uint32_t k) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_lo(tmem + s * 128, q + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4), sdesc_hi(1024), k + Tile::feature_step(kk),
                       Tile::kHi, kIdescS, kk > 0);
        tc_commit(sh.bar(B_SFULL + s));
      };
      auto issue_pv = [&](int s, uint32_t v, bool acc) {
#pragma unroll
        for (int kk = 0; kk < kPagedTile / 16; ++kk)
          // P of keys 0-63 in columns 0-31 of the S buffer, keys 64-127 in 64-95
          tc_mma_ts_lo(tmem + 256 + s * 128, tmem + s * 128 + kk * 8 + (kk >= 4 ? 32 : 0), v + Tile::key_step(kk), Tile::kHi,
                       kIdescPV, (acc || kk > 0) ? 1u : 0u);
      };
      auto full = [&](int bar, int x, uint32_t site) {  // of tile x's stage
        return wait_bar(sh, sh.bar(bar + (x & 1)), (x >> 1) & 1, a.status, site);
      };
      for (PagedWalk<kTurns> w(a, share); w.more() && ok; w.next(), ++it) {
        const int tiles = w.j1 - w.j;
        if (!wait_bar(sh, sh.bar(B_QFULL), it & 1, a.status, 0x8101)) break;
        if (!full(B_KFULL, kv_it, 0x8102)) break;
        tc_fence_after();
        if (two(w)) {
          // both turns on every tile
          const uint32_t kb = k0 + (kv_it & 1) * kTile;
          issue_s(0, q0, kb);
          issue_s(1, q0 + kTile, kb);
          tc_commit(sh.bar(B_KEMPTY + (kv_it & 1)));
          if (tiles == 1) tc_commit(sh.bar(B_QEMPTY));
          for (int j = 0; j < tiles; ++j) {
            const int x = kv_it + j, st = x & 1;
            const uint32_t v = v0 + st * kTile, k = k0 + (st ^ 1) * kTile;
            const bool more = j + 1 < tiles;
            ok = full(B_VFULL, x, 0x8104) && wait_bar(sh, sh.bar(B_PFULL + 0), pc[0] & 1, a.status, 0x8103);
            if (!ok) break;
            tc_fence_after();
            issue_pv(0, v, j > 0);
            if (more) {
              ok = full(B_KFULL, x + 1, 0x8105);
              if (!ok) break;
              tc_fence_after();
              issue_s(0, q0, k);
            }
            ok = wait_bar(sh, sh.bar(B_PFULL + 1), pc[1] & 1, a.status, 0x8106);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, v, j > 0);
            tc_commit(sh.bar(B_VEMPTY + st));
            if (more) {
              issue_s(1, q0 + kTile, k);
              tc_commit(sh.bar(B_KEMPTY + (st ^ 1)));
              if (j + 2 == tiles) tc_commit(sh.bar(B_QEMPTY));
            }
            ++pc[0];
            ++pc[1];
          }
        } else {
          // turn A on tiles 0, 2, .., turn B on 1, 3, ..: a tile per step
          auto start = [&](int s, int j) {
            const int x = kv_it + j;
            issue_s(s, q0, k0 + (x & 1) * kTile);
            tc_commit(sh.bar(B_KEMPTY + (x & 1)));
            if (j + 1 == tiles) tc_commit(sh.bar(B_QEMPTY));
          };
          auto step = [&](int s, int j) {
            const int x = kv_it + j;
            if (!full(B_VFULL, x, 0x8107) || !wait_bar(sh, sh.bar(B_PFULL + s), pc[s] & 1, a.status, 0x8108)) return false;
            ++pc[s];
            tc_fence_after();
            issue_pv(s, v0 + (x & 1) * kTile, j >= 2);
            tc_commit(sh.bar(B_VEMPTY + (x & 1)));
            if (j + 2 < tiles) {
              if (!full(B_KFULL, x + 2, 0x8109)) return false;
              tc_fence_after();
              start(s, j + 2);
            }
            return true;
          };
          start(0, 0);
          if (tiles > 1) {
            ok = full(B_KFULL, kv_it + 1, 0x810a);
            if (!ok) break;
            tc_fence_after();
            start(1, 1);
          }
          for (int j = 0; j < tiles && ok; j += 2) ok = step(0, j) && (j + 1 == tiles || step(1, j + 1));
        }
        if (!ok) break;
        tc_commit(sh.bar(B_ORDY));
        kv_it += tiles;
      }
    }
  } else {
    // --------------------------------------------- softmax + epilogue -----
    // As in the V2 forward: warpgroup wg takes keys [64 wg, 64 wg + 64) of every
    // tile (thread = row = TMEM lane); the two halves of a row share a running
    // maximum, taken on a turn's first tile and raised on the rare tile whose sum
    // leaves the guard.  Both warpgroups reach named barrier 1 in the same order:
    // it depends on the part, the step and barrier reductions only, and a failed
    // wait leaves at the end of a part, for all of them.
    const int wg = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float sl2 = a.scale_log2;
    const uint64_t sl2x2 = f2(sl2, sl2);
    const int c0 = wg * 64;
    const int my_tok = row / a.G;
    const bool in_tile = row < a.tq1 * a.G;  // 128 need not be a multiple of G
    float* xm = sh.xm();
    int it = 0, kv_it = 0, done = 0;  // done: shares whose parts are all described
    uint32_t sc[2] = {0, 0};
    PagedDesc desc{0, 0, 0, 0};
    bool ok = true, synced = false;
    for (PagedWalk<kTurns> w(a, share); w.more(); w.next(), ++it) {
      for (; kTurns > 1 && done < w.k; ++done) {
        if (threadIdx.x == 0) a.desc[done * gridDim.x + blockIdx.x] = desc;
        desc = PagedDesc{0, 0, 0, 0};
      }
      const bool dual = two(w);
      const int tiles = w.j1 - w.j, steps = dual ? 2 * tiles : tiles;
      float m_run[2] = {0.f, 0.f}, l_half[2] = {0.f, 0.f};
#pragma unroll 1
      for (int k = 0; k < steps; ++k) {
        const int s = k & 1, x = dual ? k >> 1 : k, key0 = (w.j + x) * kPagedTile;
        const int first_tok = dual && s ? a.tq1 : 0;             // of this turn's Q tile
        const int pos0 = w.first_position() + first_tok;          // its position
        const bool masked = key0 + kPagedTile - 1 > pos0;
        const int lim = pos0 + my_tok - key0;                     // the last key column that the row sees
        const bool valid = in_tile && first_tok + my_tok < w.tokens;
        if (!wait_bar(sh, sh.bar(B_SFULL + s), sc[s] & 1, a.status, 0x8201)) ok = false;
        ++sc[s];
        tc_fence_after();
        const uint32_t t_s = tmem + lane_off + s * 128 + c0;
        uint32_t sv[64];
        tmem_ld32(t_s, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_ld_wait();
        auto exps = [&](float m) {
          return masked ? exp_half<true>(sv, c0, lim, sl2x2, m, t_s) : exp_half<false>(sv, c0, lim, sl2x2, m, t_s);
        };
        // the maximum of both halves, in log2 units; a row that sees none of the tile's keys has -inf
        auto tile_max = [&]() {
          const float hm = masked ? half_max<true>(sv, c0, lim) : half_max<false>(sv, c0, lim);
          xm[(s * 2 + wg) * 128 + row] = hm;
          named_sync_256();
          return fmaxf(hm, xm[(s * 2 + (wg ^ 1)) * 128 + row]) * sl2;
        };
        if (k < 2) {
          // a row that sees nothing of its first tile sees nothing of later ones
          const float m = tile_max();
          m_run[s] = m == -INFINITY ? 0.f : m;
          l_half[s] = exps(m_run[s]);
        } else {
          float lsum = exps(m_run[s]);
          if (named_red_or_256(valid && !(lsum <= kPagedSumGuard))) {
            // O is at rest: the commit that signalled these scores covers the turn's last product
            const float m_new = fmaxf(m_run[s], tile_max());
            const float alpha = fast_exp2(m_run[s] - m_new);
            m_run[s] = m_new;
            lsum = exps(m_new);
            l_half[s] = l_half[s] * alpha + lsum;
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
              const uint32_t t_o = tmem + lane_off + 256 + s * 128 + wg * (D / 2);
#pragma unroll 1
              for (int c = 0; c < D / 64; ++c) {
                uint32_t o[32];
                tmem_ld32(t_o + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(t_o + c * 32, o);
              }
            }
          } else {
            l_half[s] += lsum;
          }
        }
        if (key0 + kPagedTile > w.L && (!dual || s == 0)) {
          // values behind the sequence's end: zeros.  These scores were issued behind
          // the product of the tile that had the stage before, so the parity is this one's.
          const int st = (kv_it + x) & 1, r0 = w.L - key0;
          if (!wait_bar(sh, sh.bar(B_VFULL + st), ((kv_it + x) >> 1) & 1, a.status, 0x8203)) ok = false;
          uint8_t* v = sh.gen + kOffV + st * Tile::kBytes;
          for (int e = threadIdx.x; e < (kPagedTile - r0) * 8 * kNB; e += 256)
            *reinterpret_cast<uint4*>(v + Tile::row(r0 + e / (8 * kNB)) + e % (8 * kNB) / 8 * 1024 + e % 8 * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(sh.bar(B_PFULL + s));
      }
      kv_it += tiles;
      // ----------------------------------------------------- epilogue ----
      const bool whole = w.begins() && w.ends();
      if (whole && !synced) {
        cudaGridDependencySynchronize();  // the gate
        synced = true;
      }
      // what the row's output is scaled by: 1 (even heads) or the gate, fetched
      // while the last products run
      const int pair = w.g * (a.G / 2) + ((row - my_tok * a.G) >> 1);
      const int64_t t_item = w.t0 + static_cast<int64_t>(w.i) * a.tq;
      float factor[2] = {1.f, 1.f};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int tok = (s ? a.tq1 : 0) + my_tok;
        if (whole && (row & 1) && in_tile && tok < w.tokens && (dual || s == 0)) factor[s] = a.gate[(t_item + tok) * a.h + pair];
      }
      if (!wait_bar(sh, sh.bar(B_ORDY), it & 1, a.status, 0x8202)) ok = false;
      tc_fence_after();
      float* lx = sh.lx();
#pragma unroll
      for (int s = 0; s < 2; ++s) lx[(s * 2 + wg) * 128 + row] = l_half[s];
      if (named_red_or_256(!ok || *sh.abort_flag())) {
        ok = false;
        break;
      }
      const int64_t part = static_cast<int64_t>(2 * w.number() + (w.begins() ? 1 : 0)) * a.rows;
#pragma unroll 1
      for (int s = 0; s < (dual ? 2 : 1); ++s) {
        const int tok = (s ? a.tq1 : 0) + my_tok;
        const bool valid = in_tile && tok < w.tokens;
        // one Q tile: turn B has the odd key tiles, where there are any
        const bool join = !dual && steps > 1;
        float l = lx[s * 256 + row] + lx[s * 256 + 128 + row];
        float m = l == 0.f ? -INFINITY : (s ? m_run[1] : m_run[0]);
        float fa = 1.f, fb = 0.f;
        if (join) {
          const float lb = lx[256 + row] + lx[256 + 128 + row], mb = lb == 0.f ? -INFINITY : m_run[1];
          const float mm = fmaxf(m, mb), base = mm == -INFINITY ? 0.f : mm;
          fa = exp2f(m - base);
          fb = exp2f(mb - base);
          l = l * fa + lb * fb;
          m = mm;
        }
        const float coef = (s ? factor[1] : factor[0]) / l;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.ptr) + (t_item + tok) * a.out.st + pair * a.out.sh + wg * (D / 2);
        // the parts' rows lie side by side, four features each: a warp writes 512 bytes on end
        float* po = a.part_o + part * D + (s * 128 + row) * a.part_row + wg * (D / 8) * a.part_group;
        const uint32_t t_o = tmem + lane_off + 256 + s * 128 + wg * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          tmem_ld32(t_o + c * 32, o);
          if (join) {
            uint32_t ob[32];
            tmem_ld32(t_o + 128 + c * 32, ob);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * fa + __uint_as_float(ob[e]) * fb);
          } else {
            tmem_ld_wait();
          }
          if (whole) {
            // rows 2p and 2p + 1 are neighbouring lanes: each keeps half of the
            // columns and takes the other's share of them.  The products are
            // rounded apart, so that equal heads cancel with gate 1.
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float lo = __fmul_rn(__uint_as_float(o[e]), coef), hi = __fmul_rn(__uint_as_float(o[16 + e]), coef);
              const float got = __shfl_xor_sync(0xffffffffu, row & 1 ? lo : hi, 1);
              y[e] = row & 1 ? __fsub_rn(got, hi) : __fsub_rn(lo, got);
            }
            if (valid) {
              uint4 v[2];
              uint32_t* u = reinterpret_cast<uint32_t*>(v);
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
              uint4* dst = reinterpret_cast<uint4*>(out + c * 32 + (row & 1) * 16);
              dst[0] = v[0];
              dst[1] = v[1];
            }
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(po + (c * 8 + e) * a.part_group) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (!whole && valid && wg == 0)
          *reinterpret_cast<float2*>(a.part_ml + (part + s * 128 + row) * 2) = make_float2(m, l);
      }
      if (!w.begins() && w.ends()) desc.flags |= kPagedEnds;
      if (w.begins() && !w.ends()) desc = PagedDesc{desc.flags | kPagedOpen, w.t0 + w.i * a.tq, w.tokens, w.g};
      tc_fence_before();
    }
    for (; done < kTurns; ++done) {
      if (threadIdx.x == 0) a.desc[done * gridDim.x + blockIdx.x] = ok ? desc : PagedDesc{0, 0, 0, 0};
      desc = PagedDesc{0, 0, 0, 0};
    }
    if (!synced) cudaGridDependencySynchronize();  // the merge counts on the gate's end
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D, int kTurns>
cudaError_t launch_d(const PagedArgs& a, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  const da_paged_cache& c = a.cache;
  if (!encode_queries(&tq, a, a.tq1) || !encode_pages(&tk, c.k_pages, c, a.box) || !encode_pages(&tv, c.v_pages, c, a.box))
    return cudaErrorInvalidValue;
  static OncePerDevice once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(paged_fwd_kernel<D, kTurns>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_ahead(paged_fwd_kernel<D, kTurns>, dim3(a.grid), dim3(kThreads), kSmemBytes, s, a.after_gate, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (a.turns > 1)
    e = a.cache.d == 128 ? launch_d<128, kPagedMaxTurns>(a, s) : launch_d<64, kPagedMaxTurns>(a, s);
  else
    e = a.cache.d == 128 ? launch_d<128, 1>(a, s) : launch_d<64, 1>(a, s);
  return e == cudaSuccess ? launch_paged_merge(a, s) : e;
}

}  // namespace da
