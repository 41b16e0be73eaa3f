// paged.cuh — how the attention over a paged cache shares its work, for the
// kernels that do it (paged_fwd.cu) and the one that joins their parts
// (paged_merge.cu).
//
// The work is tiles of 128 keys for items: up to `tq` new tokens of one sequence
// with all G query heads of one KV head.  A tile is a unit of work, and an item by
// itself (its queries, its end) is a few more, before its first tile: without that
// the CTA with the first items of a long prompt, of one tile each, would be the
// last (8192 of 8192 tokens, 64 query heads: 843 us, 724 with it).  The units of a
// call form a line, (sequence, KV head, item, key tile) in this order, and share c
// of C is its c-th equal piece, wherever that begins and ends.  So a batch of any
// lengths loads the SMs evenly, whether it is one long sequence or many short
// ones, and only the items that a share's end cuts are left to be joined: at most
// C - 1, whatever the batch.  A share has at most two such parts, the rest of an
// item that an earlier one began (slot 2c) and the beginning of one that a later
// one ends (slot 2c + 1); an item that runs through whole shares has its middle
// parts in the slots 2c.
// There are as many shares as CTAs, or a few times as many where a prompt's keys
// and values do not fit L2 and are read for many items: the CTAs then take the
// first shares of all, the next ones, and so on, so that what is read at a time is
// a stretch of the line that fits (4 x 2048 tokens of 16384, 64 query and 8 KV
// heads: 2870 us with one share to a CTA, 2715 with four).
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tma.cuh"

namespace da {

constexpr int kPagedTile = 128;  // keys
// What an item costs beside its tiles, in tiles' time: about 4 us of 1.3 to 1.5 in
// the kernel for chunks (an item with one MMA tile waits longer for each of its
// steps than one with two has to compute, and its tiles count no less: 8 chunks of
// 1000 tokens among 40 single ones, up to 6000 keys: 242 us with two thirds, 215 so,
// 229 with four); in the one for few tokens 1 to 2 us of 0.8 to 1.1 at d 64 and 1.5
// at d 128, and as much again where a cut makes one item two (300 ragged sequences
// up to 500, d 128, 4 tokens: 115, 104, 102 us with 1, 2, 3; up to 1000, 128 of
// them, d 64: 62, 60, 62 with 2, 3, 4, single tokens 51, 45, 47 with 1, 3, 4).
constexpr int kItem = 3;
// A row's maximum is taken on a part's first tile and raised where a later tile's
// weights pass 2^kRaise: so 2^30 keys' sum to 2^54 at most, and values of up to 2^73
// stay within fp32 (2^64, as in the V2 forward, would leave 2^33).
constexpr int kRaise = 24;
constexpr float kPagedSumGuard = 1 << kRaise;
constexpr int64_t kTurnBytes = 48 << 20;  // of keys and values that one turn of the CTAs reads
constexpr int kTurnTiles = 128;           // of a share, where there are several turns
enum { kPagedOpen = 1, kPagedEnds = 2 };  // PagedDesc::flags

__device__ __forceinline__ bool paged_sequence_ok(const da_paged_cache& c, int t0, int t1, int L) {
  return t0 >= 0 && t0 <= t1 && t1 <= c.T && L >= t1 - t0 && L <= static_cast<int64_t>(c.max_pages) * c.page_size;
}

// sum over i < n of floor((a i + b) / m): the points of a lattice below a line.
// Whole parts of a / m and b / m are summed directly; what is left is counted along
// the other axis, which turns (a, m) into (m, a mod m), as in Euclid's algorithm
// (Graham, Knuth and Patashnik, Concrete Mathematics, 3.5: sums of floors).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t s = 0;
  while (n > 0) {
    s += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return s;
}

// Units of the first i items of a sequence with n new tokens, length L; all but its
// last item are whole.
__device__ __forceinline__ int64_t units_before(const PagedArgs& a, int i, int n, int L) {
  return floor_sum(i, kPagedTile, a.tq, static_cast<int64_t>(L) - n + a.tq + kPagedTile - 1) + static_cast<int64_t>(kItem) * i;
}

// A sequence of the batch as the arrays have it.
struct PagedSequence {
  int t0, t1, L;
  __device__ __forceinline__ void load(const da_paged_cache& c, int b) {
    t0 = c.cu_seqlens[b];
    t1 = c.cu_seqlens[b + 1];
    L = c.seqlens[b];
  }
};

// Its units for one KV head, 0 if it is out of bounds (then *bad).
__device__ __forceinline__ int64_t sequence_units(const PagedArgs& a, const PagedSequence& s, bool* bad) {
  if (!paged_sequence_ok(a.cache, s.t0, s.t1, s.L)) {
    *bad = true;
    return 0;
  }
  const int n = s.t1 - s.t0;
  if (n == 0) return 0;
  const int before = n <= a.tq ? 0 : (n - 1) / a.tq;  // items before the last
  const int64_t last = (static_cast<int64_t>(s.L) + kPagedTile - 1) / kPagedTile + kItem;
  return before ? units_before(a, before, n, s.L) + last : last;
}

// x / y, in 32 bits where that will do (a 64-bit division takes some 100 instructions)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// A CTA's shares: where each begins and how long it is.
struct PagedShare {
  int b, g, i;
  int from;       // its first unit in that item
  int64_t units;
};
template <int kTurns>  // the most that a CTA may have
struct PagedShares {
  int count;  // of this CTA; its k-th is share k * gridDim.x + blockIdx.x
  int bad;    // some sequence is out of bounds
  PagedShare share[kTurns];
};

// Fills *out (shared memory); called by all kThreads of a block, with sequence
// threadIdx.x (where there is one) in `mine`: fetched at the kernel's start, since
// the rest waits for it.
template <int kThreads, int kTurns>
__device__ void paged_share(const PagedArgs& a, const PagedSequence& mine, PagedShares<kTurns>* out) {
  static_assert(kThreads % 32 == 0, "whole warps");
  constexpr int kW = kThreads / 32;
  __shared__ int64_t sums[kW], lengths[kW];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.cache.B;
  bool bad = false;
  // inclusive sums over the warp's sequences, and each round's over the warps:
  // the first round's stay in registers, which for kThreads sequences are all
  int64_t per = tid < B ? sequence_units(a, mine, &bad) : 0;
  int64_t incl = per * a.cache.h_kv, rest = 0, keys = per ? mine.L : 0;
  for (int b = tid + kThreads; b < B; b += kThreads) {
    PagedSequence s;
    s.load(a.cache, b);
    const int64_t u = sequence_units(a, s, &bad);
    rest += u * a.cache.h_kv;
    keys += u ? s.L : 0;
  }
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if constexpr (kTurns > 1) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) keys += __shfl_xor_sync(0xffffffffu, keys, o);
  }
  if (B > kThreads) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  }
  if (lane == 31) {
    sums[warp] = incl;
    if constexpr (kTurns > 1) lengths[warp] = keys;
  }
  const bool any_bad = __syncthreads_or(bad);
  int64_t before = incl - per * a.cache.h_kv, total = 0;
  keys = 0;
#pragma unroll
  for (int v = 0; v < kW; ++v) {
    if (v < warp) before += sums[v];
    total += sums[v];
    if constexpr (kTurns > 1) keys += lengths[v];
  }
  int64_t base = total;  // of the first round
  if (B > kThreads) {
    __syncthreads();
    if (lane == 0) sums[warp] = rest;
    __syncthreads();
    for (int v = 0; v < kW; ++v) total += sums[v];
  }
  // turns of the CTAs: a stretch of the line reads about kTurnBytes of keys and
  // values, and a share is long enough to outweigh its two cut items
  int turns = 1;
  if constexpr (kTurns > 1) {
    const int64_t by_bytes = (keys * a.cache.h_kv * a.cache.d * 4) / kTurnBytes;
    const int64_t by_units = quotient(total, static_cast<int64_t>(gridDim.x) * kTurnTiles);
    const int64_t t = by_bytes < by_units ? by_bytes : by_units;
    turns = static_cast<int>(t < 1 ? 1 : t < kTurns ? t : kTurns);
  }
  // equal shares, the first `more` of them one unit longer; none is empty between
  // others, so that an item's parts follow each other without a gap
  const int64_t all = static_cast<int64_t>(turns) * gridDim.x, shares = total < 1 ? 1 : total < all ? total : all;
  const int64_t each = quotient(total, shares), more = total - each * shares;
  auto begin = [&](int64_t c) { return c * each + (c < more ? c : more); };
  auto length = [&](int64_t c) { return c < shares ? each + (c < more) : 0; };
  if (tid == 0) {
    out->count = turns;
    out->bad = any_bad;
    for (int k = 0; k < turns; ++k) out->share[k].units = length(static_cast<int64_t>(k) * gridDim.x + blockIdx.x);
  }
  PagedSequence s = mine;
  for (int r = 0;;) {
    const int64_t w = per * a.cache.h_kv;
    for (int k = 0; k < turns; ++k) {
      const int64_t c = static_cast<int64_t>(k) * gridDim.x + blockIdx.x, u0 = begin(c);
      if (length(c) == 0 || u0 < before || u0 >= before + w) continue;
      const int n = s.t1 - s.t0;
      int64_t off = u0 - before;
      const int g = static_cast<int>(quotient(off, per));
      off -= g * per;
      int lo = 0, hi = (n + a.tq - 1) / a.tq;  // the item: the last that begins at or before off
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (units_before(a, mid, n, s.L) <= off)
          lo = mid;
        else
          hi = mid;
      }
      out->share[k].b = r + tid;
      out->share[k].g = g;
      out->share[k].i = lo;
      out->share[k].from = static_cast<int>(off - (lo ? units_before(a, lo, n, s.L) : 0));
    }
    r += kThreads;
    if (r >= B || begin(static_cast<int64_t>(turns - 1) * gridDim.x + blockIdx.x) < base) break;
    // the next kThreads sequences
    per = 0;
    if (r + tid < B) {
      s.load(a.cache, r + tid);
      per = sequence_units(a, s, &bad);
    }
    incl = per * a.cache.h_kv;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();  // sums has been read
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    before = base + incl - per * a.cache.h_kv;
    for (int v = 0; v < kW; ++v) {
      if (v < warp) before += sums[v];
      base += sums[v];
    }
  }
  __syncthreads();
}

// A CTA's way along its shares, part by part; every warp walks by itself.
template <int kTurns>
struct PagedWalk {
  const PagedArgs& a;
  const PagedShares<kTurns>& s;
  int k;                // the share, of this CTA's
  int b, g, i, j;       // the part's item and first key tile
  int t0, n, L;         // the sequence
  int tokens, tiles, j1;  // the item's tokens and key tiles; the part ends before tile j1
  __device__ __forceinline__ PagedWalk(const PagedArgs& a_, const PagedShares<kTurns>& s_) : a(a_), s(s_), k(0) { share(); }
  // the share's number, of all
  __device__ __forceinline__ int number() const { return (kTurns > 1 ? k * static_cast<int>(gridDim.x) : 0) + static_cast<int>(blockIdx.x); }
  __device__ __forceinline__ bool more() const { return j < j1; }
  __device__ __forceinline__ bool begins() const { return j == 0; }
  __device__ __forceinline__ bool ends() const { return j1 == tiles; }
  // position of the item's first token
  __device__ __forceinline__ int first_position() const { return L - n + i * a.tq; }
  __device__ __forceinline__ void next() {
    advance();
    find();
  }

 private:
  int64_t left;  // units that are left of the share, this part's counted in
  int from, end;  // this part's units in the item (at most 2^23 tiles)
  // to the first part with a tile, in this share or the next; none: j = j1
  __device__ __forceinline__ void find() {
    while (true) {
      if (left <= 0) {
        if (kTurns == 1 || k + 1 >= s.count) {
          j = j1 = 0;
          return;
        }
        ++k;
        start();
        continue;
      }
      item();
      if (j < j1) return;
      advance();
    }
  }
  __device__ __forceinline__ void advance() {
    left -= end - from;
    from = 0;
    if (left <= 0) return;
    if ((i + 1) * a.tq < n) {
      ++i;
    } else {
      i = 0;
      if (++g == a.cache.h_kv) {
        g = 0;
        ++b;
        sequence();
      }
    }
  }
  __device__ __forceinline__ void share() {
    j = j1 = 0;
    start();
    find();
  }
  __device__ __forceinline__ void start() {
    const PagedShare& x = s.share[k];
    left = x.units;
    if (left <= 0) return;
    b = x.b;
    g = x.g;
    i = x.i;
    from = x.from;
    sequence();
  }
  __device__ __forceinline__ void sequence() {
    for (;; ++b) {  // there is one with work, since units are left
      t0 = a.cache.cu_seqlens[b];
      const int t1 = a.cache.cu_seqlens[b + 1];
      L = a.cache.seqlens[b];
      n = t1 - t0;
      if (b >= a.cache.B - 1 || (n > 0 && paged_sequence_ok(a.cache, t0, t1, L))) break;
    }
  }
  __device__ __forceinline__ void item() {
    tokens = min(a.tq, n - i * a.tq);
    tiles = (first_position() + tokens + kPagedTile - 1) / kPagedTile;
    const int all = tiles + kItem;
    end = left < all - from ? from + static_cast<int>(left) : all;
    j = max(from - kItem, 0);
    j1 = max(end - kItem, 0);
  }
};

// ------------------------------------------------------- tiles of pages ----
// A tile of 128 keys (or values) of a KV head in shared memory: groups of 8 rows,
// in each group D / 64 atoms of 8 rows x 128 bytes (64 features, 128-byte
// swizzle).  So any number of rows that is a multiple of 8 is one contiguous
// piece with all features, and a page's share of a tile is one TMA copy: the
// tensor map's dimensions are (64 features, 8 rows, blocks of 64 features counted
// through all heads, groups of 8 rows, pages).  Copies of 4 KB (two of 2 KB each
// in a layout with a box per 64 features) are what a page of 16 leaves.
// As an MMA operand with the features along K the groups are (D / 64) KB apart;
// with the features along M or N so are the groups along K, and the 64-feature
// blocks 1 KB.
template <int D>
struct KeyTile {
  static constexpr int kNB = D / 64;
  static constexpr int kGroup = kNB * 1024;
  static constexpr int kBytes = 16 * kGroup;
  static constexpr uint32_t kHi = sdesc_hi(kGroup);
  // descriptor units (16 bytes) to K step kk (16 features or 16 keys)
  static constexpr __device__ uint32_t feature_step(int kk) { return ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4; }
  static constexpr __device__ uint32_t key_step(int kk) { return kk * 2 * kGroup >> 4; }
  static __device__ uint32_t row(int r) { return (r >> 3) * kGroup + (r & 7) * 128; }
};

inline bool encode_pages(CUtensorMap* map, const da_t4& t, const da_paged_cache& c, int box) {
  const int64_t dims[5] = {64, 8, c.h_kv > 1 ? (c.h_kv - 1) * (t.sh / 64) + c.d / 64 : c.d / 64, c.page_size / 8, c.n_pages};
  const int64_t strides[4] = {t.sn, 64, 8 * t.sn, t.sb};
  const int boxes[5] = {64, 8, c.d / 64, box / 8, 1};
  return encode_tmap_bf16_box(map, t.ptr, 5, dims, strides, boxes);
}

// Queries: boxes of 64 features, all heads of a KV head, `tokens` tokens.
inline bool encode_queries(CUtensorMap* map, const PagedArgs& a, int tokens) {
  const int64_t dims[3] = {a.cache.d, 2 * a.h, a.cache.T}, strides[2] = {a.q.sh, a.q.st};
  const int boxes[3] = {64, a.G, tokens};
  return encode_tmap_bf16_box(map, a.q.ptr, 3, dims, strides, boxes);
}

// A producer lane's copies: lanes 0 .. 128 / box - 1 each look up and copy `box`
// rows of every tile, from the page that the block table names.  A page that is
// none reads as zeros: it is taken to be the one behind the last.
struct PageCopies {
  const PagedArgs& a;
  int row0, k_block, v_block;  // first row of this lane's copies; 64-feature blocks per head
  bool mine;
  __device__ __forceinline__ PageCopies(const PagedArgs& a_, int lane) : a(a_) {
    row0 = lane * a.box;
    mine = row0 < kPagedTile;
    k_block = static_cast<int>(a.cache.k_pages.sh / 64);
    v_block = static_cast<int>(a.cache.v_pages.sh / 64);
  }
  // whether tile j's copy holds any of a sequence's L keys
  __device__ __forceinline__ bool used(int L, int j) const { return mine && j * kPagedTile + row0 < L; }
  // its entry in the block table (`page` looks at it: what it waits for is the load)
  __device__ __forceinline__ int entry(int b, int L, int j) const {
    if (!used(L, j)) return 0;
    return a.cache.block_table[static_cast<int64_t>(b) * a.cache.max_pages + (j * kPagedTile + row0) / a.cache.page_size];
  }
  __device__ __forceinline__ int page(int entry, int L, int j) const {
    const bool in = entry >= 0 && entry < a.cache.n_pages;
    if (used(L, j) && in) return entry;
    if (!in) record_status(a.status, DA_ERR_BOUNDS, 0x0F02);
    return a.cache.n_pages;
  }
  __device__ __forceinline__ int group(int j) const { return (j * kPagedTile + row0) % a.cache.page_size / 8; }
};

// A block's way where some sequence is out of bounds: the outputs of those, where
// their rows are within the array, are zeros, all threads of the grid sharing them.
// Where the offsets fall somewhere the rows of two sequences could be the same: no
// sequence is taken then, and all rows are zeros.  A call, since its registers would
// be the kernels' (8192 of 8192 tokens: 716 us, 744 with it in line).
template <int kTurns>
__device__ __noinline__ void paged_out_of_bounds(const PagedArgs& a, PagedShares<kTurns>* shares) {
  const da_paged_cache& c = a.cache;
  const int per = a.h * c.d / 8;
  auto zero = [&](int64_t row, int64_t rows, int64_t first, int64_t step) {
    for (int64_t x = first; x < rows * per; x += step) {
      const int64_t t = row + x / per;
      const int r = static_cast<int>(x % per);
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out.ptr) + t * a.out.st + r / (c.d / 8) * a.out.sh + r % (c.d / 8) * 8;
      *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
    }
  };
  if (threadIdx.x == 0) record_status(a.status, DA_ERR_BOUNDS, 0x0F01);
  bool falls = false;
  for (int b = threadIdx.x; b < c.B; b += blockDim.x) falls |= c.cu_seqlens[b + 1] < c.cu_seqlens[b];
  if (__syncthreads_or(falls)) {
    for (int k = threadIdx.x; k < kTurns; k += blockDim.x) shares->share[k].units = 0;
    zero(0, c.T, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, static_cast<int64_t>(gridDim.x) * blockDim.x);
    return;
  }
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    const int t0 = c.cu_seqlens[b], t1 = c.cu_seqlens[b + 1];
    if (paged_sequence_ok(c, t0, t1, c.seqlens[b])) continue;
    const int64_t lo = max(t0, 0);  // (in 64 bits: t1 may be any number)
    zero(lo, min(t1, c.T) - lo, threadIdx.x, blockDim.x);
  }
}

}  // namespace da
