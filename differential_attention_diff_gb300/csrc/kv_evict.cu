// kv_evict.cu — eviction by gathered weight: which slots of each (sequence,
// KV head) stay, and the rows that move into the slots they leave.
//
// Every slot has a 32-bit rank: all ones for a protected slot, else an
// order-preserving image of its weight.  Select finds the rank of the m-th
// highest slot by its digits, eleven bits at a time from the top: a histogram
// of the digit over the slots that match the digits so far, and the bin that
// the m-th falls into.  Two digits (sign, exponent and 13 bits of mantissa)
// mostly leave one slot in that bin, and the search ends there.  Slots above
// that rank stay, and of those at it the lowest ones until m stay.  Each
// 32-slot word's answer is kept as a mask; the slots below m that go
// (destinations) and the slots at or above m that stay (sources) are listed
// from the masks, a word per lane, and paired in ascending order.
//
// A head's slots are spread over a cluster of CTAs, each holding its slice's
// ranks in shared memory, so weights and positions are read once; histograms
// and counts are summed over distributed shared memory.  One launch serves
// few long heads and many short ones: the cluster's size is chosen so that
// the GPU is filled (see launch_kv_evict).
//
// Move: rows from sources to destinations, 16 bytes per thread.  Sources lie
// at or above m and destinations below it, so no order is needed, and only as
// many rows move as there are holes, fewer than a compaction in order moves.
#include <cooperative_groups.h>

#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace da {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kDigit = 11;        // bits looked at together
constexpr int kBins = 1 << kDigit;
constexpr int kMaxRanks = 49152;  // of a slice kept in shared memory (192 KB); those behind are read again
constexpr int kMaxSelectSmem = 208 * 1024;  // ranks and masks: slices up to 131,072 slots, kEvictMaxSlots in all
constexpr int kMoveThreads = 256;

// Rank of slot j: protected, then NaN, then weights in ascending order (-0 as 0).
__device__ __forceinline__ uint32_t rank_of(float w, int pos, int sinks, int recent_from) {
  if (pos < sinks || pos >= recent_from) return 0xffffffffu;
  w += 0.f;
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int T>
struct Shared {
  uint32_t hist[2][kBins];  // this slice's histogram, read by the cluster; two, so that one barrier a digit suffices
  int counts[3];            // this slice's ties, destinations, sources
  int warp_counts[3][T / 32];
  int digit, above, in_bin;
};

// Whether the array that the new lengths go to is read by the heads.
__host__ __device__ inline bool lengths_read(const EvictArgs& a) {
  return a.p.seqlens_out == a.p.seqlens || a.p.seqlens_out == a.p.next_position;
}

// A barrier over the cluster in two halves: all threads arrive, and wait later
// (not as whole warps: the loops before end at different times for each thread).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Move n rows of a head from slots src[i] to dst[i], 16 bytes per thread and
// step, four steps in flight, and the slots' weights and positions with them.
// Thread x0 of `step`.
__device__ void move_rows(const EvictArgs& a, int unit, const int* dst, const int* src, int n, unsigned x0, unsigned step) {
  const int b = unit / a.p.h_kv, g = unit % a.p.h_kv;
  for (int k = 0; k < a.p.n_rows; ++k) {
    const unsigned chunks = a.p.row_bytes[k] / 16, total = n * chunks;
    uint8_t* rows = static_cast<uint8_t*>(a.p.rows[k].ptr) + b * a.p.rows[k].sb + g * a.p.rows[k].sh;
    for (unsigned x = x0; x < total; x += 4 * step) {
      uint4 v[4];
      unsigned at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const unsigned y = x + u * step;
        if (y < total) {
          at[u] = y / chunks;
          v[u] = __ldcs(reinterpret_cast<const uint4*>(rows + src[at[u]] * a.p.rows[k].sn + (y - at[u] * chunks) * 16));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const unsigned y = x + u * step;
        if (y < total)
          *reinterpret_cast<uint4*>(rows + dst[at[u]] * a.p.rows[k].sn + (y - at[u] * chunks) * 16) = v[u];
      }
    }
  }
  const int64_t base = static_cast<int64_t>(unit) * a.p.L_max;
  for (unsigned i = x0; i < static_cast<unsigned>(n); i += step) {
    const int t = dst[i], f = src[i];
    a.p.weights_out[base + t] = a.p.weights_in[base + f];
    if (a.p.positions_out) a.p.positions_out[base + t] = a.p.positions_in ? a.p.positions_in[base + f] : f;
  }
}

// T threads; kAll: every slice fits in `cached` ranks; kMove: a head is one
// CTA's, which also moves the rows (from lists that take the ranks' place) and
// writes the new length.  Where other heads read that in the same place, the
// heads of a sequence are a cluster and it is written behind a barrier, if
// `lengths`, or by a kernel of its own.
template <int T, bool kAll, bool kMove>
__global__ void __launch_bounds__(T, kMove ? 1536 / T : 2048 / T) evict_select_kernel(EvictArgs a, int cached, bool lengths) {
  constexpr int kThreads = T, kWarps = T / 32;
  extern __shared__ __align__(16) uint32_t ranks[];  // and behind them the masks
  __shared__ Shared<T> sh;
  cg::cluster_group cluster = cg::this_cluster();
  // with kMove a cluster is the heads of a sequence instead, if `lengths`
  const int cs = kMove ? 1 : static_cast<int>(cluster.num_blocks()), part = kMove ? 0 : static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / cs, b = unit / a.p.h_kv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t base = static_cast<int64_t>(unit) * a.p.L_max;
  const int L = a.p.seqlens ? a.p.seqlens[b] : a.p.L_max;
  const bool bad = L < 0 || L > a.p.L_max;
  const int m = bad ? L : min(L, a.p.keep);
  if (part == 0 && tid == 0) {
    if (bad) record_status(a.status, DA_ERR_BOUNDS, 0x4B03);
    if (unit % a.p.h_kv == 0) {
      a.new_len[b] = m;
      if (kMove && !lengths && !lengths_read(a)) a.p.seqlens_out[b] = m;
    }
  }
  const float* w_in = a.p.weights_in + base;
  float* w_out = a.p.weights_out + base;
  const int* p_in = a.p.positions_in ? a.p.positions_in + base : nullptr;
  int* p_out = a.p.positions_out ? a.p.positions_out + base : nullptr;
  const bool copy_w = w_out != w_in, copy_p = p_out != nullptr && p_out != p_in;
  if (bad || L <= a.p.keep) {  // the whole cluster leaves
    if (part == 0 && tid == 0) a.n_moves[unit] = 0;
    if (!bad)
      for (int j = part * kThreads + tid; j < L; j += cs * kThreads) {
        if (copy_w) w_out[j] = w_in[j];
        if (copy_p) p_out[j] = p_in ? p_in[j] : j;
      }
    if (kMove && lengths) {
      cluster_arrive();
      cluster_wait();
      if (tid == 0 && unit % a.p.h_kv == 0) a.p.seqlens_out[b] = m;
    }
    return;
  }
  const int end = a.p.next_position ? a.p.next_position[b] : L;
  const int recent_from = end >= INT_MIN + a.p.recent ? end - a.p.recent : INT_MIN;
  // this CTA has read the length (which may be the next position's array too)
  if (kMove && lengths) cluster_arrive();
  const bool alone = cs == 1;
  auto sync_all = [&]() {
    if (alone)
      __syncthreads();
    else
      cluster.sync();
  };
  const int slice = ((L + cs - 1) / cs + 31) / 32 * 32;
  const int j0 = min(L, part * slice), j1 = min(L, j0 + slice);
  auto read_rank = [&](int j) { return rank_of(w_in[j], p_in ? p_in[j] : j, a.p.sinks, recent_from); };
  auto rank = [&](int j) { return kAll || j - j0 < cached ? ranks[j - j0] : read_rank(j); };
  for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(sh.hist[0])[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  // Read the slots; their first digit is counted on the way, and what lies
  // below m is copied whether it stays or not: the slots that go are written
  // again when their successors move in.  Four neighbouring slots per access
  // where the arrays allow it (L_max a multiple of 4): a quarter of the address
  // arithmetic, which is most of this pass.
  auto count_digit = [&](uint32_t r) { atomicAdd(&sh.hist[0][r >> (32 - kDigit)], 1u); };
  auto quad_ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool quads = kAll && quad_ok(w_in) && quad_ok(w_out) && quad_ok(p_in) && quad_ok(p_out);
  const int full = quads ? j0 + (j1 - j0) / 4 * 4 : j0;  // slots up to here go by fours
#pragma unroll 2
  for (int j = j0 + 4 * tid; j < full; j += 4 * kThreads) {
    const float4 w = *reinterpret_cast<const float4*>(w_in + j);
    const int4 p = p_in ? *reinterpret_cast<const int4*>(p_in + j) : make_int4(j, j + 1, j + 2, j + 3);
    const uint4 r = make_uint4(rank_of(w.x, p.x, a.p.sinks, recent_from), rank_of(w.y, p.y, a.p.sinks, recent_from),
                               rank_of(w.z, p.z, a.p.sinks, recent_from), rank_of(w.w, p.w, a.p.sinks, recent_from));
    *reinterpret_cast<uint4*>(ranks + (j - j0)) = r;
    count_digit(r.x);
    count_digit(r.y);
    count_digit(r.z);
    count_digit(r.w);
    if (j + 3 < m) {
      if (copy_w) *reinterpret_cast<float4*>(w_out + j) = w;
      if (copy_p) *reinterpret_cast<int4*>(p_out + j) = p;
    } else {
      const float ws[4] = {w.x, w.y, w.z, w.w};
      const int ps[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (copy_w && j + k < m) w_out[j + k] = ws[k];
        if (copy_p && j + k < m) p_out[j + k] = ps[k];
      }
    }
  }
  for (int i0 = full + tid; i0 < j1; i0 += 4 * kThreads) {
    float w[4];
    int p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = i0 + k * kThreads;
      w[k] = j < j1 ? w_in[j] : 0.f;
      p[k] = j < j1 && p_in ? p_in[j] : j;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = i0 + k * kThreads;
      if (j < j1) {
        const uint32_t r = rank_of(w[k], p[k], a.p.sinks, recent_from);
        if (kAll || j - j0 < cached) ranks[j - j0] = r;
        count_digit(r);
        if (copy_w && j < m) w_out[j] = w[k];
        if (copy_p && j < m) p_out[j] = p[k];
      }
    }
  }

  // ---- the rank of the m-th highest slot ----
  uint32_t prefix = 0;  // its digits so far
  int need = m;         // how many of the slots that match them stay
  int shift = 32;       // bits not looked at yet
  bool all = false;     // every slot that matches stays
  for (int round = 0; shift > 0 && !all; ++round) {
    const int bits = min(shift, kDigit), above_shift = shift;
    shift -= bits;
    uint32_t* hist = sh.hist[round & 1];
    if (round) {
      for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      auto count = [&](uint32_t r) {
        if ((r >> above_shift) == prefix) atomicAdd(&hist[(r >> shift) & ((1u << bits) - 1)], 1u);
      };
      const int by_four = kAll ? j0 + (j1 - j0) / 4 * 4 : j0;
#pragma unroll 2
      for (int j = j0 + 4 * tid; j < by_four; j += 4 * kThreads) {
        const uint4 r = *reinterpret_cast<const uint4*>(ranks + (j - j0));
        count(r.x);
        count(r.y);
        count(r.z);
        count(r.w);
      }
      for (int j = by_four + tid; j < j1; j += kThreads) count(rank(j));
    }
    sync_all();
    constexpr int kMine = kBins / kThreads;  // neighbouring bins per thread
    int bin[kMine], up = 0;
#pragma unroll
    for (int k = 0; k < kMine; ++k) bin[k] = 0;
    for (int c = 0; c < cs; ++c) {
      const uint2* h = reinterpret_cast<const uint2*>(alone ? hist : cluster.map_shared_rank(hist, c)) + tid * (kMine / 2);
#pragma unroll
      for (int k = 0; k < kMine / 2; ++k) {
        const uint2 v = h[k];
        bin[2 * k] += v.x;
        bin[2 * k + 1] += v.y;
      }
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) up += bin[k];
    const int own = up;
    // slots in this thread's bins and those above: sums from the top
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_down_sync(0xffffffffu, up, o);
      if (lane + o < 32) up += y;
    }
    if (lane == 0) sh.warp_counts[0][warp] = up;
    __syncthreads();
    up += __reduce_add_sync(0xffffffffu, lane > warp && lane < kWarps ? sh.warp_counts[0][lane] : 0);
    if (up >= need && up - own < need) {  // one thread, and one of its bins
      int above = up - own;
#pragma unroll
      for (int k = kMine - 1; k >= 0; --k) {
        if (above < need && above + bin[k] >= need) {
          sh.digit = tid * kMine + k;
          sh.above = above;
          sh.in_bin = bin[k];
        }
        above += bin[k];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | static_cast<uint32_t>(sh.digit);
    need -= sh.above;
    all = sh.in_bin == need;
  }

  // ---- who stays, a mask per 32-slot word; each warp takes a run of words ----
  __syncthreads();
  uint32_t* masks = ranks + cached;
  const int words = (j1 - j0 + 31) / 32, w0 = words * warp / kWarps, w1 = words * (warp + 1) / kWarps;
  // numbers before this warp's run, from per-warp counts and the slices before
  auto before = [&](int k, int n) {
    if (lane == 0) sh.warp_counts[k][warp] = n;
    __syncthreads();
    const int c = lane < kWarps ? sh.warp_counts[k][lane] : 0;
    if (warp == 0) {
      const int all_warps = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) sh.counts[k] = all_warps;
    }
    return __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
  };
  auto slices = [&](int k, int n) {  // over the first n slices
    if (alone) return n ? sh.counts[k] : 0;
    int s = 0;
    for (int c = 0; c < n; ++c) s += cluster.map_shared_rank(&sh.counts[0], c)[k];
    return s;
  };
  int ties = 0;  // before this warp's run
  if (!all) {
    int n = 0;
#pragma unroll 4
    for (int w = w0; w < w1; ++w) {
      const int j = j0 + w * 32 + lane;
      n += __popc(__ballot_sync(0xffffffffu, j < j1 && (rank(j) >> shift) == prefix));
    }
    ties = before(0, n);
    sync_all();
    ties += slices(0, part);
  }
  int n_dst = 0, n_src = 0;
#pragma unroll 4
  for (int w = w0; w < w1; ++w) {
    const int j = j0 + w * 32 + lane;
    const uint32_t r = j < j1 ? rank(j) >> shift : 0u;
    bool stays = j < j1 && r >= prefix;
    if (!all) {
      const bool tie = stays && r == prefix;
      const unsigned t = __ballot_sync(0xffffffffu, tie);
      if (tie) stays = ties + __popc(t & ((1u << lane) - 1)) < need;
      ties += __popc(t);
    }
    const unsigned mask = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) masks[w] = mask;
  }
  __syncwarp();
  // a word per lane: its slots that go below m, and those that stay from m on
  auto split = [&](int w, uint32_t& d, uint32_t& s) {
    d = s = 0;
    if (w >= w1) return;
    const int first = j0 + w * 32;  // the word's slots below m, and those that exist
    const uint32_t low = m >= first + 32 ? ~0u : m > first ? (1u << (m - first)) - 1 : 0u;
    const uint32_t live = j1 >= first + 32 ? ~0u : (1u << (j1 - first)) - 1;
    d = ~masks[w] & low & live;
    s = masks[w] & ~low;
  };
  for (int w = w0 + lane; w - lane < w1; w += 32) {
    uint32_t d, s;
    split(w, d, s);
    n_dst += __popc(d);
    n_src += __popc(s);
  }
  n_dst = __reduce_add_sync(0xffffffffu, n_dst);
  n_src = __reduce_add_sync(0xffffffffu, n_src);
  n_dst = before(1, n_dst);
  n_src = before(2, n_src);
  sync_all();
  n_dst += slices(1, part);
  n_src += slices(2, part);
  // at most half of a head's slots move: both lists fit where its ranks were
  int* dst = kMove ? reinterpret_cast<int*>(ranks) : a.dst + static_cast<int64_t>(unit) * a.max_moves;
  int* src = kMove ? dst + cached / 2 : a.src + static_cast<int64_t>(unit) * a.max_moves;
  for (int w = w0 + lane; w - lane < w1; w += 32) {
    uint32_t d, s;
    split(w, d, s);
    int di = __popc(d), si = __popc(s);  // up to and with this lane's word
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, di, o), y = __shfl_up_sync(0xffffffffu, si, o);
      if (lane >= o) di += x, si += y;
    }
    const int td = __shfl_sync(0xffffffffu, di, 31), ts = __shfl_sync(0xffffffffu, si, 31);
    di += n_dst - __popc(d);
    si += n_src - __popc(s);
    n_dst += td;
    n_src += ts;
    const int first = j0 + w * 32;
    for (; d; d &= d - 1) dst[di++] = first + __ffs(d) - 1;
    for (; s; s &= s - 1) src[si++] = first + __ffs(s) - 1;
  }
  if constexpr (kMove) {
    __syncthreads();
    move_rows(a, unit, dst, src, sh.counts[1], tid, kThreads);
    if (lengths) {
      cluster_wait();
      if (tid == 0 && unit % a.p.h_kv == 0) a.p.seqlens_out[b] = m;
    }
  } else {
    if (part == 0 && tid == 0) a.n_moves[unit] = slices(1, cs);
    if (!alone) cluster.sync();  // no CTA leaves while another may still read its counts
  }
}

// Block (part of a head's moves, head).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, int blocks_per_unit) {
  cudaGridDependencySynchronize();  // the lists
  const int unit = blockIdx.x / blocks_per_unit, part = blockIdx.x % blocks_per_unit;
  if (part == 0 && unit % a.p.h_kv == 0 && threadIdx.x == 0) a.p.seqlens_out[unit / a.p.h_kv] = a.new_len[unit / a.p.h_kv];
  const int64_t list = static_cast<int64_t>(unit) * a.max_moves;
  move_rows(a, unit, a.dst + list, a.src + list, a.n_moves[unit], part * kMoveThreads + threadIdx.x,
            blocks_per_unit * kMoveThreads);
}

__global__ void __launch_bounds__(kMoveThreads) evict_lengths_kernel(EvictArgs a) {
  cudaGridDependencySynchronize();
  const int b = blockIdx.x * kMoveThreads + threadIdx.x;
  if (b < a.p.B) a.p.seqlens_out[b] = a.new_len[b];
}

template <int T, bool kAll, bool kMove = false>
cudaError_t launch_select(const EvictArgs& a, int cs, int cached, size_t smem, cudaStream_t s, bool lengths = false) {
  auto* kernel = evict_select_kernel<T, kAll, kMove>;
  static OncePerDevice once;
  const cudaError_t e = once.run(
      [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSelectSmem); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3(a.p.B * a.p.h_kv * cs);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = lengths ? a.p.h_kv : cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, cached, lengths);
}

}  // namespace

namespace {

struct Plan {
  int cs, per;  // CTAs per head, slots of each
  bool small;   // 256 threads instead of 1024
};
Plan plan_of(int64_t units, int L_max, int sms) {
  // Spread a head over a cluster while that leaves no SM two CTAs and each
  // still has 8192 slots (64 heads of 33000: 1, 2, 4, 8 CTAs took 32, 27, 33,
  // 68 us; 8 heads of 131072: 231, 112, 35, 31; 8 of 4097: 11.5 and, with 2,
  // 14.0); a slice that would pass kMaxRanks asks for more too.
  int cs = 1;
  while (cs < kMaxCluster && ((units * cs * 2 <= sms && L_max / cs > 8192) || L_max / cs > kMaxRanks)) cs *= 2;
  const int per = ((L_max + cs - 1) / cs + 31) / 32 * 32;
  // 1024 threads, but 256 for short heads that are many: their CTAs then share
  // an SM six or more at a time (512 heads of 4352: 32 us, 34 with 512 threads,
  // 41 with 1024; 128 of 8192: 46, 43, 41)
  return {cs, per, per <= 1024 || (per <= 6144 && units * cs > 2 * sms)};
}

}  // namespace

bool evict_moves_unlisted(int64_t units, int L_max, int sms) {
  const Plan p = plan_of(units, L_max, sms);
  return p.cs == 1 && p.small && units >= sms;
}

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s) {
  const int units = a.p.B * a.p.h_kv;
  const auto [cs, per, small] = plan_of(units, a.p.L_max, a.num_sms);
  const int cached = per < kMaxRanks ? per : kMaxRanks;
  const size_t smem = (static_cast<size_t>(cached) + per / 32) * sizeof(uint32_t);
  if (smem > kMaxSelectSmem) return cudaErrorInvalidValue;  // refused by the entry point before
  int64_t chunks = 0;
  for (int k = 0; k < a.p.n_rows; ++k) chunks += a.p.row_bytes[k] / 16;
  // Each CTA moves its own rows, which saves a launch and the wait for it,
  // unless there are many rows and many SMs without a head to share them with
  // (512 heads, 256 of 4352 slots moved: 29.4 us in two launches, 25.6 in one
  // and one for the lengths, 22.1 in one; 8 heads, 1 of 4097: 11.9 and 9.9; 128
  // heads, 2048 of 8192: 41.6 and 38.2; but 96 of them 33.0 and 34.2, 16 heads,
  // 1000 of 3000: 12.4 and 16.8).  Clusters of 1024-thread CTAs, one to an SM,
  // would leave SMs empty: those lengths get the launch.
  const int64_t idle = units < a.num_sms ? a.num_sms - units : 0;
  const bool own = small || (per <= 8192 && units <= a.num_sms);
  if (cs == 1 && own && a.max_moves * chunks * idle <= int64_t{12288} * a.num_sms) {
    const bool in_place = lengths_read(a), lengths = in_place && small && a.p.h_kv <= kMaxCluster;
    const cudaError_t e = small ? launch_select<256, true, true>(a, cs, cached, smem, s, lengths)
                                : launch_select<1024, true, true>(a, cs, cached, smem, s);
    if (e != cudaSuccess || !in_place || lengths) return e;
    return launch_ahead(evict_lengths_kernel, dim3((a.p.B + kMoveThreads - 1) / kMoveThreads), dim3(kMoveThreads), 0, s, true, a);
  }
  cudaError_t e = per > kMaxRanks ? launch_select<1024, false>(a, cs, cached, smem, s)
                  : small         ? launch_select<256, true>(a, cs, cached, smem, s)
                                  : launch_select<1024, true>(a, cs, cached, smem, s);
  if (e != cudaSuccess) return e;
  // enough blocks for the most rows that can move, 4 steps of a block each
  int64_t per_unit = (a.max_moves * chunks + 4 * kMoveThreads - 1) / (4 * kMoveThreads);
  const int64_t most = (16 * a.num_sms + units - 1) / units;  // and no more than fill the GPU twice
  per_unit = per_unit < 1 ? 1 : per_unit > most ? most : per_unit;
  return launch_ahead(evict_move_kernel, dim3(static_cast<unsigned>(units * per_unit)), dim3(kMoveThreads), 0, s, true, a,
                      static_cast<int>(per_unit));
}

}  // namespace da
