// kv_evict.cu — eviction by gathered weight: which slots of each (sequence,
// KV head) stay, and the rows that move into the slots they leave.
//
// Every slot has a 32-bit rank: all ones for a protected slot, else an
// order-preserving image of its weight.  Select finds the rank of the m-th
// highest slot by its digits, eight bits at a time from the top: a histogram
// of the digit over the slots that match the digits so far, and the bin that
// the m-th falls into.  Slots above that rank stay, and of those at it the
// lowest ones until m stay.  A pass in slot order then lists the slots below m
// that go (destinations) and the slots at or above m that stay (sources),
// paired in ascending order.
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

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kCopies = 8;        // of the histogram, by lane: weights crowd into few bins
constexpr int kMaxRanks = 49152;  // of a slice kept in shared memory (192 KB); those behind are read again
constexpr int kMoveThreads = 256;

// Rank of slot j: protected, then NaN, then weights in ascending order (-0 as 0).
__device__ __forceinline__ uint32_t rank_of(float w, int pos, int sinks, int64_t recent_from) {
  if (pos < sinks || pos >= recent_from) return 0xffffffffu;
  w += 0.f;
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Shared {
  uint32_t hist[256 * kCopies];
  int sums[2][256];  // this slice's histogram, for the cluster; two, so that one barrier a digit suffices
  int counts[3];     // this slice's ties, destinations, sources
  int warp_counts[3][kWarps];
  int digit, above;
};

__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a, int cached) {
  extern __shared__ uint32_t ranks[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / cs, b = unit / a.p.h_kv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t base = static_cast<int64_t>(unit) * a.p.L_max;
  const int L = a.p.seqlens ? a.p.seqlens[b] : a.p.L_max;
  const bool bad = L < 0 || L > a.p.L_max;
  const int m = bad ? L : min(L, a.p.keep);
  if (part == 0 && tid == 0) {
    if (bad) record_status(a.status, DA_ERR_BOUNDS, 0x4B03);
    if (unit % a.p.h_kv == 0) a.new_len[b] = m;
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
    return;
  }
  const int64_t recent_from = (a.p.next_position ? a.p.next_position[b] : L) - static_cast<int64_t>(a.p.recent);
  const int slice = ((L + cs - 1) / cs + 31) / 32 * 32;
  const int j0 = min(L, part * slice), j1 = min(L, j0 + slice);
  auto read_rank = [&](int j) { return rank_of(w_in[j], p_in ? p_in[j] : j, a.p.sinks, recent_from); };
  auto rank = [&](int j) { return j - j0 < cached ? ranks[j - j0] : read_rank(j); };
  {
    const int n = min(j1 - j0, cached);
    for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {  // four reads in flight
      float w[4];
      int p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kThreads;
        w[k] = i < n ? w_in[j0 + i] : 0.f;
        p[k] = i < n && p_in ? p_in[j0 + i] : j0 + i;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * kThreads < n) ranks[i0 + k * kThreads] = rank_of(w[k], p[k], a.p.sinks, recent_from);
    }
  }

  // ---- the rank of the m-th highest slot ----
  uint32_t prefix = 0;  // its digits so far
  int need = m;         // how many of the slots that match them stay
  int shift = 32;       // bits not looked at yet
  bool all = false;     // every slot that matches stays
  for (int round = 0; shift > 0 && !all; ++round) {
    shift -= 8;
    for (int i = tid; i < 256 * kCopies; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int j = j0 + tid; j < j1; j += kThreads) {
      const uint32_t r = rank(j);
      if (shift == 24 || (r >> (shift + 8)) == prefix) atomicAdd(&sh.hist[((r >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1u);
    }
    __syncthreads();
    static_assert(kThreads == 256, "one thread per bin");
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) mine += sh.hist[tid * kCopies + k];
    if (cs > 1) {
      sh.sums[round & 1][tid] = mine;
      cluster.sync();
      mine = 0;
      for (int c = 0; c < cs; ++c) mine += cluster.map_shared_rank(&sh.sums[round & 1][0], c)[tid];
    }
    // slots in the bins above this thread's: sums from the top
    const int bin_count = mine;
    int up = bin_count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_down_sync(0xffffffffu, up, o);
      if (lane + o < 32) up += y;
    }
    if (lane == 0) sh.warp_counts[0][warp] = up;
    __syncthreads();
    for (int w = warp + 1; w < kWarps; ++w) up += sh.warp_counts[0][w];
    if (up >= need && up - bin_count < need) {  // one bin
      sh.digit = tid;
      sh.above = up - bin_count;
      sh.counts[0] = bin_count;
    }
    __syncthreads();
    prefix = (prefix << 8) | static_cast<uint32_t>(sh.digit);
    need -= sh.above;
    all = sh.counts[0] == need;
    __syncthreads();
  }

  // ---- who stays, in slot order: each warp takes a run of 32-slot words ----
  const int words = (j1 - j0 + 31) / 32, w0 = words * warp / kWarps, w1 = words * (warp + 1) / kWarps;
  auto state = [&](int word, int ties_before, bool& stays, unsigned& tie) {
    const int j = j0 + word * 32 + lane;
    const uint32_t r = j < j1 ? rank(j) >> shift : 0u;
    const bool t = j < j1 && r == prefix;
    tie = __ballot_sync(0xffffffffu, t);
    stays = j < j1 && (r > prefix || (t && (all || ties_before + __popc(tie & ((1u << lane) - 1)) < need)));
    return j;
  };
  // numbers before this warp's run, from per-warp counts and the slices before
  auto before = [&](int k, int n) {
    if (lane == 0) sh.warp_counts[k][warp] = n;
    __syncthreads();
    if (tid == 0) {
      int s = 0;
      for (int w = 0; w < kWarps; ++w) s += sh.warp_counts[k][w];
      sh.counts[k] = s;
    }
    int s = 0;
    for (int w = 0; w < warp; ++w) s += sh.warp_counts[k][w];
    return s;
  };
  auto slices_before = [&](int k) {
    int s = 0;
    for (int c = 0; c < part; ++c) s += cluster.map_shared_rank(&sh.counts[0], c)[k];
    return s;
  };
  int ties = 0;
  bool stays;
  unsigned tie;
  if (!all) {
    int n = 0;
    for (int w = w0; w < w1; ++w) {
      state(w, 0, stays, tie);
      n += __popc(tie);
    }
    ties = before(0, n);
    cluster.sync();
    ties += slices_before(0);
  }
  int n_dst = 0, n_src = 0, seen = ties;
  for (int w = w0; w < w1; ++w) {
    const int j = state(w, seen, stays, tie);
    seen += __popc(tie);
    n_dst += __popc(__ballot_sync(0xffffffffu, j < j1 && j < m && !stays));
    n_src += __popc(__ballot_sync(0xffffffffu, j >= m && stays));
  }
  n_dst = before(1, n_dst);
  n_src = before(2, n_src);
  cluster.sync();
  n_dst += slices_before(1);
  n_src += slices_before(2);
  int* dst = a.dst + static_cast<int64_t>(unit) * a.max_moves;
  int* src = a.src + static_cast<int64_t>(unit) * a.max_moves;
  seen = ties;
  for (int w = w0; w < w1; ++w) {
    const int j = state(w, seen, stays, tie);
    seen += __popc(tie);
    const bool is_dst = j < j1 && j < m && !stays, is_src = j >= m && stays;
    const unsigned db = __ballot_sync(0xffffffffu, is_dst), sb = __ballot_sync(0xffffffffu, is_src);
    const unsigned low = (1u << lane) - 1;
    if (is_dst) dst[n_dst + __popc(db & low)] = j;
    if (is_src) src[n_src + __popc(sb & low)] = j;
    n_dst += __popc(db);
    n_src += __popc(sb);
    if (j < m && stays) {
      if (copy_w) w_out[j] = w_in[j];
      if (copy_p) p_out[j] = p_in ? p_in[j] : j;
    }
  }
  if (part == 0 && tid == 0) {
    int s = 0;
    for (int c = 0; c < cs; ++c) s += cluster.map_shared_rank(&sh.counts[0], c)[1];
    a.n_moves[unit] = s;
  }
  cluster.sync();  // no CTA leaves while another may still read its counts
}

// Block (part of a head's moves, head): 16 bytes per thread and step, four
// steps in flight; the moved slots' weights and positions with them.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, int blocks_per_unit) {
  cudaGridDependencySynchronize();  // the lists
  const int unit = blockIdx.x / blocks_per_unit, part = blockIdx.x % blocks_per_unit;
  const int b = unit / a.p.h_kv, g = unit % a.p.h_kv;
  if (part == 0 && g == 0 && threadIdx.x == 0) a.p.seqlens_out[b] = a.new_len[b];
  const int n = a.n_moves[unit];
  const int* dst = a.dst + static_cast<int64_t>(unit) * a.max_moves;
  const int* src = a.src + static_cast<int64_t>(unit) * a.max_moves;
  const unsigned step = blocks_per_unit * kMoveThreads, x0 = part * kMoveThreads + threadIdx.x;
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

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s) {
  const int units = a.p.B * a.p.h_kv;
  // Double the cluster while the CTAs are fewer than four per SM and each has
  // more than 2048 slots; a slice that would pass kMaxRanks asks for more too.
  int cs = 1;
  while (cs < kMaxCluster && ((static_cast<int64_t>(units) * cs * 2 <= 4 * a.num_sms && a.p.L_max / cs > 2048) ||
                              a.p.L_max / cs > kMaxRanks))
    cs *= 2;
  const int per = ((a.p.L_max + cs - 1) / cs + 31) / 32 * 32;
  const int cached = per < kMaxRanks ? per : kMaxRanks;
  const size_t smem = static_cast<size_t>(cached) * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxRanks * static_cast<int>(sizeof(uint32_t)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3(units * cs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cached);
  if (e != cudaSuccess) return e;
  // enough blocks for the most rows that can move, 4 steps of a block each
  int64_t chunks = 0;
  for (int k = 0; k < a.p.n_rows; ++k) chunks += a.p.row_bytes[k] / 16;
  int64_t per_unit = a.max_moves * chunks / (4 * kMoveThreads);
  const int64_t most = (16 * a.num_sms + units - 1) / units;  // and no more than fill the GPU twice
  per_unit = per_unit < 1 ? 1 : per_unit > most ? most : per_unit;
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * per_unit));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a, static_cast<int>(per_unit));
}

}  // namespace da
