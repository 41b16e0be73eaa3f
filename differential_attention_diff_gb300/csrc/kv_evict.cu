// kv_evict.cu — eviction by gathered weight: which slots of each (sequence,
// KV head) stay, and the rows that move into the slots they leave.
//
// Select (one CTA per head): every slot has a 32-bit rank, all ones for a
// protected slot, else an order-preserving image of its weight.  The rank of
// the keep-th highest slot is found bit by bit; slots above it stay, and of
// those at it the lowest ones until m stay.  A pass in slot order then lists
// the slots below m that go (destinations) and the slots at or above m that
// stay (sources), paired in ascending order.
// Move: rows from sources to destinations, 16 bytes per thread.  Sources lie
// at or above m and destinations below it, so no order is needed.
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kThreads = 1024;

// Rank of slot j: protected, then NaN, then weights in ascending order (-0 as 0).
__device__ __forceinline__ uint32_t rank_of(const EvictArgs& a, int64_t base, int j, int64_t recent_from) {
  const int pos = a.p.positions_in ? a.p.positions_in[base + j] : j;
  if (pos < a.p.sinks || pos >= recent_from) return 0xffffffffu;
  const float w = a.p.weights_in[base + j] + 0.f;
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
  const int unit = blockIdx.x, b = unit / a.p.h_kv, tid = threadIdx.x;
  const int64_t base = static_cast<int64_t>(unit) * a.p.L_max;
  const int L = a.p.seqlens ? a.p.seqlens[b] : a.p.L_max;
  const bool bad = L < 0 || L > a.p.L_max;
  const int m = bad ? L : min(L, a.p.keep);
  if (tid == 0) {
    if (bad) record_status(a.status, DA_ERR_BOUNDS, 0x4B03);
    if (unit % a.p.h_kv == 0) a.new_len[b] = m;
  }
  if (bad || L <= a.p.keep) {
    if (tid == 0) a.n_moves[unit] = 0;
    if (!bad)
      for (int j = tid; j < L; j += kThreads) {
        a.p.weights_out[base + j] = a.p.weights_in[base + j];
        if (a.p.positions_out) a.p.positions_out[base + j] = a.p.positions_in ? a.p.positions_in[base + j] : j;
      }
    return;
  }
  const int64_t recent_from = (a.p.next_position ? a.p.next_position[b] : L) - static_cast<int64_t>(a.p.recent);
  // the m-th highest rank, from its highest bit down
  uint32_t cut = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = cut | (1u << bit);
    int n = 0;
    for (int j = tid; j < L; j += kThreads) n += rank_of(a, base, j, recent_from) >= cand;
    __shared__ int total;
    if (tid == 0) total = 0;
    __syncthreads();
    atomicAdd(&total, n);
    __syncthreads();
    if (total >= m) cut = cand;
    __syncthreads();
  }
  __shared__ int above;
  if (tid == 0) above = 0;
  __syncthreads();
  {
    int n = 0;
    for (int j = tid; j < L; j += kThreads) n += rank_of(a, base, j, recent_from) > cut;
    atomicAdd(&above, n);
  }
  __syncthreads();
  const int ties = m - above;  // slots at the cut that stay, the lowest first
  // slots in order, one tile of kThreads at a time
  __shared__ int scan[3][kThreads / 32];
  int seen_ties = 0, seen_dst = 0, seen_src = 0;
  const int warp = tid >> 5, lane = tid & 31;
  int* dst = a.dst + static_cast<int64_t>(unit) * a.max_moves;
  int* src = a.src + static_cast<int64_t>(unit) * a.max_moves;
  for (int j0 = 0; j0 < L; j0 += kThreads) {
    const int j = j0 + tid;
    const uint32_t r = j < L ? rank_of(a, base, j, recent_from) : 0u;
    const bool tie = j < L && r == cut;
    const unsigned tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) scan[0][warp] = __popc(tb);
    __syncthreads();
    int before = seen_ties + __popc(tb & ((1u << lane) - 1));
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[0][w];
      seen_ties += scan[0][w];
    }
    const bool stays = j < L && (r > cut || (tie && before < ties));
    const bool is_dst = j < m && !stays, is_src = j >= m && stays;
    const unsigned db = __ballot_sync(0xffffffffu, is_dst), sb = __ballot_sync(0xffffffffu, is_src);
    if (lane == 0) scan[1][warp] = __popc(db), scan[2][warp] = __popc(sb);
    __syncthreads();
    int di = seen_dst + __popc(db & ((1u << lane) - 1)), si = seen_src + __popc(sb & ((1u << lane) - 1));
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) di += scan[1][w], si += scan[2][w];
      seen_dst += scan[1][w];
      seen_src += scan[2][w];
    }
    if (is_dst) dst[di] = j;
    if (is_src) src[si] = j;
    if (j < m && stays) {
      a.p.weights_out[base + j] = a.p.weights_in[base + j];
      if (a.p.positions_out) a.p.positions_out[base + j] = a.p.positions_in ? a.p.positions_in[base + j] : j;
    }
    __syncthreads();
  }
  if (tid == 0) a.n_moves[unit] = seen_dst;
  for (int i = tid; i < seen_dst; i += kThreads) {
    const int t = dst[i], f = src[i];
    a.p.weights_out[base + t] = a.p.weights_in[base + f];
    if (a.p.positions_out) a.p.positions_out[base + t] = a.p.positions_in ? a.p.positions_in[base + f] : f;
  }
}

// Block (chunk of a head's moves, head): 16 bytes per thread and step.
__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a, int blocks_per_unit) {
  const int unit = blockIdx.x / blocks_per_unit, part = blockIdx.x % blocks_per_unit;
  const int b = unit / a.p.h_kv, g = unit % a.p.h_kv;
  if (part == 0 && g == 0 && threadIdx.x == 0 && a.p.seqlens_out) a.p.seqlens_out[b] = a.new_len[b];
  const int n = a.n_moves[unit];
  const int* dst = a.dst + static_cast<int64_t>(unit) * a.max_moves;
  const int* src = a.src + static_cast<int64_t>(unit) * a.max_moves;
  for (int k = 0; k < a.p.n_rows; ++k) {
    const int chunks = a.p.row_bytes[k] / 16;
    uint8_t* rows = static_cast<uint8_t*>(a.p.rows[k].ptr) + b * a.p.rows[k].sb + g * a.p.rows[k].sh;
    const int64_t total = static_cast<int64_t>(n) * chunks;
    for (int64_t x = static_cast<int64_t>(part) * 256 + threadIdx.x; x < total; x += static_cast<int64_t>(blocks_per_unit) * 256) {
      const int i = static_cast<int>(x / chunks), c = static_cast<int>(x % chunks);
      *reinterpret_cast<uint4*>(rows + dst[i] * a.p.rows[k].sn + c * 16) =
          *reinterpret_cast<const uint4*>(rows + src[i] * a.p.rows[k].sn + c * 16);
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s) {
  const int units = a.p.B * a.p.h_kv;
  evict_select_kernel<<<units, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per_unit = a.max_moves / 64 < 1 ? 1 : a.max_moves / 64 > 64 ? 64 : a.max_moves / 64;
  evict_move_kernel<<<units * per_unit, 256, 0, s>>>(a, per_unit);
  return cudaGetLastError();
}

}  // namespace da
