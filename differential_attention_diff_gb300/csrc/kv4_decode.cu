// kv4_decode.cu — V2 decode over a 4-bit KV cache (records of kv4.cu).
//
// out_p = (A_2p - gate_p A_2p+1) V with A_j = softmax(scale q_j K^T), K and V
// the values s n + m that the records stand for (n a 4-bit code; s, m per
// half row).  A record is 144 bytes for 512 bytes of bf16 rows, so at the
// memory's rate an SM gets 23 bytes, 47 codes, a cycle: there are about 2.7
// lane-instructions per code.  Turning every code into s n + m first would
// spend twice that.  The kernel therefore multiplies the codes themselves:
//   score_j  = sum_groups s (q . n) + m (sum of q),
//   output_f = sum_j (p_j s_j) n_jf + sum_j p_j m_j,
// with s and m applied to a group's 32 or 64 products at once.  A code masked
// out of its word IS an fp16 number, the subnormal n 2^-24 (or 16 n 2^-24 for
// the upper code of a byte), which the tensor cores take exactly, so a pair
// of codes costs one AND (and a shift per two pairs); 2^24 and 1/16 are
// powers of two that move into q and the final factor.
//
// Scores are taken transposed, S^T[16 keys x 8 heads] = K Q^T, so that the
// codes are the A operand and the heads (2h/h_kv of them, up to 16) fill the
// small side of m16n8k16; the products p s go through movmatrix into the B
// operand of O^T[16 features x 8 heads] += V^T P^T, whose pairs of keys are
// put side by side by two byte permutes per four pairs.
//
// A chunk's value product starts from zero and is then added to O.  Codes are
// not negative, so over thousands of keys their sum outgrows what is left
// once the minima are added, by a factor of hundreds; chained through the
// tensor cores, whose accumulators are truncated at each step, it lost 2.2e-3
// of the output (B64 L32768), more than the output's own rounding.  Sums of 32
// keys, added with rounding, lose nothing that shows, for an addition per
// accumulator and chunk; at d 128 two accumulators share one (64 x 32768:
// 398 -> 388.5 us; at d 64 it measured slower, 78.6 -> 83.5 at 64 x 8192).
//
// P is fp16 (11 bits, against 8 of a bf16 P).  Its range is kept by a factor
// per head and half row, vs, beside the running maximum m of the scores: they are
// references that only move when a value would pass 2^-2 (p) or 2^14 (p s vs),
// or is NaN, by a warp vote, so the common path has no reductions.  vs follows p s and
// not s, so a large value row of a key with no weight costs no precision, and
// each half has its own, so neither does a half beside a larger one (a factor
// for both lost a half's codes behind one 2^30 larger).
// Sums of p, of p m and the score corrections are fp32.
//
// Schedule: the batch's work is one line of 32-key chunks in (sequence, KV
// head) order, cut into equal parts, one per warp (16 warps on each SM, 8
// where two head tiles need the registers), so ragged lengths balance
// exactly.  A warp streams its part through a ring of its own and shares
// nothing with the others: where a head ends it writes its partial (max, sum,
// O) and goes on to the next, and no block-wide barrier stops the loads (warps
// that shared a head and summed their partials in shared memory took 63 us for
// 64 sequences of 2048 keys where this takes 46).  A second kernel merges the
// parts of each head and applies the gate.  Where the heads are few and short, a
// block takes a whole head instead, merges its warps' partials in shared memory
// and is done in one launch (the rule and both sides: own_blocks in kv_api.cu).
//
// Measured (64 query heads, 8 KV heads, d 128): 64 x 32768 keys 384 us with the
// gate from x, 6.3 TB/s of records over the whole call, 0.93 of a copy; 2 x
// 131072 with the keys' weights 88 us; one sequence of 1000 keys 10 us, in one
// launch.  Up to about 64 x 8192 keys the instructions bound it (580 a chunk and
// warp, issue slots 64 % busy, ALU pipe 61 %, tensor pipe 28 %, at 5.6 TB/s; at
// d 64 455, 71 %, 58 % and 20 %, at 4.5 TB/s), above that the memory nearly does.
#include "common.cuh"
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "decode_merge.cuh"
#include "fp32_pair.cuh"
#include "kernels.h"
#include "tma.cuh"

namespace cg = cooperative_groups;

namespace da {
namespace {

constexpr int kChunk = kKv4ChunkKeys;  // keys per ring slot

template <int D, int NT>
struct Cfg {
  // 128 registers a thread allow 16 warps; two head tiles need more
  static constexpr int kWarps = NT == 1 ? 16 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRec = D + 16;
  static constexpr int kSlot = kChunk * kRec;  // bytes
  static constexpr int kStages = NT == 1 ? 3 : 5;
  static constexpr int kRing = kWarps * kStages * kSlot;  // 221,184 (D 128, 16 warps) or less
  static constexpr int kWords = D / 64;     // 4-byte code words per lane, group and key row (K side)
  static constexpr int kTiles = D / 16;     // 16-feature tiles of O^T
  static constexpr int kGroupTiles = kTiles / 2;
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// D = A(16x16, row) * B(16x8, col) + D, fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero accumulators.
__device__ __forceinline__ void mma_f16_16816_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// x[0..1] += y[0..1], in one instruction if kOne.
template <bool kOne>
__device__ __forceinline__ void add_pair(float* x, const float* y) {
  if constexpr (kOne) {
    const uint2 r = add2(F2(x[0], x[1]), F2(y[0], y[1])).bits();
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
  } else {
    x[0] += y[0];
    x[1] += y[1];
  }
}
// 8x8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Untiled bulk copy, both addresses and the size multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t x;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(x));
  return x;
}
// The same with an L2 policy.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
template <class T>
__device__ __forceinline__ T lds(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}
// 2^k for k in -126 .. 127, the exponent of a normal number, and 1 / x of a power of two in 2^-126 .. 2^126.
__device__ __forceinline__ float power(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float inverse_power(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// 16-byte copies that a barrier counts: each lane's arrival comes when its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Chunks of one head of sequence b: 0 for a bad length.
__device__ __forceinline__ int seq_chunks(const Kv4DecodeArgs& a, int b) {
  const int L = a.seqlens ? a.seqlens[b] : a.L_max;
  return L < 1 || L > a.L_max ? 0 : (L + kChunk - 1) / kChunk;
}

// A warp's place on the line of chunks: the next chunk of head b * h_kv + g,
// and where its part of that head ends.
struct Cursor {
  int b, g, chunk, end;
  int L;     // the sequence's length
  int left;  // chunks of this warp's part behind this head (its records fit the memory: 32 bits do)
};
// About what a warp takes in the 8 us of the gate's projection (64 x 8192 with
// 0, 3, 4, 5, 6: 122.4, 117.6, 117.2, 117.0, 119.8 us).
constexpr int kLateChunks = 4;

// The reference of a head that has seen no key: any score above it sends p past kTop.
constexpr float kNoMax = -0x1.fffffep127f;

// A moved reference lies kHeadroom above the largest score, and p may grow by
// 2^8 before it moves again: p stays below 1, so that sums of p m and of p s n
// of values at the end of their range stay within it (as in a softmax about
// its true maximum, and with a reference at the maximum they did not).
constexpr int kHeadroom = 10;
constexpr float kTop = 0x1p-2f;

// What the products of codes are multiplied by where a query is so large that
// its score factor is divided by it.
constexpr float kLift = 0x1p32f;

// kOwn: a block (1), or a cluster of a.own blocks (2), takes a whole head, shares
// its chunks out to its warps, merges them and writes the output (and the keys'
// weights) itself: one launch for short sequences of few heads.
template <int D, int NT, bool kScores, int kOwn>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) kv4_split_kernel(Kv4DecodeArgs a) {
  using C = Cfg<D, NT>;
  constexpr int kW = C::kWarps, kS = C::kStages, kRec = C::kRec, kWords = C::kWords, kGT = C::kGroupTiles;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kW * kS];
  __shared__ int64_t warp_sum[kOwn ? 1 : kW];
  __shared__ int64_t ends[kOwn ? 1 : C::kThreads];  // of a tile of sequences: chunks of one head up to each one's end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, tq = lane & 3;
  const int H2 = 2 * a.h, G = H2 / a.h_kv;
  const bool dense = a.cache.sn == kRec;

  if (tid < kW * kS) mbar_init(smem_u32(&bars[tid]), dense ? 1 : 32);
  fence_mbar_init();

  Cursor at;
  int64_t me = 0;
  int take = 0;  // chunks of this warp's part
  if constexpr (kOwn) {
    __syncthreads();  // the barriers
    const int own = kOwn == 1 ? 1 : a.own, unit = blockIdx.x / own, part = blockIdx.x % own;
    at.b = unit / a.h_kv;
    at.g = unit % a.h_kv;
    const int n = seq_chunks(a, at.b);
    if (n == 0) {  // a bad length: recorded, zeros (and the whole cluster leaves)
      if (tid == 0 && part == 0) record_status(a.status, DA_ERR_BOUNDS, 0x4B02);
      for (int x = part * C::kThreads + tid; x < G / 2 * D; x += own * C::kThreads)
        static_cast<__nv_bfloat16*>(a.out)[(static_cast<int64_t>(at.b) * a.h + at.g * (G / 2)) * D + x] = __float2bfloat16_rn(0.f);
      cudaGridDependencySynchronize();
      return;
    }
    const int w = part * kW + warp;
    at.chunk = w * n / (own * kW);
    take = (w + 1) * n / (own * kW) - at.chunk;
  } else {
    // ---- this warp's part of the line ----
    // sequences b0 .. b0 + kThreads - 1 into `ends`; returns the sum up to their end
    auto sum_tile = [&](int b0, int64_t carry) {
      const int b = b0 + tid;
      int64_t x = b < a.B ? seq_chunks(a, b) : 0;
      if (blockIdx.x == 0 && b < a.B && x == 0) record_status(a.status, DA_ERR_BOUNDS, 0x4B02);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      for (int w = 0; w < warp; ++w) x += warp_sum[w];
      x += carry;
      ends[tid] = x;
      __syncthreads();
      return ends[C::kThreads - 1];
    };
    int64_t sum = 0;
    for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
      if (b0) __syncthreads();
      sum = sum_tile(b0, sum);
    }
    const int64_t total = sum * a.h_kv;
    const int64_t parts = kv4_parts(total, static_cast<int64_t>(gridDim.x) * kW);
    // Few parts go to an SM each; as many as there are warps go to each SM side
    // by side, where they touch fewer pages.
    me = parts < static_cast<int64_t>(gridDim.x) * kW ? static_cast<int64_t>(warp) * gridDim.x + blockIdx.x
                                                                    : static_cast<int64_t>(blockIdx.x) * kW + warp;
    const bool works = me < parts;
    // Beside the gate's projection the grid's last blocks start when it ends,
    // on the SMs that it had: their warps get kLateChunks fewer than the others.
    const int64_t late = parts == static_cast<int64_t>(gridDim.x) * kW && total >= 24 * parts ? a.late_blocks * kW : 0;
    auto cut = [&](int64_t w) {
      const int64_t x = w * (total + late * kLateChunks) / parts, behind = w - (parts - late);
      return behind > 0 ? x - behind * kLateChunks : x;
    };
    const int64_t first = works ? cut(me) : 0, last = works ? cut(me + 1) : 0;
    take = static_cast<int>(last - first);
    at.b = -1;
    int64_t from = 0;  // chunks before the tile, of one head
    for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
      if (a.B > C::kThreads) {  // more than one tile: the last one is in `ends` now
        __syncthreads();
        sum_tile(b0, from);
      }
      if (works && at.b < 0 && first < ends[C::kThreads - 1] * a.h_kv) {
        // the sequence whose end is the first above `first`
        for (int i = 0; at.b < 0; i += 32) {
          const unsigned hit = __ballot_sync(0xffffffffu, ends[i + lane] * a.h_kv > first);
          if (hit) {
            const int k = i + __ffs(hit) - 1;
            at.b = b0 + k;
            const int64_t before = k ? ends[k - 1] : from;
            const int n = static_cast<int>(ends[k] - before);
            const int64_t in = first - before * a.h_kv;
            at.g = static_cast<int>(in / n);
            at.chunk = static_cast<int>(in - static_cast<int64_t>(at.g) * n);
          }
        }
      }
      from = ends[C::kThreads - 1];
    }
    if (!works) {
      cudaGridDependencySynchronize();  // the gate, where it runs beside this kernel: the merge counts on its end
      return;
    }
  }

  auto enter = [&](Cursor& c, int begin) {  // chunks begin .. of head (c.b, c.g), as far as the part goes
    c.L = a.seqlens ? a.seqlens[c.b] : a.L_max;
    const int n = (c.L + kChunk - 1) / kChunk;
    const int take = min(n - begin, c.left);
    c.end = begin + take;
    c.left -= take;
    c.chunk = begin;
  };
  auto next_head = [&](Cursor& c) {  // c.left > 0: another head with chunks follows
    do {
      if (++c.g == a.h_kv) c.g = 0, ++c.b;
    } while (seq_chunks(a, c.b) == 0);
    enter(c, 0);
  };
  at.left = take;
  enter(at, at.chunk);

  const uint32_t ring = smem_u32(smem) + warp * kS * C::kSlot;
  const uint32_t bar0 = smem_u32(&bars[warp * kS]);
  const uint8_t* cache = static_cast<const uint8_t*>(a.cache.ptr);
  bool dead = false;  // a wait ran out: nothing more is issued or read

  // fill the ring's next slot with the chunk that `ahead` is at
  Cursor ahead = at;
  const int64_t chunk_bytes = kChunk * a.cache.sn;
  // Where scores are stored the records are the first that L2 lets go, so that
  // the weights' kernel finds the scores there (2 x 131072: 90.1 -> 85.6 us,
  // 64 x 2048: 59.0 -> 54.3).  The 16-byte copies of records that lie apart go
  // without (a kernel whose copies carried one ended with an illegal instruction).
  const uint64_t once = evict_first_policy();
  auto source = [&]() { return cache + ahead.b * a.cache.sb + ahead.g * a.cache.sh + ahead.chunk * chunk_bytes; };
  const uint8_t* src = source();
  int in_flight = 0, fill = 0;    // chunks, and the slot that the next one goes to
  int slot = 0;                   // the slot to read next
  uint32_t parity = 0;            // of each slot's barrier, one bit each
  auto issue = [&]() {
    if (ahead.chunk >= ahead.end) {
      if (ahead.left == 0) return;
      next_head(ahead);
      src = source();
    }
    if (dead) return;
    const int n = min(kChunk, ahead.L - ahead.chunk * kChunk);
    const uint32_t dst = ring + fill * C::kSlot, bar = bar0 + fill * 8;
    if (dense) {  // one bulk copy
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, n * kRec);
        if constexpr (kScores)
          bulk_load(dst, src, n * kRec, bar, once);
        else
          bulk_load(dst, src, n * kRec, bar);
      }
    } else {  // records apart: a bulk copy each measured slower than 16 bytes per lane
      constexpr int kPieces = kRec / 16;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int x = i * 32 + lane, r = x / kPieces, c = x % kPieces;
        if (r < n) cp_async_16(dst + x * 16, src + r * a.cache.sn + c * 16, 16);
      }
      cp_async_arrive(bar);
    }
    ++in_flight;
    fill = fill == kS - 1 ? 0 : fill + 1;
    ++ahead.chunk;
    src += chunk_bytes;
  };
#pragma unroll 1
  for (int i = 0; i < kS - 1; ++i) issue();

  // row gr of a 16-key tile is key row_key, row gr + 8 the key after it: an
  // order that keeps both the K and the V loads off each other's banks
  const int b2 = gr >> 2, b1 = (gr >> 1) & 1, b0 = gr & 1;
  const int row_key = 8 * b2 + 2 * b1 + 4 * (b0 ^ b2);
  auto key_of = [](int r) { return 8 * (r >> 2) + 2 * ((r >> 1) & 1) + 4 * ((r & 1) ^ (r >> 2)); };
  const int vkey0 = key_of(2 * tq), vkey1 = key_of(2 * tq + 1);

  while (true) {
    // ---- a head: its queries ----
    const int64_t unit = static_cast<int64_t>(at.b) * a.h_kv + at.g;
    uint32_t qf[NT][4 * kWords][2];  // B fragments: [2 groups x kWords x 2 MMAs]
    float qs0[NT][2], qs1[NT][2], fac[NT][2];  // of heads 2 tq, 2 tq + 1: group sums of q, score factor
    unsigned lifted[NT];  // bit 4 j: head j's products take kLift
    bool careful = false;  // whole chunks go the way of partial ones (see take_chunk)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int head = t * 8 + gr;
      float q[2][8 * kWords];
      float mx = 0.f;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (head < G)
            v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                (static_cast<int64_t>(at.b) * H2 + at.g * G + head) * D + p * (D / 2) +
                                                tq * (D / 8) + w * 8);
          const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            q[p][w * 8 + 2 * e] = lo_bf16(ws[e]);
            q[p][w * 8 + 2 * e + 1] = hi_bf16(ws[e]);
            mx = fmaxf(mx, fmaxf(fabsf(lo_bf16(ws[e])), fabsf(hi_bf16(ws[e]))));
          }
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // largest query feature in [2^14, 2^15): exact in fp16 down to 2^-31 of it,
      // 2^-27 where a feature meets upper codes and is divided by 16
      const float up = mx > 0.f ? power(min(max(14 - exponent(mx), -126), 126)) : 1.f;
      const bool lift = up < 0x1p-64f;  // 2^24 / up would pass the largest number at 2^-104
      lifted[t] = __ballot_sync(0xffffffffu, lift);
      careful |= lifted[t] != 0;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int i = 0; i < 8 * kWords; ++i) {
          q[p][i] *= up;
          sum[p] += q[p][i];
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float* x = &q[p][w * 8 + 2 * m];
            qf[t][(p * kWords + w) * 2 + m][0] = pack_f16x2(x[0], x[4]);
            qf[t][(p * kWords + w) * 2 + m][1] = pack_f16x2(x[1] * 0.0625f, x[5] * 0.0625f);
          }
        sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], 1);
        sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], 2);
        sum[p] *= 0x1p-24f;
      }
      const float f = (lift ? 0x1p24f / kLift : 0x1p24f) * inverse_power(up) * a.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs0[t][e] = __shfl_sync(0xffffffffu, sum[0], (2 * tq + e) * 4);
        qs1[t][e] = __shfl_sync(0xffffffffu, sum[1], (2 * tq + e) * 4);
        fac[t][e] = __shfl_sync(0xffffffffu, f, (2 * tq + e) * 4);
      }
    }
    float o[NT][C::kTiles][4];
    // reference max, value factors (per group), sums of p and of p m (per group)
    float mx[NT][2], vs[NT][2][2], l[NT][2], mn[NT][2][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < C::kTiles; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[t][e] = kNoMax;
        vs[t][0][e] = vs[t][1][e] = 0x1p126f;
        l[t][e] = mn[t][0][e] = mn[t][1][e] = 0.f;
      }
    }

    const int begin = at.chunk;
    for (; at.chunk < at.end; ++at.chunk) {
      issue();  // into the slot read last
      if (dead) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(bar0 + slot * 8, (parity >> slot) & 1, a.status, 0x4B04))) {
        dead = true;
        continue;
      }
      --in_flight;
      parity ^= 1u << slot;
      const uint8_t* base = smem + (warp * kS + slot) * C::kSlot;
      slot = slot == kS - 1 ? 0 : slot + 1;
      const int valid = at.L - at.chunk * kChunk;  // keys of this chunk

      // kPartial: a chunk that is not whole, or a head that asks for care.  In
      // the others scores are held as their fac-th part, and p = 2^(s fac - m) is
      // one multiply-add.  Its unrounded product is off from the rounded one by up
      // to half an ulp, which passes the range of p from scores of about 2^30 on:
      // there, and wherever a reference moves, s fac is rounded first.
      auto take_chunk = [&](auto partial) {
        constexpr bool kPartial = decltype(partial)::value;
        // ---- scores (of fac log2 units), two 16-key tiles ----
        [[maybe_unused]] float* const score_row = kScores ? a.scores + (unit * a.L_max + at.chunk * kChunk + row_key) * G + 2 * tq : nullptr;
        uint4 par[2][2];  // [tile][row half]: K s0 s1 | K m0 m1 | V s0 s1 | V m0 m1
        float s[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* ra = base + (u * 16 + row_key) * kRec;
          par[u][0] = lds<uint4>(ra + D);
          par[u][1] = lds<uint4>(ra + kRec + D);
          if constexpr (kPartial) {  // what lies behind the last key may be anything: zero parameters
            if (u * 16 + row_key >= valid) par[u][0] = make_uint4(0, 0, 0, 0);
            if (u * 16 + row_key + 1 >= valid) par[u][1] = make_uint4(0, 0, 0, 0);
          }
          float acc[2][NT][4];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t wa[kWords], wb[kWords];
            const uint32_t off = p * (D / 4) + tq * (D / 16);
            if constexpr (kWords == 2) {
              const uint2 x = lds<uint2>(ra + off), y = lds<uint2>(ra + kRec + off);
              wa[0] = x.x, wa[1] = x.y, wb[0] = y.x, wb[1] = y.y;
            } else {
              wa[0] = lds<uint32_t>(ra + off);
              wb[0] = lds<uint32_t>(ra + kRec + off);
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w)
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const uint32_t x = wa[w] >> (8 * m), y = wb[w] >> (8 * m);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  const uint32_t* b = qf[t][(p * kWords + w) * 2 + m];
                  if (w == 0 && m == 0)
                    mma_f16_16816_first(acc[p][t], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u, b[0],
                                        b[1]);
                  else
                    mma_f16_16816(acc[p][t], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u, b[0], b[1]);
                }
              }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4& r = par[u][e >> 1];
              const int c = e & 1;
              float x = hi_bf16(r.y) * qs1[t][c];
              x = fmaf(lo_bf16(r.y), qs0[t][c], x);
              x = fmaf(lo_bf16(r.x), acc[0][t][e], x);
              x = fmaf(hi_bf16(r.x), acc[1][t][e], x);
              s[u][t][e] = kPartial ? x * fac[t][c] * ((lifted[t] >> (8 * tq + 4 * c)) & 1 ? kLift : 1.f) : x;
            }
          if constexpr (kPartial) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (u * 16 + row_key + (e >> 1) >= valid) s[u][t][e] = -INFINITY;
          }
          if constexpr (kScores) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int k = u * 16 + row_key + r;
                if ((!kPartial || k < valid) && t * 8 + 2 * tq < G)
                  *reinterpret_cast<float2*>(score_row + (u * 16 + r) * G + t * 8) =
                      kPartial ? make_float2(s[u][t][2 * r], s[u][t][2 * r + 1])
                               : make_float2(s[u][t][2 * r] * fac[t][0], s[u][t][2 * r + 1] * fac[t][1]);
              }
          }
        }

        // ---- softmax against the references ----
        float p[2][NT][4], lsum[NT][2];
        uint32_t pf[2][NT][2][2];  // [tile][head tile][group][row half], fp16 pairs of heads
        auto weigh = [&](auto rounded) {  // rounded: s is s fac already
          constexpr bool kRounded = decltype(rounded)::value, kTwo = kRounded || !kScores;
          bool over = false;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float sx = s[u][t][2 * r], sy = s[u][t][2 * r + 1];
                const float x = fast_exp2(kRounded ? sx - mx[t][0] : fmaf(sx, fac[t][0], -mx[t][0]));
                const float y = fast_exp2(kRounded ? sy - mx[t][1] : fmaf(sy, fac[t][1], -mx[t][1]));
                p[u][t][2 * r] = x;
                p[u][t][2 * r + 1] = y;
                const float s0 = lo_bf16(par[u][r].z), s1 = hi_bf16(par[u][r].z);
                const F2 xy(x, y);
                const uint2 v0 = mul2(xy, F2(vs[t][0][0], vs[t][0][1])).bits();
                const uint2 v1 = kTwo ? mul2(xy, F2(vs[t][1][0], vs[t][1][1])).bits() : v0;
                pf[u][t][0][r] = pack_f16x2(__uint_as_float(v0.x) * s0, __uint_as_float(v0.y) * s0);
                pf[u][t][1][r] = pack_f16x2(__uint_as_float(v1.x) * s1, __uint_as_float(v1.y) * s1);
              }
            lsum[t][0] = (p[0][t][0] + p[0][t][2]) + (p[1][t][0] + p[1][t][2]);
            lsum[t][1] = (p[0][t][1] + p[0][t][3]) + (p[1][t][1] + p[1][t][3]);
            over |= !(lsum[t][0] <= kTop && lsum[t][1] <= kTop);
            // none of them is negative: their sum bounds each (and its adds do
            // not take the pipe that the code masks fill)
            __half2 top = *reinterpret_cast<__half2*>(&pf[0][t][0][0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) top = __hadd2(top, *reinterpret_cast<__half2*>(&pf[i >> 2][t][(i >> 1) & 1][i & 1]));
            over |= !__hle(__hadd(__low2half(top), __high2half(top)), __float2half(16384.f));
          }
          return over;
        };
        if (__any_sync(0xffffffffu, weigh(partial))) {
          if constexpr (!kPartial) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[u][t][e] *= fac[t][e & 1];
          }
          // new references from this chunk's keys: a whole number kHeadroom above
          // the score maximum, then powers of two from each half's largest p s under it, so
          // that what was summed so far is scaled exactly
          careful = false;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            careful |= lifted[t] != 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(fmaxf(s[0][t][e], s[0][t][2 + e]), fmaxf(s[1][t][e], s[1][t][2 + e]));
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              const float old = mx[t][e], now = fmaxf(old, ceilf(top) + kHeadroom);
              float big[2] = {0.f, 0.f};
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const float w = fast_exp2(s[u][t][2 * r + e] - now);
                  big[0] = fmaxf(big[0], w * lo_bf16(par[u][r].z));
                  big[1] = fmaxf(big[1], w * hi_bf16(par[u][r].z));
                }
              // the upper halves of both, which order as whole numbers do (without a zero's sign)
              uint32_t both = __byte_perm(__float_as_uint(big[0]), __float_as_uint(big[1]), 0x7632) & 0x7fff7fffu;
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, x));
              // O stands for O / vs: a higher maximum raises vs and leaves O alone
              const int rise = static_cast<int>(fminf(now - old, 512.f));
              int had[2], k[2];
#pragma unroll
              for (int g2 = 0; g2 < 2; ++g2) {
                const uint32_t top16 = g2 ? both >> 16 : both & 0xffffu;
                had[g2] = exponent(vs[t][g2][e]) + rise;
                k[g2] = min(had[g2], 126);
                if (top16) k[g2] = max(min(k[g2], 8 + 127 - static_cast<int>(top16 >> 7)), -126);
              }
              careful |= fabsf(now) > 0x1p22f;
              // Where scores are stored, halves of about the same size take one
              // factor, and others ask for care: fewer multiplications in the
              // common path (64 x 8192: 169.5 -> 163.7 us, 169.2 for halves 2^10
              // apart; without scores two factors are as fast, 112.5 and 112.5).
              if constexpr (kScores) {
                const int low = min(k[0], k[1]);
                if (max(k[0], k[1]) <= low + 4) k[0] = k[1] = low;
                careful |= k[0] != k[1];
              }
              const float down = rise > 126 ? 0.f : power(-rise);
              mx[t][e] = now;
              l[t][e] *= down;
#pragma unroll
              for (int g2 = 0; g2 < 2; ++g2) {
                mn[t][g2][e] *= down;
                const float by = k[g2] < had[g2] - 126 ? 0.f : power(k[g2] - had[g2]);
                vs[t][g2][e] = power(k[g2]);
#pragma unroll
                for (int i = g2 * kGT; i < (g2 + 1) * kGT; ++i) {
                  o[t][i][e] *= by;
                  o[t][i][2 + e] *= by;
                }
              }
            }
          }
          careful = __any_sync(0xffffffffu, careful);
          weigh(std::true_type{});
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[t][e] += lsum[t][e];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                mn[t][0][e] = fmaf(p[u][t][2 * r + e], lo_bf16(par[u][r].w), mn[t][0][e]);
                mn[t][1][e] = fmaf(p[u][t][2 * r + e], hi_bf16(par[u][r].w), mn[t][1][e]);
              }
          }

        // ---- O^T += V^T P^T, a chunk's product first, then its sum in fp32 ----
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          uint32_t bf[2][NT][2], w[2][4];  // [tile]; codes of keys (vkey0, vkey1) and the ones after them
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint8_t *va = base + (u * 16 + vkey0) * kRec + D / 2, *vb = base + (u * 16 + vkey1) * kRec + D / 2;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              bf[u][t][0] = movmatrix(pf[u][t][g2][0]);
              bf[u][t][1] = movmatrix(pf[u][t][g2][1]);
            }
            if constexpr (D == 128) {
              const uint32_t off = g2 * 32 + gr * 4;
              w[u][0] = lds<uint32_t>(va + off), w[u][1] = lds<uint32_t>(vb + off);
              w[u][2] = lds<uint32_t>(va + kRec + off), w[u][3] = lds<uint32_t>(vb + kRec + off);
            } else {
              const uint32_t off = g2 * 16 + gr * 2;
              w[u][0] = lds<uint16_t>(va + off), w[u][1] = lds<uint16_t>(vb + off);
              w[u][2] = lds<uint16_t>(va + kRec + off), w[u][3] = lds<uint16_t>(vb + kRec + off);
            }
          }
#pragma unroll
          for (int hw = 0; hw < kWords; ++hw) {
            float even[NT][4], odd[NT][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // four features of both keys side by side
              const uint32_t sel = hw ? 0x7632 : 0x5410;
              const uint32_t x = __byte_perm(w[u][0], w[u][1], sel), y = __byte_perm(w[u][2], w[u][3], sel);
              const uint32_t xs = x >> 8, ys = y >> 8;
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (u == 0) {
                  mma_f16_16816_first(even[t], x & 0x000f000fu, xs & 0x000f000fu, y & 0x000f000fu, ys & 0x000f000fu,
                                      bf[u][t][0], bf[u][t][1]);
                  mma_f16_16816_first(odd[t], x & 0x00f000f0u, xs & 0x00f000f0u, y & 0x00f000f0u, ys & 0x00f000f0u,
                                      bf[u][t][0], bf[u][t][1]);
                } else {
                  mma_f16_16816(even[t], x & 0x000f000fu, xs & 0x000f000fu, y & 0x000f000fu, ys & 0x000f000fu,
                                bf[u][t][0], bf[u][t][1]);
                  mma_f16_16816(odd[t], x & 0x00f000f0u, xs & 0x00f000f0u, y & 0x00f000f0u, ys & 0x00f000f0u,
                                bf[u][t][0], bf[u][t][1]);
                }
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                add_pair<D == 128>(&o[t][g2 * kGT + hw * 2][i], &even[t][i]);
                add_pair<D == 128>(&o[t][g2 * kGT + hw * 2 + 1][i], &odd[t][i]);
              }
          }
        }
      };
      if (valid >= kChunk && !careful)
        take_chunk(std::false_type{});
      else
        take_chunk(std::true_type{});
      __syncwarp();  // the slot is read before it is filled again
    }

    if constexpr (kOwn) {
      // ---- the head's end: all warps' partials, in the ring's place ----
      __shared__ float2 wml[kW][8 * NT];
      __shared__ float2 norm[8 * NT];      // maximum and 1 / sum
      __shared__ float factor[kW][8 * NT];  // of each warp's part in its head's sum
      float* park = reinterpret_cast<float*>(smem);  // [warp][head][D]
      __syncthreads();  // the ring is read (a warp without chunks has m = kNoMax, l = 0, O = 0)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lt = l[t][e], m0 = mn[t][0][e], m1 = mn[t][1][e];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            lt += __shfl_xor_sync(0xffffffffu, lt, x);
            m0 += __shfl_xor_sync(0xffffffffu, m0, x);
            m1 += __shfl_xor_sync(0xffffffffu, m1, x);
          }
          const int head = t * 8 + 2 * tq + e;
          const float f[2] = {inverse_power(vs[t][0][e]), inverse_power(vs[t][1][e])};
          if (gr == 0) wml[warp][head] = make_float2(mx[t][e], lt);
#pragma unroll
          for (int g2 = 0; g2 < 2; ++g2)
#pragma unroll
            for (int hw = 0; hw < kWords; ++hw) {
              const float* x = o[t][g2 * kGT + hw * 2];
              const float* y = o[t][g2 * kGT + hw * 2 + 1];
              const float m = g2 ? m1 : m0;
              *reinterpret_cast<float4*>(park + (warp * 8 * NT + head) * D + g2 * (D / 2) + gr * (D / 16) + hw * 4) =
                  make_float4(fmaf(x[e] * 0x1p24f, f[g2], m), fmaf(y[e] * 0x1p20f, f[g2], m),
                              fmaf(x[2 + e] * 0x1p24f, f[g2], m), fmaf(y[2 + e] * 0x1p20f, f[g2], m));
            }
        }
      __syncthreads();
      if (tid < 8 * NT * kW) {  // kW lanes side by side for each head
        const int w = tid % kW, head = tid / kW;
        const float2 part = wml[w][head];
        float top = part.x;
#pragma unroll
        for (int x = 1; x < kW; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float down = exp2f(part.x - top);
        float sum = part.y * down;
#pragma unroll
        for (int x = 1; x < kW; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        // a sum of 0 is keys that are all -inf: zeros, as in decode.cu; NaN stays
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        factor[w][head] = kOwn == 2 ? down : down * inv;
        if (w == 0) norm[head] = make_float2(top, kOwn == 2 ? sum : inv);
      }
      cudaGridDependencySynchronize();  // the gate, where it runs beside this kernel
      __syncthreads();
      const int64_t pair0 = static_cast<int64_t>(at.b) * a.h + at.g * (G / 2);
      if constexpr (kOwn == 2) {  // this block's sums, then those of the cluster's blocks
        __shared__ float2 block_norm[8 * NT];
        cg::cluster_group cluster = cg::this_cluster();
        float* mine = park + kW * 8 * NT * D;  // [head][D]
        static_assert((kW + 1) * 8 * NT * D * 4 <= C::kRing, "the blocks' sums lie behind the warps'");
        for (int x = tid; x < G * D; x += C::kThreads) {
          const int head = x / D;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kW; ++w) sum = fmaf(park[(w * 8 * NT + head) * D + x % D], factor[w][head], sum);
          mine[x] = sum;
        }
        if (tid < 8 * NT) block_norm[tid] = norm[tid];
        cluster.sync();
        if (tid < 8 * NT) {
          float top = kNoMax, sum = 0.f;
          for (int c = 0; c < a.own; ++c) top = fmaxf(top, cluster.map_shared_rank(block_norm, c)[tid].x);
          for (int c = 0; c < a.own; ++c) {
            const float2 x = cluster.map_shared_rank(block_norm, c)[tid];
            sum += x.y * exp2f(x.x - top);
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          norm[tid] = make_float2(top, inv);
          for (int c = 0; c < a.own; ++c) factor[c][tid] = exp2f(cluster.map_shared_rank(block_norm, c)[tid].x - top) * inv;
        }
        __syncthreads();
        const int part = static_cast<int>(cluster.block_rank());
        for (int x = part * C::kThreads + tid; x < G / 2 * D; x += a.own * C::kThreads) {
          const int p = x / D, f = x % D;
          float res[2] = {0.f, 0.f};
          for (int c = 0; c < a.own; ++c) {
            const float* theirs = cluster.map_shared_rank(mine, c);
#pragma unroll
            for (int e = 0; e < 2; ++e) res[e] = fmaf(theirs[(2 * p + e) * D + f], factor[c][2 * p + e], res[e]);
          }
          store_pair(a.out, a.gate, pair0 + p, D, f, res[0], res[1]);
        }
      } else {
        for (int x = tid; x < G / 2 * D; x += C::kThreads) {
          const int p = x / D, f = x % D;
          float res[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 0; w < kW; ++w)
              res[e] = fmaf(park[(w * 8 * NT + 2 * p + e) * D + f], factor[w][2 * p + e], res[e]);
          store_pair(a.out, a.gate, pair0 + p, D, f, res[0], res[1]);
        }
      }
      if constexpr (kScores) {  // written by this block, read after its barriers
        const float* t0 = a.scores + unit * a.L_max * G;
        const int n = (at.L + kChunk - 1) / kChunk, own = kOwn == 1 ? 1 : a.own, part = blockIdx.x % own;
        const int k0 = part * n / own * kChunk, k1 = min(at.L, (part + 1) * n / own * kChunk);  // this block's keys
        for (int key = k0 + tid; key < k1; key += C::kThreads) {
          float w = a.weights_in ? a.weights_in[unit * a.L_max + key] : 0.f;
          for (int p = 0; p < G / 2; ++p) {
            const float2 t = reinterpret_cast<const float2*>(t0 + static_cast<int64_t>(key) * G)[p];
            const float2 n0 = norm[2 * p], n1 = norm[2 * p + 1];
            w += fabsf(__fsub_rn(__fmul_rn(exp2f(t.x - n0.x), n0.y), __fmul_rn(exp2f(t.y - n1.x), n1.y * a.gate[pair0 + p])));
          }
          a.weights_out[unit * a.L_max + key] = w;
        }
      }
      if constexpr (kOwn == 2) cg::this_cluster().sync();  // no block leaves while another may still read its sums
      break;
    }
    // ---- the head's end: this warp's partial ----
    const int64_t number = me + unit, row = number * G;
    if (lane == 0) {
      if (begin == 0) a.parts[unit].first = static_cast<int>(number);
      if (at.end * kChunk >= at.L) a.parts[unit].last = static_cast<int>(number);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lt = l[t][e], m0 = mn[t][0][e], m1 = mn[t][1][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          lt += __shfl_xor_sync(0xffffffffu, lt, x);
          m0 += __shfl_xor_sync(0xffffffffu, m0, x);
          m1 += __shfl_xor_sync(0xffffffffu, m1, x);
        }
        const int head = t * 8 + 2 * tq + e;
        if (head >= G) continue;
        const float f[2] = {inverse_power(vs[t][0][e]), inverse_power(vs[t][1][e])};
        float* po = a.part_o + (row + head) * D;
        if (gr == 0) *reinterpret_cast<float2*>(a.part_ml + (row + head) * 2) = make_float2(mx[t][e], lt);
        // four neighbouring features: rows gr and gr + 8 of two tiles.  2^24
        // and f are applied apart: their product may overflow
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2)
#pragma unroll
          for (int hw = 0; hw < kWords; ++hw) {
            const float* x = o[t][g2 * kGT + hw * 2];
            const float* y = o[t][g2 * kGT + hw * 2 + 1];
            const float m = g2 ? m1 : m0;
            *reinterpret_cast<float4*>(po + g2 * (D / 2) + gr * (D / 16) + hw * 4) =
                make_float4(fmaf(x[e] * 0x1p24f, f[g2], m), fmaf(y[e] * 0x1p20f, f[g2], m),
                            fmaf(x[2 + e] * 0x1p24f, f[g2], m), fmaf(y[2 + e] * 0x1p20f, f[g2], m));
          }
      }
    if (at.left == 0) break;
    next_head(at);
  }
  // a warp that gave up waits (bounded) for what it still has in flight
  if (dead)
    for (; in_flight > 0; --in_flight) {
      mbar_wait(bar0 + slot * 8, (parity >> slot) & 1, nullptr, 0);
      slot = slot == kS - 1 ? 0 : slot + 1;
    }
  cudaGridDependencySynchronize();
}

// One output head's parts merged, even - gate * odd; also the two heads'
// normalisers for the keys' weights.  Grid (h, B, SLICES of the features).
// First the maximum and the sum over each head's parts: by a warp per head, or
// where the parts may be many (kMany) by the whole block; then threads are
// (way, head, four features) and the ways share out the parts.
template <int D, int SLICES, int WAYS, bool kMany>
__global__ void __launch_bounds__(WAYS * D / SLICES / 2) kv4_merge_kernel(Kv4DecodeArgs a) {
  constexpr int kCols = D / SLICES / 4, kThreads = WAYS * 2 * kCols, kWarps = kThreads / 32;
  __shared__ float2 part[kWarps][2];
  __shared__ float4 sums[WAYS][2][kCols];
  const int p = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = 2 * a.h / a.h_kv, g = 2 * p / G, r = 2 * p % G;
  const int L = a.seqlens ? a.seqlens[b] : a.L_max;
  const bool bad = L < 1 || L > a.L_max;  // recorded by the split kernel
  cudaGridDependencySynchronize();        // the parts
  // the weights' kernel may start: its scores are there, it waits for the norms
  cudaTriggerProgrammaticLaunchCompletion();
  int64_t first = 0;
  int count = 0;
  if (!bad) {
    const Kv4Parts s = a.parts[static_cast<int64_t>(b) * a.h_kv + g];
    first = s.first;
    count = s.last - s.first + 1;
  }
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + first * G + r;
  const int f = tid % kCols, e = tid / kCols % 2, way = tid / (2 * kCols);
  const float4* po = reinterpret_cast<const float4*>(a.part_o) + (first * G + r + e) * (D / 4) + blockIdx.z * kCols + f;
  // The first parts' rows, on their way while the maximum and the sum are found
  // (64 x 2048: 45.6 -> 44.7 us, 4 x 4096: 15.5 -> 15.1).  Blocks of 8 ways are
  // many and hide the wait by their number, up to where registers leave fewer of
  // them (16 x 4096 of 128 heads with 0, 1, 2, 4: 38.3, 36.7, 38.7, 39.2).
  constexpr int kEarly = WAYS == 8 ? 1 : 4;
  float4 early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int i = way + k * WAYS;
    early[k] = i < count ? po[static_cast<int64_t>(i) * G * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // of each head: maximum and 1 / sum.  A sum of 0 is an empty sequence or
  // keys that are all -inf: zeros, as in decode.cu; NaN stays
  float2 both[2];
  auto norm_of = [](float m, float l) { return make_float2(m, l == 0.f ? 0.f : 1.f / l); };
  if constexpr (kMany) {
    auto join = [](float2& x, float2 y) {  // (maximum, sum) of both
      const float m = fmaxf(x.x, y.x), nb = m == -INFINITY ? 0.f : m;
      x.y = x.y * exp2f(x.x - nb) + y.y * exp2f(y.x - nb);
      x.x = m;
    };
    float2 tot = make_float2(-INFINITY, 0.f);
#pragma unroll 4
    for (int i = tid >> 1; i < count; i += kThreads / 2) join(tot, ml[static_cast<int64_t>(i) * G + (tid & 1)]);
#pragma unroll
    for (int o = 2; o < 32; o <<= 1)
      join(tot, make_float2(__shfl_xor_sync(0xffffffffu, tot.x, o), __shfl_xor_sync(0xffffffffu, tot.y, o)));
    if (lane < 2) part[warp][lane] = tot;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      tot = lane < kWarps ? part[lane][e] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        join(tot, make_float2(__shfl_xor_sync(0xffffffffu, tot.x, o), __shfl_xor_sync(0xffffffffu, tot.y, o)));
      both[e] = norm_of(tot.x, tot.y);
    }
  } else {
    for (int e = warp; e < 2; e += kWarps) {
      float2 v[4];  // the first 128 parts at once, one wait for all
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = lane + 32 * k;
        v[k] = i < count ? ml[static_cast<int64_t>(i) * G + e] : make_float2(-INFINITY, 0.f);
      }
      float mt = fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x)), lt = 0.f;
      for (int i = lane + 128; i < count; i += 32) mt = fmaxf(mt, ml[static_cast<int64_t>(i) * G + e].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float nb = mt == -INFINITY ? 0.f : mt;
#pragma unroll
      for (int k = 0; k < 4; ++k) lt += v[k].y * exp2f(v[k].x - nb);
      for (int i = lane + 128; i < count; i += 32) {
        const float2 w = ml[static_cast<int64_t>(i) * G + e];
        lt += w.y * exp2f(w.x - nb);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
      if (lane == 0) part[0][e] = norm_of(mt, lt);
    }
    __syncthreads();
    both[0] = part[0][0];
    both[1] = part[0][1];
  }
  if (tid < 2 && blockIdx.z == 0 && a.norm) a.norm[static_cast<int64_t>(b) * 2 * a.h + 2 * p + tid] = both[tid & 1];
  const float mt = e ? both[1].x : both[0].x;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](int i, float4 v) {
    const float c = exp2f(ml[static_cast<int64_t>(i) * G + e].x - mt);
    x.x = fmaf(v.x, c, x.x);
    x.y = fmaf(v.y, c, x.y);
    x.z = fmaf(v.z, c, x.z);
    x.w = fmaf(v.w, c, x.w);
  };
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (way + k * WAYS < count) take(way + k * WAYS, early[k]);
#pragma unroll 4
  for (int i = way + kEarly * WAYS; i < count; i += WAYS) take(i, po[static_cast<int64_t>(i) * G * (D / 4)]);
  sums[way][e][f] = x;
  __syncthreads();
  if (tid < 4 * kCols) {
    float res[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll 8
      for (int w = 0; w < WAYS; ++w) res[k] += reinterpret_cast<const float*>(&sums[w][k][0])[tid];
      res[k] *= both[k].y;
    }
    const int64_t at = static_cast<int64_t>(b) * a.h + p;
    static_cast<__nv_bfloat16*>(a.out)[at * D + blockIdx.z * 4 * kCols + tid] =
        __float2bfloat16_rn(__fsub_rn(res[0], __fmul_rn(a.gate[at], res[1])));
  }
}

template <int D, int SLICES, int WAYS, bool kMany>
cudaError_t launch_merge(const Kv4DecodeArgs& a, cudaStream_t s) {
  constexpr int kThreads = WAYS * D / SLICES / 2;
  static_assert(kThreads >= D / SLICES && kThreads % 32 == 0 && kThreads <= 1024, "a thread per feature of the slice");
  return launch_ahead(kv4_merge_kernel<D, SLICES, WAYS, kMany>, dim3(a.h, a.B, SLICES), dim3(kThreads), 0, s, true, a);
}

// Ways by the parts that a head can have (as many as its chunks, or its share
// of the warps) and by the blocks that there are to fill the SMs with.
template <int D>
cudaError_t launch_merge_for(const Kv4DecodeArgs& a, cudaStream_t s) {
  const int64_t heads = static_cast<int64_t>(a.B) * a.h_kv, chunks = (static_cast<int64_t>(a.L_max) + kChunk - 1) / kChunk;
  const int64_t share = static_cast<int64_t>(a.grid) * kKv4MaxWarps / heads + 2, most = chunks < share ? chunks : share;
  const int64_t blocks = static_cast<int64_t>(a.h) * a.B;
  constexpr int kThin = D / 32;  // slices of 32 features
  if (most <= 16) return launch_merge<D, 1, 2, false>(a, s);
  if (most <= 128) return blocks > a.grid ? launch_merge<D, 1, 8, false>(a, s) : launch_merge<D, 1, 16, false>(a, s);
  return blocks * kThin > a.grid ? launch_merge<D, kThin / 2, 32, true>(a, s) : launch_merge<D, kThin, 64, true>(a, s);
}

template <int D, int NT, bool kScores, int kOwn>
cudaError_t launch_split(const Kv4DecodeArgs& a, cudaStream_t s) {
  using C = Cfg<D, NT>;
  static_assert(C::kRing <= 220 * 1024, "the ring and the static arrays fit an SM");
  static_assert(C::kWarps <= kKv4MaxWarps, "the workspace has room for every warp's parts");
  auto* kernel = kv4_split_kernel<D, NT, kScores, kOwn>;
  static OncePerDevice once;
  const cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kRing);
  });
  if (e != cudaSuccess) return e;
  return launch_clustered(kernel, dim3(kOwn ? a.B * a.h_kv * a.own : a.grid), dim3(C::kThreads), C::kRing, s, a.after_gate,
                          kOwn ? a.own : 1, a);
}

template <int D, int NT, int kOwn>
cudaError_t launch_scored(const Kv4DecodeArgs& a, cudaStream_t s) {
  return a.scores ? launch_split<D, NT, true, kOwn>(a, s) : launch_split<D, NT, false, kOwn>(a, s);
}

template <int kOwn>
cudaError_t launch_shaped(const Kv4DecodeArgs& a, cudaStream_t s) {
  const bool two = 2 * a.h / a.h_kv > 8;
  if (a.d == 128) return two ? launch_scored<128, 2, kOwn>(a, s) : launch_scored<128, 1, kOwn>(a, s);
  return two ? launch_scored<64, 2, kOwn>(a, s) : launch_scored<64, 1, kOwn>(a, s);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s) {
  if (a.own) return a.own == 1 ? launch_shaped<1>(a, s) : launch_shaped<2>(a, s);
  cudaError_t e = launch_shaped<0>(a, s);
  if (e != cudaSuccess) return e;
  e = a.d == 128 ? launch_merge_for<128>(a, s) : launch_merge_for<64>(a, s);
  if (e != cudaSuccess || a.weights_out == nullptr) return e;
  // a launch of its own: merged by the same kernel as a bf16 cache's splits, the
  // parts took 3 us more (64 x 2048 keys), since that kernel's blocks hold
  // twice the registers
  const FinishArgs f{a.B, a.h, a.h_kv, a.d, a.L_max, 0, a.norm, a.seqlens, a.gate, nullptr, nullptr, a.scores,
                     a.weights_in, a.weights_out, nullptr};
  return launch_decode_finish(f, s);
}

}  // namespace da
