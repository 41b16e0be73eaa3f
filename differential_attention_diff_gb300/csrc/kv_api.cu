// kv_api.cu — the extern "C" entry points of the 4-bit KV cache (append, read
// back, V2 decode) and of eviction: argument checks, workspace carving and the
// launches.  As in api.cu, nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <cmath>

#include "diffattn.h"
#include "kernels.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
da_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DA_OK : DA_ERR_CUDA; }

// Pointer and strides of a 16-byte-granular array: `unit` elements per 16 bytes.
bool ok_t4(const da_t4& t, int unit) {
  return t.ptr != nullptr && aligned(t.ptr, 16) && t.sb >= 0 && t.sn >= 0 && t.sh >= 0 && t.sb % unit == 0 &&
         t.sn % unit == 0 && t.sh % unit == 0;
}

// The checks that append and read share; DA_OK with *empty set for no rows.
da_status check_rows(int B, int N, int h_kv, int d, int L_max, const da_t4& k, const da_t4& v, const da_t4& cache,
                     const int* start, const int* counts, bool* empty) {
  *empty = false;
  if (B < 0 || N < 0 || h_kv <= 0 || d <= 0 || L_max <= 0) return DA_ERR_INVALID_ARG;
  if (diffattn_kv4_record_bytes(d) == 0) return DA_ERR_UNSUPPORTED;
  if (!aligned(start, 4) || !aligned(counts, 4)) return DA_ERR_INVALID_ARG;
  if (B == 0 || N == 0) {
    *empty = true;
    return DA_OK;
  }
  if (!ok_t4(k, 8) || !ok_t4(v, 8) || !ok_t4(cache, 16)) return DA_ERR_INVALID_ARG;
  // a sequence's rows are counted in 32 bits
  if (static_cast<int64_t>(N) * h_kv > (1 << 29)) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// CTAs of the 4-bit decode: one per SM, or as many as the fullest batch has
// parts.  The lengths are on the device, so this is an upper bound.
int decode_grid(int B, int h_kv, int L_max, int sms) {
  const int64_t chunks = (static_cast<int64_t>(L_max) + da::kKv4ChunkKeys - 1) / da::kKv4ChunkKeys;
  const int64_t most = sms < da::kKv4MaxGrid ? sms : da::kKv4MaxGrid;
  return static_cast<int>(chunks * h_kv * B < most ? chunks * h_kv * B : most);
}

// Blocks (a cluster) that take a whole head and write its output themselves,
// 0 for the line of chunks that is cut over all warps: heads that all find SMs
// at once, and sequences of at most 1024 keys a block (512 where the SMs allow
// it, 2048 from 64 heads on).  With up to 8 query heads per KV head a block has
// 16 warps, so that is two chunks a warp (one, four); with more it has 8, and
// twice the chunks.  Not all SMs of a GPU are in groups of 4 or 8 that
// a cluster fits (36 clusters of 4 ran at once, 11.4 us for 2000 keys, and 37 in
// two turns, 20.9; 16 of 8 took 21.7 us for 8000 keys, 14.5 on the line), hence
// the shares below.  One launch instead of two, three with weights, and room for
// the scores only.  Called eagerly, own blocks and line: 8 heads of 1000 keys
// 11.7 and 14.3 us, of 2000 12.7 and 17.2, of 8000 16.5 and 16.6; 32 of 4000
// 14.9 and 17.3; with weights 8 of 2000 14.7 and 20.1, 32 of 4000 16.6 and 20.4.
// Replayed, where a launch less counts for less: 8 of 1000 9.6 and 9.0, of 2000
// 10.2 and 9.4, of 8000 12.8 and 13.0; 32 of 4000 12.3 and 15.6; 128 of 2000
// 13.5 and 18.8; 64 of 4096 21.3 and 18.4; with weights 8 of 2000 11.5 and 11.1,
// 32 of 4000 14.2 and 18.6.  These are for 8 query heads per KV head.  For 16 (d 128, replayed) the limits
// fit less well: 8 heads of 1000 keys 11.9 and 10.6 us, with weights 15.3 and
// 12.6; 64 of 2000 17.8 and 17.2, with weights 24.1 and 20.6; but 32 of 2000
// 11.9 and 16.0 (14.1 and 19.3), 128 of 2000 18.1 and 25.0 (24.4 and 29.9).
int own_blocks(int B, int h_kv, int L_max, int sms) {
  const int64_t heads = static_cast<int64_t>(B) * h_kv;
  if (heads <= sms && (L_max <= 1024 || (L_max <= 2048 && heads >= 64))) return 1;
  for (int keys = 512; keys <= 1024; keys *= 2)
    for (int n = 2; n <= 8; n *= 2)
      if (heads * n <= (n == 8 ? sms / 2 : n == 4 ? sms * 7 / 8 : sms) && L_max <= keys * n) return n;
  return 0;
}

// Blocks that take whole heads need room for the scores and the gate only; the
// others for a part per warp, or per chunk where there are fewer, and head.
struct DecodeSpace {
  size_t ml, parts, norm, scores, gate, total;  // offsets; the partial O rows are at 0
};
DecodeSpace decode_space(int B, int h, int h_kv, int d, int L_max, int gate_given, int weights, int sms) {
  const int64_t heads = static_cast<int64_t>(B) * h_kv;
  const bool own = own_blocks(B, h_kv, L_max, sms) != 0;
  const int64_t chunks = (static_cast<int64_t>(L_max) + da::kKv4ChunkKeys - 1) / da::kKv4ChunkKeys * heads;
  const int64_t warps = static_cast<int64_t>(decode_grid(B, h_kv, L_max, sms)) * da::kKv4MaxWarps;
  const size_t rows = own ? 0 : static_cast<size_t>((chunks < warps ? chunks : warps) + heads) * (2 * h / h_kv);
  DecodeSpace w;
  w.ml = align256(rows * d * sizeof(float));
  w.parts = w.ml + align256(rows * 2 * sizeof(float));
  w.norm = w.parts + (own ? 0 : align256(heads * sizeof(da::Kv4Parts)));
  w.scores = w.norm + (own ? 0 : align256(static_cast<size_t>(B) * 2 * h * sizeof(float2)));
  w.gate = w.scores + (weights ? align256(static_cast<size_t>(B) * 2 * h * L_max * sizeof(float)) : 0);
  w.total = w.gate + (gate_given ? 0 : align256(static_cast<size_t>(B) * h * sizeof(float)));
  return w;
}

struct EvictSpace {
  size_t len, dst, src, total;  // offsets; the move counts are at 0
  int max_moves;
};
EvictSpace evict_space(int B, int h_kv, int L_max, int keep, int sms) {
  const size_t units = static_cast<size_t>(B) * h_kv;
  EvictSpace w;
  // a head moves one row per slot below m that goes: at most min(m, L - m)
  w.max_moves = keep >= L_max ? 0 : (keep < L_max - keep ? keep : L_max - keep);
  w.len = align256(units * sizeof(int));
  w.dst = w.len + align256(static_cast<size_t>(B) * sizeof(int));
  const size_t listed = da::evict_moves_unlisted(units, L_max, sms) ? 0 : units * w.max_moves;
  w.src = w.dst + align256(listed * sizeof(int));
  w.total = w.src + align256(listed * sizeof(int));
  return w;
}

}  // namespace

extern "C" {

int diffattn_kv4_record_bytes(int d) { return d == 64 || d == 128 ? d + 16 : 0; }

da_status diffattn_kv4_append(const da_kv4_append_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  bool empty;
  const da_status chk =
      check_rows(p->B, p->N, p->h_kv, p->d, p->L_max, p->k, p->v, p->cache, p->start, p->counts, &empty);
  if (chk != DA_OK) return chk;
  if (!aligned(p->key_weights, 4) || !aligned(p->positions, 4) || !aligned(p->first_position, 4))
    return DA_ERR_INVALID_ARG;
  if (empty) return DA_OK;
  uint32_t* status;
  int sms;
  if (!da::device_handles(&status, &sms)) return DA_ERR_CUDA;
  const da::Kv4RowsArgs a{p->B, p->N, p->h_kv, p->d, p->L_max, p->k, p->v, p->cache, p->start, p->counts,
                          p->key_weights, p->positions, p->first_position, status, 0, 0};
  return cuda_status(da::launch_kv4_append(a, static_cast<cudaStream_t>(stream)));
}

da_status diffattn_kv4_read(const da_kv4_read_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  bool empty;
  const da_status chk =
      check_rows(p->B, p->N, p->h_kv, p->d, p->L_max, p->k_out, p->v_out, p->cache, p->start, p->counts, &empty);
  if (chk != DA_OK || empty) return chk;
  uint32_t* status;
  int sms;
  if (!da::device_handles(&status, &sms)) return DA_ERR_CUDA;
  const da::Kv4RowsArgs a{p->B, p->N, p->h_kv, p->d, p->L_max, p->k_out, p->v_out, p->cache, p->start, p->counts,
                          nullptr, nullptr, nullptr, status, 0, 0};
  return cuda_status(da::launch_kv4_read(a, static_cast<cudaStream_t>(stream)));
}

size_t diffattn_v2_decode_kv4_workspace_size(int B, int h, int h_kv, int d, int L_max, int gate_given, int weights) {
  if (B <= 0 || h <= 0 || h_kv <= 0 || d <= 0 || L_max <= 0) return 0;
  uint32_t* status;
  int sms = 152;
  if (!da::device_handles(&status, &sms)) sms = 152;
  return decode_space(B, h, h_kv, d, L_max, gate_given, weights, sms).total;
}

da_status diffattn_v2_decode_kv4(const da_v2_decode_kv4_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  // the checks of diffattn_v2_decode on what both take; the cache's own below
  da_v2_decode_params q{};
  q.B = p->B;
  q.h = p->h;
  q.h_kv = p->h_kv;
  q.d = p->d;
  q.L_max = p->L_max;
  q.d_model = p->d_model;
  q.q = p->q;
  q.k_cache = q.v_cache = p->cache;
  q.gate = p->gate;
  q.x = p->x;
  q.w_lambda = p->w_lambda;
  q.out = p->out;
  const da_status chk = da::check_v2_decode_args(&q);
  if (chk != DA_OK) return chk;
  if (!ok_t4(p->cache, 16) || !aligned(p->seqlens, 4)) return DA_ERR_INVALID_ARG;
  if (!aligned(p->weights_in, 4) || !aligned(p->weights_out, 4) || (p->weights_in && !p->weights_out))
    return DA_ERR_INVALID_ARG;
  if (p->gate == nullptr && (!aligned(p->x, 16) || !aligned(p->w_lambda, 16))) return DA_ERR_INVALID_ARG;
  // sequences and KV heads are grid dimensions; partials are numbered in 32 bits
  if (p->B > 65535 || p->h_kv > 65535 || static_cast<int64_t>(p->B) * p->h_kv > (1 << 28) || p->L_max > (1 << 30))
    return DA_ERR_UNSUPPORTED;
  uint32_t* status;
  int sms = 152;
  const bool device = da::device_handles(&status, &sms);
  if (!device) sms = 152;  // the workspace is checked first, as the size query would have it
  int grid = decode_grid(p->B, p->h_kv, p->L_max, sms);
  const DecodeSpace w =
      decode_space(p->B, p->h, p->h_kv, p->d, p->L_max, p->gate != nullptr, p->weights_out != nullptr, sms);
  if (w.total > 0 && (p->workspace == nullptr || p->workspace_bytes < w.total || !aligned(p->workspace, 256)))
    return DA_ERR_WORKSPACE;
  if (!device) return DA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  const float* gate = p->gate;
  if (gate == nullptr) {
    float* g = reinterpret_cast<float*>(ws + w.gate);
    const da::GateArgs ga{p->B, p->d_model, p->h, p->x, p->d_model, p->w_lambda, g, status};
    if (da::launch_gate(ga, s) != cudaSuccess) return DA_ERR_CUDA;
    gate = g;
  }
  // The gate projection takes 8 SMs for about 8 us (more from 65 sequences on).
  // Short work leaves them alone (64 x 2048 keys: 51 us on all SMs, 46 on the
  // others); long work takes them too, and the blocks that start there last get
  // a little less of it (64 x 5120, 34 chunks a warp: 83.5 and 82.4 us; x 7000:
  // 106.5 and 103.7; x 32768: 409 and 390, 396 with equal parts).
  const int64_t chunks = (static_cast<int64_t>(p->L_max) + da::kKv4ChunkKeys - 1) / da::kKv4ChunkKeys * p->h_kv * p->B;
  int late = 0;
  if (p->gate == nullptr && grid > sms - 8 && sms > 16) {
    if (chunks <= (p->B <= 64 ? 32LL : 48LL) * da::kKv4MaxWarps * sms)
      grid = sms - 8;
    else if (p->B <= 64)  // 8 CTAs of gate.cu, a cluster
      late = 8;
  }
  const float scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.f / std::sqrt(static_cast<float>(p->d));
  const da::Kv4DecodeArgs a{p->B, p->h, p->h_kv, p->d, p->L_max, grid,
                            scale * kLog2e, p->q, p->cache, p->seqlens, gate, p->out,
                            reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + w.ml),
                            reinterpret_cast<da::Kv4Parts*>(ws + w.parts),
                            p->weights_out ? reinterpret_cast<float2*>(ws + w.norm) : nullptr,
                            p->weights_out ? reinterpret_cast<float*>(ws + w.scores) : nullptr,
                            p->weights_in, p->weights_out, status, p->gate == nullptr,
                            own_blocks(p->B, p->h_kv, p->L_max, sms), late};
  return cuda_status(da::launch_kv4_decode(a, s));
}

size_t diffattn_kv_evict_workspace_size(int B, int h_kv, int L_max, int keep) {
  if (B <= 0 || h_kv <= 0 || L_max <= 0 || keep <= 0) return 0;
  uint32_t* status;
  int sms = 152;
  if (!da::device_handles(&status, &sms)) sms = 152;
  return evict_space(B, h_kv, L_max, keep, sms).total;
}

da_status diffattn_kv_evict(const da_kv_evict_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  if (p->B < 0 || p->h_kv <= 0 || p->L_max <= 0) return DA_ERR_INVALID_ARG;
  if (p->keep < 1 || p->sinks < 0 || p->recent < 0 || p->sinks > p->keep - p->recent) return DA_ERR_INVALID_ARG;
  if (p->n_rows < 1 || p->n_rows > DIFFATTN_EVICT_MAX_ROWS) return DA_ERR_INVALID_ARG;
  if (p->B == 0) return DA_OK;
  if (!p->weights_in || !p->weights_out || !p->seqlens_out || (p->positions_in && !p->positions_out))
    return DA_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(p->weights_in), static_cast<const void*>(p->weights_out),
                        static_cast<const void*>(p->positions_in), static_cast<const void*>(p->positions_out),
                        static_cast<const void*>(p->seqlens), static_cast<const void*>(p->seqlens_out),
                        static_cast<const void*>(p->next_position)})
    if (!aligned(q, 4)) return DA_ERR_INVALID_ARG;
  for (int k = 0; k < p->n_rows; ++k)
    if (!ok_t4(p->rows[k], 16) || p->row_bytes[k] <= 0 || p->row_bytes[k] % 16) return DA_ERR_INVALID_ARG;
  // heads are a grid dimension, up to 8 CTAs each; a head's 16-byte pieces are counted in 32 bits
  if (static_cast<int64_t>(p->B) * p->h_kv > (1 << 24) || p->L_max > da::kEvictMaxSlots) return DA_ERR_UNSUPPORTED;
  for (int k = 0; k < p->n_rows; ++k)
    if (static_cast<int64_t>(p->L_max) * (p->row_bytes[k] / 16) > (1 << 30)) return DA_ERR_UNSUPPORTED;
  uint32_t* status;
  int sms = 152;
  const bool device = da::device_handles(&status, &sms);
  if (!device) sms = 152;  // the workspace is checked first, as the size query would have it
  const EvictSpace w = evict_space(p->B, p->h_kv, p->L_max, p->keep, sms);
  if (p->workspace == nullptr || p->workspace_bytes < w.total || !aligned(p->workspace, 256)) return DA_ERR_WORKSPACE;
  if (!device) return DA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  const da::EvictArgs a{*p, reinterpret_cast<int*>(ws), reinterpret_cast<int*>(ws + w.len),
                        reinterpret_cast<int*>(ws + w.dst), reinterpret_cast<int*>(ws + w.src), w.max_moves, status, sms};
  return cuda_status(da::launch_kv_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
