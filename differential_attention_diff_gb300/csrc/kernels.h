// kernels.h — internal launch interface between api.cu (argument checks,
// workspace carving, stream handling) and the kernel translation units.
// Every launcher returns a cudaError_t from the launch itself.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "diffattn.h"
#include "kv4.cuh"

namespace da {

// ---- V2 gate: gate[t, p] = sigmoid(x[t, :] . w[:, p]) ---------------------
struct GateArgs {
  int T, d_model, h;
  const void* x;
  int64_t x_stride;
  const void* w;
  float* gate;
  uint32_t* status;  // device status word for bounded waits (may be null)
};
cudaError_t launch_gate(const GateArgs& a, cudaStream_t s);
// dX = dz W^T of the gate projection on tensor cores (gate_grads.cu), for
// T >= 128, h <= 64 with h % 8 == 0, d_model % 64 == 0
bool gate_dx_tc_ok(int T, int d_model, int h);
// partial sums of dW = X^T dz per chunk of chunk_tokens tokens (a multiple of
// 64) on tensor cores, part = fp32 [chunks][d_model][h]; for T >= 64, h <= 64
// with h % 8 == 0, d_model % 128 == 0
bool gate_dw_tc_ok(int T, int d_model, int h);
cudaError_t launch_gate_dw_tc(int T, int d_model, int h, int chunk_tokens, int chunks, const float* dz, const void* X,
                              float* part, uint32_t* status, cudaStream_t s);
cudaError_t launch_gate_dx_tc(int T, int d_model, int h, const float* dz, const void* W, void* dx, uint32_t* status,
                              cudaStream_t s);

// ---- V2 decode: split-KV partials, then merge + even/odd gate ------------
struct DecodeArgs {
  int B, h, h_kv, d, L_max, num_splits;
  float scale_log2;  // softmax scale * log2(e)
  const void* q;
  da_t4 k, v;
  const int* seqlens;
  const float* gate;  // [B, h]
  void* out;          // bf16 [B, h, d]
  float* part_o;      // [splits, B, 2h, d]
  float* part_ml;     // [splits, B, 2h, 2]  (running max in log2 units, sum)
  uint32_t* status;
  float* scores;      // [B, h_kv, L_max, G] scaled scores in log2 units, or null
  bool after_gate;    // the kernel launched just before is this call's gate (used with scores)
};
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
// The split count is a grid dimension (at most 65535).
constexpr int kMaxDecodeSplits = 65535;
// Every argument check of diffattn_v2_decode except the split count chosen
// by the library and the workspace; DA_OK or the status the call returns.
da_status check_v2_decode_args(const da_v2_decode_params* p);

// ---- device handles shared by the entry points ------------------------------
// The current device's status word and SM count; false if they cannot be had.
bool device_handles(uint32_t** status, int* num_sms);

// Launches a kernel that may start before the one launched just before it has
// ended (programmatic stream serialization): it waits for that one's end itself
// (cudaGridDependencySynchronize) before it reads what that one writes, or
// before its own end.  With `cluster` blocks to a cluster, along x.
template <class... P, class... A>
cudaError_t launch_clustered(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool ahead,
                             unsigned cluster, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  if (ahead) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
template <class... P, class... A>
cudaError_t launch_ahead(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool ahead, A... args) {
  return launch_clustered(kernel, grid, block, smem, s, ahead, 1, args...);
}

// Runs a set-up call (a kernel attribute, say) once on each device: with its
// result on the first call there, cudaSuccess on later ones.
class OncePerDevice {
 public:
  template <class F>
  cudaError_t run(F&& f) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done_.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t r = f();
    if (r == cudaSuccess && dev < 64) done_.fetch_or(bit, std::memory_order_release);
    return r;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// ---- 4-bit KV cache: append and read back -----------------------------------
struct Kv4RowsArgs {
  int B, N, h_kv, d, L_max;
  da_t4 k, v;      // bf16 [B, N, h_kv, d]: read by append, written by read
  da_t4 cache;     // records [B, L_max, h_kv], byte strides
  const int* start;
  const int* counts;
  float* key_weights;
  int* positions;
  const int* first_position;
  uint32_t* status;
  int step_i, step_g;  // a pass of rows onward, in tokens and heads (set by the launchers)
};
cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s);

// ---- V2 decode over a 4-bit KV cache ----------------------------------------
struct Kv4DecodeArgs {
  int B, h, h_kv, d, L_max;
  int grid;           // CTAs that share the work
  float scale_log2;
  const void* q;
  da_t4 cache;        // records [B, L_max, h_kv], byte strides
  const int* seqlens;
  const float* gate;  // [B, h]
  void* out;          // bf16 [B, h, d]
  float* part_o;      // [grid * warps + B * h_kv, G, d] (numbered as in kv4.cuh)
  float* part_ml;     // [grid * warps + B * h_kv, G, 2]
  Kv4Parts* parts;    // [B * h_kv]
  float2* norm;       // [B, 2h] each head's maximum and 1 / sum, or null
  float* scores;      // [B, h_kv, L_max, G] scaled scores in log2 units, or null
  const float* weights_in;
  float* weights_out;
  uint32_t* status;
  bool after_gate;    // the kernel launched just before is this call's gate
  int own;            // blocks (a cluster) per head, no partials; 0: the work is cut over all heads
  int late_blocks;    // of the grid's end, which have to wait for the gate's SMs
};
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s);

// ---- the end of a decode that gathers the keys' weights -----------------------
struct FinishArgs {
  int B, h, h_kv, d, L_max;
  int splits;            // key-range splits, where norm is null
  const float2* norm;    // [B, 2h] each head's maximum and 1 / sum, or null: taken from part_ml
  const int* seqlens;
  const float* gate;
  const float* part_o;   // [splits, B, 2h, d]
  const float* part_ml;  // [splits, B, 2h, 2]
  const float* scores;   // [B, h_kv, L_max, G]
  const float* weights_in;
  float* weights_out;
  void* out;             // bf16 [B, h, d]: merged too, or null
};
cudaError_t launch_decode_finish(const FinishArgs& a, cudaStream_t s);

// ---- eviction from a cache -----------------------------------------------------
constexpr int kEvictMaxSlots = 1 << 20;  // of a head: 8 slices whose masks fit shared memory beside their ranks
struct EvictArgs {
  da_kv_evict_params p;
  int* n_moves;  // [B * h_kv]
  int* new_len;  // [B]
  int* dst;      // [B * h_kv, max_moves], but for evict_moves_unlisted
  int* src;
  int max_moves;
  uint32_t* status;
  int num_sms;
};
cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s);
// Whether every head's own block moves its rows, whatever they are: no lists in memory.
bool evict_moves_unlisted(int64_t units, int L_max, int sms);

// ---- queries and keys normed and rotated; append to a paged cache ---------------
// Rows of one kind: queries, keys, or (paged) values, which are copied.
struct RopeKind {
  int heads;
  da_t4 src, dst;          // paged: of the packed rows sb is unused, sn the token's stride; k and v go to the pages
  const float* weight;
  // set by the launchers: passes over a token's heads, and in how many shares (units)
  int passes, chunk_passes, chunks;
  uint32_t unit0;          // the kind's first unit
};
struct RopeArgs {
  int64_t tokens;
  int N;                   // tokens are [B, N] (not paged)
  int rot, interleaved, norm;
  float rope_scale, norm_eps;
  const float* inv_freq;
  const int* positions;
  RopeKind kind[3];
  uint32_t units;          // of all kinds (set by the launchers)
  da_paged_cache cache;    // paged
  uint32_t* status;
};
struct RopeBwdArgs {
  RopeArgs a;              // kind[].dst: the gradients to write
  da_t4 dq_out, dk_out;
  float* part;             // [blocks, 2, d] sums of the weights' gradients, or null
  float *dq_weight, *dk_weight;
};
constexpr int kRopeBlocksPerSm = 2;  // of the grid at most
cudaError_t launch_rope_fwd(const RopeArgs& a, int d, bool f32, int sms, cudaStream_t s);
cudaError_t launch_rope_bwd(const RopeBwdArgs& g, int d, bool f32, int sms, cudaStream_t s);
// The checks of a paged cache: sizes and types, then pointers and strides (which
// an empty call need not give).
da_status check_paged_cache(const da_paged_cache& c);
bool paged_cache_given(const da_paged_cache& c);
cudaError_t launch_paged_append(const RopeArgs& a, int d, int sms, cudaStream_t s);

// ---- V2 attention over a paged cache --------------------------------------------
constexpr int kPagedMaxTurns = 4;  // shares of a CTA (paged.cuh)
struct PagedDesc {
  int flags;             // paged.cuh; the rest: the item that is begun and not ended
  int token, tokens, g;  // its rows of the packed arrays, its KV head
};
struct PagedArgs {
  da_paged_cache cache;
  int h, G;            // output heads, query heads per KV head
  int tq, tq1;         // tokens of an item, and of one of its MMA tiles
  int box;             // keys of a page that one TMA copy takes
  float scale_log2;
  da_t3 q, out;
  const float* gate;   // [T, h]
  float* part_o;       // [2 grid turns, rows, d] unnormalised outputs of the parts, d in
                       // groups of four: row r's group q at r * part_row + q * part_group
  float* part_ml;      // [2 grid turns, rows, 2] their maxima (log2 units) and sums
  PagedDesc* desc;     // [grid turns]
  int part_row, part_group;
  int turns;           // the most shares that a CTA may have
  int rows;            // of a part: 128 per MMA tile, or the columns of the kernel for few tokens
  int grid;
  uint32_t* status;
  bool after_gate;     // the kernel launched just before is this call's gate
};
constexpr int kPagedDecodeCols = 32;  // the most (token, query head) columns that the kernel for few tokens has
cudaError_t launch_paged_fwd(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t s);

// ---- V1 decode: split-KV partials of both streams, then merge + RMSNorm ----
struct V1DecodeArgs {
  int B, H, d_qk, d_v, L_max, num_splits;  // (d_qk, d_v) = (128, 256) or (64, 128)
  float scale_log2, lambda_init, rms_eps;
  const void* q1;  // bf16 [B, H, d_qk]
  const void* q2;
  da_t4 k1, k2, v;  // [B, L_max, H, d_qk | d_qk | d_v]
  const int* seqlens;
  const float *lq1, *lk1, *lq2, *lk2;
  void* out;       // bf16 [B, H, d_v]
  float* part_o;   // [splits, B, H, 2, d_v]
  float* part_ml;  // [splits, B, H, 2, 2]  (running max in log2 units, sum)
  uint32_t* status;
  const float* rms_weight;  // [d_v] or nullptr (unit)
};
cudaError_t launch_v1_decode(const V1DecodeArgs& a, cudaStream_t s);

// ---- V1 forward, fp32 SIMT path ------------------------------------------
struct V1F32Args {
  int B, N, H, d_qk, d_v, causal;
  float scale, lambda_init, rms_eps;
  da_t4 q1, q2, k1, k2, v, out, o2;
  const float *lq1, *lk1, *lq2, *lk2;
  float *lse1, *lse2, *rstd, *lambda_out;
  const float* rms_weight;  // [d_v] or nullptr (unit)
};
cudaError_t launch_v1_fwd_f32(const V1F32Args& a, cudaStream_t s);

// ---- V2 forward, tcgen05 -------------------------------------------------
struct V2FwdArgs {
  int B, N, h, h_kv, d, causal;
  float scale_log2;
  da_t4 q, k, v, out;
  const float* gate;  // [B, N, h]
  float* lse;         // optional [B, 2h, N] (natural log)
  da_t4 o_heads;      // optional [B, N, 2h, d] per-head outputs
  uint32_t* status;
  int num_sms;
  int fault;          // test hook: CTA 0 skips its first K tile load
};
cudaError_t launch_v2_fwd(const V2FwdArgs& a, cudaStream_t s);

// ---- grouped differential attention: combine per-head outputs -------------
struct GroupedArgs {
  int B, N, h, ratio;   // h output (signal) heads, ratio signal heads per noise head
  int d;                // head dim (a multiple of 8)
  da_t4 o_heads;        // [B, N, h (ratio + 1) / ratio, d] bf16
  const float* gate;    // [B, N, h]
  da_t4 out;            // [B, N, h, d] bf16
};
cudaError_t launch_grouped_combine(const GroupedArgs& a, cudaStream_t s);

// ---- V2 backward, bf16, tcgen05 --------------------------------------------
struct V2BwdArgs {
  int B, N, h, h_kv, d, d_model, causal;
  float scale;
  da_t4 q, k, v, o_heads, dout, dq, dk, dv;
  const float* gate;   // [B, N, h], or NULL: computed from x, w into the workspace
  const float* lse;    // [B, 2h, N] natural log
  const void* x;       // bf16 [B, N, d_model] (optional)
  const void* w;       // bf16 [d_model, h] (optional)
  float* dz;           // optional [B, N, h] output (else kept in the workspace)
  void* dx;            // optional bf16 [B, N, d_model]
  float* dw;           // optional fp32 [d_model, h]
  void* workspace;
  size_t workspace_bytes;
  uint32_t* status;
  int num_sms;
  // Grouped differential attention (ratio >= 2): the 2h query heads come in
  // groups of `ratio` signal heads and one noise head; dout, gate, dz, w and
  // dw have h_out = 2h ratio / (ratio + 1) output heads.  ratio <= 1 is V2
  // (h_out = h, even/odd pairs).
  int ratio;
  int h_out;
};
size_t v2_bwd_workspace_bytes(int B, int N, int h, int d_model);
// grouped: h_attn = Hq / 2 (half the query heads), h_out = the output heads
size_t grouped_bwd_workspace_bytes(int B, int N, int h_attn, int h_out, int d_model);
cudaError_t launch_v2_bwd(const V2BwdArgs& a, cudaStream_t s);

// ---- V1 forward, bf16, tcgen05 ---------------------------------------------
struct V1FwdArgs {
  int B, N, H, d_qk, d_v, causal;
  float scale_log2, lambda_init, rms_eps;
  da_t4 q1, q2, k1, k2, v, out, o2;
  const float *lq1, *lk1, *lq2, *lk2;
  float *lse1, *lse2, *rstd, *lambda_out;
  void* workspace;  // exchange slots of the CTA pairs
  size_t workspace_bytes;
  uint32_t* status;
  int num_sms;
  const float* rms_weight;  // [d_v] or nullptr (unit)
};
size_t v1_fwd_workspace_bytes(int num_sms);
cudaError_t launch_v1_fwd(const V1FwdArgs& a, cudaStream_t s);

// ---- V1 backward, bf16 -----------------------------------------------------
struct V1BwdArgs {
  int B, N, H, d_qk, d_v, causal;
  float scale, lambda_init, rms_eps;
  da_t4 q1, q2, k1, k2, v, out, dout, o2;
  const float *lq1, *lk1, *lq2, *lk2;
  const float *lse1, *lse2, *rstd;
  da_t4 dq1, dq2, dk1, dk2, dv;
  float *dlq1, *dlk1, *dlq2, *dlk2;
  void* workspace;
  size_t workspace_bytes;
  uint32_t* status;
  int num_sms;
  int deterministic;  // dQ through per-key-tile slots summed in a fixed order
  const float* rms_weight;  // [d_v] or nullptr (unit); entries nonzero
};
// deterministic dQ slots: the causal tile pairs when causal, all pairs otherwise
size_t v1_bwd_workspace_bytes(int B, int N, int H, int d_qk, int d_v, int deterministic, int causal);
cudaError_t launch_v1_bwd(const V1BwdArgs& a, cudaStream_t s);

// TMA descriptor encoding (driver entry point fetched through the runtime).
bool tma_available();

}  // namespace da
