// rope_api.cu — the extern "C" entry points of the norm and rotation of queries
// and keys and of the append to a paged cache: argument checks and launches.  As
// in api.cu, nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <cmath>

#include "diffattn.h"
#include "kernels.h"

namespace {

constexpr int kMostTokens = 1 << 29;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
da_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DA_OK : DA_ERR_CUDA; }

// A tensor whose rows are read and written in 16-byte pieces, `unit` elements each.
bool ok_t4(const da_t4& t, int unit) {
  return t.ptr != nullptr && aligned(t.ptr, 16) && t.sb >= 0 && t.sn >= 0 && t.sh >= 0 && t.sb % unit == 0 &&
         t.sn % unit == 0 && t.sh % unit == 0;
}
bool ok_t3(const da_t3& t) { return ok_t4(da_t4{t.ptr, 0, t.st, t.sh}, 8); }
da_t4 as_t4(const da_t3& t) { return da_t4{t.ptr, 0, t.st, t.sh}; }

// The rotation's and the norm's arguments.
da_status check_rope(int d, int rot_dim, const float* inv_freq, float rope_scale, int norm, float norm_eps,
                     const float* q_weight, const float* k_weight, const int* positions) {
  if (rot_dim < 0 || rot_dim > d) return DA_ERR_INVALID_ARG;
  if (rot_dim % 8) return DA_ERR_UNSUPPORTED;
  if (rot_dim > 0 && (inv_freq == nullptr || !aligned(inv_freq, 4) || !std::isfinite(rope_scale))) return DA_ERR_INVALID_ARG;
  if (norm && (!(norm_eps >= 0.f) || !aligned(q_weight, 4) || !aligned(k_weight, 4))) return DA_ERR_INVALID_ARG;
  return aligned(positions, 4) ? DA_OK : DA_ERR_INVALID_ARG;
}

// The checks of the forward and the backward up to their tensors; *empty for no rows.
da_status check_qk(const da_qk_rope_fwd_params* p, bool* empty) {
  if (p->B < 0 || p->N < 0 || p->h_q < 0 || p->h_k < 0 || p->d <= 0) return DA_ERR_INVALID_ARG;
  if (p->dtype != DA_F32 && p->dtype != DA_BF16) return DA_ERR_INVALID_ARG;
  if (p->d != 16 && p->d != 32 && p->d != 64 && p->d != 128) return DA_ERR_UNSUPPORTED;
  const da_status chk = check_rope(p->d, p->rot_dim, p->inv_freq, p->rope_scale, p->norm, p->norm_eps, p->q_weight,
                                   p->k_weight, p->positions);
  if (chk != DA_OK) return chk;
  // tokens, a token's heads and the shares of them are counted in 32 bits
  if (static_cast<int64_t>(p->B) * p->N > kMostTokens || p->h_q > (1 << 24) || p->h_k > (1 << 24)) return DA_ERR_UNSUPPORTED;
  *empty = p->B == 0 || p->N == 0 || (p->h_q == 0 && p->h_k == 0);
  return DA_OK;
}

da::RopeKind rows(int heads, const da_t4& src, const da_t4& dst, const float* weight) {
  da::RopeKind k{};
  k.heads = heads;
  k.src = src;
  k.dst = dst;
  k.weight = weight;
  return k;
}

da::RopeArgs rope_args(const da_qk_rope_fwd_params* p, const da_t4& q_to, const da_t4& k_to) {
  da::RopeArgs a{};
  a.tokens = static_cast<int64_t>(p->B) * p->N;
  a.N = p->N;
  a.rot = p->rot_dim;
  a.interleaved = p->interleaved != 0;
  a.norm = p->norm != 0;
  a.rope_scale = p->rope_scale;
  a.norm_eps = p->norm_eps;
  a.inv_freq = p->inv_freq;
  a.positions = p->positions;
  a.kind[0] = rows(p->h_q, p->q, q_to, p->q_weight);
  a.kind[1] = rows(p->h_k, p->k, k_to, p->k_weight);
  return a;
}

}  // namespace

extern "C" {

da_status diffattn_rope_inv_freq(int rot_dim, double base, da_rope_stretch stretch, double factor, int trained_len,
                                 float* inv_freq, float* rope_scale) {
  if (rot_dim <= 0 || rot_dim % 8 || !(base > 1.0) || !std::isfinite(base) || inv_freq == nullptr || rope_scale == nullptr)
    return DA_ERR_INVALID_ARG;
  const bool stretched = stretch != DA_ROPE_NONE;
  if (stretch != DA_ROPE_NONE && stretch != DA_ROPE_LINEAR && stretch != DA_ROPE_BASE && stretch != DA_ROPE_RAMP)
    return DA_ERR_INVALID_ARG;
  if (stretched && (!(factor >= 1.0) || !std::isfinite(factor))) return DA_ERR_INVALID_ARG;
  if (stretch == DA_ROPE_RAMP && trained_len <= 0) return DA_ERR_INVALID_ARG;
  if (stretch == DA_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (stretch == DA_ROPE_LINEAR) f /= factor;
    if (stretch == DA_ROPE_RAMP) {
      const double turns = trained_len * f / 6.283185307179586;
      const double keep = std::fmin(std::fmax((turns - 1.0) / 31.0, 0.0), 1.0);
      f = f * keep + f / factor * (1.0 - keep);
    }
    inv_freq[i] = static_cast<float>(f);
  }
  *rope_scale = stretch == DA_ROPE_RAMP ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return DA_OK;
}

da_status diffattn_qk_rope_fwd(const da_qk_rope_fwd_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  bool empty = false;
  const da_status chk = check_qk(p, &empty);
  if (chk != DA_OK || empty) return chk;
  const int unit = p->dtype == DA_BF16 ? 8 : 4;
  if (p->h_q > 0 && (!ok_t4(p->q, unit) || !ok_t4(p->q_out, unit))) return DA_ERR_INVALID_ARG;
  if (p->h_k > 0 && (!ok_t4(p->k, unit) || !ok_t4(p->k_out, unit))) return DA_ERR_INVALID_ARG;
  uint32_t* status;
  int sms;
  if (!da::device_handles(&status, &sms)) return DA_ERR_CUDA;
  return cuda_status(da::launch_rope_fwd(rope_args(p, p->q_out, p->k_out), p->d, p->dtype == DA_F32, sms, static_cast<cudaStream_t>(stream)));
}

size_t diffattn_qk_rope_bwd_workspace_size(int B, int N, int h_q, int h_k, int d) {
  if (B <= 0 || N <= 0 || h_q < 0 || h_k < 0 || d <= 0) return 0;
  uint32_t* status;
  int sms = 152;
  if (!da::device_handles(&status, &sms)) sms = 152;
  // the sums of every block that the grid can have
  return align256(static_cast<size_t>(sms) * da::kRopeBlocksPerSm * 2 * d * sizeof(float));
}

da_status diffattn_qk_rope_bwd(const da_qk_rope_bwd_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  bool empty = false;
  const da_status chk = check_qk(&p->fwd, &empty);
  if (chk != DA_OK) return chk;
  const bool weights = p->dq_weight != nullptr || p->dk_weight != nullptr;
  if (weights && (!p->fwd.norm || !aligned(p->dq_weight, 4) || !aligned(p->dk_weight, 4))) return DA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) {
    for (float* w : {p->dq_weight, p->dk_weight})
      if (w != nullptr && cudaMemsetAsync(w, 0, p->fwd.d * sizeof(float), s) != cudaSuccess) return DA_ERR_CUDA;
    return DA_OK;
  }
  const int unit = p->fwd.dtype == DA_BF16 ? 8 : 4;
  if (p->fwd.h_q > 0 && (!ok_t4(p->dq_out, unit) || !ok_t4(p->dq, unit) || (p->fwd.norm && !ok_t4(p->fwd.q, unit))))
    return DA_ERR_INVALID_ARG;
  if (p->fwd.h_k > 0 && (!ok_t4(p->dk_out, unit) || !ok_t4(p->dk, unit) || (p->fwd.norm && !ok_t4(p->fwd.k, unit))))
    return DA_ERR_INVALID_ARG;
  const size_t need =
      weights ? diffattn_qk_rope_bwd_workspace_size(p->fwd.B, p->fwd.N, p->fwd.h_q, p->fwd.h_k, p->fwd.d) : 0;
  if (need && (p->workspace == nullptr || p->workspace_bytes < need || !aligned(p->workspace, 256))) return DA_ERR_WORKSPACE;
  uint32_t* status;
  int sms;
  if (!da::device_handles(&status, &sms)) return DA_ERR_CUDA;
  const da::RopeBwdArgs g{rope_args(&p->fwd, p->dq, p->dk), p->dq_out, p->dk_out,
                          weights ? static_cast<float*>(p->workspace) : nullptr, p->dq_weight, p->dk_weight};
  return cuda_status(da::launch_rope_bwd(g, p->fwd.d, p->fwd.dtype == DA_F32, sms, s));
}

da_status diffattn_paged_append(const da_paged_append_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  da_status chk = da::check_paged_cache(p->cache);
  if (chk != DA_OK) return chk;
  const int d = p->cache.d;
  chk = check_rope(d, p->rot_dim, p->inv_freq, p->rope_scale, p->norm, p->norm_eps, p->q_weight, p->k_weight, p->positions);
  if (chk != DA_OK) return chk;
  if (p->h_q < 0) return DA_ERR_INVALID_ARG;
  if (p->h_q > (1 << 24) || p->cache.h_kv > (1 << 24) || p->cache.T > kMostTokens) return DA_ERR_UNSUPPORTED;
  if (p->cache.T == 0 || p->cache.B == 0) return DA_OK;
  if (!da::paged_cache_given(p->cache) || !ok_t3(p->k) || !ok_t3(p->v)) return DA_ERR_INVALID_ARG;
  if (p->h_q > 0 && (!ok_t3(p->q) || !ok_t3(p->q_out))) return DA_ERR_INVALID_ARG;
  uint32_t* status;
  int sms;
  if (!da::device_handles(&status, &sms)) return DA_ERR_CUDA;
  da::RopeArgs a{};
  a.tokens = p->cache.T;
  a.rot = p->rot_dim;
  a.interleaved = p->interleaved != 0;
  a.norm = p->norm != 0;
  a.rope_scale = p->rope_scale;
  a.norm_eps = p->norm_eps;
  a.inv_freq = p->inv_freq;
  a.positions = p->positions;
  a.kind[0] = rows(p->h_q, as_t4(p->q), as_t4(p->q_out), p->q_weight);
  a.kind[1] = rows(p->cache.h_kv, as_t4(p->k), p->cache.k_pages, p->k_weight);
  a.kind[2] = rows(p->cache.h_kv, as_t4(p->v), p->cache.v_pages, nullptr);
  a.cache = p->cache;
  a.status = status;
  return cuda_status(da::launch_paged_append(a, d, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// Sizes and types of a paged cache.
da_status da::check_paged_cache(const da_paged_cache& c) {
  if (c.B < 0 || c.T < 0 || c.h_kv <= 0 || c.d <= 0 || c.page_size <= 0 || c.n_pages < 0 || c.max_pages < 0)
    return DA_ERR_INVALID_ARG;
  if (c.d != 64 && c.d != 128) return DA_ERR_UNSUPPORTED;
  // sequences are counted in 32 bits, a block's threads of them a step
  if (c.B > (1 << 30) || static_cast<int64_t>(c.max_pages) * c.page_size > (1 << 30) ||
      static_cast<int64_t>(c.B) * c.max_pages > (int64_t(1) << 31) - 1)
    return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// Its pointers and strides.
bool da::paged_cache_given(const da_paged_cache& c) {
  if (!c.cu_seqlens || !aligned(c.cu_seqlens, 4) || !c.seqlens || !aligned(c.seqlens, 4)) return false;
  if (c.max_pages > 0 && (!c.block_table || !aligned(c.block_table, 4))) return false;
  return c.n_pages == 0 || (ok_t4(c.k_pages, 8) && ok_t4(c.v_pages, 8));
}
