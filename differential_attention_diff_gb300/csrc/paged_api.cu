// paged_api.cu — the extern "C" entry points of the V2 attention over a paged
// cache: argument checks, the choice of its shares, workspace carving and the
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

// Strides that TMA copies can take: 16-byte multiples, above 0 where they are used.
bool ok_stride(int64_t stride, int64_t extent) { return extent <= 1 || (stride > 0 && stride % 8 == 0); }

// How a call's work is cut (paged.cuh), and by which kernel: sequences whose new
// tokens fit the columns of the kernel for few tokens read their keys once there;
// with more the 128-row tiles pay.
struct Cut {
  int tq, tq1, rows, grid, turns;
  bool few;
};
Cut cut(int T, int max_new, int G, int h_kv, int sms) {
  Cut c;
  c.turns = 1;
  const int64_t cols = static_cast<int64_t>(max_new > 0 && max_new < T ? max_new : T) * G;
  c.few = cols <= da::kPagedDecodeCols;
  if (c.few) {
    c.rows = cols <= 8 ? 8 : cols <= 16 ? 16 : 32;
    c.tq = c.tq1 = c.rows / G;
  } else {
    c.tq1 = 128 / G;
    c.tq = 2 * c.tq1;
    c.rows = 256;
    // a long prompt's chunk reads its keys for many items, four and more to a CTA:
    // room for finer shares, which the lengths, on the device, decide on
    if (static_cast<int64_t>(T) / c.tq * h_kv >= 4 * static_cast<int64_t>(sms)) c.turns = da::kPagedMaxTurns;
  }
  c.grid = sms;
  return c;
}

struct Space {
  size_t ml, desc, gate, total;  // offsets; the parts' outputs are at 0
};
Space space(const Cut& c, int T, int h, int d, int gate_given) {
  Space w;
  const size_t rows = static_cast<size_t>(2) * c.grid * c.turns * c.rows;
  w.ml = align256(rows * d * sizeof(float));
  w.desc = w.ml + align256(rows * 2 * sizeof(float));
  w.gate = w.desc + align256(static_cast<size_t>(c.grid) * c.turns * sizeof(da::PagedDesc));
  w.total = w.gate + (gate_given ? 0 : align256(static_cast<size_t>(T) * h * sizeof(float)));
  return w;
}

}  // namespace

extern "C" {

size_t diffattn_v2_paged_fwd_workspace_size(int T, int B, int max_new, int h, int h_kv, int d, int gate_given) {
  if (T <= 0 || B <= 0 || h <= 0 || h_kv <= 0 || d <= 0 || (2 * static_cast<int64_t>(h)) % h_kv) return 0;
  const int64_t G = 2 * static_cast<int64_t>(h) / h_kv;
  if (G > 128 || max_new < 0) return 0;
  uint32_t* status;
  int sms = 152;
  if (!da::device_handles(&status, &sms)) sms = 152;
  return space(cut(T, max_new, static_cast<int>(G), h_kv, sms), T, h, d, gate_given).total;
}

da_status diffattn_v2_paged_fwd(const da_v2_paged_fwd_params* p, void* stream) {
  if (p == nullptr) return DA_ERR_INVALID_ARG;
  const da_paged_cache& c = p->cache;
  const da_status chk = da::check_paged_cache(c);
  if (chk != DA_OK) return chk;
  if (p->h <= 0 || p->max_new < 0 || (2 * static_cast<int64_t>(p->h)) % c.h_kv) return DA_ERR_INVALID_ARG;
  const int64_t G = 2 * static_cast<int64_t>(p->h) / c.h_kv;
  if (G % 2) return DA_ERR_INVALID_ARG;  // a pair must sit in one K/V group
  // a CTA passes over empty sequences one at a time while others of its warps wait
  // for the next tile: 2^20 of them stay well within those waits' limit
  if (c.B > (1 << 20)) return DA_ERR_UNSUPPORTED;
  if (G > 128 || c.page_size % 16 || c.h_kv > 65535 || static_cast<int64_t>(c.T) * 2 * p->h > (int64_t(1) << 31) - 1)
    return DA_ERR_UNSUPPORTED;
  if (c.T == 0 || c.B == 0) return DA_OK;
  if (c.n_pages == 0 || c.max_pages == 0 || !da::paged_cache_given(c)) return DA_ERR_INVALID_ARG;
  for (const da_t4* t : {&c.k_pages, &c.v_pages})
    if (!ok_stride(t->sb, c.n_pages) || !ok_stride(t->sn, c.page_size) || !ok_stride(t->sh, c.h_kv)) return DA_ERR_INVALID_ARG;
  // a head's place in a page is counted in blocks of 64 features
  if (c.h_kv > 1 && (c.k_pages.sh % 64 || c.v_pages.sh % 64)) return DA_ERR_UNSUPPORTED;
  for (const da_t3* t : {&p->q, &p->out})
    if (t->ptr == nullptr || !aligned(t->ptr, 16) || !ok_stride(t->st, c.T) || !ok_stride(t->sh, 2)) return DA_ERR_INVALID_ARG;
  if (p->gate == nullptr) {
    if (!p->x || !p->w_lambda || p->d_model <= 0 || !aligned(p->x, 16) || !aligned(p->w_lambda, 16)) return DA_ERR_INVALID_ARG;
    if ((p->d_model % 64) || p->h > 64) return DA_ERR_UNSUPPORTED;
  } else if (!aligned(p->gate, 4)) {
    return DA_ERR_INVALID_ARG;
  }
  uint32_t* status;
  int sms = 152;
  const bool device = da::device_handles(&status, &sms);
  if (!device) sms = 152;  // the workspace is checked first, as the size query would have it
  const Cut k = cut(c.T, p->max_new, static_cast<int>(G), c.h_kv, sms);
  const Space w = space(k, c.T, p->h, c.d, p->gate != nullptr);
  if (p->workspace == nullptr || p->workspace_bytes < w.total || !aligned(p->workspace, 256)) return DA_ERR_WORKSPACE;
  if (!device || !da::tma_available()) return DA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  const float* gate = p->gate;
  if (gate == nullptr) {
    float* g = reinterpret_cast<float*>(ws + w.gate);
    const da::GateArgs ga{c.T, p->d_model, p->h, p->x, p->d_model, p->w_lambda, g, status};
    if (da::launch_gate(ga, s) != cudaSuccess) return DA_ERR_CUDA;
    gate = g;
  }
  const float scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.f / std::sqrt(static_cast<float>(c.d));
  da::PagedArgs a{};
  a.cache = c;
  a.h = p->h;
  a.G = static_cast<int>(G);
  a.tq = k.tq;
  a.tq1 = k.tq1;
  a.box = 16;
  while (a.box < 128 && c.page_size % (2 * a.box) == 0) a.box *= 2;
  a.scale_log2 = scale * kLog2e;
  a.q = p->q;
  a.out = p->out;
  a.gate = gate;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml);
  a.desc = reinterpret_cast<da::PagedDesc*>(ws + w.desc);
  a.rows = k.rows;
  a.part_row = k.few ? c.d : 4;
  a.part_group = k.few ? 4 : 4 * k.rows;
  // finer shares only where the keys and values that there can be do not fit L2
  const int64_t bytes = static_cast<int64_t>(c.B) * c.max_pages * c.page_size * c.h_kv * c.d * 4;
  a.turns = bytes >= (int64_t(96) << 20) ? k.turns : 1;
  a.grid = k.grid;
  a.status = status;
  a.after_gate = p->gate == nullptr;
  return cuda_status(k.few ? da::launch_paged_decode(a, s) : da::launch_paged_fwd(a, s));
}

}  // extern "C"
