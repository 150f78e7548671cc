// C-ABI entry points of the latent-row operators (include/sfa_grad.h):
// validation and launches of norm_rope, its gradient, the cache append and the
// paged attention, over rows of 16 and of 4 bits, and of the page plans.
#include <cmath>
#include <cstdio>

#include "sfa_grad.h"
#include "kernels.h"
#include "cache4.cuh"

namespace sfa {
namespace {

sfa_status fail(cudaError_t e, const char* what) {
  char msg[200];
  snprintf(msg, sizeof(msg), "%s (CUDA error %d) in %s", cudaGetErrorString(e), (int)e, what);
  set_last_error(msg);
  (void)cudaGetLastError();
  return SFA_ERR_RUNTIME;
}

// The kernels hold the scale, its product with log2(e) and eps in fp32.
bool fits(double x) { return std::isfinite(static_cast<float>(x)); }

bool aligned(const void* p, size_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
template <typename... Ts>
bool all_aligned(Ts... ps) {
  return (... && aligned(ps));
}
// int32 and fp32 arrays read and written by element
template <typename... Ts>
bool words_aligned(Ts... ps) {
  return (... && aligned(ps, 4));
}

sfa_status check_rows(const sfa_rows_params* p) {
  if (!p) return SFA_ERR_NULLPTR;
  if (p->dtype != SFA_DTYPE_BF16 && p->dtype != SFA_DTYPE_FP16) return SFA_ERR_PARAM_INVALID;
  if (p->interleaved != 0 && p->interleaved != 1) return SFA_ERR_PARAM_INVALID;
  if (p->N1 < 1 || p->N1 > 128 || p->T1 < 0 || p->T1 > INT32_MAX / 2 || p->T1 * p->N1 > INT32_MAX / 2)
    return SFA_ERR_SHAPE;
  if (p->table_len < 0 || p->table_len > INT32_MAX) return SFA_ERR_SHAPE;
  if (!fits(p->eps) || p->eps < 0) return SFA_ERR_SHAPE;
  return SFA_OK;
}

RowsArgs rows_args(const sfa_rows_params* p, const int32_t* pos, const float* cs) {
  RowsArgs a{};
  a.pos = pos;
  a.cs = cs;
  a.table_len = p->table_len;
  a.T = (int)p->T1;
  a.G = (int)p->N1;
  a.interleaved = p->interleaved;
  a.eps = (float)p->eps;
  return a;
}

// Sizes of the two paged calls.
sfa_status check_paged(const sfa_paged_params* p, Paged* out) {
  if (!p) return SFA_ERR_NULLPTR;
  if (p->dtype != SFA_DTYPE_BF16 && p->dtype != SFA_DTYPE_FP16) return SFA_ERR_PARAM_INVALID;
  if (p->layout != SFA_LAYOUT_BSND && p->layout != SFA_LAYOUT_TND) return SFA_ERR_PARAM_INVALID;
  if (p->interleaved != 0 && p->interleaved != 1) return SFA_ERR_PARAM_INVALID;
  if (p->wait_limit_us < 0) return SFA_ERR_PARAM_INVALID;
  if (p->D != 512 || (p->Dr != 64 && p->Dr != 0) || p->N1 < 1 || p->N1 > 128) return SFA_ERR_SHAPE;
  if (p->B < 1 || p->B > (1 << 20)) return SFA_ERR_SHAPE;
  if (p->page_size < 16 || p->page_size > 1024 || p->page_size % 16) return SFA_ERR_SHAPE;
  if (p->num_pages < 1 || p->num_pages > INT32_MAX / 2 / p->page_size) return SFA_ERR_SHAPE;
  if (p->max_pages < 1 || p->max_pages > INT32_MAX / 2 / p->page_size) return SFA_ERR_SHAPE;
  if (p->sparse_mode != 0 && p->sparse_mode != 3) return SFA_ERR_SHAPE;
  if (!fits(p->scale * 1.4426950408889634)) return SFA_ERR_SHAPE;
  const bool tnd = p->layout == SFA_LAYOUT_TND;
  const int64_t n = tnd ? p->T1 : p->S1;
  if (n < 0 || n > INT32_MAX / 2) return SFA_ERR_SHAPE;
  const int64_t T = tnd ? n : p->B * n;
  if (T > INT32_MAX / 2 || T * p->N1 > INT32_MAX / 2) return SFA_ERR_SHAPE;
  Paged g{};
  g.tnd = tnd;
  g.B = (int)p->B;
  g.S1 = tnd ? 0 : (int)p->S1;
  g.T = (int)T;
  g.G = (int)p->N1;
  g.row = (int)(p->D + p->Dr);
  g.num_pages = (int)p->num_pages;
  g.page_size = (int)p->page_size;
  g.max_pages = (int)p->max_pages;
  g.mode = (int)p->sparse_mode;
  *out = g;
  return SFA_OK;
}

// The axis of each rotated pair as two bits; axes null: all of them the first.
bool pack_axes(int32_t n, const uint8_t* axes, unsigned long long* map) {
  *map = 0;
  if (n < 1 || n > 4) return false;
  for (int i = 0; axes && i < 32; ++i) {
    if (axes[i] >= n) return false;
    *map |= (unsigned long long)axes[i] << (2 * i);
  }
  return true;
}

// The unit of a 4-bit cache as its exponent.
bool scale_exponent(double scale, int* k) {
  int e = 0;
  if (!std::isfinite(scale) || std::frexp(scale, &e) != 0.5) return false;
  *k = e - 1;
  return *k >= kScaleExpMin && *k <= kScaleExpMax;
}

sfa_status check_cache(const sfa_cache_params* p, Paged* g, int* k) {
  if (!p) return SFA_ERR_NULLPTR;
  if (p->dtype != SFA_DTYPE_BF16 && p->dtype != SFA_DTYPE_FP16) return SFA_ERR_PARAM_INVALID;
  if (p->bits != 16 && p->bits != 4) return SFA_ERR_PARAM_INVALID;
  if (p->Dr != 64 && p->Dr != 0) return SFA_ERR_SHAPE;
  if (p->page_size < 16 || p->page_size > 1024 || p->page_size % 16) return SFA_ERR_SHAPE;
  if (p->num_pages < 1 || p->num_pages > INT32_MAX / 2 / p->page_size) return SFA_ERR_SHAPE;
  *k = 0;
  if (p->bits == 4 && !scale_exponent(p->scale, k)) return SFA_ERR_SHAPE;
  *g = Paged{};
  g->row = (int)(512 + p->Dr);
  g->num_pages = (int)p->num_pages;
  g->page_size = (int)p->page_size;
  return SFA_OK;
}

sfa_status norm_rope(const sfa_rows_params* p, int32_t n_axes, const uint8_t* axes, const int32_t* positions,
                     const float* cos_sin, const void* q, const void* q_weight, const void* q_rope, const void* k,
                     const void* k_weight, const void* k_rope, void* q_out, void* q_rope_out, void* k_out,
                     void* k_rope_out, float* q_rstd, float* k_rstd, void* stream) {
  const sfa_status s = check_rows(p);
  if (s != SFA_OK) return s;
  unsigned long long map;
  if (!pack_axes(n_axes, axes, &map)) return SFA_ERR_PARAM_INVALID;
  if ((q && (!q_weight || !q_out)) || (k && (!k_weight || !k_out)) || (q_rope && !q_rope_out) ||
      (k_rope && !k_rope_out))
    return SFA_ERR_NULLPTR;
  if ((q_rope || k_rope || n_axes > 1) && (!positions || !cos_sin)) return SFA_ERR_NULLPTR;
  if ((q_rope || k_rope || n_axes > 1) && p->table_len < 1) return SFA_ERR_SHAPE;
  if (!all_aligned(cos_sin, q, q_weight, q_rope, k, k_weight, k_rope, q_out, q_rope_out, k_out, k_rope_out) ||
      !words_aligned(positions, q_rstd, k_rstd))
    return SFA_ERR_PARAM_INVALID;
  if (p->T1 == 0) return SFA_OK;
  RowsArgs a = rows_args(p, positions, cos_sin);
  a.axes = n_axes;
  a.axis_map = map;
  a.q = q; a.qw = q_weight; a.qr = q_rope; a.k = k; a.kw = k_weight; a.kr = k_rope;
  a.qo = q_out; a.qro = q_rope_out; a.ko = k_out; a.kro = k_rope_out;
  a.q_rstd = q_rstd; a.k_rstd = k_rstd;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == SFA_DTYPE_FP16 ? launch_norm_rope<__half>(a, st)
                                                   : launch_norm_rope<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_norm_rope");
}

sfa_status norm_rope_grad(const sfa_rows_params* p, int32_t n_axes, const uint8_t* axes, const int32_t* positions,
                          const float* cos_sin, const void* q, const void* q_weight, const float* q_rstd,
                          const void* k, const void* k_weight, const float* k_rstd, const void* d_q,
                          const void* d_q_rope, const void* d_k, const void* d_k_rope, void* dq, void* dq_rope,
                          void* dk, void* dk_rope, float* dq_weight, float* dk_weight, void* workspace,
                          size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const sfa_status s = sfa_norm_rope_grad_workspace_size(p, &need);
  if (s != SFA_OK) return s;
  unsigned long long map;
  if (!pack_axes(n_axes, axes, &map)) return SFA_ERR_PARAM_INVALID;
  if ((d_q && (!q || !q_weight || !q_rstd || !dq || !dq_weight)) ||
      (d_k && (!k || !k_weight || !k_rstd || !dk || !dk_weight)) || (d_q_rope && !dq_rope) ||
      (d_k_rope && !dk_rope))
    return SFA_ERR_NULLPTR;
  const bool rope = d_q_rope || d_k_rope || n_axes > 1;
  if (rope && (!positions || !cos_sin)) return SFA_ERR_NULLPTR;
  if ((d_q || d_k) && !workspace) return SFA_ERR_NULLPTR;
  if (rope && p->table_len < 1) return SFA_ERR_SHAPE;
  if (!all_aligned(cos_sin, q, q_weight, k, k_weight, d_q, d_q_rope, d_k, d_k_rope, dq, dq_rope, dk, dk_rope) ||
      !words_aligned(positions, q_rstd, k_rstd, dq_weight, dk_weight))
    return SFA_ERR_PARAM_INVALID;
  if ((d_q || d_k) && (workspace_bytes < need || !aligned(workspace, 256))) return SFA_ERR_PARAM_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (p->T1 == 0) {
    // no token: the weights' gradients are empty sums
    if (d_q) e = cudaMemsetAsync(dq_weight, 0, 512 * sizeof(float), st);
    if (d_k && e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, 512 * sizeof(float), st);
    return e == cudaSuccess ? SFA_OK : fail(e, "sfa_norm_rope_grad");
  }
  RowsArgs a = rows_args(p, positions, cos_sin);
  a.axes = n_axes;
  a.axis_map = map;
  a.q = q; a.qw = q_weight; a.k = k; a.kw = k_weight;
  a.q_rstd = const_cast<float*>(q_rstd);
  a.k_rstd = const_cast<float*>(k_rstd);
  a.dq = d_q; a.dk = d_k; a.qr = d_q_rope; a.kr = d_k_rope;
  a.qo = dq; a.ko = dk; a.qro = dq_rope; a.kro = dk_rope;
  a.dqw = dq_weight; a.dkw = dk_weight;
  a.part = static_cast<float*>(workspace);
  int nsm = device_sm_count();
  if (nsm > kMaxSms) nsm = kMaxSms;
  e = p->dtype == SFA_DTYPE_FP16 ? launch_norm_rope_grad<__half>(a, nsm, st)
                                 : launch_norm_rope_grad<__nv_bfloat16>(a, nsm, st);
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_norm_rope_grad");
}

// The rows that both forms of the append take, and its launch.
sfa_status append(AppendArgs a, bool f16, const void* k, const void* k_rope, const void* k_weight, double eps,
                  const float* cos_sin, int64_t table_len, const void* q_rope, void* q_rope_out, int32_t* error,
                  const char* what, void* stream) {
  const bool rope = a.pg.row == 576;
  if (!a.cache || !k) return SFA_ERR_NULLPTR;
  if (rope && (!k_rope || !cos_sin || (q_rope && !q_rope_out))) return SFA_ERR_NULLPTR;
  if (rope && (table_len < 1 || table_len > INT32_MAX)) return SFA_ERR_SHAPE;
  if (!fits(eps) || eps < 0) return SFA_ERR_SHAPE;
  if (!all_aligned(a.cache, k, k_rope, k_weight, cos_sin, q_rope, q_rope_out) ||
      !words_aligned(a.pg.table, a.pg.act_q, a.pg.act_kv, a.slots, a.pos, error))
    return SFA_ERR_PARAM_INVALID;
  a.k = k; a.kw = k_weight;
  a.kr = rope ? k_rope : nullptr;
  a.qr = rope ? q_rope : nullptr;
  a.qro = q_rope_out;
  a.cs = rope ? cos_sin : nullptr;
  a.table_len = table_len;
  a.error = error;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = f16 ? launch_append<__half>(a, st) : launch_append<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? SFA_OK : fail(e, what);
}

sfa_status append_by_table(const sfa_paged_params* p, const double* scale, void* cache, const int32_t* block_table,
                           const int32_t* act_seq_q, const int32_t* act_seq_kv, const void* k, const void* k_rope,
                           const void* k_weight, double eps, const float* cos_sin, int64_t table_len,
                           const void* q_rope, void* q_rope_out, int32_t* error, const char* what, void* stream) {
  AppendArgs a{};
  const sfa_status s = check_paged(p, &a.pg);
  if (s != SFA_OK) return s;
  a.packed = scale != nullptr;
  if (scale && !scale_exponent(*scale, &a.scale_exp)) return SFA_ERR_SHAPE;
  if (a.pg.T == 0) return SFA_OK;   // no new token: the tensors are empty, and may be null
  if (!block_table || !act_seq_kv || (a.pg.tnd && !act_seq_q)) return SFA_ERR_NULLPTR;
  a.pg.table = block_table;
  a.pg.act_q = act_seq_q;
  a.pg.act_kv = act_seq_kv;
  a.cache = cache;
  a.interleaved = p->interleaved;
  return append(a, p->dtype == SFA_DTYPE_FP16, k, k_rope, k_weight, eps, cos_sin, table_len, q_rope, q_rope_out,
                error, what, stream);
}

sfa_status paged_fwd(const sfa_paged_params* p, const double* scale, const void* q, const void* q_rope,
                     const void* cache, const int32_t* block_table, const int32_t* act_seq_q,
                     const int32_t* act_seq_kv, void* out, float* softmax_max, float* softmax_sum, void* workspace,
                     size_t workspace_bytes, const char* what, void* stream) {
  PagedArgs a{};
  const sfa_status s = check_paged(p, &a.pg);
  if (s != SFA_OK) return s;
  a.packed = scale != nullptr;
  if (scale && !scale_exponent(*scale, &a.scale_exp)) return SFA_ERR_SHAPE;
  const bool rope = p->Dr == 64;
  if (!workspace) return SFA_ERR_NULLPTR;
  if (!aligned(workspace, 256) || workspace_bytes < (scale ? paged4_workspace(a.pg) : paged_workspace(a.pg))) return SFA_ERR_PARAM_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.pg.T == 0) {
    // no query row: the tensors are empty, and may be null
    const cudaError_t e = cudaMemsetAsync(workspace, 0, 4, st);
    return e == cudaSuccess ? SFA_OK : fail(e, what);
  }
  if (!q || !cache || !block_table || !act_seq_kv || !out || !softmax_max || !softmax_sum ||
      (a.pg.tnd && !act_seq_q) || (rope && !q_rope))
    return SFA_ERR_NULLPTR;
  if (!all_aligned(q, rope ? q_rope : nullptr, cache, out) ||
      !words_aligned(block_table, act_seq_q, act_seq_kv, softmax_max, softmax_sum))
    return SFA_ERR_PARAM_INVALID;
  a.pg.table = block_table;
  a.pg.act_q = act_seq_q;
  a.pg.act_kv = act_seq_kv;
  a.q = q;
  a.qr = rope ? q_rope : nullptr;
  a.cache = cache;
  a.out = out;
  a.smax = softmax_max;
  a.ssum = softmax_sum;
  a.scale = (float)p->scale;
  a.wait_ns = p->wait_limit_us > 0 ? (unsigned long long)p->wait_limit_us * 1000ull : kWaitNsDefault;
  a.brief = a.wait_ns < 40000;   // four suspensions of at most 10 us
  a.ws = static_cast<uint8_t*>(workspace);
  int nsm = device_sm_count();
  if (nsm > kMaxSms) nsm = kMaxSms;
  const cudaError_t e = p->dtype == SFA_DTYPE_FP16 ? launch_paged<__half>(a, nsm, st)
                                                   : launch_paged<__nv_bfloat16>(a, nsm, st);
  return e == cudaSuccess ? SFA_OK : fail(e, what);
}

}  // namespace
}  // namespace sfa

using namespace sfa;

extern "C" {

sfa_status sfa_norm_rope(const sfa_rows_params* p, const int32_t* positions, const float* cos_sin, const void* q,
                         const void* q_weight, const void* q_rope, const void* k, const void* k_weight,
                         const void* k_rope, void* q_out, void* q_rope_out, void* k_out, void* k_rope_out,
                         float* q_rstd, float* k_rstd, void* stream) {
  return norm_rope(p, 1, nullptr, positions, cos_sin, q, q_weight, q_rope, k, k_weight, k_rope, q_out, q_rope_out,
                   k_out, k_rope_out, q_rstd, k_rstd, stream);
}

sfa_status sfa_norm_rope_axes(const sfa_rows_params* p, int32_t n_axes, const uint8_t* axes, const int32_t* positions,
                              const float* cos_sin, const void* q, const void* q_weight, const void* q_rope,
                              const void* k, const void* k_weight, const void* k_rope, void* q_out, void* q_rope_out,
                              void* k_out, void* k_rope_out, float* q_rstd, float* k_rstd, void* stream) {
  if (!axes) return SFA_ERR_NULLPTR;
  return norm_rope(p, n_axes, axes, positions, cos_sin, q, q_weight, q_rope, k, k_weight, k_rope, q_out, q_rope_out,
                   k_out, k_rope_out, q_rstd, k_rstd, stream);
}

sfa_status sfa_norm_rope_grad_workspace_size(const sfa_rows_params* p, size_t* bytes) {
  const sfa_status s = check_rows(p);
  if (s != SFA_OK) return s;
  if (!bytes) return SFA_ERR_NULLPTR;
  // one partial sum of 512 a block, for the keys' and the queries' weight;
  // sized for the most SMs this library runs on
  const int n = norm_grad_blocks(p->T1, kMaxSms) + norm_grad_blocks(p->T1 * p->N1, kMaxSms);
  *bytes = (size_t)(n > 0 ? n : 1) * 512 * sizeof(float);
  return SFA_OK;
}

sfa_status sfa_norm_rope_grad(const sfa_rows_params* p, const int32_t* positions, const float* cos_sin, const void* q,
                              const void* q_weight, const float* q_rstd, const void* k, const void* k_weight,
                              const float* k_rstd, const void* d_q, const void* d_q_rope, const void* d_k,
                              const void* d_k_rope, void* dq, void* dq_rope, void* dk, void* dk_rope,
                              float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                              void* stream) {
  return norm_rope_grad(p, 1, nullptr, positions, cos_sin, q, q_weight, q_rstd, k, k_weight, k_rstd, d_q, d_q_rope, d_k,
                        d_k_rope, dq, dq_rope, dk, dk_rope, dq_weight, dk_weight, workspace, workspace_bytes, stream);
}

sfa_status sfa_norm_rope_axes_grad(const sfa_rows_params* p, int32_t n_axes, const uint8_t* axes,
                                   const int32_t* positions, const float* cos_sin, const void* q,
                                   const void* q_weight, const float* q_rstd, const void* k, const void* k_weight,
                                   const float* k_rstd, const void* d_q, const void* d_q_rope, const void* d_k,
                                   const void* d_k_rope, void* dq, void* dq_rope, void* dk, void* dk_rope,
                                   float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!axes) return SFA_ERR_NULLPTR;
  return norm_rope_grad(p, n_axes, axes, positions, cos_sin, q, q_weight, q_rstd, k, k_weight, k_rstd, d_q, d_q_rope,
                        d_k, d_k_rope, dq, dq_rope, dk, dk_rope, dq_weight, dk_weight, workspace, workspace_bytes,
                        stream);
}

sfa_status sfa_cache_append(const sfa_paged_params* p, void* cache, const int32_t* block_table,
                            const int32_t* act_seq_q, const int32_t* act_seq_kv, const void* k, const void* k_rope,
                            const void* k_weight, double eps, const float* cos_sin, int64_t table_len,
                            const void* q_rope, void* q_rope_out, int32_t* error, void* stream) {
  return append_by_table(p, nullptr, cache, block_table, act_seq_q, act_seq_kv, k, k_rope, k_weight, eps, cos_sin,
                         table_len, q_rope, q_rope_out, error, "sfa_cache_append", stream);
}

sfa_status sfa_cache4_append(const sfa_paged_params* p, double cache_scale, void* cache, const int32_t* block_table,
                             const int32_t* act_seq_q, const int32_t* act_seq_kv, const void* k, const void* k_rope,
                             const void* k_weight, double eps, const float* cos_sin, int64_t table_len,
                             const void* q_rope, void* q_rope_out, int32_t* error, void* stream) {
  return append_by_table(p, &cache_scale, cache, block_table, act_seq_q, act_seq_kv, k, k_rope, k_weight, eps,
                         cos_sin, table_len, q_rope, q_rope_out, error, "sfa_cache4_append", stream);
}

sfa_status sfa_cache_append_slots(const sfa_cache_params* c, const sfa_rows_params* p, void* cache,
                                  const int32_t* slots, int32_t n_axes, const uint8_t* axes, const int32_t* positions,
                                  const void* k, const void* k_rope, const void* k_weight, const float* cos_sin,
                                  const void* q_rope, void* q_rope_out, int32_t* error, void* stream) {
  AppendArgs a{};
  sfa_status s = check_cache(c, &a.pg, &a.scale_exp);
  if (s == SFA_OK) s = check_rows(p);
  if (s != SFA_OK) return s;
  if (p->dtype != c->dtype || !pack_axes(n_axes, axes, &a.axis_map)) return SFA_ERR_PARAM_INVALID;
  if (p->T1 == 0) return SFA_OK;   // no token: the tensors are empty, and may be null
  if (!slots || (a.pg.row == 576 && !positions)) return SFA_ERR_NULLPTR;
  a.pg.T = (int)p->T1;
  a.pg.G = (int)p->N1;
  a.packed = c->bits == 4;
  a.cache = cache;
  a.slots = slots;
  a.pos = positions;
  a.axes = n_axes;
  a.interleaved = p->interleaved;
  return append(a, p->dtype == SFA_DTYPE_FP16, k, k_rope, k_weight, p->eps, cos_sin, p->table_len, q_rope, q_rope_out,
                error, "sfa_cache_append_slots", stream);
}

sfa_status sfa_cache4_unpack(const sfa_cache_params* c, const void* cache, void* out, void* stream) {
  UnpackArgs a{};
  const sfa_status s = check_cache(c, &a.pg, &a.scale_exp);
  if (s != SFA_OK) return s;
  if (c->bits != 4) return SFA_ERR_PARAM_INVALID;
  if (!cache || !out) return SFA_ERR_NULLPTR;
  if (!all_aligned(cache, out)) return SFA_ERR_PARAM_INVALID;
  a.cache = cache;
  a.out = out;
  a.rows = c->num_pages * c->page_size;
  a.width = a.pg.row;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->dtype == SFA_DTYPE_FP16 ? launch_unpack<__half>(a, device_sm_count(), st)
                                                   : launch_unpack<__nv_bfloat16>(a, device_sm_count(), st);
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_cache4_unpack");
}

sfa_status sfa_page_plan(const sfa_plan_params* p, int32_t* block_table, const int32_t* act_seq_kv,
                         const int32_t* new_tokens, int32_t* free_pages, const int32_t* free_count,
                         int32_t* act_seq_q_out, int32_t* act_seq_kv_out, int32_t* free_count_out, int32_t* slots,
                         int32_t* positions, int32_t* error, void* stream) {
  if (!p) return SFA_ERR_NULLPTR;
  if (p->B < 1 || p->B > kPlanRequests) return SFA_ERR_SHAPE;
  if (p->page_size < 16 || p->page_size > 1024 || p->page_size % 16) return SFA_ERR_SHAPE;
  if (p->num_pages < 1 || p->num_pages > INT32_MAX / 2 / p->page_size) return SFA_ERR_SHAPE;
  if (p->max_pages < 1 || p->max_pages > INT32_MAX / 2 / p->page_size) return SFA_ERR_SHAPE;
  if (p->tokens < 0 || p->tokens > INT32_MAX / 2) return SFA_ERR_SHAPE;
  if (!block_table || !act_seq_kv || !new_tokens || !free_pages || !free_count || !act_seq_q_out || !act_seq_kv_out ||
      !free_count_out || (p->tokens && (!slots || !positions)))
    return SFA_ERR_NULLPTR;
  if (!words_aligned(block_table, act_seq_kv, new_tokens, free_pages, free_count, act_seq_q_out, act_seq_kv_out,
                     free_count_out, slots, positions, error))
    return SFA_ERR_PARAM_INVALID;
  // blocks read the inputs while others write the outputs
  struct {
    const int32_t* at;
    size_t n;
  } const part[] = {{act_seq_q_out, (size_t)p->B}, {act_seq_kv_out, (size_t)p->B}, {free_count_out, 1},
                    {slots, (size_t)p->tokens}, {positions, (size_t)p->tokens}, {error, error ? 1u : 0u},
                    {block_table, (size_t)(p->B * p->max_pages)}, {free_pages, (size_t)p->num_pages},
                    {act_seq_kv, (size_t)p->B}, {new_tokens, (size_t)p->B}, {free_count, 1}};
  for (int i = 0; i < 8; ++i)   // (the last three are only read)
    for (int k = i + 1; k < 11; ++k)
      if (part[i].n && part[k].n && part[i].at < part[k].at + part[k].n && part[k].at < part[i].at + part[i].n)
        return SFA_ERR_PARAM_INVALID;
  PlanArgs a{block_table, act_seq_kv, new_tokens, free_pages, free_count, act_seq_q_out, act_seq_kv_out, free_count_out,
             slots, positions, error, (int)p->B, (int)p->max_pages, (int)p->num_pages, (int)p->page_size,
             (int)p->tokens};
  const cudaError_t e = launch_plan(a, device_sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_page_plan");
}

sfa_status sfa_paged_workspace_size(const sfa_paged_params* p, size_t* bytes) {
  Paged g;
  const sfa_status s = check_paged(p, &g);
  if (s != SFA_OK) return s;
  if (!bytes) return SFA_ERR_NULLPTR;
  *bytes = paged_workspace(g);
  return SFA_OK;
}

sfa_status sfa_paged4_workspace_size(const sfa_paged_params* p, size_t* bytes) {
  Paged g;
  const sfa_status s = check_paged(p, &g);
  if (s != SFA_OK) return s;
  if (!bytes) return SFA_ERR_NULLPTR;
  *bytes = paged4_workspace(g);
  return SFA_OK;
}

sfa_status sfa_paged_fwd(const sfa_paged_params* p, const void* q, const void* q_rope, const void* cache,
                         const int32_t* block_table, const int32_t* act_seq_q, const int32_t* act_seq_kv, void* out,
                         float* softmax_max, float* softmax_sum, void* workspace, size_t workspace_bytes,
                         void* stream) {
  return paged_fwd(p, nullptr, q, q_rope, cache, block_table, act_seq_q, act_seq_kv, out, softmax_max, softmax_sum,
                   workspace, workspace_bytes, "sfa_paged_fwd", stream);
}

sfa_status sfa_paged4_fwd(const sfa_paged_params* p, double cache_scale, const void* q, const void* q_rope,
                          const void* cache, const int32_t* block_table, const int32_t* act_seq_q,
                          const int32_t* act_seq_kv, void* out, float* softmax_max, float* softmax_sum,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return paged_fwd(p, &cache_scale, q, q_rope, cache, block_table, act_seq_q, act_seq_kv, out, softmax_max,
                   softmax_sum, workspace, workspace_bytes, "sfa_paged4_fwd", stream);
}

}  // extern "C"
