// C-ABI entry points of the latent-row operators (include/sfa_grad.h):
// validation and launches of norm_rope, its gradient, the cache append and the
// paged attention.
#include <cmath>
#include <cstdio>

#include "sfa_grad.h"
#include "kernels.h"

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

}  // namespace
}  // namespace sfa

using namespace sfa;

extern "C" {

sfa_status sfa_norm_rope(const sfa_rows_params* p, const int32_t* positions, const float* cos_sin, const void* q,
                         const void* q_weight, const void* q_rope, const void* k, const void* k_weight,
                         const void* k_rope, void* q_out, void* q_rope_out, void* k_out, void* k_rope_out,
                         float* q_rstd, float* k_rstd, void* stream) {
  const sfa_status s = check_rows(p);
  if (s != SFA_OK) return s;
  if ((q && (!q_weight || !q_out)) || (k && (!k_weight || !k_out)) || (q_rope && !q_rope_out) ||
      (k_rope && !k_rope_out))
    return SFA_ERR_NULLPTR;
  if ((q_rope || k_rope) && (!positions || !cos_sin)) return SFA_ERR_NULLPTR;
  if ((q_rope || k_rope) && p->table_len < 1) return SFA_ERR_SHAPE;
  if (!all_aligned(cos_sin, q, q_weight, q_rope, k, k_weight, k_rope, q_out, q_rope_out, k_out, k_rope_out) ||
      !words_aligned(positions, q_rstd, k_rstd))
    return SFA_ERR_PARAM_INVALID;
  if (p->T1 == 0) return SFA_OK;
  RowsArgs a = rows_args(p, positions, cos_sin);
  a.q = q; a.qw = q_weight; a.qr = q_rope; a.k = k; a.kw = k_weight; a.kr = k_rope;
  a.qo = q_out; a.qro = q_rope_out; a.ko = k_out; a.kro = k_rope_out;
  a.q_rstd = q_rstd; a.k_rstd = k_rstd;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == SFA_DTYPE_FP16 ? launch_norm_rope<__half>(a, st)
                                                   : launch_norm_rope<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_norm_rope");
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
  size_t need = 0;
  const sfa_status s = sfa_norm_rope_grad_workspace_size(p, &need);
  if (s != SFA_OK) return s;
  if ((d_q && (!q || !q_weight || !q_rstd || !dq || !dq_weight)) ||
      (d_k && (!k || !k_weight || !k_rstd || !dk || !dk_weight)) || (d_q_rope && !dq_rope) ||
      (d_k_rope && !dk_rope))
    return SFA_ERR_NULLPTR;
  const bool rope = d_q_rope || d_k_rope;
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

sfa_status sfa_cache_append(const sfa_paged_params* p, void* cache, const int32_t* block_table,
                            const int32_t* act_seq_q, const int32_t* act_seq_kv, const void* k, const void* k_rope,
                            const void* k_weight, double eps, const float* cos_sin, int64_t table_len,
                            const void* q_rope, void* q_rope_out, int32_t* error, void* stream) {
  AppendArgs a{};
  const sfa_status s = check_paged(p, &a.pg);
  if (s != SFA_OK) return s;
  if (a.pg.T == 0) return SFA_OK;   // no new token: the tensors are empty, and may be null
  const bool rope = p->Dr == 64;
  if (!cache || !block_table || !act_seq_kv || !k || (a.pg.tnd && !act_seq_q)) return SFA_ERR_NULLPTR;
  if (rope && (!k_rope || !cos_sin || (q_rope && !q_rope_out))) return SFA_ERR_NULLPTR;
  if (rope && (table_len < 1 || table_len > INT32_MAX)) return SFA_ERR_SHAPE;
  if (!fits(eps) || eps < 0) return SFA_ERR_SHAPE;
  if (!all_aligned(cache, k, k_rope, k_weight, cos_sin, q_rope, q_rope_out) ||
      !words_aligned(block_table, act_seq_q, act_seq_kv, error))
    return SFA_ERR_PARAM_INVALID;
  a.pg.table = block_table;
  a.pg.act_q = act_seq_q;
  a.pg.act_kv = act_seq_kv;
  a.cache = cache;
  a.k = k; a.kw = k_weight;
  a.kr = rope ? k_rope : nullptr;
  a.qr = rope ? q_rope : nullptr;
  a.qro = q_rope_out;
  a.cs = rope ? cos_sin : nullptr;
  a.table_len = table_len;
  a.error = error;
  a.eps = (float)eps;
  a.interleaved = p->interleaved;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == SFA_DTYPE_FP16 ? launch_append<__half>(a, st)
                                                   : launch_append<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_cache_append");
}

sfa_status sfa_paged_workspace_size(const sfa_paged_params* p, size_t* bytes) {
  Paged g;
  const sfa_status s = check_paged(p, &g);
  if (s != SFA_OK) return s;
  if (!bytes) return SFA_ERR_NULLPTR;
  *bytes = paged_workspace(g);
  return SFA_OK;
}

sfa_status sfa_paged_fwd(const sfa_paged_params* p, const void* q, const void* q_rope, const void* cache,
                         const int32_t* block_table, const int32_t* act_seq_q, const int32_t* act_seq_kv, void* out,
                         float* softmax_max, float* softmax_sum, void* workspace, size_t workspace_bytes,
                         void* stream) {
  PagedArgs a{};
  const sfa_status s = check_paged(p, &a.pg);
  if (s != SFA_OK) return s;
  const bool rope = p->Dr == 64;
  if (!workspace) return SFA_ERR_NULLPTR;
  if (!aligned(workspace, 256) || workspace_bytes < paged_workspace(a.pg)) return SFA_ERR_PARAM_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.pg.T == 0) {
    // no query row: the tensors are empty, and may be null
    const cudaError_t e = cudaMemsetAsync(workspace, 0, 4, st);
    return e == cudaSuccess ? SFA_OK : fail(e, "sfa_paged_fwd");
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
  return e == cudaSuccess ? SFA_OK : fail(e, "sfa_paged_fwd");
}

}  // extern "C"
