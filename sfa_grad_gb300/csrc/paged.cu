// Attention of new tokens over the paged latent cache (sfa_paged_fwd).
//
//   x_j = scale [q || q_rope] . row_j,  out = sum_j exp(x_j - m) row_j[:512] / l
//
// One warp a (token, head): q and the output row stay in registers, 16 + 2 and
// 16 values a lane, the keys pass one by one with a running max and sum.
#include "kernels.h"
#include "rows.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) paged_kernel(PagedArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* err = reinterpret_cast<int*>(a.ws);
  const Paged& p = a.pg;
  // lengths: every warp checks all of them
  bool bad = false;
  long long total = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int q = p.act_q ? __ldg(p.act_q + b) : p.S1, kv = __ldg(p.act_kv + b);
    bad |= q < 0 || kv < 0 || (!p.tnd && q > p.S1) || kv > (long long)p.max_pages * p.page_size;
    total += q;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  bad |= p.tnd && total > p.T;
  if (__any_sync(~0u, bad)) {
    *err = kErrSeqLens;
    return;
  }
  const long long item = (long long)blockIdx.x * kWarps + warp;
  if (item >= (long long)p.T * p.G) return;
  const int t = (int)(item / p.G);
  const SeqTok s = find_token(p, t);
  if (s.seq < 0) return;
  const int kv = __ldg(p.act_kv + s.seq);
  const long long keys = p.mode == 3 ? min((long long)kv, (long long)kv - s.qlen + s.i + 1) : kv;
  float q[16], qr[2] = {0.f, 0.f}, o[16], m = -INFINITY, l = 0.f;
  load_row512((const T*)a.q + (size_t)item * 512, lane, q);
  if (p.row == 576) {
    const T* r = (const T*)a.qr + (size_t)item * 64 + 2 * lane;
    qr[0] = Elt<T>::to_f(r[0]);
    qr[1] = Elt<T>::to_f(r[1]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const int* table = p.table + (size_t)s.seq * p.max_pages;
  for (long long j = 0; j < keys; ++j) {
    const int page = __ldg(table + j / p.page_size);
    float c[16], r[2] = {0.f, 0.f};
    if (page < 0 || page >= p.num_pages) {
      *err = kErrPage;
#pragma unroll
      for (int i = 0; i < 16; ++i) c[i] = 0.f;
    } else {
      const T* row = (const T*)a.cache + ((size_t)page * p.page_size + j % p.page_size) * p.row;
      load_row512(row, lane, c);
      if (p.row == 576) {
        r[0] = Elt<T>::to_f(row[512 + 2 * lane]);
        r[1] = Elt<T>::to_f(row[513 + 2 * lane]);
      }
    }
    float d = q[0] * c[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) d = fmaf(q[i], c[i], d);
    d = fmaf(qr[0], r[0], fmaf(qr[1], r[1], d));
    const float x = warp_sum(d) * a.scale;
    const float top = fmaxf(m, x);
    const float f = m == top ? 1.f : ex2((m - top) * kLog2e), e = x == top ? 1.f : ex2((x - top) * kLog2e);
    l = l * f + e;
    m = top;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = o[i] * f + e * c[i];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] *= inv;
  store_row512((T*)a.out + (size_t)item * 512, lane, o);
  if (lane == 0) {
    a.smax[item] = m;
    a.ssum[item] = l;
  }
}

}  // namespace

size_t paged_workspace(const Paged&) { return 256; }

template <typename T>
cudaError_t launch_paged(const PagedArgs& a, int, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(a.ws, 0, 4, st);
  if (e != cudaSuccess) return e;
  const long long n = ((long long)a.pg.T * a.pg.G + kWarps - 1) / kWarps;
  paged_kernel<T><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_paged<__nv_bfloat16>(const PagedArgs&, int, cudaStream_t);
template cudaError_t launch_paged<__half>(const PagedArgs&, int, cudaStream_t);

}  // namespace sfa
