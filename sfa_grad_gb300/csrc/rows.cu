// Norm and position rotation of the attention's input rows, and their
// gradients (sfa_norm_rope, sfa_norm_rope_grad).
//
//   y = x r w, r = 1 / sqrt(mean x^2 + eps)          (rows of 512)
//   dx = r (g - x^ mean(g x^)), g = dy w, x^ = x r;   dw = sum dy x^
//   rotation by the position's angles, gradient by their negatives (rows of 64)
//
// Bound by HBM: every row is read once and written once, in 16-byte pieces, a
// row of 512 by one warp that keeps it in registers between the sum and the
// scaling.  One launch covers all four tensors: ranges of blocks take the key
// rows, the query rows and the rotated rows.
#include "kernels.h"
#include "rows.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 8;       // warps of a block
constexpr int kPieces = 4;      // 16-byte pieces a lane rotates at once (16 rows of 64 a warp)

__device__ __forceinline__ bool padded(const RowsArgs& a, int t) {
  if (!a.pos) return false;
  const int p = __ldg(a.pos + t);
  return p < 0 || p >= a.table_len;
}

// Rows of 512: x -> x r w, one warp a row.
template <typename T>
__device__ void norm_rows(const RowsArgs& a, const T* x, const T* w, T* y, float* rstd, int heads, long long row) {
  const int lane = threadIdx.x & 31;
  const bool pad = padded(a, (int)(row / heads));
  float v[16], g[16];
  load_row512(x + row * 512, lane, v);
  load_row512(w, lane, g);
  const float r = pad ? 0.f : row_rstd(v, a.eps);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = pad ? 0.f : v[i] * r * g[i];
  store_row512(y + row * 512, lane, v);
  if (rstd && lane == 0) rstd[row] = r;
}

// Rows of 64 of one token, heads h0 .. h0 + 15: rotated by the token's angles.
template <typename T, bool INTER>
__device__ void rotate_rows(const RowsArgs& a, const T* x, T* y, int heads, int t, int h0, float sgn) {
  const int lane = threadIdx.x & 31;
  const int pos = __ldg(a.pos + t);
  const bool pad = pos < 0 || pos >= a.table_len;
  const size_t base = ((size_t)t * heads + h0) * 8;
  const int n = min(heads - h0, 4 * kPieces) * 8;
  const uint4* src = reinterpret_cast<const uint4*>(x) + base;
  uint4* dst = reinterpret_cast<uint4*>(y) + base;
  uint4 w[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    w[j] = make_uint4(0, 0, 0, 0);
    if (lane + 32 * j < n) w[j] = src[lane + 32 * j];
  }
  Angles ang;
  load_angles<INTER>(a.cs + (size_t)(pad ? 0 : pos) * 64, lane & 7, &ang);
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    float v[8];
    unpack8<T>(w[j], v);
    rotate8<INTER>(v, ang, sgn);
    if (lane + 32 * j < n) dst[lane + 32 * j] = pad ? make_uint4(0, 0, 0, 0) : pack8<T>(v);
  }
}

// The rotated rows' warp items: 16 heads of one token each, the queries'
// first, then one a token for the keys.
template <typename T, bool INTER>
__device__ void rotate_item(const RowsArgs& a, const T* qr, T* qro, const T* kr, T* kro, long long item, float sgn) {
  const int per = (a.G + 4 * kPieces - 1) / (4 * kPieces);
  const long long nq = qr ? (long long)a.T * per : 0;
  if (item < nq) {
    rotate_rows<T, INTER>(a, qr, qro, a.G, (int)(item / per), (int)(item % per) * 4 * kPieces, sgn);
  } else if (kr && item - nq < a.T) {
    rotate_rows<T, INTER>(a, kr, kro, 1, (int)(item - nq), 0, sgn);
  }
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(RowsArgs a) {
  const int warp = threadIdx.x >> 5;
  int b = blockIdx.x;
  if (b < a.blocks_k) {
    const long long row = (long long)b * kWarps + warp;
    if (row < a.T) norm_rows<T>(a, (const T*)a.k, (const T*)a.kw, (T*)a.ko, a.k_rstd, 1, row);
    return;
  }
  b -= a.blocks_k;
  if (b < a.blocks_q) {
    const long long row = (long long)b * kWarps + warp;
    if (row < (long long)a.T * a.G) norm_rows<T>(a, (const T*)a.q, (const T*)a.qw, (T*)a.qo, a.q_rstd, a.G, row);
    return;
  }
  b -= a.blocks_q;
  rotate_item<T, INTER>(a, (const T*)a.qr, (T*)a.qro, (const T*)a.kr, (T*)a.kro, (long long)b * kWarps + warp, 1.f);
}

// Gradient of rows of 512: warps of `nblk` blocks take rows in strides, keep
// their part of dw in registers and leave one fp32 sum a block in `part`.
template <typename T>
__device__ void norm_grad_rows(const RowsArgs& a, const T* x, const T* w, const float* rstd, const T* dy, T* dx,
                               int heads, int blk, int nblk, float* part, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long rows = (long long)a.T * heads;
  float g[16], acc[16];
  load_row512(w, lane, g);
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (long long row = (long long)blk * kWarps + warp; row < rows; row += (long long)nblk * kWarps) {
    const bool pad = padded(a, (int)(row / heads));
    const float r = __ldg(rstd + row);
    float v[16], d[16], s = 0.f;
    load_row512(x + row * 512, lane, v);
    load_row512(dy + row * 512, lane, d);
    if (pad) {
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i] = 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] *= r;
        acc[i] = fmaf(d[i], v[i], acc[i]);
        d[i] *= g[i];
        s = fmaf(d[i], v[i], s);
      }
      s = warp_sum(s) * (1.0f / 512.0f);
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i] = r * (d[i] - v[i] * s);
    }
    store_row512(dx + row * 512, lane, d);
  }
  // the block's warps in ascending order
  float* mine = sm + warp * 512;
#pragma unroll
  for (int i = 0; i < 16; ++i) mine[(i < 8 ? 0 : 256) + lane * 8 + (i & 7)] = acc[i];
  __syncthreads();
  for (int f = threadIdx.x; f < 512; f += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) s += sm[k * 512 + f];
    part[(size_t)blk * 512 + f] = s;
  }
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_grad_kernel(RowsArgs a) {
  __shared__ float sm[kWarps * 512];
  int b = blockIdx.x;
  if (b < a.blocks_k) {
    norm_grad_rows<T>(a, (const T*)a.k, (const T*)a.kw, a.k_rstd, (const T*)a.dk, (T*)a.ko, 1, b, a.blocks_k, a.part,
                      sm);
    return;
  }
  b -= a.blocks_k;
  if (b < a.blocks_q) {
    norm_grad_rows<T>(a, (const T*)a.q, (const T*)a.qw, a.q_rstd, (const T*)a.dq, (T*)a.qo, a.G, b, a.blocks_q,
                      a.part + (size_t)a.blocks_k * 512, sm);
    return;
  }
  b -= a.blocks_q;
  rotate_item<T, INTER>(a, (const T*)a.qr, (T*)a.qro, (const T*)a.kr, (T*)a.kro,
                        (long long)b * kWarps + (threadIdx.x >> 5), -1.f);
}

// dw of 32 features: the blocks' partial sums in a fixed order.  Block
// 0..15: keys, 16..31: queries.
__global__ void __launch_bounds__(256) weight_grad_kernel(RowsArgs a) {
  __shared__ float sm[8][32];
  const bool q = blockIdx.x >= 16;
  float* out = q ? a.dqw : a.dkw;
  const int n = q ? a.blocks_q : a.blocks_k;
  if (!n) return;
  const float* part = a.part + (q ? (size_t)a.blocks_k * 512 : 0);
  const int f = (blockIdx.x & 15) * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float s = 0.f;
  for (int i = w; i < n; i += 8) s += part[(size_t)i * 512 + f];
  sm[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[i][threadIdx.x];
    out[f] = s;
  }
}

long long rope_blocks(const RowsArgs& a) {
  const long long per = (a.G + 4 * kPieces - 1) / (4 * kPieces);
  const long long items = (a.qr ? a.T * per : 0) + (a.kr ? a.T : 0);
  return (items + kWarps - 1) / kWarps;
}

}  // namespace

int norm_grad_blocks(long long rows, int nsm) {
  // enough warps to fill the GPU: 8 blocks of 8 warps an SM at most, each of
  // at least one row a warp
  const long long n = (rows + kWarps - 1) / kWarps, cap = 6LL * nsm;
  return (int)(n < cap ? n : cap);
}

template <typename T>
cudaError_t launch_norm_rope(RowsArgs a, cudaStream_t st) {
  a.blocks_k = a.k ? (int)((a.T + kWarps - 1) / kWarps) : 0;
  a.blocks_q = a.q ? (int)(((long long)a.T * a.G + kWarps - 1) / kWarps) : 0;
  const long long n = a.blocks_k + (long long)a.blocks_q + rope_blocks(a);
  if (n == 0) return cudaSuccess;
  if (a.interleaved)
    norm_rope_kernel<T, true><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
  else
    norm_rope_kernel<T, false><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_rope_grad(RowsArgs a, int nsm, cudaStream_t st) {
  a.blocks_k = a.dk ? norm_grad_blocks(a.T, nsm) : 0;
  a.blocks_q = a.dq ? norm_grad_blocks((long long)a.T * a.G, nsm) : 0;
  const long long n = a.blocks_k + (long long)a.blocks_q + rope_blocks(a);
  if (n > 0) {
    if (a.interleaved)
      norm_rope_grad_kernel<T, true><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
    else
      norm_rope_grad_kernel<T, false><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.blocks_k || a.blocks_q) weight_grad_kernel<<<32, 256, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_norm_rope<__nv_bfloat16>(RowsArgs, cudaStream_t);
template cudaError_t launch_norm_rope<__half>(RowsArgs, cudaStream_t);
template cudaError_t launch_norm_rope_grad<__nv_bfloat16>(RowsArgs, int, cudaStream_t);
template cudaError_t launch_norm_rope_grad<__half>(RowsArgs, int, cudaStream_t);

}  // namespace sfa
