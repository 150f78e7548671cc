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
// rows, the query rows and the rotated rows.  Measured (a plain copy reaches
// 6.8 TB/s): 4096 tokens, keys normed, 128 query heads rotated, bf16: 24.6 us,
// 5.9 TB/s; their gradients 32.4 us, 4.6 TB/s, with the second launch that adds
// up the weight's; 16381 tokens x 16 normed heads, fp16, gradients: 166 us, 5.6
// TB/s.
#include "kernels.h"
#include "rows.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 8;       // warps of a block
// Blocks of the gradient's rows of 512 an SM.  Two leave the keys of 4096
// tokens waiting (the gradients of that step 43 us instead of 37), four take
// registers away from the row in flight (16381 x 16 heads 240 instead of 166).
constexpr int kGradBlocks = 3;
// 16-byte pieces a lane rotates at once (32 rows of 64 a warp): the gradients
// of 4096 x 128 heads took 41 us with two, 37 with four, 32 with eight.
constexpr int kPieces = 8;

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

// Rows of 64 of one token, heads h0 .. h0 + 31: rotated by the token's angles.
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

// The rotated rows' warp items: 32 heads of one token each, the queries'
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
// their part of dw in registers and leave one fp32 sum a block in `part`.  A
// row's 2 KB are on their way while the row before is worked on; packed, so
// that the registers allow three blocks an SM.
template <typename T>
__device__ void norm_grad_rows(const RowsArgs& a, const T* x, const T* w, const float* rstd, const T* dy, T* dx,
                               int heads, int blk, int nblk, float* part, float* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long rows = (long long)a.T * heads, step = (long long)nblk * kWarps;
  const uint4* pw = reinterpret_cast<const uint4*>(w);
  const uint4 g[2] = {pw[lane], pw[lane + 32]};
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  uint4 nx[2], nd[2];
  float nr = 0.f;
  int npos = 0;
  auto fetch = [&](long long row) {
    const uint4* px = reinterpret_cast<const uint4*>(x + row * 512);
    const uint4* pd = reinterpret_cast<const uint4*>(dy + row * 512);
    nx[0] = __ldcs(px + lane); nx[1] = __ldcs(px + lane + 32);
    nd[0] = __ldcs(pd + lane); nd[1] = __ldcs(pd + lane + 32);
    nr = __ldg(rstd + row);
    if (a.pos) npos = __ldg(a.pos + row / heads);
  };
  long long row = (long long)blk * kWarps + warp;
  if (row < rows) fetch(row);
  for (; row < rows; row += step) {
    const uint4 rx[2] = {nx[0], nx[1]}, rd[2] = {nd[0], nd[1]};
    const float r = nr;
    const bool pad = a.pos && (npos < 0 || npos >= a.table_len);
    if (row + step < rows) fetch(row + step);
    uint4* out = reinterpret_cast<uint4*>(dx + row * 512);
    if (pad) {
      out[lane] = out[lane + 32] = make_uint4(0, 0, 0, 0);
      continue;
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8], d[8], gw[8];
      unpack8<T>(rx[k], v);
      unpack8<T>(rd[k], d);
      unpack8<T>(g[k], gw);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = v[i] * r;
        acc[k * 8 + i] = fmaf(d[i], xh, acc[k * 8 + i]);
        s = fmaf(d[i] * gw[i], xh, s);
      }
    }
    s = warp_sum(s) * (1.0f / 512.0f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8], d[8], gw[8];
      unpack8<T>(rx[k], v);
      unpack8<T>(rd[k], d);
      unpack8<T>(g[k], gw);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = r * (d[i] * gw[i] - v[i] * r * s);
      __stcs(out + lane + 32 * k, pack8<T>(d));
    }
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
__global__ void __launch_bounds__(kWarps * 32, kGradBlocks) norm_rope_grad_kernel(RowsArgs a) {
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

// dw of 16 features: the blocks' partial sums in a fixed order, 64 chains of
// them a feature.  Block 0..31: keys, 32..63: queries.
__global__ void __launch_bounds__(1024) weight_grad_kernel(RowsArgs a) {
  __shared__ float sm[64][17];
  const bool q = blockIdx.x >= 32;
  float* out = q ? a.dqw : a.dkw;
  const int n = q ? a.blocks_q : a.blocks_k;
  if (!n) return;
  const float* part = a.part + (q ? (size_t)a.blocks_k * 512 : 0);
  const int c = threadIdx.x & 15, w = threadIdx.x >> 4, f = (blockIdx.x & 31) * 16 + c;
  float s = 0.f;
#pragma unroll 8
  for (int i = w; i < n; i += 64) s += part[(size_t)i * 512 + f];
  sm[w][c] = s;
  __syncthreads();
  if (threadIdx.x < 512) {   // warp k: feature k
    const int k = threadIdx.x >> 5, lane = threadIdx.x & 31;
    s = warp_sum(sm[lane][k] + sm[lane + 32][k]);
    if (lane == 0) out[(blockIdx.x & 31) * 16 + k] = s;
  }
}

long long rope_blocks(const RowsArgs& a) {
  const long long per = (a.G + 4 * kPieces - 1) / (4 * kPieces);
  const long long items = (a.qr ? a.T * per : 0) + (a.kr ? a.T : 0);
  return (items + kWarps - 1) / kWarps;
}

}  // namespace

int norm_grad_blocks(long long rows, int nsm) {
  // as many blocks as the GPU holds at once, each of at least one row a warp
  const long long n = (rows + kWarps - 1) / kWarps, cap = (long long)kGradBlocks * nsm;
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
  if (a.blocks_k || a.blocks_q) weight_grad_kernel<<<64, 1024, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_norm_rope<__nv_bfloat16>(RowsArgs, cudaStream_t);
template cudaError_t launch_norm_rope<__half>(RowsArgs, cudaStream_t);
template cudaError_t launch_norm_rope_grad<__nv_bfloat16>(RowsArgs, int, cudaStream_t);
template cudaError_t launch_norm_rope_grad<__half>(RowsArgs, int, cudaStream_t);

}  // namespace sfa
