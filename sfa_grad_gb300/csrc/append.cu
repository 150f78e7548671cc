// Append of new tokens' latent rows to the paged cache, with the norm of the
// latent part and the position rotation on the way (sfa_cache_append).
//
// One warp a token writes its 1152-byte row straight to its page; further
// warps rotate the tokens' query rows, 32 heads each, so that a decoding step
// has one launch ahead of its attention.  Bound by the rows' bytes, and with
// few tokens by the latency of the lengths, the block table and the row, read
// one after the other.  Measured, bf16: 64 single tokens x 128 heads 6.2 us;
// 8 chunks, 13,045 tokens x 64 heads, 47.3 us, 5.2 TB/s.
#include "kernels.h"
#include "paged.cuh"
#include "rows.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 4;
// 16-byte pieces a lane rotates at once (32 heads a warp): the chunks took 62
// us with two, 49 with four, 47 with eight.
constexpr int kPieces = 8;

// Where a new token goes: its position, or -1 (left out).
__device__ __forceinline__ int token_position(const AppendArgs& a, int t, int* seq) {
  const SeqTok s = find_token(a.pg, t);
  if (s.seq < 0) {
    if (s.bad && a.error) *a.error = kErrSeqLens;
    return -1;
  }
  const int kv = __ldg(a.pg.act_kv + s.seq);
  const long long pos = (long long)kv - s.qlen + s.i;
  if (pos < 0 || kv > (long long)a.pg.max_pages * a.pg.page_size) {
    if (a.error) *a.error = kErrSeqLens;
    return -1;
  }
  if (a.cs && pos >= a.table_len) {
    if (a.error) *a.error = kErrPosition;
    return -1;
  }
  *seq = s.seq;
  return (int)pos;
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(AppendArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int seq = 0;
  if ((int)blockIdx.x < a.blocks_k) {
    const int t = blockIdx.x * kWarps + warp;
    if (t >= a.pg.T) return;
    // the row does not depend on where it goes: its loads are in flight
    // during the search
    float v[16], rope[8], g[16];
    load_row512((const T*)a.k + (size_t)t * 512, lane, v);
    if (a.cs) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (lane < 8) w = reinterpret_cast<const uint4*>((const T*)a.kr + (size_t)t * 64)[lane];
      unpack8<T>(w, rope);
    }
    if (a.kw) load_row512((const T*)a.kw, lane, g);
    const int pos = token_position(a, t, &seq);
    if (pos < 0) return;
    const int ps = a.pg.page_size;
    const int page = __ldg(a.pg.table + (size_t)seq * a.pg.max_pages + pos / ps);
    if (page < 0 || page >= a.pg.num_pages) {
      if (a.error && lane == 0) *a.error = kErrPage;
      return;
    }
    T* dst = (T*)a.cache + ((size_t)page * ps + pos % ps) * a.pg.row;
    if (a.kw) {
      const float r = row_rstd(v, a.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= r * g[i];
    }
    store_row512(dst, lane, v);
    if (a.cs) {
      Angles ang;
      load_angles<INTER>(a.cs + (size_t)pos * 64, lane & 7, &ang);
      rotate8<INTER>(rope, ang, 1.f);
      if (lane < 8) reinterpret_cast<uint4*>(dst + 512)[lane] = pack8<T>(rope);
    }
    return;
  }
  // query rows: 32 heads of one token a warp
  const int per = (a.pg.G + 4 * kPieces - 1) / (4 * kPieces);
  const long long item = (long long)(blockIdx.x - a.blocks_k) * kWarps + warp;
  if (item >= (long long)a.pg.T * per) return;
  const int t = (int)(item / per), h0 = (int)(item % per) * 4 * kPieces;
  const size_t base = ((size_t)t * a.pg.G + h0) * 8;
  const int n = min(a.pg.G - h0, 4 * kPieces) * 8;
  uint4 w[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    w[j] = make_uint4(0, 0, 0, 0);
    if (lane + 32 * j < n) w[j] = (reinterpret_cast<const uint4*>(a.qr) + base)[lane + 32 * j];
  }
  const int pos = token_position(a, t, &seq);
  if (pos < 0) return;
  Angles ang;
  load_angles<INTER>(a.cs + (size_t)pos * 64, lane & 7, &ang);
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    float v[8];
    unpack8<T>(w[j], v);
    rotate8<INTER>(v, ang, 1.f);
    if (lane + 32 * j < n) (reinterpret_cast<uint4*>(a.qro) + base)[lane + 32 * j] = pack8<T>(v);
  }
}

}  // namespace

template <typename T>
cudaError_t launch_append(AppendArgs a, cudaStream_t st) {
  const int per = (a.pg.G + 4 * kPieces - 1) / (4 * kPieces);
  a.blocks_k = (a.pg.T + kWarps - 1) / kWarps;
  const long long n = a.blocks_k + (a.qr ? ((long long)a.pg.T * per + kWarps - 1) / kWarps : 0);
  if (n == 0) return cudaSuccess;
  if (a.interleaved)
    append_kernel<T, true><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
  else
    append_kernel<T, false><<<(unsigned)n, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_append<__nv_bfloat16>(AppendArgs, cudaStream_t);
template cudaError_t launch_append<__half>(AppendArgs, cudaStream_t);

}  // namespace sfa
