// Values of a 4-bit cache in 16 bits (sfa_cache4_unpack), and of the pages
// that a call's block tables name.
//
// Bound by HBM: a warp takes four rows at once, a lane two 4-byte words of codes
// of each to two 16-byte pieces (and eight lanes a piece of the rotated part),
// so that reads and writes are whole lines and twelve loads are in flight a lane.
// 2^20 rows 244 us, 6.8 TB/s; 131,072 rows 33 us, 6.3 TB/s.  A small cache is
// bound by latency, one round of reads and one of writes, which stay in L2:
// 13,168 rows 5.4 us from cold caches and 3.8 from warm ones (a thread a piece: 8.2
// us cold by the profiler, where this takes 6.2).
#include "kernels.h"
#include "cache4.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 8, kRowsAtOnce = 4;

// Rows first .. first + n - 1 (n <= kRowsAtOnce) of `src` to `dst`, by one warp.
template <typename T, bool ROPE>
__device__ __forceinline__ void unpack_rows(const uint8_t* src, uint4* dst, int n, const Dec4<T>& dec) {
  constexpr int kPieces = ROPE ? 72 : 64, kBytes = kRopeAt + (ROPE ? 128 : 0);
  const int lane = threadIdx.x & 31;
  uint32_t code[kRowsAtOnce][2], scale[kRowsAtOnce][2];
  uint4 rope[kRowsAtOnce];
#pragma unroll
  for (int r = 0; r < kRowsAtOnce; ++r) {
    if (r >= n) break;
    const uint8_t* row = src + r * kBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      code[r][h] = __ldg(reinterpret_cast<const uint32_t*>(row) + lane + 32 * h);
      scale[r][h] = __ldg(row + kCodes + (lane >> 1) + 16 * h);
    }
    if (ROPE && lane < 8) rope[r] = __ldg(reinterpret_cast<const uint4*>(row + kRopeAt) + lane);
  }
#pragma unroll
  for (int r = 0; r < kRowsAtOnce; ++r) {
    if (r >= n) break;
    uint4* to = dst + r * kPieces;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t s[2];
      dec.scales(scale[r][h], s);
      to[lane + 32 * h] = dec.eight(code[r][h], s[0]);
    }
    if (ROPE && lane < 8) to[64 + lane] = rope[r];
  }
}

template <typename T, bool ROPE>
__global__ void __launch_bounds__(32 * kWarps) unpack_kernel(const UnpackArgs a) {
  constexpr int kPieces = ROPE ? 72 : 64, kBytes = kRopeAt + (ROPE ? 128 : 0);
  const Dec4<T> dec(a.scale_exp);
  const long long step = (long long)gridDim.x * kWarps * kRowsAtOnce;
  for (long long r = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRowsAtOnce; r < a.rows; r += step)
    unpack_rows<T, ROPE>((const uint8_t*)a.cache + r * kBytes, reinterpret_cast<uint4*>(a.out) + r * kPieces,
                         (int)min((long long)kRowsAtOnce, a.rows - r), dec);
}

// Block table entry by entry (a block each): its page's values, as far as the
// sequence reaches; none of a sequence without query rows, which nobody reads.
// By page, they go where the page lies in the cache, so that the caller's table
// serves, and a page that several entries name is unpacked once: an entry takes
// the rows beyond those that others have taken (64 sequences of one token x 128
// heads over one history of 16384 rows: 337 us, 64 times the same rows; so 223,
// where the call over 16-bit rows takes 192).  Else every entry has a page of
// its own and an entry in a table over them, where pages that are none stay
// none.
template <typename T, bool ROPE>
__global__ void __launch_bounds__(32 * kWarps) unpack_tables_kernel(const UnpackArgs a) {
  constexpr int kPieces = ROPE ? 72 : 64, kBytes = kRopeAt + (ROPE ? 128 : 0);
  const Dec4<T> dec(a.scale_exp);
  const Paged& g = a.pg;
  __shared__ int taken;
  const long long entries = (long long)g.B * g.max_pages;
  for (long long e = blockIdx.x; e < entries; e += gridDim.x) {
    const int b = (int)(e / g.max_pages), j = (int)(e - (long long)b * g.max_pages);
    const long long kv = min((long long)__ldg(g.act_kv + b), (long long)g.max_pages * g.page_size);
    const int rows = (int)max(0LL, min((long long)g.page_size, kv - (long long)j * g.page_size));
    if (!rows || (g.act_q && __ldg(g.act_q + b) <= 0)) continue;
    const int id = __ldg(g.table + e);
    const bool ok = id >= 0 && id < g.num_pages;
    if (!a.by_page && threadIdx.x == 0) a.table[e] = ok ? (int)e : -1;
    if (!ok) continue;
    const long long to = a.by_page ? id : e;
    int from = 0;
    if (a.by_page) {
      if (threadIdx.x == 0) taken = atomicMax(a.table + id, rows);
      __syncthreads();
      from = taken;
      __syncthreads();   // before the next entry's
    }
    const uint8_t* src = (const uint8_t*)a.cache + (size_t)id * g.page_size * kBytes;
    uint4* dst = reinterpret_cast<uint4*>(a.out) + (size_t)to * g.page_size * kPieces;
    for (int r = from + (threadIdx.x >> 5) * kRowsAtOnce; r < rows; r += kWarps * kRowsAtOnce)
      unpack_rows<T, ROPE>(src + (size_t)r * kBytes, dst + (size_t)r * kPieces, min(kRowsAtOnce, rows - r), dec);
  }
}

}  // namespace

template <typename T>
cudaError_t launch_unpack(const UnpackArgs& a, int nsm, cudaStream_t st) {
  const long long per = kWarps * kRowsAtOnce, blocks = (a.rows + per - 1) / per, most = (long long)nsm * 32;
  auto kern = a.width == 576 ? unpack_kernel<T, true> : unpack_kernel<T, false>;
  kern<<<(unsigned)(blocks < most ? blocks : most), 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_unpack_tables(const UnpackArgs& a, int nsm, cudaStream_t st) {
  const long long blocks = (long long)a.pg.B * a.pg.max_pages, most = (long long)nsm * 32;
  if (a.by_page) {
    const cudaError_t e = cudaMemsetAsync(a.table, 0, (size_t)a.pg.num_pages * sizeof(int), st);
    if (e != cudaSuccess) return e;
  }
  auto kern = a.width == 576 ? unpack_tables_kernel<T, true> : unpack_tables_kernel<T, false>;
  kern<<<(unsigned)(blocks < most ? blocks : most), 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_unpack<__nv_bfloat16>(const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_unpack<__half>(const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_unpack_tables<__nv_bfloat16>(const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_unpack_tables<__half>(const UnpackArgs&, int, cudaStream_t);

}  // namespace sfa
