// Values of a 4-bit cache in 16 bits (sfa_cache4_unpack), and of the pages
// that a call's block tables name.
//
// Bound by HBM: a thread takes four bytes of codes to one 16-byte piece of a
// row (or copies a piece of its rotated part), neighbouring threads
// neighbouring pieces.
#include "kernels.h"
#include "cache4.cuh"

namespace sfa {
namespace {

// Piece p of a row: 8 elements of the latent part, or of the rotated one.
template <typename T>
__device__ __forceinline__ uint4 piece_of(const uint8_t* row, int p, const Dec4<T>& dec) {
  if (p >= 64) return __ldg(reinterpret_cast<const uint4*>(row + kRopeAt) + (p - 64));
  uint32_t s[2];
  dec.scales(__ldg(row + kCodes + (p >> 1)), s);
  return dec.eight(__ldg(reinterpret_cast<const uint32_t*>(row) + p), s[0]);
}

template <typename T, bool ROPE>
__global__ void __launch_bounds__(256) unpack_kernel(const UnpackArgs a) {
  constexpr int kPieces = ROPE ? 72 : 64, kBytes = kRopeAt + (ROPE ? 128 : 0);
  const Dec4<T> dec(a.scale_exp);
  const long long n = a.rows * kPieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long row = i / kPieces;
    reinterpret_cast<uint4*>(a.out)[i] =
        piece_of<T>((const uint8_t*)a.cache + row * kBytes, (int)(i - row * kPieces), dec);
  }
}

// Block table entry by entry (a block each): its page's values, as far as the
// sequence reaches, and the entry of the table over them.  Pages that are
// none stay none.
template <typename T, bool ROPE>
__global__ void __launch_bounds__(256) unpack_tables_kernel(const UnpackArgs a) {
  constexpr int kPieces = ROPE ? 72 : 64, kBytes = kRopeAt + (ROPE ? 128 : 0);
  const Dec4<T> dec(a.scale_exp);
  const Paged& g = a.pg;
  const long long entries = (long long)g.B * g.max_pages;
  for (long long e = blockIdx.x; e < entries; e += gridDim.x) {
    const int b = (int)(e / g.max_pages), j = (int)(e - (long long)b * g.max_pages);
    const long long kv = min((long long)__ldg(g.act_kv + b), (long long)g.max_pages * g.page_size);
    const int rows = (int)max(0LL, min((long long)g.page_size, kv - (long long)j * g.page_size));
    if (!rows) continue;
    const int id = __ldg(g.table + e);
    const bool ok = id >= 0 && id < g.num_pages;
    const long long to = a.by_page ? id : e;
    if (threadIdx.x == 0) a.table[e] = ok ? (int)to : -1;
    if (!ok) continue;
    const uint8_t* src = (const uint8_t*)a.cache + (size_t)id * g.page_size * kBytes;
    uint4* dst = reinterpret_cast<uint4*>(a.out) + (size_t)to * g.page_size * kPieces;
    for (int i = threadIdx.x; i < rows * kPieces; i += 256) {
      const int row = i / kPieces;
      dst[i] = piece_of<T>(src + (size_t)row * kBytes, i - row * kPieces, dec);
    }
  }
}

}  // namespace

template <typename T>
cudaError_t launch_unpack(const UnpackArgs& a, int nsm, cudaStream_t st) {
  const bool rope = a.width == 576;
  const long long blocks = (a.rows * (rope ? 72 : 64) + 255) / 256, most = (long long)nsm * 32;
  auto kern = rope ? unpack_kernel<T, true> : unpack_kernel<T, false>;
  kern<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_unpack_tables(const UnpackArgs& a, int nsm, cudaStream_t st) {
  const long long blocks = (long long)a.pg.B * a.pg.max_pages, most = (long long)nsm * 32;
  auto kern = a.width == 576 ? unpack_tables_kernel<T, true> : unpack_tables_kernel<T, false>;
  kern<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_unpack<__nv_bfloat16>(const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_unpack<__half>(const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_unpack_tables<__nv_bfloat16>(const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_unpack_tables<__half>(const UnpackArgs&, int, cudaStream_t);

}  // namespace sfa
