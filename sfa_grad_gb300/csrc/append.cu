// Append of new tokens' latent rows to the paged cache, with the norm of the
// latent part and the position rotation on the way (sfa_cache_append).
//
// One warp a token writes its 1152-byte row straight to its page; further
// warps rotate the tokens' query rows, 32 heads each, so that a decoding step
// has one launch ahead of its attention.  Bound by the rows' bytes, and with
// few tokens by the latency of the lengths, the block table and the row, read
// one after the other.  Measured, bf16: 64 single tokens x 128 heads 6.2 us;
// 8 chunks, 13,045 tokens x 64 heads, 47.3 us, 5.2 TB/s.
#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "cache4.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 4;
// 16-byte pieces a lane rotates at once (32 heads a warp): the chunks took 62
// us with two, 49 with four, 47 with eight.
constexpr int kPieces = 8;

// Where a new token goes and what turns it.
struct Spot {
  bool ok;         // else: left out
  long long row;   // of the cache
  Places at;
};
// The row follows from the token's position and its sequence's block table;
// page = false: only the position is wanted.
__device__ __forceinline__ Spot by_table(const AppendArgs& a, int t, bool page) {
  const SeqTok s = find_token(a.pg, t);
  Spot r{};
  if (s.seq < 0) {
    if (s.bad && a.error) *a.error = kErrSeqLens;
    return r;
  }
  const int kv = __ldg(a.pg.act_kv + s.seq);
  const long long pos = (long long)kv - s.qlen + s.i;
  if (pos < 0 || kv > (long long)a.pg.max_pages * a.pg.page_size) {
    if (a.error) *a.error = kErrSeqLens;
    return r;
  }
  if (a.cs && pos >= a.table_len) {
    if (a.error) *a.error = kErrPosition;
    return r;
  }
  r.at.p[0] = (int)pos;
  if (page) {
    const int ps = a.pg.page_size;
    const int id = __ldg(a.pg.table + (size_t)s.seq * a.pg.max_pages + (int)pos / ps);
    if (id < 0 || id >= a.pg.num_pages) {
      if (a.error) *a.error = kErrPage;
      return r;
    }
    r.row = (long long)id * ps + (int)pos % ps;
  }
  r.ok = true;
  return r;
}
// The row stands in the slot map; a negative slot is a token of no sequence.
__device__ __forceinline__ Spot by_slot(const AppendArgs& a, int t) {
  Spot r{};
  const int slot = __ldg(a.slots + t);
  if (a.cs) r.at = load_places(a.pos, t, a.pg.T, a.axes);
  if (slot < 0) return r;
  if (slot >= (long long)a.pg.num_pages * a.pg.page_size) {
    if (a.error) *a.error = kErrPage;
    return r;
  }
  if (a.cs && outside(r.at, a.table_len)) {
    if (a.error) *a.error = kErrPosition;
    return r;
  }
  r.row = slot;
  r.ok = true;
  return r;
}
template <bool INTER, bool SLOTS>
__device__ __forceinline__ void spot_angles(const AppendArgs& a, const Spot& s, int piece, Angles* ang) {
  if constexpr (SLOTS)
    load_angles<INTER>(a.cs, s.at, a.axis_map, piece, ang);
  else
    load_angles<INTER>(a.cs + (size_t)s.at.p[0] * 64, piece, ang);
}

// ------------------------------------------------------------------ rows of 4 bits
// y / 2^k in blocks of 16: the scale is max|y| / 6 in e4m3, a code the value
// nearest to y / scale, ties to even, both of the exact y: a value that fp32's
// roundings could carry over a border between two codes or two scales is
// found, and its row is quantised again from y in 64 bits.
//
// Steps of fp32 on the way: squares are exact or 2^-24 off, their sum 16 + 5
// additions, the square root halves that, and a root, a reciprocal, two
// products, the division by 6, the reciprocal of the scale and the product
// with it add 2^-24 each: less than 19 x 2^-24 in all.  32 of them (2^-19) are
// taken as near.
constexpr float kNear = 1.0f / (1 << 19);

__device__ __forceinline__ uint32_t to_e4m3(float x) {   // one byte, to nearest, at most 448
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xff;
}
__device__ __forceinline__ uint32_t to_e2m1(float a, float b) {   // two codes, a in the low half
  uint32_t r;
  asm("{\n.reg .b8 x;\ncvt.rn.satfinite.e2m1x2.f32 x, %1, %2;\ncvt.u32.u8 %0, x;\n}" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const uint32_t h = e4m3_f16(byte);
  __half2 v;
  memcpy(&v, &h, 4);
  return __low2float(v);
}
// The nearest scale to top / 6; a block with a value that is not finite gets
// a scale that is not a number.
template <typename F>
__device__ __forceinline__ uint32_t exact_scale(F top) {
  const F want = top / (F)6;
  int e;
  frexp(want, &e);
  const F step = ldexp((F)1, max(e - 1, -6) - 3);
  return to_e4m3(fminf((float)(rint(want / step) * step), 448.f));
}
template <typename F>
__device__ __forceinline__ uint32_t exact_code(F y, F s) {
  const F a = fabs(y);
  // (products of a border's 3 bits and a scale's 4 are exact)
  const int n = (a > (F)0.25 * s) + (a >= (F)0.75 * s) + (a > (F)1.25 * s) + (a >= (F)1.75 * s) + (a > (F)2.5 * s) +
                (a >= (F)3.5 * s) + (a > (F)5 * s);
  return (s > (F)0 ? n : 0) + (y < (F)0 ? 8 : 0);
}

struct Row4 {
  uint32_t scale[2], code[2];   // of the lane's elements 8 l .. 8 l + 7 and 256 + 8 l ..
};
// A lane's 16 values and the neighbour's (a block is two lanes').
template <typename F>
__device__ __forceinline__ Row4 quantise_exact(const F* y) {
  Row4 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    F top = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F x = fabs(y[8 * h + i]);
      bad |= !(x < (F)INFINITY);
      top = x > top ? x : top;
    }
    const F o = __shfl_xor_sync(~0u, top, 1);
    top = o > top ? o : top;
    bad = __shfl_xor_sync(~0u, (int)bad, 1) || bad;
    r.scale[h] = bad ? 0x7f : exact_scale(top);
    r.code[h] = 0;
    const F s = bad ? (F)0 : (F)e4m3_value(r.scale[h]);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.code[h] |= exact_code(y[8 * h + i], s) << (4 * i);
  }
  return r;
}
// The same in fp32; *near: a border is too close for that.
__device__ __forceinline__ Row4 quantise_fast(const float* y, bool* near) {
  Row4 r;
  bool close = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* v = y + 8 * h;
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bad |= !(fabsf(v[i]) < INFINITY);
      top = fmaxf(top, fabsf(v[i]));
    }
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    bad = __shfl_xor_sync(~0u, (int)bad, 1) || bad;
    const float want = top * (1.f / 6.f);
    const uint32_t sc = to_e4m3(want);
    close |= to_e4m3(want * (1.f + kNear)) != to_e4m3(want * (1.f - kNear));
    const float s = e4m3_value(sc), inv = s > 0.f && !bad ? 1.f / s : 0.f;
    r.scale[h] = bad ? 0x7f : sc;
    uint32_t c = 0, up = 0, down = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = v[2 * i] * inv, q = v[2 * i + 1] * inv;
      c |= to_e2m1(p, q) << (8 * i);
      up |= to_e2m1(p * (1.f + kNear), q * (1.f + kNear)) << (8 * i);
      down |= to_e2m1(p * (1.f - kNear), q * (1.f - kNear)) << (8 * i);
    }
    r.code[h] = bad ? 0 : c;
    close |= up != down && !bad;
  }
  *near = close;
  return r;
}

// x r w / 2^k (r = rstd, or x / 2^k) in codes; the whole warp calls this.
// Rows whose sums, weights or values leave the middle of fp32's range take the
// 64 bits too, where no finite row's do.
constexpr float kLarge = 1.2676506e30f, kSmall = 1.f / kLarge;   // 2^100
template <typename T, bool NORM>
__device__ __forceinline__ Row4 quantise(const AppendArgs& a, const float* x, const T* w) {
  const int lane = threadIdx.x & 31;
  const float unit = __uint_as_float((uint32_t)(127 - a.scale_exp) << 23);   // 2^-k
  float v[16];
  bool far = false;
  if constexpr (NORM) {
    float g[16], s = 0.f;
    load_row512(w, lane, g);
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(x[i], x[i], s);
    s = warp_sum(s) * (1.0f / 512.0f) + (float)a.eps;
    far = !(s > kSmall && s < kLarge);
    const float r = 1.0f / sqrtf(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float h = g[i] * unit;
      far |= !(fabsf(h) < kLarge);
      v[i] = x[i] * r * h;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = x[i] * unit;
      far |= !(fabsf(x[i]) < kLarge);
    }
  }
  bool near;
  const Row4 fast = quantise_fast(v, &near);
  far = __any_sync(~0u, far);
  if (!far && !__any_sync(~0u, near)) return fast;
  if (!NORM && !far) return quantise_exact(v);   // v is exact, and so is every comparison in fp32
  // (of normal rows about one in a hundred)
  double y[16];
  if constexpr (NORM) {
    float g[16];
    load_row512(w, lane, g);
    double s = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fma((double)x[i], (double)x[i], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    const double r = 1.0 / sqrt(s * (1.0 / 512.0) + a.eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = (double)x[i] * r * (double)g[i] * (double)unit;
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = (double)x[i] * (double)unit;
  }
  return quantise_exact(y);
}

template <typename T, bool INTER, bool SLOTS, bool PACKED>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(AppendArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    if (!PACKED && a.kw) load_row512((const T*)a.kw, lane, g);
    const Spot s = SLOTS ? by_slot(a, t) : by_table(a, t, true);
    if (!s.ok) return;
    T* dst_rope;
    if constexpr (PACKED) {
      uint8_t* dst = (uint8_t*)a.cache + (size_t)s.row * (kRopeAt + (a.pg.row - 512) * 2);
      const Row4 q = a.kw ? quantise<T, true>(a, v, (const T*)a.kw) : quantise<T, false>(a, v, nullptr);
      uint32_t* codes = reinterpret_cast<uint32_t*>(dst);
      codes[lane] = q.code[0];
      codes[lane + 32] = q.code[1];
      if (!(lane & 1)) {
        dst[kCodes + (lane >> 1)] = (uint8_t)q.scale[0];
        dst[kCodes + 16 + (lane >> 1)] = (uint8_t)q.scale[1];
      }
      dst_rope = reinterpret_cast<T*>(dst + kRopeAt);
    } else {
      T* dst = (T*)a.cache + (size_t)s.row * a.pg.row;
      if (a.kw) {
        const float r = row_rstd(v, (float)a.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= r * g[i];
      }
      store_row512(dst, lane, v);
      dst_rope = dst + 512;
    }
    if (a.cs) {
      Angles ang;
      spot_angles<INTER, SLOTS>(a, s, lane & 7, &ang);
      rotate8<INTER>(rope, ang, 1.f);
      if (lane < 8) reinterpret_cast<uint4*>(dst_rope)[lane] = pack8<T>(rope);
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
  const Spot s = SLOTS ? by_slot(a, t) : by_table(a, t, false);
  if (!s.ok) return;
  Angles ang;
  spot_angles<INTER, SLOTS>(a, s, lane & 7, &ang);
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
  auto pick = [&](auto inter) {
    constexpr bool I = decltype(inter)::value;
    return a.slots ? (a.packed ? append_kernel<T, I, true, true> : append_kernel<T, I, true, false>)
                   : (a.packed ? append_kernel<T, I, false, true> : append_kernel<T, I, false, false>);
  };
  auto kern = a.interleaved ? pick(std::true_type{}) : pick(std::false_type{});
  kern<<<(unsigned)n, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template cudaError_t launch_append<__nv_bfloat16>(AppendArgs, cudaStream_t);
template cudaError_t launch_append<__half>(AppendArgs, cudaStream_t);

}  // namespace sfa
