// Append of new tokens' latent rows to the paged cache, with the norm of the
// latent part and the position rotation on the way (sfa_cache_append), in 16 or
// in 4 bits (sfa_cache4_append), by block tables or by a slot map
// (sfa_cache_append_slots).
//
// One warp a token writes its 1152-byte row straight to its page; further
// warps rotate the tokens' query rows, 32 heads each, so that a decoding step
// has one launch ahead of its attention.  Bound by the rows' bytes, and with
// few tokens by the latency of the lengths, the block table and the row, read
// one after the other.  Measured, bf16: 64 single tokens x 128 heads 6.2 us;
// 8 chunks, 13,045 tokens x 64 heads, 47.3 us, 5.2 TB/s.  By slots, fp16, 13,045 tokens
// with 16 heads from cold caches: into 4 bits 26.0 us, into 16 bits 24.1; keys alone
// 23.3 and 15.1; from warm caches 20.6 and 17.3, keys alone 17.4 and 8.6.  Into 4 bits
// a row close to a border takes its warp some 6 us, and a launch of four waves
// waits for the last.
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
template <bool INTER>
struct Spot {
  bool ok;         // else: left out
  long long row;   // of the cache
  int pos;         // by table: the position
  PairsAt<INTER> at;   // by slot: the pairs'
};
// The row follows from the token's position and its sequence's block table;
// page = false: only the position is wanted.
template <bool INTER>
__device__ __forceinline__ Spot<INTER> by_table(const AppendArgs& a, int t, bool page) {
  const SeqTok s = find_token(a.pg, t);
  Spot<INTER> r{};
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
  r.pos = (int)pos;
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
template <bool INTER>
__device__ __forceinline__ Spot<INTER> by_slot(const AppendArgs& a, int t) {
  Spot<INTER> r{};
  const int slot = __ldg(a.slots + t);
  if (a.cs) r.at.load(a.pos, t, a.pg.T, a.axes, a.axis_map, a.table_len);
  if (slot < 0) return r;
  if (slot >= (long long)a.pg.num_pages * a.pg.page_size) {
    if (a.error) *a.error = kErrPage;
    return r;
  }
  if (a.cs && r.at.pad) {
    if (a.error) *a.error = kErrPosition;
    return r;
  }
  r.row = slot;
  r.ok = true;
  return r;
}
template <bool INTER, bool SLOTS>
__device__ __forceinline__ void spot_angles(const AppendArgs& a, const Spot<INTER>& s, int piece, Angles* ang) {
  if constexpr (SLOTS)
    s.at.angles(a.cs, a.axis_map, piece, ang);
  else
    load_angles<INTER>(a.cs + (size_t)s.pos * 64, piece, ang);
}

// ------------------------------------------------------------------ rows of 4 bits
// y / 2^k in blocks of 16: the scale is max|y| / 6 in e4m3, a code the value
// nearest to y / scale, ties to even, both of the exact y: a value that fp32's
// roundings could carry over a border between two codes or two scales is
// found, and its row is quantised again from its inputs, in more bits.  A code
// takes y's sign, zeros' too (as the conversion does it), so that a row's bytes
// do not depend on the way it took.
//
// Roundings of fp32 on the way, 2^-24 each: 4 + 2 + 5 additions of squares and
// the one of eps, halved by the square root; root, reciprocal, two products; the
// division by 6 or by the scale, two more; 12 in all, and one to look aside.
// What is within 16 of them (2^-20) of a border is near: a scale of one normal row in
// 1400, a code of one in 480.
constexpr float kNear = 1.0f / (1 << 20);

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
struct Row4 {
  uint32_t scale[2], code[2];   // of the lane's elements 8 l .. 8 l + 7 and 256 + 8 l ..
};
// The scale nearest to top / 6, top exact (a border between two scales is 3 times
// their sum, exact too; scales ascend with their bytes, a tie goes to the even
// one): fp32's, or one of its neighbours.
template <typename Above, typename Is>
__device__ __forceinline__ uint32_t next_scale(uint32_t b, Above above, Is is, float* up, float* down) {
  *up = 3.f * (e4m3_value(b) + e4m3_value(min(b + 1, 126u)));
  *down = 3.f * (e4m3_value(max(b, 1u) - 1) + e4m3_value(b));
  if (b < 126 && (above(*up) || (is(*up) && (b & 1)))) return b + 1;
  if (b > 0 && !above(*down) && !(is(*down) && !(b & 1))) return b - 1;
  return b;
}
// The code nearest to a / s: borders between codes, times the scale, are exact.
template <typename Above, typename Is>
__device__ __forceinline__ uint32_t code_of(float s, Above above, Is is) {
  constexpr float borders[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
  uint32_t n = 0;
#pragma unroll
  for (int k = 0; k < 7; ++k) n += above(borders[k] * s) || ((k & 1) && is(borders[k] * s));   // ties to the even code
  return s > 0.f ? n : 0;
}

// A lane's 16 values (a block is two lanes') in fp32; *near: some border is too
// close for that, unless the values are EXACT.  A block with a value that is
// not finite gets a scale that is not a number.
template <bool EXACT>
__device__ __forceinline__ Row4 quantise(const float* y, bool* near) {
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
    uint32_t sc = to_e4m3(want);
    if constexpr (EXACT) {
      float up, down;
      sc = next_scale(sc, [&](float b) { return top > b; }, [&](float b) { return top == b; }, &up, &down);
      const float s = e4m3_value(sc);
      r.scale[h] = bad ? 0x7f : sc;
      r.code[h] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(v[i]);
        const uint32_t n = code_of(s, [&](float b) { return a > b; }, [&](float b) { return a == b; });
        r.code[h] |= (bad ? 0 : n + (signbit(v[i]) ? 8 : 0)) << (4 * i);
      }
      continue;
    }
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

// Sums and products of fp32 with their rounding errors (Knuth, Dekker): the
// result is x.h + x.l.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(const Two& a, const Two& b) {
  const Two s = two_sum(a.h, b.h);
  return two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ bool above(const Two& a, float b) { return a.h > b || (a.h == b && a.l > 0.f); }
__device__ __forceinline__ bool is(const Two& a, float b) { return a.h == b && a.l == 0.f; }

// The whole row from its inputs, two blocks at a time: in pairs of fp32, which
// are 2^-43 off and say so (false) where that does not decide, or (WIDE) in 64
// bits.  (In 64 bits alone, whose operations take this GPU some 100 clk each,
// 13,045 rows took 35 us instead of 25, 41 with the loop rolled.)
template <typename T, bool NORM, bool WIDE>
__device__ __noinline__ bool quantise_exact(const T* x, const T* w, double eps, float unit, uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  Two r = {1.f, 0.f};
  double wide = 1;
  static_assert(NORM || WIDE, "without a norm fp32 holds the values");
  if constexpr (!WIDE) {
    Two s = {0.f, 0.f};
#pragma unroll 4
    for (int i = lane; i < 512; i += 32) {
      const float v = Elt<T>::to_f(x[i]);
      s = add(s, Two{__fmul_rn(v, v), 0.f});   // the square of 11 bits is exact
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) s = add(s, Two{__shfl_xor_sync(~0u, s.h, o), __shfl_xor_sync(~0u, s.l, o)});
    const float e = (float)eps;
    s = add(Two{s.h * (1.f / 512.f), s.l * (1.f / 512.f)}, Two{e, (float)(eps - (double)e)});
    // one step of Newton's from fp32's root: what 1 - s r^2 leaves, halved
    r.h = 1.0f / sqrtf(s.h);
    const float p = __fmul_rn(r.h, r.h), pl = fmaf(r.h, r.h, -p), q = __fmul_rn(s.h, p), ql = fmaf(s.h, p, -q);
    const float rest = __fsub_rn(__fsub_rn(1.f, q), __fadd_rn(ql, fmaf(s.h, pl, __fmul_rn(s.l, p))));
    r.l = 0.5f * r.h * rest;
  } else if constexpr (NORM) {
    double s = 0;
#pragma unroll 1
    for (int i = lane; i < 512; i += 32) {
      const double v = Elt<T>::to_f(x[i]);
      s = fma(v, v, s);
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    wide = rsqrt(s * (1.0 / 512.0) + eps);
  }
  bool sure = true;
#pragma unroll(WIDE ? 1 : 4)
  for (int i = 0; i < 16; ++i) {
    const int e = 32 * i + lane;
    Two a;
    bool negative;
    if constexpr (WIDE) {
      double y = (double)Elt<T>::to_f(x[e]) * (double)unit;
      if (NORM) y = y * wide * (double)Elt<T>::to_f(w[e]);
      negative = signbit(y);
      y = fmin(fabs(y), 1e38);   // far past the largest scale
      y = Elt<T>::to_f(x[e]) - Elt<T>::to_f(x[e]) == 0.f && (!NORM || Elt<T>::to_f(w[e]) - Elt<T>::to_f(w[e]) == 0.f) &&
                  wide - wide == 0
              ? y
              : (double)INFINITY;
      a.h = (float)y;
      a.l = a.h < INFINITY ? (float)(y - (double)a.h) : 0.f;
    } else {
      const float c = __fmul_rn(Elt<T>::to_f(x[e]), Elt<T>::to_f(w[e])) * unit;   // exact
      negative = signbit(c);
      a.h = __fmul_rn(fabsf(c), r.h);
      a.l = fmaf(fabsf(c), r.h, -a.h) + fabsf(c) * r.l;
      if (a.h < INFINITY) a = two_sum(a.h, a.l);
    }
    const bool bad = !(a.h < INFINITY);
    Two top = bad ? Two{0.f, 0.f} : a;
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      const Two u = {__shfl_xor_sync(~0u, top.h, o), __shfl_xor_sync(~0u, top.l, o)};
      if (u.h > top.h || (u.h == top.h && u.l > top.l)) top = u;
    }
    const bool none = (__ballot_sync(~0u, bad) >> (lane & 16)) & 0xffff;
    float up, down;
    const uint32_t b = next_scale(to_e4m3(fminf(top.h, 2688.f) * (1.f / 6.f)), [&](float x) { return above(top, x); },
                                  [&](float x) { return is(top, x); }, &up, &down);
    auto unsure = [&](const Two& v, float border) {
      return !WIDE && v.h == border && border != 0.f && fabsf(v.l) <= v.h * (1.f / (1ull << 42));
    };
    sure &= !unsure(top, up) && !unsure(top, down);
    const float s = e4m3_value(b);
    uint32_t n = code_of(
        s, [&](float x) { return sure &= none || !unsure(a, x), above(a, x); }, [&](float x) { return is(a, x); });
    n = none ? 0 : n + (negative ? 8 : 0);
    const uint32_t high = __shfl_xor_sync(~0u, n, 1);
    if (!(lane & 1)) dst[16 * i + (lane >> 1)] = (uint8_t)(n | high << 4);
    if (!(lane & 15)) dst[kCodes + 2 * i + (lane >> 4)] = none ? 0x7f : (uint8_t)b;
  }
  return __all_sync(~0u, sure);
}

// y = x r w / 2^k (r = rstd, or x / 2^k) into a row; the whole warp calls this
// with the row in its lanes.  Rows whose sums, weights or values leave the middle
// of fp32's range take the 64 bits too, where no finite row's do.  (A square root
// of 512 sums below 2^100 times a weight below 2^60 leaves products with weights,
// which come before the factor r, below 2^119.)
constexpr float kLarge = 1.2676506e30f, kSmall = 1.f / kLarge;   // 2^100
constexpr float kLargeWeight = 1.1529215e18f;                    // 2^60
template <typename T, bool NORM>
__device__ __forceinline__ void store_row4(const AppendArgs& a, int t, const float* x, uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  const float unit = __uint_as_float((uint32_t)(127 - a.scale_exp) << 23);   // 2^-k
  float v[16];
  bool far = false;
  if constexpr (NORM) {
    float g[16], sum[4] = {0.f, 0.f, 0.f, 0.f};
    load_row512((const T*)a.kw, lane, g);
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i & 3] = fmaf(x[i], x[i], sum[i & 3]);
    const float s = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3])) * (1.0f / 512.0f) + (float)a.eps;
    far = !(s > kSmall && s < kLarge);
    const float r = 1.0f / sqrtf(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float h = g[i] * unit;
      far |= !(fabsf(h) < kLargeWeight);
      v[i] = x[i] * r * h;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = x[i] * unit;
      far |= !(fabsf(x[i]) < kLarge);
    }
  }
  bool near = false;
  const Row4 q = quantise<!NORM>(v, &near);
  far = __any_sync(~0u, far);
  if (far || __any_sync(~0u, near)) {
    const T* row = (const T*)a.k + (size_t)t * 512;
    bool done = false;
    if constexpr (NORM) done = !far && quantise_exact<T, true, false>(row, (const T*)a.kw, a.eps, unit, dst);
    if (!done) quantise_exact<T, NORM, true>(row, (const T*)a.kw, a.eps, unit, dst);
    return;
  }
  uint32_t* codes = reinterpret_cast<uint32_t*>(dst);
  codes[lane] = q.code[0];
  codes[lane + 32] = q.code[1];
  if (!(lane & 1)) {
    dst[kCodes + (lane >> 1)] = (uint8_t)q.scale[0];
    dst[kCodes + 16 + (lane >> 1)] = (uint8_t)q.scale[1];
  }
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
    const Spot<INTER> s = SLOTS ? by_slot<INTER>(a, t) : by_table<INTER>(a, t, true);
    if (!s.ok) return;
    T* dst_rope;
    if constexpr (PACKED) {
      uint8_t* dst = (uint8_t*)a.cache + (size_t)s.row * (kRopeAt + (a.pg.row - 512) * 2);
      if (a.kw)
        store_row4<T, true>(a, t, v, dst);
      else
        store_row4<T, false>(a, t, v, dst);
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
  const Spot<INTER> s = SLOTS ? by_slot<INTER>(a, t) : by_table<INTER>(a, t, false);
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
