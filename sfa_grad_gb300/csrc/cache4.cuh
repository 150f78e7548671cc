// Rows of the 4-bit cache: 256 bytes of codes (element 2j in the low half of
// byte j, 2j + 1 in the high one: sign, then 0 .5 1 1.5 2 3 4 6), 32 scales of 8
// bits (e4m3, one for 16 elements), then the rotated elements in 16 bits.  An
// element is code * scale * 2^k; at most 6 significant bits, so it is exact in
// bf16 and fp16 for the k that the calls take.
#pragma once
#include "rows.cuh"

namespace sfa {

constexpr int kCodes = 256, kScales = 32;             // bytes of a row
constexpr int kRopeAt = kCodes + kScales;
// 2^k, k = -14 .. 4: 6 * 448 * 2^4 and half the smallest scale times 2^-14 are fp16 numbers
constexpr int kScaleExpMin = -14, kScaleExpMax = 4;

// Eight codes as fp16 pairs.  The bytes are named as parts of the register, which
// the conversion takes as they are: shifted into place one by one, 8 warps took
// 153 clk for 32 elements a lane instead of 104.
__device__ __forceinline__ void e2m1_f16(uint32_t w, uint32_t* h) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two scales as fp16.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hmul2(x, y);
  memcpy(&a, &x, 4);
  return a;
}
// A pair of fp16 in T.
template <typename T>
__device__ __forceinline__ uint32_t to_pair(uint32_t h) {
  if constexpr (Elt<T>::is_f16) return h;
  __half2 x;
  memcpy(&x, &h, 4);
  const float2 f = __half22float2(x);
  return Elt<T>::pack(f.x, f.y);
}

// Values are formed in fp16, where every product of the unit's range is exact;
// bf16 takes them from there, exactly too.  (8 warps, 32 elements a lane: 104
// clk in fp16, 216 in bf16; 293 with exponents moved by shifts and masks, 268
// with codes shifted into place, 354 looked up by byte permutations.)
template <typename T>
struct Dec4 {
  uint32_t unit;   // 2^k, twice (normal: k >= -14)
  __device__ explicit Dec4(int k) { unit = (uint32_t)((15 + k) << 10) * 0x10001u; }
  // Scales of two neighbouring blocks (bytes), times the unit, each as a pair.
  __device__ __forceinline__ void scales(uint32_t two, uint32_t* s) const {
    const uint32_t h = mul2(e4m3_f16(two), unit);
    s[0] = __byte_perm(h, h, 0x1010);
    s[1] = __byte_perm(h, h, 0x3232);
  }
  // Eight elements of a block as pairs.
  __device__ __forceinline__ uint4 eight(uint32_t w, uint32_t s) const {
    uint32_t h[4];
    e2m1_f16(w, h);
    return make_uint4(to_pair<T>(mul2(h[0], s)), to_pair<T>(mul2(h[1], s)), to_pair<T>(mul2(h[2], s)),
                      to_pair<T>(mul2(h[3], s)));
  }
};

}  // namespace sfa
