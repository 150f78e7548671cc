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

// Two codes (a byte of w, b = 0 .. 3) as fp16.
__device__ __forceinline__ uint32_t e2m1_f16(uint32_t w, int b) {
  uint32_t r;
  asm("{\n.reg .b8 x, y, z, u;\nmov.b32 {x, y, z, u}, %1;\ncvt.rn.f16x2.e2m1x2 %0, x;\n}" : "=r"(r) : "r"(w >> (8 * b)));
  return r;
}
// Two scales as fp16.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
template <typename T2>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  T2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  const T2 r = __hmul2(x, y);
  uint32_t u;
  memcpy(&u, &r, 4);
  return u;
}
// fp16 pairs as bf16 pairs times 2^-112: both exponents then count from the
// same place.  For values with at most 7 mantissa bits, none subnormal.
__device__ __forceinline__ uint32_t f16_bf16(uint32_t h) { return (h & 0x80008000u) | ((h >> 3) & 0x0FFF0FFFu); }

template <typename T>
struct Dec4;
template <>
struct Dec4<__half> {
  uint32_t unit;   // 2^k, twice (normal: k >= -14)
  __device__ explicit Dec4(int k) { unit = (uint32_t)((15 + k) << 10) * 0x10001u; }
  // Scales of two neighbouring blocks (bytes), times the unit, each as a pair.
  __device__ __forceinline__ void scales(uint32_t two, uint32_t* s) const {
    const uint32_t h = mul2<__half2>(e4m3_f16(two), unit);
    s[0] = __byte_perm(h, h, 0x1010);
    s[1] = __byte_perm(h, h, 0x3232);
  }
  // Eight elements of a block as pairs.
  __device__ __forceinline__ uint4 eight(uint32_t w, uint32_t s) const {
    return make_uint4(mul2<__half2>(e2m1_f16(w, 0), s), mul2<__half2>(e2m1_f16(w, 1), s),
                      mul2<__half2>(e2m1_f16(w, 2), s), mul2<__half2>(e2m1_f16(w, 3), s));
  }
};
// (bf16: codes have no conversion of their own.  Through fp16, two logical
// operations and the multiplication, which also takes the 2^112 back, measured
// less than codes shifted into place or looked up by byte permutations.)
template <>
struct Dec4<__nv_bfloat16> {
  uint32_t unit;   // 2^(112 + k), twice: k <= 4 leaves it and 448 of it finite
  __device__ explicit Dec4(int k) { unit = (uint32_t)((127 + 112 + k) << 7) * 0x10001u; }
  __device__ __forceinline__ void scales(uint32_t two, uint32_t* s) const {
    // an e4m3 NaN's mantissa survives the shift; 2^112 takes the shift's factor back
    constexpr uint32_t up = ((127 + 112) << 7) * 0x10001u;
    const uint32_t t = e4m3_f16(two);
    uint32_t h = f16_bf16(t);
    // (the shift makes an fp16 NaN, all exponent bits set, a finite bf16)
    if ((t & 0x7C00u) == 0x7C00u) h |= 0x7FC0u;
    if ((t & 0x7C000000u) == 0x7C000000u) h |= 0x7FC00000u;
    h = mul2<__nv_bfloat162>(mul2<__nv_bfloat162>(h, up), unit);
    s[0] = __byte_perm(h, h, 0x1010);
    s[1] = __byte_perm(h, h, 0x3232);
  }
  __device__ __forceinline__ uint4 eight(uint32_t w, uint32_t s) const {
    return make_uint4(mul2<__nv_bfloat162>(f16_bf16(e2m1_f16(w, 0)), s), mul2<__nv_bfloat162>(f16_bf16(e2m1_f16(w, 1)), s),
                      mul2<__nv_bfloat162>(f16_bf16(e2m1_f16(w, 2)), s), mul2<__nv_bfloat162>(f16_bf16(e2m1_f16(w, 3)), s));
  }
};

}  // namespace sfa
