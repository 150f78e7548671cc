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
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
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
// Products of two pairs of fp16, in T.
template <typename T>
__device__ __forceinline__ uint32_t product(uint32_t a, uint32_t b) {
  if constexpr (Elt<T>::is_f16) return mul2(a, b);
  float x, y;
  asm("{\n.reg .b16 a0, a1, b0, b1;\nmov.b32 {a0, a1}, %2;\nmov.b32 {b0, b1}, %3;\n"
      "fma.rn.f32.f16 %0, a0, b0, 0f80000000;\nfma.rn.f32.f16 %1, a1, b1, 0f80000000;\n}"
      : "=f"(x), "=f"(y)
      : "r"(a), "r"(b));
  return Elt<T>::pack(x, y);
}

// Codes and scales have conversions to fp16 alone, and every product of the unit's
// range is exact there; for bf16 the products are formed in fp32 and packed,
// exactly too.  (8 warps, 32 elements a lane: 104 clk in fp16, 203 in bf16; 216
// from products in fp16, 293 with exponents moved by shifts and masks, 268 with
// codes shifted into place, 354 looked up by byte permutations.)
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
    return make_uint4(product<T>(h[0], s), product<T>(h[1], s), product<T>(h[2], s), product<T>(h[3], s));
  }
};

}  // namespace sfa
