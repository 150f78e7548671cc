// Pieces of the latent-row kernels (rows.cu, append.cu): 16-byte pieces of
// 16-bit elements as fp32 values, the 512-wide norm of a row held by one warp
// and the position rotation of a 16-byte piece of a 64-wide row.
#pragma once
#include "common.cuh"

namespace sfa {

// Element pairs of a 16-byte piece as fp32.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    T h[2];
    memcpy(h, &u[i], 4);
    v[2 * i] = Elt<T>::to_f(h[0]);
    v[2 * i + 1] = Elt<T>::to_f(h[1]);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(Elt<T>::pack(v[0], v[1]), Elt<T>::pack(v[2], v[3]), Elt<T>::pack(v[4], v[5]),
                    Elt<T>::pack(v[6], v[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// One warp's row of 512: lane l holds elements 8l .. 8l+7 (v[0..7]) and
// 256 + 8l .. (v[8..15]).
template <typename T>
__device__ __forceinline__ void load_row512(const T* row, int lane, float* v) {
  const uint4* p = reinterpret_cast<const uint4*>(row);
  const uint4 a = p[lane], b = p[lane + 32];
  unpack8<T>(a, v);
  unpack8<T>(b, v + 8);
}
template <typename T>
__device__ __forceinline__ void store_row512(T* row, int lane, const float* v) {
  uint4* p = reinterpret_cast<uint4*>(row);
  p[lane] = pack8<T>(v);
  p[lane + 32] = pack8<T>(v + 8);
}
// 1 / sqrt(mean of squares + eps), by every lane.
__device__ __forceinline__ float row_rstd(const float* v, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s = fmaf(v[i], v[i], s);
  return 1.0f / sqrtf(warp_sum(s) * (1.0f / 512.0f) + eps);
}

// Angles of piece c (0..7) of a 64-wide row at one position: interleaved, the
// piece holds pairs 4c .. 4c+3 (c[0..3], s[0..3]); else elements 8c .. 8c+7
// belong to pairs 8(c % 4) .. + 7 (c[0..7], s[0..7]).
struct Angles {
  float c[8], s[8];
};
template <bool INTER>
__device__ __forceinline__ void load_angles(const float* cs_row, int piece, Angles* a) {
  const float4* p = reinterpret_cast<const float4*>(cs_row);
  if (INTER) {
    const float4 c = __ldg(p + piece), s = __ldg(p + 8 + piece);
    a->c[0] = c.x; a->c[1] = c.y; a->c[2] = c.z; a->c[3] = c.w;
    a->s[0] = s.x; a->s[1] = s.y; a->s[2] = s.z; a->s[3] = s.w;
  } else {
    const int q = (piece & 3) * 2;
    const float4 c0 = __ldg(p + q), c1 = __ldg(p + q + 1), s0 = __ldg(p + 8 + q), s1 = __ldg(p + 9 + q);
    a->c[0] = c0.x; a->c[1] = c0.y; a->c[2] = c0.z; a->c[3] = c0.w;
    a->c[4] = c1.x; a->c[5] = c1.y; a->c[6] = c1.z; a->c[7] = c1.w;
    a->s[0] = s0.x; a->s[1] = s0.y; a->s[2] = s0.z; a->s[3] = s0.w;
    a->s[4] = s1.x; a->s[5] = s1.y; a->s[6] = s1.z; a->s[7] = s1.w;
  }
}
// Positions of a token on up to four axes; pair i turns by the one that bits
// 2i, 2i + 1 of a `map` name.  Axes that are not there repeat the first.
struct Places {
  int p[4];
};
__device__ __forceinline__ Places load_places(const int* pos, int t, int tokens, int axes) {
  Places r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = __ldg(pos + (i < axes ? (size_t)i * tokens : 0) + t);
  return r;
}
__device__ __forceinline__ bool outside(const Places& r, long long table_len) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= r.p[i] < 0 || r.p[i] >= table_len;
  return bad;
}
// Where a token's pairs are turned to, on several axes, and the angles of a
// piece; by a whole warp.  Interleaved, a lane reads its piece's four pairs.
// Else a piece has eight: a lane reads its own pair's angle, and the pieces take
// theirs from the lanes.  (Each the other way: 4096 tokens x 128 heads
// interleaved 28.5 instead of 24 us, 16381 x 64 not interleaved 53 instead of 51,
// the append of 13,045 rows of 4 bits with 16 heads 29 instead of 25.)
template <bool INTER>
struct PairsAt {
  Places all;
  int own;
  bool pad;   // outside the table on some axis
  __device__ __forceinline__ void load(const int* pos, int t, int tokens, int axes, unsigned long long map,
                                       long long table_len) {
    if constexpr (INTER) {
      all = load_places(pos, t, tokens, axes);
      pad = outside(all, table_len);
      if (pad) all = Places{{0, 0, 0, 0}};
    } else {
      const int lane = threadIdx.x & 31;
      const int p = lane < axes ? __ldg(pos + (size_t)lane * tokens + t) : 0;
      pad = __any_sync(~0u, p < 0 || p >= table_len);
      own = __shfl_sync(~0u, p, (int)(map >> (2 * lane)) & 3);
      if (pad) own = 0;
    }
  }
  __device__ __forceinline__ void angles(const float* cs, unsigned long long map, int piece, Angles* a) const {
    if constexpr (INTER) {
      const uint32_t m = (uint32_t)(map >> (8 * piece));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t axis = m >> (2 * i) & 3;
        const int at = axis == 0 ? all.p[0] : axis == 1 ? all.p[1] : axis == 2 ? all.p[2] : all.p[3];
        const float* row = cs + (size_t)at * 64 + piece * 4 + i;
        a->c[i] = __ldg(row);
        a->s[i] = __ldg(row + 32);
      }
    } else {
      const float* row = cs + (size_t)own * 64 + (threadIdx.x & 31);
      const float c = __ldg(row), s = __ldg(row + 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a->c[i] = __shfl_sync(~0u, c, (piece & 3) * 8 + i);
        a->s[i] = __shfl_sync(~0u, s, (piece & 3) * 8 + i);
      }
    }
  }
};
// Rotates the lane's piece (lane % 8 = piece) by +angle, or by -angle
// (sgn = -1).  Not interleaved, a pair's halves sit four lanes apart: every
// lane of the warp calls this.
template <bool INTER>
__device__ __forceinline__ void rotate8(float* v, const Angles& a, float sgn) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1], s = a.s[i] * sgn;
      v[2 * i] = x * a.c[i] - y * s;
      v[2 * i + 1] = y * a.c[i] + x * s;
    }
  } else {
    // first half: a c - b s; second half: b c + a s
    const float d = (threadIdx.x & 4) ? sgn : -sgn;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_xor_sync(~0u, v[i], 4);
      v[i] = v[i] * a.c[i] + o * (a.s[i] * d);
    }
  }
}

}  // namespace sfa
