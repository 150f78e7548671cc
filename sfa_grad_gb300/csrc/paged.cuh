// What the paged kernels share: a call's sizes and index arrays, and the
// search for a new token's sequence.
#pragma once
#include "common.cuh"

namespace sfa {

// Device error codes of the paged calls, beside common.cuh's.
constexpr int kErrPage = 3;          // a block table entry outside the cache
constexpr int kErrPosition = 4;      // append: a position outside the rotation table
constexpr int kErrPool = 5;          // plan: fewer free pages than the step needs, or more than there are

struct Paged {
  const int* table;    // (B, max_pages)
  const int* act_q;    // (B) or null (BSND: every sequence has S1 new tokens)
  const int* act_kv;   // (B)
  int tnd, B, S1, T;   // T: rows of q, tokens (BSND: B * S1)
  int G, row;          // query heads; elements of a cache row (512 or 576)
  int num_pages, page_size, max_pages;
  int mode;            // 0 or 3
};

struct SeqTok {
  int seq;    // -1: the token belongs to no sequence
  int i;      // index among its sequence's new tokens
  int qlen;
  bool bad;   // seq = -1 because of a negative or too large length
};

// The sequence of token t (row of q), found by one warp; every lane gets it.
__device__ __forceinline__ SeqTok find_token(const Paged& p, int t) {
  SeqTok r{-1, 0, 0, false};
  const int lane = threadIdx.x & 31;
  if (!p.tnd) {
    const int b = t / p.S1, i = t - b * p.S1;
    const int q = p.act_q ? __ldg(p.act_q + b) : p.S1;
    r.bad = q < 0 || q > p.S1;
    if (!r.bad && i < q) r = SeqTok{b, i, q, false};
    return r;
  }
  long long before = 0;   // tokens of the sequences behind us
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int q = b0 + lane < p.B ? __ldg(p.act_q + b0 + lane) : 0;
    const unsigned neg = __ballot_sync(~0u, q < 0);   // sequences before a negative length still stand
    long long sum = max(q, 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += u;
    }
    const unsigned hit = __ballot_sync(~0u, before + sum > t);
    if (neg && (!hit || __ffs(neg) < __ffs(hit))) {
      r.bad = true;
      return r;
    }
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int ql = __shfl_sync(~0u, q, l);
      const long long end = __shfl_sync(~0u, sum, l);
      r.bad = before + end > p.T;   // more tokens than there are
      if (r.bad) return r;
      return SeqTok{b0 + l, (int)(t - (before + end - ql)), ql, false};
    }
    before += __shfl_sync(~0u, sum, 31);
  }
  return r;
}

}  // namespace sfa
