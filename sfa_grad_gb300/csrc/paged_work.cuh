// What the kernels of the paged attention share: the work of a call and its
// even split over workers (a CTA, or a pair of them), the bounded waits, the
// scaling of scores, and the pieces that the merge adds up.
#pragma once
#include "kernels.h"
#include "rows.cuh"

namespace sfa {

constexpr float kRaise = 8.0f;              // log2 growth of a row's max that rescales O
// How scores are scaled.  The sign is taken out first, so that a larger score
// is a larger weight, and a scale of zero becomes one that leaves every finite
// score zero and a masked one -inf.
struct Scale {
  bool negative;
  float scale, log2;   // |scale|, times log2(e)
};
// (The tensor core adds each step of 16 products to a score in fp32, rounding
// towards zero.  Scores whose partial sums fp32 holds exactly lose nothing by
// that; measured, others come out short by 1 to 16 (bf16) and 4 to 54 (fp16) x 2^-24 of
// themselves, normal rows by 9 and 11, rows of one sign by the most.  No factor
// makes that up: it would have to know the rows.)
__device__ __forceinline__ Scale score_scale(float scale) {
  const float s = fabsf(scale);
  return {scale < 0.f, s, fmaxf(s * kLog2e, 1.4e-45f)};   // at least fp32's smallest value
}

// One piece of work: key tiles kt0 .. kt1 - 1 of a row tile.
struct Seg {
  int row0, nrows;        // rows of q, row0 the first
  int i0;                 // first row's index in its sequence (token * heads + head)
  int kt0, kt1;           // kt1 = 0: end of the work
  int kend;               // keys any row sees
  int base;               // mode 3: last key of the sequence's first new token; mode 0: of every token
  int slot;               // -1: whole row tile; else where the piece's result goes
};

// A piece's place in the workspace, for the merge.
struct Piece {
  int valid, row0, nrows;
  int first, last;        // begins / ends its row tile
  int pad[3];
};

// A worker's share of the work: where it begins, and its size in key tiles.
struct Share {
  int seq, row, tile, kt;      // sequence, its first row, row tile of it, key tile of that
  int bad, ntiles;
  // the two ends: sequence, offset into its cost, key tiles before it
  int end_seq[2];
  long long end_off[2], end_before[2], end_units[2];
};

// Bounded waits of these kernels: as common.cuh's, with the limit in SM clocks
// (a read of the global timer costs more than most waits here last).  The
// first look at a barrier does not suspend, so that the limit counts from the
// beginning, and where the limit is short none does: a suspension, 10 us at
// most, would outlast it (waits of 1 to 4 us did not notice a limit of 1, with
// a hint of 0.25 us for the suspension neither).  512 tokens x 128 heads over
// 16384 keys take 1369 us so, and 1361 with a first look that suspends.
struct Limit {
  volatile int* abort;
  int* gerr;
  long long clocks;
  int brief;               // no suspensions
};
__device__ __forceinline__ Limit wait_limit(int* abort, int* status, const PagedArgs& a) {
  return {abort, status, (long long)(a.wait_ns * 21 / 10), a.brief};   // SM clock at most 2.1 GHz
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const Limit& w) {
  const uint32_t a = smem_u32(bar);
  if (mbar_poll(a, parity)) return true;
  const long long t0 = clock64();
  while (!(w.brief ? mbar_poll(a, parity) : mbar_test(a, parity))) {
    if (*w.abort) return false;
    if (clock64() - t0 > w.clocks) {
      *w.abort = 1;
      atomicExch(w.gerr, kErrTimeout);
      return false;
    }
  }
  return true;
}
// Wait by a whole warp: one answer for all lanes, and the lanes together again
// before what follows (tcgen05.ld and .st want a converged warp).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Limit& w) {
  const bool ok = wait_bar(bar, parity, w);
  return __all_sync(~0u, ok);
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ the work
struct SeqWork {
  int qlen, kvlen, rows, tiles;
};
// The work in row tiles of kRows and key tiles of kKeys.
template <int kRows, int kKeys, int kThreads, int kOwn>
struct Work {
  static_assert(kRows == 32 || kRows == 64 || kRows == 128, "a shift");
  static_assert(kKeys % kRows == 0, "whole units of d");
  // Row tile j of a sequence: keys its last row sees, and its key tiles (at
  // least one: a tile without keys still writes its rows).
  static __device__ __forceinline__ SeqWork seq_work(const Paged& p, int b) {
    SeqWork s;
    s.qlen = p.act_q ? __ldg(p.act_q + b) : p.S1;
    s.kvlen = __ldg(p.act_kv + b);
    s.rows = s.qlen * p.G;
    s.tiles = (s.rows + kRows - 1) / kRows;
    return s;
  }
  static __device__ __forceinline__ int tile_keys(const Paged& p, const SeqWork& s, int j) {
    if (p.mode == 0) return s.kvlen;
    const int tok = min((j + 1) * kRows - 1, s.rows - 1) / p.G;
    return max(0, s.kvlen - s.qlen + tok + 1);
  }
  static __device__ __forceinline__ int tile_units(const Paged& p, const SeqWork& s, int j) {
    return max(1, (tile_keys(p, s, j) + kKeys - 1) / kKeys);
  }
  // Key tiles of row tiles 0 .. n-1, n < tiles (mode 3).  Tile j ends at token
  // (128 j + 127) / G, so its units are max(1, (j + e) / d) rounded down with d =
  // 2 G and e = (127 + G (base + 256)) / 128 rounded down: ones while j + e <
  // 2 d, then a sum over i / d.
  static __device__ __forceinline__ long long units_before(const Paged& p, const SeqWork& s, int n) {
    if (n <= 0) return 0;
    if (p.mode == 0) return (long long)n * max(1, (s.kvlen + kKeys - 1) / kKeys);
    const int d = kKeys / kRows * p.G;
    const long long x = kRows - 1 + (long long)p.G * (s.kvlen - s.qlen + kKeys);
    const long long e = x >> (kRows == 128 ? 7 : kRows == 64 ? 6 : 5);   // / kRows, rounded down
    const long long ones = min((long long)n, max(0LL, 2LL * d - e));
    auto sum = [&](long long m) {   // sum of i / d over i < m
      const long long q = (long long)((unsigned)m / (unsigned)d), r = m - q * d;
      return d * (q * (q - 1) / 2) + q * r;
    };
    return ones + (ones < n ? sum(n + e) - sum(ones + e) : 0);
  }
  static __device__ __forceinline__ long long seq_units(const Paged& p, const SeqWork& s) {
    return s.tiles ? units_before(p, s, s.tiles - 1) + tile_units(p, s, s.tiles - 1) : 0;
  }

  // Row tiles cost their key tiles and kOwn more, their beginning and end (none
  // where the workers get a key tile each at most): the cost before row tile n.
  static __device__ __forceinline__ long long cost_before(const Paged& p, const SeqWork& s, int n, int own) {
    return units_before(p, s, n) + (long long)own * n;
  }

  // Block-wide: checks the lengths, adds up the work and splits its cost evenly
  // and in order; this worker's share is in `c` after the next block barrier.
  // scan: 3 * kThreads / 32 elements.
  static __device__ void plan(const Paged& p, Share* c, long long* scan, int worker, int workers) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long units = 0, toks = 0;
    int tiles = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const SeqWork s = seq_work(p, b);
      const bool no = s.qlen < 0 || s.kvlen < 0 || s.qlen > (p.tnd ? p.T : p.S1) ||
                      s.kvlen > (long long)p.max_pages * p.page_size;
      bad |= no;
      if (!no) units += seq_units(p, s), tiles += s.tiles, toks += s.qlen;
    }
    // inclusive scans over the block's threads
    long long u = units, t = toks;
    int g = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long du = __shfl_up_sync(~0u, u, o), dt = __shfl_up_sync(~0u, t, o);
      const int dg = __shfl_up_sync(~0u, g, o);
      if (lane >= o) u += du, t += dt, g += dg;
    }
    if (lane == 31) scan[w] = u, scan[kWarps + w] = t, scan[2 * kWarps + w] = g;
    const bool any = __syncthreads_or(bad);
    long long total = 0, toks_all = 0, tiles_all = 0;
    if constexpr (kWarps <= 17) {
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < w) u += scan[i], t += scan[kWarps + i], g += (int)scan[2 * kWarps + i];
        total += scan[i];
        toks_all += scan[kWarps + i];
        tiles_all += scan[2 * kWarps + i];
      }
    } else {
      // More warps (rows of 4 bits): their sums one a lane.  As above the 20 warps of
      // single CTAs took 4400 clk, most of it for fetching the code, which runs
      // once a launch (one sequence of 1000 keys 25 us instead of 21); the 16
      // and 17 of the 16-bit kernels lose nothing by it.
      static_assert(kWarps <= 32, "a lane a warp");
      long long x[3], all[3], ahead[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) x[i] = lane < kWarps ? scan[i * kWarps + lane] : 0;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        long long y[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) y[i] = __shfl_up_sync(~0u, x[i], o);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (lane >= o) x[i] += y[i];
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        all[i] = __shfl_sync(~0u, x[i], 31);
        ahead[i] = __shfl_sync(~0u, x[i], (w + 31) & 31);
      }
      if (w) u += ahead[0], t += ahead[1], g += (int)ahead[2];
      total = all[0], toks_all = all[1], tiles_all = all[2];
    }
    const bool wrong = any || (p.tnd && toks_all > p.T) || total > (long long)workers * (INT32_MAX / 2);
    const int np = total < 1 ? 1 : total < workers ? (int)total : workers;
    const int own = total > workers ? kOwn : 0;
    // shares of cost / np, the first cost % np workers one more
    const long long cost = total + own * tiles_all;
    const long long share = cost >> 32 ? cost / np : (unsigned)cost / (unsigned)np;
    const int rest = (int)(cost - share * np);
    const bool mine = !wrong && total > 0 && worker < np;
    const long long first = share * worker + min(worker, rest), last = first + share + (worker < rest);
    const long long from = u - units + (long long)own * (g - tiles), to = u + (long long)own * g;
    if (tid == 0) {
      c->bad = wrong;
      c->ntiles = 0;
      if (last == cost) c->end_seq[1] = -1, c->end_units[1] = total;
    }
#pragma unroll(kWarps <= 17 ? 2 : 1)
    for (int e = 0; e < 2; ++e) {
      const long long at = e ? last : first;
      if (!mine || at < from || at >= to) continue;
      long long before = u - units, row = t - toks, cum = from;
      for (int b = b0; b < b1; ++b) {
        const SeqWork s = seq_work(p, b);
        const long long k = seq_units(p, s), all = k + (long long)own * s.tiles;
        if (at < cum + all) {
          c->end_seq[e] = b;
          c->end_off[e] = at - cum;
          c->end_before[e] = before;
          if (e == 0) c->row = (int)(p.tnd ? row : (long long)b * p.S1) * p.G;
          break;
        }
        cum += all;
        before += k;
        row += s.qlen;
      }
    }
    __syncthreads();
    if (mine && w < 2) {
      // warp e: the row tile and key tile of end e
      const int b = c->end_seq[w];
      if (b >= 0) {
        const SeqWork s = seq_work(p, b);
        const long long off = c->end_off[w];
        const int j = find_tile(p, s, off, own);
        const int kt = (int)max(0LL, off - cost_before(p, s, j, own) - own);
        if (lane == 0) {
          c->end_units[w] = c->end_before[w] + units_before(p, s, j) + kt;
          if (w == 0) c->seq = b, c->tile = j, c->kt = kt;
        }
      }
    }
    __syncthreads();
    if (mine && tid == 0) c->ntiles = (int)(c->end_units[1] - c->end_units[0]);
  }

  // The row tile at an offset into a sequence's cost: the last j with
  // cost_before(j) <= off; all lanes of a warp search together.
  static __device__ __forceinline__ int find_tile(const Paged& p, const SeqWork& s, long long off, int own) {
    int lo = 0, hi = s.tiles;   // cost_before(lo) <= off < cost_before(hi)
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
      const int step = (hi - lo + 32) / 33;
      const int j = lo + (lane + 1) * step;
      const unsigned ok = __ballot_sync(~0u, j < hi && cost_before(p, s, j, own) <= off);
      const int n = __popc(ok);   // a prefix of the lanes
      lo += n * step;
      hi = min(hi, lo + step);
    }
    return lo;
  }
};

struct Args {
  PagedArgs a;
  int workers, ctas;       // that share the work; CTAs of the grid
  int kbox, vbox;          // rows of a box of the cache (16 .. 128 and 16 .. 64)
  int* status;             // one word a CTA
  Piece* piece;
  float4* stats;           // (slot, row) x {max, the max P is relative to, sum, -}
  float* part;             // (slot, row, 512); slots 2 w and 2 w + 1 are worker w's
};

// Adds up the pieces of row tiles of `rows` rows (32, 64 or 128).
template <typename T>
cudaError_t launch_paged_merge(const Args& g, int rows, cudaStream_t st);
// The kernel of row tiles of 32 or 64 rows, one CTA each, and its merge.
template <typename T>
cudaError_t launch_paged_few(const Args& g, int rows, cudaStream_t st);

}  // namespace sfa
