// Block tables and slot maps of a step from the requests' lengths
// (sfa_page_plan).
//
// Three running sums over the requests (new tokens, pages they need, pages
// that ended requests give back) decide everything: the free pages and, behind
// them, the ones given back are one stack, new pages come from its end, and an
// item (a token, a new page, a page that stays free) finds its request by a
// search in the sums.  Every block adds the sums up for itself and takes a
// share of the items; what one reads no other writes (the table's rows that
// grow are not those that end, and the stack is read above the place up to
// which it is written), so one launch does without a wait in between.
//
// Bound by latency: the lengths, the sums, the table's and the stack's entries,
// one after the other.  64 requests 5.2 us; 1024, 24 of them prompts, with
// 52,627 new tokens and 24,130 pages that move 7.0 us; from cold caches 6.4 and 8.7.
// 8192 requests 28 us: every block adds up all of them.
#include "kernels.h"

namespace sfa {
namespace {

constexpr int kThreads = 512;

// First i < n with sum[i] > x (n: none).
__device__ __forceinline__ int find(const int* sum, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (sum[m] > x) hi = m;
    else lo = m + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  extern __shared__ int sums[];   // inclusive, of requests: new tokens, new pages, pages back
  int *toks = sums, *grown = sums + a.B, *back = sums + 2 * a.B;
  __shared__ long long part[3][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, ps = a.page_size;
  const long long cap = (long long)a.max_pages * ps;
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  auto pages = [&](int n) { return (n + ps - 1) / ps; };   // lengths stay below 2^30

  long long s[3] = {0, 0, 0};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int kv = __ldg(a.kv + b), n = __ldg(a.fresh + b);
    if (kv < 0 || (long long)kv + max(n, 0) > cap) {
      bad = true;
      continue;
    }
    const int held = pages(kv);
    if (n < 0) {
      s[2] += held;
    } else {
      s[0] += n;
      s[1] += pages(kv + n) - held;
    }
  }
  long long run[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    long long x = s[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += u;
    }
    if (lane == 31) part[i][w] = x;
    run[i] = x - s[i];
  }
  bad = __syncthreads_or(bad);
  long long all[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < w) run[i] += part[i][k];
      all[i] += part[i][k];
    }
  const int count = __ldg(a.count);
  const long long total = count + all[2], left = total - all[1];   // the stack with what comes back; without what goes
  int err = 0;
  if (bad || all[0] > a.tokens)
    err = kErrSeqLens;
  else if (count < 0 || total > a.num_pages || left < 0)
    err = kErrPool;

  const int first = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  if (err) {   // nothing changes
    if (first == 0) {
      if (a.error) *a.error = err;
      *a.count_out = count;
    }
    for (int b = first; b < a.B; b += step) a.q_out[b] = 0, a.kv_out[b] = __ldg(a.kv + b);
    for (int t = first; t < a.tokens; t += step) a.slots[t] = -1, a.pos[t] = -1;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    const int kv = __ldg(a.kv + b), n = __ldg(a.fresh + b), held = pages(kv);
    if (n < 0) {
      run[2] += held;
    } else {
      run[0] += n;
      run[1] += pages(kv + n) - held;
    }
    toks[b] = (int)run[0];
    grown[b] = (int)run[1];
    back[b] = (int)run[2];
    if (blockIdx.x == 0) a.q_out[b] = max(n, 0), a.kv_out[b] = n < 0 ? 0 : kv + n;
  }
  __syncthreads();
  const int ntok = (int)all[0], ngrown = (int)all[1], top = (int)total, rest = (int)left;
  if (first == 0) *a.count_out = rest;

  // entry k of the stack with what comes back
  auto stack = [&](int k) {
    if (k < count) return a.free[k];
    const int r = k - count, b = find(back, a.B, r);
    return a.table[(size_t)b * a.max_pages + (r - (b ? back[b - 1] : 0))];
  };
  for (int t = first; t < a.tokens; t += step) {
    int slot = -1, pos = -1;
    if (t < ntok) {
      const int b = find(toks, a.B, t), kv = __ldg(a.kv + b);
      pos = kv + t - (b ? toks[b - 1] : 0);
      const int j = pos / ps, held = pages(kv);
      const int id = j < held ? a.table[(size_t)b * a.max_pages + j]
                              : stack(top - 1 - ((b ? grown[b - 1] : 0) + j - held));
      if (id >= 0 && id < a.num_pages)
        slot = id * ps + (pos - j * ps);
      else if (a.error)
        *a.error = kErrPage;
    }
    a.slots[t] = slot;
    a.pos[t] = pos;
  }
  for (int i = first; i < ngrown; i += step) {
    const int b = find(grown, a.B, i);
    a.table[(size_t)b * a.max_pages + pages(__ldg(a.kv + b)) + (i - (b ? grown[b - 1] : 0))] = stack(top - 1 - i);
  }
  for (int k = count + first; k < rest; k += step) a.free[k] = stack(k);
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, int nsm, cudaStream_t st) {
  const int bytes = 3 * a.B * (int)sizeof(int);
  if (bytes > 40 * 1024) {   // beyond what a launch has without asking
    const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               3 * kPlanRequests * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  // A thread an item, of tokens and of pages that may move: what comes back or
  // is handed out only the device knows.  (Blocks for the tokens alone: 512 of
  // 1024 requests of up to 16384 tokens end, 512 have a token, 496 us instead of
  // 10; where few pages move the blocks that find nothing cost nothing, 64
  // requests 4.2 us with one or 152.)
  const long long held = (long long)a.B * a.max_pages, pages = held < a.num_pages ? held : a.num_pages;
  const long long items = pages > a.tokens ? pages : a.tokens, want = (items + kThreads - 1) / kThreads;
  plan_kernel<<<(unsigned)(want < nsm ? want : nsm), kThreads, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sfa
