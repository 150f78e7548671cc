// The merge of the paged attention's pieces (paged.cu, paged_few.cu).
#include "paged_work.cuh"

namespace sfa {
namespace {

static_assert(2 * kMaxSms <= 512, "a thread a piece");
// Pieces of row tiles, added in order.  The worker whose last piece begins a row
// tile owns it.  A tile of few pieces takes a warp a row, one of many (few
// rows over a long cache) a block a row, its warps a share of the pieces each.
// Block 0 also sums up the error words.
constexpr int kMergeThreads = 512;
constexpr int kManyPieces = 16;

template <typename T, int kRows>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const Args args) {
  constexpr int kW = kMergeThreads / 32;
  __shared__ int few_before[kMaxSms + 1], many_before[kMaxSms + 1], pieces[kMaxSms], slot0[kMaxSms];
  __shared__ Piece pc[2 * kMaxSms];
  __shared__ float part_sum[kW];
  __shared__ float4 part[kW][128];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, np = args.workers;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int e = tid < args.ctas ? args.status[tid] : 0;
  if (tid < 2 * np) pc[tid] = args.piece[tid];
  if (blockIdx.x == 0) {
    const int t1 = __syncthreads_or(e == kErrTimeout), t2 = __syncthreads_or(e == kErrSeqLens),
              t3 = __syncthreads_or(e == kErrPage);
    if (tid == 0) *reinterpret_cast<int*>(args.a.ws) = t1 ? kErrTimeout : t2 ? kErrSeqLens : t3 ? kErrPage : 0;
  }
  __syncthreads();
  if (tid < np) {
    const int s = pc[2 * tid + 1].valid ? 2 * tid + 1 : 2 * tid;
    int n = 0;
    if (pc[s].valid && pc[s].first) {
      // this piece, then every following worker's first, up to the tile's end
      // (a call that gave up a wait leaves the chain without its end)
      n = 1;
      for (int q = s; !pc[q].last && tid + n < np && pc[2 * (tid + n)].valid; ++n) q = 2 * (tid + n);
    }
    slot0[tid] = s;
    pieces[tid] = n;
  }
  __syncthreads();
  if (warp < 2) {   // prefix sums of the rows of tiles of few and of many pieces
    int* before = warp ? many_before : few_before;
    int sum = 0;
    for (int i0 = 0; i0 < np; i0 += 32) {
      const int i = i0 + lane;
      int v = i < np && pieces[i] > 0 && (pieces[i] > kManyPieces) == (warp == 1) ? pc[slot0[i]].nrows : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
      }
      if (i < np) before[i + 1] = sum + v;
      sum += __shfl_sync(~0u, v, 31);
    }
    if (lane == 0) before[0] = 0;
  }
  __syncthreads();
  const Scale sc = score_scale(args.a.scale);
  auto owner = [&](const int* before, int task) {   // before[lo] <= task < before[lo + 1]
    int lo = 0, hi = np;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= task) lo = mid; else hi = mid;
    }
    return lo;
  };
  // One warp's share of a row: pieces first, first + step, ... of n, relative
  // to the max m of all of them.  Lane l holds columns 4 l + 128 i.
  auto gather = [&](int worker, int r, int n, int first, int step, float m, float4* o) {
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = first; i < n; i += step) {
      const int s = i == 0 ? slot0[worker] : 2 * (worker + i);
      const float4 st = args.stats[s * kRows + r];
      const float4* p = reinterpret_cast<const float4*>(args.part + ((size_t)s * kRows + r) * 512) + lane;
      const float4 v[4] = {p[0], p[32], p[64], p[96]};
      if (st.x == -INFINITY && st.z == 0.f) continue;
      const float f = ex2((st.y - m) * sc.log2);
      l += st.z * f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k].x += v[k].x * f; o[k].y += v[k].y * f; o[k].z += v[k].z * f; o[k].w += v[k].w * f;
      }
    }
    return l;
  };
  auto top = [&](int worker, int r, int n) {
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, args.stats[(i == 0 ? slot0[worker] : 2 * (worker + i)) * kRows + r].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    return m;
  };
  auto finish = [&](int worker, int r, float m, float l, const float4* o) {
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    const size_t row = (size_t)pc[slot0[worker]].row0 + r;
    uint2* dst = reinterpret_cast<uint2*>((T*)args.a.out + row * 512) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      dst[32 * k] = make_uint2(Elt<T>::pack(o[k].x * inv, o[k].y * inv), Elt<T>::pack(o[k].z * inv, o[k].w * inv));
    if (lane == 0) {
      args.a.smax[row] = m == -INFINITY ? m : m * sc.scale;
      args.a.ssum[row] = l;
    }
  };
  for (int task = blockIdx.x; task < many_before[np]; task += gridDim.x) {
    const int worker = owner(many_before, task), r = task - many_before[worker], n = pieces[worker];
    const float m = top(worker, r, n);
    float4 o[4];
    const float share = gather(worker, r, n, warp, kW, m, o);
    __syncthreads();   // the row before has been read
#pragma unroll
    for (int k = 0; k < 4; ++k) part[warp][lane + 32 * k] = o[k];
    if (lane == 0) part_sum[warp] = share;
    __syncthreads();
    if (tid < 256) {   // two columns a thread, the warps in ascending order
      float l = 0.f;
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float2 v = reinterpret_cast<const float2*>(part[w])[tid];
        l += part_sum[w];
        a.x += v.x; a.y += v.y;
      }
      const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
      const size_t row = (size_t)pc[slot0[worker]].row0 + r;
      reinterpret_cast<uint32_t*>((T*)args.a.out + row * 512)[tid] = Elt<T>::pack(a.x * inv, a.y * inv);
      if (tid == 0) {
        args.a.smax[row] = m == -INFINITY ? m : m * sc.scale;
        args.a.ssum[row] = l;
      }
    }
  }
  for (int task = warp * gridDim.x + blockIdx.x; task < few_before[np]; task += kW * gridDim.x) {
    const int worker = owner(few_before, task), r = task - few_before[worker], n = pieces[worker];
    const float m = top(worker, r, n);
    float4 o[4];
    const float l = gather(worker, r, n, 0, 1, m, o);
    finish(worker, r, m, l, o);
  }
}

}  // namespace

template <typename T>
cudaError_t launch_paged_merge(const Args& g, int rows, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * device_sm_count());
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return rows == 32   ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 32>, g)
         : rows == 64 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 64>, g)
                      : cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 128>, g);
}

template cudaError_t launch_paged_merge<__nv_bfloat16>(const Args&, int, cudaStream_t);
template cudaError_t launch_paged_merge<__half>(const Args&, int, cudaStream_t);

}  // namespace sfa
