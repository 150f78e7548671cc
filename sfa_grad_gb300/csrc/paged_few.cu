// Attention over the paged cache for few query rows a sequence: row tiles of
// R = 32 or 64 (token, head) rows, one CTA each (paged.cu takes tiles of 128
// with pairs of CTAs and decides which calls come here).
//
// With few rows the cache's bytes decide, so a tile of 64 keys is loaded once:
// its panels (64 keys x 64 features, 128-byte swizzle) are the K-major operand
// of S^T = K Q^T and, two at a time, the MN-major one of O^T = V^T P^T.  Keys
// and features lie on M and the rows on N, so both products cost what the rows
// that are there cost: 36 MMAs and 16, of 25 and 41 clk each at 32 rows, of 33
// and 49 at 64.
//
// A warp reads the scores of 16 keys as matrix fragments, so that all lanes
// have work (M = 64 leaves half the lanes of tensor memory empty).  A thread
// keeps its own maximum and sum of every row it meets and P stays relative to
// a row's stale reference: the rows' maxima are brought together only when a
// score exceeds its reference by 2^8, and at the end.
//
// The ring holds ten slots of two panels (eight at 64 rows), four a tile, so
// up to 2.5 tiles are on their way or worked on.  Each product has a warp of
// its own: one warp that looked at both products' barriers in turn spent 650
// clk a slot where its eight MMAs take 200, and the loads waited for it.
//
// Measured: 128 sequences x 16 heads of 2048 .. 16384 keys 233 us, 6.1 TB/s of
// the cache's bytes (302 with the rows on M); 128 x 64 heads of 2048 .. 8192
// keys 158 us, 4.8 TB/s: with eight slots the loads wait
// for the products, a tile takes 3900 clk.
//
// Rows of 4 bits (R = 32): groups of 16 rows come as they are, by bulk copies, and
// eight warps unpack them into the ring's panels, which both products read as
// above.  What bounds this is shared memory: a tile of 64 keys is written twice
// and read three times, 2440 clk at 128 bytes a clk, and takes 3100.  128 sequences x
// 16 heads of 2048 .. 16384 keys 225 us (16 bits: 230, bound by HBM), one of 1000
// keys 17.3 us.  (Bytes read by the unpacking warps themselves, by global
// loads of rows 416 bytes apart: 254 us.  Eight slots and four groups, which
// fill shared memory, 234 where seven and eight took 250.  Sixteen unpacking
// warps, or tiles of 16 rows with a slot more: 2 %.)
//
// Work is split and merged as in paged.cu.
//
// Warps: 0..7 softmax, rescaling, epilogue, 8 the scores' MMAs, 15 the values',
// 9 the walk with the page table and the query rows, 10..13 the loads of a
// tile's slots, one each, 14 those of its rope panel.  Rows of 4 bits: 10 the
// copies of groups, 11..14 and 16..19 the unpacking.
#include "cache4.cuh"
#include "paged_work.cuh"

namespace sfa {
namespace {

constexpr int kKeys = 64;
constexpr int kSoft = 8;                    // softmax warps, the first ones
constexpr int kDecode = 8;                  // warps that unpack rows of 4 bits
constexpr int kSegs = 4;                    // work descriptors in flight
constexpr int kTiles = 8;                   // tiles whose cache rows are known in advance
constexpr int kMaxSlots = 10;
constexpr int kGroup = 16;                  // rows of 4 bits that arrive together: never of two pages
// Groups on their way: a multiple of a tile's four, so that a place belongs to
// the warps of one group, which meet every phase of it.
constexpr int kRaw = 4;
constexpr uint32_t kPanel = 8192;           // 64 rows of 128 bytes
constexpr uint32_t kSlot = 2 * kPanel;
constexpr uint32_t kColS = 256;             // tensor memory: O^T, 64 columns a block of 128 features, then two S^T

// What follows from the rows of a row tile, and from the cache's.
template <int R, bool Q4, bool ROPE>
struct Few {
  static constexpr int kThreads = 32 * (kSoft + 8 + (Q4 ? kDecode - 4 : 0));
  static constexpr int kWide = R / 2;                  // rows of a softmax warp
  // Rows of 4 bits: a sum of its own for each slot of a tile, added up in fp32.
  // The tensor core rounds every step of a sum towards zero, by the sum so far.
  static constexpr int kSums = Q4 ? 4 : 1;
  static constexpr int kSlots = R == 32 && !Q4 ? 10 : 8;
  static constexpr uint32_t kRowBytes = kRopeAt + (ROPE ? 128 : 0);
  static constexpr uint32_t kQPanel = R * 128;
  static constexpr uint32_t kOffP = 9 * kQPanel;       // P^T: 64 keys x 64 rows
  static constexpr uint32_t kOffRope = kOffP + kPanel;
  static constexpr uint32_t kOffRing = kOffRope + 2 * kPanel;
  static constexpr uint32_t kOffRaw = kOffRing + kSlots * kSlot;
  static constexpr uint32_t kOffCtl = kOffRaw + (Q4 ? kRaw * kGroup * kRowBytes : 0);
  using W = Work<R, kKeys, kThreads, 2>;
};

struct Ctl {
  uint64_t full[kMaxSlots], empty[kMaxSlots], rfull[2], rempty[2];
  uint64_t qfull, qempty, sfull[2], sfree[2], pready, pfree, ofree;
  uint64_t xch, fch, settle[2];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t tile_full[kTiles], tile_empty[kTiles];
  uint64_t flags[2];                        // a byte a softmax warp: some row's max rises
  Share share;
  uint32_t tmem;
  int abort;
  Seg seg[kSegs];
  int y[kTiles][4];                         // cache row of each box of a tile
  int loads[kMaxSlots], rloads[2];          // uses of a slot (4 bits: of a group's place) that have been issued
  int none[kRaw];                        // a group without a page: zeros
  alignas(16) float rbuf[64];               // a row's reference, times log2
  float fbuf[64];                           // ... and its factor for O
};
template <int R, bool Q4, bool ROPE>
constexpr uint32_t kSmem = Few<R, Q4, ROPE>::kOffCtl + sizeof(Ctl) + 1024;
static_assert(kSmem<32, false, true> <= 227 * 1024 && kSmem<64, false, true> <= 227 * 1024, "shared memory");
static_assert(kSmem<32, true, true> <= 227 * 1024, "shared memory");
static_assert(kSmem<32, false, false> > kOneCtaSmem && kSmem<64, false, false> > kOneCtaSmem &&
                  kSmem<32, true, false> > kOneCtaSmem,
              "one CTA an SM: it allocates all of tensor memory");

// The four steps of a contraction over 64 elements, by the elected lane of a
// converged warp; SA, SB: a step in encoded descriptor units.
template <uint32_t SA, uint32_t SB>
__device__ __forceinline__ void mma_k64(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %11, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %6, %3, 1;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %8, %3, 1;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %9, %10, %3, 1;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "l"(a + SA), "l"(b + SB), "l"(a + 2 * SA), "l"(b + 2 * SB),
      "l"(a + 3 * SA), "l"(b + 3 * SB), "r"(el)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// 16 lanes x 8 N columns of tensor memory as matrix fragments: v[4 j + 2 h + e]
// is lane (thread / 4) + 8 h, column 8 j + 2 (thread % 4) + e.
template <int N>
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float* v) {
  static_assert(N == 2 || N == 4, "");
  uint32_t r[4 * N];
  if constexpr (N == 2)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) v[i] = __uint_as_float(r[i]);
}

// The same at `Sums` places, `step` columns apart: the first in v, the others in w.
template <int N, int Sums, int Step>
__device__ __forceinline__ void tmem_ld_frags(uint32_t taddr, float* v, float (*w)[4 * N]) {
  static_assert(N == 2, "");
  uint32_t r[Sums][8];
#pragma unroll
  for (int k = 0; k < Sums; ++k)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[k][0]), "=r"(r[k][1]), "=r"(r[k][2]), "=r"(r[k][3]), "=r"(r[k][4]), "=r"(r[k][5]),
                   "=r"(r[k][6]), "=r"(r[k][7])
                 : "r"(taddr + k * Step));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < Sums; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) (k ? w[k - 1] : v)[i] = __uint_as_float(r[k][i]);
}

struct MapsFew {
  CUtensorMap q, qr;   // boxes of 64 columns x R rows
  CUtensorMap c2, c1;  // the cache, boxes of vbox rows of two panels (vbox = 64 only) and of one
};

// Bytes of packed rows into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <typename T, bool ROPE, int R, bool Q4>
__global__ void __launch_bounds__((Few<R, Q4, ROPE>::kThreads), 1)
    paged_few_kernel(const __grid_constant__ MapsFew maps, const Args args) {
  using F = Few<R, Q4, ROPE>;
  using W = typename F::W;
  constexpr int kSlots = F::kSlots;
  constexpr uint32_t kQPanel = F::kQPanel, kOffP = F::kOffP, kOffRope = F::kOffRope, kOffRing = F::kOffRing;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Ctl* c = reinterpret_cast<Ctl*>(sm + F::kOffCtl);
  const Paged& p = args.a.pg;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  constexpr int kPanels = ROPE ? 9 : 8;
  int* status = args.status + cta;

  // programmatic launch: the merge may be set up from now on (it waits for
  // this grid's end before it reads anything)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    *status = 0;
    args.piece[2 * cta].valid = 0;
    args.piece[2 * cta + 1].valid = 0;
    c->abort = 0;
    c->flags[0] = c->flags[1] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->rfull[i], Q4 ? kDecode : 1);
      mbar_init(&c->rempty[i], 1);
      c->rloads[i] = 0;
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->sfree[i], kSoft);
    }
    mbar_init(&c->qfull, 1);
    mbar_init(&c->qempty, 1);
    mbar_init(&c->pready, kSoft);
    mbar_init(&c->pfree, 1);
    mbar_init(&c->ofree, kSoft);
    mbar_init(&c->xch, kSoft);
    mbar_init(&c->fch, kSoft);
    mbar_init(&c->settle[0], 1);
    mbar_init(&c->settle[1], 1);
    mbar_fence_init();
  } else if (warp == 1) {
    if (lane < kSegs) mbar_init(&c->seg_full[lane], 1), mbar_init(&c->seg_empty[lane], kSoft + 2);
    c->rbuf[lane] = c->rbuf[lane + 32] = -INFINITY;
    if (lane < kTiles) mbar_init(&c->tile_full[lane], 1), mbar_init(&c->tile_empty[lane], Q4 ? 1 : 4 + ROPE);
    if (lane < kSlots) {
      mbar_init(&c->full[lane], Q4 ? kDecode : 1);
      mbar_init(&c->empty[lane], 1);
    }
    if (lane < kMaxSlots) c->loads[lane] = 0;
    if (Q4 && lane < kRaw) mbar_init(&c->raw_full[lane], 1), mbar_init(&c->raw_empty[lane], kDecode / 4);
    mbar_fence_init();
  } else if (warp == 2 && lane < (Q4 ? 2 : 4)) {
    const CUtensorMap* m = lane == 0 ? &maps.q : lane == 1 ? &maps.qr : lane == 2 ? &maps.c2 : &maps.c1;
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  if (warp == kSoft + 1) tmem_alloc(&c->tmem, 512);
  // (the scan's sums lie in the ring, which nothing has been loaded into yet)
  W::plan(p, &c->share, reinterpret_cast<long long*>(sm + kOffRing), cta, args.workers);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  const Limit w = wait_limit(&c->abort, status, args.a);
  const int ntiles = c->share.ntiles;
  const bool work = ntiles > 0;
  const uint32_t ring = smem_u32(sm + kOffRing), rope = smem_u32(sm + kOffRope);

  if (c->share.bad && tid == 0) *status = kErrSeqLens;

  if (work && warp == kSoft + 1) {
    // ---------------------------------------------------------------- the walk
    const int none = p.num_pages * p.page_size;     // a row outside the map: zeros
    const int boxes = kKeys / args.vbox;
    int b = c->share.seq, left = ntiles, tile = 0, issued = 0;
    SeqWork s = W::seq_work(p, b);
    int j = c->share.tile, kt = c->share.kt, row = c->share.row;   // row: the sequence's first
    bool ok = true;
    for (int n = 0; ok; ++n) {
      Seg g;
      g.kt1 = 0;
      if (left > 0) {
        while (j >= s.tiles) {
          row += (p.tnd ? s.qlen : p.S1) * p.G;
          s = W::seq_work(p, ++b);
          j = 0;
        }
        const int units = W::tile_units(p, s, j);
        g.row0 = row + j * R;
        g.i0 = j * R;
        g.nrows = min(R, s.rows - g.i0);
        g.kt0 = kt;
        g.kt1 = min(units, kt + left);
        g.kend = W::tile_keys(p, s, j);
        g.base = p.mode == 3 ? s.kvlen - s.qlen : s.kvlen - 1;
        g.slot = g.kt0 == 0 && g.kt1 == units ? -1 : n == 0 ? 2 * cta : 2 * cta + 1;
        left -= g.kt1 - g.kt0;
        if (g.slot >= 0 && lane == 0)
          args.piece[g.slot] = Piece{1, g.row0, g.nrows, g.kt0 == 0, g.kt1 == units, {0, 0, 0}};
        kt = 0;
        ++j;
      }
      const int r = n % kSegs;
      if (n >= kSegs && !(ok = warp_wait(&c->seg_empty[r], (n / kSegs - 1) & 1, w))) break;
      if (lane == 0) {
        c->seg[r] = g;
        mbar_arrive(&c->seg_full[r]);
      }
      if (g.kt1 == 0) break;
      const int* table = p.table + (size_t)b * p.max_pages;
      // (an entry may hold any value, so none marks a box that is not needed)
      auto needed = [&](int t) { return lane < boxes && t * kKeys + lane * args.vbox < g.kend; };
      auto fetch = [&](int t) { return needed(t) ? __ldg(table + (t * kKeys + lane * args.vbox) / p.page_size) : -1; };
      int page = fetch(g.kt0);
      for (int t = g.kt0; t < g.kt1; ++t, ++tile) {
        int y = none;
        if (page >= 0 && page < p.num_pages)
          y = page * p.page_size + (t * kKeys + lane * args.vbox) % p.page_size;
        else if (needed(t))
          atomicCAS(status, 0, kErrPage);   // a timeout stays
        if (t + 1 < g.kt1) page = fetch(t + 1);   // in flight during the waits
        const int i = tile % kTiles;
        if (tile >= kTiles && !(ok = warp_wait(&c->tile_empty[i], (tile / kTiles - 1) & 1, w))) break;
        if (lane < boxes) c->y[i][lane] = y;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->tile_full[i]);
        if (t == g.kt0) {
          // the query rows, once the piece before has done its products
          if (n > 0 && !(ok = warp_wait(&c->qempty, (n - 1) & 1, w))) break;
          if (lane == 0) mbar_expect_tx(&c->qfull, kPanels * kQPanel);
          __syncwarp();
          if (lane < kPanels)
            tma_2d(smem_u32(sm) + lane * kQPanel, lane < 8 ? &maps.q : &maps.qr, (lane & 7) * 64, g.row0, &c->qfull);
          issued = n + 1;
        }
      }
    }
    // rows on their way, where another warp gave up
    if (issued > 0) mbar_settle(&c->qfull, (issued - 1) & 1, status);
  } else if (Q4 && work && warp == kSoft + 2) {
    // ---------------------------------------------------------------- packed rows, a group a place
    const int none = p.num_pages * p.page_size;
    for (int t = 0; t < ntiles; ++t) {
      const int i = t % kTiles;
      if (!warp_wait(&c->tile_full[i], (t / kTiles) & 1, w)) break;
      const int y = c->y[i][lane & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->tile_empty[i]);
      bool ok = true;
      for (int g = 0; g < 4 && ok; ++g) {
        const int u = 4 * t + g, s = u % kRaw, use = u / kRaw;
        if (use > 0 && !(ok = warp_wait(&c->raw_empty[s], (use - 1) & 1, w))) break;
        if (lane == g) {
          c->none[s] = y == none;
          c->loads[s] = use + 1;
          if (y == none) {
            mbar_arrive(&c->raw_full[s]);
          } else {
            mbar_expect_tx(&c->raw_full[s], kGroup * F::kRowBytes);
            bulk_load(smem_u32(sm) + F::kOffRaw + s * kGroup * F::kRowBytes,
                      (const uint8_t*)args.a.cache + (size_t)y * F::kRowBytes, kGroup * F::kRowBytes, &c->raw_full[s]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
    }
  } else if (Q4 && work && ((warp > kSoft + 2 && warp < kSoft + 7) || warp > kSoft + 7)) {
    // ---------------------------------------------------------------- rows of 4 bits to panels
    // Warp: a group's keys, one of a slot's two panels.  Lane: a key and half
    // a panel's row, 32 features; eight neighbouring lanes have four keys and
    // both halves, which keeps the reads (416 bytes apart) and the swizzled
    // writes free of bank conflicts.
    const int d = warp < kSoft + 7 ? warp - (kSoft + 3) : warp - (kSoft + 4);
    const int g = d & 3, half = d >> 2;
    const int key = (lane & 3) + 4 * (lane >> 3), part = (lane >> 2) & 1;
    const uint32_t row = (g * kGroup + key) * 128, swz = key & 7;
    const Dec4<T> dec(args.a.scale_exp);
    int s = 0, ph = 1;   // ring slot, and the phase of its release (the first use waits for none)
    bool ok = true;
    for (int t = 0; t < ntiles && ok; ++t) {
      const int u = 4 * t + g, rs = u % kRaw;
      if (!(ok = warp_wait(&c->raw_full[rs], (u / kRaw) & 1, w))) break;
      const uint32_t src = smem_u32(sm) + F::kOffRaw + (rs * kGroup + key) * F::kRowBytes;
      uint4 code[4], rope4[2];
      uint32_t two[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int panel = 2 * i + half;
        code[i] = lds128(src + panel * 32 + part * 16);
        two[i] = lds_u16(src + kCodes + panel * 4 + part * 2);
      }
      if (ROPE) {
#pragma unroll
        for (int i = 0; i < 2; ++i) rope4[i] = lds128(src + kRopeAt + (4 * half + 2 * i + part) * 16);
      }
      if (c->none[rs]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) code[i] = make_uint4(0, 0, 0, 0), two[i] = 0;
        rope4[0] = rope4[1] = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->raw_empty[rs]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t sc[2];
        dec.scales(two[i], sc);
        const uint4 v[4] = {dec.eight(code[i].x, sc[0]), dec.eight(code[i].y, sc[0]), dec.eight(code[i].z, sc[1]),
                            dec.eight(code[i].w, sc[1])};
        if (!(ok = warp_wait(&c->empty[s], ph, w))) break;
        const uint32_t dst = ring + s * kSlot + half * kPanel + row;
#pragma unroll
        for (int k = 0; k < 4; ++k) sts128(dst + (((4 * part + k) ^ swz) << 4), v[k]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->full[s]);
        if (++s == kSlots) s = 0, ph ^= 1;
      }
      if (!ok || !ROPE) continue;
      const int b = t & 1;
      if (t >= 2 && !(ok = warp_wait(&c->rempty[b], ((t >> 1) - 1) & 1, w))) break;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sts128(rope + b * kPanel + row + (((4 * half + 2 * i + part) ^ swz) << 4), rope4[i]);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->rfull[b]);
    }
  } else if (!Q4 && work && warp >= kSoft + 2 && warp < kSoft + 6 + ROPE) {
    // ---------------------------------------------------------------- TMA loads
    const int boxes = kKeys / args.vbox;
    const int pl = boxes == 1 ? 0 : lane / boxes, pb = boxes == 1 ? 0 : lane % boxes;   // panel, box of a lane
    const int k = warp - (kSoft + 2);   // slot of the tile, 4: rope
    const bool is_rope = k == 4;
    for (int t = 0; t < ntiles; ++t) {
      const int i = t % kTiles, u = 4 * t + k;
      if (!warp_wait(&c->tile_full[i], (t / kTiles) & 1, w)) break;
      const int y = c->y[i][pb];
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->tile_empty[i]);
      const int s = is_rope ? t & 1 : u % kSlots, use = is_rope ? t >> 1 : u / kSlots;
      uint64_t* full = is_rope ? &c->rfull[s] : &c->full[s];
      if (use > 0 && !warp_wait(is_rope ? &c->rempty[s] : &c->empty[s], (use - 1) & 1, w)) break;
      if (lane == 0) {
        mbar_expect_tx(full, is_rope ? kPanel : kSlot);
        (is_rope ? c->rloads : c->loads)[s] = use + 1;
      }
      __syncwarp();
      const uint32_t dst = is_rope ? rope + s * kPanel : ring + s * kSlot;
      if (boxes == 1 && !is_rope) {
        if (lane == 0) tma_3d(dst, &maps.c2, 0, y, 2 * k, full);
      } else if (boxes == 1 ? lane == 0 : pl < (is_rope ? 1 : 2)) {
        tma_3d(dst + pl * kPanel + pb * args.vbox * 128, &maps.c1, 0, y, 2 * k + pl, full);
      }
    }
  } else if (work && warp == kSoft) {
    // ---------------------------------------------------------------- scores
    const uint32_t el = elect_one();
    constexpr uint32_t ids = idesc_f16(kKeys, R, Elt<T>::is_f16, false, false);
    const uint64_t dq = sdesc_kmajor(smem_u32(sm), 0), dk = sdesc_kmajor(ring, 0), dr = sdesc_kmajor(rope, 0);
    int s = 0, ph = 0, segs = 0, left = 0;   // ring slot and its phase; pieces; tiles of the piece to come
    bool ok = true;
    for (int t = 0; t < ntiles && ok; ++t) {
      if (left == 0) {   // a new piece
        const int r = segs % kSegs;
        if (!(ok = warp_wait(&c->seg_full[r], (segs / kSegs) & 1, w))) break;
        left = c->seg[r].kt1 - c->seg[r].kt0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->seg_empty[r]);
        if (!(ok = warp_wait(&c->qfull, segs & 1, w))) break;
        ++segs;
      }
      const int buf = t & 1;
      if (t >= 2 && !(ok = warp_wait(&c->sfree[buf], (t / 2 - 1) & 1, w))) break;
      tc_fence_after();   // the softmax warps' reads of this S buffer
      const uint32_t d0 = tmem + kColS + buf * (Q4 ? 128 : 64);
#pragma unroll 2
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = d0 + (Q4 ? i * R : 0);
        if (!(ok = warp_wait(&c->full[s], ph, w))) break;
        const uint64_t a = dk + desc_off(s * kSlot), b = dq + desc_off(2 * i * kQPanel);
        mma_k64<2, 2>(el, d, a, b, ids, !Q4 && i > 0);
        mma_k64<2, 2>(el, d, a + desc_off(kPanel), b + desc_off(kQPanel), ids, 1);
        if (++s == kSlots) s = 0, ph ^= 1;
      }
      if (!ok) break;
      if (ROPE) {
        if (!(ok = warp_wait(&c->rfull[buf], (t >> 1) & 1, w))) break;
        mma_k64<2, 2>(el, d0 + (Q4 ? 3 * R : 0), dr + desc_off(buf * kPanel), dq + desc_off(8 * kQPanel), ids, 1);
        commit(el, &c->rempty[buf]);
      }
      commit(el, &c->sfull[buf]);
      if (--left == 0) commit(el, &c->qempty);
    }
    commit(el, &c->settle[0]);
    mbar_settle(&c->settle[0], 0, status);
  } else if (work && warp == kSoft + 7) {
    // ---------------------------------------------------------------- products with the values
    // (a warp of their own: neither product waits for the other's slots)
    const uint32_t el = elect_one();
    const uint64_t dp = sdesc_mnmajor(smem_u32(sm + kOffP), 0, 64), dv = sdesc_mnmajor(ring, 0, 64);
    int s = 0, segs = 0, left = 0;
    uint32_t idv = 0;
    bool ok = true;
    for (int t = 0; t < ntiles && ok; ++t) {
      const bool first = left == 0;
      if (first) {
        const int r = segs % kSegs;
        if (!(ok = warp_wait(&c->seg_full[r], (segs / kSegs) & 1, w))) break;
        left = c->seg[r].kt1 - c->seg[r].kt0;
        idv = idesc_f16(128, (c->seg[r].nrows + 15) / 16 * 16, Elt<T>::is_f16, true, true);
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->seg_empty[r]);
        if (segs++ > 0 && !(ok = warp_wait(&c->ofree, (segs - 2) & 1, w))) break;
      }
      if (!(ok = warp_wait(&c->pready, t & 1, w))) break;
      tc_fence_after();   // ... and reads and rescaling of O
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        mma_k64<128, 128>(el, tmem + i * 64, dv + desc_off(s * kSlot), dp, idv, !first);
        commit(el, &c->empty[s]);
        if (++s == kSlots) s = 0;
      }
      commit(el, &c->pfree);
      --left;
    }
    commit(el, &c->settle[1]);
    mbar_settle(&c->settle[1], 0, status);
  } else if (work && warp < kSoft) {
    // ---------------------------------------------------------------- softmax, epilogue
    // Warps q and q + 4: keys 16 q .. 16 q + 15 of a tile (M = 64 puts 16 keys
    // in each warp's quarter of tensor memory), rows c0 .. c0 + kWide - 1.  A
    // thread has keys key and key + 8 and, of every eight rows, two:
    // row(i) = c0 + 8 (i / 2) + 2 (lane % 4) + i % 2.  Every lane: feature 32 q +
    // lane of two blocks of O^T.  Lane l of a warp with q = 0 brings row c0 + l
    // together.
    constexpr int kWide = F::kWide, kHas = kWide / 4;   // rows of a warp, of a thread
    const int wq = warp & 3, cg = warp >> 2, c0 = cg * kWide, r0 = c0 + 2 * (lane & 3);
    const bool owner = wq == 0 && lane < kWide;
    const int key = wq * 16 + (lane >> 2);
    const uint32_t tq = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t pkey = smem_u32(sm + kOffP) + key * 128 + (lane & 3) * 4;   // P's row of key; key + 8: 1024 on
    float* scratch = reinterpret_cast<float*>(sm + kOffP);   // P's place, when no product reads it
    const Scale sc = score_scale(args.a.scale);
    int tile = 0, nx = 0, nf = 0;
    // all softmax warps: has any of them a flag
    auto exchange = [&](bool flag, bool* any) {
      if (lane == 0) {
        reinterpret_cast<uint8_t*>(&c->flags[nx & 1])[warp] = flag;
        mbar_arrive(&c->xch);
      }
      if (!warp_wait(&c->xch, nx & 1, w)) return false;
      *any = c->flags[nx & 1] != 0;
      ++nx;
      return true;
    };
    auto sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->fch);
      return warp_wait(&c->fch, nf++ & 1, w);
    };
    // a value of each row over a warp's keys, into the scratch: each step
    // halves the rows a lane keeps
    auto gather = [&](const float* v, bool sum, int at) {
      float u[kHas];
#pragma unroll
      for (int i = 0; i < kHas; ++i) u[i] = v[i];
      int i = 0;
#pragma unroll
      for (int o = 16, n = kHas / 2; o >= 4; o >>= 1, n >>= 1) {
        const bool up = lane & o;
        if (n == 0) {   // one row left: both lanes keep it
          const float e = __shfl_xor_sync(~0u, u[0], o);
          u[0] = sum ? u[0] + e : fmaxf(u[0], e);
          continue;
        }
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const float e = __shfl_xor_sync(~0u, up ? u[k] : u[k + n], o), x = up ? u[k + n] : u[k];
          u[k] = sum ? x + e : fmaxf(x, e);
        }
        if (up) i += n;
      }
      if (kHas == 8 || !(lane & 4)) scratch[at * 256 + wq * 64 + r0 + 8 * (i >> 1) + (i & 1)] = u[0];
    };
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int sr = n % kSegs;
      if (!warp_wait(&c->seg_full[sr], (n / kSegs) & 1, w)) break;
      const Seg g = c->seg[sr];
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->seg_empty[sr]);
      if (g.kt1 == 0) break;
      const int least = p.mode == 3 ? g.base + g.i0 / p.G : g.base;   // last key the tile's first row sees
      const int cols = (g.nrows + 15) / 16 * 16;
      // of this thread's keys, by row: the max of their scores, the sum of
      // their weights
      float m[kHas], l[kHas];
#pragma unroll
      for (int i = 0; i < kHas; ++i) m[i] = -INFINITY, l[i] = 0.f;
      float mtop = -INFINITY, mref = -INFINITY;   // an owner's row: its max, its reference
      for (int kt = g.kt0; kt < g.kt1; ++kt, ++tile) {
        const int buf = tile & 1;
        if (!(ok = warp_wait(&c->sfull[buf], (tile >> 1) & 1, w))) break;
        tc_fence_after();
        const bool edge = (kt + 1) * kKeys > least + 1;
        float x[2 * kHas];   // [4 j + 2 h + e]: key + 8 h, row(2 j + e)
        if constexpr (Q4) {
          float y[F::kSums - 1][2 * kHas];
          tmem_ld_frags<kWide / 8, F::kSums, R>(tq + kColS + buf * 128 + c0, x, y);
#pragma unroll
          for (int i = 0; i < 2 * kHas; ++i) x[i] = (x[i] + y[0][i]) + (y[1][i] + y[2][i]);
        } else {
          tmem_ld_frag<kWide / 8>(tq + kColS + buf * 64 + c0, x);
        }
        if (sc.negative) {
#pragma unroll
          for (int i = 0; i < 2 * kHas; ++i) x[i] = -x[i];
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < 2 * kHas; ++i) {
            const int j = kt * kKeys + key + 4 * (i & 2), r = r0 + 8 * (i >> 2) + (i & 1);
            if (j >= g.kend || j > (p.mode == 3 ? g.base + (g.i0 + r) / p.G : g.base)) x[i] = -INFINITY;
          }
        }
        bool rises = false;
#pragma unroll
        for (int j = 0; j < kHas / 2; ++j) {
          const float2 ref = *reinterpret_cast<const float2*>(c->rbuf + r0 + 8 * j);
          const float t0 = fmaxf(x[4 * j], x[4 * j + 2]), t1 = fmaxf(x[4 * j + 1], x[4 * j + 3]);
          m[2 * j] = fmaxf(m[2 * j], t0);
          m[2 * j + 1] = fmaxf(m[2 * j + 1], t1);
          rises |= fmaf(t0, sc.log2, -ref.x) > kRaise || fmaf(t1, sc.log2, -ref.y) > kRaise;
        }
        tc_fence_before();
        rises = __any_sync(~0u, rises);
        if (lane == 0) mbar_arrive(&c->sfree[buf]);
        bool any;
        if (!(ok = exchange(rises, &any))) break;
        // P and O belong to the products of the tile before until they end
        if (any) {
          if (tile > 0 && !(ok = warp_wait(&c->pfree, (tile - 1) & 1, w))) break;
          gather(m, false, 0);
          if (!(ok = sync())) break;
          if (owner) {
            // a stale reference keeps P below 2^8, which both types hold as
            // exactly as values below one; O is rescaled only beyond that
            const float* s = scratch + c0 + lane;
            mtop = fmaxf(fmaxf(s[0], s[64]), fmaxf(s[128], s[192]));
            float f = 1.f;
            if ((mtop - mref) * sc.log2 > kRaise) {
              f = ex2((mref - mtop) * sc.log2);
              mref = mtop;
            }
            c->rbuf[c0 + lane] = mref == -INFINITY ? mref : mref * sc.log2;
            c->fbuf[c0 + lane] = f;
          }
          if (!(ok = sync())) break;
#pragma unroll
          for (int i = 0; i < kHas; ++i) l[i] *= c->fbuf[r0 + 8 * (i >> 1) + (i & 1)];
          if (kt > g.kt0) {
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 2 * cols; q += 16) {
              const int blk = q >= cols, col = q - (blk ? cols : 0);
              const uint32_t at = tq + (2 * cg + blk) * 64 + col;
              float o[16];
              tmem_ld16(at, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= c->fbuf[col + i];
              tmem_st16(at, o);
            }
          }
        }
        uint32_t pk[kHas];   // [2 j + h]
#pragma unroll
        for (int j = 0; j < kHas / 2; ++j) {
          const float2 ref = *reinterpret_cast<const float2*>(c->rbuf + r0 + 8 * j);
          const float a = ref.x == -INFINITY ? 0.f : ref.x, b = ref.y == -INFINITY ? 0.f : ref.y;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float u = ex2(fmaf(x[4 * j + 2 * h], sc.log2, -a)), v = ex2(fmaf(x[4 * j + 2 * h + 1], sc.log2, -b));
            l[2 * j] += u;
            l[2 * j + 1] += v;
            pk[2 * j + h] = Elt<T>::pack(u, v);
          }
        }
        if (!any && tile > 0 && !(ok = warp_wait(&c->pfree, (tile - 1) & 1, w))) break;
        if (edge) {
          // Values of masked keys: rows no query row sees become zeros (they
          // may hold anything), and non-finite values of the others, which
          // would reach rows that do not see them as 0 x inf (a row that sees
          // them has a non-finite score from the same cache row).
          const int u = 4 * tile + (warp >> 1), s = u % kSlots;   // the warp's panel
          if (!(ok = warp_wait(&c->full[s], (u / kSlots) & 1, w))) break;
          const int first = max(0, least + 1 - kt * kKeys), end = g.kend - kt * kKeys;
          const uint32_t base = ring + s * kSlot + (warp & 1) * kPanel + ((lane & 7) << 4);
          for (int q = first + (lane >> 3); q < kKeys; q += 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (q < end) {
              v = lds128(base + q * 128);
              float e[8];
              unpack8<T>(v, e);
#pragma unroll
              for (int z = 0; z < 8; ++z) e[z] = fabsf(e[z]) < INFINITY ? e[z] : 0.f;
              v = pack8<T>(e);
            }
            sts128(base + q * 128, v);
          }
        }
#pragma unroll
        for (int j = 0; j < kHas / 2; ++j) {
          const uint32_t at = pkey + (((c0 / 8 + j) ^ (key & 7)) << 4);
          sts32(at, pk[2 * j]);
          sts32(at + 1024, pk[2 * j + 1]);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->pready);
      }
      if (!ok) break;
      if (!(ok = warp_wait(&c->pfree, (tile - 1) & 1, w))) break;
      gather(m, false, 0);
      gather(l, true, 1);
      if (!(ok = sync())) break;
      const bool whole = g.slot < 0;
      float lsum = 0.f;
      if (owner) {
        const float* s = scratch + c0 + lane;
        mtop = fmaxf(fmaxf(s[0], s[64]), fmaxf(s[128], s[192]));
        lsum = (s[256] + s[320]) + (s[384] + s[448]);
        c->fbuf[c0 + lane] = lsum > 0.f || lsum != lsum ? 1.0f / lsum : 0.f;
        c->rbuf[c0 + lane] = -INFINITY;   // for the next piece
      }
      if (!(ok = sync())) break;
      tc_fence_after();
      // a lane has one feature of every row: a store covers 32 of a row
      const int feat = cg * 256 + wq * 32 + lane;
#pragma unroll 1
      for (int q = 0; q < 2 * cols; q += 16) {
        const int blk = q >= cols, col = q - (blk ? cols : 0);
        float o[16];
        tmem_ld16(tq + (2 * cg + blk) * 64 + col, o);
        if (whole) {
          T* dst = (T*)args.a.out + ((size_t)g.row0 + col) * 512 + feat + blk * 128;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (col + i < g.nrows) dst[i * 512] = Elt<T>::from_f(o[i] * c->fbuf[col + i]);
        } else {
          float* dst = args.part + ((size_t)g.slot * R + col) * 512 + feat + blk * 128;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (col + i < g.nrows) dst[i * 512] = o[i];
        }
      }
      if (owner && c0 + lane < g.nrows) {
        if (whole) {
          const size_t row = (size_t)g.row0 + c0 + lane;
          args.a.smax[row] = mtop == -INFINITY ? mtop : mtop * sc.scale;
          args.a.ssum[row] = lsum > 0.f ? lsum * ex2((mref - mtop) * sc.log2) : lsum;
        } else {
          args.stats[g.slot * R + c0 + lane] = make_float4(mtop, mref, lsum, 0.f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->ofree);
    }
  }

  // ---------------------------------------------------------------- end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (Q4) {
    if (c->abort && tid < kRaw && c->loads[tid] > 0) mbar_settle(&c->raw_full[tid], (c->loads[tid] - 1) & 1, status);
  } else if (c->abort && tid < kSlots + 2) {   // copies on their way, where some warp gave up
    const int s = tid < kSlots ? tid : tid - kSlots, n = tid < kSlots ? c->loads[s] : c->rloads[s];
    if (n > 0) mbar_settle(tid < kSlots ? &c->full[s] : &c->rfull[s], (n - 1) & 1, status);
  }
  if (warp == kSoft + 1) tmem_dealloc(tmem, 512);
}

}  // namespace

template <typename T, int R, bool Q4, bool ROPE>
static cudaError_t launch_few(const Args& g, cudaStream_t st) {
  const Paged& p = g.a.pg;
  MapsFew m{};
  const bool f16 = Elt<T>::is_f16;
  const uint64_t rows = (uint64_t)p.T * p.G, cached = (uint64_t)p.num_pages * p.page_size;
  if (!encode_map2d(&m.q, f16, g.a.q, 512, rows, R) ||
      !encode_map2d(&m.qr, f16, ROPE ? g.a.qr : g.a.q, ROPE ? 64 : 512, rows, R) ||
      (!Q4 && (!encode_map_panels(&m.c2, f16, g.a.cache, p.row, cached, g.vbox, g.vbox == 64 ? 2 : 1) ||
               !encode_map_panels(&m.c1, f16, g.a.cache, p.row, cached, g.vbox, 1))))
    return cudaErrorInvalidValue;
  auto kern = paged_few_kernel<T, ROPE, R, Q4>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<R, Q4, ROPE>);
  if (e != cudaSuccess) return e;
  kern<<<g.ctas, Few<R, Q4, ROPE>::kThreads, kSmem<R, Q4, ROPE>, st>>>(m, g);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_paged_merge<T>(g, R, st);
}

template <typename T>
cudaError_t launch_paged_few(const Args& g, int rows, cudaStream_t st) {
  const bool rope = g.a.pg.row == 576;
  if (g.a.packed) return rope ? launch_few<T, 32, true, true>(g, st) : launch_few<T, 32, true, false>(g, st);
  if (rows == 32) return rope ? launch_few<T, 32, false, true>(g, st) : launch_few<T, 32, false, false>(g, st);
  return rope ? launch_few<T, 64, false, true>(g, st) : launch_few<T, 64, false, false>(g, st);
}

template cudaError_t launch_paged_few<__nv_bfloat16>(const Args&, int, cudaStream_t);
template cudaError_t launch_paged_few<__half>(const Args&, int, cudaStream_t);

}  // namespace sfa
