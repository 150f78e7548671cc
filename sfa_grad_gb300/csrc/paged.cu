// Attention of new tokens over the paged latent cache (sfa_paged_fwd).
//
//   x_j = scale [q || q_rope] . row_j,  out = sum_j exp(x_j - m) row_j[:512] / l
//
// Query rows (token, head) are packed 128 to a row tile, keys pass in tiles of
// 256 with a running max m and sum l.  A row tile belongs to a pair of CTAs
// (one cluster), each with 64 of its rows: O needs 512 fp32 columns a row, so
// 128 rows would fill the tensor memory of an SM and leave nothing for S,
// while M = 64 on one SM runs at half rate.  With cta_group::2 and M = 128
// both SMs run at full rate (64 clk an MMA of N = 256), O takes 256 columns of
// 128 lanes (lanes 64..127 hold columns N/2.. of the same 64 rows), and each
// SM stages only half of every B operand: the keys of its half of the tile for
// S = Q K^T, its half of the features for O += P V.
//
// Work: every row tile counts its key tiles, and one more for its beginning and
// end; the pairs split the total evenly and in order, so a pair takes some
// whole row tiles and at most one piece of a tile at each end.  (Without the
// one more, a chunk of 532 tokens x 128 heads over 768 keys took 159 us, with
// it 109: the first pairs got twice the row tiles of the last.)  Pieces leave
// (m, l, O) in fp32 and a second kernel merges them in order: few rows over a
// long cache spread over all SMs, and the result does not depend on timing.
//
// P is rounded to the call's type, for the MMAs take both operands in one, the
// values' (its sum l is of the fp32 weights).  The roundings are independent from key
// to key, so the output's error in the mean square grows little by them: 0.0018
// to 0.0019 of its size in bf16, where its own rounding gives 0.0017, in fp16
// 0.00023 and 0.00021.
//
// Measured, bf16, pages of 64: 512 tokens x 128 heads over 16384 keys 1380 us
// (1667 TFLOP/s; back to back the power limit makes it 1500 to 1525; the tensor
// pipe is busy 74 % of the cycles, the rest is switches between the two
// products and late slots); 64 sequences
// x 128 heads, one token each, 262,000 keys, 98 us: there bound by the bytes
// into shared memory, which keys and values pass separately.
//
// Rows of 4 bits, up to 512 of q a sequence: codes and scales come by TMA in units
// of 128 keys x 256 features, warps unpack them into the ring's slots, and the
// products are as above.  Keys and values are unpacked separately, each CTA its
// own half: the half of the keys that S needs and the half of the features that
// O needs share only a quarter of a tile, and it would have to stay in shared
// memory until P is ready.  Bound by shared memory, which a slot crosses with
// 49 to 53 KB (384 to 415 clk at 128 bytes a clk, where its MMAs take 256), and in bf16
// by the unpacking beside it: 630 clk a slot, fp16 480.  64 sequences x 128 heads of
// 1024 .. 8192 keys, bf16, 100 us (16 bits: 98, bound by the bytes into shared
// memory); one of 131071 keys 61 us.  On the way there, 64 x 128 heads: bytes read by
// global loads 187; staged by TMA 116; rotated parts a tile ahead in a place of their
// own and conversions that take a register's bytes 103.  (Fetching a unit before
// the one in hand is unpacked: no gain.)
//
// Warps of a CTA: 0..3, 5, 7 and 16 the TMA loads of one ring slot each, 4 the
// MMAs (only in the pair's first CTA), 6 the walk over the work with the page
// table and the query rows, 8..15 softmax and epilogue.  Rows of 4 bits: 5 the
// loads of units, 7 those of rotated parts, 0..3 and 16..27 the unpacking.
#include "cache4.cuh"
#include "paged_work.cuh"

namespace sfa {
namespace {

template <bool Q4>
constexpr int kThreads = Q4 ? 896 : 544;
constexpr int kTiles = 4;                   // tiles whose cache rows are known in advance
constexpr int kSoft = 8;                    // softmax warps, from warp 8
constexpr int kRows = 128;                  // rows of a row tile
constexpr int kKeys = 256;                  // keys of a tile
constexpr int kMaxSlots = 7;                // ring slots; rows of 4 bits leave room for fewer
template <bool Q4>
constexpr int kRingSlots = Q4 ? 4 : 7;
constexpr uint32_t kPanel = 8192;           // 64 rows of 128 bytes
constexpr uint32_t kSlot = 2 * kPanel;      // keys: 128 rows x 64 features; values: 64 rows x 128 features
constexpr int kVSlots = 8;                  // ring slots of a tile's values
constexpr uint32_t kOffP = 9 * kPanel;      // P: 64 rows x 256 keys
constexpr uint32_t kOffRing = kOffP + 4 * kPanel;
// Rows of 4 bits arrive in units of 128 keys x 256 features, codes and scales,
// each the source of four slots: sets of four warps unpack a slot each.  Their
// rotated parts have a place of their own, loaded a tile ahead.
constexpr int kSets = 4, kSetWarps = 4, kUnits = 2;
constexpr uint32_t kUnitScales = 128 * 128, kUnit = kUnitScales + 128 * 16;
template <bool Q4>
constexpr uint32_t kOffRope4 = kOffRing + kRingSlots<Q4> * kSlot;
constexpr uint32_t kOffUnits = kOffRope4<true> + kSlot;
template <bool Q4>
constexpr uint32_t kOffCtl = Q4 ? kOffUnits + kUnits * kUnit : kOffRope4<Q4>;
constexpr uint32_t kColS = 256;             // tensor memory: O, then two S tiles of 128 columns
constexpr int kSegs = 8;                    // work descriptors in flight
// What the loads of a key tile need.
struct Tile {
  int y[kKeys / 16];      // cache row of each box of vbox keys
  int key0, kend, least;  // first key; keys any row sees; last key the first row sees
};

struct Ctl {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t qfull, qempty;
  uint64_t sfull[2], sfree[2];
  uint64_t pready, pfree, ofree, vloc[kMaxSlots];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t tile_full[kTiles], tile_empty[kTiles];
  uint64_t xch[2];
  uint64_t unit_full[kUnits], unit_empty[kUnits], rfull, rempty;   // rows of 4 bits
  uint64_t settle;
  Seg seg[kSegs];
  Tile tile[kTiles];
  float xbuf[2][4][64];
  long long scan64[3 * kThreads<true> / 32];
  Share share;
  uint32_t tmem;
  int abort, peer_abort;
  // what this CTA's loaders have issued, for the end after a wait that gave up
  int loads[kMaxSlots];   // uses of a slot
  int q_issued, rope_issued;
};

template <bool Q4>
constexpr uint32_t kSmem = kOffCtl<Q4> + sizeof(Ctl) + 1024;
static_assert(kSmem<false> <= 227 * 1024 && kSmem<true> <= 227 * 1024, "shared memory");
static_assert(kSmem<false> > kOneCtaSmem && kSmem<true> > kOneCtaSmem,
              "one CTA an SM: it allocates all of tensor memory");

// ------------------------------------------------------------------ cluster
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// Cluster-window address of `a` in CTA `rank` of the pair.
__device__ __forceinline__ uint32_t map_to(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
// Arrival at a barrier of either CTA.  What it announces lies in this CTA's
// shared or tensor memory, complete before it (tcgen05.wait, proxy fence), so
// CTA scope does: a release at cluster scope measured 1100 clk a call.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void expect_at(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void store_at(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ int load_from(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
// ------------------------------------------------------------------ tensor cores, both SMs of the pair
// The MMA warp runs as a whole and one elected lane issues: descriptors then
// stay in uniform registers.  Four MMAs of N = 256 from a single-lane branch
// measured 650 clk (their descriptors move to uniform registers one by one),
// from a converged warp 257, the tensor core's own time.
// Steps 0..2, and 3, of a contraction over 64 elements; SA, SB: a step in
// encoded descriptor units.
template <uint32_t SA, uint32_t SB>
__device__ __forceinline__ void pair_mma_first3(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                uint32_t acc_first) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %9, 0;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %5, %6, %3, 1;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %7, %8, %3, 1;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc_first), "l"(a + SA), "l"(b + SB), "l"(a + 2 * SA), "l"(b + 2 * SB), "r"(el)
      : "memory");
}
template <uint32_t SA, uint32_t SB>
__device__ __forceinline__ void pair_mma_last(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %4, 0;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, 1;\n}" ::"r"(d),
      "l"(a + 3 * SA), "l"(b + 3 * SB), "r"(idesc), "r"(el)
      : "memory");
}
// Arrives on `bar` of both CTAs once the elected lane's MMAs so far are
// complete.
__device__ __forceinline__ void pair_commit(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3), "r"(el)
      : "memory");
}
// A box into this CTA's shared memory; the bytes count on `bar`, a barrier of
// either CTA (cluster address).
__device__ __forceinline__ void pair_tma(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_tma3(uint32_t dst, const CUtensorMap* map, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// (a row tile's beginning and end take about as long as a key tile and a half)
template <bool Q4>
using PairWork = Work<kRows, kKeys, kThreads<Q4>, 1>;

struct Maps2 {
  CUtensorMap q, qr;   // boxes of 64 columns x 64 rows
  // the cache as (64 columns, rows, panels); k: boxes of kbox rows of a
  // panel, v: of vbox rows, of two panels when vbox = 64.  Rows of 4 bits: k:
  // boxes of kbox rows x 128 bytes, v: x 16 bytes
  CUtensorMap k, v;
};

template <typename T, bool ROPE, bool Q4>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<Q4>, 1)
    paged_kernel(const __grid_constant__ Maps2 maps, const Args args) {
  using W = PairWork<Q4>;
  constexpr int kSlots = kRingSlots<Q4>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Ctl* c = reinterpret_cast<Ctl*>(sm + kOffCtl<Q4>);
  const Paged& p = args.a.pg;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1;
  const bool leader = rank == 0;
  constexpr int kKSlots = ROPE && !Q4 ? 9 : 8;   // ring slots of a tile's keys
  int* status = args.status + blockIdx.x;

  // programmatic launch: the merge may be set up from now on (it waits for
  // this grid's end before it reads anything)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    *status = 0;
    c->abort = 0;
    c->q_issued = c->rope_issued = 0;
    mbar_init(&c->qfull, 2);
    mbar_init(&c->qempty, 1);
    mbar_init(&c->settle, 1);
    mbar_init(&c->pready, 2 * kSoft);
    mbar_init(&c->pfree, 1);
    mbar_init(&c->ofree, 2 * kSoft);
    if (leader) {
      // a piece at the beginning, a piece at the end: none until the walk says so
      args.piece[2 * pair].valid = 0;
      args.piece[2 * pair + 1].valid = 0;
    }
    mbar_fence_init();
  } else if (warp == 1) {
    if (lane < kSlots) {
      mbar_init(&c->vloc[lane], 1);
      mbar_init(&c->full[lane], Q4 ? 2 * kSetWarps : 2);
      mbar_init(&c->empty[lane], 1);
      c->loads[lane] = 0;
    }
    mbar_fence_init();
  } else if (warp == 2) {
    if (lane < 2) {
      mbar_init(&c->sfull[lane], 1);
      mbar_init(&c->sfree[lane], 2 * kSoft);
      mbar_init(&c->xch[lane], 4);
    }
    if (lane < kSegs) {
      mbar_init(&c->seg_full[lane], 1);
      mbar_init(&c->seg_empty[lane], kSoft + (leader ? 1 : 0));
    }
    if (Q4 && lane < kUnits) {
      mbar_init(&c->unit_full[lane], 1);
      mbar_init(&c->unit_empty[lane], kSets * kSetWarps);
      if (lane == 0) mbar_init(&c->rfull, 2), mbar_init(&c->rempty, 1);
    }
    if (lane < kTiles) {
      mbar_init(&c->tile_full[lane], 1);
      mbar_init(&c->tile_empty[lane], Q4 ? kSets * kSetWarps + 1 + ROPE : kSlots);
    }
    mbar_fence_init();
  } else if (warp == 3 && lane < 4) {
    const CUtensorMap* m = lane == 0 ? &maps.q : lane == 1 ? &maps.qr : lane == 2 ? &maps.k : &maps.v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  if (warp == 6) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  W::plan(p, &c->share, c->scan64, pair, args.workers);   // with block barriers
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  const Limit w = wait_limit(&c->abort, status, args.a);
  const int ntiles = c->share.ntiles;
  const bool work = ntiles > 0;
  // the ring holds, slot after slot, K(0) K(1) V(0) K(2) V(1) ... K(N-1) V(N-2) V(N-1),
  // over the ends of pieces too: V(t) before K(t+1) there cost every tile more in
  // code than it gained (512 tokens x 128 heads over 16384 keys took 3 % longer)
  const uint32_t ring = smem_u32(sm + kOffRing), lead = 0;

  if (c->share.bad && tid == 0) *status = kErrSeqLens;

  if (work && warp == 6) {
    // ---------------------------------------------------------------- the walk
    // Pieces for the softmax and the MMAs, tiles for the loads, and the query
    // rows.
    const int none = p.num_pages * p.page_size;     // a row outside the maps: zeros
    const int boxes = kKeys / args.vbox;
    const uint32_t qfull = map_to(smem_u32(&c->qfull), lead);
    int b = c->share.seq, left = ntiles, tile = 0;
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
        g.row0 = row + j * kRows;
        g.i0 = j * kRows;
        g.nrows = min(kRows, s.rows - g.i0);
        g.kt0 = kt;
        g.kt1 = min(units, kt + left);
        g.kend = W::tile_keys(p, s, j);
        g.base = p.mode == 3 ? s.kvlen - s.qlen : s.kvlen - 1;
        g.slot = g.kt0 == 0 && g.kt1 == units ? -1 : n == 0 ? 2 * pair : 2 * pair + 1;
        left -= g.kt1 - g.kt0;
        if (g.slot >= 0 && leader && lane == 0)
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
        if (lane < boxes) c->tile[i].y[lane] = y;
        if (lane == 0) {
          c->tile[i].key0 = t * kKeys;
          c->tile[i].kend = g.kend;
          c->tile[i].least = p.mode == 3 ? g.base + g.i0 / p.G : g.base;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->tile_full[i]);
        if (t == g.kt0) {
          // the query rows, once the piece before has done its products
          if (n > 0 && !(ok = warp_wait(&c->qempty, (n - 1) & 1, w))) break;
          if (lane == 0) {
            expect_at(qfull, (8 + ROPE) * kPanel);
            c->q_issued = n + 1;
          }
          __syncwarp();
          if (lane < 8 + ROPE)
            pair_tma(smem_u32(sm) + lane * kPanel, lane < 8 ? &maps.q : &maps.qr, (lane & 7) * 64,
                     g.row0 + rank * 64, qfull);
        }
      }
      // (the last query release: none is on its way to a CTA that has ended)
      if (ok && left == 0) ok = warp_wait(&c->qempty, n & 1, w);
    }
  } else if (Q4 && work && warp == 5) {
    // ---------------------------------------------------------------- rows of 4 bits: TMA loads of units
    // Two of a tile's keys (this CTA's 128, each half of the features), two of
    // its values (each half of the keys, this CTA's 256 features).
    const int nb = 128 / args.kbox, b = lane & 7, kstep = args.kbox / 16;
    const bool codes = lane < nb, issues = codes || (lane >= 8 && lane < 8 + nb);
    const uint32_t bytes = codes ? 128 : 16;
    bool ok = true;
    int u = 0;
    auto load = [&](const Tile& t, int first, int half) {   // rows from key 128 * first, bytes of this half
      const int s = u % kUnits, use = u / kUnits;
      const int y = issues ? t.y[first * 8 + b * kstep] : 0;
      if (use > 0 && !(ok = warp_wait(&c->unit_empty[s], (use - 1) & 1, w))) return;
      if (lane == 0) mbar_expect_tx(&c->unit_full[s], kUnit);
      __syncwarp();
      if (issues)
        tma_2d(smem_u32(sm) + kOffUnits + s * kUnit + (codes ? 0 : kUnitScales) + b * args.kbox * bytes,
               codes ? &maps.k : &maps.v, codes ? half * 128 : kCodes + half * 16, y, &c->unit_full[s]);
      ++u;
    };
    for (int t = -1; t < ntiles && ok; ++t) {
      if (t + 1 < ntiles) {
        const int i = (t + 1) % kTiles;
        if (!(ok = warp_wait(&c->tile_full[i], ((t + 1) / kTiles) & 1, w))) break;
        for (int h = 0; h < 2 && ok; ++h) load(c->tile[i], rank, h);
      }
      if (t >= 0) {
        for (int h = 0; h < 2 && ok; ++h) load(c->tile[t % kTiles], h, rank);
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->tile_empty[t % kTiles]);
      }
    }
    // the copies on their way, whatever else gave up
    for (int k = max(0, u - kUnits); k < u; ++k) mbar_settle(&c->unit_full[k % kUnits], (k / kUnits) & 1, status);
  } else if (Q4 && ROPE && work && warp == 7) {
    // ---------------------------------------------------------------- rows of 4 bits: rotated parts
    const int nb = 128 / args.kbox, kstep = args.kbox / 16;
    const uint32_t bar = map_to(smem_u32(&c->rfull), lead);
    bool ok = true;
    for (int t = 0; t < ntiles && ok; ++t) {
      const int i = t % kTiles;
      if (!(ok = warp_wait(&c->tile_full[i], (t / kTiles) & 1, w))) break;
      const int y = lane < nb ? c->tile[i].y[(int)rank * 8 + lane * kstep] : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->tile_empty[i]);
      if (t > 0 && !(ok = warp_wait(&c->rempty, (t - 1) & 1, w))) break;
      if (lane == 0) {
        expect_at(bar, kSlot);
        c->rope_issued = t + 1;
      }
      __syncwarp();
      if (lane < nb) pair_tma(smem_u32(sm) + kOffRope4<true> + lane * args.kbox * 128, &maps.k, kRopeAt, y, bar);
    }
    if (ok) warp_wait(&c->rempty, (ntiles - 1) & 1, w);   // the last release: none is on its way to a CTA that has ended
  } else if (Q4 && work && (warp < 4 || warp > 15)) {
    // ---------------------------------------------------------------- rows of 4 bits: units to slots
    // Set k takes slot k of every unit; a warp 32 keys of a slot of keys (two
    // steps of 16), or 16 keys of a slot of values (two steps of a panel).
    // Lane: a key of a step's 16 and 32 of its 64 features, so that neighbouring
    // lanes read and write the same piece of eight swizzled rows.
    const int d = warp < 4 ? warp : warp - 12;
    const int set = d >> 2, j = d & 3;
    const int key16 = lane & 15, part = lane >> 4, swz = lane & 7;
    const uint32_t units = smem_u32(sm) + kOffUnits;
    static_assert(!Q4 || kSlots == kSets, "a set has a slot of its own");
    const Dec4<T> dec(args.a.scale_exp);
    const int n_units = 4 * ntiles;
    const uint32_t full = map_to(smem_u32(&c->full[set & 3]), lead);
    uint4 code[2];
    uint32_t two[2];
    // a unit's codes and scales: K(0) K(1) V(0) K(2) V(1) ... K(N-1) V(N-2) V(N-1), two units each
    auto fetch = [&](int n) {
      const int m = (n >> 1) - 1, end = 2 * (ntiles - 1);
      const bool values = m >= 0 && ((m & 1) || m == end);
      const int t = max(m >> 1, 0);   // of values
      const uint32_t src = units + (n % kUnits) * kUnit;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // key of the unit, panel of its four
        const int key = values ? (set >> 1) * 64 + 16 * j + key16 : 32 * j + 16 * h + key16;
        const int panel = values ? (set & 1) * 2 + h : set;
        code[h] = lds128(src + key * 128 + (((2 * panel + part) ^ swz) << 4));
        two[h] = lds_u16(src + kUnitScales + key * 16 + panel * 4 + part * 2);
      }
      const Tile& tl = c->tile[t % kTiles];
      const int at = tl.key0 + (n & 1) * 128 + (set >> 1) * 64 + 16 * j + key16;
      if (values && at > tl.least) {
        // Values of masked keys: rows no query row sees become zeros (they may
        // hold anything), and non-finite values of the others, which would
        // reach rows that do not see them as 0 x inf (a row that sees them has
        // a non-finite score from the same cache row).
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (at >= tl.kend) code[h] = make_uint4(0, 0, 0, 0), two[h] = 0;
          if ((two[h] & 0x7f) == 0x7f) two[h] &= 0xff00;
          if ((two[h] & 0x7f00) == 0x7f00) two[h] &= 0xff;
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&c->unit_empty[n % kUnits]);
        if (values && (n & 1)) mbar_arrive(&c->tile_empty[t % kTiles]);
      }
    };
    bool ok = warp_wait(&c->unit_full[0], 0, w);
    if (ok) fetch(0);
    for (int n = 0; n < n_units && ok; ++n) {
      // (unpacked before the slot is free: what follows its release is short)
      uint4 v[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t sc[2];
        dec.scales(two[h], sc);
        v[h][0] = dec.eight(code[h].x, sc[0]);
        v[h][1] = dec.eight(code[h].y, sc[0]);
        v[h][2] = dec.eight(code[h].z, sc[1]);
        v[h][3] = dec.eight(code[h].w, sc[1]);
      }
      // the next unit's codes now, if they are there, else after the slot
      const int next = n + 1;
      uint64_t* arrived = &c->unit_full[next % kUnits];
      const uint32_t phase = (next / kUnits) & 1;
      const bool early = next < n_units && __all_sync(~0u, mbar_poll(smem_u32(arrived), phase));
      const int m = (n >> 1) - 1;
      const bool values = m >= 0 && ((m & 1) || m == 2 * (ntiles - 1));
      if (early) fetch(next);
      if (n > 0 && !(ok = warp_wait(&c->empty[set], (n - 1) & 1, w))) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at =
            ring + set * kSlot + (values ? h * kPanel + (16 * j + key16) * 128 : (32 * j + 16 * h + key16) * 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) sts128(at + (((4 * part + i) ^ swz) << 4), v[h][i]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) arrive_at(full);
      if (!early && next < n_units) {
        if (!(ok = warp_wait(arrived, phase, w))) break;
        fetch(next);
      }
    }
    // the slot's last release has arrived: none is on its way to a CTA that has ended
    if (ok && j == 0) warp_wait(&c->empty[set], (n_units - 1) & 1, w);
  } else if (!Q4 && work && (warp < 4 || warp == 5 || warp == 7 || warp == 16)) {
    // ---------------------------------------------------------------- TMA loads
    // Slot s: the ring's uses s, s + kSlots, ...
    const int s = warp < 4 ? warp : warp == 5 ? 4 : warp == 7 ? 5 : 6;
    const uint32_t bar = map_to(smem_u32(&c->full[s]), lead), dst = ring + s * kSlot;
    // a slot of keys takes 128 / kbox boxes, one of values 64 / vbox boxes of
    // each panel (or one of both)
    const int nk = 128 / args.kbox, nv = 64 / args.vbox, kstep = args.kbox / args.vbox;
    const int vp = nv == 1 ? 0 : lane / nv, vb = nv == 1 ? 0 : lane - vp * nv;
    const bool vissues = nv == 1 ? lane == 0 : vp < 2;
    const int ky = (int)rank * 2 * nv + lane * kstep;
    const uint32_t kdst = dst + lane * args.kbox * 128, vdst = dst + vp * kPanel + vb * args.vbox * 128;
    int k = 0, nclean = 0;   // uses so far; of them values cleaned here
    bool ok = true;
    auto free_slot = [&]() { return k == 0 || (ok = warp_wait(&c->empty[s], (k - 1) & 1, w)); };
    auto load_k = [&](const Tile& t, int panel) {
      const int y = lane < nk ? t.y[ky] : 0;
      if (!free_slot()) return;
      if (lane < nk) pair_tma3(kdst, &maps.k, y, panel, bar);
      if (lane == 0) {
        expect_at(bar, kSlot);
        c->loads[s] = k + 1;
      }
      ++k;
    };
    // 64 keys, 128 features: part i of the tile's values
    auto load_v = [&](const Tile& t, int i) {
      const int key0 = t.key0 + (i >> 1) * 64, panel = (int)rank * 4 + (i & 1) * 2 + vp;
      const int y = vissues ? t.y[(i >> 1) * nv + vb] : 0;
      // keys that a box brings in; those past `least` are masked for some row
      const int loaded = min(64, (max(0, t.kend - key0) + args.vbox - 1) / args.vbox * args.vbox);
      const bool clean = loaded > 0 && t.least + 1 < key0 + loaded;
      const int first = max(0, t.least + 1 - key0), end = t.kend - key0;
      if (!free_slot()) return;
      if (!clean) {
        if (vissues) pair_tma3(vdst, &maps.v, y, panel, bar);
        if (lane == 0) {
          expect_at(bar, kSlot);
          c->loads[s] = k + 1;
        }
        ++k;
        return;
      }
      // Values of masked keys: rows no query row sees become zeros (they may
      // hold anything), and non-finite values of the others, which would
      // reach rows that do not see them as 0 x inf (a row that sees them has
      // a non-finite score from the same cache row).
      if (lane == 0) mbar_expect_tx(&c->vloc[s], kSlot);
      __syncwarp();
      if (vissues) pair_tma3(vdst, &maps.v, y, panel, smem_u32(&c->vloc[s]));
      mbar_settle(&c->vloc[s], nclean++ & 1, status);   // the copy is on its way, whatever else gave up
      __syncwarp();
      for (int q = first + (lane >> 4); q < loaded; q += 2) {
        const uint32_t at = dst + ((lane >> 3) & 1) * kPanel + q * 128 + ((lane & 7) << 4);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q < end) {
          v = lds128(at);
          float e[8];
          unpack8<T>(v, e);
#pragma unroll
          for (int z = 0; z < 8; ++z) e[z] = fabsf(e[z]) < INFINITY ? e[z] : 0.f;
          v = pack8<T>(e);
        }
        sts128(at, v);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        arrive_at(bar);
        c->loads[s] = k + 1;
      }
      ++k;
    };
    int u = s, base = 0;   // the slot's next use; the first use of the block below
    for (int t = -1; t < ntiles && ok; ++t) {
      if (t + 1 < ntiles) {
        const int i = (t + 1) % kTiles;
        if (!(ok = warp_wait(&c->tile_full[i], ((t + 1) / kTiles) & 1, w))) break;
#pragma unroll 1
        for (; u < base + kKSlots && ok; u += kSlots) load_k(c->tile[i], u - base);
        base += kKSlots;
      }
      if (t >= 0) {
#pragma unroll 1
        for (; u < base + kVSlots && ok; u += kSlots) load_v(c->tile[t % kTiles], u - base);
        base += kVSlots;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->tile_empty[t % kTiles]);
      }
    }
    // the slot's last release has arrived: none is on its way to a CTA that
    // has ended
    if (ok && k > 0) warp_wait(&c->empty[s], (k - 1) & 1, w);
  } else if (work && leader && warp == 4) {
    // ---------------------------------------------------------------- MMAs
    // In the ring's order, S one tile ahead: S(0) S(1) PV(0) S(2) PV(1) ...  The
    // loops over slots are unrolled by 3 and 4: by 1 they cost 6 % each in loop
    // code between the MMAs, by 9 and 8 24 % in fetching it.
    // One warp takes every slot in turn: two, one for each product, could
    // meet a slot's barrier a whole phase early and mistake it for a phase
    // late.  The next slot's barrier is looked at before a slot's last MMA,
    // while the tensor core still has the others to do.
    const uint32_t el = elect_one();
    constexpr uint32_t ids = idesc_f16(kRows, kKeys, Elt<T>::is_f16, false, false);
    constexpr uint32_t idv = idesc_f16(kRows, 256, Elt<T>::is_f16, false, true);
    const uint64_t dq = sdesc_kmajor(smem_u32(sm), 0), dk = sdesc_kmajor(ring, 0);
    const uint64_t dp = sdesc_kmajor(smem_u32(sm + kOffP), 0), dv = sdesc_mnmajor(ring, 0, 64);
    int use = 0, segs = 0, s_left = 0, pv_left = 0, pv_next = 0, pv_segs = 0;
    bool ok = true;
    bool ready = false;   // the next slot is known to be full
    auto slot = [&]() {   // the next slot, full
      const int s = use % kSlots;
      if (!ready) ok = warp_wait(&c->full[s], (use / kSlots) & 1, w);
      ++use;
      return s;
    };
    auto peek = [&]() {
      ready = __all_sync(~0u, mbar_poll(smem_u32(&c->full[use % kSlots]), (use / kSlots) & 1));
    };
    auto products_s = [&](int t) {
      if (s_left == 0) {   // a new piece
        const int r = segs % kSegs;
        if (!(ok = warp_wait(&c->seg_full[r], (segs / kSegs) & 1, w))) return;
        pv_next = s_left = c->seg[r].kt1 - c->seg[r].kt0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->seg_empty[r]);
        if (!(ok = warp_wait(&c->qfull, segs & 1, w))) return;
        ++segs;
      }
      if (t >= 2 && !(ok = warp_wait(&c->sfree[t & 1], (t / 2 - 1) & 1, w))) return;
      tc_fence_after();   // the softmax warps' reads of this S buffer
      const uint32_t d = tmem + kColS + (t & 1) * 128;
      if (Q4 && ROPE) {
        if (!(ok = warp_wait(&c->rfull, t & 1, w))) return;
        const uint64_t a = dq + desc_off(8 * kPanel), b = dk + desc_off(kSlots * kSlot);
        pair_mma_first3<2, 2>(el, d, a, b, ids, 0);
        pair_mma_last<2, 2>(el, d, a, b, ids);
        pair_commit(el, &c->rempty);
      }
#pragma unroll 3
      for (int i = 0; i < kKSlots; ++i) {
        const int s = slot();
        if (!ok) return;
        const uint64_t a = dq + desc_off(i * kPanel), b = dk + desc_off(s * kSlot);
        pair_mma_first3<2, 2>(el, d, a, b, ids, (Q4 && ROPE) || i > 0);
        peek();
        pair_mma_last<2, 2>(el, d, a, b, ids);
        pair_commit(el, &c->empty[s]);
      }
      pair_commit(el, &c->sfull[t & 1]);
      if (--s_left == 0) pair_commit(el, &c->qempty);
    };
    auto products_v = [&](int t, int len) {
      const bool first = pv_left == 0;
      if (first) {
        pv_left = len;
        if (pv_segs++ > 0 && !(ok = warp_wait(&c->ofree, (pv_segs - 2) & 1, w))) return;
      }
      if (!(ok = warp_wait(&c->pready, t & 1, w))) return;
      tc_fence_after();   // ... and reads and rescaling of O
#pragma unroll 4
      for (int i = 0; i < kVSlots; ++i) {
        const int s = slot();
        if (!ok) return;
        const uint32_t d = tmem + (i & 1) * 128;
        const uint64_t a = dp + desc_off((i >> 1) * kPanel), b = dv + desc_off(s * kSlot);
        pair_mma_first3<2, 128>(el, d, a, b, idv, !first || i > 1);
        peek();
        pair_mma_last<2, 128>(el, d, a, b, idv);
        pair_commit(el, &c->empty[s]);
      }
      pair_commit(el, &c->pfree);
      --pv_left;
    };
    for (int t = -1; t < ntiles && ok; ++t) {
      const int len = pv_left == 0 ? pv_next : 0;   // of the piece that tile t begins
      if (t + 1 < ntiles) products_s(t + 1);
      if (t >= 0 && ok) products_v(t, len);
    }
    if (ok) {   // the end mark
      const int r = segs % kSegs;
      ok = warp_wait(&c->seg_full[r], (segs / kSegs) & 1, w);
      if (ok && lane == 0) mbar_arrive(&c->seg_empty[r]);
    }
    // every product done, and the other CTA's last arrivals received
    pair_commit(el, &c->settle);
    mbar_settle(&c->settle, 0, status);
    __syncwarp();
    for (int t = max(0, ntiles - 2); t < ntiles && ok; ++t) ok = warp_wait(&c->sfree[t & 1], (t >> 1) & 1, w);
    if (ok) warp_wait(&c->ofree, (pv_segs - 1) & 1, w);
  } else if (work && warp >= 8 && warp < 16) {
    // ---------------------------------------------------------------- softmax, epilogue
    // Thread: row r of this CTA's 64, keys 128 h + 64 g .. + 63 of a tile, and
    // features 256 h + 128 g .. + 127 of O; the four threads of a row exchange
    // its max.
    const int wq = warp & 3, cg = (warp >> 2) & 1;
    const int l = wq * 32 + lane, r = l & 63, h = l >> 6;
    const uint32_t tq = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t prow = smem_u32(sm + kOffP) + (2 * h + cg) * kPanel + r * 128;
    const uint32_t pready = map_to(smem_u32(&c->pready), lead), ofree = map_to(smem_u32(&c->ofree), lead);
    const uint32_t sfree0 = map_to(smem_u32(&c->sfree[0]), lead);
    const Scale sc = score_scale(args.a.scale);
    int tile = 0, nx = 0;
    // one value of each of the row's four threads
    auto exchange = [&](float v, float* o) {
      c->xbuf[nx & 1][2 * h + cg][r] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->xch[wq & 1]);
      if (!warp_wait(&c->xch[wq & 1], nx & 1, w)) return false;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = c->xbuf[nx & 1][i][r];
      ++nx;
      return true;
    };
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int sr = n % kSegs;
      if (!warp_wait(&c->seg_full[sr], (n / kSegs) & 1, w)) break;
      const Seg g = c->seg[sr];
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->seg_empty[sr]);
      if (g.kt1 == 0) break;
      const int myrow = (int)rank * 64 + r;
      const int least = p.mode == 3 ? g.base + g.i0 / p.G : g.base;   // last key the tile's first row sees
      // ... and this row, counted from the thread's first column of tile 0
      const int last = min(p.mode == 3 ? g.base + (g.i0 + myrow) / p.G : g.base, g.kend - 1) - (h * 128 + cg * 64);
      // the max so far and the one P is relative to (scores before the scale)
      float mtop = -INFINITY, mref = -INFINITY, lsum = 0.f;
      for (int kt = g.kt0; kt < g.kt1; ++kt, ++tile) {
        if (!(ok = warp_wait(&c->sfull[tile & 1], (tile >> 1) & 1, w))) break;
        tc_fence_after();
        const bool edge = (kt + 1) * kKeys > least + 1;
        // half a thread's scores; they are read twice, for the max and for P
        float x[32];
        auto scores = [&](int half) {
          tmem_ld32(tq + kColS + (tile & 1) * 128 + cg * 64 + half * 32, x);
          if (sc.negative) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = -x[i];
          }
          if (edge) {
            const int see = last - kt * kKeys - half * 32;   // last column this row sees
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i > see) x[i] = -INFINITY;
          }
        };
        float top = -INFINITY;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          scores(half);
#pragma unroll
          for (int i = 0; i < 32; i += 2) top = fmaxf(top, fmaxf(x[i], x[i + 1]));
        }
        float mx[4];
        if (!(ok = exchange(top, mx))) break;
        top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        mtop = fmaxf(mtop, top);
        // a stale reference keeps P below 2^8, which both types hold as
        // exactly as values below one; O is rescaled only beyond that
        const bool raise = (top - mref) * sc.log2 > kRaise;
        float f = 1.f;
        if (raise) {
          f = ex2((mref - mtop) * sc.log2);
          mref = mtop;
          lsum *= f;
        }
        const float ref = mref == -INFINITY ? 0.f : mref * sc.log2;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          scores(half);
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(sfree0 + (tile & 1) * 8);
          }
          uint32_t pk[16];
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float a = ex2(fmaf(x[2 * i], sc.log2, -ref)), b = ex2(fmaf(x[2 * i + 1], sc.log2, -ref));
            s0 += a;
            s1 += b;
            pk[i] = Elt<T>::pack(a, b);
          }
          lsum += s0 + s1;
          // P and O belong to the products of the tile before until they end
          if (half == 0) {
            if (tile > 0 && !(ok = warp_wait(&c->pfree, (tile - 1) & 1, w))) break;
            if (kt > g.kt0 && __any_sync(~0u, raise)) {
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < 128; q += 16) {
                float o[16];
                tmem_ld16(tq + cg * 128 + q, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f;
                tmem_st16(tq + cg * 128 + q, o);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(prow + (((half * 4 + i) ^ (r & 7)) << 4),
                   make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]));
        }
        if (!ok) break;
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(pready);
      }
      if (!ok) break;
      float ls[4];
      if (!(ok = exchange(lsum, ls))) break;
      lsum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
      if (!(ok = warp_wait(&c->pfree, (tile - 1) & 1, w))) break;
      tc_fence_after();
      const bool mine = myrow < g.nrows;
      const size_t row = (size_t)g.row0 + myrow;
      const int col = h * 256 + cg * 128;
      const bool whole = g.slot < 0;
      const float inv = lsum > 0.f || lsum != lsum ? 1.0f / lsum : 0.f;
      // O leaves through the 4 KB of the P buffer that this warp alone writes,
      // so that a store covers 128 bytes of 4 rows instead of 16 bytes of 32
      const uint32_t stage = prow - lane * 128;
      const int row0 = (int)rank * 64 + (wq & 1) * 32;   // the warp's first row
      char* dst = whole ? (char*)args.a.out + ((size_t)(g.row0 + row0) * 512 + col) * sizeof(T)
                        : (char*)(args.part + ((size_t)g.slot * kRows + row0) * 512 + col);
      const int stride = 512 * (whole ? (int)sizeof(T) : 4);
      const int fill = whole ? 3 : 1;   // 16 columns are 32 or 64 of a row's 128 staged bytes
      const int piece = lane & 7;
      // (rolled: this code runs once a piece, and fetching it takes longer than
      // running it; unrolled, 6300 clk instead of 4800)
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        float o[16];
        tmem_ld16(tq + cg * 128 + q * 16, o);
        const uint32_t line = stage + lane * 128;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= inv;
          const int at = 2 * (q & 3);
          sts128(line + ((at ^ (lane & 7)) << 4), pack8<T>(o));
          sts128(line + (((at + 1) ^ (lane & 7)) << 4), pack8<T>(o + 8));
        } else {
          const int at = 4 * (q & 1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(line + (((at + i) ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]), __float_as_uint(o[4 * i + 2]),
                              __float_as_uint(o[4 * i + 3])));
        }
        if ((q & fill) != fill) continue;
        __syncwarp();
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
          const int k = i * 4 + (lane >> 3);
          const uint4 u = lds128(stage + k * 128 + ((piece ^ (k & 7)) << 4));
          if (row0 + k < g.nrows) *reinterpret_cast<uint4*>(dst + (size_t)k * stride + piece * 16) = u;
        }
        dst += 128;
        __syncwarp();
      }
      if (mine && h == 0 && cg == 0) {
        if (whole) {
          args.a.smax[row] = mtop == -INFINITY ? mtop : mtop * sc.scale;
          args.a.ssum[row] = lsum > 0.f ? lsum * ex2((mref - mtop) * sc.log2) : lsum;
        } else {
          args.stats[g.slot * kRows + myrow] = make_float4(mtop, mref, lsum, 0.f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(ofree);
    }
  }

  // ---------------------------------------------------------------- end
  __syncthreads();
  if (tid == 0) {
    // the last of the MMA warp's arrivals has come here too
    if (work && !leader) mbar_settle(&c->settle, 0, status);
    store_at(map_to(smem_u32(&c->peer_abort), rank ^ 1), c->abort);
  }
  cluster_sync();
  const bool gave_up = c->abort || c->peer_abort;   // the same in both CTAs
  if (gave_up && tid == 0) {
    // Loads on their way.  The first CTA's barriers count those of both, and
    // the two may have stopped at different places (a slot's uses at most one
    // apart): a phase that one of them has begun gets the other's arrival,
    // then the last phase of every slot is waited for.
    if (leader) {
      auto finish = [&](uint64_t* bar, int mine, int peer) {
        if (mine != peer) mbar_arrive(bar);
        if (max(mine, peer) > 0) mbar_settle(bar, (max(mine, peer) - 1) & 1, status);
      };
      for (int i = 0; i < kSlots; ++i) finish(&c->full[i], c->loads[i], load_from(map_to(smem_u32(&c->loads[i]), 1)));
      finish(&c->qfull, c->q_issued, load_from(map_to(smem_u32(&c->q_issued), 1)));
      if (Q4) finish(&c->rfull, c->rope_issued, load_from(map_to(smem_u32(&c->rope_issued), 1)));
    }
  }
  if (gave_up) cluster_sync();
  if (warp == 6)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
constexpr size_t kOffStatus = 256;
const size_t kOffPiece = kOffStatus + up256(kMaxSms * sizeof(int));
// two pieces a worker: pairs with pieces of 128 rows, or CTAs with pieces of at most 64
const size_t kOffStats = kOffPiece + up256(2 * kMaxSms * sizeof(Piece));
const size_t kOffPart = kOffStats + up256(kMaxSms * kRows * sizeof(float4));

}  // namespace

size_t paged_workspace(const Paged&) { return kOffPart + (size_t)kMaxSms * kRows * 512 * sizeof(float); }

// Few query rows a sequence, on the mean, go to paged_few.cu: their time is the
// cache's bytes, which this file's kernel takes twice (keys, then values).  128
// sequences of 2048 .. 8192 keys took 199 us here and 142 there with 32 rows,
// 200 and 162 with 64; with 128 rows 207 and, cut in two, 296.  Not where the
// tables cannot hold a tile of 64 keys an SM, or ten with more than 32 rows,
// for it takes longer to begin and to end: with 16 rows one sequence of 1000
// keys 23 and 27 us, 128 of 30 .. 300 30.8 and 29.6, 4 of 4000 31 and 27; with
// 64 rows one of 1000 25 and 31, 16 of 3000 33 and 37, 32 of 3000 57 and 49.
static int few_rows(const Paged& p, int nsm) {
  const long long rows = (long long)(p.tnd ? (p.T + p.B - 1) / p.B : p.S1) * p.G;
  const long long keys = (long long)p.B * p.max_pages * p.page_size;
  if (rows <= 32) return keys >= 64LL * nsm ? 32 : 0;
  return rows <= 64 && keys >= 640LL * nsm ? 64 : 0;
}

// Rows of 4 bits that are unpacked on the way to the MMAs cost every row tile
// its unpacking; unpacked ahead of the call, once, and then they pass HBM in 16
// bits.  16 sequences of 4096 keys with 128 heads, on the way and ahead: 128 rows 40 us
// and 55 (bf16), 39 and 58 (fp16), 512 rows 98 and 95, 91 and 100, 768 rows 132 and
// 120, 121 and 125; one sequence of 16384 keys with 1024 rows 59 and 52, 55 and 53, with
// 65,536 rows 2167 and 1384, 1954 and 1400.  Unpacking ahead also takes a workspace.
//
// The mean counts the room of the tensors (T, S1), for the lengths are the
// device's, and one choice serves all sequences.  So a chunk of 512 tokens x 128
// heads beside 63 single tokens of 1024 .. 8192 keys has all of them unpacked: 868 us in
// one call, 711 and 110 in two.  The single tokens alone in tensors with that
// much room to spare take 176 us instead of 110.
static bool many_rows4(const Paged& p) {
  return (long long)(p.tnd ? (p.T + p.B - 1) / p.B : p.S1) * p.G > 512;
}

// Single CTAs for few rows, as for 16 bits, but whatever the tables hold: 128
// sequences of 2048 .. 16384 keys with 16 heads 231 us, in pairs 310; one of 1000 keys 26
// and 27.  (With 64 rows a tile of theirs 187 us for 64 sequences x 128 heads, where
// pairs take 105.)
static int few_rows4(const Paged& p) {
  return (long long)(p.tnd ? (p.T + p.B - 1) / p.B : p.S1) * p.G <= 32 ? 32 : 0;
}

// Where a packed cache's values go: tables, then pages.  Where the cache has no
// more pages than the tables have entries, a page as it lies in the cache (pages
// shared by sequences then are unpacked once, and the tables' place counts
// their rows); else a page for each entry.
static bool by_page(const Paged& p) { return p.num_pages <= (long long)p.B * p.max_pages; }
static size_t table_bytes(const Paged& p) { return up256((size_t)p.B * p.max_pages * sizeof(int)); }

size_t paged4_workspace(const Paged& p) {
  if (!many_rows4(p)) return paged_workspace(p);
  const size_t pages = by_page(p) ? (size_t)p.num_pages : (size_t)p.B * p.max_pages;
  return paged_workspace(p) + table_bytes(p) + pages * p.page_size * p.row * 2;
}

template <typename T>
static cudaError_t launch_unpacked(PagedArgs a, int nsm, cudaStream_t st) {
  const size_t base = paged_workspace(a.pg);
  UnpackArgs u{};
  u.cache = a.cache;
  u.width = a.pg.row;
  u.scale_exp = a.scale_exp;
  u.pg = a.pg;
  u.by_page = by_page(a.pg);
  u.table = reinterpret_cast<int*>(a.ws + base);
  u.out = a.ws + base + table_bytes(a.pg);
  const cudaError_t e = launch_unpack_tables<T>(u, nsm, st);
  if (e != cudaSuccess) return e;
  a.packed = 0;
  a.cache = u.out;
  if (!u.by_page) {
    a.pg.table = u.table;
    a.pg.num_pages = a.pg.B * a.pg.max_pages;
  }
  return launch_paged<T>(a, nsm, st);
}

template <typename T, bool ROPE, bool Q4>
static cudaError_t launch_pairs(const Args& g, cudaStream_t st) {
  const Paged& p = g.a.pg;
  Maps2 m{};
  const bool f16 = Elt<T>::is_f16;
  const uint64_t rows = (uint64_t)p.T * p.G, cached = (uint64_t)p.num_pages * p.page_size;
  if (!encode_map2d(&m.q, f16, g.a.q, 512, rows, 64) ||
      !encode_map2d(&m.qr, f16, ROPE ? g.a.qr : g.a.q, ROPE ? 64 : 512, rows, 64) ||
      (!Q4 && (!encode_map_panels(&m.k, f16, g.a.cache, p.row, cached, g.kbox, 1) ||
               !encode_map_panels(&m.v, f16, g.a.cache, p.row, cached, g.vbox, g.vbox == 64 ? 2 : 1))) ||
      (Q4 && (!encode_map_bytes(&m.k, g.a.cache, kRopeAt + (ROPE ? 128 : 0), cached, 128, g.kbox) ||
              !encode_map_bytes(&m.v, g.a.cache, kRopeAt + (ROPE ? 128 : 0), cached, 16, g.kbox))))
    return cudaErrorInvalidValue;
  auto kern = paged_kernel<T, ROPE, Q4>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<Q4>);
  if (e != cudaSuccess) return e;
  kern<<<g.ctas, kThreads<Q4>, kSmem<Q4>, st>>>(m, g);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_paged_merge<T>(g, kRows, st);
}

template <typename T>
cudaError_t launch_paged(const PagedArgs& a, int nsm, cudaStream_t st) {
  const Paged& p = a.pg;
  if (a.packed && many_rows4(p)) return launch_unpacked<T>(a, nsm, st);
  Args g;
  g.a = a;
  g.workers = nsm / 2;
  g.ctas = 2 * g.workers;
  g.kbox = p.page_size % 128 == 0 ? 128 : p.page_size % 64 == 0 ? 64 : p.page_size % 32 == 0 ? 32 : 16;
  g.vbox = g.kbox < 64 ? g.kbox : 64;
  g.status = reinterpret_cast<int*>(a.ws + kOffStatus);
  g.piece = reinterpret_cast<Piece*>(a.ws + kOffPiece);
  g.stats = reinterpret_cast<float4*>(a.ws + kOffStats);
  g.part = reinterpret_cast<float*>(a.ws + kOffPart);
  if (a.packed) g.vbox = 16;   // the walk's grain
  if (const int few = a.packed ? few_rows4(p) : few_rows(p, nsm)) {
    g.workers = g.ctas = nsm;
    return launch_paged_few<T>(g, few, st);
  }
  return a.packed ? (p.row == 576 ? launch_pairs<T, true, true>(g, st) : launch_pairs<T, false, true>(g, st))
                  : (p.row == 576 ? launch_pairs<T, true, false>(g, st) : launch_pairs<T, false, false>(g, st));
}

template cudaError_t launch_paged<__nv_bfloat16>(const PagedArgs&, int, cudaStream_t);
template cudaError_t launch_paged<__half>(const PagedArgs&, int, cudaStream_t);

}  // namespace sfa
