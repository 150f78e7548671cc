// Internal launcher declarations shared by the C-ABI host code and the kernels.
#pragma once
#include "common.cuh"
#include "paged.cuh"

namespace sfa {

constexpr int kModeBwd = 0;       // S and dP -> P, dS
// S -> partial max / sum statistics; the per-token kernel (sdp.cu) also
// stages P relative to each partial max (one partial per 32 keys)
constexpr int kModeFwdStats = 1;

// Score / softmax-gradient kernel (sdp.cu).  The staged P^T / dS^T rows go
// through the store maps maps.Pw / maps.dSw.
template <typename T>
cudaError_t launch_sdp(const Maps& maps, const Prob& p, int mode, float* tile_stats, int* gerr, int nsm,
                       cudaStream_t st);

// Key-major dK / dV for block-sparse indices (kvb.cu): group the chunk's
// (token, index) pairs by block start (count, scan, scatter), then accumulate
// every group's block in tensor memory and add it to acc once.  res >= 0
// (deterministic mode; entries sorted within each group): only the groups
// whose start is res modulo bs, whose blocks share no key row.
// pst / dsst (optional): the staged P^T / dS^T; the rows no group covers
// (pairs left out, padding slots) are zeroed.  tile_stats (optional, the
// forward's per-pair statistics): a left-out pair's entries are set to
// {-inf, 0}.
cudaError_t launch_blk_count(const Prob& p, int* cnt, void* pst, void* dsst, float* tile_stats, cudaStream_t st);
// nres (optional, bs entries): non-empty bins per residue modulo bs.
cudaError_t launch_blk_scan(const int* cnt, int nbins, int* cursor, int* groups, int* gbeg, int* ngroups, int bs,
                            int* nres, cudaStream_t st);
cudaError_t launch_blk_scatter(const Prob& p, int* cursor, int* entries, cudaStream_t st);
template <typename T>
cudaError_t launch_kvb(const BlkMaps& maps, const Prob& p, int bs, const int* groups, const int* gbeg,
                       const int* ngroups, const int* entries, float* acc, int res, const int* nres, int* gerr,
                       int nsm, cudaStream_t st);

// Key-major scores for block-sparse indices (sdpb.cu): per group of pairs
// sharing a block start, S (and dP) of packs of 128 / GK tokens against the
// block's resident key (and value) rows.  mode kModeBwd writes the pairs'
// staged P^T / dS^T rows; kModeFwdStats the pairs' partial statistics
// (tile_stats, (token, index, head) x {max, sum}) and their P^T rows relative
// to each pair's max.
template <typename T>
cudaError_t launch_sdpb(const Maps& maps, const Prob& p, int mode, const int* groups, const int* gbeg,
                        const int* ngroups, const int* entries, void* pst, void* dsst, float* tile_stats, int* gerr,
                        int nsm, cudaStream_t st);

// Key-side and query-side contractions in one launch, two pipelines per CTA
// (kvq.cu): key-side reductions into acc, dQ / dQRope out.  tile_group: key
// tiles per key-side work item, at least 1 (items run tile-group major; a
// group of all tiles gives token-major order).  part:
// deterministic mode; acc is then the chunk's partial-row buffer (bf16
// elements) and every valid (token, slot) row is stored there instead of
// reduced.
template <typename T>
cudaError_t launch_kvq(const Maps& maps, const Prob& p, float* acc, void* dq, void* dqr, int tile_group, bool part,
                       int* gerr, int nsm, cudaStream_t st);

// dQ / dQRope for block-sparse indices with at most 64 heads (dqb.cu):
// features on the MMA's M, heads on N, over each token's selected blocks.
// pv: the companion forward's O = P V instead (value rows; dq is the
// output, dqr unused), from P staged by sdpb's statistics pass relative to
// each (token, block) pair's max and rescaled to the final statistics
// p.smax, p.ssum; part_stats: that pass's (pair, head) x {max, sum}.
template <typename T>
cudaError_t launch_dqb(const Maps& maps, const Prob& p, bool pv, void* dq, void* dqr, const float* part_stats,
                       int* gerr, int nsm, cudaStream_t st);

// Companion forward's output O = P V over each token's selected keys (dq.cu),
// from the P staged by sdp.cu's statistics pass relative to each 32-key
// group's max, rescaled per (group, head) to the final statistics p.smax,
// p.ssum.  part_stats: that pass's (token, Kpad / 32 groups, head) x {max of
// the raw score, sum}.
template <typename T>
cudaError_t launch_pv(const Maps& maps, const Prob& p, const float* part_stats, void* out, int* gerr, int nsm,
                      cudaStream_t st);

// Small kernels (prep.cu).
cudaError_t launch_rowtab(const Prob& p, cudaStream_t st);
cudaError_t launch_batch_prefix(const Prob& p, int B, const int* act_q, const int* act_kv, int* batch_ofs, int* gerr,
                                cudaStream_t st);
cudaError_t launch_meta(const Prob& p, int layout, int B, int S1, int S2, int mode, const int* act_q, const int* act_kv,
                        int* batch_ofs, TokMeta* meta, int* gerr, cudaStream_t st);
// Dsum of tokens tok0 .. tok0 + ntok - 1 (all heads).
template <typename T>
cudaError_t launch_dsum(const Prob& p, int tok0, int ntok, float* dsum, cudaStream_t st);
template <typename T>
cudaError_t launch_cast(const float* acc, int T2, void* dk, void* dkr, void* dv, int has_rope, cudaStream_t st);
// ntiles: partial statistics per token (32-key groups, or block indices).
cudaError_t launch_stats_combine(const Prob& p, const float* tile_stats, int ntiles, float* smax, float* ssum,
                                 cudaStream_t st);

// Records a message for sfa_last_error_message on the calling thread (api.cu).
void set_last_error(const char* msg);
// SMs of the current device (api.cu).
int device_sm_count();
// 2-D map of rows x cols 16-bit elements, boxes of 64 columns x box_rows rows
// with 128-byte swizzle; false when the driver refuses it (api.cu).
bool encode_map2d(CUtensorMap* m, bool f16, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows);
// The same rows as (64 columns, rows, cols / 64 panels), boxes of 64 x
// box_rows x box_panels.
bool encode_map_panels(CUtensorMap* m, bool f16, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows,
                       uint32_t box_panels);
// Rows of bytes, boxes of box_bytes (128 with 128-byte swizzle, or fewer) x box_rows.
bool encode_map_bytes(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_bytes,
                      uint32_t box_rows);

// Deterministic key-side reduction (det.cu): counting sort of the chunk's
// (kv row, token, slot) entries by row (count, then launch_blk_scan over the
// T2 rows, scatter, per-row sort), then one fixed-order sum per row.
cudaError_t launch_det_count(const Prob& p, int* cnt, cudaStream_t st);
cudaError_t launch_det_scatter(const Prob& p, int* cursor, int* ent, cudaStream_t st);
// Sorts each row's segment of entry ids ascending: long_segs = false sorts the
// segments of up to 1024 entries, true the longer ones (two launches).
cudaError_t launch_det_sort(const Prob& p, const int* gbeg, const int* ngroups, int* ent, int* scratch, bool long_segs,
                            cudaStream_t st);
cudaError_t launch_det_reduce(const Prob& p, const int* groups, const int* gbeg, const int* ngroups, const int* ent,
                              const uint16_t* partials, float* acc, cudaStream_t st);

// Workspaces that grow with the grid are sized for this many SMs, and grids
// are cut to it.
constexpr int kMaxSms = 160;

// Norm and rotation of input rows (rows.cu).  Forward: q, k, qr, kr -> qo, ko,
// qro, kro.  Gradient: dq, dk with q, k -> qo, ko and the weights' gradients;
// qr, kr are then the rotated rows' gradients.
struct RowsArgs {
  const int* pos;        // (axes, T) or null
  const float* cs;       // (table_len, 64)
  long long table_len;
  int axes;                      // 1..4
  unsigned long long axis_map;   // two bits a pair: the axis whose position turns it
  const void *q, *qw, *qr, *k, *kw, *kr;
  void *qo, *qro, *ko, *kro;
  float *q_rstd, *k_rstd;
  const void *dq, *dk;
  float *dqw, *dkw, *part;
  int T, G, interleaved, backward;
  float eps;
  int blocks_k, blocks_q;   // set by the launchers
};
template <typename T>
cudaError_t launch_norm_rope(RowsArgs a, cudaStream_t st);
template <typename T>
cudaError_t launch_norm_rope_grad(RowsArgs a, int nsm, cudaStream_t st);
// Blocks (partial sums of dw) of the gradient over `rows` rows of 512.
int norm_grad_blocks(long long rows, int nsm);

// Append to the paged cache (append.cu).  Where the rows go follows from the
// lengths and the block table, or (slots not null) stands in a map, with the
// positions beside it; of pg that case uses T, G, row and the cache's sizes.
struct AppendArgs {
  Paged pg;
  const int* slots;      // (T) or null
  const int* pos;        // (axes, T), with slots
  int axes;
  unsigned long long axis_map;
  int packed, scale_exp; // rows of 4 bits, in units of 2^scale_exp
  void* cache;
  const void *k, *kr, *kw, *qr;
  void* qro;
  const float* cs;       // null without rope
  long long table_len;
  int* error;            // or null
  double eps;
  int interleaved;
  int blocks_k;          // set by the launcher
};
template <typename T>
cudaError_t launch_append(AppendArgs a, cudaStream_t st);

// Values of a 4-bit cache (cache4.cu): all of it, rows in order
// (launch_unpack), or the pages that the block tables of pg name
// (launch_unpack_tables).
struct UnpackArgs {
  const void* cache;
  void* out;
  long long rows;        // all of it: num_pages * page_size
  int width, scale_exp;  // elements of a row: 512 or 576
  Paged pg;              // the tables' form
  int by_page;           // out's pages lie as the cache's do; else one for each entry of the tables
  int* table;            // by page: rows taken of each page (num_pages); else the tables of `out`
};
template <typename T>
cudaError_t launch_unpack(const UnpackArgs& a, int nsm, cudaStream_t st);
template <typename T>
cudaError_t launch_unpack_tables(const UnpackArgs& a, int nsm, cudaStream_t st);

// Block tables and slot maps of a step (plan.cu).
struct PlanArgs {
  int* table;            // (B, max_pages)
  const int *kv, *fresh; // (B): tokens in the cache; new ones, negative where the request has ended
  int* free;             // (num_pages): the free pages, the first *count
  const int* count;
  int *q_out, *kv_out, *count_out, *slots, *pos;
  int* error;            // or null
  int B, max_pages, num_pages, page_size, tokens;
};
constexpr int kPlanRequests = 8192;   // most of a call: their sums lie in shared memory
cudaError_t launch_plan(const PlanArgs& a, int nsm, cudaStream_t st);

// Attention over the paged cache (paged.cu).
struct PagedArgs {
  Paged pg;
  const void *q, *qr, *cache;
  void* out;
  float *smax, *ssum;
  float scale;
  int packed, scale_exp; // rows of 4 bits, in units of 2^scale_exp
  int brief;             // the wait limit is short against a suspension
  unsigned long long wait_ns;
  uint8_t* ws;
};
size_t paged_workspace(const Paged& p);
size_t paged4_workspace(const Paged& p);   // rows of 4 bits
template <typename T>
cudaError_t launch_paged(const PagedArgs& a, int nsm, cudaStream_t st);

}  // namespace sfa
