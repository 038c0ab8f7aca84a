// Internal launch interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "si_select.cuh"

namespace si {

// Parameters of the fused score + select kernel.
struct ScoreParams {
  SelParams sel;
  UnitGrid ug;
  const float* w;      // [B*S, H] fp32 head weights
  const float* w_tail; // bf16: [QT, H] copy of the last batch's last query tile's
                       // rows of w, zero past S (read instead of w by that tile)
  const float* s_q;    // FP8 only: [B*S, H] query row scales
  const float* s_k;    // FP8 only: [B*T] key row scales
  int* counter;        // shared unit counter; this launch's ids start at ug.id_base
  uint32_t* err;       // device error word
  uint64_t timeout_ns; // limit of any single wait
  int nst;             // key-tile pipeline stages
  int nslot;           // strip ring slots
  int debug_flags;     // bit 0: skip the first key-tile load (timeout test)
  unsigned long long* role;  // role counters of a profiling build, else null
};

// Parameters of the sparse attention kernel (128 heads of dim 128).
struct AttnParams {
  const uint16_t* ka;  // [B*T, 128] bf16 key rows
  const uint16_t* va;  // [B*T, 128] bf16 value rows
  const int32_t* idx;  // [B*S, k] listed entries (-1: none)
  float* out;          // [B*S, 128, 128] fp32
  int B, S, T, k;
  float scale_log2;    // softmax scale times log2(e)
  uint32_t* err;       // device error word
  uint64_t timeout_ns; // limit of any single wait
};
size_t sparse_attn_smem_bytes();
cudaError_t launch_sparse_attn(const CUtensorMap& tm_q, const AttnParams& p, int grid,
                               cudaStream_t stream);

// Sizes of a query-group candidate scan (k_pivot.cu): groups of G queries,
// ng = S/G per batch, C candidates per group.
struct PivotParams {
  int B, S, T, H, D, m, G, C, ng;
};
cudaError_t launch_pivot_reps(const uint16_t* q, const float* w, const PivotParams& p,
                              uint16_t* qr, float* wr, cudaStream_t stream);
cudaError_t launch_pivot_cands(const int32_t* rep_idx, const uint16_t* kc, const PivotParams& p,
                               int32_t* cand, uint16_t* kcg, int* vis, cudaStream_t stream);
cudaError_t launch_pivot_remap(int32_t* out_idx, const int32_t* cand, const PivotParams& p, int K,
                               int sms, cudaStream_t stream);

// Shared-memory plan of the fused kernel for one problem shape.
struct ScorePlan {
  int QT;        // queries per tile (nq / H)
  int nq;        // MMA N: query-tile rows (QT * H), 256 or 128
  int CS;        // keys per score strip
  int nst;       // pipeline stages
  int nslot;     // strip ring slots
  int cap;       // selection pool entries per query
  size_t smem;   // dynamic shared memory bytes
  bool ok;
  int err;       // when !ok: 1 = the pools of this topk do not fit, 2 = cs_req
                 // above the largest strip either tile width allows
};

// cs_req: keys per score strip (128 .. 1024), nsl_req: strip ring slots
// (2 .. 4); 0 = the planner's choice.
// rows: queries per batch when known and small (0: many), see k_score_topk.cu
ScorePlan plan_score(bool fp8, int D, int H, int K, int max_smem, int cs_req, int nsl_req,
                     int rows);

cudaError_t launch_score_topk(bool fp8, int D, int H, int nq, const CUtensorMap& tm_q,
                              const CUtensorMap& tm_kc, const ScoreParams& p, int grid,
                              size_t smem, cudaStream_t stream);

size_t topk_scores_smem_bytes(int QT, int cap, int CS);
cudaError_t launch_topk_scores(const float* X, const SelParams& sp, const UnitGrid& ug,
                               int* counter, uint32_t* err, uint64_t timeout_ns, int grid,
                               cudaStream_t stream);

cudaError_t launch_merge(const uint64_t* partial, const SelParams& sp, const UnitGrid& ug,
                         cudaStream_t stream);

// True when the merge kernel already writes sorted rows (small K).
bool merge_sorts_rows(int K);

// Exact sorted rows from a single candidate list per query (one key chunk);
// every row comes out sorted, whatever K.
// The finishing kernel takes a query's one or two lists when they hold at
// most this many keys together (its shared memory, and the fallback select's
// byte counters: at most 255 * 32 keys); other sets go through the merge kernel.
constexpr int kFinishMaxKeys = 8160;
bool finish_takes(int L, int nch);
cudaError_t launch_finish_rows(const uint64_t* partial, const SelParams& sp, const UnitGrid& ug,
                               cudaStream_t stream);

// Sorts each of the rows [rows, K] of (idx, score) in place into the output
// order (score descending, index ascending, padding last).
cudaError_t launch_sort_rows(int32_t* idx, float* score, int64_t rows, int K, int sms,
                             cudaStream_t stream);

cudaError_t launch_quantize_fp8(const uint16_t* x, int64_t rows, int cols, uint8_t* x8,
                                float* scale, cudaStream_t stream);

// How the CTAs of a call over a key/value cache share its tiles' keys: a CTA a
// tile or a fixed chunk of one, a cluster a tile, or equal parts of all of them.
enum { kSplit = 0, kCluster = 1, kShared = 2 };

// Attention of few query rows over a key/value cache (k_attn_rows.cu).
struct RowsParams {
  const uint16_t* q;   // [B,S,H,D] bf16
  uint16_t* out;       // [B,S,H,D] bf16
  float* lse;          // [B,S,H] fp32, or null
  const uint16_t *k, *v;  // bf16 keys and values [B,T,Hk,D]; null: 4-bit pages
  const uint8_t* pages;   // [n_pages, page_bytes]
  const int32_t* table;   // [B, width] pages of each sequence
  int width, n_pages, page_shift;
  int64_t page_bytes;
  const int32_t* idx;  // [B,S,topk] listed entries, or null: the keys a query sees
  int topk;
  const int32_t* lens;    // [B] tokens of each sequence, or null: T
  const int32_t* q_lens;  // [B] its query rows, or null: S
  int B, S, T, H, Hk, G;
  int window, sinks;   // window <= 2^30
  float scale_log2;    // softmax scale (and K scale) times log2(e)
  float v_scale;
  int row_tile, tiles; // rows of a tile (8, 16, 32 or 128); tiles per kv head
  int share;           // how the CTAs share the tiles' keys
  int splits;          // kSplit, kCluster: CTAs of a tile, chunk_keys each;
  int chunk_keys;      // kShared: pieces of a tile at most; the least keys of a CTA
  int ctas;            // kShared
  float* part_o;       // kSplit, kShared: [B*Hk*S*G, splits, D] partial sums
  float2* part_ml;     // [B*Hk*S*G, splits] (maximum in log2 units, sum)
  int64_t* tile_start; // kShared: [B*Hk*tiles] where a tile's steps begin
  int64_t* share_out;  // kShared: steps of a CTA
  int debug_flags;     // 128-row tiles, bit 0: no first block (timeout test)
};
// CTAs of a tile width that an SM holds.
int attn_rows_ctas(int D, bool cache4, int row_tile);
cudaError_t launch_attn_rows(const RowsParams& p, int D, cudaStream_t stream);
// The same over a 4-bit cache in tiles of 128 rows (k_cache4_tiles.cu), and the
// join of its chunks (blocks of 64 keys).
size_t cache4_tiles_smem(int D);
cudaError_t launch_cache4_tiles(const RowsParams& p, int D, int grid, uint32_t* err,
                                uint64_t timeout_ns, cudaStream_t stream);
cudaError_t launch_attn_join_tiles(const RowsParams& p, int D, cudaStream_t stream);

// Window attention of many rows on the tensor cores (k_window_tiles.cu).
struct WinParams {
  const uint16_t *q, *k, *v;  // [B,S,H,D], [B,T,Hk,D] bf16
  uint16_t* out;
  float* lse;                 // or null
  const int32_t *lens, *q_lens;  // [B], or null
  int B, S, T, H, Hk, G;
  int QT;                     // queries of a 128-row tile: 128 / G
  int pairs;                  // pairs of tiles per batch and kv head
  int splits, chunk;          // chunks of a pair's keys at most; blocks of 64 keys of a chunk
  float* part_o;              // splits > 1: [B*S*H, splits, D] partial results
  float2* part_ml;            // [B*S*H, splits] (maximum in log2 units, sum)
  int64_t items;              // B * Hk * pairs * splits
  int window, sinks;
  float scale_log2;
  uint32_t* err;
  uint64_t timeout_ns;
  int debug_flags;            // bit 0: the first K block is never loaded (timeout test)
};
size_t window_tiles_smem(int D);
// tm_vs: the sinks' values alone.
cudaError_t launch_window_tiles(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                const CUtensorMap& tm_v, const CUtensorMap& tm_vs,
                                const WinParams& p, int D, int grid, cudaStream_t stream);

// Rows of a 4-bit paged cache (k_cache4.cu): append reads k, v [B,S,Hk,D]
// bf16, read writes k_out, v_out of that shape.
struct Cache4Params {
  uint8_t* pages;
  const int32_t* table;
  const int32_t* lens;    // [B]
  const int32_t* q_lens;  // [B], or null: S
  int B, S, Hk, width, n_pages, page_shift;
  int cap;                // tokens that a table row can hold
  int64_t page_bytes;
  const uint16_t *k, *v;
  uint16_t *k_out, *v_out;
  float k_scale, v_scale;
};
cudaError_t launch_cache4_rows(const Cache4Params& p, int D, bool append, cudaStream_t stream);

// The life of a cache's pages (k_cache_pages.cu).
struct ForkChild {
  int32_t len;          // its length; -1: not made
  int32_t full;         // pages shared with its parent
  int32_t last, fresh;  // the parent's partly filled page and the copy, or -1
};
struct PagesParams {
  uint8_t* pages;       // [n_pages, page_bytes]
  int64_t page_bytes;
  int32_t* refs;        // [n_pages]
  int32_t* table;       // [B, width]
  int32_t* lens;        // [B]
  int B, width, n_pages, page_shift;
  const int32_t *rows, *src, *dst;  // [n] rows of a call
  int n;
  int32_t* missing;     // extend, fork: what was not done; compact: live pages
  int32_t *refs_out, *table_out;  // compact
  // workspace
  int32_t* order;       // extend, fork: [n_pages] pages taken, by rank
  int32_t* claim;       // fork: [B]
  ForkChild* child;     // fork: [n]
  int32_t *lr, *hole, *mover, *mref, *moves;  // compact: [n_pages] each, [1]
};
cudaError_t launch_pages_extend(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t stream);

// Number of units (query tile x key chunk x batch) in a launch.
int host_count_units(const UnitGrid& u);
int host_tile_chunks(const UnitGrid& u, int g);

}  // namespace si
