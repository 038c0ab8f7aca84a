// The C ABI of the key/value cache (include/streamindex.h): attention with a
// window and sinks, the 4-bit paged cache, and the life of its pages.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "si_api.h"
#include "si_kernels.h"

namespace si {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int kWindowMax = 1 << 30;  // longer than any sequence

// log2 of a page size, or -1.
int page_shift_of(int page, int lo, int hi) {
  if (page < lo || page > hi || (page & (page - 1))) return -1;
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

// Softmax scales, finite in log2 units too; false for NaN.
bool scale_finite(float s) { return s >= 0.0f && s * 1.4426950408889634f <= FLT_MAX; }

bool scale_ok(float g) { return g >= 0x1p-60f && g <= 0x1p60f; }  // false for NaN

// Sizes that the two attention calls share.
int check_attention(int B, int S, int H, int H_k, int d) {
  if (B < 1 || S < 1 || H < 1 || H_k < 1 || H % H_k || !(d == 64 || d == 128)) return SI_ERR_DIM;
  if ((int64_t)B * S * H >= ((int64_t)1 << 31)) return SI_ERR_DIM;
  return SI_OK;
}

// The plan over a call's keys: the tile width, how the CTAs share the tiles'
// keys, and the bytes of partial results.  keys: what one query may see at
// most; spread: how far the sequences may differ in what they see.
//
// Tile width: the narrowest of 8, 16 and 32 rows that holds a kv head's rows,
// so that keys are read once; over a 4-bit cache 128-row tensor-core tiles from
// 17 rows on.  (B200, one kv head's 32 rows and 64 of them at D = 128: 28.8 us in
// 32-row tiles and 17 in 128-row ones for one sequence of 4,096 keys, 72.8 and
// 63.6 for eight of 16,384, 76.7 and 51.4 for 32 of 4,096.  With 16 rows the
// 16-row tiles take 20.7, 44.5 and 45.4.)
//
// Sharing, tiles below 128 rows:
//  kSplit, a CTA a tile, where tiles see as much and the places that the last
//    round of CTAs leaves idle would save less than a join costs: 32 steps of
//    rows of 128 elements (of any rows where a cluster would do).  (bf16, 32
//    sequences, 8 kv heads, window 1,024: 25.4 us; 33.9 in equal shares, 37 in
//    fixed chunks and a join.  12 such sequences, 96 tiles: window 512 13.3 us
//    and 18.5 in shares, window 2,048 34.9 and 29.  64 sequences, two rounds on
//    296 places, window 1,024: 61.4 and 71.7, with rows of 64 36.9 and 47.5; 48
//    sequences, window 2,048: 98.3 and 92.1, with rows of 64 55.8 and 61.7.
//    4-bit, 128 sequences on 592 places, window 512: 32.7 and 43.)
//    A window of more than half the table may be longer than most sequences; the
//    imbalance then counts as an eighth of the places left idle.  (bf16, 37
//    ragged sequences and 37 full ones, a window as long as the table: 77.8 and
//    111.7 us against 76.1 and 117.1 in shares at 4,096 tokens, 269 and 365
//    against 201 and 369 at 16,384; 32 of 4,096: 75.5 and 100.4 against 68.5 and
//    112.  4-bit, 74 sequences of up to 8,192: 139 and 154 against 113 and 160.)
//    Also where tiles are many times the places.
//  kCluster, a tile's chunks in one cluster that joins them, for calls of few
//    steps whose clusters are all resident (three drafted tokens of four
//    sequences: 13.9 us, with a join kernel 19.3; 32 ragged sequences of up to
//    8,192 keys in clusters 81 us, in shares 58).
//  kShared else: one wave of CTAs, each with an equal share of all steps.
enum { kAlike, kUnknown, kUnlike };
int plan_rows(RowsParams* p, int64_t keys, bool cache4, int spread, int key_chunk, int sms, int d,
              size_t* bytes) {
  const bool listed = p->topk > 0;
  const int64_t rows = listed ? p->G : std::min<int64_t>((int64_t)p->S * p->G, 1 << 20);
  p->row_tile = rows <= 8 ? 8 : rows <= 16 ? 16 : cache4 ? 128 : 32;
  const int rt = p->row_tile;
  const int64_t per = listed ? (int64_t)p->S * ((p->G + rt - 1) / rt)
                             : ((int64_t)p->S * p->G + rt - 1) / rt;
  const int64_t tiles = (int64_t)p->B * p->Hk * per;
  if (tiles >= ((int64_t)1 << 31)) return SI_ERR_DIM;
  p->tiles = (int)per;
  // a tile's queries see a little more than one of them; the sinks and the
  // window's two ends come in whole steps (32 keys, 64 in 128-row tiles)
  const int64_t span = listed ? keys : std::min<int64_t>(p->T, keys + rt / p->G + 1);
  const int64_t steps = (span + 31) / 32 + (listed ? (rt == 128 ? 1 : 0) : (rt == 128 ? 6 : 3));
  const int64_t all = (int64_t)p->B * p->S * p->H;
  int64_t chunk = steps;
  *bytes = 0;
  if (rt == 128) {
    // a persistent CTA per SM: the number of chunks that makes the rounds of
    // CTAs times a chunk's cost least, a chunk costing 256 keys besides its own
    if (key_chunk > 0) {
      chunk = std::max<int64_t>(key_chunk / 32, (steps + 1023) / 1024);
    } else if (tiles < sms) {
      int64_t best = -1;
      for (int64_t n = 1; n <= 64; ++n) {
        const int64_t c = ((steps + n - 1) / n + 3) / 4 * 4;
        const int64_t cost = (tiles * ((steps + c - 1) / c) + sms - 1) / sms * (c + 8);
        if (best < 0 || cost < best) best = cost, chunk = c;
      }
    }
    chunk = (chunk + 3) / 4 * 4;  // whole pairs of blocks
    p->share = kSplit;
  } else {
    const int64_t room = (int64_t)sms * attn_rows_ctas(d, cache4, rt);
    const int64_t least = 8;  // two steps of 32 keys for each of a CTA's warps
    // clusters of up to eight, as long as the GPU holds all of them at once
    const int64_t n = std::min<int64_t>(8, std::max<int64_t>(1, room / tiles));
    const bool few = n > 1 && steps <= n * least * 2;  // a cluster's share is a few steps
    const int64_t idle = (room - tiles % room) % room + (spread == kUnknown ? room / 8 : 0);
    if (key_chunk == 0 && steps <= least) {
      p->share = kSplit;
    } else if (key_chunk == 0 &&
               ((spread != kUnlike && 2 * tiles > sms &&
                 steps * idle * (few ? 128 : d) <= 32 * room * 128) ||
                tiles > 8 * room)) {
      p->share = kSplit;
    } else if (key_chunk == 0 && few) {
      p->share = kCluster;
      chunk = std::max<int64_t>(least, (steps + n - 1) / n);
    } else {
      // equal shares: a tile falls into at most so many pieces
      const int64_t pieces = std::min<int64_t>(96, std::max<int64_t>(8, 8 * room / tiles));
      chunk = std::max<int64_t>(key_chunk > 0 ? key_chunk / 32 : least,
                                (steps + pieces - 3) / (pieces - 2));
      p->share = kShared;
      p->ctas = (int)room;
      p->splits = (int)std::min<int64_t>(pieces, (steps - 1) / chunk + 2);
    }
  }
  p->chunk_keys = (int)chunk * 32;
  if (rt == 128 && (steps + chunk - 1) / chunk <= 8) p->share = kCluster;
  if (p->share != kShared) p->splits = (int)((steps + chunk - 1) / chunk);
  if (p->share == kCluster && p->splits == 1) p->share = kSplit;
  if (tiles * p->splits >= ((int64_t)1 << 31)) return SI_ERR_DIM;
  if (p->share != kCluster && p->splits > 1)
    *bytes = align256((size_t)all * p->splits * d * sizeof(float)) +
             align256((size_t)all * p->splits * sizeof(float2)) +
             (p->share == kShared ? align256((size_t)(tiles + 1) * sizeof(int64_t)) : 0);
  return SI_OK;
}

int place_partials(RowsParams* p, int d, size_t need, void* ws, size_t ws_bytes) {
  if (!need) return SI_OK;
  if (!ws || ws_bytes < need) return SI_ERR_WORKSPACE;
  if (!aligned16(ws)) return SI_ERR_ALIGN;
  const int64_t rows = (int64_t)p->B * p->S * p->H;
  char* at = static_cast<char*>(ws);
  p->part_o = reinterpret_cast<float*>(at);
  at += align256((size_t)rows * p->splits * d * sizeof(float));
  p->part_ml = reinterpret_cast<float2*>(at);
  at += align256((size_t)rows * p->splits * sizeof(float2));
  p->share_out = reinterpret_cast<int64_t*>(at);
  p->tile_start = p->share_out + 1;
  return SI_OK;
}

// Whether a window call runs in 128-row tensor-core tiles: from so many
// (query, head) rows per kv head on, unless the caller fixed key chunks.  (B200,
// 8 heads a kv head, D = 128: 32 rows over a window of 512 take 22.7 us in 32-row
// tiles and 14.5 in 128-row ones for one sequence, 37.2 and 26.5 for 64; 16 rows
// 14.5 in 16-row tiles and 14.5, 19.2 and 26.2.)
constexpr int kTileRows = 17;
// What a pair of tiles costs besides its blocks of 64 keys, and the join of
// chunks of them, in blocks.
constexpr int kItemBlocks = 6, kJoinBlocks = 20;
bool window_in_tiles(int S, int G, int key_chunk) {
  return G <= 128 && (int64_t)S * G >= kTileRows && key_chunk == 0;
}

// How 128-row tiles share a pair's keys, and the bytes of partial results: the
// number of chunks that makes rounds of CTAs times a chunk's cost least.  (B200,
// D = 64, 256 rows of each of two kv heads over 32,768 keys: 483 us whole, 37 in
// chunks; D = 128, four kv heads, window 2,048: 40.2 and 26.3, window 512: 16.5
// and 24.7, where the rule takes them whole.)
int plan_window_tiles(const RowsParams& p, int sms, int d, WinParams* w, size_t* bytes) {
  w->QT = 128 / p.G;
  w->pairs = (int)(((int64_t)p.S + 2 * w->QT - 1) / (2 * w->QT));
  const int64_t pairs = (int64_t)p.B * p.Hk * w->pairs;
  // a pair's queries see a little more than one of them
  const int64_t most = std::min<int64_t>(p.S, 2 * w->QT);
  const int64_t blocks = (std::min<int64_t>(p.T, (int64_t)p.window + most - 1) + 63) / 64 +
                         (std::min<int64_t>(p.sinks, p.T) + 63) / 64;
  int64_t best = (pairs + sms - 1) / sms * (blocks + kItemBlocks);
  w->splits = 1;
  w->chunk = (int)blocks;
  for (int64_t n = 2; n <= 32 && pairs * n <= 2 * sms; ++n) {
    const int64_t c = (blocks + n - 1) / n, s = (blocks + c - 1) / c;
    const int64_t cost = (pairs * s + sms - 1) / sms * (c + kItemBlocks) + kJoinBlocks;
    if (cost < best) best = cost, w->chunk = (int)c, w->splits = (int)s;
  }
  w->items = pairs * w->splits;
  if (w->items >= ((int64_t)1 << 31)) return SI_ERR_DIM;
  const int64_t rows = (int64_t)p.B * p.S * p.H * w->splits;
  *bytes = w->splits == 1 ? 0 : align256((size_t)rows * d * sizeof(float)) +
                                    align256((size_t)rows * sizeof(float2));
  return SI_OK;
}

// Whether tokens see about as many keys in every sequence: where the window is
// what bounds them.
int spread_of(int window, int T) { return 2 * (int64_t)window <= T ? kAlike : kUnknown; }

// Sizes of a window call and its plan.  full: all sequences have T tokens.  (A
// size query does not know; what it answers is no less, see plan_rows.)
int window_problem(int B, int S, int T, int H, int H_k, int d, int window, int sinks, bool full,
                   const si_options* opt, RowsParams* p, WinParams* w, Opts* o, size_t* bytes) {
  int rc = check_attention(B, S, H, H_k, d);
  if (rc) return rc;
  if (T < 1 || T >= (1 << 30) || (int64_t)B * T * H_k >= ((int64_t)1 << 31)) return SI_ERR_DIM;
  if (window < 1 || sinks < 0) return SI_ERR_OPTIONS;
  if ((rc = read_opts(opt, o))) return rc;
  p->B = B, p->S = S, p->T = T, p->H = H, p->Hk = H_k, p->G = H / H_k;
  p->window = std::min(window, kWindowMax);
  p->sinks = std::min(sinks, kWindowMax);
  int max_smem = 0, sms = 0;
  plan_limits(&max_smem, &sms);
  if (window_in_tiles(S, p->G, o->key_chunk)) return plan_window_tiles(*p, sms, d, w, bytes);
  return plan_rows(p, std::min<int64_t>(T, (int64_t)p->window + p->sinks), false,
                   full ? kAlike : spread_of(window, T), o->key_chunk, sms, d, bytes);
}

int cache4_problem(int width, int page, int topk, int B, int S, int H, int H_k, int d, int window,
                   int sinks, const si_options* opt, RowsParams* p, Opts* o, size_t* bytes) {
  int rc = check_attention(B, S, H, H_k, d);
  if (rc) return rc;
  const int sh = page_shift_of(page, 16, 256);
  if (sh < 0 || width < 1 || (int64_t)width * page >= (1 << 30) ||
      (int64_t)B * width >= ((int64_t)1 << 31))
    return SI_ERR_DIM;
  if (topk < 0 || topk > SI_MAX_TOPK) return SI_ERR_TOPK;
  if (window < 0 || sinks < 0 || (window == 0 && sinks) || (topk && window)) return SI_ERR_OPTIONS;
  if ((rc = read_opts(opt, o))) return rc;
  p->B = B, p->S = S, p->T = width * page, p->H = H, p->Hk = H_k, p->G = H / H_k;
  p->width = width;
  p->page_shift = sh;
  p->page_bytes = (int64_t)H_k * page * (d + d / 8);
  p->topk = topk;
  p->window = window ? std::min(window, kWindowMax) : kWindowMax;
  p->sinks = std::min(sinks, kWindowMax);
  int max_smem = 0, sms = 0;
  plan_limits(&max_smem, &sms);
  const int64_t keys =
      topk ? topk : std::min<int64_t>(p->T, (int64_t)p->window + p->sinks);
  return plan_rows(p, keys, true, topk ? kAlike : window ? spread_of(window, p->T) : kUnlike,
                   o->key_chunk, sms, d, bytes);
}

// The sizes of a call on the rows of a 4-bit cache.
int cache4_rows(int B, int S, int H_k, int d, int n_pages, int width, int page, float k_scale,
                float v_scale, Cache4Params* p) {
  if (B < 1 || S < 1 || H_k < 1 || !(d == 64 || d == 128) || n_pages < 1 || width < 1)
    return SI_ERR_DIM;
  const int sh = page_shift_of(page, 16, 256);
  if (sh < 0 || (int64_t)width * page >= (1 << 30) || (int64_t)B * width >= ((int64_t)1 << 31) ||
      (int64_t)B * S * H_k >= ((int64_t)1 << 31))
    return SI_ERR_DIM;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return SI_ERR_OPTIONS;
  p->B = B, p->S = S, p->Hk = H_k, p->width = width, p->n_pages = n_pages;
  p->page_shift = sh;
  p->cap = width * page;
  p->page_bytes = (int64_t)H_k * page * (d + d / 8);
  p->k_scale = k_scale, p->v_scale = v_scale;
  return SI_OK;
}

// Workspace of the page calls, laid out for any of them.
struct PagesLayout {
  size_t a, b, c, d, e, total;
};
PagesLayout pages_layout(int n_pages, int B, int n) {
  PagesLayout l;
  const size_t pool = align256((size_t)n_pages * 4);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += bytes;
    return r;
  };
  l.a = take(pool);                                    // order, or live ranks
  l.b = take(std::max(pool, align256((size_t)B * 4))); // claims, or holes
  l.c = take(std::max(pool, align256((size_t)n * sizeof(ForkChild))));  // children, or movers
  l.d = take(pool);                                    // the movers' counts
  l.e = take(256);                                     // the number of moves
  l.total = at;
  return l;
}

int check_pool(int n_pages, int B, int width) {
  if (n_pages < 1 || B < 1 || width < 1 || (int64_t)B * width >= ((int64_t)1 << 31))
    return SI_ERR_DIM;
  return SI_OK;
}

int pages_call(int32_t* refs, int n_pages, int32_t* table, int B, int width, int32_t* lens,
               int page, PagesParams* p) {
  int rc = check_pool(n_pages, B, width);
  if (rc) return rc;
  const int sh = page_shift_of(page, 1, 1 << 16);
  if (sh < 0) return SI_ERR_DIM;
  if (!aligned4(refs) || !aligned4(table) || !aligned4(lens)) return SI_ERR_ALIGN;
  p->refs = refs, p->n_pages = n_pages, p->table = table, p->B = B, p->width = width;
  p->lens = lens;
  p->page_shift = sh;
  return SI_OK;
}

int place_pages(PagesParams* p, void* ws, size_t ws_bytes) {
  const PagesLayout l = pages_layout(p->n_pages, p->B, p->n);
  if (!ws || ws_bytes < l.total) return SI_ERR_WORKSPACE;
  if (!aligned16(ws)) return SI_ERR_ALIGN;
  char* w = static_cast<char*>(ws);
  p->order = p->lr = reinterpret_cast<int32_t*>(w + l.a);
  p->claim = p->hole = reinterpret_cast<int32_t*>(w + l.b);
  p->mover = reinterpret_cast<int32_t*>(w + l.c);
  p->child = reinterpret_cast<ForkChild*>(w + l.c);
  p->mref = reinterpret_cast<int32_t*>(w + l.d);
  p->moves = reinterpret_cast<int32_t*>(w + l.e);
  return SI_OK;
}

// A pool's pages and the CTAs that copy n of them.
int check_pages(const void* pages, int64_t page_bytes, int64_t n) {
  if (page_bytes < 16 || page_bytes % 16 || page_bytes > ((int64_t)1 << 30)) return SI_ERR_DIM;
  if (n * ((page_bytes + 16383) / 16384) >= ((int64_t)1 << 31)) return SI_ERR_DIM;
  return aligned16(pages) ? SI_OK : SI_ERR_ALIGN;
}

int status(cudaError_t e) { return e == cudaSuccess ? SI_OK : SI_ERR_CUDA; }

}  // namespace
}  // namespace si

using namespace si;

extern "C" {

// ------------------------------------------------------------ window attention
int si_window_attention_workspace_size(int B, int S, int T, int H, int H_k, int d, int window,
                                       int sinks, const si_options* opt, size_t* bytes) {
  if (!bytes) return SI_ERR_NULL;
  RowsParams p{};
  WinParams w{};
  Opts o;
  size_t need = 0;
  const int rc = window_problem(B, S, T, H, H_k, d, window, sinks, false, opt, &p, &w, &o, &need);
  if (rc == SI_OK) *bytes = need;
  return rc;
}

int si_window_attention(const void* qa, const void* ka, const void* va, const int32_t* lens,
                        const int32_t* q_lens, int B, int S, int T, int H, int H_k, int d,
                        int window, int sinks, float scale, void* out, float* lse,
                        const si_options* opt, void* workspace, size_t ws_bytes, void* stream) {
  if (!qa || !ka || !va || !out) return SI_ERR_NULL;
  RowsParams p{};
  WinParams w{};
  Opts o;
  size_t need = 0;
  int rc = window_problem(B, S, T, H, H_k, d, window, sinks, !lens, opt, &p, &w, &o, &need);
  if (rc) return rc;
  if (!scale_finite(scale)) return SI_ERR_OPTIONS;
  if (!aligned16(qa) || !aligned16(ka) || !aligned16(va) || !aligned16(out) || !aligned4(lens) ||
      !aligned4(q_lens) || !aligned4(lse))
    return SI_ERR_ALIGN;
  const bool tiles = window_in_tiles(S, p.G, o.key_chunk);
  p.splits = tiles ? w.splits : p.splits;
  if ((rc = place_partials(&p, d, need, workspace, ws_bytes))) return rc;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  p.q = static_cast<const uint16_t*>(qa);
  p.k = static_cast<const uint16_t*>(ka);
  p.v = static_cast<const uint16_t*>(va);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.lens = lens;
  p.q_lens = q_lens;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.v_scale = 1.0f;
  if (!tiles) return status(launch_attn_rows(p, d, static_cast<cudaStream_t>(stream)));
  if (window_tiles_smem(d) > (size_t)dev->max_smem) return SI_ERR_UNSUPPORTED;
  w.q = p.q, w.k = p.k, w.v = p.v, w.out = p.out, w.lse = lse;
  w.lens = lens, w.q_lens = q_lens;
  w.B = B, w.S = S, w.T = T, w.H = H, w.Hk = H_k, w.G = p.G;
  w.part_o = p.part_o, w.part_ml = p.part_ml;
  w.window = p.window, w.sinks = p.sinks;
  w.scale_log2 = std::max(p.scale_log2, FLT_MIN);  // times -inf for an unseen key: not NaN
  w.err = dev->err;
  w.timeout_ns = (uint64_t)o.timeout_ms * 1000000ull;
  w.debug_flags = o.debug_flags;
  CUtensorMap tm_q, tm_k, tm_v, tm_vs;
  if ((rc = make_map4(&tm_q, qa, d, H, S, B, p.G, w.QT, S)) ||
      (rc = make_map4(&tm_k, ka, d, H_k, T, B, 1, 32, T)) ||
      (rc = make_map4(&tm_v, va, d, H_k, T, B, 1, 32, T)) ||
      (rc = make_map4(&tm_vs, va, d, H_k, p.sinks > 0 ? std::min(p.sinks, T) : T, B, 1, 32, T)))
    return rc;
  const int most = o.grid_ctas > 0 ? o.grid_ctas : dev->sms;
  return status(launch_window_tiles(tm_q, tm_k, tm_v, tm_vs, w, d, (int)std::min<int64_t>(most, w.items),
                                    static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------ 4-bit cache
int si_cache4_page_bytes(int H_k, int d, int page, size_t* bytes) {
  if (!bytes) return SI_ERR_NULL;
  if (H_k < 1 || H_k > (1 << 16) || !(d == 64 || d == 128) || page_shift_of(page, 16, 256) < 0)
    return SI_ERR_DIM;
  *bytes = (size_t)H_k * page * (d + d / 8);
  return SI_OK;
}

int si_cache4_append(const void* k, const void* v, int B, int S, int H_k, int d, void* pages,
                     int n_pages, const int32_t* table, int width, int page, const int32_t* lens,
                     const int32_t* q_lens, float k_scale, float v_scale, void* stream) {
  if (!k || !v || !pages || !table || !lens) return SI_ERR_NULL;
  Cache4Params p{};
  int rc = cache4_rows(B, S, H_k, d, n_pages, width, page, k_scale, v_scale, &p);
  if (rc) return rc;
  if (!aligned16(k) || !aligned16(v) || !aligned16(pages) || !aligned4(table) ||
      !aligned4(lens) || !aligned4(q_lens))
    return SI_ERR_ALIGN;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  p.pages = static_cast<uint8_t*>(pages);
  p.table = table;
  p.lens = lens;
  p.q_lens = q_lens;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  return status(launch_cache4_rows(p, d, true, static_cast<cudaStream_t>(stream)));
}

int si_cache4_read(void* k, void* v, int B, int S, int H_k, int d, const void* pages, int n_pages,
                   const int32_t* table, int width, int page, const int32_t* lens,
                   const int32_t* q_lens, float k_scale, float v_scale, void* stream) {
  if (!k || !v || !pages || !table || !lens) return SI_ERR_NULL;
  Cache4Params p{};
  int rc = cache4_rows(B, S, H_k, d, n_pages, width, page, k_scale, v_scale, &p);
  if (rc) return rc;
  if (!aligned16(k) || !aligned16(v) || !aligned16(pages) || !aligned4(table) ||
      !aligned4(lens) || !aligned4(q_lens))
    return SI_ERR_ALIGN;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  p.pages = const_cast<uint8_t*>(static_cast<const uint8_t*>(pages));
  p.table = table;
  p.lens = lens;
  p.q_lens = q_lens;
  p.k_out = static_cast<uint16_t*>(k);
  p.v_out = static_cast<uint16_t*>(v);
  return status(launch_cache4_rows(p, d, false, static_cast<cudaStream_t>(stream)));
}

int si_cache4_attention_workspace_size(int width, int page, int topk, int B, int S, int H, int H_k,
                                       int d, int window, int sinks, const si_options* opt,
                                       size_t* bytes) {
  if (!bytes) return SI_ERR_NULL;
  RowsParams p{};
  Opts o;
  size_t need = 0;
  const int rc =
      cache4_problem(width, page, topk, B, S, H, H_k, d, window, sinks, opt, &p, &o, &need);
  if (rc == SI_OK) *bytes = need;
  return rc;
}

int si_cache4_attention(const void* qa, const void* pages, int n_pages, const int32_t* table,
                        int width, int page, const int32_t* lens, const int32_t* q_lens,
                        const int32_t* idx, int topk, int B, int S, int H, int H_k, int d,
                        int window, int sinks, float scale, float k_scale, float v_scale,
                        void* out, float* lse, const si_options* opt, void* workspace,
                        size_t ws_bytes, void* stream) {
  if (!qa || !pages || !table || !lens || !out) return SI_ERR_NULL;
  if (idx ? topk < 1 : topk != 0) return SI_ERR_TOPK;
  if (n_pages < 1) return SI_ERR_DIM;
  RowsParams p{};
  Opts o;
  size_t need = 0;
  int rc = cache4_problem(width, page, topk, B, S, H, H_k, d, window, sinks, opt, &p, &o, &need);
  if (rc) return rc;
  if (!scale_ok(k_scale) || !scale_ok(v_scale) || !scale_finite(scale * k_scale))
    return SI_ERR_OPTIONS;
  if (!aligned16(qa) || !aligned16(pages) || !aligned16(out) || !aligned4(table) ||
      !aligned4(lens) || !aligned4(q_lens) || !aligned4(idx) || !aligned4(lse))
    return SI_ERR_ALIGN;
  if ((rc = place_partials(&p, d, need, workspace, ws_bytes))) return rc;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  p.q = static_cast<const uint16_t*>(qa);
  p.pages = static_cast<const uint8_t*>(pages);
  p.n_pages = n_pages;
  p.table = table;
  p.lens = lens;
  p.q_lens = q_lens;
  p.idx = idx;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.scale_log2 = scale * k_scale * 1.4426950408889634f;
  p.v_scale = v_scale;
  p.debug_flags = o.debug_flags;
  if (p.row_tile < 128)
    return status(launch_attn_rows(p, d, static_cast<cudaStream_t>(stream)));
  if (cache4_tiles_smem(d) > (size_t)dev->max_smem) return SI_ERR_UNSUPPORTED;
  const int64_t items = (int64_t)B * H_k * p.tiles * p.splits;
  const int most = o.grid_ctas > 0 ? o.grid_ctas : dev->sms;
  return status(launch_cache4_tiles(p, d, (int)std::min<int64_t>(most, items), dev->err,
                                    (uint64_t)o.timeout_ms * 1000000ull,
                                    static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------ pages
int si_cache_workspace_size(int n_pages, int B, int n, size_t* bytes) {
  if (!bytes) return SI_ERR_NULL;
  if (n_pages < 1 || B < 1 || n < 0) return SI_ERR_DIM;
  *bytes = pages_layout(n_pages, B, n).total;
  return SI_OK;
}

int si_cache_extend(int32_t* refs, int n_pages, int32_t* table, int B, int width,
                    const int32_t* lens, int page, int32_t* missing, void* workspace,
                    size_t ws_bytes, void* stream) {
  if (!refs || !table || !lens || !missing) return SI_ERR_NULL;
  PagesParams p{};
  int rc = pages_call(refs, n_pages, table, B, width, const_cast<int32_t*>(lens), page, &p);
  if (rc) return rc;
  if (!aligned4(missing)) return SI_ERR_ALIGN;
  if ((rc = place_pages(&p, workspace, ws_bytes))) return rc;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  p.missing = missing;
  return status(launch_pages_extend(p, static_cast<cudaStream_t>(stream)));
}

int si_cache_fork(void* pages, int64_t page_bytes, int32_t* refs, int n_pages, int32_t* table,
                  int B, int width, int32_t* lens, const int32_t* src, const int32_t* dst, int n,
                  int page, int32_t* missing, void* workspace, size_t ws_bytes, void* stream) {
  if (!pages || !refs || !table || !lens || !missing || (n > 0 && (!src || !dst)))
    return SI_ERR_NULL;
  if (n < 0) return SI_ERR_DIM;
  PagesParams p{};
  int rc = pages_call(refs, n_pages, table, B, width, lens, page, &p);
  if (rc) return rc;
  if ((rc = check_pages(pages, page_bytes, n))) return rc;
  if (!aligned4(missing) || !aligned4(src) || !aligned4(dst)) return SI_ERR_ALIGN;
  p.pages = static_cast<uint8_t*>(pages);
  p.page_bytes = page_bytes;
  p.src = src, p.dst = dst, p.n = n;
  p.missing = missing;
  if ((rc = place_pages(&p, workspace, ws_bytes))) return rc;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  return status(launch_pages_fork(p, static_cast<cudaStream_t>(stream)));
}

int si_cache_free(int32_t* refs, int n_pages, int32_t* table, int B, int width, int32_t* lens,
                  const int32_t* rows, int n, void* stream) {
  if (!refs || !table || !lens || (n > 0 && !rows)) return SI_ERR_NULL;
  if (n < 0) return SI_ERR_DIM;
  PagesParams p{};
  int rc = pages_call(refs, n_pages, table, B, width, lens, 1, &p);
  if (rc) return rc;
  if (!aligned4(rows)) return SI_ERR_ALIGN;
  p.rows = rows;
  p.n = n;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  return status(launch_pages_free(p, static_cast<cudaStream_t>(stream)));
}

int si_cache_compact(void* pages, int64_t page_bytes, const int32_t* refs, int n_pages,
                     const int32_t* table, int B, int width, int32_t* refs_out,
                     int32_t* table_out, int32_t* live, void* workspace, size_t ws_bytes,
                     void* stream) {
  if (!pages || !refs || !table || !refs_out || !table_out || !live) return SI_ERR_NULL;
  int rc = check_pool(n_pages, B, width);
  if (rc) return rc;
  if ((rc = check_pages(pages, page_bytes, 1))) return rc;
  if (!aligned4(refs) || !aligned4(table) || !aligned4(refs_out) || !aligned4(table_out) ||
      !aligned4(live))
    return SI_ERR_ALIGN;
  PagesParams p{};
  p.pages = static_cast<uint8_t*>(pages);
  p.page_bytes = page_bytes;
  p.refs = const_cast<int32_t*>(refs);
  p.n_pages = n_pages;
  p.table = const_cast<int32_t*>(table);
  p.B = B, p.width = width;
  p.refs_out = refs_out, p.table_out = table_out;
  p.missing = live;
  if ((rc = place_pages(&p, workspace, ws_bytes))) return rc;
  DevInfo* dev;
  if ((rc = dev_info(&dev))) return rc;
  return status(launch_pages_compact(p, dev->sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
