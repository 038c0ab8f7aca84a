// Attention of few query rows over a key/value cache: the decode form of the
// window attention (bf16 keys) and of the attention over a 4-bit paged cache.
//
//   o[row] = sum_j softmax_j(scale * q[row] . k[j]) v[j],  lse[row] = ln sum_j exp(...)
//
// over the keys the row's query sees (si_attn.cuh), or over the entries that a
// row of the indexer lists.  The G = H / H_k query heads of a kv head share its
// keys, so (query, head) pairs are the rows of a tile of 16.
//
// What bounds it: a decode step reads every visible key once and multiplies it
// with few rows, so HBM does.  One warp takes KS keys at a time from a ring of
// its own in shared memory (cp.async, no barrier between warps), the running
// maximum and sum stay in registers, and the warps of a CTA (and, with few
// sequences, several CTAs: `splits`) share a sequence's keys; their results
// are joined at the end, by k_attn_join when there are several CTAs.  16-row
// mma.sync tiles are what this shape needs: tcgen05's 128 rows would be empty
// but for a few, and its operands would have to pass through shared memory as
// 16-bit numbers, four times the bytes of the 4-bit codes.
//
// 4-bit keys (E2M1 codes, an E4M3 scale per 16 elements): code x scale has six
// significant bits, so it is exact in fp16, and the products run in fp16 with
// fp32 accumulation.  A query row is scaled by a power of two into fp16's
// range (bf16 to fp16 drops no bit of an element within 2^-25 of the row's
// largest).  The dot product does not depend on the order of its terms, so a
// thread's fragment of a key row is simply 16 consecutive bytes of codes: no
// shuffle, no transposition.  A value fragment pairs two keys for one element;
// taking the nibbles of two code words together gives the pairs without a
// transposition too.  Probabilities are rounded to fp16 after a scale of 2^10
// (2^-11 relative down to 2^-24 of the row's largest); the sum takes them
// unrounded.
//
// bf16 keys: bf16 products, probabilities rounded to bf16 (2^-8).
#include <type_traits>

#include "si_attn.cuh"

namespace si {
namespace {

constexpr int kRowWarps = 4;
constexpr int kRowTile = 16;
constexpr float kProbShift = 10.0f;  // 4-bit path: probabilities times 2^10

// What a warp holds of its tile while it walks over keys.
template <int D>
struct RowState {
  float o[D / 8][4];
  float m[2], l[2];
};

// ------------------------------------------------------------ 4-bit pages
// Key order inside a group of 16: column n of score tile t is this key.  A
// quad's columns 2c, 2c+1 then are keys whose value rows lie in different
// banks, and so are the key rows that a quarter-warp reads.
SI_DEV int group_key(int t, int n) { return 8 * t + ((n & 1) ? 4 + ((n >> 1) ^ 1) : (n >> 1)); }

template <int D>
struct Cache4 {
  static constexpr int KS = 32;
  static constexpr int kStages = 3;
  static constexpr int kCodes = KS * D / 2, kScales = KS * D / 16;
  static constexpr int kStageBytes = 2 * kCodes + 2 * kScales;

  uint32_t qf[D / 16][4];
  float row_factor[2];

  // Byte of a value row's 16-byte chunk in its stage (a swizzle by key).
  static SI_DEV int v_off(int key, int chunk) {
    return key * (D / 2) + ((D == 128 ? chunk ^ (((key >> 1) & 1) << 1) : chunk) << 4);
  }

  SI_DEV void load_q(const RowsParams& p, const uint16_t* const (&qr)[2], int lane) {
    const int c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[D / 8];  // D/4 elements of the row: D/4 * c ...
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = qr[h] ? __ldg(reinterpret_cast<const uint4*>(qr[h] + (D / 4) * c) + i)
                              : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      // 2^(10 - e) for a largest element in [2^e, 2^(e+1)); 1 for rows of
      // zeros or with an infinity, 2^126 at most
      const int e = (int)(__float_as_uint(top) >> 23);
      const int up = (e == 0 || e == 255) ? 0 : min(126, 137 - e);
      const float f = __uint_as_float((uint32_t)(127 + max(up, -126)) << 23);
      row_factor[h] = __uint_as_float((uint32_t)(127 - max(up, -126)) << 23);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][h] = pack_f16x2(bf16_lo(w[2 * s]) * f, bf16_hi(w[2 * s]) * f);
        qf[s][2 + h] = pack_f16x2(bf16_lo(w[2 * s + 1]) * f, bf16_hi(w[2 * s + 1]) * f);
      }
    }
  }

  // Scores of 16 keys (two tiles of 8 columns) from a stage.
  SI_DEV void scores(uint32_t kc, uint32_t ks, int lane, float (&s)[2][4]) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int key = group_key(t, r);
      uint32_t w[D / 32];
      uint32_t sc;
      if constexpr (D == 128) {
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(kc + key * 64 + c * 16));
        asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                     : "=r"(sc)
                     : "r"(ks + key * 8 + c * 2));
      } else {
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                     : "=r"(w[0]), "=r"(w[1])
                     : "r"(kc + key * 32 + c * 8));
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sc) : "r"(ks + key * 4 + c));
      }
      const uint32_t s2 = e4m3x2(sc);
      const uint32_t slo = __byte_perm(s2, 0, 0x1010), shi = __byte_perm(s2, 0, 0x3232);
      s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t sf = (D == 128 && i >= 2) ? shi : slo;
        mma_f16(s[t], qf[2 * i], hmul2(e2m1x2<0>(w[i]), sf), hmul2(e2m1x2<1>(w[i]), sf));
        mma_f16(s[t], qf[2 * i + 1], hmul2(e2m1x2<2>(w[i]), sf), hmul2(e2m1x2<3>(w[i]), sf));
      }
    }
  }

  // o += P V over 16 keys; `live`: which keys of the group may be read (their
  // codes count as zero else).
  SI_DEV void values(uint32_t vc, uint32_t vs, int lane, const uint32_t (&pf)[4], uint32_t live,
                     RowState<D>& st) const {
    const int n = lane >> 2, c = lane & 3;
    uint32_t sp[2], w[4][D / 64];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = group_key(t, 2 * c + i);
        if constexpr (D == 128) {
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                       : "=r"(w[2 * t + i][0]), "=r"(w[2 * t + i][1])
                       : "r"(vc + v_off(key, n >> 1) + (n & 1) * 8));
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b[i]) : "r"(vs + key * 8 + n));
        } else {
          asm volatile("ld.shared.b32 %0, [%1];"
                       : "=r"(w[2 * t + i][0])
                       : "r"(vc + key * 32 + n * 4));
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b[i]) : "r"(vs + key * 4 + (n >> 1)));
        }
        if (!((live >> key) & 1u)) b[i] = 0u;
      }
      sp[t] = e4m3x2(b[0] | (b[1] << 8));
    }
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      // even elements of both keys of a pair in the bytes of lo, odd ones in hi
      uint32_t lo[2], hi[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t a = w[2 * t][x], b = w[2 * t + 1][x];
        lo[t] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
        hi[t] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
      }
#define SI_PV(BYTE)                                                                          \
  mma_f16(st.o[8 * x + 2 * BYTE], pf, hmul2(e2m1x2<BYTE>(lo[0]), sp[0]),                     \
          hmul2(e2m1x2<BYTE>(lo[1]), sp[1]));                                                \
  mma_f16(st.o[8 * x + 2 * BYTE + 1], pf, hmul2(e2m1x2<BYTE>(hi[0]), sp[0]),                 \
          hmul2(e2m1x2<BYTE>(hi[1]), sp[1]));
      SI_PV(0)
      SI_PV(1)
      SI_PV(2)
      SI_PV(3)
#undef SI_PV
    }
  }

  // Element of the row that accumulator o[i][.] column e (0, 1) of a thread is.
  static SI_DEV int element(int i, int c, int e) { return (D / 8) * (2 * c + e) + i; }
};

// ------------------------------------------------------------ bf16 rows
template <int D>
struct Bf16Rows {
  static constexpr int KS = D == 128 ? 16 : 32;
  static constexpr int kStages = 3;
  static constexpr int kRows = KS * D * 2;
  static constexpr int kStageBytes = 2 * kRows;

  uint32_t qf[D / 16][4];
  float row_factor[2];

  static SI_DEV int off(int key, int chunk) {
    return key * (D * 2) + ((chunk ^ (key & 7)) << 4);
  }

  SI_DEV void load_q(const RowsParams& p, const uint16_t* const (&qr)[2], int lane) {
    const int c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row_factor[h] = 1.0f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][h] = qr[h] ? __ldg(reinterpret_cast<const uint32_t*>(qr[h] + 16 * s + 2 * c)) : 0u;
        qf[s][2 + h] =
            qr[h] ? __ldg(reinterpret_cast<const uint32_t*>(qr[h] + 16 * s + 8 + 2 * c)) : 0u;
      }
    }
  }

  SI_DEV void scores(uint32_t kb, int g, int lane, float (&s)[2][4]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
      const int key = 16 * g + 8 * t + (lane & 7);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t b[4];
        ldmatrix4(b, kb + off(key, 4 * i + (lane >> 3)));
        mma_bf16(s[t], qf[2 * i], b[0], b[1]);
        mma_bf16(s[t], qf[2 * i + 1], b[2], b[3]);
      }
    }
  }

  SI_DEV void values(uint32_t vb, int g, int lane, const uint32_t (&pf)[4], RowState<D>& st) const {
    const int key = 16 * g + (lane & 15);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t b[4];
      ldmatrix4_t(b, vb + off(key, 2 * i + (lane >> 4)));
      mma_bf16(st.o[2 * i], pf, b[0], b[1]);
      mma_bf16(st.o[2 * i + 1], pf, b[2], b[3]);
    }
  }

  static SI_DEV int element(int i, int c, int e) { return 8 * i + 2 * c + e; }
};

// The tile's rows and what its queries see.
struct Tile {
  int b, hk, row0, rows;  // rows: live rows of the tile
  int len, q_len, t_min, t_max;
  int64_t part;           // index of its first row among all rows
};

SI_DEV bool find_tile(const RowsParams& p, int64_t id, Tile& ti) {
  const int tile = (int)(id % p.tiles);
  const int64_t bh = id / p.tiles;
  ti.b = (int)(bh / p.Hk);
  ti.hk = (int)(bh % p.Hk);
  ti.len = seq_len(p.lens, ti.b, p.T);
  ti.q_len = seq_len(p.q_lens, ti.b, p.S);
  int last;  // one past the tile's last row
  if (p.idx) {  // a tile's rows belong to one query
    const int per = (p.G + kRowTile - 1) / kRowTile;
    const int i = tile / per;
    ti.row0 = i * p.G + (tile % per) * kRowTile;
    last = min((i + 1) * p.G, ti.q_len * p.G);
  } else {
    ti.row0 = tile * kRowTile;
    last = ti.q_len * p.G;
  }
  ti.rows = min(kRowTile, last - ti.row0);
  if (ti.rows <= 0) return false;
  ti.t_min = ti.len - ti.q_len + ti.row0 / p.G;
  ti.t_max = ti.len - ti.q_len + (ti.row0 + ti.rows - 1) / p.G;
  ti.part = bh * p.S * p.G + ti.row0;
  return true;
}

SI_DEV int64_t out_row(const RowsParams& p, const Tile& ti, int row) {
  const int i = row / p.G;
  return ((int64_t)ti.b * p.S + i) * p.H + ti.hk * p.G + row % p.G;
}

}  // namespace

// MODE 0: bf16 keys [B,T,H_k,D]; 1: 4-bit pages; 2: 4-bit pages, listed entries.
template <int D, int MODE>
__global__ void __launch_bounds__(kRowWarps * 32, 3)
    k_attn_rows(const __grid_constant__ RowsParams p) {
  using Src = typename std::conditional<MODE == 0, Bf16Rows<D>, Cache4<D>>::type;
  constexpr int KS = Src::KS, NST = Src::kStages, NG = KS / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sh_m[kRowWarps][kRowTile], sh_l[kRowWarps][kRowTile];
  __shared__ uint32_t sh_nan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int split = (int)(blockIdx.x % p.splits);
  Tile ti;
  if (!find_tile(p, blockIdx.x / p.splits, ti)) return;
  if (threadIdx.x == 0) sh_nan = 0u;

  const KeySpan span = MODE == 2 ? KeySpan{0, 0, p.topk, 0, 0, (p.topk + KS - 1) / KS}
                                 : key_span<KS>(ti.t_min, ti.t_max, ti.len, p.window, p.sinks);
  const int u_lo = (int)((int64_t)span.steps * split / p.splits);
  const int u_hi = (int)((int64_t)span.steps * (split + 1) / p.splits);

  Src src;
  int t_row[2];
  {
    const uint16_t* qr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = r + 8 * h;
      const bool live = row < ti.rows;
      qr[h] = live ? p.q + out_row(p, ti, ti.row0 + row) * D : nullptr;
      t_row[h] = ti.len - ti.q_len + (ti.row0 + min(row, ti.rows - 1)) / p.G;
    }
    src.load_q(p, qr, lane);
  }
  const float f_row[2] = {src.row_factor[0] * p.scale_log2, src.row_factor[1] * p.scale_log2};

  RowState<D> st;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.0f;
  st.m[0] = st.m[1] = neg_inf();
  st.l[0] = st.l[1] = 0.0f;

  const uint32_t ring = smem_u32(smem) + warp * NST * Src::kStageBytes;
  uint32_t vmask[NST];  // keys of a stage that lie in a page
#pragma unroll
  for (int i = 0; i < NST; ++i) vmask[i] = 0u;

  // What the next step to be loaded needs from memory first (its pages, or its
  // entries), read one step ahead.
  int ahead[NG];        // MODE 1: page of each group of 16 keys; -1: none
  int64_t a_off = 0;    // MODE 2: this lane's entry
  int a_slot = 0;
  bool a_ok = false;
  const int32_t* table = MODE ? p.table + (int64_t)ti.b * p.width : nullptr;
  const int32_t* irow =
      MODE == 2 ? p.idx + ((int64_t)ti.b * p.S + ti.row0 / p.G) * p.topk : nullptr;
  auto look_ahead = [&](int u) {
    if constexpr (MODE == 1) {
      const int j0 = step_key<KS>(span, u);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int j = j0 + 16 * g;
        const bool in = u < u_hi && j < (u < span.sink_steps ? span.sink_end : span.end) &&
                        (j + 16 > span.lo || j < p.sinks);
        const int pg = in ? __ldg(table + (j >> p.page_shift)) : -1;
        ahead[g] = pg >= 0 && pg < p.n_pages ? pg : -1;
      }
    } else if constexpr (MODE == 2) {
      const int e = u * KS + lane;
      const int j = u < u_hi && e < p.topk ? __ldg(irow + e) : -1;
      a_ok = j >= 0 && j < ti.len;
      const int pg = a_ok ? __ldg(table + (j >> p.page_shift)) : -1;
      a_ok = pg >= 0 && pg < p.n_pages;
      a_off = (int64_t)(a_ok ? pg : 0) * p.page_bytes;
      a_slot = a_ok ? j & ((1 << p.page_shift) - 1) : 0;
    }
  };
  const int page = MODE ? 1 << p.page_shift : 0;
  const uint8_t* head_block = MODE ? p.pages + (int64_t)ti.hk * cache4_block<D>(page) : nullptr;

  // Start the copies of step u into a stage.
  auto issue = [&](int u, int stage, uint32_t& vm) {
    const uint32_t dst = ring + stage * Src::kStageBytes;
    if constexpr (MODE == 0) {
      if (u < u_hi) {
        const int j0 = step_key<KS>(span, u);
        constexpr int kChunks = D / 8;  // 16-byte chunks of a row
        const int64_t stride = (int64_t)p.Hk * D;
        const int64_t first = ((int64_t)ti.b * p.T) * stride + (int64_t)ti.hk * D;
#pragma unroll
        for (int x = 0; x < KS * kChunks / 32; ++x) {
          const int key = (x * 32 + lane) / kChunks, ch = lane % kChunks;
          const int j = j0 + key;
          const bool ok = span_holds(span, u, j, p.sinks);
          const int64_t at = first + (ok ? j : 0) * stride + ch * 8;
          cp_async16(dst + Src::off(key, ch), p.k + at, ok ? 16u : 0u);
          cp_async16(dst + Src::kRows + Src::off(key, ch), p.v + at, ok ? 16u : 0u);
        }
        vm = 0xFFFFFFFFu;
      }
    } else {
      constexpr int kCodes = Src::kCodes, kScales = Src::kScales;
      constexpr int kChunks = D / 32;  // 16-byte chunks of a row's codes
      if (u < u_hi) {
        if constexpr (MODE == 1) {
          const int j0 = step_key<KS>(span, u);
          uint32_t m = 0u;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const int pg = ahead[g];
            const bool ok = pg >= 0;
            if (ok) m |= 0xFFFFu << (16 * g);
            const int slot = (j0 + 16 * g) & (page - 1);
            const uint8_t* blk = head_block + (int64_t)(ok ? pg : 0) * p.page_bytes;
            const uint8_t* kc = blk + slot * (D / 2);
            const uint8_t* vc = kc + page * (D / 2);
            const uint8_t* ks = blk + page * D + slot * (D / 16);
            const uint8_t* vs = ks + page * (D / 16);
#pragma unroll
            for (int x = 0; x < 16 * kChunks / 32; ++x) {
              const int i = x * 32 + lane, key = 16 * g + i / kChunks, ch = i % kChunks;
              cp_async16(dst + key * (D / 2) + ch * 16, kc + i * 16, ok ? 16u : 0u);
              cp_async16(dst + kCodes + Src::v_off(key, ch), vc + i * 16, ok ? 16u : 0u);
            }
            if (lane < D / 8) {  // D bytes of K scales, then as many of V scales
              const int i = lane % (D / 16);
              const bool is_v = lane >= D / 16;
              cp_async16(dst + 2 * kCodes + (is_v ? kScales : 0) + g * D + i * 16,
                         (is_v ? vs : ks) + i * 16, ok ? 16u : 0u);
            }
          }
          vm = m;
        } else {
          vm = __ballot_sync(0xFFFFFFFFu, a_ok);
#pragma unroll
          for (int x = 0; x < kChunks; ++x) {
            const int key = (x * 32 + lane) / kChunks, ch = lane % kChunks;
            const int64_t off = __shfl_sync(0xFFFFFFFFu, a_off, key);
            const int slot = __shfl_sync(0xFFFFFFFFu, a_slot, key);
            const uint32_t n = (vm >> key) & 1u ? 16u : 0u;
            const uint8_t* kc = head_block + off + slot * (D / 2) + ch * 16;
            cp_async16(dst + key * (D / 2) + ch * 16, kc, n);
            cp_async16(dst + kCodes + Src::v_off(key, ch), kc + page * (D / 2), n);
          }
          const uint8_t* ks = head_block + a_off + page * D + a_slot * (D / 16);
          const uint32_t n = a_ok ? D / 16 : 0;
          cp_async_small<D / 16>(dst + 2 * kCodes + lane * (D / 16), ks, n);
          cp_async_small<D / 16>(dst + 2 * kCodes + kScales + lane * (D / 16),
                                 ks + page * (D / 16), n);
        }
      }
    }
    cp_async_commit();
  };

  const int u0 = u_lo + warp;
  if (MODE) look_ahead(u0);
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    issue(u0 + i * kRowWarps, i, vmask[i]);
    if (MODE) look_ahead(u0 + (i + 1) * kRowWarps);
  }
  int stage = 0;
  for (int u = u0; u < u_hi; u += kRowWarps) {
    cp_async_wait<NST - 2>();
    __syncwarp();
    const uint32_t at = ring + stage * Src::kStageBytes;
    const uint32_t vm = vmask[0];
    float s[NG][2][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if constexpr (MODE == 0)
        src.scores(at, g, lane, s[g]);
      else
        src.scores(at + g * 8 * D, at + 2 * Src::kCodes + g * D, lane, s[g]);
    }
    // scores to log2 units, unseen keys to -inf
    const int j0 = MODE == 2 ? 0 : step_key<KS>(span, u);
    const bool whole = vm == 0xFFFFFFFFu &&
                       (MODE == 2 || (j0 + KS - 1 <= ti.t_min && j0 + KS <= ti.len &&
                                      (j0 > ti.t_max - p.window || j0 + KS <= p.sinks) &&
                                      (u >= span.sink_steps || j0 + KS <= span.sink_end)));
    uint32_t live = 0xFFFFFFFFu;  // keys whose values may be read
    if (whole) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][t][e] *= f_row[e >> 1];
    } else {
      if constexpr (MODE == 1) {
        const int j = j0 + lane;
        live = __ballot_sync(0xFFFFFFFFu, ((vm >> lane) & 1u) && span_holds(span, u, j, p.sinks));
      } else if constexpr (MODE == 2) {
        live = vm;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = 2 * c + (e & 1);
            const int key = 16 * g + (MODE == 0 ? 8 * t + n : group_key(t, n));
            bool see = (live >> key) & 1u;
            if constexpr (MODE != 2)
              see = see && span_holds(span, u, j0 + key, p.sinks) &&
                    sees(j0 + key, t_row[e >> 1], ti.len, p.window, p.sinks);
            s[g][t][e] = see ? s[g][t][e] * f_row[e >> 1] : neg_inf();
          }
    }
    // running maximum of the two rows
    float mx[2] = {st.m[0], st.m[1]};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[g][t][e]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
    }
    if (__any_sync(0xFFFFFFFFu, mx[0] > st.m[0] || mx[1] > st.m[1])) {
      const float a0 = mx[0] > st.m[0] ? ex2(st.m[0] - mx[0]) : 1.0f;
      const float a1 = mx[1] > st.m[1] ? ex2(st.m[1] - mx[1]) : 1.0f;
      st.m[0] = mx[0];
      st.m[1] = mx[1];
      st.l[0] *= a0;
      st.l[1] *= a1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        st.o[i][0] *= a0;
        st.o[i][1] *= a0;
        st.o[i][2] *= a1;
        st.o[i][3] *= a1;
      }
    }
    // a row that has seen nothing keeps its maximum at -inf: its weights are 2^-inf
    const float shift = MODE == 0 ? 0.0f : kProbShift;
    const float b0 = (st.m[0] == neg_inf() ? 0.0f : st.m[0]) - shift;
    const float b1 = (st.m[1] == neg_inf() ? 0.0f : st.m[1]) - shift;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t pf[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2(s[g][t][e] - (e < 2 ? b0 : b1));
          st.l[e >> 1] += w[e];
        }
        pf[2 * t] = MODE == 0 ? pack_bf16x2(w[0], w[1]) : pack_f16x2(w[0], w[1]);
        pf[2 * t + 1] = MODE == 0 ? pack_bf16x2(w[2], w[3]) : pack_f16x2(w[2], w[3]);
      }
      if constexpr (MODE == 0)
        src.values(at + Src::kRows, g, lane, pf, st);
      else
        src.values(at + Src::kCodes + g * 8 * D, at + 2 * Src::kCodes + Src::kScales + g * D, lane,
                   pf, live >> (16 * g), st);
    }
    __syncwarp();
    // the stage just read takes the step NST - 1 further on
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) vmask[i] = vmask[i + 1];
    const int nxt = u + (NST - 1) * kRowWarps;
    issue(nxt, stage == 0 ? NST - 1 : stage - 1, vmask[NST - 2]);
    if (MODE) look_ahead(nxt + kRowWarps);
    stage = stage + 1 == NST ? 0 : stage + 1;
  }
  cp_async_wait<0>();

  // ---------------------------------------------------------------- join the warps
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    st.l[h] += __shfl_xor_sync(0xFFFFFFFFu, st.l[h], 1);
    st.l[h] += __shfl_xor_sync(0xFFFFFFFFu, st.l[h], 2);
    if (c == 0) {
      sh_m[warp][r + 8 * h] = st.m[h];
      sh_l[warp][r + 8 * h] = st.l[h];
    }
  }
  __syncthreads();  // the ring is free from here on
  constexpr int kPad = D + 4;
  float* sh_o = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = r + 8 * h;
    float top = neg_inf();
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, sh_m[w][row]);
    const float f = st.m[h] == neg_inf() ? 0.0f : ex2(st.m[h] - top);
    float* orow = sh_o + (warp * kRowTile + row) * kPad;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      // a weight of zero times a sum that is NaN stays NaN: found below
      orow[Src::element(i, c, 0)] = st.o[i][2 * h] * f;
      orow[Src::element(i, c, 1)] = st.o[i][2 * h + 1] * f;
    }
  }
  __syncthreads();
  // eight threads a row, D/8 elements each
  constexpr int kPer = D / 8;
  const int row = threadIdx.x >> 3, part = threadIdx.x & 7;
  float top = neg_inf(), sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, sh_m[w][row]);
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w)
    sum += sh_m[w][row] == neg_inf() ? 0.0f * sh_l[w][row] : sh_l[w][row] * ex2(sh_m[w][row] - top);
  float o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    o[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w)
      o[i] += sh_o[(w * kRowTile + row) * kPad + part * kPer + i];
  }
  if constexpr (MODE == 0) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) bad |= o[i] != o[i];
    if (bad && row < ti.rows) atomicOr(&sh_nan, 1u << row);
    __syncthreads();
    if (sh_nan) {  // rows by the formula (see exact_row_keys)
      const int64_t stride = (int64_t)p.Hk * D;
      const int64_t first = ((int64_t)ti.b * p.T) * stride + (int64_t)ti.hk * D;
      for (int x = warp; x < ti.rows; x += kRowWarps) {
        if (!((sh_nan >> x) & 1u)) continue;
        const int t = ti.len - ti.q_len + (ti.row0 + x) / p.G;
        float m = neg_inf(), l = 0.0f, acc[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
        for (int u = u_lo; u < u_hi; ++u) {
          const int j0 = step_key<KS>(span, u);
          const int hi = min(j0 + KS, u < span.sink_steps ? span.sink_end : span.end);
          exact_row_keys<D>(p.q + out_row(p, ti, ti.row0 + x) * D, p.k + first, p.v + first, stride,
                            j0, hi, t, ti.len, p.window, p.sinks, p.scale_log2, lane, m, l, acc);
        }
#pragma unroll
        for (int e = 0; e < D / 32; ++e) sh_o[x * kPad + lane * (D / 32) + e] = acc[e];
        if (lane == 0) {
          sh_m[0][x] = m;
          sh_l[0][x] = l;
        }
      }
      __syncthreads();
      if ((sh_nan >> row) & 1u) {
        top = sh_m[0][row];
        sum = sh_l[0][row];
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = sh_o[row * kPad + part * kPer + i];
      }
    }
  }
  if (row >= ti.rows) return;
  if (MODE) top -= kProbShift;  // the weights' common factor
  if (p.splits > 1) {
    const int64_t at = (ti.part + row) * p.splits + split;
    float* po = p.part_o + at * D + part * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 4)
      *reinterpret_cast<float4*>(po + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    if (part == 0) p.part_ml[at] = make_float2(sum == 0.0f ? neg_inf() : top, sum);
    return;
  }
  const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
  const int64_t orow = out_row(p, ti, ti.row0 + row);
  uint32_t w[kPer / 2];
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) w[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
#pragma unroll
  for (int i = 0; i < kPer / 8; ++i)
    reinterpret_cast<uint4*>(p.out + orow * D + part * kPer)[i] =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  if (part == 0 && p.lse)
    p.lse[orow] = sum == 0.0f ? neg_inf() : (top + log2f(sum)) * 0.6931471805599453f;
}

// Joins the splits of a row: one warp per row, D/32 elements per lane.
template <int D>
__global__ void __launch_bounds__(128) k_attn_join(const __grid_constant__ RowsParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t rows = (int64_t)p.S * p.G;
  if (at >= (int64_t)p.B * p.Hk * rows) return;
  const int row = (int)(at % rows);
  const int64_t bh = at / rows;
  const int b = (int)(bh / p.Hk), hk = (int)(bh % p.Hk);
  if (row >= seq_len(p.q_lens, b, p.S) * p.G) return;
  const float2* ml = p.part_ml + at * p.splits;
  float top = neg_inf();
  for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, ml[s].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
  float o[E], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 v = ml[s];
    if (v.y == 0.0f) continue;
    const float f = ex2(v.x - top);
    sum = fmaf(v.y, f, sum);
    const float* po = p.part_o + (at * p.splits + s) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(po[e], f, o[e]);
  }
  const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
  const int64_t orow = ((int64_t)b * p.S + row / p.G) * p.H + hk * p.G + row % p.G;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0 && p.lse)
    p.lse[orow] = sum == 0.0f ? neg_inf() : (top + log2f(sum)) * 0.6931471805599453f;
}

namespace {

template <int D, int MODE>
cudaError_t launch(const RowsParams& p, cudaStream_t stream) {
  using Src = typename std::conditional<MODE == 0, Bf16Rows<D>, Cache4<D>>::type;
  const size_t ring = (size_t)kRowWarps * Src::kStages * Src::kStageBytes;
  const size_t join = (size_t)kRowWarps * kRowTile * (D + 4) * sizeof(float);
  const size_t smem = ring > join ? ring : join;
  cudaError_t e = cudaFuncSetAttribute(k_attn_rows<D, MODE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)p.B * p.Hk * p.tiles * p.splits;
  k_attn_rows<D, MODE><<<(unsigned)ctas, kRowWarps * 32, smem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)p.B * p.Hk * p.S * p.G;
  k_attn_join<D><<<(unsigned)((rows + 3) / 4), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace


cudaError_t launch_attn_rows(const RowsParams& p, int D, cudaStream_t stream) {
  const int mode = !p.pages ? 0 : (p.idx ? 2 : 1);
  if (D == 128)
    return mode == 0   ? launch<128, 0>(p, stream)
           : mode == 1 ? launch<128, 1>(p, stream)
                       : launch<128, 2>(p, stream);
  return mode == 0   ? launch<64, 0>(p, stream)
         : mode == 1 ? launch<64, 1>(p, stream)
                     : launch<64, 2>(p, stream);
}

}  // namespace si
