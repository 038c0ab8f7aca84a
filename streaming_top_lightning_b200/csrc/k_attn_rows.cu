// Attention of few query rows over a key/value cache: the decode form of the
// window attention (bf16 keys) and of the attention over a 4-bit paged cache.
//
//   o[row] = sum_j softmax_j(scale * q[row] . k[j]) v[j],  lse[row] = ln sum_j exp(...)
//
// over the keys the row's query sees (si_attn.cuh), or over the entries that a
// row of the indexer lists.  The G = H / H_k query heads of a kv head share its
// keys, so (query, head) pairs are the rows of a tile of 8, 16 or 32.
//
// What bounds it: a decode step reads every visible key once and multiplies it
// with few rows, so HBM does, and for 4-bit keys the instructions that turn
// codes into fp16 come near it.  One warp takes KS keys at a time from a ring
// of its own in shared memory (cp.async, no barrier between warps), the running
// maximum and sum stay in registers, and the warps of a CTA (and several CTAs,
// each with a chunk of the keys, unless there are tiles enough) share a
// sequence's keys.  A small call's CTAs, up to eight a tile, are clusters that
// join their results through one another's shared memory.  A large call's are
// one wave, each with an equal share of all tiles' steps, however ragged the
// sequences: a share begins and ends inside tiles, and k_attn_join joins the
// pieces of those.
//
// Keys are the M side of the products, rows the N side (mma.sync m16n8k16):
//   S^T = K Q^T,   O^T += V^T P^T
// so a tile can be as small as 8 rows, and a key's fragment, once built, serves
// all of the tile's rows.  S^T's fragments become P^T's by one 8 x 8
// transposition each (movmatrix).  tcgen05's 128 rows would be empty but for a
// few, and its operands would have to pass through shared memory as 16-bit
// numbers, four times the bytes of the 4-bit codes.
//
// 4-bit keys (E2M1 codes, an E4M3 scale per 16 elements): code x scale has six
// significant bits, so it is exact in fp16, and the products run in fp16 with
// fp32 accumulation.  A query row is scaled by a power of two into fp16's
// range (bf16 to fp16 drops no bit of an element within 2^-25 of the row's
// largest).  The dot product does not depend on the order of its terms, so a
// thread's fragment of a key row is simply D/8 consecutive bytes of codes: no
// shuffle, no transposition.  A value fragment pairs two keys for one element;
// taking the nibbles of two code words together gives the pairs without a
// transposition too.  Probabilities are rounded to fp16 after a scale of 2^10
// (2^-11 relative down to 2^-24 of the row's largest); the sum takes them
// unrounded.
//
// Measured on B200 (D = 128): 32 sequences, 32 heads on 8 kv heads, a window of
// 1,024 bf16 keys, 25.4 us, 5.3 TB/s; the same heads over ragged 4-bit caches of
// up to 8,192 keys, 55 us, 2.8 TB/s of the 6.6 that a copy reaches: the warps'
// instructions (about 800 for 32 keys: codes to fp16, products, transpositions)
// take 59 % of the issue slots and half of the ALUs' time.  Five CTAs an SM with
// two stages took 64 us, shares weighted by a CTA's start 60.  Tiles of 16 rows of
// 128 elements spill 96 to 224 bytes a thread at three CTAs an SM, 8-row tiles up to
// 24 at four, 32-row tiles 208 at 255 registers.
//
// bf16 keys: bf16 products, probabilities rounded to bf16 (2^-8).  The output is
// divided by the sum of the probabilities as rounded, so that a weight near one
// is not off by its rounding (of bf16's 2^-9 half steps the unrounded sum gave up
// to two: 0.0021 of the norm on one token of 300; 0.0017 being the output's own).
#include <cooperative_groups.h>

#include <type_traits>

#include "si_attn.cuh"

namespace cg = cooperative_groups;

namespace si {
namespace {

constexpr int kRowWarps = 4;
constexpr float kProbShift = 10.0f;  // 4-bit path: probabilities times 2^10

SI_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// What a warp holds of its tile while it walks over keys.  Accumulators and
// running values of n-tile x: the thread's rows are 8 x + 2 c and the next.
// l: the sum of the weights; lr: of the weights as rounded (bf16 keys).
template <int D, int NT>
struct RowState {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2], lr[NT][2];
};

// ------------------------------------------------------------ 4-bit pages
// Key order inside a group of 16: row 8 t + n of a fragment is this key.  A
// quad's pairs 2c, 2c+1 then are keys whose value rows lie in different banks,
// and so are the key rows that a quarter-warp reads.
SI_DEV int group_key(int t, int n) { return 8 * t + ((n & 1) ? 4 + ((n >> 1) ^ 1) : (n >> 1)); }

template <int D, int NT>
struct Cache4 {
  static constexpr int KS = 32;
  static constexpr int kStages = 3;
  static constexpr int kCodes = KS * D / 2, kScales = KS * D / 16;
  static constexpr int kStageBytes = 2 * kCodes + 2 * kScales;

  uint32_t qf[NT][D / 16][2];
  float row_factor[NT];  // of row 8 x + lane / 4

  // Byte of a value row's 16-byte chunk in its stage (a swizzle by key).
  static SI_DEV int v_off(int key, int chunk) {
    return key * (D / 2) + ((D == 128 ? chunk ^ (((key >> 1) & 1) << 1) : chunk) << 4);
  }

  // Fragments of n-tile x: the thread's row is 8 x + lane / 4.
  SI_DEV void load_q(int x, const uint16_t* qr, int lane) {
    const int c = lane & 3;
    uint32_t w[D / 8];  // D/4 elements of the row: D/4 * c ...
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = qr ? __ldg(reinterpret_cast<const uint4*>(qr + (D / 4) * c) + i)
                         : make_uint4(0, 0, 0, 0);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // 2^(10 - e) for a largest element in [2^e, 2^(e+1)); 1 for rows of zeros
    // or with an infinity, 2^126 at most
    const int e = (int)(__float_as_uint(top) >> 23);
    const int up = (e == 0 || e == 255) ? 0 : max(-126, min(126, 137 - e));
    const float f = __uint_as_float((uint32_t)(127 + up) << 23);
    row_factor[x] = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      qf[x][s][0] = pack_f16x2(bf16_lo(w[2 * s]) * f, bf16_hi(w[2 * s]) * f);
      qf[x][s][1] = pack_f16x2(bf16_lo(w[2 * s + 1]) * f, bf16_hi(w[2 * s + 1]) * f);
    }
  }

  // Scores of 16 keys from a stage: s[x][t] are the keys group_key(t, lane / 4)
  // against the rows 8 x + 2 c + (0, 1), [2 t] and [2 t + 1].
  SI_DEV void scores(uint32_t kc, uint32_t ks, int lane, float (&s)[NT][4]) const {
    const int r = lane >> 2, c = lane & 3;
    uint32_t w[2][D / 32], slo[2], shi[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int key = group_key(t, r);
      uint32_t sc;
      if constexpr (D == 128) {
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[t][0]), "=r"(w[t][1]), "=r"(w[t][2]), "=r"(w[t][3])
                     : "r"(kc + key * 64 + c * 16));
        asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                     : "=r"(sc)
                     : "r"(ks + key * 8 + c * 2));
      } else {
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                     : "=r"(w[t][0]), "=r"(w[t][1])
                     : "r"(kc + key * 32 + c * 8));
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sc) : "r"(ks + key * 4 + c));
      }
      const uint32_t s2 = e4m3x2(sc);
      slo[t] = __byte_perm(s2, 0, 0x1010);
      shi[t] = __byte_perm(s2, 0, 0x3232);
    }
#pragma unroll
    for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t f0 = (D == 128 && i >= 2) ? shi[0] : slo[0];
      const uint32_t f1 = (D == 128 && i >= 2) ? shi[1] : slo[1];
      uint32_t a[4] = {hmul2(e2m1x2<0>(w[0][i]), f0), hmul2(e2m1x2<0>(w[1][i]), f1),
                       hmul2(e2m1x2<1>(w[0][i]), f0), hmul2(e2m1x2<1>(w[1][i]), f1)};
#pragma unroll
      for (int x = 0; x < NT; ++x) mma_f16(s[x], a, qf[x][2 * i][0], qf[x][2 * i][1]);
      uint32_t b[4] = {hmul2(e2m1x2<2>(w[0][i]), f0), hmul2(e2m1x2<2>(w[1][i]), f1),
                       hmul2(e2m1x2<3>(w[0][i]), f0), hmul2(e2m1x2<3>(w[1][i]), f1)};
#pragma unroll
      for (int x = 0; x < NT; ++x) mma_f16(s[x], b, qf[x][2 * i + 1][0], qf[x][2 * i + 1][1]);
    }
  }

  // O^T += V^T P^T over 16 keys; MASKED: `live` says which keys of the group may
  // be read (the others' codes count as zero).
  template <bool MASKED>
  SI_DEV void values(uint32_t vc, uint32_t vs, int lane, const uint32_t (&pf)[NT][2], uint32_t live,
                     RowState<D, NT>& st) const {
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
        if (MASKED && !((live >> key) & 1u)) b[i] = 0u;
      }
      sp[t] = e4m3x2(__byte_perm(b[0], b[1], 0x0040));
    }
#pragma unroll
    for (int y = 0; y < D / 64; ++y) {
      // even elements of both keys of a pair in the bytes of lo, odd ones in hi
      uint32_t lo[2], hi[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t a = w[2 * t][y], b = w[2 * t + 1][y];
        lo[t] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
        hi[t] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
      }
#define SI_PV(BYTE)                                                                             \
  {                                                                                             \
    uint32_t a[4] = {hmul2(e2m1x2<BYTE>(lo[0]), sp[0]), hmul2(e2m1x2<BYTE>(hi[0]), sp[0]),      \
                     hmul2(e2m1x2<BYTE>(lo[1]), sp[1]), hmul2(e2m1x2<BYTE>(hi[1]), sp[1])};     \
    _Pragma("unroll") for (int x = 0; x < NT; ++x)                                              \
        mma_f16(st.o[x][4 * y + BYTE], a, pf[x][0], pf[x][1]);                                  \
  }
      SI_PV(0)
      SI_PV(1)
      SI_PV(2)
      SI_PV(3)
#undef SI_PV
    }
  }

  // Element of the row that accumulator o[.][i] row half h of a thread is.
  static SI_DEV int element(int i, int r, int h) { return (D / 8) * r + 2 * i + h; }
};

// ------------------------------------------------------------ bf16 rows
template <int D, int NT>
struct Bf16Rows {
  static constexpr int KS = D == 128 ? 16 : 32;
  static constexpr int kStages = 3;
  static constexpr int kRows = KS * D * 2;
  static constexpr int kStageBytes = 2 * kRows;

  uint32_t qf[NT][D / 16][2];
  float row_factor[NT];

  static SI_DEV int off(int key, int chunk) {
    return key * (D * 2) + ((chunk ^ (key & 7)) << 4);
  }

  SI_DEV void load_q(int x, const uint16_t* qr, int lane) {
    const int c = lane & 3;
    row_factor[x] = 1.0f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      qf[x][s][0] = qr ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 2 * c)) : 0u;
      qf[x][s][1] = qr ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 8 + 2 * c)) : 0u;
    }
  }

  SI_DEV void scores(uint32_t kb, int g, int lane, float (&s)[NT][4]) const {
#pragma unroll
    for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.0f;
    const int key = 16 * g + (lane & 15);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      ldmatrix4(a, kb + off(key, 2 * i + (lane >> 4)));
#pragma unroll
      for (int x = 0; x < NT; ++x) mma_bf16(s[x], a, qf[x][i][0], qf[x][i][1]);
    }
  }

  SI_DEV void values(uint32_t vb, int g, int lane, const uint32_t (&pf)[NT][2],
                     RowState<D, NT>& st) const {
    // matrices: keys 0-7 and elements 0-7, then 8-15; keys 8-15 the same
    const int key = 16 * g + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      ldmatrix4_t(a, vb + off(key, 2 * i + ((lane >> 3) & 1)));
#pragma unroll
      for (int x = 0; x < NT; ++x) mma_bf16(st.o[x][i], a, pf[x][0], pf[x][1]);
    }
  }

  static SI_DEV int element(int i, int r, int h) { return 16 * i + r + 8 * h; }
};

// exact_row_keys for the keys [s_lo, s_hi) and [w_lo, w_hi) of a row's sequence in
// 4-bit pages; the results to out [D] and ml.  (A call: inline, drafted tokens
// took 10.8 us for 10.3.)
template <int D>
__device__ __noinline__ void exact_row_pages(const uint16_t* qr, const int32_t* table,
                                             const uint8_t* head, int64_t page_bytes, int n_pages,
                                             int page_shift, int s_lo, int s_hi, int w_lo, int w_hi,
                                             int t, int len, int window, int sinks,
                                             float scale_log2, float* out, float2* ml) {
  const int page = 1 << page_shift, lane = threadIdx.x & 31;
  const uint2 qw = value_bits<D>(qr, lane);
  float m = neg_inf(), l = 0.0f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.0f;
  // The lane's elements of a row from its codes and scale.  An E2M1 number's lower
  // bits are the fp16 number 2^-14 of it.
  auto numbers = [&](const uint8_t* codes, const uint8_t* scales, float (&x)[D / 32]) {
    const uint32_t c = D == 128 ? (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(codes) + lane)
                                : (uint32_t)__ldg(codes + lane);
    const float f = __half2float(__ushort_as_half(
                        (uint16_t)e4m3x2((uint32_t)__ldg(scales + lane * (D / 32) / 16)))) *
                    16384.0f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const uint32_t n = c >> (4 * e);
      x[e] = __half2float(__ushort_as_half((uint16_t)((n & 7u) << 9 | (n & 8u) << 12))) * f;
    }
  };
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int j_hi = part ? w_hi : s_hi;
#pragma unroll 1
    for (int j0 = part ? w_lo : s_lo; j0 < j_hi; j0 += 4) {
      float dot[4], v[4][D / 32];
      bool see[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int j = j0 + x;
        see[x] = j < j_hi && sees(j, t, len, window, sinks);
        const int pg = see[x] ? __ldg(table + (j >> page_shift)) : -1;
        see[x] = see[x] && pg >= 0 && pg < n_pages;
        const int slot = see[x] ? j & (page - 1) : 0;
        const uint8_t* kc = head + (int64_t)(see[x] ? pg : 0) * page_bytes + slot * (D / 2);
        const uint8_t* ks = kc - slot * (D / 2) + page * D + slot * (D / 16);
        float k[D / 32];
        numbers(kc, ks, k);
        numbers(kc + page * (D / 2), ks + page * (D / 16), v[x]);
        dot[x] = bf16_lo(qw.x) * k[0] + bf16_hi(qw.x) * k[1];
        if constexpr (D == 128) dot[x] += bf16_lo(qw.y) * k[2] + bf16_hi(qw.y) * k[3];
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1)
#pragma unroll
        for (int x = 0; x < 4; ++x) dot[x] += __shfl_xor_sync(0xFFFFFFFFu, dot[x], i);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (see[x]) exact_key<D>(dot[x] * scale_log2, v[x], m, l, o);
    }
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) out[lane * (D / 32) + e] = o[e];
  if (lane == 0) *ml = make_float2(m, l);
}

// MODE 0: bf16 keys; 1: 4-bit pages; 2: 4-bit pages, listed entries.
template <int D, int MODE, int NT>
using Source = typename std::conditional<MODE == 0, Bf16Rows<D, NT>, Cache4<D, NT>>::type;

// Steps of a (batch, tile) pair: the same for each kv head.
template <int RT, int KS>
SI_DEV int pair_steps(const RowsParams& p, int pair) {
  Tile ti;
  const int b = pair / p.tiles;
  if (!find_tile<RT>(p, (uint32_t)(b * p.Hk * p.tiles + pair % p.tiles), ti)) return 0;
  return tile_span<KS>(p, ti).steps;
}

// A CTA's share of all work, which stands in a row: (batch, tile), kv head,
// and in a tile first kTileCost for beginning it and joining its warps, then
// its steps.  at: the next one's place; left: how much; off: its place in its
// tile.
template <int KS>
constexpr int kTileCost = 256 / KS;
struct Share {
  int64_t at, share, left;
  int pair, hk, off;
};

// Sum and exclusive prefix sum over the CTA's 128 threads.
SI_DEV int64_t scan128(int64_t v, int64_t* total) {
  __shared__ int64_t sh[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < warp) before += sh[i];
    all += sh[i];
  }
  *total = all;
  return before + x - v;
}

// The share of this CTA (in shared memory): the steps of all tiles in equal
// parts, found from the lengths by every CTA for itself.  False: there is none.
template <int RT, int KS>
SI_DEV bool share_of(const RowsParams& p, Share& job) {
  const int pairs = p.B * p.tiles, per = (pairs + 127) / 128;
  const int lo = min(pairs, (int)threadIdx.x * per), hi = min(pairs, lo + per);
  int64_t mine = 0, total;
  auto cost = [&](int i) {
    const int n = pair_steps<RT, KS>(p, i);
    return n ? n + kTileCost<KS> : 0;
  };
  for (int i = lo; i < hi; ++i) mine += cost(i);
  const int64_t before = scan128(mine, &total) * p.Hk;
  total *= p.Hk;
  const int64_t share =
      max((total + gridDim.x - 1) / gridDim.x, (int64_t)(p.chunk_keys / KS));
  const int64_t at = blockIdx.x * share;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.share_out = share;
  if (at >= total) return false;
  if (at >= before && at < before + mine * p.Hk) {  // one thread's tiles hold its beginning
    int64_t x = before;
    for (int i = lo; i < hi; ++i) {
      const int n = cost(i);
      if (at < x + (int64_t)n * p.Hk) {
        job = Share{at, share, min(share, total - at), i, (int)((at - x) / n), (int)((at - x) % n)};
        break;
      }
      x += (int64_t)n * p.Hk;
    }
  }
  __syncthreads();
  return true;
}

// Dynamic shared memory of a CTA: its warps' rings, or the join of the warps.
template <int D, int MODE, int NT>
constexpr size_t row_smem() {
  constexpr size_t ring = (size_t)kRowWarps * Source<D, MODE, NT>::kStages *
                          Source<D, MODE, NT>::kStageBytes;
  constexpr size_t join = (size_t)kRowWarps * 8 * NT * (D + 4) * sizeof(float);
  return ring > join ? ring : join;
}

// CTAs that an SM holds: of those that its registers do, as many as its 228 KB
// of shared memory do (a CTA has 1 KB of the system's and its static arrays
// besides: up to three numbers a warp and row, and 256 bytes).  bf16 rings of 96
// KB leave room for two.
template <int D, int MODE, int NT>
constexpr int row_ctas() {
  constexpr int regs = NT == 1 ? 4 : (NT == 2 ? 3 : 2);
  constexpr int smem =
      (int)(228 * 1024 / (row_smem<D, MODE, NT>() + 1024 + 12 * kRowWarps * 8 * NT + 256));
  return regs < smem ? regs : smem;
}

}  // namespace

// MANY: calls of several queries a sequence, whose tiles' rows may see different
// keys (bf16 keys: every call).  Over 4-bit pages a decode batch takes 55.7 us with
// the code for that and 54.7 without.
template <int D, int MODE, int NT, bool MANY>
__global__ void __launch_bounds__(kRowWarps * 32, row_ctas<D, MODE, NT>())
    k_attn_rows(const __grid_constant__ RowsParams p) {
  using Src = Source<D, MODE, NT>;
  constexpr int KS = Src::KS, NST = Src::kStages, NG = KS / 16, RT = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sh_m[kRowWarps][RT], sh_l[kRowWarps][RT];
  __shared__ float sh_lr[kRowWarps][MODE == 0 ? RT : 1];
  __shared__ uint32_t sh_nan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  Tile ti;
  KeySpan span;
  int u_lo, u_hi, split;
  __shared__ Share job;
  if (p.share == kShared) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join, see launch_join
    if (!share_of<RT, KS>(p, job)) return;
  } else {
    const uint32_t tile = blockIdx.x / (uint32_t)p.splits;
    split = (int)(blockIdx.x - tile * (uint32_t)p.splits);
    if (!find_tile<RT>(p, tile, ti)) return;
    // a sequence without keys still has rows to write
    span = tile_span<KS>(p, ti);
    u_lo = split * p.chunk_keys / KS;
    u_hi = split + 1 == p.splits ? span.steps : min(span.steps, (split + 1) * p.chunk_keys / KS);
  }
  for (;;) {
  if (p.share == kShared) {
    // the next piece of this CTA's steps
    const int at_tile = job.pair % p.tiles;
    find_tile<RT>(p, (uint32_t)((job.pair / p.tiles * p.Hk + job.hk) * p.tiles + at_tile), ti);
    span = tile_span<KS>(p, ti);
    u_lo = max(0, job.off - kTileCost<KS>);
    u_hi = (int)min((int64_t)span.steps, job.off - kTileCost<KS> + job.left);
    const int64_t start = job.at - job.off + kTileCost<KS>;  // where the tile's steps begin
    split = (int)(blockIdx.x - start / job.share);
    if (threadIdx.x == 0 && u_lo == 0 && u_hi > 0)
      p.tile_start[(int64_t)(ti.b * p.Hk + ti.hk) * p.tiles + at_tile] = start;
    if (u_hi <= u_lo) return;  // the share ends before the tile's first step
  }
  if (threadIdx.x == 0) sh_nan = 0u;

  Src src;
  float f_row[NT][2];  // scale of the thread's score columns
#pragma unroll
  for (int x = 0; x < NT; ++x) {
    const int row = 8 * x + r;
    src.load_q(x, row < ti.rows ? p.q + out_row(p, ti, ti.row0 + row) * D : nullptr, lane);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      f_row[x][e] = __shfl_sync(0xFFFFFFFFu, src.row_factor[x], 8 * c + 4 * e) * p.scale_log2;
  }

  RowState<D, NT> st;
#pragma unroll
  for (int x = 0; x < NT; ++x) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      st.o[x][i][0] = st.o[x][i][1] = st.o[x][i][2] = st.o[x][i][3] = 0.0f;
    st.m[x][0] = st.m[x][1] = neg_inf();
    st.l[x][0] = st.l[x][1] = st.lr[x][0] = st.lr[x][1] = 0.0f;
  }

  const uint32_t ring = smem_u32(smem) + warp * NST * Src::kStageBytes;
  uint32_t vmask[NST];  // keys of a stage that lie in a page
#pragma unroll
  for (int i = 0; i < NST; ++i) vmask[i] = 0u;

  // What the next step to be loaded needs from memory first, read ahead and not
  // looked at before the step is loaded: its pages (MODE 1), or its entries'
  // pages (MODE 2, whose entries are read another step ahead).
  int ahead[NG];             // MODE 1: page of each group of 16 keys
  int e_now = -1, e_next = -1, pg_now = -1;  // MODE 2: this lane's entry and page
  const int32_t* table = MODE ? p.table + (int64_t)ti.b * p.width : nullptr;
  const int32_t* irow =
      MODE == 2 ? p.idx + ((int64_t)ti.b * p.S + ti.row0 / p.G) * p.topk : nullptr;
  auto entry = [&](int u) {
    const int e = u * KS + lane;
    return u < u_hi && e < p.topk ? __ldg(irow + e) : -1;
  };
  auto look_ahead = [&](int u) {
    if constexpr (MODE == 1) {
      const int j0 = step_key<KS>(span, u);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int j = j0 + 16 * g;
        const bool in = u < u_hi && j < (u < span.sink_steps ? span.sink_end : span.end) &&
                        (j + 16 > span.lo || j < p.sinks);
        ahead[g] = in ? __ldg(table + (j >> p.page_shift)) : -1;
      }
    } else if constexpr (MODE == 2) {
      e_now = e_next;
      e_next = entry(u + kRowWarps);
      pg_now = e_now >= 0 && e_now < ti.len ? __ldg(table + (e_now >> p.page_shift)) : -1;
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
            const bool ok = pg >= 0 && pg < p.n_pages;
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
          const bool a_ok = pg_now >= 0 && pg_now < p.n_pages;
          const int64_t a_off = (int64_t)(a_ok ? pg_now : 0) * p.page_bytes;
          const int a_slot = a_ok ? e_now & (page - 1) : 0;
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

  // One step from a stage: scores, running maximum, weights, values.
  auto step = [&](auto masked, int u, uint32_t at, uint32_t vm) {
    constexpr bool MASKED = decltype(masked)::value;
    float s[NG][NT][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if constexpr (MODE == 0)
        src.scores(at, g, lane, s[g]);
      else
        src.scores(at + g * 8 * D, at + 2 * Src::kCodes + g * D, lane, s[g]);
    }
    uint32_t live = 0xFFFFFFFFu;  // keys whose values may be read
    const int j0 = MASKED && MODE != 2 ? step_key<KS>(span, u) : 0;
    if constexpr (MASKED && MODE == 1)
      live = __ballot_sync(0xFFFFFFFFu,
                           ((vm >> lane) & 1u) && span_holds(span, u, j0 + lane, p.sinks));
    if constexpr (MASKED && MODE == 2) live = vm;
    // scores to log2 units, unseen keys to -inf
    float mx[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      mx[x][0] = st.m[x][0];
      mx[x][1] = st.m[x][1];
      int t_row[2] = {0, 0};
      if constexpr (MASKED && MODE != 2)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          t_row[e] = ti.len - ti.q_len + (ti.row0 + min(8 * x + 2 * c + e, ti.rows - 1)) / p.G;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[g][x][e] * f_row[x][e & 1];
          if constexpr (MASKED) {
            const int key = 16 * g + (MODE == 0 ? 8 * (e >> 1) + r : group_key(e >> 1, r));
            bool see = (live >> key) & 1u;
            if constexpr (MODE != 2)
              see = see && span_holds(span, u, j0 + key, p.sinks) &&
                    sees(j0 + key, t_row[e & 1], ti.len, p.window, p.sinks);
            v = see ? v : neg_inf();
          }
          s[g][x][e] = v;
          mx[x][e & 1] = fmaxf(mx[x][e & 1], v);
        }
    }
    bool grown = false;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          mx[x][e] = fmaxf(mx[x][e], __shfl_xor_sync(0xFFFFFFFFu, mx[x][e], o));
        grown |= mx[x][e] > st.m[x][e];
      }
    if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          a[e] = mx[x][e] > st.m[x][e] ? ex2(st.m[x][e] - mx[x][e]) : 1.0f;
          st.m[x][e] = mx[x][e];
          st.l[x][e] *= a[e];
          if (MODE == 0) st.lr[x][e] *= a[e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[x][i][0] *= a[0];
          st.o[x][i][1] *= a[1];
          st.o[x][i][2] *= a[0];
          st.o[x][i][3] *= a[1];
        }
      }
    }
    // a row that has seen nothing keeps its maximum at -inf: its weights are 2^-inf
    const float shift = MODE == 0 ? 0.0f : kProbShift;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t pf[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const float b0 = (st.m[x][0] == neg_inf() ? 0.0f : st.m[x][0]) - shift;
        const float b1 = (st.m[x][1] == neg_inf() ? 0.0f : st.m[x][1]) - shift;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float w0 = ex2(s[g][x][2 * t] - b0), w1 = ex2(s[g][x][2 * t + 1] - b1);
          st.l[x][0] += w0;
          st.l[x][1] += w1;
          const uint32_t both = MODE == 0 ? pack_bf16x2(w0, w1) : pack_f16x2(w0, w1);
          if (MODE == 0) {
            st.lr[x][0] += bf16_lo(both);
            st.lr[x][1] += bf16_hi(both);
          }
          pf[x][t] = transpose8x8(both);
        }
      }
      if constexpr (MODE == 0)
        src.values(at + Src::kRows, g, lane, pf, st);
      else
        src.template values<MASKED>(at + Src::kCodes + g * 8 * D,
                                    at + 2 * Src::kCodes + Src::kScales + g * D, lane, pf,
                                    live >> (16 * g), st);
    }
  };

  const int u0 = u_lo + warp;
  if (MODE == 2) e_next = entry(u0);
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
    bool whole = vm == 0xFFFFFFFFu;  // every row sees every key of the step
    if (MODE != 2) {
      const int j0 = step_key<KS>(span, u);
      whole = whole && j0 + KS - 1 <= ti.t_min && j0 + KS <= ti.len &&
              (j0 > ti.t_max - p.window || j0 + KS <= p.sinks) &&
              (u >= span.sink_steps || j0 + KS <= span.sink_end);
    }
    if (whole)
      step(std::false_type{}, u, at, vm);
    else
      step(std::true_type{}, u, at, vm);
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
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        st.l[x][e] += __shfl_xor_sync(0xFFFFFFFFu, st.l[x][e], o);
      if (MODE == 0)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          st.lr[x][e] += __shfl_xor_sync(0xFFFFFFFFu, st.lr[x][e], o);
      if (r == 0) {
        sh_m[warp][8 * x + 2 * c + e] = st.m[x][e];
        sh_l[warp][8 * x + 2 * c + e] = st.l[x][e];
        if (MODE == 0) sh_lr[warp][8 * x + 2 * c + e] = st.lr[x][e];
      }
    }
  __syncthreads();  // the ring is free from here on
  constexpr int kPad = D + 4;
  float* sh_o = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * x + 2 * c + e;
      float top = neg_inf();
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, sh_m[w][row]);
      const float f = st.m[x][e] == neg_inf() ? 0.0f : ex2(st.m[x][e] - top);
      float* orow = sh_o + (warp * RT + row) * kPad;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // a weight of zero times a sum that is NaN stays NaN: found below
        orow[Src::element(i, r, 0)] = st.o[x][i][e] * f;
        orow[Src::element(i, r, 1)] = st.o[x][i][2 + e] * f;
      }
    }
  __syncthreads();
  // 128 / RT threads a row
  constexpr int kParts = kRowWarps * 32 / RT, kPer = D / kParts;
  const int row = threadIdx.x / kParts, part = threadIdx.x % kParts;
  // rsum: of the weights as rounded
  float top = neg_inf(), sum = 0.0f, rsum = 0.0f;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, sh_m[w][row]);
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    const float f = sh_m[w][row] == neg_inf() ? 0.0f : ex2(sh_m[w][row] - top);
    sum = fmaf(sh_l[w][row], f, sum);
    if (MODE == 0) rsum = fmaf(sh_lr[w][row], f, rsum);
  }
  float o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    o[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) o[i] += sh_o[(w * RT + row) * kPad + part * kPer + i];
  }
  if constexpr (MODE == 0) {
    // the values' mean is that over the weights as rounded; sum is what the other
    // chunks and lse take
    const float fit = sum == 0.0f ? 0.0f : __fdividef(sum, rsum);
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] *= fit;
  }
  // Rows that are NaN by a value that they do not see, by the formula (si_attn.cuh).
  // Rows of one query see the same keys; where the sum is NaN too, a score that the
  // row sees is.
  if (MANY && ti.t_min != ti.t_max) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) bad |= o[i] != o[i];
    if (bad && row < ti.rows && sum == sum) atomicOr(&sh_nan, 1u << row);
    __syncthreads();
    if (sh_nan) {
      // the keys that the steps have brought
      const int u_w = max(u_lo, span.sink_steps), ss = span.sink_steps;
      const int w_lo = step_key<KS>(span, u_w), w_hi = min(span.end, step_key<KS>(span, max(u_hi, ss)));
      const int s_lo = min(u_lo, ss) * KS, s_hi = min(span.sink_end, min(u_hi, ss) * KS);
      for (int x = warp; x < ti.rows; x += kRowWarps) {
        if (!((sh_nan >> x) & 1u)) continue;
        const int t = ti.len - ti.q_len + (ti.row0 + x) / p.G;
        const uint16_t* qr = p.q + out_row(p, ti, ti.row0 + x) * D;
        if constexpr (MODE == 1) {
          exact_row_pages<D>(qr, p.table + (int64_t)ti.b * p.width,
                             p.pages + (int64_t)ti.hk * cache4_block<D>(page), p.page_bytes, p.n_pages, p.page_shift, s_lo,
                             s_hi, w_lo, w_hi, t, ti.len, p.window, p.sinks, p.scale_log2,
                             sh_o + x * kPad, reinterpret_cast<float2*>(sh_o + x * kPad + D));
        } else {
          const int64_t stride = (int64_t)p.Hk * D;
          const int64_t first = ((int64_t)ti.b * p.T) * stride + (int64_t)ti.hk * D;
          uint32_t nans = 0u;
          if (unseen_bad<D>(p.v + first, stride, max(w_lo, span.lo), w_hi, t, p.window, p.sinks,
                            lane) ||
              unseen_bad<D>(p.v + first, stride, s_lo, s_hi, t, p.window, p.sinks, lane)) {
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
              float y = 0.0f;
#pragma unroll
              for (int w = 0; w < kRowWarps; ++w)
                y += sh_o[(w * RT + x) * kPad + lane * (D / 32) + e];
              nans |= (uint32_t)(y != y) << e;
            }
            nans = unexplained<D>(p.v + first, stride, w_lo, w_hi, t, ti.len, p.window, p.sinks,
                                  lane, nans);
            nans = unexplained<D>(p.v + first, stride, s_lo, s_hi, t, ti.len, p.window, p.sinks,
                                  lane, nans);
          }
          if (!__any_sync(0xFFFFFFFFu, nans != 0u)) {
            if (lane == 0) atomicAnd(&sh_nan, ~(1u << x));
            continue;
          }
          float m = neg_inf(), l = 0.0f, acc[D / 32];
#pragma unroll
          for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
          exact_row_keys<D>(qr, p.k + first, p.v + first, stride, s_lo, s_hi, t, ti.len, p.window,
                            p.sinks, p.scale_log2, lane, m, l, acc);
          exact_row_keys<D>(qr, p.k + first, p.v + first, stride, w_lo, w_hi, t, ti.len, p.window,
                            p.sinks, p.scale_log2, lane, m, l, acc);
#pragma unroll
          for (int e = 0; e < D / 32; ++e) sh_o[x * kPad + lane * (D / 32) + e] = acc[e];
          if (lane == 0) *reinterpret_cast<float2*>(sh_o + x * kPad + D) = make_float2(m, l);
        }
      }
      __syncthreads();
      if ((sh_nan >> row) & 1u) {
        // in the weights' units, 2^kProbShift over 4-bit pages
        const float unit = MODE == 1 ? 1024.0f : 1.0f;
        top = sh_o[row * kPad + D];
        sum = sh_o[row * kPad + D + 1] * unit;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = sh_o[row * kPad + part * kPer + i] * unit;
      }
    }
  }
  if (MODE) top -= kProbShift;  // the weights' common factor
  if (p.share == kCluster) {
    // the chunks' CTAs are one cluster: each joins the rows that its rank gives
    cg::cluster_group cl = cg::this_cluster();
    __syncthreads();  // everyone is done with sh_o
    float* mine = sh_o + row * D + part * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 4)
      *reinterpret_cast<float4*>(mine + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    if (part == 0) {
      sh_m[0][row] = sum == 0.0f ? neg_inf() : top;
      sh_l[0][row] = sum;
    }
    cl.sync();
    for (int x = split + warp * p.splits; x < ti.rows; x += kRowWarps * p.splits) {
      float all = neg_inf(), tot = 0.0f, acc[D / 32];
      for (int s = 0; s < p.splits; ++s) all = fmaxf(all, *cl.map_shared_rank(&sh_m[0][x], s));
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
#pragma unroll 2
      for (int s = 0; s < p.splits; ++s) {
        const float l = *cl.map_shared_rank(&sh_l[0][x], s);
        const float f = l == 0.0f ? 0.0f : ex2(*cl.map_shared_rank(&sh_m[0][x], s) - all);
        tot = fmaf(l, f, tot);
        const float* po = cl.map_shared_rank(sh_o + x * D + lane * (D / 32), s);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(po[e], f, acc[e]);
      }
      const float inv = tot == 0.0f ? 0.0f : p.v_scale / tot;
      const int64_t orow = out_row(p, ti, ti.row0 + x);
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * (D / 64);
#pragma unroll
      for (int e = 0; e < D / 64; ++e)
        dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      if (lane == 0 && p.lse)
        p.lse[orow] = tot == 0.0f ? neg_inf() : (all + log2f(tot)) * 0.6931471805599453f;
    }
    cl.sync();  // nobody leaves while its results are read
    return;
  }
  if (row < ti.rows) {
    if (p.share == kShared && (u_lo > 0 || u_hi < span.steps)) {
      // (a tile has at most p.splits pieces: a share is at least chunk_keys)
      const int64_t at = (ti.part + row) * p.splits + split;
      float* po = p.part_o + at * D + part * kPer;
#pragma unroll
      for (int i = 0; i < kPer; i += 4)
        *reinterpret_cast<float4*>(po + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      if (part == 0) p.part_ml[at] = make_float2(sum == 0.0f ? neg_inf() : top, sum);
    } else {
      const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
      const int64_t orow = out_row(p, ti, ti.row0 + row);
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D + part * kPer);
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i)
        reinterpret_cast<uint2*>(dst)[i] =
            make_uint2(pack_bf16x2(o[4 * i] * inv, o[4 * i + 1] * inv),
                       pack_bf16x2(o[4 * i + 2] * inv, o[4 * i + 3] * inv));
      if (part == 0 && p.lse)
        p.lse[orow] = sum == 0.0f ? neg_inf() : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
  if (p.share != kShared) return;
  __syncthreads();  // everyone is done with the join's shared memory and this piece
  if (threadIdx.x == 0) {
    const int done = u_hi + kTileCost<KS> - job.off;
    job.left -= done;
    job.at += done;
    // on to the next kv head, or the next tile with keys
    job.off = 0;
    if (++job.hk == p.Hk) {
      job.hk = 0;
      do {
        ++job.pair;
      } while (job.pair < p.B * p.tiles && pair_steps<RT, KS>(p, job.pair) == 0);
      if (job.pair == p.B * p.tiles) job.left = 0;
    }
  }
  __syncthreads();
  if (job.left <= 0) return;
  }
}

// Joins the chunks of a row: W warps per row (1 for few chunks, 4 for many),
// D/32 elements a lane.
template <int D, int KS, int RT, int W, bool SHARED>
__global__ void __launch_bounds__(128) k_attn_join(const __grid_constant__ RowsParams p) {
  constexpr int E = D / 32;
  __shared__ float sh_o[4][D], sh_l[4], sh_top[4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rows = (uint32_t)(p.S * p.G), at32 = W == 1 ? blockIdx.x * 4 + warp : blockIdx.x;
  if (at32 >= (uint32_t)(p.B * p.Hk) * rows) return;  // B*S*H < 2^31
  const int64_t at = at32;
  const uint32_t bh = at32 / rows;
  const int row = (int)(at32 - bh * rows);
  // the row's tile, for the chunks that its keys filled
  Tile ti;
  int tile;
  if (p.idx) {
    const int per = (p.G + RT - 1) / RT;
    tile = row / p.G * per + row % p.G / RT;
  } else {
    tile = row / RT;
  }
  if (!find_tile<RT>(p, bh * (uint32_t)p.tiles + tile, ti) || row >= ti.row0 + ti.rows) return;
  const int steps = tile_span<KS>(p, ti).steps;
  int n;
  if constexpr (SHARED) {
    n = 0;
    if (steps > 0) {
      // the CTAs that had a part of the tile; one alone has written the rows
      const int64_t start = p.tile_start[(int64_t)bh * p.tiles + tile], share = *p.share_out;
      n = (int)((start + steps - 1) / share - start / share) + 1;
      if (n == 1) return;
    }
  } else {
    n = min(p.splits, (steps * KS + p.chunk_keys - 1) / p.chunk_keys);
  }
  const float2* ml = p.part_ml + at * p.splits;
  const int s0 = W == 1 ? 0 : warp;
  float top = neg_inf();
  for (int s = s0 + W * lane; s < n; s += W * 32) top = fmaxf(top, ml[s].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
  if constexpr (W > 1) {
    if (lane == 0) sh_top[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(sh_top[0], sh_top[1]), fmaxf(sh_top[2], sh_top[3]));
  }
  float o[E], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
  for (int s = s0; s < n; s += W) {
    const float2 v = ml[s];
    const float f = v.y == 0.0f ? 0.0f : ex2(v.x - top);
    sum = fmaf(v.y, f, sum);
    const float* po = p.part_o + (at * p.splits + s) * D + lane * E;
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(po);
      o[0] = fmaf(x.x, f, o[0]), o[1] = fmaf(x.y, f, o[1]);
      o[2] = fmaf(x.z, f, o[2]), o[3] = fmaf(x.w, f, o[3]);
    } else {
      const float2 x = *reinterpret_cast<const float2*>(po);
      o[0] = fmaf(x.x, f, o[0]), o[1] = fmaf(x.y, f, o[1]);
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) sh_o[warp][lane * E + e] = o[e];
    if (lane == 0) sh_l[warp] = sum;
    __syncthreads();
    if (warp) return;
    sum = (sh_l[0] + sh_l[1]) + (sh_l[2] + sh_l[3]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane * E + e;
      o[e] = (sh_o[0][d] + sh_o[1][d]) + (sh_o[2][d] + sh_o[3][d]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
  const int64_t orow = out_row(p, ti, row);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0 && p.lse)
    p.lse[orow] = sum == 0.0f ? neg_inf() : (top + log2f(sum)) * 0.6931471805599453f;
}

namespace {

// Up to 24 chunks a warp takes a row, beyond that four.  (500 ragged sequences
// of up to 1,024 keys, few pieces each: 62.9 us with one warp, 75 with four; one
// sequence of 131,072 keys: 47.2 and 29.1.)  The join's CTAs are brought up
// while the chunks' run out and wait for their end (32 ragged sequences of up to
// 8,192 keys: 54.9 us, else 56.5; 200 of up to 2,048: 71 and 76.8).
template <int D, int KS, int RT, bool SHARED>
cudaError_t launch_join(const RowsParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.B * p.Hk * p.S * p.G;
  const bool few = p.splits <= 24;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(few ? (rows + 3) / 4 : rows));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, few ? k_attn_join<D, KS, RT, 1, SHARED> : k_attn_join<D, KS, RT, 4, SHARED>, p);
}

template <int D, int MODE, int NT, bool MANY>
cudaError_t launch(const RowsParams& p, cudaStream_t stream) {
  using Src = Source<D, MODE, NT>;
  constexpr size_t smem = row_smem<D, MODE, NT>();
  cudaError_t e = cudaFuncSetAttribute(k_attn_rows<D, MODE, NT, MANY>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas =
      p.share == kShared ? p.ctas : (int64_t)p.B * p.Hk * p.tiles * p.splits;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.share == kCluster ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, k_attn_rows<D, MODE, NT, MANY>, p);
  if (e != cudaSuccess || p.share != kShared) return e;
  return launch_join<D, Src::KS, 8 * NT, true>(p, stream);
}

template <int D, int MODE>
cudaError_t launch_nt(const RowsParams& p, cudaStream_t stream) {
  if constexpr (MODE == 0)
    if (p.row_tile == 32) return launch<D, MODE, 4, true>(p, stream);
  if (MODE == 0 || (MODE == 1 && p.S > 1))
    return p.row_tile == 8 ? launch<D, MODE, 1, MODE != 2>(p, stream)
                           : launch<D, MODE, 2, MODE != 2>(p, stream);
  return p.row_tile == 8 ? launch<D, MODE, 1, MODE == 0>(p, stream)
                         : launch<D, MODE, 2, MODE == 0>(p, stream);
}

}  // namespace

cudaError_t launch_attn_join_tiles(const RowsParams& p, int D, cudaStream_t stream) {
  return D == 128 ? launch_join<128, 64, 128, false>(p, stream)
                  : launch_join<64, 64, 128, false>(p, stream);
}

template <int D>
static int rows_ctas(bool cache4, int row_tile) {
  if (cache4) return row_tile == 8 ? row_ctas<D, 1, 1>() : row_ctas<D, 1, 2>();
  return row_tile == 8    ? row_ctas<D, 0, 1>()
         : row_tile == 16 ? row_ctas<D, 0, 2>()
                          : row_ctas<D, 0, 4>();
}

int attn_rows_ctas(int D, bool cache4, int row_tile) {
  return D == 128 ? rows_ctas<128>(cache4, row_tile) : rows_ctas<64>(cache4, row_tile);
}

cudaError_t launch_attn_rows(const RowsParams& p, int D, cudaStream_t stream) {
  const int mode = !p.pages ? 0 : (p.idx ? 2 : 1);
  if (D == 128)
    return mode == 0   ? launch_nt<128, 0>(p, stream)
           : mode == 1 ? launch_nt<128, 1>(p, stream)
                       : launch_nt<128, 2>(p, stream);
  return mode == 0   ? launch_nt<64, 0>(p, stream)
         : mode == 1 ? launch_nt<64, 1>(p, stream)
                     : launch_nt<64, 2>(p, stream);
}

}  // namespace si
