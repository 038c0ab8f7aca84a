// Shared pieces of the attention kernels that read a key/value cache: which
// keys a query sees, and small PTX wrappers.
//
// Query row i of batch b (i < q_len) sits at position t = len - q_len + i of a
// sequence of len tokens, and sees key j when
//   j <= t  and  j < len  and  (j > t - window  or  j < sinks).
#pragma once

#include <cuda_fp16.h>

#include "si_common.cuh"
#include "si_kernels.h"

namespace si {

SI_DEV float neg_inf() { return __int_as_float(0xFF800000); }

SI_DEV bool sees(int j, int t, int len, int window, int sinks) {
  return j <= t && j < len && (j > t - window || j < sinks);
}

SI_DEV int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Length of sequence b and how many of the S query rows it has.
SI_DEV int seq_len(const int32_t* lens, int b, int cap) {
  return lens ? clampi(__ldg(lens + b), 0, cap) : cap;
}

// The keys that some query of a tile sees, [lo, end) and the sinks before it,
// as steps of KS keys: first the sinks' steps, then those from `base` on (lo
// rounded down to a step).
struct KeySpan {
  int lo, base, end, sink_end, sink_steps, steps;
};

template <int KS>
SI_DEV KeySpan key_span(int t_min, int t_max, int len, int window, int sinks) {
  KeySpan s;
  s.end = min(len, t_max + 1);
  s.lo = max(0, t_min - window + 1);
  if (s.end <= 0) return KeySpan{0, 0, 0, 0, 0, 0};
  s.base = s.lo / KS * KS;
  if (s.base > s.end) s.base = s.end / KS * KS;
  s.sink_end = min(min(sinks, s.base), s.end);
  s.sink_steps = (s.sink_end + KS - 1) / KS;
  s.steps = s.sink_steps + (s.end - s.base + KS - 1) / KS;
  return s;
}

// First key of a step, and whether a key of it is one that the span holds.
template <int KS>
SI_DEV int step_key(const KeySpan& s, int u) {
  return u < s.sink_steps ? u * KS : s.base + (u - s.sink_steps) * KS;
}
SI_DEV bool span_holds(const KeySpan& s, int u, int j, int sinks) {
  return u < s.sink_steps ? j < s.sink_end : (j < s.end && (j >= s.lo || j < sinks));
}

SI_DEV void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
template <int N>
SI_DEV void cp_async_small(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
               "r"(bytes)
               : "memory");
}
SI_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SI_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

SI_DEV float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
SI_DEV float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
SI_DEV uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
SI_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^x, -inf to 0.
SI_DEV float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 numbers in a register pair, and arithmetic on both at once.
SI_DEV uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
SI_DEV void unpair2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
SI_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SI_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SI_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The largest magnitude of three; a NaN among them is the result.
SI_DEV float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest of three; a NaN among them is the result.
SI_DEV float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// D (+)= A B, 16 x 8 x 16, fp32 accumulation.
SI_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
SI_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
SI_DEV void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
SI_DEV void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Two E2M1 numbers of a byte, and two E4M3 numbers of a half-word, as fp16
// (both exact; the lower bits give the lower half).
template <int BYTE>
SI_DEV uint32_t e2m1x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(r)
      : "r"(w), "n"(BYTE));
  return r;
}
SI_DEV uint32_t e4m3x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
// Whether an E4M3 byte is NaN, and a word's NaN bytes (0x80 in their places).
SI_DEV bool e4m3_nan(uint32_t b) { return (b & 0x7Fu) == 0x7Fu; }
SI_DEV uint32_t e4m3_nans(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
SI_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The block of one kv head in a 4-bit page: K codes, V codes, K scales, V
// scales, each [page, ...].
template <int D>
SI_DEV int64_t cache4_block(int page) {
  return (int64_t)page * (D + D / 8);
}

// The tile's rows and what its queries see.
struct Tile {
  int b, hk, row0, rows;  // rows: live rows of the tile
  int len, q_len, t_min, t_max;
  int64_t part;           // index of its first row among all rows
};

template <int RT>
SI_DEV bool find_tile(const RowsParams& p, uint32_t id, Tile& ti) {
  const uint32_t bh = id / (uint32_t)p.tiles;
  const int tile = (int)(id - bh * (uint32_t)p.tiles);
  ti.b = (int)(bh / (uint32_t)p.Hk);
  ti.hk = (int)(bh - (uint32_t)ti.b * (uint32_t)p.Hk);
  ti.len = seq_len(p.lens, ti.b, p.T);
  ti.q_len = seq_len(p.q_lens, ti.b, p.S);
  int last;  // one past the tile's last row
  if (p.idx) {  // a tile's rows belong to one query
    const int per = (p.G + RT - 1) / RT;
    const int i = tile / per;
    ti.row0 = i * p.G + (tile % per) * RT;
    last = min((i + 1) * p.G, ti.q_len * p.G);
  } else {
    ti.row0 = tile * RT;
    last = ti.q_len * p.G;
  }
  ti.rows = min(RT, last - ti.row0);
  if (ti.rows <= 0) return false;
  ti.t_min = ti.len - ti.q_len + ti.row0 / p.G;
  ti.t_max = ti.len - ti.q_len + (ti.row0 + ti.rows - 1) / p.G;
  ti.part = (int64_t)bh * p.S * p.G + ti.row0;
  return true;
}

// The steps of KS keys that a tile takes.
template <int KS>
SI_DEV KeySpan tile_span(const RowsParams& p, const Tile& ti) {
  if (p.idx) return KeySpan{0, 0, p.topk, 0, 0, (p.topk + KS - 1) / KS};
  return key_span<KS>(ti.t_min, ti.t_max, ti.len, p.window, p.sinks);
}

SI_DEV int64_t out_row(const RowsParams& p, const Tile& ti, int row) {
  const int i = row / p.G;
  return ((int64_t)ti.b * p.S + i) * p.H + ti.hk * p.G + row % p.G;
}

// ------------------------------------------------------------ tensor-core tiles
// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands (idesc says which).
SI_DEV void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// Descriptor of an MN-major operand in the 128-byte swizzle: 64-element blocks
// along N lie lbo_bytes apart, 8-row groups along K 1024.
SI_DEV uint64_t sdesc_mn(uint32_t saddr, uint32_t lbo_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)64u << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

SI_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
SI_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

SI_DEV void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Keeps values read from TMEM behind the wait for them.
SI_DEV void pin32(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]),
                 "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7]));
}

// The first lane's value, which the compiler then knows to be the warp's.
template <class T>
SI_DEV T uniform(T x) {
  return (T)__shfl_sync(0xFFFFFFFFu, (int)x, 0);
}
SI_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0u;
}

// Waits, at most a millisecond, for the MMAs issued so far (a CTA that gives up
// frees its TMEM only then).  By the warp that issued them.
SI_DEV void umma_drain(uint64_t* bar, bool leader) {
  if (leader) {
    umma_commit(smem_u32(bar));
    const uint64_t end = globaltimer() + 1000000ull;
    while (!mbar_try_wait(smem_u32(bar), 0u) && globaltimer() < end) {
    }
  }
  __syncwarp();
}

// Transposes the 4 x 4 pieces of four neighbouring lanes: lane q's piece e
// becomes lane e's piece q.
SI_DEV uint4 shfl_xor4(uint4 x, int m) {
  return make_uint4(__shfl_xor_sync(0xFFFFFFFFu, x.x, m), __shfl_xor_sync(0xFFFFFFFFu, x.y, m),
                    __shfl_xor_sync(0xFFFFFFFFu, x.z, m), __shfl_xor_sync(0xFFFFFFFFu, x.w, m));
}
SI_DEV void transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e & m) continue;
      // lanes without the bit give their piece e | m for the others' piece e
      const uint4 give = up ? x[e] : x[e | m];
      const uint4 got = shfl_xor4(give, m);
      if (up)
        x[e] = got;
      else
        x[e | m] = got;
    }
  }
}

// The n lowest bits.
SI_DEV uint32_t below(int n) { return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u); }

SI_DEV void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Kernels that multiply whole tiles give a row NaN when the value of a key that
// it does not see holds an infinity or NaN (0 times that value).  Rows that came
// out NaN are looked at by a whole warp, D/32 elements of a bf16 row per lane:
// where unseen_bad finds such a value, and a NaN of the row is not one that it has
// seen itself (unexplained), the row is computed again (exact_row_keys).  A key
// is unseen by some row of a tile, but in its blocks, for a few tiles only, so
// one bad value costs a few tiles' rows however many see it.  (B200, 8,192 queries
// of 64 heads, window 1,024, 0.30 ms: with a NaN token among the sinks 0.8 ms, with
// one elsewhere 8.3, the time of one tile's rows; 169 and 172 when every row that
// came out NaN was computed again.)
template <int D>
SI_DEV uint2 value_bits(const uint16_t* v, int lane) {
  if constexpr (D == 128) return __ldg(reinterpret_cast<const uint2*>(v) + lane);
  return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(v) + lane), 0u);
}

// Whether one of the keys [lo, hi) that the query at t does not see has a value
// that is not finite.
template <int D>
SI_DEV bool unseen_bad(const uint16_t* v, int64_t key_stride, int lo, int hi, int t, int window,
                       int sinks, int lane) {
  uint32_t bad = 0u;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int a = part ? max(lo, t + 1) : max(lo, sinks);
    const int b = part ? hi : min(hi, t - window + 1);
#pragma unroll 4
    for (int j = a; j < b; ++j) {
      const uint2 w = value_bits<D>(v + j * key_stride, lane);
      // an exponent of ones carries into the sign's place
      bad |= (((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u)) & 0x80008000u;
    }
  }
  return __any_sync(0xFFFFFFFFu, bad != 0u);
}

// Of a lane's elements in `nans` those that are not NaN in any key of [lo, hi)
// that the query sees.
template <int D>
SI_DEV uint32_t unexplained(const uint16_t* v, int64_t key_stride, int lo, int hi, int t, int len,
                            int window, int sinks, int lane, uint32_t nans) {
  for (int j0 = lo; j0 < hi && __any_sync(0xFFFFFFFFu, nans != 0u); j0 += 8) {
    uint2 w[8];  // asked for together
#pragma unroll
    for (int x = 0; x < 8; ++x)
      w[x] = value_bits<D>(v + (int64_t)min(j0 + x, hi - 1) * key_stride, lane);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if (j0 + x >= hi || !sees(j0 + x, t, len, window, sinks)) continue;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        if ((((e < 2 ? w[x].x : w[x].y) >> (16 * (e & 1))) & 0x7FFFu) > 0x7F80u) nans &= ~(1u << e);
    }
  }
  return nans;
}

// A key of score s (log2 units) into a row's running maximum, sum and values.
template <int D>
SI_DEV void exact_key(float s, const float (&v)[D / 32], float& m, float& l, float (&o)[D / 32]) {
  const float mn = fmaxf(m, s);  // ignores a NaN score, which makes the weight NaN below
  const float a = mn == neg_inf() ? 1.0f : ex2(m - mn);
  const float w = mn == neg_inf() && s == s ? 0.0f : ex2(s - mn);
  l = l * a + w;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = fmaf(o[e], a, w * v[e]);
  m = mn;
}

// One query row by the formula, by a whole warp: the keys [j_lo, j_hi) of a
// bf16 source that the row sees.
template <int D>
SI_DEV void exact_row_keys(const uint16_t* qr, const uint16_t* k, const uint16_t* v,
                           int64_t key_stride, int j_lo, int j_hi, int t, int len, int window,
                           int sinks, float scale_log2, int lane, float& m, float& l,
                           float (&o)[D / 32]) {
  const uint2 qw = value_bits<D>(qr, lane);
  for (int j0 = j_lo; j0 < j_hi; j0 += 8) {
    uint2 kw[8], vw[8];  // asked for together; keys that the row does not see are not used
    float dot[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int64_t at = (int64_t)min(j0 + x, j_hi - 1) * key_stride;
      kw[x] = value_bits<D>(k + at, lane);
      vw[x] = value_bits<D>(v + at, lane);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      dot[x] = fmaf(bf16_hi(qw.x), bf16_hi(kw[x].x), bf16_lo(qw.x) * bf16_lo(kw[x].x));
      if (D == 128)
        dot[x] = fmaf(bf16_hi(qw.y), bf16_hi(kw[x].y),
                      fmaf(bf16_lo(qw.y), bf16_lo(kw[x].y), dot[x]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int x = 0; x < 8; ++x) dot[x] += __shfl_xor_sync(0xFFFFFFFFu, dot[x], o);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if (j0 + x >= j_hi || !sees(j0 + x, t, len, window, sinks)) continue;
      float vv[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const uint32_t two = e < 2 ? vw[x].x : vw[x].y;
        vv[e] = (e & 1) ? bf16_hi(two) : bf16_lo(two);
      }
      exact_key<D>(dot[x] * scale_log2, vv, m, l, o);
    }
  }
}

}  // namespace si
