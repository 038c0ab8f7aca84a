// Rows into and out of a 4-bit paged cache (layout: include/streamindex.h).
//
// Append rounds blocks of 16 elements of a bf16 row: with the row scale g,
//   s = E4M3(min(amax / (6 g), 448)),  code = E2M1(x / (g s)),
// both to nearest with ties to even; an element whose quotient passes 6 is
// stored as 6, a block whose s rounds to zero as zeros, and a NaN as zero.
// One thread takes one block: 32 bytes in, 8 bytes of codes and one scale
// out, neighbouring threads on neighbouring blocks.  Measured on B200: chunks
// of up to 4,096 rows of four ragged sequences, 8 kv heads of 128 elements,
// appended in 14 us and read in 12.5 (24 MB and as much: launch, lengths, table
// and data are a chain of loads).  Before NaNs and saturated blocks had a path of
// their own the rounding's instructions bound the append, at 17.  Append and read
// together take 31 us, with two blocks a thread 39.  The quotient
// is Markstein's correctly rounded one (reciprocal rounded to nearest, product,
// one residual step; "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), a third of a division's instructions: ties
// are common (x and s are short), so a quotient that is off by one unit would
// show.
#include "si_attn.cuh"

namespace si {
namespace {

constexpr int kThreads = 256;

// One block of a call's rows: (batch, row, kv head, key or value, block).
template <int D>
struct Block {
  bool live;
  bool is_v;
  int64_t src;          // element offset in k or v
  int64_t codes, scale; // byte offsets in the pages
};

template <int D>
SI_DEV Block<D> find_block(const Cache4Params& p, uint32_t block, int thread) {
  constexpr int NB = D / 16;
  Block<D> r;
  // (row, key or value, kv head, block): `block` counts rows of blocks, and
  // B * S * Hk < 2^31
  const int blk = thread % NB;
  const uint32_t x = block * (kThreads / NB) + thread / NB;
  const uint32_t row2 = x / (uint32_t)p.Hk;
  const int hk = (int)(x - row2 * (uint32_t)p.Hk);
  r.is_v = (row2 & 1u) != 0;  // all of a row's key blocks, then its value blocks
  const uint32_t row = row2 >> 1;
  const int b = (int)(row / (uint32_t)p.S);
  const int i = (int)(row - (uint32_t)b * (uint32_t)p.S);
  r.live = false;
  if (b >= p.B) return r;
  const int page = 1 << p.page_shift;
  const int len = clampi(__ldg(p.lens + b), 0, p.cap);
  const int q_len = seq_len(p.q_lens, b, p.S);
  const int pos = len - q_len + i;
  if (i >= q_len || pos < 0) return r;
  const int pg = __ldg(p.table + (int64_t)b * p.width + (pos >> p.page_shift));
  if (pg < 0 || pg >= p.n_pages) return r;
  const int slot = pos & (page - 1);
  const int64_t base = (int64_t)pg * p.page_bytes + hk * cache4_block<D>(page);
  r.live = true;
  r.src = (((int64_t)b * p.S + i) * p.Hk + hk) * D + blk * 16;
  r.codes = base + (r.is_v ? page * (D / 2) : 0) + slot * (D / 2) + blk * 8;
  r.scale = base + page * D + (r.is_v ? page * (D / 16) : 0) + slot * (D / 16) + blk;
  return r;
}

SI_DEV uint32_t e2m1_byte(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b32 %0, {b, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads) k_cache4_append(const Cache4Params p) {
  const Block<D> bl = find_block<D>(p, blockIdx.x, threadIdx.x);
  if (!bl.live) return;
  const uint4* src = reinterpret_cast<const uint4*>((bl.is_v ? p.v : p.k) + bl.src);
  const uint4 a = __ldcs(src), b = __ldcs(src + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    amax = max3_abs_nan(amax, x[2 * i], x[2 * i + 1]);
  }
  const float g = bl.is_v ? p.v_scale : p.k_scale;
  // a NaN, or elements that the largest scale does not reach
  const bool odd = !(amax <= 6.0f * 448.0f * g);
  if (odd) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = x[i] == x[i] ? x[i] : 0.0f;
      amax = fmaxf(amax, fabsf(x[i]));
    }
  }
  uint16_t sb;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(sb)
      : "f"(0.0f), "f"(fminf(__fdiv_rn(amax, 6.0f * g), 448.0f)));
  const float gs = g * __half2float(__ushort_as_half((uint16_t)e4m3x2(sb)));
  const float rcp = gs > 0.0f ? __frcp_rn(gs) : 0.0f;
  uint32_t out[2] = {0u, 0u};
  if (gs > 0.0f) {
    float y[16];
    if (!odd) {
      // quotients of less than 9, two at a time
      const uint64_t rcp2 = pair2(rcp, rcp), neg2 = pair2(-gs, -gs);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint64_t m = pair2(x[i], x[i + 1]), q = mul2(m, rcp2);
        unpair2(fma2(fma2(q, neg2, m), rcp2, q), y[i], y[i + 1]);
        y[i] = copysignf(y[i], x[i]);  // of zeros
        y[i + 1] = copysignf(y[i + 1], x[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // up to 8 the quotient is exact to rounding; past that it is stored as 6
        const float m = fabsf(x[i]);
        const float q = fminf(m * rcp, 8.0f);
        y[i] = copysignf(fmaf(fmaf(-q, gs, m), rcp, q), x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i >> 2] |= e2m1_byte(y[2 * i], y[2 * i + 1]) << (8 * (i & 3));
  }
  *reinterpret_cast<uint2*>(p.pages + bl.codes) = make_uint2(out[0], out[1]);
  p.pages[bl.scale] = (uint8_t)sb;
}

// The rows back as bf16: code x (g s), rounded once.
template <int D>
__global__ void __launch_bounds__(kThreads) k_cache4_read(const Cache4Params p) {
  const Block<D> bl = find_block<D>(p, blockIdx.x, threadIdx.x);
  if (!bl.live) return;
  const uint2 c = *reinterpret_cast<const uint2*>(p.pages + bl.codes);
  const float gs = (bl.is_v ? p.v_scale : p.k_scale) *
                   __half2float(__ushort_as_half((uint16_t)e4m3x2(p.pages[bl.scale])));
  uint32_t w[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = h ? c.y : c.x;
    const uint32_t v[4] = {e2m1x2<0>(x), e2m1x2<1>(x), e2m1x2<2>(x), e2m1x2<3>(x)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      w[4 * h + i] = pack_bf16x2(f.x * gs, f.y * gs);
    }
  }
  uint4* dst = reinterpret_cast<uint4*>((bl.is_v ? p.v_out : p.k_out) + bl.src);
  __stcs(dst, make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(dst + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

cudaError_t launch_cache4_rows(const Cache4Params& p, int D, bool append, cudaStream_t stream) {
  const int64_t blocks = (int64_t)p.B * p.S * p.Hk * 2 * (D / 16);
  const unsigned grid = (unsigned)((blocks + kThreads - 1) / kThreads);
  if (append) {
    if (D == 128)
      k_cache4_append<128><<<grid, kThreads, 0, stream>>>(p);
    else
      k_cache4_append<64><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (D == 128)
      k_cache4_read<128><<<grid, kThreads, 0, stream>>>(p);
    else
      k_cache4_read<64><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace si
