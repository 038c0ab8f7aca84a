// Attention of many query rows over a 4-bit paged cache on the tensor cores:
// 17 and more (query, head) rows of a kv head, as a layer has whose 128 heads
// share one key row.  Formula, key rule, number formats and roundings are those
// of k_attn_rows.cu's 4-bit path.
//
// What bounds it: per key 4 D operations for each of 128 rows against 4.5 bits
// per element, so the tensor cores and the exponentials (a 128 x 64 block of
// scores takes 256 + 256 cycles of MMA at D = 128 and 512 of the SM's 16
// exponentials a cycle), with the conversion of the codes beside them (16,384
// fp16 numbers a block into shared memory).
//
// One persistent CTA per SM takes (row tile, chunk of keys) items.  The blocks
// of 64 keys of an item go alternately to two pipelines that share Q and have
// everything else of their own, the running maximum, sum and O too:
//   4 producer warps  codes from the pages into registers (one block ahead; the
//                     page two ahead, the listed entry three), to fp16 and into
//                     the 128-byte swizzled layout; keys that are not there
//                     become zeros and a cleared mask bit
//   an MMA warp       S = Q K^T into one of two TMEM buffers, two blocks ahead of
//                     the softmax, then O += P V with P read from TMEM
//   4 softmax warps   a thread a row, P = 2^(s - m) in fp16 over S's columns;
//                     at the start of an item they bring Q in
// At the end of an item each softmax group writes one half of the row's
// elements, from both pipelines' O.  The CTAs of a tile whose keys are split are
// a cluster (of up to eight): each joins a part of the rows, which the others
// write into its ring.  O is rescaled when a row's maximum has
// grown by more than 2^5 since it was last fixed; with the scale of 2^10 a
// probability then stays below fp16's largest number.
// Measured on B200: 64 queries of 128 heads over 2,048 listed entries each (one
// kv head, D = 128) take 33 us, 261 TFLOP/s; in 32-row tiles 117, and 62 before
// clusters joined the chunks.  8.6 GFLOP and 24 MB would take 5.2 us: with 16
// blocks a pipeline most of the time goes into the page and entry loads before
// the first block, the producers' conversions and the join.  Eight sequences of
// 16,384 keys, 128 rows of each of 4 kv heads: 65 us.
// Registers: the softmax threads take what the producers and MMA warps leave.
// Every wait is bounded; a CTA that gives up records the error word, lets its
// MMAs end, still meets its cluster, and leaves.
#include <cooperative_groups.h>

#include "si_attn.cuh"

namespace cg = cooperative_groups;

namespace si {
namespace {

constexpr int kM = 128;
constexpr int kN = 64;
constexpr int kThreads = 640;  // softmax 0, 1; producers 0, 1; MMA warps 16, 17
constexpr int kSlots = 3;      // K and V blocks of a pipeline
constexpr float kShift = 10.0f, kGrow = 5.0f;
template <int D>
constexpr int kRowPad = D + 4;  // floats of a row in a cluster's join: O, maximum, sum

template <int D>
struct TileCfg {
  static constexpr uint32_t kQ = kM * D * 2, kQHalf = kM * 128;
  static constexpr uint32_t kBlock = kN * D * 2, kHalf = kN * 128;  // K or V block
  static constexpr size_t kRing = 2 * kSlots * 2 * (size_t)kBlock;
};

struct TileCtl {
  uint64_t kv_full[2][kSlots], kv_empty[2][kSlots];
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];
  uint64_t q_full, q_empty, ml_full, o_free;
  uint64_t idle[2];               // a CTA that gives up: its MMAs are done
  uint64_t mask[2][kSlots];       // keys of a block that are there
  uint64_t nans[2][kSlots];       // not 0: a value scale of the block is NaN
  float factor[kM];               // 2^-x of the rows scaled by 2^x
  float xm[2][kM], xl[2][kM];     // the pipelines' maxima and sums
  uint32_t tmem_base;
  uint32_t abort;
};

// An item: its tile, its blocks [lo, hi) and its chunk.
struct TileItem {
  Tile ti;
  KeySpan span;
  int lo, hi, split;
};

SI_DEV bool tile_item(const RowsParams& p, int id, TileItem& it) {
  const int tile = id / p.splits;
  it.split = id - tile * p.splits;
  if (!find_tile<kM>(p, tile, it.ti)) return false;
  it.span = tile_span<kN>(p, it.ti);
  const int per = p.chunk_keys / kN;
  it.lo = it.split * per;
  it.hi = it.split + 1 == p.splits ? it.span.steps : min(it.span.steps, it.lo + per);
  // a row without keys is still written, and the CTAs of a cluster stay together
  return it.lo < it.hi || p.splits == 1 || p.share == kCluster;
}
// All threads of the cluster's CTAs.
SI_DEV void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The two meetings of a cluster's join, for warps with no part in it.
SI_DEV void stand_by(const RowsParams& p) {
  Tile ti;
  if (p.share != kCluster || !find_tile<kM>(p, blockIdx.x / p.splits, ti)) return;
  cluster_sync();
  cluster_sync();
}

// The blocks of 16 elements whose NaN value scale a row at position t sees, among
// the 64 keys from j0 on that are there.  By the whole warp.
template <int D>
SI_DEV uint32_t nan_blocks(const RowsParams& p, const Tile& ti, int j0, uint64_t there, int t,
                           int lane) {
  const int page = 1 << p.page_shift;
  uint32_t seen = 0u;
#pragma unroll 1
  for (int h = 0; h < kN; h += 32) {
    const int j = j0 + h + lane;
    uint32_t bits = 0u;
    if ((there >> (h + lane)) & 1u) {
      const int64_t pg = __ldg(p.table + (int64_t)ti.b * p.width + (j >> p.page_shift));
      const uint8_t* s = p.pages + pg * p.page_bytes + (int64_t)ti.hk * cache4_block<D>(page) +
                         page * D + (page + (j & (page - 1))) * (D / 16);
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) bits |= (uint32_t)e4m3_nan(__ldg(s + c)) << c;
    }
#pragma unroll 1
    for (int x = 0; x < 32; ++x) {
      const uint32_t b = __shfl_sync(0xFFFFFFFFu, bits, x);
      if (b && sees(j0 + h + x, t, ti.len, p.window, p.sinks)) seen |= b;
    }
  }
  return seen;
}

// Blocks of pipeline i.
SI_DEV int pipe_blocks(const TileItem& it, int i) { return max(0, it.hi - it.lo + 1 - i) >> 1; }

}  // namespace

template <int D, bool LISTED>
__global__ void __launch_bounds__(kThreads, 1) k_cache4_tiles(const __grid_constant__ RowsParams p,
                                                              int items, uint32_t* err,
                                                              uint64_t timeout_ns) {
  using C = TileCfg<D>;
  // [Q | pipeline 0: K V K V K V | pipeline 1 | ctl], with no room to align it by hand
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem), ring = base + C::kQ;
  TileCtl* cs = reinterpret_cast<TileCtl*>(smem + C::kQ + C::kRing);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (base & 1023u) {  // the swizzled layout needs it
    if (tid == 0) atomicOr(err, SI_DEVERR_BAD_STATE);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int x = 0; x < kSlots; ++x) {
        mbar_init(smem_u32(&cs->kv_full[i][x]), 128);
        mbar_init(smem_u32(&cs->kv_empty[i][x]), 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_u32(&cs->s_full[i][x]), 1);
        mbar_init(smem_u32(&cs->p_ready[i][x]), kM);
        mbar_init(smem_u32(&cs->pv_done[i][x]), 1);
      }
    }
    mbar_init(smem_u32(&cs->q_full), 2 * kM);
    mbar_init(smem_u32(&cs->q_empty), 2);
    mbar_init(smem_u32(&cs->ml_full), 2 * kM);
    mbar_init(smem_u32(&cs->o_free), 2 * kM);
    mbar_init(smem_u32(&cs->idle[0]), 1);
    mbar_init(smem_u32(&cs->idle[1]), 1);
    cs->abort = 0u;
    mbar_fence_init();
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(&cs->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = cs->tmem_base;
  const Ctl ctl{err, &cs->abort, timeout_ns, nullptr};

  if (warp >= 16) {
    // ------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp < 18) {
      const int i = warp - 16;
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = idesc_make(0, 0, kM, kN);               // fp16
      constexpr uint32_t idesc_o = idesc_make(0, 0, kM, D) | (1u << 16);   // V is MN-major
      const uint32_t u_tmem = uniform(tmem);
      const uint32_t s_tmem = u_tmem + i * 128, o_tmem = u_tmem + 256 + i * 128;
      const uint64_t qd = sdesc_sw128(uniform(base));
      const uint32_t my_ring = uniform(ring) + i * (kSlots * 2 * C::kBlock);
      const uint64_t kd0 = sdesc_sw128(my_ring), vd0 = sdesc_mn(my_ring + C::kBlock, C::kHalf);
      uint32_t kslot = 0, kphase = 0, vslot = 0, n_items = 0, np = 0;
      bool ok = true;
      for (int id = blockIdx.x; ok && id < items; id += gridDim.x) {
        int blocks, any;
        {
          TileItem it;
          if (!uniform(tile_item(p, id, it))) continue;
          any = uniform(it.hi - it.lo);
          blocks = uniform(pipe_blocks(it, i));
        }
        if (any <= 0) continue;
        if (!mbar_wait_warp(smem_u32(&cs->q_full), n_items & 1u, ctl)) break;
        ++n_items;
        if (blocks == 0 && leader) mbar_arrive(smem_u32(&cs->q_empty));
        for (int n = -2; n < blocks; ++n) {
          const int m = n + 2;
          if (n >= 0) {  // O += P V
            const int buf = n & 1;
            if (!(ok = mbar_wait_warp(smem_u32(&cs->p_ready[i][buf]), (np >> buf) & 1u, ctl))) break;
            np ^= 1u << buf;
            tc_fence_after();
            if (leader) {
              const uint64_t vd = vd0 + (uint64_t)(vslot * (2 * C::kBlock >> 4));
              const uint32_t a = s_tmem + buf * kN;
#pragma unroll
              for (int kk = 0; kk < kN / 16; ++kk)
                umma_ts(o_tmem, a + kk * 8, vd + kk * (2048 >> 4), idesc_o,
                        (kk > 0 || n > 0) ? 1u : 0u);
              umma_commit(smem_u32(&cs->pv_done[i][buf]));
              umma_commit(smem_u32(&cs->kv_empty[i][vslot]));
            }
            __syncwarp();
            if (++vslot == (uint32_t)kSlots) vslot = 0;
          }
          if (m < blocks) {  // S = Q K^T
            if (!(ok = mbar_wait_warp(smem_u32(&cs->kv_full[i][kslot]), kphase, ctl))) break;
            tc_fence_after();
            if (leader) {
              const uint64_t kd = kd0 + (uint64_t)(kslot * (2 * C::kBlock >> 4));
              const uint32_t d = s_tmem + (m & 1) * kN;
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16(d, qd + (((kk >> 2) * C::kQHalf + (kk & 3) * 32) >> 4),
                          kd + (((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4), idesc_s,
                          kk > 0 ? 1u : 0u);
              umma_commit(smem_u32(&cs->s_full[i][m & 1]));
              if (m == blocks - 1) umma_commit(smem_u32(&cs->q_empty));
            }
            __syncwarp();
            if (++kslot == (uint32_t)kSlots) kslot = 0, kphase ^= 1u;
          }
        }
      }
      if (*ctl.abort) umma_drain(&cs->idle[i], leader);
    }
    stand_by(p);
  } else if (warp >= 8) {
    // ------------------------------------------------------------ producers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // A warp takes 32 rows: keys 0-31 or 32-63 of a block, as K or as V rows.
    // Its lanes look up a row each; L lanes then share a row, 16 bytes of codes
    // (32 elements) each, 32 / L rows at a time, so that a load instruction
    // touches few lines.
    constexpr int L = D / 32, R = 32 / L;
    const int i = (warp - 8) >> 2;
    const bool is_v = (warp & 2) != 0;
    const int key0 = (warp & 1) * 32, key = key0 + lane;
    const int c = lane % L, sub = lane / L;
    const int page = 1 << p.page_shift;
    const uint32_t my_ring = ring + i * (kSlots * 2 * C::kBlock) + (is_v ? C::kBlock : 0);
    uint32_t slot = 0, phase = 0;
    bool ok = true;
    for (int id = blockIdx.x; ok && id < items; id += gridDim.x) {
      TileItem it;
      if (!tile_item(p, id, it) || it.hi <= it.lo) continue;
      const int blocks = pipe_blocks(it, i);
      const int32_t* table = p.table + (int64_t)it.ti.b * p.width;
      const int32_t* irow =
          LISTED ? p.idx + ((int64_t)it.ti.b * p.S + it.ti.row0 / p.G) * p.topk : nullptr;
      const uint8_t* head = p.pages + (int64_t)it.ti.hk * cache4_block<D>(page);
      // The key of this thread's row of the pipeline's n-th block (-1: none), its
      // page, and the head's block there (null: the row is not there), each
      // asked for a block before it is looked at.
      auto key_of = [&](int n) {
        if (n >= blocks) return -1;
        const int u = it.lo + 2 * n + i;
        if constexpr (LISTED) {
          const int e = u * kN + key;
          return e < p.topk ? __ldg(irow + e) : -1;
        } else {
          const int j = step_key<kN>(it.span, u) + key;
          return span_holds(it.span, u, j, p.sinks) ? j : -1;
        }
      };
      auto page_of = [&](int j) {
        return j >= 0 && j < it.ti.len ? __ldg(table + (j >> p.page_shift)) : -1;
      };
      // A row's place in the pool, its page's offset plus its slot (page_bytes
      // is a multiple of the page's tokens), or -1: it is not there.
      auto place = [&](int j, int pg) -> int64_t {
        return pg >= 0 && pg < p.n_pages ? (int64_t)pg * p.page_bytes + (j & (page - 1)) : -1;
      };
      // codes and scales of this lane's part of L rows; at: its own row's place
      uint4 code[L];
      uint32_t sc[L];
      auto load = [&](int64_t at) {
#pragma unroll
        for (int x = 0; x < L; ++x) {
          const int64_t o = __shfl_sync(0xFFFFFFFFu, at, x * R + sub);
          const int sl = (int)o & (page - 1);
          const uint8_t* blk = head + (o - sl);
          const int row = (is_v ? page : 0) + sl;
          code[x] = o >= 0 ? __ldg(reinterpret_cast<const uint4*>(blk + row * (D / 2)) + c)
                           : make_uint4(0, 0, 0, 0);
          sc[x] = o >= 0 ? __ldg(reinterpret_cast<const uint16_t*>(blk + page * D + row * (D / 16)) + c)
                         : 0u;
        }
      };
      int j0 = key_of(0), j1 = key_of(1), j2 = key_of(2);
      int pg1 = page_of(j1);
      int64_t here = place(j0, page_of(j0));
      load(here);
      for (int n = 0; ok && n < blocks; ++n) {
        if (!mbar_wait_warp(smem_u32(&cs->kv_empty[i][slot]), phase ^ 1u, ctl)) {
          ok = false;
          break;
        }
        const uint32_t dst = my_ring + slot * (2 * C::kBlock);
        uint4 cur[L];
        uint32_t cur_s[L];
#pragma unroll
        for (int x = 0; x < L; ++x) cur[x] = code[x], cur_s[x] = sc[x];
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, here >= 0);
        here = place(j1, pg1);
        load(here);
        pg1 = page_of(j2);
        j1 = j2;
        j2 = key_of(n + 3);
        if (!LISTED && is_v) {
          // A NaN scale counts as zero in the products (a weight of zero times it
          // would be NaN); the softmax looks up which rows it reaches.  The rows
          // of a listed tile all see the same keys.
          uint32_t odd = 0u;
#pragma unroll
          for (int x = 0; x < L; ++x) odd |= e4m3_nans(cur_s[x]);
          const bool any = __any_sync(0xFFFFFFFFu, odd != 0u);
          if (any)
#pragma unroll
            for (int x = 0; x < L; ++x) cur_s[x] &= ~((e4m3_nans(cur_s[x]) >> 7) * 0xFFu);
          if (lane == 0) reinterpret_cast<uint32_t*>(&cs->nans[i][slot])[warp & 1] = any;
        }
#pragma unroll
        for (int x = 0; x < L; ++x) {
          const int row = key0 + x * R + sub;
          const uint32_t s2 = e4m3x2(cur_s[x]);
          const uint32_t f[2] = {__byte_perm(s2, 0, 0x1010), __byte_perm(s2, 0, 0x3232)};
          const uint32_t w[4] = {cur[x].x, cur[x].y, cur[x].z, cur[x].w};
          const uint32_t to = dst + row * 128 + (c >> 1) * C::kHalf;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // the upper half's lanes store in another order: no bank twice
            const int q = k ^ (c & 2);
            const uint32_t ww = (c & 2) ? w[k ^ 2] : w[k];
            const uint32_t s = (c & 2) ? f[(k ^ 2) >> 1] : f[k >> 1];
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             to + (((4 * (c & 1) + q) ^ (row & 7)) << 4)),
                         "r"(hmul2(e2m1x2<0>(ww), s)), "r"(hmul2(e2m1x2<1>(ww), s)),
                         "r"(hmul2(e2m1x2<2>(ww), s)), "r"(hmul2(e2m1x2<3>(ww), s))
                         : "memory");
          }
        }
        if (!is_v && lane == 0)
          reinterpret_cast<uint32_t*>(&cs->mask[i][slot])[warp & 1] = m;
        fence_async();
        if (!((p.debug_flags & 1) && n == 0)) mbar_arrive(smem_u32(&cs->kv_full[i][slot]));
        if (++slot == (uint32_t)kSlots) slot = 0, phase ^= 1u;
      }
    }
    stand_by(p);
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int i = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + i * 128, o_all = lane_base + 256, o_col = o_all + i * 128;
    // parities: each pipeline's values per buffer, this one's scores per buffer
    uint32_t mine = 0, theirs = 0, ns = 0, kslot = 0, kphase = 0, n_items = 0, n_ml = 0;
    bool stop = false, met = false;
    for (int id = blockIdx.x; !stop && id < items; id += gridDim.x) {
      TileItem it;
      if (!tile_item(p, id, it)) continue;
      const Tile& ti = it.ti;
      const bool live = row < ti.rows;
      const int t = ti.len - ti.q_len + (ti.row0 + min(row, ti.rows - 1)) / p.G;
      const int blocks = pipe_blocks(it, i), others = pipe_blocks(it, i ^ 1);
      float m = neg_inf(), limit = neg_inf(), l = 0.0f, f = 0.0f;
      uint32_t bad = 0u;  // blocks of 16 elements that a NaN scale reaches
      if (it.hi > it.lo) {
        // Q to fp16, scaled by a power of two a row (k_attn_rows.cu): 16 rows a
        // warp, D/8 lanes a row
        constexpr int LQ = D / 8, RQ = 32 / LQ;
        uint4 x[16 / RQ];
#pragma unroll
        for (int y = 0; y < 16 / RQ; ++y) {
          const int r = warp * 16 + y * RQ + lane / LQ;
          x[y] = r < ti.rows ? __ldg(reinterpret_cast<const uint4*>(
                                         p.q + out_row(p, ti, ti.row0 + r) * D) +
                                     lane % LQ)
                             : make_uint4(0, 0, 0, 0);
        }
        if (!mbar_wait_warp(smem_u32(&cs->q_empty), (n_items & 1u) ^ 1u, ctl)) break;
#pragma unroll
        for (int y = 0; y < 16 / RQ; ++y) {
          const int r = warp * 16 + y * RQ + lane / LQ, c = lane % LQ;
          const uint32_t w[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
          float big = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            big = fmaxf(big, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
#pragma unroll
          for (int o = 1; o < LQ; o <<= 1)
            big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
          const int e = (int)(__float_as_uint(big) >> 23);
          const int up = (e == 0 || e == 255) ? 0 : max(-126, min(126, 137 - e));
          const float g = __uint_as_float((uint32_t)(127 + up) << 23);
          if (c == 0) cs->factor[r] = __uint_as_float((uint32_t)(127 - up) << 23);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           base + (c >> 3) * C::kQHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                       "r"(pack_f16x2(bf16_lo(w[0]) * g, bf16_hi(w[0]) * g)),
                       "r"(pack_f16x2(bf16_lo(w[1]) * g, bf16_hi(w[1]) * g)),
                       "r"(pack_f16x2(bf16_lo(w[2]) * g, bf16_hi(w[2]) * g)),
                       "r"(pack_f16x2(bf16_lo(w[3]) * g, bf16_hi(w[3]) * g))
                       : "memory");
        }
        fence_async();
        mbar_arrive(smem_u32(&cs->q_full));
        if (!mbar_wait_warp(smem_u32(&cs->q_full), n_items & 1u, ctl)) break;
        ++n_items;
        // above zero: times -inf for an unseen key it is not NaN
        f = fmaxf(cs->factor[row] * p.scale_log2, 1.17549435e-38f);
      }
      for (int n = 0; n < blocks; ++n) {
        const int buf = n & 1;
        const uint32_t b_col = s_col + buf * kN;
        const int u = it.lo + 2 * n + i;
        if (!mbar_wait_warp(smem_u32(&cs->kv_full[i][kslot]), kphase, ctl) ||
            !mbar_wait_warp(smem_u32(&cs->s_full[i][buf]), (ns >> buf) & 1u, ctl)) {
          stop = true;
          break;
        }
        const uint64_t there = cs->mask[i][kslot];
        const bool odd = !LISTED && cs->nans[i][kslot] != 0u;
        if (++kslot == (uint32_t)kSlots) kslot = 0, kphase ^= 1u;
        ns ^= 1u << buf;
        tc_fence_after();
        float v[kN / 32][32];
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) tmem_ld32(b_col + c * 32, v[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) pin32(v[c]);
        bool clean = there == ~0ull;
        int j0 = 0;
        if constexpr (!LISTED) {
          j0 = step_key<kN>(it.span, u);
          clean = clean && j0 + kN - 1 <= ti.t_min &&
                  (j0 > ti.t_max - p.window || j0 + kN <= p.sinks);
        }
        if (!clean) {
#pragma unroll
          for (int c = 0; c < kN / 32; ++c) {
            uint32_t seen = (uint32_t)(there >> (32 * c));
            if constexpr (!LISTED) {
              const int a = j0 + 32 * c;
              seen &= below(min(t + 1, ti.len) - a) &
                      (~below(t + 1 - p.window - a) | below(p.sinks - a));
            }
            asm volatile("" ::"r"(seen));  // a branch, and not 64 selections for every block
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((seen >> e) & 1u)) v[c][e] = neg_inf();
          }
        }
        if (odd) bad |= nan_blocks<D>(p, ti, j0, there, t, lane);
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < kN / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = max3_nan(mx[(e >> 1) & 3], v[c][e], v[c][e + 1]);
        float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * f;
        const bool grow = !(top <= limit);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          // a score that is infinite or NaN makes the row NaN, as in the formula
          if (!(top < __int_as_float(0x7F800000))) top = m = __int_as_float(0x7FC00000);
          const float a = grow ? ex2(m - top) : 1.0f;
          if (n > 0) {
            // nobody writes O once the values of the block before are in it
            const int last = buf ^ 1;
            if (!mbar_wait_warp(smem_u32(&cs->pv_done[i][last]), ((mine >> last) & 1u) ^ 1u,
                                ctl)) {
              stop = true;
              break;
            }
            tc_fence_after();
            l *= a;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t w[16];
              tmem_ld16(o_col + c * 16, w);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+r"(w[e]));
                w[e] = __float_as_uint(__uint_as_float(w[e]) * a);
              }
              tmem_st16(o_col + c * 16, w);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          if (grow) {
            m = top;
            limit = top + kGrow;
          }
        }
        // the other group may still read this pipeline's O of the item before
        if (n == 0 && n_ml > 0 &&
            !mbar_wait_warp(smem_u32(&cs->o_free), (n_ml - 1) & 1u, ctl)) {
          stop = true;
          break;
        }
        const float sub = kShift - (m == neg_inf() ? 0.0f : m);
        const uint64_t f2 = pair2(f, f), sub2 = pair2(sub, sub);
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            uint64_t xy = fma2(pair2(v[c][e], v[c][e + 1]), f2, sub2);
            float x, y;
            unpair2(xy, x, y);
            x = ex2(x);
            y = ex2(y);
            xy = pair2(x, y);
            ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], xy);
            w[e >> 1] = pack_f16x2(x, y);
          }
          tmem_st16(b_col + c * 16, w);
        }
        float l0, l1;
        unpair2(add2(ls[0], ls[1]), l0, l1);
        l += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&cs->p_ready[i][buf]));
        mine ^= 1u << buf;
      }
      if (stop) break;
      // both pipelines' results: this group writes half of the elements
      // (the other pipeline has used its buffers in turn)
      theirs ^= ((uint32_t)(others + 1) >> 1 & 1u) | ((uint32_t)others >> 1 & 1u) << 1;
      // (and this one's maxima and sums)
      if (blocks == 0 && n_ml > 0 &&
          !mbar_wait_warp(smem_u32(&cs->o_free), (n_ml - 1) & 1u, ctl))
        break;
      if (__any_sync(0xFFFFFFFFu, bad != 0u)) {
        // NaN into the row's elements of those blocks
        const int last = (blocks - 1) & 1;
        if (!mbar_wait_warp(smem_u32(&cs->pv_done[i][last]), ((mine >> last) & 1u) ^ 1u, ctl)) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t w[16];
          tmem_ld16(o_col + c * 16, w);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            asm volatile("" : "+r"(w[e]));
            if ((bad >> c) & 1u) w[e] = 0x7FC00000u;
          }
          tmem_st16(o_col + c * 16, w);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      cs->xm[i][row] = m;
      cs->xl[i][row] = l;
      mbar_arrive(smem_u32(&cs->ml_full));
      if (!mbar_wait_warp(smem_u32(&cs->ml_full), n_ml & 1u, ctl)) break;
      bool ready = true;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int nb = x == i ? blocks : others, last = (nb - 1) & 1;
        if (nb > 0)
          ready = ready && mbar_wait_warp(smem_u32(&cs->pv_done[x][last]),
                                          (((x == i ? mine : theirs) >> last) & 1u) ^ 1u, ctl);
      }
      if (!ready) break;
      tc_fence_after();
      const int b0 = pipe_blocks(it, 0), b1 = pipe_blocks(it, 1);
      const float m0 = cs->xm[0][row], m1 = cs->xm[1][row];
      const float top = fmaxf(m0, m1);
      const float f0 = b0 && m0 != neg_inf() ? ex2(m0 - top) : 0.0f;
      const float f1 = b1 && m1 != neg_inf() ? ex2(m1 - top) : 0.0f;
      const float sum = cs->xl[0][row] * f0 + cs->xl[1][row] * f1;
      const bool final_rows = p.splits == 1;
      const float inv = sum == 0.0f ? 0.0f : (final_rows ? p.v_scale / sum : 1.0f);
      const int64_t part = (ti.part + row) * p.splits + it.split;
      const int64_t orow = live ? out_row(p, ti, ti.row0 + row) : -1;
      // in a cluster, the CTA that joins this row, and the row's place there
      const int per = (kM + p.splits - 1) / p.splits, rank = row / per;
      float* there = nullptr;
      if (p.share == kCluster) {
        cluster_sync();  // every CTA is done with its ring
        cg::cluster_group cl = cg::this_cluster();
        float* mine = reinterpret_cast<float*>(smem + C::kQ);
        there = cl.map_shared_rank(mine, rank) + (it.split * per + row - rank * per) * kRowPad<D>;
        if (i == 0)
          *reinterpret_cast<float2*>(there + D) = make_float2(sum == 0.0f ? neg_inf() : top, sum);
      }
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        const int col = i * (D / 2) + c * 32;
        float a[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if ((x ? b1 : b0) == 0) continue;
          float o[32];
          tmem_ld32(o_all + x * 128 + col, o);
          tmem_ld_wait();
          pin32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = fmaf(o[e], x ? f1 : f0, a[e]);
        }
        if (final_rows) {
          uint4 piece[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            piece[e] = make_uint4(pack_bf16x2(a[8 * e] * inv, a[8 * e + 1] * inv),
                                  pack_bf16x2(a[8 * e + 2] * inv, a[8 * e + 3] * inv),
                                  pack_bf16x2(a[8 * e + 4] * inv, a[8 * e + 5] * inv),
                                  pack_bf16x2(a[8 * e + 6] * inv, a[8 * e + 7] * inv));
          transpose4(piece, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t o = __shfl_sync(0xFFFFFFFFu, orow, (lane & ~3) + e);
            if (o >= 0) reinterpret_cast<uint4*>(p.out + o * D + col)[lane & 3] = piece[e];
          }
        } else if (p.share == kCluster) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(there + col + 4 * e) =
                make_float4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 piece[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* v = a + 16 * h + 4 * e;
              piece[e] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                    __float_as_uint(v[2]), __float_as_uint(v[3]));
            }
            transpose4(piece, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int64_t o = __shfl_sync(0xFFFFFFFFu, live ? part : -1, (lane & ~3) + e);
              if (o >= 0)
                reinterpret_cast<uint4*>(p.part_o + o * D + col + 16 * h)[lane & 3] = piece[e];
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&cs->o_free));
      ++n_ml;
      if (p.share == kCluster) {
        cluster_sync();  // all of this CTA's rows are here
        const float* mine = reinterpret_cast<const float*>(smem + C::kQ);
        const int r0 = it.split * per;  // the split is the CTA's rank
        // D/32 threads a row, 32 elements each, in an order that spreads the banks
        constexpr int TR = D / 32;
        const int q = tid % TR;
        for (int x = tid / TR; x < per && r0 + x < ti.rows; x += 2 * kM / TR) {
          float big = neg_inf(), tot = 0.0f;
          float4 acc[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int y = 0; y < p.splits; ++y)
            big = fmaxf(big, mine[(y * per + x) * kRowPad<D> + D]);
          for (int y = 0; y < p.splits; ++y) {
            const float* from = mine + (y * per + x) * kRowPad<D>;
            const float w = from[D + 1] == 0.0f ? 0.0f : ex2(from[D] - big);
            tot = fmaf(from[D + 1], w, tot);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v =
                  *reinterpret_cast<const float4*>(from + 32 * q + 4 * ((e + 2 * q) & 7));
              acc[e].x = fmaf(v.x, w, acc[e].x), acc[e].y = fmaf(v.y, w, acc[e].y);
              acc[e].z = fmaf(v.z, w, acc[e].z), acc[e].w = fmaf(v.w, w, acc[e].w);
            }
          }
          const float fin = tot == 0.0f ? 0.0f : p.v_scale / tot;
          const int64_t to = out_row(p, ti, ti.row0 + r0 + x);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint2*>(p.out + to * D + 32 * q + 4 * ((e + 2 * q) & 7)) =
                make_uint2(pack_bf16x2(acc[e].x * fin, acc[e].y * fin),
                           pack_bf16x2(acc[e].z * fin, acc[e].w * fin));
          if (q == 0 && p.lse)
            p.lse[to] = tot == 0.0f ? neg_inf() : (big - kShift + log2f(tot)) * 0.6931471805599453f;
        }
        met = true;
      } else if (live && i == 0) {
        const float lg = top - kShift;
        if (!final_rows)
          p.part_ml[part] = make_float2(sum == 0.0f ? neg_inf() : lg, sum);
        else if (p.lse)
          p.lse[orow] = sum == 0.0f ? neg_inf() : (lg + log2f(sum)) * 0.6931471805599453f;
      }
    }
    if (!met) stand_by(p);  // gave up before the join: the others still meet
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

size_t cache4_tiles_smem(int D) {
  return (D == 128 ? TileCfg<128>::kQ + TileCfg<128>::kRing : TileCfg<64>::kQ + TileCfg<64>::kRing) +
         sizeof(TileCtl);
}

template <int D, bool LISTED>
static cudaError_t launch_tiles(const RowsParams& p, int items, int grid, uint32_t* err,
                                uint64_t timeout_ns, cudaStream_t stream) {
  const size_t smem = cache4_tiles_smem(D);
  const cudaError_t e = cudaFuncSetAttribute(
      k_cache4_tiles<D, LISTED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.share == kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_cache4_tiles<D, LISTED>, p, items, err, timeout_ns);
}

cudaError_t launch_cache4_tiles(const RowsParams& p, int D, int grid, uint32_t* err,
                                uint64_t timeout_ns, cudaStream_t stream) {
  const int items = (int)((int64_t)p.B * p.Hk * p.tiles * p.splits);
  if (p.share == kCluster) grid = items;  // an item a CTA
  const cudaError_t e =
      D == 128 ? (p.idx ? launch_tiles<128, true>(p, items, grid, err, timeout_ns, stream)
                        : launch_tiles<128, false>(p, items, grid, err, timeout_ns, stream))
               : (p.idx ? launch_tiles<64, true>(p, items, grid, err, timeout_ns, stream)
                        : launch_tiles<64, false>(p, items, grid, err, timeout_ns, stream));
  if (e != cudaSuccess || p.splits == 1 || p.share == kCluster) return e;
  return launch_attn_join_tiles(p, D, stream);
}

}  // namespace si
