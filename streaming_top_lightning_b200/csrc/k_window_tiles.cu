// Window attention of many query rows (prompts and their chunks) on the tensor
// cores.  The formula and the key rule are those of k_attn_rows.cu's bf16 path.
//
//   o[row] = sum_j softmax_j(scale * q[row] . k[j]) v[j] over j <= t with
//            j > t - window or j < sinks
//
// What bounds it: 4 D operations per (row, key) pair on the tensor cores, and
// as many cycles of exponentials (a 128 x 128 score tile takes 512 + 512 cycles
// of MMA at D = 128, and 1,024 of the SM's 16 exponentials a cycle).  K and V
// come from L2: neighbouring tiles share nearly all of their keys.
//
// The G = H / H_k query heads of a kv head share its keys, so a tile's 128 rows
// are (query, head) pairs, 128 / G whole queries of them.  One persistent CTA
// per SM takes two such tiles at a time over the union of their keys, so every
// key block is loaded once for 256 rows, and the softmax of one tile runs while
// the tensor cores work for the other:
//   warp 0       K and V blocks by TMA into a ring, in the order of use
//                (K0 K1 V0 K2 V1 K3 ...); rows of V past the sequence's end
//                are overwritten with zeros (0 times whatever they hold would
//                reach the sums)
//   warp 2       the two Q tiles by TMA
//   warps 1, 3   a tile each: S = Q K^T of a block into one of two buffers in
//                TMEM, two blocks ahead of the softmax, then O += P V with P
//                read from TMEM
//   warps 4-11   softmax, four warps a tile, a thread a row: the block's 64
//                scores to registers, their maximum, then P = 2^(s - m) in bf16
//                over the first half of the buffer's columns, and the row's
//                sum.  O is rescaled only when a row's maximum has grown by more
//                than 2^16 since it was last fixed: bf16 and fp32 keep their
//                relative precision up there.  The output is divided by the sum
//                of the P's as rounded, so that a weight near one is not off by
//                its rounding (error against 64 bits on rows with a few large
//                logits: 0.0023 of the norm with the unrounded sum, which lse
//                takes, 0.0016 being the output's own rounding).
// Keys are taken from the first one that the pair of tiles sees, 64 at a time,
// the last block and the sinks' block cut to multiples of 32 columns, so a
// window costs about its own length and not whole tiles of it.  Only columns
// that a boundary crosses are compared with positions.
//
// A masked column's probability is 0, and 0 times an infinity or NaN in V is
// NaN; a row that comes out NaN by a value that it does not see is computed again
// by the formula (si_attn.cuh), so what a row does not see does not reach it.  The
// values behind the sinks in their block, which no row sees there but every item
// loads, are zeros of the TMA.  While rows are computed again the waits' clocks
// stand still.
// Where pairs of tiles are few and their keys many, the keys are cut into chunks
// that are items of their own (SPLIT), their results kept in fp32 and joined by
// k_window_join (plan_window_tiles says when, with the times).
//
// Measured on B200: 8,192 queries of 64 heads, 8 kv heads, D = 128, window 1,024
// take 293 us in a burst (880 TFLOP/s) and 331-337 sustained at the power limit
// (770 TFLOP/s); the tensor cores alone would take 156 at the dense peak.  They
// are active for 46 % of the time and the exponentials' unit for 47 %: two softmax
// warps a scheduler do not hide one another's chains (scores from TMEM, maximum,
// exponentials, store), and the two units work in turn more than at once.  Before,
// with 128-key blocks and one score buffer 489, scores read from TMEM twice 510.
// A part of the exponentials as polynomials on the FMA units gave nothing under
// the power limit and is not kept.
// Every wait is bounded; a CTA that gives up records the error word, lets its
// copies and MMAs end and leaves.
#include "si_attn.cuh"

namespace si {
namespace {

constexpr int kM = 128;        // rows of a tile (MMA M)
constexpr int kN = 64;         // keys of a block
constexpr int kWinThreads = 384;
constexpr int kSoftWarp = 4;   // softmax warps 4-7: tile 0, 8-11: tile 1
constexpr float kGrow = 16.0f; // log2 growth of a maximum that rescales O

constexpr int kListed = 256;  // sequences whose live pairs a CTA lists

struct WinCtl {
  uint64_t kv_full[12], kv_empty[12], kv_land;
  uint64_t idle[2];  // a CTA that gives up: its MMAs are done
  uint64_t q_full, q_empty, s_full[2][2], p_ready[2][2], pv_done[2][2];  // [tile][buffer]
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t busy;  // softmax warps that compute rows again
  int starts[kListed + 1];  // LISTED: live pairs of the sequences before each one
  int items;
};

template <int D>
struct WinCfg {
  static constexpr uint32_t kQ = kM * D * 2;      // one Q tile
  static constexpr uint32_t kQHalf = kM * 128;    // its 64-column half
  static constexpr uint32_t kBlock = kN * D * 2;  // one K or V block
  static constexpr uint32_t kHalf = kN * 128;     // its 64-column half
  static constexpr int kSlots = D == 128 ? 10 : 12;
  static constexpr size_t kSmem =
      2 * (size_t)kQ + kSlots * (size_t)kBlock + 1024 + sizeof(WinCtl);
};

SI_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                        int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// A pair of tiles: its queries, their positions and the key blocks.
struct WinItem {
  int b, hk, i0;     // batch, kv head, first query
  int len, q_len;
  int live, QT;      // live queries of the pair, queries of a full tile
  int t0;            // position of the first query
  KeySpan span;      // of both tiles, cut to the item's chunk of it
  int sink_base;     // first sink of the chunk
  int chunk, pieces; // the chunk, of so many that hold the pair's keys
  int blocks, win_blocks;
  // the window blocks that each tile sees, and whether it sees the sinks' blocks
  // (where there are any, every query of the pair lies behind them)
  int from[2], to[2];
  bool sinks[2];
  // live queries of tile i (0: none) and the position of its first
  SI_DEV int nq(int i) const { return clampi(live - i * QT, 0, QT); }
  SI_DEV int first(int i) const { return t0 + i * QT; }
};

template <bool SPLIT, bool LISTED>
SI_DEV bool win_item(const WinParams& p, int id, const int* starts, WinItem& it) {
  int pairs = p.pairs, b = 0;
  if constexpr (LISTED) {  // the sequence whose live pairs hold the item
    const int unit = id / (SPLIT ? p.Hk * p.splits : p.Hk);
    for (int hi = p.B; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (starts[mid] <= unit)
        b = mid;
      else
        hi = mid;
    }
    pairs = starts[b + 1] - starts[b];
    id -= starts[b] * (SPLIT ? p.Hk * p.splits : p.Hk);
  }
  const int all = SPLIT ? pairs * p.splits : pairs, bh = id / all;
  it.chunk = SPLIT ? (id - bh * all) / pairs : 0;
  const int pair = id - bh * all - it.chunk * pairs;
  it.b = LISTED ? b : bh / p.Hk;
  it.hk = LISTED ? bh : bh - it.b * p.Hk;
  it.i0 = pair * 2 * p.QT;
  it.len = seq_len(p.lens, it.b, p.T);
  it.q_len = seq_len(p.q_lens, it.b, p.S);
  it.QT = p.QT;
  it.live = min(it.q_len - it.i0, 2 * p.QT);
  if (it.live <= 0) return false;
  it.t0 = it.len - it.q_len + it.i0;
  it.span = key_span<1>(it.t0, it.t0 + it.live - 1, it.len, p.window, p.sinks);
  it.win_blocks = (it.span.end - it.span.base + kN - 1) / kN;
  it.blocks = it.win_blocks + (it.span.sink_end + kN - 1) / kN;
  it.pieces = 1;
  it.sink_base = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // first key of the tile's first query, last position of its last
    const int nq = it.nq(i), lo = max(0, it.first(i) - p.window + 1);
    const int hi = min(it.span.end, it.first(i) + nq);
    it.from[i] = max(0, (p.sinks > it.span.base ? 0 : lo - it.span.base) / kN);
    it.to[i] = nq == 0 || hi <= 0 ? 0 : (hi - it.span.base + kN - 1) / kN;
    it.sinks[i] = it.to[i] > 0 && it.span.sink_end > 0;
  }
  if (SPLIT && it.blocks > p.chunk) {
    it.pieces = (it.blocks + p.chunk - 1) / p.chunk;
    // the window blocks of the chunk, then the sinks'
    const int w0 = min(it.chunk * p.chunk, it.win_blocks), s0 = it.chunk * p.chunk - w0;
    it.blocks = min(p.chunk, it.blocks - it.chunk * p.chunk);
    it.win_blocks = min(it.blocks, it.win_blocks - w0);
    it.span.base += w0 * kN;
    it.span.end = min(it.span.end, it.span.base + it.win_blocks * kN);
    it.sink_base = s0 * kN;
    it.span.sink_end = min(it.span.sink_end, (s0 + it.blocks - it.win_blocks) * kN);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      it.from[i] = clampi(it.from[i] - w0, 0, it.win_blocks);
      it.to[i] = clampi(it.to[i] - w0, 0, it.win_blocks);
      it.sinks[i] = it.sinks[i] && it.blocks > it.win_blocks;
      if (it.to[i] <= it.from[i]) it.from[i] = it.to[i] = it.win_blocks;
    }
  }
  return !SPLIT || it.chunk < it.pieces;
}

// First key of block n, the keys it holds, and its columns (a multiple of 32).
// The sinks' blocks come last: the first maximum is then that of many keys.
SI_DEV int block_key(const WinItem& it, int n) {
  return n < it.win_blocks ? it.span.base + n * kN : it.sink_base + (n - it.win_blocks) * kN;
}
SI_DEV int block_keys(const WinItem& it, int n) {
  return min(kN, (n < it.win_blocks ? it.span.end : it.span.sink_end) - block_key(it, n));
}
SI_DEV int columns(int keys) { return (keys + 31) & ~31; }

// The x-th block of an item's ring, in the order of use: K0 K1 V0 K2 V1 K3 ...
// (with one block: K0 V0).
SI_DEV int ring_block(int blocks, int x, bool& is_v) {
  if (x < 2 && x < blocks) {
    is_v = false;
    return x;
  }
  if (x >= 2 * blocks - 2 || blocks < 2) {  // the last two values
    is_v = true;
    return x - blocks;
  }
  is_v = (x & 1) == 0;
  return is_v ? (x - 2) >> 1 : (x + 1) >> 1;
}
}  // namespace

// SPLIT: chunks of a pair's keys are items of their own.  LISTED: sequences have
// query rows of their own number, and a CTA's items are every so-many-th of
// those that have rows (8 ragged chunks of up to 1,024 queries, window 1,024:
// 99 us, 113-118 without; the longer way to an item costs a full prompt 5 %).
template <int D, bool SPLIT, bool LISTED>
__global__ void __launch_bounds__(kWinThreads, 1)
    k_window_tiles(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_vs, const WinParams p) {
  using C = WinCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  // [Q0 | Q1 | ring | ctl]
  const uint32_t base = smem_u32(smem);
  const uint32_t ring = base + 2 * C::kQ;
  WinCtl* cs = reinterpret_cast<WinCtl*>(smem + 2 * (size_t)C::kQ + C::kSlots * (size_t)C::kBlock);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&cs->kv_full[i]), 1);
      mbar_init(smem_u32(&cs->kv_empty[i]), 2);  // both MMA warps
    }
    mbar_init(smem_u32(&cs->idle[0]), 1);
    mbar_init(smem_u32(&cs->idle[1]), 1);
    mbar_init(smem_u32(&cs->kv_land), 1);
    mbar_init(smem_u32(&cs->q_full), 1);
    mbar_init(smem_u32(&cs->q_empty), 2);
    for (int i = 0; i < 2; ++i) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_u32(&cs->s_full[i][x]), 1);
        mbar_init(smem_u32(&cs->p_ready[i][x]), kM);
        mbar_init(smem_u32(&cs->pv_done[i][x]), 1);
      }
    }
    cs->abort = 0u;
    cs->busy = 0u;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&cs->tmem_base), 512);
    tmem_relinquish();
  }
  if (LISTED && warp == 2) {
    int live[kListed / 32], sum = 0;
#pragma unroll
    for (int e = 0; e < kListed / 32; ++e) {
      const int b = lane * (kListed / 32) + e;
      live[e] = b < p.B ? (seq_len(p.q_lens, b, p.S) + 2 * p.QT - 1) / (2 * p.QT) : 0;
      sum += live[e];
    }
    int at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, at, o);
      if (lane >= o) at += y;
    }
    at -= sum;
#pragma unroll
    for (int e = 0; e < kListed / 32; ++e) {
      cs->starts[lane * (kListed / 32) + e] = at;
      at += live[e];
    }
    if (lane == 31) {
      cs->starts[kListed] = at;
      cs->items = at * p.Hk * p.splits;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = cs->tmem_base;
  const Ctl ctl{p.err, &cs->abort, p.timeout_ns, nullptr, &cs->busy};

  if (warp == 0) {
    // ------------------------------------------------------------ K and V
    uint32_t at = 0, lands = 0;  // blocks issued; blocks mended
    bool ok = true;
    for (int id = blockIdx.x; ok && id < (LISTED ? cs->items : p.items); id += gridDim.x) {
      WinItem it;
      if (!win_item<SPLIT, LISTED>(p, id, cs->starts, it)) continue;
      for (int x = 0; ok && x < 2 * it.blocks; ++x, ++at) {
        bool is_v;
        const int n = ring_block(it.blocks, x, is_v);
        const int slot = (int)(at % C::kSlots);
        if (!mbar_wait_warp(smem_u32(&cs->kv_empty[slot]), ((at / C::kSlots) & 1u) ^ 1u, ctl)) {
          ok = false;
          break;
        }
        const int j0 = block_key(it, n), cols = columns(block_keys(it, n));
        const uint32_t dst = ring + slot * C::kBlock;
        // keys past the sequence's end lie in the block's last columns
        const bool mend = is_v && j0 + cols > it.len;
        const uint32_t bar = smem_u32(mend ? &cs->kv_land : &cs->kv_full[slot]);
        // keys behind the sinks in their block read as zeros (seen by no row there)
        const CUtensorMap* map = !is_v ? &tm_k : (n < it.win_blocks ? &tm_v : &tm_vs);
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, (uint32_t)cols * D * 2);
          for (int c = (p.debug_flags & 1) && at == 0 ? cols : 0; c < cols; c += 32)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(dst + h * C::kHalf + c * 128, map, bar, 64 * h, it.hk, j0 + c, it.b);
        }
        __syncwarp();
        if (mend) {
          if (!mbar_wait_warp(bar, lands & 1u, ctl)) {
            ok = false;
            break;
          }
          ++lands;
          // whole 128-byte rows, so the swizzle does not matter
          const int first = max(0, it.len - j0);
          for (int y = lane; y < (cols - first) * 8 * (D / 64); y += 32) {
            const int h = y / ((cols - first) * 8), z = y % ((cols - first) * 8);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             dst + h * C::kHalf + first * 128 + z * 16),
                         "r"(0)
                         : "memory");
          }
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&cs->kv_full[slot]));
        }
      }
    }
    if (*ctl.abort && lane == 0) {
      // let the copies in flight land before the CTA leaves
      const uint64_t t_end = globaltimer() + 1000000ull;
      for (uint32_t x = at > C::kSlots ? at - C::kSlots : 0; x < at; ++x)
        while (!mbar_try_wait(smem_u32(&cs->kv_full[x % C::kSlots]), (x / C::kSlots) & 1u) &&
               globaltimer() < t_end) {
        }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ Q
    if (lane == 0) {
      uint32_t n = 0;
      for (int id = blockIdx.x; id < (LISTED ? cs->items : p.items); id += gridDim.x) {
        WinItem it;
        if (!win_item<SPLIT, LISTED>(p, id, cs->starts, it) || it.blocks == 0) continue;
        if (!mbar_wait(smem_u32(&cs->q_empty), (n & 1u) ^ 1u, ctl)) break;
        ++n;
        const int tiles = it.live > p.QT ? 2 : 1;
        const uint32_t bar = smem_u32(&cs->q_full);
        mbar_arrive_expect_tx(bar, (uint32_t)(tiles * p.QT * p.G * D * 2));
        for (int i = 0; i < tiles; ++i)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(base + i * C::kQ + h * C::kQHalf, &tm_q, bar, 64 * h, it.hk * p.G,
                        it.i0 + i * p.QT, it.b);
      }
      if (*ctl.abort && n > 0) {
        const uint64_t t_end = globaltimer() + 1000000ull;
        while (!mbar_try_wait(smem_u32(&cs->q_full), (n - 1) & 1u) && globaltimer() < t_end) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA
    // Warp 1 for tile 0, warp 3 for tile 1.  The whole warp goes through the
    // loop with values that are the same in every lane, and one lane issues:
    // descriptors then stay in uniform registers.  (Issued from code that one
    // lane alone runs, each of an MMA's operands is moved there first, about 90
    // cycles an instruction.)
    const int i = warp >> 1;
    const bool leader = elect_one();
    constexpr uint32_t idesc_o = idesc_make(1, 1, kM, D) | (1u << 16);  // V is MN-major
    const uint32_t u_tmem = uniform(tmem);
    const uint32_t s_tmem = u_tmem + i * 128, o_tmem = u_tmem + 256 + i * 128;
    const uint64_t qd = sdesc_sw128(uniform(base) + i * C::kQ);
    const uint64_t kd0 = sdesc_sw128(uniform(ring)), vd0 = sdesc_mn(uniform(ring), C::kHalf);
    uint32_t slot = 0, phase = 0;  // of the next block in the ring
    uint32_t nq = 0, np = 0;
    bool ok = true;
    for (int id = blockIdx.x; ok && id < (LISTED ? cs->items : p.items); id += gridDim.x) {
      WinItem it;
      if (!uniform(win_item<SPLIT, LISTED>(p, id, cs->starts, it))) continue;
      const int blocks = uniform(it.blocks), wins = uniform(it.win_blocks);
      if (blocks == 0) continue;
      const int from = uniform(i ? it.from[1] : it.from[0]), to = uniform(i ? it.to[1] : it.to[0]);
      // columns of the last window block and the last of the sinks
      const int win_cols = uniform(columns(block_keys(it, it.win_blocks - 1)));
      const int sink_cols = uniform(columns(block_keys(it, it.blocks - 1)));
      const bool sinks = uniform(i ? it.sinks[1] : it.sinks[0]);
      if (!mbar_wait_warp(smem_u32(&cs->q_full), nq & 1u, ctl)) break;
      ++nq;
      uint32_t begun = 0u;
      // The first two blocks' scores, then for each block its values and the
      // scores of the one two further on, into the buffer of the same parity:
      // the ring holds them in this order.  see, cols: of blocks n, n + 1, n + 2.
      uint32_t see = 0u;
      int cols0 = kN, cols1 = kN, cols2 = kN;
      for (int n = -2; n < blocks; ++n) {
        const int m = n + 2;
        see >>= 1;
        cols0 = cols1;
        cols1 = cols2;
        cols2 = m == wins - 1 ? win_cols : (m == blocks - 1 ? sink_cols : kN);
        if (m < blocks && ((m >= from && m < to) || (m >= wins && sinks))) see |= 4u;
        if (n >= 0) {
          if (!(ok = mbar_wait_warp(smem_u32(&cs->kv_full[slot]), phase, ctl))) break;
          if (see & 1u) {  // O += P V
            const int buf = n & 1;
            if (!(ok = mbar_wait_warp(smem_u32(&cs->p_ready[i][buf]), (np >> buf) & 1u, ctl))) break;
            np ^= 1u << buf;
            tc_fence_after();
            const uint64_t vd = vd0 + (uint64_t)(slot * (C::kBlock >> 4));
            const uint32_t a = s_tmem + buf * kN;
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kN / 16; ++kk)
                if (kk * 16 < cols0)
                  umma_ts(o_tmem, a + kk * 8, vd + kk * (2048 >> 4), idesc_o,
                               kk > 0 ? 1u : begun);
              umma_commit(smem_u32(&cs->pv_done[i][buf]));
            }
            __syncwarp();
            begun = 1u;
          }
          if (leader) umma_commit(smem_u32(&cs->kv_empty[slot]));
          __syncwarp();
          if (++slot == (uint32_t)C::kSlots) slot = 0, phase ^= 1u;
        }
        if (m < blocks) {
          if (!(ok = mbar_wait_warp(smem_u32(&cs->kv_full[slot]), phase, ctl))) break;
          if (see & 4u) {  // S = Q K^T
            tc_fence_after();
            const uint64_t kd = kd0 + (uint64_t)(slot * (C::kBlock >> 4));
            const uint32_t idesc_s = idesc_make(1, 1, kM, (uint32_t)cols2);
            const uint32_t d = s_tmem + (m & 1) * kN;
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16(d, qd + (((kk >> 2) * C::kQHalf + (kk & 3) * 32) >> 4),
                          kd + (((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4), idesc_s,
                          kk > 0 ? 1u : 0u);
              umma_commit(smem_u32(&cs->s_full[i][m & 1]));
            }
            __syncwarp();
          }
          if (leader) {
            umma_commit(smem_u32(&cs->kv_empty[slot]));
            if (m == blocks - 1) umma_commit(smem_u32(&cs->q_empty));
          }
          __syncwarp();
          if (++slot == (uint32_t)C::kSlots) slot = 0, phase ^= 1u;
        }
      }
    }
    if (*ctl.abort) umma_drain(&cs->idle[i], leader);
  } else if (warp >= kSoftWarp) {
    // ------------------------------------------------------------ softmax
    const int i = (warp - kSoftWarp) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + i * 128, o_col = lane_base + 256 + i * 128;
    const float sl2 = p.scale_log2;
    // parities of each buffer's next scores and next values; the buffer whose
    // values were the last (a barrier per buffer, because those of the block
    // before the last are known to be done only where they had the same one)
    uint32_t ns = 0, npv = 0;
    int last = 0;
    bool stop = false;
    for (int id = blockIdx.x; !stop && id < (LISTED ? cs->items : p.items); id += gridDim.x) {
      WinItem it;
      if (!win_item<SPLIT, LISTED>(p, id, cs->starts, it) || it.nq(i) == 0) continue;
      const int qi = row / p.G;  // query of the row within the tile
      const int nq = it.nq(i);
      const int ta = it.first(i), tb = ta + nq - 1;
      const int t = ta + min(qi, nq - 1);
      // limit: the maximum that asks for a new m; nothing before the first block
      // l: the sum of the weights; lr: of the weights as P holds them
      float m = neg_inf(), limit = neg_inf(), l = 0.0f, lr = 0.0f;
      const int from = i ? it.from[1] : it.from[0], to = i ? it.to[1] : it.to[0];
      const bool any = to > from || (i ? it.sinks[1] : it.sinks[0]);
      for (int n = from; n < it.blocks && any; ++n) {
        if (n == to) {  // on to the sinks
          n = it.win_blocks;
          if (n == it.blocks) break;
        }
        const int buf = n & 1;
        const uint32_t b_col = s_col + buf * kN;
        const int j0 = block_key(it, n), keys = block_keys(it, n), chunks = columns(keys) / 32;
        // whether every row of the tile sees every key of the block
        const bool clean = keys == kN && j0 + kN - 1 <= ta &&
                           (j0 > tb - p.window || j0 + kN - 1 < p.sinks);
        if (!mbar_wait_warp(smem_u32(&cs->s_full[i][buf]), (ns >> buf) & 1u, ctl)) {
          stop = true;
          break;
        }
        ns ^= 1u << buf;
        tc_fence_after();
        // the tile's columns, 32 at a time, stay in registers from here on
        float v[kN / 32][32];
#pragma unroll
        for (int c = 0; c < kN / 32; ++c)
          if (c < chunks) tmem_ld32(b_col + c * 32, v[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) pin32(v[c]);
        if (!clean) {
          // columns that a row does not see: its own are an interval and the sinks
#pragma unroll
          for (int c = 0; c < kN / 32; ++c) {
            const int a = j0 + 32 * c;
            const uint32_t seen = below(min(t + 1, j0 + keys) - a) &
                                  (~below(t + 1 - p.window - a) | below(p.sinks - a));
            asm volatile("" ::"r"(seen));  // a branch, and not 64 selections for every block
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((seen >> e) & 1u)) v[c][e] = neg_inf();
          }
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < kN / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = max3_nan(mx[(e >> 1) & 3], v[c][e], v[c][e + 1]);
        float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * sl2;
        // the first maximum is taken as it is; later ones once they pass it by 2^16
        const bool grow = !(top <= limit);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          // a score that is infinite or NaN makes the row NaN, as in the formula
          if (!(top < __int_as_float(0x7F800000))) top = m = __int_as_float(0x7FC00000);
          const float a = grow ? ex2(m - top) : 1.0f;
          if (n != from) {
            // nobody writes O once the values of the block before are in it
            if (!mbar_wait_warp(smem_u32(&cs->pv_done[i][last]), ((npv >> last) & 1u) ^ 1u, ctl)) {
              stop = true;
              break;
            }
            tc_fence_after();
            l *= a;
            lr *= a;
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
        const float sub = m == neg_inf() ? 0.0f : -m;
        const uint64_t sl22 = pair2(sl2, sl2), sub2 = pair2(sub, sub);
        uint64_t ls = 0ull, lsr = 0ull;
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) {
          if (c < chunks) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x, y;
              unpair2(fma2(pair2(v[c][e], v[c][e + 1]), sl22, sub2), x, y);
              x = ex2(x);
              y = ex2(y);
              const uint32_t both = pack_bf16x2(x, y);
              w[e >> 1] = both;
              ls = add2(ls, pair2(x, y));
              lsr = add2(lsr, pair2(bf16_lo(both), bf16_hi(both)));
            }
            tmem_st16(b_col + c * 16, w);
          }
        }
        float l0, l1;
        unpair2(ls, l0, l1);
        l += l0 + l1;
        unpair2(lsr, l0, l1);
        lr += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&cs->p_ready[i][buf]));
        npv ^= 1u << buf;
        last = buf;
      }
      if (stop) break;
      const bool live = qi < nq;
      const int64_t orow =
          ((int64_t)it.b * p.S + it.i0 + i * p.QT + qi) * p.H + it.hk * p.G + row % p.G;
      // a chunk of a row's keys: its place among the row's partial results
      const bool whole = !SPLIT || it.pieces == 1;
      const int64_t at = orow * p.splits + it.chunk;
      bool bad = false;
      if (any) {
        if (!mbar_wait_warp(smem_u32(&cs->pv_done[i][last]), ((npv >> last) & 1u) ^ 1u, ctl)) break;
        tc_fence_after();
        // a chunk's sums are those of the weights before their rounding, which is
        // what the join divides by
        const float inv = l == 0.0f ? 0.0f : (whole ? 1.0f : l) / lr;
        int64_t row_of[4];  // rows of this lane's group of four, -1: not live
#pragma unroll
        for (int e = 0; e < 4; ++e)
          row_of[e] = __shfl_sync(0xFFFFFFFFu, live ? orow : -1, (lane & ~3) + e);
        float v[32];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          tmem_ld32(o_col + c * 32, v);
          tmem_ld_wait();
          pin32(v);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            v[e] *= inv, v[e + 1] *= inv;
            bad |= v[e] != v[e] || v[e + 1] != v[e + 1];
            w[e >> 1] = pack_bf16x2(v[e], v[e + 1]);
          }
          if (!whole) {
            if (live) {
              float4* po = reinterpret_cast<float4*>(p.part_o + at * D + c * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                po[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
            continue;
          }
          // four lanes exchange 16-byte pieces, so that a store writes 64
          // consecutive bytes of each of eight rows
          uint4 piece[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            piece[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          transpose4(piece, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t o = row_of[e];
            if (o >= 0)
              reinterpret_cast<uint4*>(p.out + o * D + c * 32)[lane & 3] = piece[e];
          }
        }
        tc_fence_before();
      } else if (live && whole) {
        for (int c = 0; c < D / 8; ++c)
          reinterpret_cast<uint4*>(p.out + orow * D)[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (live && !whole)
        p.part_ml[at] = make_float2(l == 0.0f ? neg_inf() : m, l);
      else if (live && p.lse)
        p.lse[orow] = l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
      // rows by the formula (see the head of the file); a row whose maximum is NaN
      // has seen a score that makes it NaN
      __syncwarp();
      uint32_t again = __ballot_sync(0xFFFFFFFFu, bad && live && m == m);
      if (again && lane == 0) atomicAdd(&cs->busy, 1u);
      const bool looked = again != 0u;
      while (again) {
        const int r = __ffs(again) - 1;
        again &= again - 1;
        const int tr = __shfl_sync(0xFFFFFFFFu, t, r);
        const int64_t orr = __shfl_sync(0xFFFFFFFFu, orow, r);
        const int64_t stride = (int64_t)p.Hk * D;
        const int64_t first = (int64_t)it.b * p.T * stride + (int64_t)it.hk * D;
        // the keys that its blocks have brought
        const int last_s = it.blocks - 1, last_w = it.win_blocks - 1;
        const int w_end = last_w < 0 ? it.span.base
                                     : min(it.len, block_key(it, last_w) +
                                                       columns(block_keys(it, last_w)));
        const int s_end = last_s == last_w ? it.sink_base
                                           : min(min(it.len, p.sinks),
                                                 block_key(it, last_s) +
                                                     columns(block_keys(it, last_s)));
        // (behind the sinks in their block no row sees a key, though it may in a block
        // of the window: as from before the sequence)
        if (!unseen_bad<D>(p.v + first, stride, it.span.base, w_end, tr, p.window, p.sinks, lane) &&
            !unseen_bad<D>(p.v + first, stride, it.span.sink_end, s_end, -1, p.window, p.sinks, lane))
          continue;
        uint32_t nans = 0u;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const int d = lane * (D / 32) + e;
          const float x = whole ? __uint_as_float((uint32_t)p.out[orr * D + d] << 16)
                                : p.part_o[(orr * p.splits + it.chunk) * D + d];
          nans |= (uint32_t)(x != x) << e;
        }
        nans = unexplained<D>(p.v + first, stride, it.span.base, it.span.end, tr, it.len, p.window,
                              p.sinks, lane, nans);
        nans = unexplained<D>(p.v + first, stride, it.sink_base, it.span.sink_end, tr, it.len,
                              p.window, p.sinks, lane, nans);
        if (!__any_sync(0xFFFFFFFFu, nans != 0u)) continue;
        float rm = neg_inf(), rl = 0.0f, ro[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) ro[e] = 0.0f;
#pragma unroll 1
        for (int part = 0; part < 2; ++part)
          exact_row_keys<D>(p.q + orr * D, p.k + first, p.v + first, stride,
                            part ? it.span.base : it.sink_base,
                            part ? it.span.end : it.span.sink_end, tr, it.len, p.window, p.sinks,
                            sl2, lane, rm, rl, ro);
        if (!whole) {
          const int64_t to = orr * p.splits + it.chunk;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) p.part_o[to * D + lane * (D / 32) + e] = ro[e];
          if (lane == 0) p.part_ml[to] = make_float2(rl == 0.0f ? neg_inf() : rm, rl);
          continue;
        }
        const float rinv = rl == 0.0f ? 0.0f : 1.0f / rl;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orr * D) + lane * (D / 64);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) dst[e] = pack_bf16x2(ro[2 * e] * rinv, ro[2 * e + 1] * rinv);
        if (lane == 0 && p.lse)
          p.lse[orr] = rl == 0.0f ? neg_inf() : (rm + log2f(rl)) * 0.6931471805599453f;
      }
      __syncwarp();
      if (looked && lane == 0) atomicSub(&cs->busy, 1u);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the chunks of a row, a warp a row; rows of one chunk are written already.
template <int D>
__global__ void __launch_bounds__(128) k_window_join(const WinParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, heads = p.G;
  const int at = blockIdx.x * 4 + (threadIdx.x >> 5);  // B*S*H < 2^31
  if (at >= p.B * p.S * p.H) return;
  // (b, query, head) and the item that its pair of tiles is
  const int head = at % p.H, bq = at / p.H, i = bq % p.S, b = bq / p.S;
  WinItem it;
  if (i >= seq_len(p.q_lens, b, p.S)) return;
  if (!win_item<true, false>(p, (b * p.Hk + head / heads) * p.pairs * p.splits + i / (2 * p.QT), nullptr,
                      it) ||
      it.pieces == 1)
    return;
  const int64_t first = (int64_t)at * p.splits;
  float top = neg_inf();
  for (int s = lane; s < it.pieces; s += 32) top = fmaxf(top, p.part_ml[first + s].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
  float o[E], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < it.pieces; ++s) {
    // a chunk without a key for the row has no sums
    const float2 v = p.part_ml[first + s];
    if (v.y == 0.0f) continue;
    const float f = ex2(v.x - top);
    sum = fmaf(v.y, f, sum);
    const float* po = p.part_o + (first + s) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(po[e], f, o[e]);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (int64_t)at * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0 && p.lse)
    p.lse[at] = sum == 0.0f ? neg_inf() : (top + log2f(sum)) * 0.6931471805599453f;
}

namespace {
template <int D>
auto window_tiles(const WinParams& p) {
  const bool listed = p.q_lens && p.B > 1 && p.B <= kListed;
  return p.splits > 1 ? (listed ? k_window_tiles<D, true, true> : k_window_tiles<D, true, false>)
                      : (listed ? k_window_tiles<D, false, true> : k_window_tiles<D, false, false>);
}
}  // namespace

size_t window_tiles_smem(int D) { return D == 128 ? WinCfg<128>::kSmem : WinCfg<64>::kSmem; }

cudaError_t launch_window_tiles(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                const CUtensorMap& tm_v, const CUtensorMap& tm_vs,
                                const WinParams& p, int D, int grid, cudaStream_t stream) {
  const size_t smem = window_tiles_smem(D);
  const auto fn = D == 128 ? window_tiles<128>(p) : window_tiles<64>(p);
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  fn<<<grid, kWinThreads, smem, stream>>>(tm_q, tm_k, tm_v, tm_vs, p);
  if (p.splits > 1) {
    const unsigned ctas = (unsigned)(((int64_t)p.B * p.S * p.H + 3) / 4);
    if (D == 128)
      k_window_join<128><<<ctas, 128, 0, stream>>>(p);
    else
      k_window_join<64><<<ctas, 128, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace si
