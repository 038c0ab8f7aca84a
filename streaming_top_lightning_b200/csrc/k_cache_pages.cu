// The life of a cache's pages: growth, forks, release and compaction.
//
// A pool of n pages has a count per page of the table rows that hold it (0:
// free); a row of the page table lists the pages of one sequence in its leading
// entries, -1 after them.  Every call takes the lowest free pages, in the order
// of its rows, so a result depends on nothing but the inputs.
//
// The counting parts read the counts and tables twice and decide with prefix
// sums over them: one CTA where a few rounds of its threads are enough, else a
// cluster of eight, each with a contiguous share, that exchange their shares'
// sums through distributed shared memory (one launch; a grid-wide scan would
// take two or three).  They are bound by latency: of a load, a barrier, a round.
// Copies of pages run in a second launch over the whole GPU, HBM-bound.
//
// Measured on B200: freeing, forking and growing 32 of 64 sequences (pool of
// 6,933 pages) takes 27.4 us in four launches, 32.7 with clusters throughout;
// compacting a pool of 23,588 pages of 74 KB, 396 MB moved, 141 us, of which the
// copies take 127 at 5.9 TB/s.
#include <cooperative_groups.h>

#include "si_attn.cuh"

namespace cg = cooperative_groups;

namespace si {
namespace {

constexpr int kClu = 8;         // CTAs of a counting kernel's cluster, or one
constexpr int kThreads = 1024;  // threads of each
constexpr int kSlice = 16384;   // bytes of a page that one CTA copies at a time

// Sum over the CTA, to every thread.
SI_DEV int cta_sum(int v, int* sh) {
  const int s = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  const int t = sh[threadIdx.x & 31];
  return __reduce_add_sync(0xFFFFFFFFu, t);
}

// Exclusive prefix sum over the CTA; *total gets the sum.
SI_DEV int cta_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int w = sh[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}

// The CTAs of a counting kernel: C = 1 or a cluster.
template <int C>
struct Team {
  unsigned rank;
  SI_DEV Team() : rank(C == 1 ? 0u : cg::this_cluster().block_rank()) {}
  // Everyone's writes, to global memory too, are seen by everyone.
  SI_DEV void sync() const {
    if constexpr (C == 1) {
      __syncthreads();
    } else {
      __threadfence();
      cg::this_cluster().sync();
    }
  }
  // Two sums of each CTA (the same in all its threads): those of the CTAs
  // before this one, and of all.  slot: two numbers in shared memory.
  SI_DEV void sums(int* slot, int a, int b, int (&before)[2], int (&all)[2]) const {
    if constexpr (C == 1) {
      before[0] = before[1] = 0;
      all[0] = a, all[1] = b;
    } else {
      if (threadIdx.x == 0) slot[0] = a, slot[1] = b;
      sync();
      cg::cluster_group cl = cg::this_cluster();
#pragma unroll
      for (int i = 0; i < 2; ++i) before[i] = all[i] = 0;
#pragma unroll
      for (unsigned r = 0; r < C; ++r) {
        const int* o = cl.map_shared_rank(slot, r);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int v = o[i];
          if (r < rank) before[i] += v;
          all[i] += v;
        }
      }
    }
  }
  // This CTA's share of n things, in whole fours.
  SI_DEV int64_t from(int64_t n) const { return C == 1 ? 0 : n * rank / C / 4 * 4; }
  SI_DEV int64_t to(int64_t n) const {
    return C == 1 || rank == C - 1 ? n : n * (rank + 1) / C / 4 * 4;
  }
};

// Four counts from i on (a multiple of four; the array 16-byte aligned or not),
// those past the end as `none`.
SI_DEV int4 four(const int32_t* a, int64_t i, int64_t end, int none) {
  if (i + 4 <= end && (reinterpret_cast<uintptr_t>(a) & 15u) == 0)
    return *reinterpret_cast<const int4*>(a + i);
  int4 v = make_int4(none, none, none, none);
  if (i < end) v.x = a[i];
  if (i + 1 < end) v.y = a[i + 1];
  if (i + 2 < end) v.z = a[i + 2];
  if (i + 3 < end) v.w = a[i + 3];
  return v;
}

// Free pages among refs [lo, hi).
SI_DEV int count_free(const int32_t* refs, int64_t lo, int64_t hi, int* sh) {
  int c = 0;
  for (int64_t i = lo + 4 * threadIdx.x; i < hi; i += 4 * kThreads) {
    const int4 v = four(refs, i, hi, 1);
    c += (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
  }
  return cta_sum(c, sh);
}

// Gives the free pages of [lo, hi) their ranks from `rank` on: the pages ranked
// below `need` go to order[rank] and get one holder.
SI_DEV void take_free(int32_t* refs, int64_t lo, int64_t hi, int rank, int need, int32_t* order,
                      int* sh) {
  for (int64_t at = lo; at < hi && rank < need; at += 4 * kThreads) {
    const int64_t i = at + 4 * threadIdx.x;
    const int4 v = four(refs, i, hi, 1);
    const int f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
    int n, r = rank + cta_scan(f[0] + f[1] + f[2] + f[3], sh, &n);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f[e]) {
        if (r < need) {
          order[r] = (int32_t)(i + e);
          refs[i + e] = 1;
        }
        ++r;
      }
    rank += n;
  }
}

SI_DEV int pages_of(int len, int page_shift, int width) {
  if (len <= 0) return 0;
  const int n = (len - 1) / (1 << page_shift) + 1;
  return n < width ? n : width;
}

}  // namespace

// ---------------------------------------------------------------- extend
// Entries of the first ceil(len / page) of each row that hold no page get one.
template <int C>
__global__ void __launch_bounds__(kThreads) k_pages_extend(const PagesParams p) {
  __shared__ int sh[32], slot[2];
  const Team<C> team;
  const int64_t r_lo = team.from(p.B), r_hi = team.to(p.B);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // what this CTA's rows want: a warp a row
  int c = 0;
  for (int64_t r = r_lo + warp; r < r_hi; r += kThreads / 32) {
    const int n = pages_of(p.lens[r], p.page_shift, p.width);
    for (int e = lane; e < n; e += 32) c += p.table[r * p.width + e] < 0;
  }
  const int64_t f_lo = team.from(p.n_pages), f_hi = team.to(p.n_pages);
  const int nfree = count_free(p.refs, f_lo, f_hi, sh);
  const int want = cta_sum(c, sh);
  int before[2], all[2];
  team.sums(slot, want, nfree, before, all);
  if (team.rank == 0 && threadIdx.x == 0) *p.missing = max(0, all[0] - all[1]);
  if (all[0] > 0) {
    take_free(p.refs, f_lo, f_hi, before[1], all[0], p.order, sh);
    team.sync();
    // rows in order: each row's wants are a prefix sum over the CTA's rows
    int at = before[0];
    for (int64_t r0 = r_lo; r0 < r_hi; r0 += kThreads / 32) {
      const int64_t r = r0 + warp;
      int n = 0, cnt = 0;
      if (r < r_hi) {
        n = pages_of(p.lens[r], p.page_shift, p.width);
        for (int e = lane; e < n; e += 32) cnt += p.table[r * p.width + e] < 0;
      }
      cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
      int sum;
      int mine = at + cta_scan(lane == 0 ? cnt : 0, sh, &sum);
      mine = __shfl_sync(0xFFFFFFFFu, mine, 0);
      if (cnt) {
        for (int e0 = 0; e0 < n; e0 += 32) {
          const int e = e0 + lane;
          const bool w = e < n && p.table[r * p.width + e] < 0;
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, w);
          const int k = mine + __popc(m & ((1u << lane) - 1u));
          if (w && k < all[1]) p.table[r * p.width + e] = __ldcg(p.order + k);
          mine += __popc(m);
        }
      }
      at += sum;
    }
  }
  if constexpr (C > 1) team.sync();  // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- free
// One CTA per listed row.  A row listed twice is released once: each entry's
// page goes to whoever takes it out of the table.
__global__ void __launch_bounds__(128) k_pages_free(const PagesParams p) {
  const int row = p.rows[blockIdx.x];
  if (row < 0 || row >= p.B) return;
  int32_t* t = p.table + (int64_t)row * p.width;
  for (int e = threadIdx.x; e < p.width; e += 128) {
    if (t[e] < 0) continue;
    const int pg = atomicExch(t + e, -1);
    if (pg < 0 || pg >= p.n_pages) continue;
    if (atomicSub(p.refs + pg, 1) <= 0) atomicAdd(p.refs + pg, 1);  // never below zero
  }
  if (threadIdx.x == 0) p.lens[row] = 0;
}

// ---------------------------------------------------------------- fork
// Per child: pages shared with its parent, the page copied (or -1) and where to.
template <int C>
__global__ void __launch_bounds__(kThreads) k_pages_fork_plan(const PagesParams p) {
  __shared__ int sh[32], slot[4];
  const Team<C> team;
  const int64_t c_lo = team.from(p.n), c_hi = team.to(p.n);
  const int64_t f_lo = team.from(p.n_pages), f_hi = team.to(p.n_pages);
  const int page = 1 << p.page_shift;
  // of several children on one row the first is made
  for (int64_t i = c_lo + threadIdx.x; i < c_hi; i += kThreads) {
    const int d = p.dst[i];
    if (d >= 0 && d < p.B) p.claim[d] = 0x7FFFFFFF;
  }
  team.sync();
  for (int64_t i = c_lo + threadIdx.x; i < c_hi; i += kThreads) {
    const int d = p.dst[i];
    if (d >= 0 && d < p.B) atomicMin(p.claim + d, (int)i);
  }
  const int nfree = count_free(p.refs, f_lo, f_hi, sh);
  team.sync();
  int need = 0;
  for (int64_t i = c_lo + threadIdx.x; i < c_hi; i += kThreads) {
    const int s = p.src[i], d = p.dst[i];
    ForkChild ch{-1, 0, -1, -1};
    if (s >= 0 && s < p.B && d >= 0 && d < p.B && s != d) {
      // (asked for together)
      const int claim = __ldcg(p.claim + d), d_len = p.lens[d], len = p.lens[s];
      const int first = p.table[(int64_t)d * p.width];
      if (claim == (int)i && d_len == 0 && first < 0 && len >= 0) {
        const int full = len >> p.page_shift;
        const bool part = (len & (page - 1)) != 0;
        if (full + (part ? 1 : 0) <= p.width) {
          const int last = part ? p.table[(int64_t)s * p.width + full] : -1;
          if (!part || (last >= 0 && last < p.n_pages)) {
            ch = ForkChild{len, full, last, -1};
            need += part;
          }
        }
      }
    }
    p.child[i] = ch;
  }
  need = cta_sum(need, sh);
  int before[2], all[2];
  team.sums(slot, need, nfree, before, all);
  take_free(p.refs, f_lo, f_hi, before[1], all[0], p.order, sh);
  team.sync();
  int bad = 0, at = before[0];
  for (int64_t i0 = c_lo; i0 < c_hi; i0 += kThreads) {
    const int64_t i = i0 + threadIdx.x;
    ForkChild ch{-1, 0, -1, -1};
    if (i < c_hi) ch = p.child[i];
    int sum;
    const int k = at + cta_scan(ch.last >= 0, sh, &sum);
    at += sum;
    if (i < c_hi) {
      if (ch.last >= 0) {
        if (k < all[1])
          ch.fresh = __ldcg(p.order + k);
        else
          ch = ForkChild{-1, 0, -1, -1};
        p.child[i] = ch;
      }
      bad += ch.len < 0;
    }
  }
  bad = cta_sum(bad, sh);
  team.sums(slot + 2, bad, 0, before, all);
  if (team.rank == 0 && threadIdx.x == 0) *p.missing = all[0];
  if constexpr (C > 1) team.sync();
}

// One CTA per child and slice of the copied page; slice 0 writes the table row.
__global__ void __launch_bounds__(256) k_pages_fork_apply(const PagesParams p, int slices) {
  const int64_t i = blockIdx.x / slices;
  const int sl = (int)(blockIdx.x % slices);
  const ForkChild ch = p.child[i];
  if (ch.len < 0) return;
  if (ch.fresh >= 0) {
    const int64_t lo = (int64_t)sl * kSlice, hi = min(lo + (int64_t)kSlice, p.page_bytes);
    const uint4* s = reinterpret_cast<const uint4*>(p.pages + (int64_t)ch.last * p.page_bytes + lo);
    uint4* d = reinterpret_cast<uint4*>(p.pages + (int64_t)ch.fresh * p.page_bytes + lo);
    const int n = (int)((hi - lo) >> 4);
    constexpr int kPer = kSlice / 16 / 256;
    uint4 v[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      if (threadIdx.x + x * 256 < n) v[x] = s[threadIdx.x + x * 256];
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      if (threadIdx.x + x * 256 < n) d[threadIdx.x + x * 256] = v[x];
  }
  if (sl != 0) return;
  const int32_t* from = p.table + (int64_t)p.src[i] * p.width;
  int32_t* to = p.table + (int64_t)p.dst[i] * p.width;
  for (int e = threadIdx.x; e < ch.full; e += 256) {
    const int pg = from[e];
    to[e] = pg;
    if (pg >= 0 && pg < p.n_pages) atomicAdd(p.refs + pg, 1);
  }
  if (threadIdx.x == 0) {
    if (ch.fresh >= 0) to[ch.full] = ch.fresh;
    p.lens[p.dst[i]] = ch.len;
  }
}

// ---------------------------------------------------------------- compact
// With L live pages, the free pages below L (holes, ascending) take the live
// pages from L on (movers, ascending).  lr[p]: live pages before p, as ~lr for
// a free page; hole[h]: the h-th hole; mover[r], mref[r]: the page that r live
// pages precede, and its count, for pages from L on.
template <int C>
__global__ void __launch_bounds__(kThreads) k_pages_compact_plan(const PagesParams p) {
  __shared__ int sh[32], slot[4];
  const Team<C> team;
  const int64_t lo = team.from(p.n_pages), hi = team.to(p.n_pages);
  int c = 0;
  for (int64_t i = lo + 4 * threadIdx.x; i < hi; i += 4 * kThreads) {
    const int4 v = four(p.refs, i, hi, 0);
    c += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
  }
  int before[2], all[2];
  team.sums(slot, cta_sum(c, sh), 0, before, all);
  const int L = all[0];
  int rank = before[0], holes = 0;
  for (int64_t at = lo; at < hi; at += 4 * kThreads) {
    const int64_t i = at + 4 * threadIdx.x;
    const int4 v = four(p.refs, i, hi, 0);
    const int ref[4] = {v.x, v.y, v.z, v.w};
    int n, r = rank + cta_scan((v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0), sh, &n);
    rank += n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t pg = i + e;
      if (pg >= hi) break;
      const bool f = ref[e] > 0;
      p.lr[pg] = f ? r : ~r;
      if (pg < L && !f) {
        p.hole[pg - r] = (int32_t)pg;
        ++holes;
      }
      if (pg >= L && f) {
        p.mover[r] = (int32_t)pg;
        p.mref[r] = ref[e];
      }
      r += f;
    }
  }
  team.sums(slot + 2, cta_sum(holes, sh), 0, before, all);
  if (team.rank == 0 && threadIdx.x == 0) {
    p.missing[0] = L;
    p.moves[0] = all[0];
  }
  if constexpr (C > 1) team.sync();
}

// Copies the movers, writes the new counts and renames the table's pages.
__global__ void __launch_bounds__(256) k_pages_compact_apply(const PagesParams p, int slices) {
  const int L = p.missing[0], M = p.moves[0];
  const int64_t units = (int64_t)M * slices;
  constexpr int kPer = kSlice / 16 / 256;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t i = u / slices;
    const int64_t lo = u % slices * kSlice, hi = min(lo + (int64_t)kSlice, p.page_bytes);
    const uint4* s =
        reinterpret_cast<const uint4*>(p.pages + (int64_t)p.mover[L - M + i] * p.page_bytes + lo);
    uint4* d = reinterpret_cast<uint4*>(p.pages + (int64_t)p.hole[i] * p.page_bytes + lo);
    const int n = (int)((hi - lo) >> 4);
    uint4 v[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      if (threadIdx.x + x * 256 < n) v[x] = __ldcs(s + threadIdx.x + x * 256);
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      if (threadIdx.x + x * 256 < n) __stcs(d + threadIdx.x + x * 256, v[x]);
  }
  const int64_t stride = (int64_t)gridDim.x * 256, t0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = t0; i < p.n_pages; i += stride) {
    const int r = p.lr[i];
    p.refs_out[i] = i >= L ? 0 : (r >= 0 ? p.refs[i] : p.mref[L - M + (i - ~r)]);
  }
  for (int64_t i = t0; i < (int64_t)p.B * p.width; i += stride) {
    const int pg = p.table[i];
    int to = pg;
    if (pg >= 0 && pg < p.n_pages) {
      const int r = p.lr[pg];
      to = r < 0 ? -1 : (pg < L ? pg : p.hole[r - (L - M)]);
    }
    p.table_out[i] = to;
  }
}

// ---------------------------------------------------------------- launches
// One CTA for up to so many pages (and four times as many table entries): four
// rounds of its threads.  A cluster's barriers cost about a microsecond each.
constexpr int kOneCta = 4 * 4 * kThreads;

template <class K>
static cudaError_t launch_team(K one, K many, bool small, const PagesParams& p,
                               cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(small ? 1 : kClu);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kClu;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = small ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, small ? one : many, p);
}

cudaError_t launch_pages_extend(const PagesParams& p, cudaStream_t stream) {
  const bool small = p.n_pages <= kOneCta && (int64_t)p.B * p.width <= 4 * kOneCta;
  return launch_team(k_pages_extend<1>, k_pages_extend<kClu>, small, p, stream);
}

cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t stream) {
  if (p.n == 0) return cudaSuccess;
  k_pages_free<<<p.n, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream) {
  const bool small = p.n_pages <= kOneCta && p.n <= 4 * kThreads;
  const cudaError_t e =
      launch_team(k_pages_fork_plan<1>, k_pages_fork_plan<kClu>, small, p, stream);
  if (e != cudaSuccess || p.n == 0) return e;
  const int slices = (int)((p.page_bytes + kSlice - 1) / kSlice);
  k_pages_fork_apply<<<(unsigned)((int64_t)p.n * slices), 256, 0, stream>>>(p, slices);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t stream) {
  const cudaError_t e = launch_team(k_pages_compact_plan<1>, k_pages_compact_plan<kClu>,
                                    p.n_pages <= kOneCta, p, stream);
  if (e != cudaSuccess) return e;
  const int slices = (int)((p.page_bytes + kSlice - 1) / kSlice);
  k_pages_compact_apply<<<sms * 8, 256, 0, stream>>>(p, slices);
  return cudaGetLastError();
}

}  // namespace si
