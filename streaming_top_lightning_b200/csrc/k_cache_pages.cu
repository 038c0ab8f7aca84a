// The life of a cache's pages: growth, forks, release and compaction.
//
// A pool of n pages has a count per page of the table rows that hold it (0:
// free); a row of the page table lists the pages of one sequence in its leading
// entries, -1 after them.  Every call takes the lowest free pages, in the order
// of its rows, so a result depends on nothing but the inputs.
//
// The counting parts read the counts and tables twice and decide with prefix
// sums over them: one cluster of eight CTAs, each with a contiguous share,
// that exchange their shares' sums through distributed shared memory (one
// launch; a grid-wide scan would take two or three).  They are bound by latency.
// Copies of pages run in a second launch over the whole GPU, HBM-bound.
#include <cooperative_groups.h>

#include "si_attn.cuh"

namespace cg = cooperative_groups;

namespace si {
namespace {

constexpr int kClu = 8;         // CTAs of the counting kernels' cluster
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

// The sums of all CTAs' `mine`: those before this CTA, and all of them.
SI_DEV void cluster_sums(cg::cluster_group& cl, int* slot, int mine, int* before, int* all) {
  if (threadIdx.x == 0) *slot = mine;
  cl.sync();
  int b = 0, t = 0;
  const unsigned rank = cl.block_rank();
#pragma unroll
  for (unsigned i = 0; i < kClu; ++i) {
    const int v = *cl.map_shared_rank(slot, i);
    if (i < rank) b += v;
    t += v;
  }
  *before = b;
  *all = t;
}

SI_DEV int64_t share(int64_t n, unsigned rank) { return n * rank / kClu; }

// Free pages among refs [lo, hi).
SI_DEV int count_free(const int32_t* refs, int64_t lo, int64_t hi, int* sh) {
  int c = 0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) c += refs[i] == 0;
  return cta_sum(c, sh);
}

// Gives the free pages of [lo, hi) their ranks from `rank` on: the pages ranked
// below `need` go to order[rank] and get one holder.
SI_DEV void take_free(int32_t* refs, int64_t lo, int64_t hi, int rank, int need, int32_t* order,
                      int* sh) {
  for (int64_t at = lo; at < hi && rank < need; at += kThreads) {
    const int64_t i = at + threadIdx.x;
    const int f = i < hi && refs[i] == 0;
    int n;
    const int r = rank + cta_scan(f, sh, &n);
    if (f && r < need) {
      order[r] = (int32_t)i;
      refs[i] = 1;
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
__global__ void __cluster_dims__(kClu, 1, 1) __launch_bounds__(kThreads)
    k_pages_extend(const PagesParams p) {
  __shared__ int sh[32];
  __shared__ int x_want, x_free;
  cg::cluster_group cl = cg::this_cluster();
  const unsigned rank = cl.block_rank();
  const int64_t r_lo = share(p.B, rank), r_hi = share(p.B, rank + 1);
  const int64_t f_lo = share(p.n_pages, rank), f_hi = share(p.n_pages, rank + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // what this CTA's rows want: a warp a row
  int c = 0;
  for (int64_t r = r_lo + warp; r < r_hi; r += kThreads / 32) {
    const int n = pages_of(p.lens[r], p.page_shift, p.width);
    for (int e = lane; e < n; e += 32) c += p.table[r * p.width + e] < 0;
  }
  const int want = cta_sum(c, sh);
  const int nfree = count_free(p.refs, f_lo, f_hi, sh);
  int want_before, want_all, free_before, free_all;
  cluster_sums(cl, &x_want, want, &want_before, &want_all);
  cluster_sums(cl, &x_free, nfree, &free_before, &free_all);
  take_free(p.refs, f_lo, f_hi, free_before, want_all, p.order, sh);
  __threadfence();
  cl.sync();
  // rows in order: each row's wants are a prefix sum over the CTA's rows
  int at = want_before;
  for (int64_t r0 = r_lo; r0 < r_hi; r0 += kThreads / 32) {
    const int64_t r = r0 + warp;
    int n = 0, cnt = 0;
    if (r < r_hi) {
      n = pages_of(p.lens[r], p.page_shift, p.width);
      for (int e = lane; e < n; e += 32) cnt += p.table[r * p.width + e] < 0;
    }
    cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
    int all;
    int mine = at + cta_scan(lane == 0 ? cnt : 0, sh, &all);
    mine = __shfl_sync(0xFFFFFFFFu, mine, 0);
    if (cnt) {
      for (int e0 = 0; e0 < n; e0 += 32) {
        const int e = e0 + lane;
        const bool w = e < n && p.table[r * p.width + e] < 0;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, w);
        const int k = mine + __popc(m & ((1u << lane) - 1u));
        if (w && k < free_all) p.table[r * p.width + e] = __ldcg(p.order + k);
        mine += __popc(m);
      }
    }
    at += all;
  }
  if (rank == 0 && threadIdx.x == 0) *p.missing = want_all > free_all ? want_all - free_all : 0;
  cl.sync();  // no CTA leaves while another reads its shared memory
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
__global__ void __cluster_dims__(kClu, 1, 1) __launch_bounds__(kThreads)
    k_pages_fork_plan(const PagesParams p) {
  __shared__ int sh[32];
  __shared__ int x_need, x_free, x_bad;
  cg::cluster_group cl = cg::this_cluster();
  const unsigned rank = cl.block_rank();
  const int64_t c_lo = share(p.n, rank), c_hi = share(p.n, rank + 1);
  const int64_t f_lo = share(p.n_pages, rank), f_hi = share(p.n_pages, rank + 1);
  const int page = 1 << p.page_shift;
  // of several children on one row the first is made
  for (int64_t i = c_lo + threadIdx.x; i < c_hi; i += kThreads) {
    const int d = p.dst[i];
    if (d >= 0 && d < p.B) p.claim[d] = 0x7FFFFFFF;
  }
  __threadfence();
  cl.sync();
  for (int64_t i = c_lo + threadIdx.x; i < c_hi; i += kThreads) {
    const int d = p.dst[i];
    if (d >= 0 && d < p.B) atomicMin(p.claim + d, (int)i);
  }
  const int nfree = count_free(p.refs, f_lo, f_hi, sh);
  __threadfence();
  cl.sync();
  int need = 0;
  for (int64_t i = c_lo + threadIdx.x; i < c_hi; i += kThreads) {
    const int s = p.src[i], d = p.dst[i];
    ForkChild ch{-1, 0, -1, -1};
    if (s >= 0 && s < p.B && d >= 0 && d < p.B && s != d && __ldcg(p.claim + d) == (int)i &&
        p.lens[d] == 0 && p.table[(int64_t)d * p.width] < 0) {
      const int len = p.lens[s];
      const int full = len > 0 ? len >> p.page_shift : 0;
      const bool part = len > 0 && (len & (page - 1)) != 0;
      if (len >= 0 && full + (part ? 1 : 0) <= p.width) {
        const int last = part ? p.table[(int64_t)s * p.width + full] : -1;
        if (!part || (last >= 0 && last < p.n_pages)) {
          ch = ForkChild{len, full, last, -1};
          need += part;
        }
      }
    }
    p.child[i] = ch;
  }
  need = cta_sum(need, sh);
  int need_before, need_all, free_before, free_all;
  cluster_sums(cl, &x_need, need, &need_before, &need_all);
  cluster_sums(cl, &x_free, nfree, &free_before, &free_all);
  take_free(p.refs, f_lo, f_hi, free_before, need_all, p.order, sh);
  __threadfence();
  cl.sync();
  int bad = 0, at = need_before;
  for (int64_t i0 = c_lo; i0 < c_hi; i0 += kThreads) {
    const int64_t i = i0 + threadIdx.x;
    ForkChild ch{-1, 0, -1, -1};
    if (i < c_hi) ch = p.child[i];
    int all;
    const int k = at + cta_scan(ch.last >= 0, sh, &all);
    at += all;
    if (i < c_hi) {
      if (ch.last >= 0) {
        if (k < free_all)
          ch.fresh = __ldcg(p.order + k);
        else
          ch = ForkChild{-1, 0, -1, -1};
        p.child[i] = ch;
      }
      bad += ch.len < 0;
    }
  }
  bad = cta_sum(bad, sh);
  int bad_before, bad_all;
  cluster_sums(cl, &x_bad, bad, &bad_before, &bad_all);
  if (rank == 0 && threadIdx.x == 0) *p.missing = bad_all;
  cl.sync();
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
__global__ void __cluster_dims__(kClu, 1, 1) __launch_bounds__(kThreads)
    k_pages_compact_plan(const PagesParams p) {
  __shared__ int sh[32];
  __shared__ int x_live, x_hole;
  cg::cluster_group cl = cg::this_cluster();
  const unsigned rank = cl.block_rank();
  const int64_t lo = share(p.n_pages, rank), hi = share(p.n_pages, rank + 1);
  int c = 0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) c += p.refs[i] > 0;
  const int live = cta_sum(c, sh);
  int before, L;
  cluster_sums(cl, &x_live, live, &before, &L);
  int holes = 0;
  for (int64_t at = lo; at < hi; at += kThreads) {
    const int64_t i = at + threadIdx.x;
    const int ref = i < hi ? p.refs[i] : 0;
    const int f = ref > 0;
    int n;
    const int r = before + cta_scan(f, sh, &n);
    before += n;
    if (i < hi) {
      p.lr[i] = f ? r : ~r;
      if (i < L && !f) {
        p.hole[i - r] = (int32_t)i;
        ++holes;
      }
      if (i >= L && f) {
        p.mover[r] = (int32_t)i;
        p.mref[r] = ref;
      }
    }
  }
  holes = cta_sum(holes, sh);
  int b, M;
  cluster_sums(cl, &x_hole, holes, &b, &M);
  if (rank == 0 && threadIdx.x == 0) {
    p.missing[0] = L;
    p.moves[0] = M;
  }
  cl.sync();
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
cudaError_t launch_pages_extend(const PagesParams& p, cudaStream_t stream) {
  k_pages_extend<<<kClu, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t stream) {
  if (p.n == 0) return cudaSuccess;
  k_pages_free<<<p.n, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream) {
  k_pages_fork_plan<<<kClu, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.n == 0) return e;
  const int slices = (int)((p.page_bytes + kSlice - 1) / kSlice);
  k_pages_fork_apply<<<(unsigned)((int64_t)p.n * slices), 256, 0, stream>>>(p, slices);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t stream) {
  k_pages_compact_plan<<<kClu, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int slices = (int)((p.page_bytes + kSlice - 1) / kSlice);
  k_pages_compact_apply<<<sms * 8, 256, 0, stream>>>(p, slices);
  return cudaGetLastError();
}

}  // namespace si
