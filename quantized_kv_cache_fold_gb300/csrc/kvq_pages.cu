// The page pool of the int4 cache (one reference count per page), the copying of pages, and the
// commit of a draft tree's accepted branch.
//
// Counts and tables: small integer work, bound by latency. Every call that hands out pages runs as
// one thread-block cluster: each warp counts the free pages of a contiguous part of the counts, the
// CTAs exchange their totals through distributed shared memory, and each warp then knows the rank
// of every free page it holds; a page of rank r goes to request r (a binary search over the
// requests' prefix sums). So the lowest free pages are handed out in order whatever the timing, in
// one launch, with no lists or locks kept between calls.
//
// Data: kvq_pages_copy and the commits move bytes; both take all layers in one launch.

#include <algorithm>
#include <mutex>

#include <cooperative_groups.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kPoolCtas = 8;  // the portable cluster size
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Inclusive sum over the CTA of one value per thread; `warp_sums` is shared [kPoolWarps].
__device__ __forceinline__ long long block_inclusive(long long v, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // warp_sums may still be read from an earlier use
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  return v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// The contiguous part [lo, hi) of `n` pages that this warp of the cluster walks: multiples of 128,
// so that every lane reads 16 aligned bytes.
__device__ __forceinline__ void warp_part(int n, int& lo, int& hi) {
  const int w = cluster_ctarank() * kPoolWarps + (threadIdx.x >> 5);
  const long long units = ((long long)n + 127) / 128, nw = kPoolCtas * kPoolWarps;
  lo = (int)min((long long)n, units * w / nw * 128);
  hi = (int)min((long long)n, units * (w + 1) / nw * 128);
}

// Counts of pages p .. p + 3 (p a multiple of 4); 1 beyond hi, so that none of those is free.
__device__ __forceinline__ int4 load_refs4(const int32_t* refs, int p, int hi, bool vec) {
  if (vec && p + 3 < hi) return __ldcg(reinterpret_cast<const int4*>(refs + p));
  int4 r = make_int4(1, 1, 1, 1);
  if (p < hi) r.x = __ldcg(refs + p);
  if (p + 1 < hi) r.y = __ldcg(refs + p + 1);
  if (p + 2 < hi) r.z = __ldcg(refs + p + 2);
  if (p + 3 < hi) r.w = __ldcg(refs + p + 3);
  return r;
}

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Exclusive sum of one value per warp over the cluster's warps in order (all lanes of a warp pass the
// same v), and the total. Contains one cluster barrier: every thread of every CTA calls it, once with one `s`; a
// CTA may leave only after a later cluster barrier (others still read its total).
struct ClusterScan {
  long long warp_sums[kPoolWarps];
  long long cta_total;
};
__device__ __forceinline__ long long cluster_exclusive(int v, ClusterScan& s, long long& total) {
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const long long incl = block_inclusive(lane == 31 ? v : 0, s.warp_sums);  // lane 31 closes each warp's sum
  const long long mine = __shfl_sync(0xffffffffu, incl, 31) - v;
  if (threadIdx.x == 0) s.cta_total = s.warp_sums[kPoolWarps - 1];
  cl.sync();
  const long long t = lane < kPoolCtas ? *cl.map_shared_rank(&s.cta_total, lane) : 0;
  long long before = 0;
  total = 0;
#pragma unroll
  for (int r = 0; r < kPoolCtas; ++r) {
    const long long x = __shfl_sync(0xffffffffu, t, r);
    if (r < (int)cluster_ctarank()) before += x;
    total += x;
  }
  return before + mine;
}

// Calls f(page, rank) for this warp's free pages in ascending order while rank < limit.
template <class F>
__device__ __forceinline__ void for_free_pages(const int32_t* refs, int lo, int hi, bool vec, long long rank,
                                               long long limit, F f) {
  const int lane = threadIdx.x & 31;
  for (int p0 = lo; p0 < hi && rank < limit; p0 += 128) {
    const int p = p0 + 4 * lane;
    const int4 r = load_refs4(refs, p, hi, vec);
    const int z[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    int c = z[0] + z[1] + z[2] + z[3];
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    long long k = rank + incl - c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (z[i] && k < limit) f(p + i, k);
      k += z[i];
    }
    rank += __shfl_sync(0xffffffffu, incl, 31);
  }
}

__device__ __forceinline__ int count_free(const int32_t* refs, int lo, int hi, bool vec) {
  int c = 0;
#pragma unroll 4
  for (int p = lo + 4 * (threadIdx.x & 31); p < hi; p += 128) {
    const int4 r = load_refs4(refs, p, hi, vec);
    c += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  return warp_sum_int(c);
}

// Whether ids[j] == id for some j < end (ids in shared memory; end per thread).
__device__ __forceinline__ bool named_before(const int32_t* ids, int id, int end) {
  bool hit = false;
#pragma unroll 8
  for (int j = 0; j < end; ++j) hit |= ids[j] == id;
  return hit;
}

struct PoolParams {
  int32_t* refs;
  int num_pages;
  int32_t* table;
  int num_seqs, max_pages;
  int n;
  const int32_t *a, *b, *c;  // alloc and free: ids, old and new length; fork: parents, children, length
  int32_t *src, *dst, *moves;
  int32_t* dev_err;
};

// Request r (0..need-1) -> the index i whose prefix range [pre[i-1], pre[i]) holds r.
__device__ __forceinline__ int request_of(const long long* pre, int n, long long r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

struct PoolSmem {
  ClusterScan scan;
  long long sums[kPoolWarps];
  long long pre[KVQ_MAX_SEQS];  // inclusive sums of the requests' pages
  int32_t id[KVQ_MAX_SEQS];
  int32_t id2[KVQ_MAX_SEQS];
};

__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    pages_alloc_kernel(const PoolParams p) {
  __shared__ PoolSmem s;
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const bool in = t < p.n;
  const int id = in ? p.a[t] : -1, l0 = in ? p.b[t] : 0, l1 = in ? p.c[t] : 0;
  s.id[t] = id;
  __syncthreads();
  bool ok = in && id >= 0 && id < p.num_seqs && l0 >= 0 && l1 >= 0 && l0 <= p.max_pages * kPage &&
            l1 <= p.max_pages * kPage && !named_before(s.id, id, t);
  if (in && !ok && cluster_ctarank() == 0) set_err(p.dev_err, KVQ_DEVERR_POS);
  const int first = pages_of(l0), cnt = ok ? max(0, pages_of(l1) - first) : 0;
  s.pre[t] = block_inclusive(cnt, s.sums);
  s.id2[t] = first;
  __syncthreads();
  const long long need = p.n > 0 ? s.pre[p.n - 1] : 0;
  int lo, hi;
  warp_part(p.num_pages, lo, hi);
  const bool vec = (reinterpret_cast<uintptr_t>(p.refs) & 15) == 0;
  long long free_total;
  const long long rank = cluster_exclusive(count_free(p.refs, lo, hi, vec), s.scan, free_total);
  for_free_pages(p.refs, lo, hi, vec, rank, need, [&](int page, long long r) {
    const int i = request_of(s.pre, p.n, r);
    const int at = s.id2[i] + (int)(r - (i > 0 ? s.pre[i - 1] : 0));
    p.table[(size_t)s.id[i] * p.max_pages + at] = page;
    p.refs[page] = 1;
  });
  if (free_total < need) {
    if (cluster_ctarank() == 0 && t == 0) set_err(p.dev_err, KVQ_DEVERR_POOL);
    for (long long r = free_total + cluster_ctarank() * kPoolThreads + t; r < need; r += kPoolCtas * kPoolThreads) {
      const int i = request_of(s.pre, p.n, r);
      const int at = s.id2[i] + (int)(r - (i > 0 ? s.pre[i - 1] : 0));
      p.table[(size_t)s.id[i] * p.max_pages + at] = -1;
    }
  }
  cg::this_cluster().sync();  // this CTA's total may still be read
}

__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    pages_fork_kernel(const PoolParams p) {
  __shared__ PoolSmem s;
  __shared__ int32_t lens[KVQ_MAX_SEQS];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const bool in = t < p.n;
  const int par = in ? p.a[t] : -1, ch = in ? p.b[t] : -1, len = in ? p.c[t] : 0;
  s.id[t] = ch;
  s.id2[t] = par;
  __syncthreads();
  // a row forked from in this call cannot be a child of it as well: the child is refused
  bool ok = in && par >= 0 && par < p.num_seqs && ch >= 0 && ch < p.num_seqs && len >= 0 &&
            len <= p.max_pages * kPage && !named_before(s.id, ch, t) && !named_before(s.id2, ch, p.n);
  if (in && !ok && cluster_ctarank() == 0) set_err(p.dev_err, KVQ_DEVERR_POS);
  int32_t tail_src = -1;  // pages with count 0 are nobody's to share or copy
  if (ok && len % kPage) {
    tail_src = p.table[(size_t)par * p.max_pages + len / kPage];
    if (tail_src < 0 || tail_src >= p.num_pages || __ldcg(p.refs + tail_src) <= 0) {
      tail_src = -1;
      if (cluster_ctarank() == 0) {
        set_err(p.dev_err, KVQ_DEVERR_PAGE);
        p.table[(size_t)ch * p.max_pages + len / kPage] = -1;
      }
    }
  }
  lens[t] = ok ? len : 0;
  s.pre[t] = block_inclusive(tail_src >= 0 ? 1 : 0, s.sums);
  __syncthreads();
  const long long need = p.n > 0 ? s.pre[p.n - 1] : 0;
  if (in && cluster_ctarank() == 0) {
    p.src[t] = tail_src;
    if (tail_src < 0) p.dst[t] = -1;
  }
  // full pages, shared: counts above 0 go up, which leaves the free pages as they are
  for (int i = cluster_ctarank() * kPoolWarps + (t >> 5); i < p.n; i += kPoolCtas * kPoolWarps) {
    const int full = lens[i] / kPage;
    if (full == 0) continue;
    const int32_t* from = p.table + (size_t)s.id2[i] * p.max_pages;
    int32_t* to = p.table + (size_t)s.id[i] * p.max_pages;
    for (int k = t & 31; k < full; k += 32) {
      int page = from[k];
      if (page < 0 || page >= p.num_pages || __ldcg(p.refs + page) <= 0) {
        set_err(p.dev_err, KVQ_DEVERR_PAGE);
        page = -1;
      } else {
        atomicAdd(p.refs + page, 1);
      }
      to[k] = page;
    }
  }
  int lo, hi;
  warp_part(p.num_pages, lo, hi);
  const bool vec = (reinterpret_cast<uintptr_t>(p.refs) & 15) == 0;
  long long free_total;
  const long long rank = cluster_exclusive(count_free(p.refs, lo, hi, vec), s.scan, free_total);
  // every share came before the exchange's barriers, so no dead entry of a parent's can meet a new page
  for_free_pages(p.refs, lo, hi, vec, rank, need, [&](int page, long long r) {
    const int i = request_of(s.pre, p.n, r);
    p.table[(size_t)s.id[i] * p.max_pages + lens[i] / kPage] = page;
    p.dst[i] = page;
    p.refs[page] = 1;
  });
  if (tail_src >= 0 && s.pre[t] > free_total && cluster_ctarank() == 0) {
    set_err(p.dev_err, KVQ_DEVERR_POOL);
    p.table[(size_t)ch * p.max_pages + len / kPage] = -1;
    p.dst[t] = -1;
  }
  cg::this_cluster().sync();  // this CTA's total may still be read
}

// One block per request; a row named by an earlier request as well is that one's.
__global__ void __launch_bounds__(128) pages_free_kernel(const PoolParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  const int id = p.a[i], l0 = p.b[i], l1 = p.c[i];
  const int most = p.max_pages * kPage;
  if (id < 0 || id >= p.num_seqs || l0 < 0 || l0 > most || l1 < 0 || l1 > most) {
    if (threadIdx.x == 0) set_err(p.dev_err, KVQ_DEVERR_POS);
    return;
  }
  bool twice = false;
  for (int j = threadIdx.x; j < i; j += blockDim.x) twice |= p.a[j] == id;
  if (__syncthreads_or(twice)) {
    if (threadIdx.x == 0) set_err(p.dev_err, KVQ_DEVERR_POS);
    return;
  }
  int32_t* row = p.table + (size_t)id * p.max_pages;
  for (int k = pages_of(l1) + threadIdx.x; k < pages_of(l0); k += blockDim.x) {
    const int page = row[k];
    if (page < 0 || page >= p.num_pages) {
      set_err(p.dev_err, KVQ_DEVERR_PAGE);
      continue;
    }
    row[k] = -1;
    if (atomicSub(p.refs + page, 1) <= 0) {
      atomicAdd(p.refs + page, 1);
      set_err(p.dev_err, KVQ_DEVERR_POOL);
    }
  }
}

// Every entry that names a moved page, by a search in the ascending list of sources; entries e, e + step, ...
__device__ __forceinline__ void remap(const PoolParams& p, int moves, long long e, long long step) {
  if (moves == 0) return;
  const int first = __ldcg(p.src);
  const long long n = (long long)p.num_seqs * p.max_pages;
  for (; e < n; e += step) {
    const int v = p.table[e];
    if (v < first || v >= p.num_pages) continue;
    int lo = 0, hi = moves - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(p.src + mid) < v) lo = mid + 1;
      else hi = mid;
    }
    if (__ldcg(p.src + lo) == v) p.table[e] = __ldcg(p.dst + lo);
    else set_err(p.dev_err, KVQ_DEVERR_PAGE);  // a page that nobody holds
  }
}

// Tables up to this many entries are rewritten by the cluster itself (8 entries a thread at most, less than the
// second launch costs: 2,600 pages, 6,048 entries, compact and copy 29.9 -> 28.8 us), larger ones by a launch
// over the whole GPU.
constexpr long long kClusterTable = 1 << 16;

// The moves: the k-th page in use at or behind L goes to the k-th free page before L.
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    pages_compact_kernel(const PoolParams p) {
  __shared__ ClusterScan scan, scan2;
  griddep_wait();
  griddep_launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  int lo, hi;
  warp_part(p.num_pages, lo, hi);
  const bool vec = (reinterpret_cast<uintptr_t>(p.refs) & 15) == 0;
  const int nfree = count_free(p.refs, lo, hi, vec);
  long long total;
  const long long before = cluster_exclusive(nfree, scan, total);
  const int L = p.num_pages - (int)total;
  // free pages before L in this warp's part and in all parts; a free page's rank in front is its rank
  // among all free pages, since only free pages behind L come after
  int fl = 0;
  for (int q = lo + 4 * lane; q < min(hi, L); q += 128) {
    const int4 r = load_refs4(p.refs, q, hi, vec);
    fl += (r.x == 0 && q < L) + (r.y == 0 && q + 1 < L) + (r.z == 0 && q + 2 < L) + (r.w == 0 && q + 3 < L);
  }
  fl = warp_sum_int(fl);
  long long moves;
  cluster_exclusive(fl, scan2, moves);
  for_free_pages(p.refs, lo, min(hi, L), vec, before, moves, [&](int page, long long k) { p.dst[k] = page; });
  // a page in use at q >= L has rank (pages in use before q) - (L - moves)
  long long rank = (long long)lo - before - (L - moves);
  for (int q0 = lo; q0 < hi; q0 += 128) {
    const int q = q0 + 4 * lane;
    const int4 r = load_refs4(p.refs, q, hi, vec);
    const int z[4] = {q < hi && r.x != 0, q + 1 < hi && r.y != 0, q + 2 < hi && r.z != 0, q + 3 < hi && r.w != 0};
    const int c = z[0] + z[1] + z[2] + z[3];
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    long long k = rank + incl - c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (z[i] && q + i >= L) p.src[k] = q + i;
      k += z[i];
    }
    rank += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (cluster_ctarank() == 0 && threadIdx.x == 0) *p.moves = (int)moves;
  __threadfence();
  cl.sync();  // the lists are complete (and no warp still reads the counts)
  for (long long k = cluster_ctarank() * kPoolThreads + threadIdx.x; k < moves; k += kPoolCtas * kPoolThreads) {
    const int from = __ldcg(p.src + k), to = __ldcg(p.dst + k);
    p.refs[to] = __ldcg(p.refs + from);
    p.refs[from] = 0;
  }
  if ((long long)p.num_seqs * p.max_pages <= kClusterTable)
    remap(p, (int)moves, cluster_ctarank() * kPoolThreads + threadIdx.x, kPoolCtas * kPoolThreads);
}

__global__ void __launch_bounds__(256) pages_remap_kernel(const PoolParams p) {
  griddep_wait();
  griddep_launch_dependents();
  remap(p, *p.moves, (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}

// ------------------------------------------------------------------ data

// One block per (pair, layer, KV head) at a time: 8704 bytes, 544 16-byte words.
constexpr int kCopyThreads = 272;  // two words a thread
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CacheSet cs, int n, const int32_t* src, const int32_t* dst,
                                                                  const int32_t* count, int32_t* dev_err) {
  griddep_wait();
  griddep_launch_dependents();
  const int m = count ? min(n, max(0, *count)) : n;
  const long long items = (long long)m * cs.count * cs.heads;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int h = (int)(it % cs.heads);
    const int l = (int)(it / cs.heads % cs.count);
    const int i = (int)(it / cs.heads / cs.count);
    const int a = src[i], b = dst[i];
    if (a == -1 || b == -1 || a == b) continue;
    if (a < 0 || a >= cs.num_pages[l] || b < 0 || b >= cs.num_pages[l]) {
      if (threadIdx.x == 0) set_err(dev_err, KVQ_DEVERR_PAGE);
      continue;
    }
    const uint4* from = reinterpret_cast<const uint4*>(cs.pages[l] + ((size_t)a * cs.heads + h) * KVQ_INT4_BLOCK_BYTES);
    uint4* to = reinterpret_cast<uint4*>(cs.pages[l] + ((size_t)b * cs.heads + h) * KVQ_INT4_BLOCK_BYTES);
    const uint4 x = __ldcs(from + threadIdx.x), y = __ldcs(from + kCopyThreads + threadIdx.x);
    to[threadIdx.x] = x;
    to[kCopyThreads + threadIdx.x] = y;
  }
}

// One block per (sequence, KV head) and two layers. The accepted records' 16-byte chunks (8 of an int4 record,
// 16 of an e4m3 one) go through registers, every load of a pass before any store. A branch of a tree names
// its tokens in ascending order, so a source never lies before its target: passes of 16 or 32 records may then
// follow one another. Any other path of more records than a pass holds is read as a whole first
// (commit_any). The chunks sit in a slot-dependent order, so a record moves chunk by chunk, not as bytes.
// Latency-bound: path -> (page) -> chunks -> stores; two layers in flight rather than one
// (64 sequences x 4 heads, up to 16 of 32 tokens, 10 + 40 layers: 19.7 -> 14.3 us; four layers take more
// registers and with them waves: 16.0 us).
constexpr int kCommitThreads = 128, kCommitLayers = 2, kCommitUnits = 2;
constexpr int kMaxPos = 1 << 30;

template <int FMT>
struct CommitAt {
  static constexpr int kChunks = FMT == 0 ? 8 : 16;  // 16-byte chunks of a record, K then V
  const CacheSet& cs;
  int b, h, l;
  int32_t* dev_err;
  // Block of a position, or null.
  __device__ __forceinline__ uint8_t* block(int pos) const {
    if (FMT == 0) {
      if (b >= cs.num_seqs[l] || pos >= cs.max_pages[l] * kPage) {
        set_err(dev_err, KVQ_DEVERR_POS);
        return nullptr;
      }
      const int page = cs.table[l][(size_t)b * cs.max_pages[l] + pos / kPage];
      if (page < 0 || page >= cs.num_pages[l]) {
        set_err(dev_err, KVQ_DEVERR_PAGE);
        return nullptr;
      }
      return cs.pages[l] + ((size_t)page * cs.heads + h) * KVQ_INT4_BLOCK_BYTES;
    }
    const int nblk = cs.max_pages[l];
    return cs.pages[l] + (((size_t)b * cs.heads + h) * nblk + (pos / kPage) % nblk) * (size_t)(2 * kPage * kRec8);
  }
  // Byte of chunk c of the record in a position's slot (a ring's capacity is a multiple of 64).
  static __device__ __forceinline__ size_t chunk(int pos, int c) {
    const int slot = pos % kPage;
    if (FMT == 0) {
      const int half = c >> 2, k = c & 3;
      return (size_t)half * kPage * kRec4 + slot * kRec4 + 16 * (k ^ (half ? (slot >> 1) & 3 : k_chunk_swz(slot)));
    }
    const int half = c >> 3, k = c & 7;
    return (size_t)half * kPage * kRec8 + slot * kRec8 + 16 * (k ^ (slot & 7));
  }
  // Word of the scales and offsets (int4): K or V of the record in a position's slot.
  static __device__ __forceinline__ size_t meta(int pos, int v) { return 2 * kPage * kRec4 + 4 * (v * kPage + pos % kPage); }
};

// Any path: one thread per chunk (and per scale word) of a record takes its chunk of all records, through local memory.
template <int FMT>
__device__ __noinline__ void commit_any(const CommitAt<FMT> at, int ctx, int A, const int32_t* path) {
  const int t = threadIdx.x;
  if (t < CommitAt<FMT>::kChunks) {
    uint4 x[KVQ_MAX_TREE];
#pragma unroll 1
    for (int i = 0; i < A; ++i) {
      const uint8_t* blk = path[i] >= 0 ? at.block(ctx + path[i]) : nullptr;
      if (blk) x[i] = *reinterpret_cast<const uint4*>(blk + at.chunk(ctx + path[i], t));
    }
#pragma unroll 1
    for (int i = 0; i < A; ++i) {
      if (path[i] < 0 || path[i] == i || !at.block(ctx + path[i])) continue;
      uint8_t* blk = at.block(ctx + i);
      if (blk) *reinterpret_cast<uint4*>(blk + at.chunk(ctx + i, t)) = x[i];
    }
  } else if (FMT == 0 && t < CommitAt<FMT>::kChunks + 2) {
    const int v = t - CommitAt<FMT>::kChunks;
    uint32_t x[KVQ_MAX_TREE];
#pragma unroll 1
    for (int i = 0; i < A; ++i) {
      const uint8_t* blk = path[i] >= 0 ? at.block(ctx + path[i]) : nullptr;
      if (blk) x[i] = *reinterpret_cast<const uint32_t*>(blk + at.meta(ctx + path[i], v));
    }
#pragma unroll 1
    for (int i = 0; i < A; ++i) {
      if (path[i] < 0 || path[i] == i || !at.block(ctx + path[i])) continue;
      uint8_t* blk = at.block(ctx + i);
      if (blk) *reinterpret_cast<uint32_t*>(blk + at.meta(ctx + i, v)) = x[i];
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CacheSet cs, int N, const int32_t* ctx_len, const int32_t* path,
                                                                const int32_t* n_accept, int32_t* ctx_out,
                                                                int32_t* dev_err) {
  constexpr int kChunks = CommitAt<FMT>::kChunks;
  constexpr int kRecs = kCommitThreads * kCommitUnits / kChunks;  // records of a pass
  __shared__ int32_t spath[KVQ_MAX_TREE];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / cs.heads, h = blockIdx.x % cs.heads, l0 = blockIdx.y * kCommitLayers;
  const int t = threadIdx.x;
  int x = t < N ? path[(size_t)b * N + t] : 0;
  const int ctx = ctx_len[b], got = n_accept[b];
  const int A = min(max(got, 0), N);
  const bool lead = h == 0 && l0 == 0;  // one block reports a sequence's errors
  if (lead && t == 0) {
    if (ctx_out) ctx_out[b] = ctx + A;
    if (A != got || ctx < 0 || ctx > kMaxPos) set_err(dev_err, KVQ_DEVERR_POS);
  }
  if (ctx < 0 || ctx > kMaxPos) return;
  if (t < KVQ_MAX_TREE) {
    if (t < A && (x < 0 || x >= N)) {
      x = -1;
      if (lead) set_err(dev_err, KVQ_DEVERR_POS);
    }
    spath[t] = x;
  }
  __syncthreads();
  if (A > kRecs) {
    const bool ascending = t >= A || (spath[t] >= t && (t == 0 || spath[t] > spath[t - 1]));
    if (!__syncthreads_and(ascending)) {
      for (int l = l0; l < min(l0 + kCommitLayers, cs.count); ++l) commit_any(CommitAt<FMT>{cs, b, h, l, dev_err}, ctx, A, spath);
      return;
    }
  }
  for (int i0 = 0; i0 < A; i0 += kRecs) {
    uint4 v[kCommitLayers][kCommitUnits];
    uint8_t* dst[kCommitLayers][kCommitUnits];  // null: nothing to move
    uint32_t meta[kCommitLayers];
    uint8_t* mdst[kCommitLayers];
#pragma unroll
    for (int ll = 0; ll < kCommitLayers; ++ll) {
      const CommitAt<FMT> at{cs, b, h, min(l0 + ll, cs.count - 1), dev_err};
#pragma unroll
      for (int u = 0; u < kCommitUnits; ++u) {
        const int i = i0 + (u * kCommitThreads + t) / kChunks, c = t % kChunks;
        dst[ll][u] = nullptr;
        if (l0 + ll < cs.count && i < A && spath[i] >= 0 && spath[i] != i) {
          const uint8_t* from = at.block(ctx + spath[i]);
          uint8_t* to = at.block(ctx + i);
          if (from && to) {
            v[ll][u] = *reinterpret_cast<const uint4*>(from + at.chunk(ctx + spath[i], c));
            dst[ll][u] = to + at.chunk(ctx + i, c);
          }
        }
      }
      mdst[ll] = nullptr;
      if (FMT == 0) {  // thread t: K (t even) or V word of record t / 2
        const int i = i0 + t / 2;
        if (t < 2 * kRecs && l0 + ll < cs.count && i < A && spath[i] >= 0 && spath[i] != i) {
          const uint8_t* from = at.block(ctx + spath[i]);
          uint8_t* to = at.block(ctx + i);
          if (from && to) {
            meta[ll] = *reinterpret_cast<const uint32_t*>(from + at.meta(ctx + spath[i], t & 1));
            mdst[ll] = to + at.meta(ctx + i, t & 1);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int ll = 0; ll < kCommitLayers; ++ll) {
#pragma unroll
      for (int u = 0; u < kCommitUnits; ++u) {
        if (FMT == 1) {  // the place again: cheaper than keeping it
          const CommitAt<FMT> at{cs, b, h, min(l0 + ll, cs.count - 1), dev_err};
          const int i = i0 + (u * kCommitThreads + t) / kChunks;
          if (dst[ll][u]) *reinterpret_cast<uint4*>(at.block(ctx + i) + at.chunk(ctx + i, t % kChunks)) = v[ll][u];
        } else if (dst[ll][u]) {
          *reinterpret_cast<uint4*>(dst[ll][u]) = v[ll][u];
        }
      }
      if (FMT == 0 && mdst[ll]) *reinterpret_cast<uint32_t*>(mdst[ll]) = meta[ll];
    }
    __syncthreads();
  }
}

template <class... A>
cudaError_t launch_pdl(void (*kern)(A...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

PoolParams params(const PoolJob& j) {
  PoolParams p{};
  p.refs = j.page_refs;
  p.num_pages = j.num_pages;
  p.table = j.block_table;
  p.num_seqs = j.num_seqs;
  p.max_pages = j.max_pages_per_seq;
  p.n = j.n;
  p.a = j.a;
  p.b = j.b;
  p.c = j.c;
  p.src = j.copy_src;
  p.dst = j.copy_dst;
  p.moves = j.n_moves;
  p.dev_err = j.dev_err;
  return p;
}

std::mutex g_sms_mu;  // guards the cache below
int g_sms[64] = {0};

}  // namespace

int device_sms() {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  std::lock_guard<std::mutex> lock(g_sms_mu);
  if (g_sms[dev] == 0) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    g_sms[dev] = n > 0 ? n : 1;
  }
  return g_sms[dev];
}

cudaError_t launch_pages_alloc(const PoolJob& j, cudaStream_t stream) {
  return launch_pdl(pages_alloc_kernel, dim3(kPoolCtas), kPoolThreads, stream, params(j));
}

cudaError_t launch_pages_fork(const PoolJob& j, cudaStream_t stream) {
  return launch_pdl(pages_fork_kernel, dim3(kPoolCtas), kPoolThreads, stream, params(j));
}

cudaError_t launch_pages_free(const PoolJob& j, cudaStream_t stream) {
  return launch_pdl(pages_free_kernel, dim3((unsigned)j.n), 128, stream, params(j));
}

cudaError_t launch_pages_compact(const PoolJob& j, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(pages_compact_kernel, dim3(kPoolCtas), kPoolThreads, stream, params(j));
  if (e != cudaSuccess) return e;
  const long long n = (long long)j.num_seqs * j.max_pages_per_seq;
  if (n <= kClusterTable) return e;
  const unsigned grid = (unsigned)std::min<long long>((n + 255) / 256, 8LL * device_sms());
  return launch_pdl(pages_remap_kernel, dim3(grid), 256, stream, params(j));
}

cudaError_t launch_pages_copy(const CacheSet& cs, int n, const int32_t* src, const int32_t* dst, const int32_t* count,
                              int32_t* dev_err, cudaStream_t stream) {
  const long long items = (long long)n * cs.count * cs.heads;
  const unsigned grid = (unsigned)std::min<long long>(items, 7LL * device_sms());
  return launch_pdl(pages_copy_kernel, dim3(grid), kCopyThreads, stream, cs, n, src, dst, count, dev_err);
}

cudaError_t launch_tree_commit(int fmt, const CacheSet& cs, int B, int N, const int32_t* ctx_len, const int32_t* path,
                               const int32_t* n_accept, int32_t* ctx_out, int32_t* dev_err, cudaStream_t stream) {
  const dim3 grid((unsigned)(B * cs.heads), (unsigned)((cs.count + kCommitLayers - 1) / kCommitLayers));
  return launch_pdl(fmt == 0 ? commit_kernel<0> : commit_kernel<1>, grid, kCommitThreads, stream, cs, N, ctx_len, path,
                    n_accept, ctx_out, dev_err);
}

}  // namespace kvq
