// Eviction from the int4 caches by gathered attention weight (kvq_evict_int4), and the masses that appended tokens start from
// (kvq_mass_start).
//
// Per layer, sequence and KV head (a pair): of the n slots the `budget` with the largest key stay, the key being the mass, or
// above all masses for a first or a newest token; of equal keys the lower slots. Kept slots behind the budget move into the
// slots before it that are given up, the i-th to the i-th: sources and targets are apart, so records move in any order, and
// no more of them than have to. (Keeping the slots in order would move nearly all of the budget every time.)
//
// One cluster of 1 to 8 CTAs per pair, its slots split into equal parts, a part's into runs of a warp, one launch for all
// layers:
//   keys     masses and token numbers are read once, 16 bytes a lane, into 32-bit keys in shared memory, ordered as the masses
//            are (first and newest tokens: the largest key), with the smallest and the largest of the others;
//   select   512 or 1,024 equal buckets between those two are counted, all CTAs read all counts, and the bucket that holds the
//            budget-th largest key is taken apart again until no more keys are left than can be ranked against one another
//            (mostly at once or twice);
//   lists    ranks of equal keys, holes and movers are prefix sums over lanes, warps and CTAs, so the outcome does not
//            depend on timing; the lists take the keys' place;
//   moves    split evenly over the cluster, eight lanes a record (16 bytes of codes each; scales, mass and number by four).
// What bounds it: records lie apart (64 bytes of K, of V, and two words in lines of their own), so a move costs about 400
// bytes of memory reads, and the moves of all pairs together run at 8 to 13 thousand a us however many are in flight; the
// selection before it by instructions and barriers, so as many CTAs as fit share an SM: parts of up to 2,560 slots have 64
// threads, 17 CTAs an SM up to 2,176 slots and 15 at 2,560. 64 sequences cut from 2,112 to 2,048 slots, 10 layers, 4 heads:
// 36 us of the kernel (load 6, selection 5, lists 4, moves 9, all CTAs at once; the rest starts and barriers); 4 of
// 20,000-32,768 cut to 2,048: 63 us. The first form (three counting passes over all 32 bits, lists by votes of 32 slots,
// records one after the other) took 102 and 153 us.

#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

// Buckets of a pass, and the most keys that are ranked against one another. Shared memory is what limits the CTAs of an SM: of
// 64 threads, which have 2,560 slots at most, half as many.
__host__ __device__ constexpr int buckets_of(int threads) { return threads == 64 ? 512 : 1024; }
__host__ __device__ constexpr int cands_of(int threads) { return buckets_of(threads) / 4; }
// CTAs that an SM's registers hold.
__host__ __device__ constexpr int resident_of(int threads) { return threads == 64 ? 17 : threads == 256 ? 5 : 2; }
constexpr int kEvictMaxThreads = 512, kEvictMaxWarps = kEvictMaxThreads / 32;
constexpr int kEvictMaxCtas = 8;     // of a cluster
constexpr int kEvictSlots = 49152;   // of a CTA: 192 KB of keys
static_assert(kEvictMaxCtas * kEvictSlots == KVQ_EVICT_MAX_TOKENS, "the limit that kvq.h names");

struct EvictParams {
  EvictJob j;
  int slots;  // shared memory of a CTA, in keys (a multiple of 128)
};

// Header of the dynamic shared memory; behind it the keys, then a word for every 32 slots of a thread (bits: which stay).
template <int T>
struct alignas(16) EvictSmem {
  uint32_t count[buckets_of(T)];     // in the end the cluster's keys of the last bucket
  uint32_t cand[cands_of(T)];        // this CTA's
  int group[32];                     // sums of 32 buckets each; this CTA's, read by the others
  uint32_t warp_min[kEvictMaxWarps], warp_max[kEvictMaxWarps];
  int warp_sum[kEvictMaxWarps];
  uint32_t lo, hi;                   // this CTA's, read by the others, as the next line's
  int first, cands, equal, moves;    // (moves: holes in the low half, movers in the high one)
  int bucket, rank, here;
  uint32_t limit;
  int need, ties;
  int hole_at[kEvictMaxCtas + 1];    // first hole and mover of every CTA
  int mover_at[kEvictMaxCtas + 1];
};

// The slots of a thread where order matters: 4 times an odd number, so that 16-byte reads of neighbouring threads fall into
// different banks.
__host__ __device__ inline int slots_of_thread(int m, int threads) { return 4 * ((m + 4 * threads - 1) / (4 * threads) | 1); }

__host__ __device__ inline size_t evict_smem(int slots, int threads) {
  const size_t head = threads == 64 ? sizeof(EvictSmem<64>) : sizeof(EvictSmem<256>);
  return head + 4 * (size_t)slots + 4 * (size_t)threads * ((slots_of_thread(slots, threads) + 31) / 32);
}

// Unsigned order of the result = order of the masses; NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kStays = 0xFFFFFFFFu;  // key of a first or newest token: above that of any mass

// Inclusive sum of v over the warp.
__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// CL: more than one CTA a pair.
template <bool CL>
__device__ __forceinline__ void sync_pair() {
  if (CL) cg::this_cluster().sync();
  else __syncthreads();
}
template <bool CL, class T>
__device__ __forceinline__ T* of_cta(T* p, int q) { return CL ? cg::this_cluster().map_shared_rank(p, q) : p; }

// The first `need` of the keys equal to `limit` stay, and all above it; `equal` of them there are.
struct Limit {
  uint32_t key;
  int need, equal;
};

template <bool CL, int T>
__device__ __forceinline__ Limit find_limit(EvictSmem<T>& s, const uint32_t* keys, int m, uint32_t lo, uint32_t hi, int have, int rank,
                                            int C) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  // f(key) for this CTA's keys in from..hi
  auto each = [&](uint32_t from, auto f) {
    for (int i = 4 * t; i < m; i += 4 * T) {
      const uint4 k4 = *reinterpret_cast<const uint4*>(keys + i);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < m && k[u] - from <= hi - from) f(k[u]);
    }
  };
  constexpr int kBuckets = buckets_of(T), kGroups = kBuckets / 32, kBits = kBuckets == 512 ? 9 : 10;
  uint32_t* const count = s.count;
  for (int pass = 0;; ++pass) {
    // The first time, if it is one of the larger half, only the top 2^27 keys (16 factors of two) are told apart, and those
    // below not counted at all: masses reach far down, and the buckets of the whole range would hold too many of the upper
    // ones (2,048 of 32,768: one pass fewer, 9 -> 7 us; 2,048 of 2,112, the other half: one more, 5 -> 10 us). The whole
    // call, with and without, masses a fourth power of even ones: 655 of 32,768 (160 pairs) 50 and 56 us, 14,745 of them 142
    // and 152; 163 of 8,192 (640 pairs) 72 and 79; 132 of 2,112 (2,560 pairs) 66 and 66; 4,096 of 65,536 (80 pairs) 83 and 81.
    const uint32_t base = pass == 0 && rank <= have / 2 && hi - lo >= 1u << 27 ? hi - ((1u << 27) - 1u) : lo;
    const int shift = max(0, 32 - kBits - __clz((int)(hi - base)));
    if (pass > 0) {
      sync_pair<CL>();  // the counts have been read
      for (int i = t; i < kBuckets; i += T) count[i] = 0u;
      __syncthreads();
    }
    each(base, [&](uint32_t k) { atomicAdd(&count[(k - base) >> shift], 1u); });
    __syncthreads();
    for (int g = warp; g < kGroups; g += T / 32) {
      const int sum = (int)__reduce_add_sync(0xffffffffu, count[32 * g + lane]);
      if (lane == 0) s.group[g] = sum;
    }
    sync_pair<CL>();
    // the group, then the bucket in it, that holds the rank-th largest key: lane 0 looks at the largest keys
    int bucket = 0, here = 0;
    if (!CL || warp == 0) {
#pragma unroll
      for (int level = 0; level < 2 && bucket >= 0; ++level) {
        const int at = level == 0 ? kGroups - 1 - lane : bucket + 31 - lane;
        int own = 0;
        for (int q = 0; q < C && at >= 0; ++q) own += level == 0 ? *of_cta<CL>(&s.group[at], q) : (int)*of_cta<CL>(&count[at], q);
        const int incl = (int)warp_inclusive((uint32_t)own, lane);
        const int counted = __shfl_sync(0xffffffffu, incl, 31);
        if (level == 0 && counted < rank) {  // below the base
          rank -= counted;
          here = have - counted;
          bucket = -1;
          break;
        }
        const int l = __ffs(__ballot_sync(0xffffffffu, incl >= rank)) - 1;
        rank -= __shfl_sync(0xffffffffu, incl - own, l);
        here = __shfl_sync(0xffffffffu, own, l);
        bucket = level == 0 ? 32 * (kGroups - 1 - l) : bucket + 31 - l;
      }
      if (CL && lane == 0) {
        s.bucket = bucket;
        s.rank = rank;
        s.here = here;
      }
    }
    __syncthreads();
    if (CL) {
      bucket = s.bucket;
      rank = s.rank;
      here = s.here;
    }
    have = here;
    if (bucket < 0) {
      hi = base - 1u;
    } else {
      lo = base + ((uint32_t)bucket << shift);
      hi = min(hi, lo + ((1u << shift) - 1u));
    }
    if (lo == hi) return Limit{lo, rank, here};
    if (here > cands_of(T)) continue;
    each(lo, [&](uint32_t k) { s.cand[atomicAdd(&s.cands, 1)] = k; });
    sync_pair<CL>();
    const uint32_t* all = s.cand;
    if (CL) {
      int at = 0;
      for (int q = 0; q < C; ++q) {
        const int n = *of_cta<CL>(&s.cands, q);
        for (int i = t; i < n; i += T) count[at + i] = of_cta<CL>(s.cand, q)[i];
        at += n;
      }
      all = count;
      __syncthreads();
    }
    for (int i = t; i < here; i += T) {
      const uint32_t k = all[i];
      int above = 0, equal = 0;
      for (int x = 0; x < here; ++x) {
        above += all[x] > k;
        equal += all[x] == k;
      }
      if (above < rank && rank <= above + equal) {  // (every thread that holds such a key writes the same)
        s.limit = k;
        s.need = rank - above;
        s.ties = equal;
      }
    }
    __syncthreads();
    return Limit{s.limit, s.need, s.ties};
  }
}

// T threads; the least CTAs an SM should hold set the registers.
template <bool CL, int T>
__global__ void __launch_bounds__(T, resident_of(T)) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvictSmem<T>& s = *reinterpret_cast<EvictSmem<T>*>(smem_raw);
  uint32_t* const keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(EvictSmem<T>));
  uint32_t* const keep = keys + p.slots;
  const EvictJob& j = p.j;
  const int C = CL ? (int)cg::this_cluster().num_blocks() : 1, c = CL ? (int)cg::this_cluster().block_rank() : 0;
  constexpr int nw = T / 32;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int pair = blockIdx.x / C;
  const int b = pair / j.cs.heads % j.B, h = pair % j.cs.heads, layer = pair / j.cs.heads / j.B;

  for (int i = t; i < buckets_of(T) / 4; i += T) reinterpret_cast<uint4*>(s.count)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (t == 0) s.cands = 0;
  griddep_wait();
  griddep_launch_dependents();

  const int width = j.cs.max_pages[layer] * kPage;
  int n = j.ctx_len[b];
  if (n < 0 || n > width) {
    if (c == 0 && h == 0 && t == 0) set_err(j.dev_err, KVQ_DEVERR_POS);
    n = min(max(n, 0), width);
  }
  const int K = min(n, j.budget);
  if (j.ctx_out && layer == 0 && h == 0 && c == 0 && t == 0) j.ctx_out[b] = K;
  if (n <= j.budget) return;  // (the whole cluster)

  // ---- keys of this CTA's slots [s0, s0 + m)
  const int part = (n + 4 * C - 1) / (4 * C) * 4;
  const int s0 = min(n, c * part), m = min(n - s0, part);
  float* const mass = j.mass[layer] + ((size_t)b * j.cs.heads + h) * j.mass_len[layer];
  int32_t* const ids = j.ids[layer] + ((size_t)b * j.cs.heads + h) * j.mass_len[layer];
  const int newest = (int)max((long long)j.seen[b] - j.recent, -2147483648LL);
  const int32_t* const table = j.cs.table[layer] + (size_t)b * j.cs.max_pages[layer];
  for (int i = 32 * t; i < (n + kPage - 1) / kPage; i += 32 * T) prefetch_l1(table + i);  // (wanted at the end)
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  int first = 0;  // first and newest tokens
  constexpr int kLoads = 2;
  for (int i0 = 4 * t; i0 < m; i0 += 4 * T * kLoads) {
    float4 w[kLoads];
    int4 d[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x)
      if (i0 + 4 * T * x < m) {
        w[x] = *reinterpret_cast<const float4*>(mass + s0 + i0 + 4 * T * x);
        d[x] = *reinterpret_cast<const int4*>(ids + s0 + i0 + 4 * T * x);
      }
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int i = i0 + 4 * T * x;
      if (i >= m) break;
      const float wv[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
      const int dv[4] = {d[x].x, d[x].y, d[x].z, d[x].w};
      uint32_t k[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool stays = dv[u] < j.sinks || dv[u] >= newest;
        k[u] = stays ? kStays : key_of(wv[u]);
        if (i + u < m) {
          first += stays;
          if (!stays) {
            lo = min(lo, k[u]);
            hi = max(hi, k[u]);
          }
        }
      }
      *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  first = __reduce_add_sync(0xffffffffu, first);
  if (lane == 0) {
    s.warp_min[warp] = lo;
    s.warp_max[warp] = hi;
    s.warp_sum[warp] = first;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < nw ? s.warp_min[lane] : 0xFFFFFFFFu);
  hi = __reduce_max_sync(0xffffffffu, lane < nw ? s.warp_max[lane] : 0u);
  first = __reduce_add_sync(0xffffffffu, lane < nw ? s.warp_sum[lane] : 0);
  if (CL) {
    if (t == 0) {
      s.lo = lo;
      s.hi = hi;
      s.first = first;
    }
    sync_pair<CL>();
    lo = __reduce_min_sync(0xffffffffu, lane < C ? *of_cta<CL>(&s.lo, lane) : 0xFFFFFFFFu);
    hi = __reduce_max_sync(0xffffffffu, lane < C ? *of_cta<CL>(&s.hi, lane) : 0u);
    first = __reduce_add_sync(0xffffffffu, lane < C ? *of_cta<CL>(&s.first, lane) : 0);
  } else {
    __syncthreads();  // the warps' values have been read
  }

  // ---- the K-th largest key
  Limit limit{kStays, K, first};
  if (K > first) limit = find_limit<CL, T>(s, keys, m, lo, hi, n - first, K - first, C);

  // ---- which slots stay; holes before K and movers behind it. A thread has the `mine` slots from a0 on, 32 a word.
  const int mine = slots_of_thread(m, T), a0 = t * mine;
  const bool ordered = limit.need < limit.equal;  // of the equal keys only the first ones stay
  int tie = 0;                                    // of them before this thread's
  auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u; };  // bits 0..x-1
  auto matches = [&](int a, auto f) {  // bits of the slots a..a+31 of this thread whose key satisfies f
    uint32_t bits = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (a + 4 * q < min(m, a0 + mine)) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + a + 4 * q);
        bits |= (uint32_t)f(k.x) << (4 * q) | (uint32_t)f(k.y) << (4 * q + 1) | (uint32_t)f(k.z) << (4 * q + 2) | (uint32_t)f(k.w) << (4 * q + 3);
      }
    return bits & below(m - a);
  };
  if (ordered) {
    int equal = 0;
    for (int a = a0; a < a0 + mine && a < m; a += 32) equal += __popc(matches(a, [&](uint32_t k) { return k == limit.key; }));
    const int incl = (int)warp_inclusive((uint32_t)equal, lane);
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    tie = incl - equal;
    int sum = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) tie += s.warp_sum[w];
      sum += s.warp_sum[w];
    }
    if (CL) {
      if (t == 0) s.equal = sum;
      sync_pair<CL>();
      for (int q = 0; q < c; ++q) tie += *of_cta<CL>(&s.equal, q);
    }
    __syncthreads();  // the warps' sums have been read
  }
  // (counts in halves of a word: holes low, movers high; a part has below 2^16 slots)
  uint32_t moves = 0;
  for (int a = a0, x = 0; a < a0 + mine && a < m; a += 32, ++x) {
    uint32_t stays = matches(a, [&](uint32_t k) { return k >= limit.key; });
    if (ordered)
      for (uint32_t e = matches(a, [&](uint32_t k) { return k == limit.key; }); e; e &= e - 1)
        if (tie++ >= limit.need) stays &= ~(e & -e);
    keep[x * T + t] = stays;
    const uint32_t front = below(min(K - s0, m) - a);
    moves += __popc(~stays & front & below(a0 + mine - a)) + (__popc(stays & ~below(K - s0 - a)) << 16);
  }
  uint32_t at = warp_inclusive(moves, lane);
  if (lane == 31) s.warp_sum[warp] = (int)at;
  at -= moves;
  __syncthreads();  // (and the keys have been read)
  const uint32_t of_warp = lane < nw ? (uint32_t)s.warp_sum[lane] : 0u;
  const uint32_t upto = warp_inclusive(of_warp, lane);
  const uint32_t sum = __shfl_sync(0xffffffffu, upto, 31);
  at += __shfl_sync(0xffffffffu, upto - of_warp, warp);
  if (t == 0) s.moves = (int)sum;
  int* const list = reinterpret_cast<int*>(keys);  // holes, then movers: no more than slots
  if (moves) {
    int hole = (int)(at & 0xFFFFu), mover = (int)((sum & 0xFFFFu) + (at >> 16));
    for (int a = a0, x = 0; a < a0 + mine && a < m; a += 32, ++x) {
      const uint32_t stays = keep[x * T + t], front = below(min(K - s0, m) - a);
      for (uint32_t hs = ~stays & front & below(a0 + mine - a); hs; hs &= hs - 1) list[hole++] = s0 + a + __ffs(hs) - 1;
      for (uint32_t ms = stays & ~below(K - s0 - a); ms; ms &= ms - 1) list[mover++] = s0 + a + __ffs(ms) - 1;
    }
  }
  sync_pair<CL>();
  if (warp == 0) {
    const uint32_t x = lane < C ? (uint32_t)*of_cta<CL>(&s.moves, lane) : 0u;
    const uint32_t hs = warp_inclusive(x & 0xFFFFu, lane), ms = warp_inclusive(x >> 16, lane);
    if (lane < C) {
      s.hole_at[lane + 1] = (int)hs;
      s.mover_at[lane + 1] = (int)ms;
    }
    if (lane == 0) s.hole_at[0] = s.mover_at[0] = 0;
  }
  __syncthreads();

  // ---- moves. Every step of two records at once: places, pages, loads, stores, so that each waits for memory once.
  const int M = s.hole_at[C];  // as many movers as holes
  const int g0 = (int)((long long)M * c / C), g1 = (int)((long long)M * (c + 1) / C);
  uint8_t* const pages = j.cs.pages[layer] + (size_t)h * KVQ_INT4_BLOCK_BYTES;
  const int num_pages = j.cs.num_pages[layer];
  const size_t page_bytes = (size_t)j.cs.heads * KVQ_INT4_BLOCK_BYTES;
  const int l8 = t & 7, groups = T / 8;
  constexpr int kUnroll = 2;
  // this lane's 16 bytes of codes: chunk l8 & 3 of the K record (l8 < 4) or of the V record
  auto chunk = [&](int slot) {
    const int r = slot % kPage;
    return l8 < 4 ? r * kRec4 + 16 * (l8 ^ k_chunk_swz(r)) : kPage * kRec4 + r * kRec4 + 16 * ((l8 & 3) ^ ((r >> 1) & 3));
  };
  // and its word: K's and V's scales and offsets, the mass, the number
  auto word_at = [&](uint8_t* block, int slot) -> uint32_t* {
    if (l8 == 2) return reinterpret_cast<uint32_t*>(mass + slot);
    if (l8 == 3) return reinterpret_cast<uint32_t*>(ids + slot);
    return reinterpret_cast<uint32_t*>(block + 2 * kPage * kRec4 + (l8 & 1) * kPage * 4 + slot % kPage * 4);
  };
  for (int g = g0 + t / 8; g < g1; g += kUnroll * groups) {
    int src[kUnroll], dst[kUnroll], from[kUnroll], to[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int gu = min(g + u * groups, g1 - 1);
      int qs = 0, qd = 0;
      if (CL) {
        while (gu >= s.mover_at[qs + 1]) ++qs;
        while (gu >= s.hole_at[qd + 1]) ++qd;
      }
      const int ahead = s.hole_at[qs + 1] - s.hole_at[qs];  // holes at the front of that CTA's list
      src[u] = *of_cta<CL>(&list[ahead + gu - s.mover_at[qs]], qs);
      dst[u] = *of_cta<CL>(&list[gu - s.hole_at[qd]], qd);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      from[u] = table[src[u] / kPage];
      to[u] = table[dst[u] / kPage];
    }
    bool lost = false;
    uint4 codes[kUnroll];
    uint32_t word[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool in = g + u * groups < g1;
      ok[u] = in && from[u] >= 0 && from[u] < num_pages && to[u] >= 0 && to[u] < num_pages;
      lost |= in && !ok[u];
      if (ok[u]) {
        uint8_t* const block = pages + from[u] * page_bytes;
        codes[u] = *reinterpret_cast<const uint4*>(block + chunk(src[u]));
        if (l8 < 4) word[u] = *word_at(block, src[u]);
      }
    }
    if (lost) set_err(j.dev_err, KVQ_DEVERR_PAGE);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (ok[u]) {
        uint8_t* const block = pages + to[u] * page_bytes;
        *reinterpret_cast<uint4*>(block + chunk(dst[u])) = codes[u];
        if (l8 < 4) *word_at(block, dst[u]) = word[u];
      }
  }
  if (CL) sync_pair<CL>();  // this CTA's list may still be read
}

// kvq_mass_start: a thread a token and KV head, tokens of a head next to each other, as their slots mostly are. Bound by the
// launch: 1.7 us for 64,000 tokens and 4 heads, one behind the other in a graph, 1.0 for a single token. (The same in single
// operations on whole arrays took 540 us of host time.)
constexpr int kStartThreads = 256;

__global__ void __launch_bounds__(kStartThreads) mass_start_kernel(const kvq_token_mass m, int T, const int32_t* seq_ids,
                                                                   const int32_t* slots, const int32_t* numbers, int fresh,
                                                                   int32_t* dev_err) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned i = blockIdx.x * kStartThreads + threadIdx.x;
  const unsigned h = i / (unsigned)T, t = i - h * (unsigned)T;
  if (h >= (unsigned)m.num_kv_heads) return;
  const int q = seq_ids[t], j = slots[t], number = numbers[t];
  if (q < 0 || q >= m.num_seqs || j < 0 || j >= m.max_tokens) {
    if (h == 0) set_err(dev_err, KVQ_DEVERR_POS);
    return;
  }
  const size_t at = ((size_t)q * m.num_kv_heads + h) * m.max_tokens + j;
  if (!fresh && m.ids[at] == number) return;
  m.mass[at] = 0.0f;
  m.ids[at] = number;
}

std::mutex g_evict_mu;  // guards the cache below
bool g_evict_attr[64] = {false};

}  // namespace

cudaError_t launch_evict(const EvictJob& job, cudaStream_t stream) {
  int width = 0;
  for (int i = 0; i < job.cs.count; ++i) width = std::max(width, job.cs.max_pages[i] * kPage);
  const long long pairs = (long long)job.cs.count * job.B * job.cs.heads;
  // CTAs a pair: the most that make no more than two rounds of what is resident at once, by shared memory and registers, with
  // parts of 2,048 slots and more (32,768 slots, 160 pairs: one CTA a pair 108 us, two 67, four 66, eight 63); where there
  // are too many pairs for that, as few as hold the keys.
  auto shape = [&](int C, EvictParams& p, int& threads) {
    p.slots = ((width + C - 1) / C + 4 + 127) / 128 * 128;  // a part is at most width / C, rounded up to 4
    // Threads by a part's slots: fewer where many small parts share an SM. Measured with 2,560 pairs cut by 64 slots: parts of
    // 512 slots 21 us with 64 threads, 29 with 256; 1,088: 29 and 33; 2,112: 40 and 40; 2,560: 52 and 44; parts of 6,144: 62
    // with 256, 92 with 512; 10,240: 101 and 113; 12,800: 134 and 132; cut to half 8,448: 543 and 449, 12,800: 812 and 669.
    // The borders look at neither the pairs nor the cut: 64 threads are slower where many records move (2,112 slots cut to
    // half: 156 us, 256 threads 119; 4,096 in clusters of two, cut by 64: 101 and 52, to half: 369 and 220) or few pairs
    // leave SMs idle (160 pairs of 2,112 slots: 20 and 13).
    threads = p.slots <= 2560 ? 64 : p.slots <= 8448 ? 256 : kEvictMaxThreads;
    const long long by_smem = 227 * 1024 / (long long)(evict_smem(p.slots, threads) + 1024);
    return device_sms() * std::min<long long>(by_smem, resident_of(threads));
  };
  EvictParams p;
  p.j = job;
  int C = kEvictMaxCtas, threads, least = 1;
  while (least * kEvictSlots < width) least *= 2;
  while (C > least && (width / C < 2048 || pairs * C > 2 * shape(C, p, threads))) C /= 2;
  shape(C, p, threads);
  using Kernel = void (*)(EvictParams);
  const Kernel kerns[2][3] = {{evict_kernel<false, 64>, evict_kernel<false, 256>, evict_kernel<false, 512>},
                              {evict_kernel<true, 64>, evict_kernel<true, 256>, evict_kernel<true, 512>}};
  const Kernel kern = kerns[C > 1][threads / 256];
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lock(g_evict_mu);
    if (dev < 0 || dev >= 64 || !g_evict_attr[dev]) {
      for (const auto& some : kerns)
        for (const Kernel k : some) {
          const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
          if (e != cudaSuccess) return e;
        }
      if (dev >= 0 && dev < 64) g_evict_attr[dev] = true;
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(pairs * C), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = evict_smem(p.slots, threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_mass_start(const kvq_token_mass& mass, int T, const int32_t* seq_ids, const int32_t* slots, const int32_t* numbers,
                              int fresh, int32_t* dev_err, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(((long long)T * mass.num_kv_heads + kStartThreads - 1) / kStartThreads), 1, 1);
  cfg.blockDim = dim3(kStartThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mass_start_kernel, mass, T, seq_ids, slots, numbers, fresh, dev_err);
}

}  // namespace kvq
