// Eviction from the int4 caches by gathered attention weight (kvq_evict_int4).
//
// Per layer, sequence and KV head (a pair): of the n slots the `budget` with the largest key stay, the key being the mass, or
// above all masses for a first or a newest token; of equal keys the lower slots. Kept slots behind the budget move into the
// slots before it that are given up, the i-th to the i-th: sources and targets are apart, so records move in any order, and
// no more of them than have to. (Keeping the slots in order would move nearly all of the budget every time.)
//
// One cluster of 1 to 8 CTAs per pair, its slots split into equal parts, one launch for all layers:
//   keys     masses and token numbers are read once, 16 bytes a thread, into 32-bit keys in shared memory, ordered as the
//            masses are;
//   select   the budget-th largest key, 11, 11 and 10 bits at a time: each CTA counts its keys by digit, then all read all
//            counts through distributed shared memory;
//   lists    warps own runs of slots, so ranks of equal keys, of holes and of movers are prefix sums over warps and CTAs, and
//            the outcome does not depend on timing; the lists take the keys' place;
//   moves    split evenly over the cluster, eight lanes a record (16 bytes of codes each; scales, mass and number by four).
// Bound by memory: 8 bytes a slot and 2 x 144 a move; for small pairs by the chain of barriers, so several CTAs share an SM.
// 64 sequences cut from 2,112 to 2,048 slots, 10 layers, 4 heads: 117 us with the copy that restores the masses; 4 of 20,000-
// 32,768 to 2,048: 166 us.

#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kBins = 2048;
constexpr int kEvictMaxThreads = 512;
constexpr int kEvictMaxCtas = 8;     // of a cluster
constexpr int kEvictSlots = 49152;   // of a CTA: 192 KB of keys
static_assert(kEvictMaxCtas * kEvictSlots == KVQ_EVICT_MAX_TOKENS, "the limit that kvq.h names");

struct EvictParams {
  EvictJob j;
  int slots;  // shared memory of a CTA, in keys (a multiple of 128)
};

// Header of the dynamic shared memory; behind it one keep bit and one key a slot.
struct alignas(16) EvictSmem {
  uint32_t hist[2][kBins];
  int warp_sum[2][kEvictMaxThreads / 32];
  int digit, rank, ties;
  int holes, movers;                 // this CTA's, read by the others
  int hole_at[kEvictMaxCtas + 1];    // first hole and mover of every CTA
  int mover_at[kEvictMaxCtas + 1];
};

__host__ __device__ inline size_t evict_smem(int slots) { return sizeof(EvictSmem) + slots / 8 + 4 * (size_t)slots; }

// Unsigned order of the result = order of the masses; NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// Inclusive sum of v over the warp.
__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

__global__ void __launch_bounds__(kEvictMaxThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvictSmem& s = *reinterpret_cast<EvictSmem*>(smem_raw);
  uint32_t* const keep = reinterpret_cast<uint32_t*>(smem_raw + sizeof(EvictSmem));
  uint32_t* const keys = keep + p.slots / 32;
  const cg::cluster_group cluster = cg::this_cluster();
  const EvictJob& j = p.j;
  const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  const int T = blockDim.x, nw = T / 32, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int pair = blockIdx.x / C;
  const int b = pair / j.cs.heads % j.B, h = pair % j.cs.heads, layer = pair / j.cs.heads / j.B;

  for (int i = t; i < 2 * kBins; i += T) (&s.hist[0][0])[i] = 0;
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
  const long long newest = (long long)j.seen[b] - j.recent;
  __syncthreads();  // counts are zero
  for (int i = 4 * t; i < m; i += 4 * T) {
    const float4 w = *reinterpret_cast<const float4*>(mass + s0 + i);
    const int4 d = *reinterpret_cast<const int4*>(ids + s0 + i);
    const float wv[4] = {w.x, w.y, w.z, w.w};
    const int dv[4] = {d.x, d.y, d.z, d.w};
    uint32_t k[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      k[u] = dv[u] < j.sinks || dv[u] >= newest ? 0xFFFFFFFFu : key_of(wv[u]);
      if (i + u < m) atomicAdd(&s.hist[0][k[u] >> 21], 1u);
    }
    *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
  }

  // ---- the K-th largest key
  int rank = K;          // of the key looked for, among those that share its upper bits
  uint32_t upper = 0;    // those bits
  int ties_before = 0;   // keys equal to it in the CTAs before this one
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* const hist = s.hist[pass & 1];
    if (pass > 0)
      for (int i = t; i < m; i += T) {
        const uint32_t k = keys[i];
        if ((k >> (shift + bits)) == upper) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
    cluster.sync();
    if (pass == 1)  // the third pass counts where the first did, which every CTA has read by now
      for (int i = t; i < kBins; i += T) s.hist[0][i] = 0;
    // thread t looks at `per` digits, the largest first
    const int bins = 1 << bits, per = bins / T;
    int own = 0;
    for (int i = 0; i < per; ++i) {
      const int d = bins - 1 - (t * per + i);
      for (int q = 0; q < C; ++q) own += (int)*cluster.map_shared_rank(&hist[d], q);
    }
    int incl = warp_inclusive(own, lane);
    if (lane == 31) s.warp_sum[0][warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += s.warp_sum[0][w];
    if (incl >= rank && incl - own < rank) {  // one thread
      int above = incl - own;
      for (int i = 0; i < per; ++i) {
        const int d = bins - 1 - (t * per + i);
        int here = 0, before = 0;
        for (int q = 0; q < C; ++q) {
          const int x = (int)*cluster.map_shared_rank(&hist[d], q);
          here += x;
          if (q < c) before += x;
        }
        if (above + here >= rank) {
          s.digit = d;
          s.rank = rank - above;
          s.ties = before;
          break;
        }
        above += here;
      }
    }
    __syncthreads();
    upper = (upper << bits) | (uint32_t)s.digit;
    rank = s.rank;
    ties_before = s.ties;
  }
  const uint32_t limit = upper;  // keys above stay, and the first `rank` equal ones

  // ---- which slots stay; holes before K and movers behind it. A warp owns the slots [w0, w1) of the part.
  const int run = (m + 32 * nw - 1) / (32 * nw) * 32;
  const int w0 = min(m, warp * run), w1 = min(m, w0 + run);
  int equal = 0;
  for (int i = w0; i < w1; i += 32) equal += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && keys[i + lane] == limit));
  if (lane == 0) s.warp_sum[0][warp] = equal;
  __syncthreads();
  int tie = ties_before;
  for (int w = 0; w < warp; ++w) tie += s.warp_sum[0][w];
  const uint32_t lower = (1u << lane) - 1u;
  int holes = 0, movers = 0;
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t k = in ? keys[i + lane] : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, in && k == limit);
    const bool stays = in && (k > limit || (k == limit && tie + __popc(eq & lower) < rank));
    tie += __popc(eq);
    const uint32_t word = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) keep[i / 32] = word;
    const int at = s0 + i + lane;
    holes += __popc(__ballot_sync(0xffffffffu, in && !stays && at < K));
    movers += __popc(__ballot_sync(0xffffffffu, stays && at >= K));
  }
  __syncthreads();  // the equal keys' sums and the keys themselves have been read
  if (lane == 0) {
    s.warp_sum[0][warp] = holes;
    s.warp_sum[1][warp] = movers;
  }
  __syncthreads();
  int hole = 0, mover = 0, all_holes = 0, all_movers = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) {
      hole = all_holes;
      mover = all_movers;
    }
    all_holes += s.warp_sum[0][w];
    all_movers += s.warp_sum[1][w];
  }
  if (t == 0) {
    s.holes = all_holes;
    s.movers = all_movers;
  }
  int* const list = reinterpret_cast<int*>(keys);  // holes, then movers: no more than slots
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1, stays = in && (keep[i / 32] >> lane & 1u);
    const int at = s0 + i + lane;
    const uint32_t hs = __ballot_sync(0xffffffffu, in && !stays && at < K);
    const uint32_t ms = __ballot_sync(0xffffffffu, stays && at >= K);
    if (hs >> lane & 1u) list[hole + __popc(hs & lower)] = at;
    if (ms >> lane & 1u) list[all_holes + mover + __popc(ms & lower)] = at;
    hole += __popc(hs);
    mover += __popc(ms);
  }
  cluster.sync();
  if (t == 0) {
    int hsum = 0, msum = 0;
    for (int q = 0; q < C; ++q) {
      s.hole_at[q] = hsum;
      s.mover_at[q] = msum;
      hsum += *cluster.map_shared_rank(&s.holes, q);
      msum += *cluster.map_shared_rank(&s.movers, q);
    }
    s.hole_at[C] = hsum;
    s.mover_at[C] = msum;
  }
  __syncthreads();

  // ---- moves
  const int M = s.hole_at[C];  // as many movers as holes
  const int g0 = (int)((long long)M * c / C), g1 = (int)((long long)M * (c + 1) / C);
  const int32_t* const table = j.cs.table[layer] + (size_t)b * j.cs.max_pages[layer];
  uint8_t* const pages = j.cs.pages[layer];
  const int num_pages = j.cs.num_pages[layer], heads = j.cs.heads;
  const int l8 = t & 7, groups = T / 8;
  constexpr int kUnroll = 4;
  auto block_of = [&](int slot) -> uint8_t* {
    const int phys = table[slot / kPage];
    if (phys < 0 || phys >= num_pages) return nullptr;
    return pages + ((size_t)phys * heads + h) * KVQ_INT4_BLOCK_BYTES;
  };
  // this lane's 16 bytes of codes: chunk l8 & 3 of the K record (l8 < 4) or of the V record
  auto chunk = [&](int slot) {
    const int r = slot % kPage;
    return l8 < 4 ? r * kRec4 + 16 * (l8 ^ k_chunk_swz(r)) : kPage * kRec4 + r * kRec4 + 16 * ((l8 & 3) ^ ((r >> 1) & 3));
  };
  for (int g = g0 + t / 8; g < g1; g += kUnroll * groups) {
    uint4 codes[kUnroll];
    uint32_t word[kUnroll];
    uint8_t* to[kUnroll];
    int dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int gu = g + u * groups;
      to[u] = nullptr;
      if (gu >= g1) continue;
      int qs = 0, qd = 0;
      while (gu >= s.mover_at[qs + 1]) ++qs;
      while (gu >= s.hole_at[qd + 1]) ++qd;
      const int ahead = s.hole_at[qs + 1] - s.hole_at[qs];  // holes at the front of that CTA's list
      const int src = *cluster.map_shared_rank(&list[ahead + gu - s.mover_at[qs]], qs);
      dst[u] = *cluster.map_shared_rank(&list[gu - s.hole_at[qd]], qd);
      const uint8_t* const from = block_of(src);
      to[u] = block_of(dst[u]);
      if (!from || !to[u]) {
        set_err(j.dev_err, KVQ_DEVERR_PAGE);
        to[u] = nullptr;
        continue;
      }
      codes[u] = *reinterpret_cast<const uint4*>(from + chunk(src));
      if (l8 < 2) word[u] = *reinterpret_cast<const uint32_t*>(from + 2 * kPage * kRec4 + l8 * kPage * 4 + src % kPage * 4);
      if (l8 == 2) word[u] = __float_as_uint(mass[src]);
      if (l8 == 3) word[u] = (uint32_t)ids[src];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!to[u]) continue;
      *reinterpret_cast<uint4*>(to[u] + chunk(dst[u])) = codes[u];
      if (l8 < 2) *reinterpret_cast<uint32_t*>(to[u] + 2 * kPage * kRec4 + l8 * kPage * 4 + dst[u] % kPage * 4) = word[u];
      if (l8 == 2) mass[dst[u]] = __uint_as_float(word[u]);
      if (l8 == 3) ids[dst[u]] = (int32_t)word[u];
    }
  }
  cluster.sync();  // this CTA's list may still be read
}

std::mutex g_evict_mu;  // guards the cache below
bool g_evict_attr[64] = {false};

}  // namespace

cudaError_t launch_evict(const EvictJob& job, cudaStream_t stream) {
  int width = 0;
  for (int i = 0; i < job.cs.count; ++i) width = std::max(width, job.cs.max_pages[i] * kPage);
  // CTAs a pair: as many as the keys need, and more while they would all find an SM and have 1,024 slots each
  const long long pairs = (long long)job.cs.count * job.B * job.cs.heads;
  int C = 1;
  while (C * kEvictSlots < width) C *= 2;
  while (C < kEvictMaxCtas && pairs * C * 2 <= 2LL * device_sms() && width / C >= 2048) C *= 2;
  EvictParams p;
  p.j = job;
  // a part is at most width / C, rounded up to 4
  p.slots = ((width + C - 1) / C + 4 + 127) / 128 * 128;
  const size_t smem = evict_smem(p.slots);
  const int threads = p.slots > 4096 ? kEvictMaxThreads : 256;
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lock(g_evict_mu);
    if (dev < 0 || dev >= 64 || !g_evict_attr[dev]) {
      const cudaError_t e =
          cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
      if (e != cudaSuccess) return e;
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
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel, p);
}

}  // namespace kvq
