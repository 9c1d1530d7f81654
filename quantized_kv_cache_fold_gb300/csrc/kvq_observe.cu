// Attention weights that a prompt's last rows put on its tokens (kvq_prompt_mass).
//
//   mass[h][j] = sum over the rows i >= n - rows (j <= i) and the query heads g of KV head h of 2^(c q_ig.k_j - a_ig),
//   a_ig = log2 sum_j 2^(c q_ig.k_j),  c = sm_scale log2(e)
//
// The sums a are needed before the first weight, so the scores are computed twice (2 x 128 operations a pair each time;
// keeping them would move 8 bytes a pair instead). Both passes are one kernel: a fixed tile of 128 rows stays, tiles of the
// other side stream through a ring, one thread of each group has one row of the fixed side and keeps its sum:
//
//   pass A  fixed: 128 / G tokens of queries with all G heads of a KV head; streamed: keys. Thread = query row: base and sum.
//           Few query tiles see long prompts, so their keys are split over `nsplit` items, joined by join_kernel.
//   pass B  fixed: 128 keys; streamed: query tiles, each with its a. Thread = key: the sum over all rows, written once.
//
// a's rounding is the only one beside those of the scores and of the power of two. tcgen05 products into four score tiles of
// tensor memory, which four groups of four warps take in turns; an item's four sums meet in one of the groups. For the 8
// prompts below: two groups 149 us, four 138; sums left without waiting and ten items an SM 127; items looked up a warp at a
// time and joined by the groups in turn 113.
//
//   warps 0-3, 4-7, 8-11, 12-15  scores to sums (a lane of tensor memory each), every fourth step
//   warp 16                      tensor-map copies
//   warp 17                      the products (one issuing thread)
//
// 8 prompts of 2,000-32,768 tokens, 20/4 heads, last 64 rows: 112 us; 4 of up to 700, last 16: 13 us (14.5 with
// tensor memory taken and pass B's start behind the wait for the grid before). A pass's first 8,000 cycles go by before its
// first sums; then a 128 x 128 tile takes 1,100 cycles in pass A and 1,350 in pass B, of which the power of two (32 a cycle
// and SM) and the products need 512 each, and no unit is full.
// Tried: bundles of four fixed tiles that stream every key once (142; with a scheduling warp 136, but the short prompts then
// 22), query tiles that stay through pass B (117), four places for the sums (115), a score tile for two groups at once (114),
// 16 columns loaded ahead (124), a maximum looked for only when a sum passes 2^30 (112).

#include <algorithm>
#include <mutex>

#include "kvq_internal.h"
#include "kvq_umma.cuh"

namespace kvq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;                  // rows of a tile
constexpr int kTileBytes = kRows * kD * 2;  // two 64-dim halves of 128 rows of 128 bytes
constexpr int kRing = 4;                    // streamed tiles, and score tiles
constexpr int kGroups = 4;                  // of four warps, a score tile each
constexpr int kThreads = 128 * kGroups + 64;
constexpr int kCopyWarp = 4 * kGroups, kIssueWarp = kCopyWarp + 1;
static_assert(kGroups == kRing, "step k is group k mod kGroups's, in score tile k mod kRing");
constexpr int kItems = 16;                  // items that a warp looks up together, a lane each
constexpr int kRec = 132;                   // floats of a query tile's record: -a of 128 rows, whether one is not finite
constexpr float kBaseLag = 30.0f;           // how far (in powers of two) a score may pass the base: sums are fp32

// Named barriers: sums left for the group that joins them, their place free again (each for even and odd items), and one
// for each group's own.
constexpr uint32_t kFullBar = 1, kFreeBar = 3, kRecBar = 5;

// Arrives at a named barrier without waiting; what the thread wrote before is seen by those who wait there.
__device__ __forceinline__ void named_arrive(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

struct ObserveParams {
  CUtensorMap mq, mk;
  ObserveJob j;
  float scale2;
  int qt;      // tokens of a query tile
  int nsplit;
  int tiles;   // most query tiles, as the workspace is laid out
};

struct Item {
  int n;
  int start;     // the sequence's first token
  int sid;       // its row of the masses
  int h;
  int first;     // first observed token
  int tile;      // pass A: this query tile's number in the workspace; pass B: that of the streamed tile 0 of (b, h)
  int at;        // pass A: first token of the query tile; pass B: first key of the key tile
  int split;
  int j0, j1;    // streamed tiles
};

struct Smem {
  uint8_t fixed[2][kTileBytes];
  uint8_t ring[kRing][kTileBytes];
  alignas(16) float rec[kRing][kRec];
  Item list[kThreads / 32][kItems];
  float2 join[2][kGroups - 1][kRows];
  uint64_t fixed_full[2], fixed_empty[2];
  uint64_t ring_full[kRing], ring_empty[kRing], s_full[kRing], s_empty[kRing];
  uint64_t fin;
  int failed;
  uint32_t taddr;
  int n[KVQ_MAX_SEQS];          // length of each sequence (0: none, or skipped)
  int items[KVQ_MAX_SEQS + 1];  // first item of each
  int tiles[KVQ_MAX_SEQS + 1];  // first query tile of each
};

template <bool B>
__device__ __forceinline__ Item find_item(const ObserveParams& p, const Smem& s, int idx) {
  int lo = 0, hi = p.j.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.items[mid] <= idx) lo = mid;
    else hi = mid - 1;
  }
  Item it;
  it.n = s.n[lo];
  it.start = p.j.cu_seqlens[lo];
  it.sid = p.j.seq_ids ? p.j.seq_ids[lo] : lo;
  const int rows = p.j.rows > 0 ? min(p.j.rows, it.n) : it.n;
  it.first = it.n - rows;
  const int tiles = (rows + p.qt - 1) / p.qt;
  const int rem = idx - s.items[lo];
  if (B) {
    const int kt = (it.n + kRows - 1) / kRows;
    it.h = rem / kt;
    it.at = (rem - it.h * kt) * kRows;
    it.tile = s.tiles[lo] + it.h * tiles;
    it.split = 0;
    it.j0 = max(0, it.at - it.first) / p.qt;
    it.j1 = tiles;
  } else {
    const int per = tiles * p.nsplit;
    it.h = rem / per;
    const int u = (rem - it.h * per) / p.nsplit;
    it.split = rem - it.h * per - u * p.nsplit;
    it.at = it.first + u * p.qt;
    it.tile = s.tiles[lo] + it.h * tiles + u;
    const int nb = (min(it.at + p.qt, it.n) + kRows - 1) / kRows;
    it.j0 = (int)((long long)it.split * nb / p.nsplit);
    it.j1 = (int)((long long)(it.split + 1) * nb / p.nsplit);
  }
  return it;
}

// The k-th item of this CTA: back and forth over the CTAs, which evens out lengths that rise or fall along the items.
__device__ __forceinline__ long long item_at(int k) {
  const int n = gridDim.x, c = blockIdx.x;
  return (long long)k * n + (k & 1 ? n - 1 - c : c);
}

// Item i of this CTA for a whole warp, which asks for 0, 1, 2, ... in turn: kItems of them are looked up together (one at a
// time, the search and its divisions took a third of the kernel's time). False behind the last one.
template <bool B>
__device__ __forceinline__ bool next_item(const ObserveParams& p, Smem& s, int i, Item& it) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, items = s.items[p.j.B];
  if ((i & (kItems - 1)) == 0) {
    __syncwarp();
    const long long idx = item_at(i + lane);
    if (lane < kItems && idx < items) s.list[warp][lane] = find_item<B>(p, s, (int)idx);
    __syncwarp();
  }
  if (item_at(i) >= items) return false;
  it = s.list[warp][i & (kItems - 1)];
  return true;
}

// Lengths and first items of the sequences; sequences that a call cannot take are flagged and have none.
template <bool B>
__device__ void lay_out(const ObserveParams& p, Smem& s) {
  const ObserveJob& j = p.j;
  bool bad = false;
  if (j.seq_ids)
    for (int b = threadIdx.x; b < j.B; b += kThreads) s.items[b] = j.seq_ids[b];  // (a place for them meanwhile)
  __syncthreads();
  for (int b = threadIdx.x; b < j.B; b += kThreads) {
    const int lo = j.cu_seqlens[b], hi = j.cu_seqlens[b + 1];
    bool ok = lo >= 0 && hi >= lo && hi <= j.T && hi - lo <= j.mass_len;
    const int row = j.seq_ids ? s.items[b] : b;
    ok &= row >= 0 && row < j.num_seqs;
    if (j.seq_ids) {
#pragma unroll 8
      for (int a = 0; a < b; ++a) ok &= s.items[a] != row;  // a row named twice: the first counts
    }
    s.n[b] = ok ? hi - lo : 0;
    bad |= !ok;
    if (!ok && blockIdx.x == 0) set_err(j.dev_err, KVQ_DEVERR_POS);
  }
  // Offsets that go back may name tokens twice, and more in all than the workspace is for: sequences that overlap an earlier
  // one are skipped too.
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      int end = 0;
      for (int b = 0; b < j.B; ++b) {
        if (s.n[b] == 0) continue;
        if (j.cu_seqlens[b] < end) s.n[b] = 0;
        else end = j.cu_seqlens[b + 1];
      }
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int items = 0, tiles = 0;
    for (int b0 = 0; b0 < j.B; b0 += 32) {
      const int n = b0 + lane < j.B ? s.n[b0 + lane] : 0;
      const int rows = j.rows > 0 ? min(j.rows, n) : n;
      const int t = (rows + p.qt - 1) / p.qt * j.Hkv;
      const int i = B ? (n + kRows - 1) / kRows * j.Hkv : t * p.nsplit;
      int ti = t, ii = i;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, ii, o);
        if (lane >= o) ti += x, ii += y;
      }
      if (b0 + lane < j.B) {
        s.items[b0 + lane] = items + ii - i;
        s.tiles[b0 + lane] = tiles + ti - t;
      }
      items += __shfl_sync(0xffffffffu, ii, 31);
      tiles += __shfl_sync(0xffffffffu, ti, 31);
    }
    if (lane == 0) s.items[j.B] = items;
  }
  __syncthreads();
}

// The record's entry of a row with base m and sum l: -(m + log2 l), -inf (no weight) for a row that is none or not finite.
__device__ __forceinline__ float minus_a(float m, float l, bool& bad) {
  const bool ok = l > 0.0f && l < INFINITY && fabsf(m) < INFINITY;
  bad = !ok && !(l < 0.0f);  // l = -1 marks places without a row
  return ok ? -(m + log2f(l)) : -INFINITY;
}

template <bool F16, bool B>
__global__ void __launch_bounds__(kThreads, 1) observe_kernel(const __grid_constant__ ObserveParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const ObserveJob& j = p.j;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* failed = &sm.failed;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.fixed_full[i], 1);
      mbar_init(&sm.fixed_empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.ring_full[i], 1);
      mbar_init(&sm.ring_empty[i], B ? 5 : 1);  // the products, and the group that reads the record
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 4);
    }
    mbar_init(&sm.fin, 1);
    sm.failed = 0;
  }
  fence_barrier_init();
  if (B) {  // the rows of a streamed tile behind those that copies write
    const int used = p.qt * (j.Hq / j.Hkv), per = (kRows - used) * 8;  // 16-byte words of a 64-dim half
    for (int i = threadIdx.x; i < 2 * kRing * per; i += kThreads)
      reinterpret_cast<uint4*>(sm.ring[i / per >> 1] + (i / per & 1) * (kTileBytes / 2) + used * 128)[i % per] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_shared();
  }
  if (warp == kCopyWarp && lane == 0) {
    prefetch_tensor_map(&p.mq);
    prefetch_tensor_map(&p.mk);
  }
  if (warp == kIssueWarp) tmem_alloc_512(&sm.taddr);
  // Pass B needs of what may still run only the records, and waits before it copies the first: whatever came before the
  // call had ended when pass A let its successors start.
  if (!B) griddep_wait();
  griddep_launch_dependents();
  lay_out<B>(p, sm);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.taddr;
  const int G = j.Hq / j.Hkv, Rq = p.qt * G;  // rows of a query tile in use

  if (warp == kCopyWarp) {
    // ---------------------------------------------------------------- copies (lane 0; the others look items up)
    fence_proxy_async_global();
    bool ok = true;
    int f = 0, k = 0;
    auto keys = [&](uint8_t* dst, const Item& it, int tok, uint64_t* bar) {
      tma_load_3d(dst, &p.mk, 0, it.h, it.start + tok, bar);
      tma_load_3d(dst + kTileBytes / 2, &p.mk, 64, it.h, it.start + tok, bar);
    };
    auto queries = [&](uint8_t* dst, const Item& it, int tok, uint64_t* bar) {
      tma_load_3d(dst, &p.mq, 0, it.h * G, it.start + tok, bar);
      tma_load_3d(dst + kTileBytes / 2, &p.mq, 64, it.h * G, it.start + tok, bar);
    };
    Item it;
    for (int i = 0; next_item<B>(p, sm, i, it); ++i) {
      if (lane > 0 || !ok || it.j0 >= it.j1) continue;
      if (f >= 2 && !(ok = role_wait(&sm.fixed_empty[f & 1], (uint32_t)((f >> 1) - 1) & 1u, failed))) continue;
      mbar_arrive_expect_tx(&sm.fixed_full[f & 1], B ? kTileBytes : 2 * Rq * 128);
      if (B) keys(sm.fixed[f & 1], it, it.at, &sm.fixed_full[f & 1]);
      else queries(sm.fixed[f & 1], it, it.at, &sm.fixed_full[f & 1]);
      ++f;
      if (B && k == 0) {
        griddep_wait();
        fence_proxy_async_global();
      }
      for (int u = it.j0; u < it.j1; ++u, ++k) {
        const int st = k % kRing;
        if (k >= kRing && !(ok = role_wait(&sm.ring_empty[st], (uint32_t)(k / kRing - 1) & 1u, failed))) break;
        mbar_arrive_expect_tx(&sm.ring_full[st], B ? 2 * Rq * 128 + kRec * 4 : kTileBytes);
        if (B) {
          queries(sm.ring[st], it, it.first + u * p.qt, &sm.ring_full[st]);
          bulk_g2s(sm.rec[st], j.rec + (size_t)(it.tile + u) * kRec, kRec * 4, &sm.ring_full[st], policy_evict_first());
        } else {
          keys(sm.ring[st], it, u * kRows, &sm.ring_full[st]);
        }
      }
    }
    if (B && k == 0) griddep_wait();  // (no record wanted: nothing that comes behind this grid may overtake pass A)
    if (!ok) {  // no copy may be in flight when the CTA ends
      for (int u = max(0, f - 2); u < f; ++u) mbar_wait_bounded(&sm.fixed_full[u & 1], (uint32_t)(u >> 1) & 1u);
      for (int u = max(0, k - kRing); u < k; ++u) mbar_wait_bounded(&sm.ring_full[u % kRing], (uint32_t)(u / kRing) & 1u);
    }
  } else if (warp == kIssueWarp) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t kId = umma_idesc_16(F16, kRows, false);
    const uint32_t leader = elect_one();
    const uint32_t tm = (uint32_t)uniform((int)tmem);
    const uint64_t da = umma_sdesc(smem_addr(sm.fixed[0]), 16, 1024), db = umma_sdesc(smem_addr(sm.ring[0]), 16, 1024);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(0xffffffffu, role_wait(bar, ph, failed)) != 0; };
    int f = 0, k = 0;
    Item it;
    for (int i = 0; ok && next_item<B>(p, sm, i, it); ++i) {
      if (it.j0 >= it.j1) continue;
      if (!(ok = wait(&sm.fixed_full[f & 1], (uint32_t)(f >> 1) & 1u))) break;
      const uint64_t a = da + (uint64_t)(uniform(f & 1) * (kTileBytes >> 4));
      for (int u = it.j0; u < it.j1; ++u, ++k) {
        const int st = uniform(k % kRing);
        if (!(ok = wait(&sm.ring_full[st], (uint32_t)(k / kRing) & 1u))) break;
        if (k >= kRing && !(ok = wait(&sm.s_empty[st], (uint32_t)(k / kRing - 1) & 1u))) break;
        tc_fence_after();
        const uint64_t bb = db + (uint64_t)(st * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * (kTileBytes / 2) + (kk & 3) * 32) >> 4);
          umma_f16_by(leader, tm + kRows * st, a + off, bb + off, kId, kk > 0);
        }
        umma_commit_by(leader, &sm.s_full[st]);
        umma_commit_by(leader, &sm.ring_empty[st]);
      }
      umma_commit_by(leader, &sm.fixed_empty[f & 1]);
      ++f;
    }
    umma_commit_by(leader, &sm.fin);  // arrives once every product issued has completed
    mbar_wait_bounded(&sm.fin, 0);
  } else {
    // ---------------------------------------------------------------- scores to sums
    const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float c = p.scale2;
    const uint64_t c2 = f2(c, c);
    bool ok = true;
    int k = 0;
    // A wait that gives up ends this warp's work, not its part in the barriers below: every warp goes through all items.
    int i = 0;
    Item it;
    for (; next_item<B>(p, sm, i, it); ++i) {
      float base = -INFINITY;
      uint64_t l2[2] = {0ull, 0ull};
      const int k0 = k;
      k += max(0, it.j1 - it.j0);
      for (int at = k0 + ((grp - k0) & (kGroups - 1)); at < k && ok; at += kGroups) {  // step at: this group's
        const int u = it.j0 + at - k0, st = grp;
        ok = __all_sync(0xffffffffu, role_wait(&sm.s_full[st], (uint32_t)(at / kRing) & 1u, failed));
        if (B && ok) ok = __all_sync(0xffffffffu, role_wait(&sm.ring_full[st], (uint32_t)(at / kRing) & 1u, failed));
        if (!ok) break;
        tc_fence_after();
        if (!B) {
          const int hi = it.at + row / G - u * kRows;  // seen: columns up to hi
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            uint32_t s[32];
            tmem_ld32u(ts + kRows * st + 32 * w, s);
            const int h = hi - 32 * w;
            const uint32_t m = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
            tmem_wait_ld_all();
            if (m != ~0u) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(m & (1u << e))) s[e] = 0xFF800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q) mx[q] = fmax3(mx[q], __uint_as_float(s[e + 2 * q]), __uint_as_float(s[e + 2 * q + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            if (top > base + kBaseLag || (base == -INFINITY && top > -INFINITY)) {
              const float alpha = fast_exp2(base - top);
              base = top;
              l2[0] = mul_f2(l2[0], f2(alpha, alpha));
              l2[1] = mul_f2(l2[1], f2(alpha, alpha));
            }
            const float neg = base == -INFINITY ? 0.0f : -base;
            const uint64_t n2 = f2(neg, neg);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t x = fma_f2(f2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, n2);
              l2[e & 1] = add_f2(l2[e & 1], f2(fast_exp2(f2lo(x)), fast_exp2(f2hi(x))));
            }
          }
        } else {
          const int q0 = it.first + u * p.qt;                   // the tile's first token
          // its columns in use (of a whole tile all: those behind its rows are zeros, with no weight)
          const int valid = it.n - q0 >= p.qt ? kRows : (it.n - q0) * G;
          const int from = max(0, it.at + row - q0) * G;        // seen: columns from here on
          const float* rec = sm.rec[st];
          const bool odd = rec[kRows] != 0.0f;
#pragma unroll 1
          for (int w = 0; w < 4 && 32 * w < valid; ++w) {
            uint32_t s[32];
            tmem_ld32u(ts + kRows * st + 32 * w, s);
            const int lo = from - 32 * w, hi = valid - 32 * w;
            uint32_t m = lo <= 0 ? ~0u : lo >= 32 ? 0u : ~0u << lo;
            if (hi < 32) m &= (1u << hi) - 1u;
            float na[32];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = *reinterpret_cast<const float4*>(rec + 32 * w + 4 * e);
              na[4 * e] = v.x;
              na[4 * e + 1] = v.y;
              na[4 * e + 2] = v.z;
              na[4 * e + 3] = v.w;
            }
            tmem_wait_ld_all();
            // Rows of zeros fill the end of a whole tile where G does not divide 128, so a quarter that has any ends with one:
            // its product is NaN for a key with an infinite or NaN element, also where all rows in use have finite sums (scores
            // of -inf), and only the masked form below leaves it out.
            const bool nan = (s[31] & 0x7FFFFFFFu) > 0x7F800000u;
            if (m == ~0u && !odd && !nan) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint64_t x = fma_f2(f2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, f2(na[2 * e], na[2 * e + 1]));
                l2[e & 1] = add_f2(l2[e & 1], f2(fast_exp2(f2lo(x)), fast_exp2(f2hi(x))));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint64_t x = fma_f2(f2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, f2(na[2 * e], na[2 * e + 1]));
                const bool s0 = (m >> (2 * e) & 1u) && na[2 * e] > -INFINITY, s1 = (m >> (2 * e + 1) & 1u) && na[2 * e + 1] > -INFINITY;
                l2[e & 1] = add_f2(l2[e & 1], f2(s0 ? fast_exp2(f2lo(x)) : 0.0f, s1 ? fast_exp2(f2hi(x)) : 0.0f));
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.s_empty[st]);
          if (B) mbar_arrive(&sm.ring_empty[st]);
        }
      }
      // The groups' sums are joined in one of them, each in its turn. The others leave theirs without waiting, two items deep:
      // whoever joined item i - 2 knows that its place is free.
      float l = (f2lo(l2[0]) + f2hi(l2[0])) + (f2lo(l2[1]) + f2hi(l2[1]));
      const int to = i % kGroups;
      if (i >= 2 && grp != (i - 2) % kGroups) named_barrier(kFreeBar + (i & 1), 128 * kGroups);
      if (grp != to) {
        sm.join[i & 1][(grp - to - 1) & (kGroups - 1)][row] = make_float2(base, l);
        named_arrive(kFullBar + (i & 1), 128 * kGroups);
        continue;
      }
      named_barrier(kFullBar + (i & 1), 128 * kGroups);
      float2 other[kGroups - 1];
#pragma unroll
      for (int q = 0; q < kGroups - 1; ++q) other[q] = sm.join[i & 1][q][row];
      named_arrive(kFreeBar + (i & 1), 128 * kGroups);
      if (B) {
#pragma unroll
        for (int q = 0; q < kGroups - 1; ++q) l += other[q].y;
        const int key = it.at + row;
        if (key < it.n) {
          const size_t at = ((size_t)it.sid * j.Hkv + it.h) * j.mass_len + key;
          j.mass[at] = l;
          j.ids[at] = key;
        }
      } else {
        float M = base;
#pragma unroll
        for (int q = 0; q < kGroups - 1; ++q) M = fmaxf(M, other[q].x);
        if (M > -INFINITY) l *= fast_exp2(base - M);
#pragma unroll
        for (int q = 0; q < kGroups - 1; ++q)  // nothing seen (0), or scores that are NaN: the sums as they are
          l += M > -INFINITY ? other[q].y * fast_exp2(other[q].x - M) : other[q].y;
        if (row >= Rq || it.at + row / G >= it.n) l = -1.0f;
        if (p.nsplit > 1) {
          j.part[((size_t)it.split * p.tiles + it.tile) * kRows + row] = make_float2(M, l);
        } else {
          bool bad;
          const float na = minus_a(M, l, bad);
          const bool any = named_barrier_or(kRecBar + grp, 128, bad);
          float* const rec = j.rec + (size_t)it.tile * kRec;
          rec[row] = na;
          if (row == 0) rec[kRows] = any ? 1.0f : 0.0f;
          fence_proxy_async_global();  // pass B reads it by bulk copies
        }
      }
    }
    for (int e = max(0, i - 2); e < i; ++e)  // the arrivals for the last two items
      if (grp != e % kGroups) named_barrier(kFreeBar + (e & 1), 128 * kGroups);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc_512(tmem);
  if (threadIdx.x == 0 && *failed) set_err(j.dev_err, KVQ_DEVERR_TIMEOUT);
}

// The splits of a query tile's rows joined in their order, one block a tile. (Tiles that no item wrote are joined as they
// lie; nothing reads them.)
__global__ void __launch_bounds__(kRows) join_kernel(const float2* part, float* rec, int nsplit, int tiles) {
  griddep_wait();
  griddep_launch_dependents();
  const int tile = blockIdx.x, row = threadIdx.x;
  float M = -INFINITY, l = 0.0f;
  bool none = false;
  for (int s = 0; s < nsplit; ++s) {
    const float2 x = part[((size_t)s * tiles + tile) * kRows + row];
    none |= x.y < 0.0f;
    const float Mn = fmaxf(M, x.x);
    l = Mn > -INFINITY ? l * fast_exp2(M - Mn) + x.y * fast_exp2(x.x - Mn) : l + x.y;
    M = Mn;
  }
  bool bad;
  const float na = minus_a(M, none ? -1.0f : l, bad);
  const int any = __syncthreads_or(bad);
  rec[(size_t)tile * kRec + row] = na;
  if (row == 0) rec[(size_t)tile * kRec + kRows] = any ? 1.0f : 0.0f;
  fence_proxy_async_global();  // pass B reads it by bulk copies
}

std::mutex g_observe_mu;  // guards the cache below
bool g_observe_attr[64][4] = {{false}};

// Query tiles of a call at most, and the splits of their keys: enough for ten items an SM (before the last two steps above:
// six 135 us, ten 129, sixteen 138) while every item keeps about four blocks of keys.
void plan(int T, int B, int Hq, int Hkv, int rows, int& tiles, int& nsplit) {
  const int qt = kRows / (Hq / Hkv);
  const long long seen = rows > 0 ? std::min<long long>(T, (long long)B * rows) : T;
  tiles = (int)((seen / qt + B) * Hkv);
  const long long want = (10LL * device_sms() + tiles - 1) / tiles;
  const long long most = std::max<long long>(1, T / ((long long)B * kRows * 4));
  nsplit = (int)std::max<long long>(1, std::min<long long>(std::min(want, most), 64));
}

}  // namespace

size_t observe_workspace_bytes(int T, int B, int Hq, int Hkv, int rows) {
  // (without asking for the device: as many splits as any has)
  const int qt = kRows / (Hq / Hkv);
  const long long seen = rows > 0 ? std::min<long long>(T, (long long)B * rows) : T;
  const long long tiles = (seen / qt + B) * Hkv;
  const size_t rec = ((size_t)tiles * kRec * 4 + 255) / 256 * 256;
  const long long most = std::max<long long>(1, T / ((long long)B * kRows * 4));
  const long long splits = std::max<long long>(1, std::min<long long>(std::min<long long>((10LL * 256 + tiles - 1) / tiles, most), 64));
  return rec + (splits > 1 ? (size_t)splits * tiles * kRows * 8 : 0) + 256;
}

cudaError_t launch_observe(const ObserveJob& job, void* workspace, cudaStream_t stream) {
  ObserveParams p;
  p.j = job;
  p.scale2 = job.sm_scale * kLog2e;
  const int G = job.Hq / job.Hkv;
  p.qt = kRows / G;
  plan(job.T, job.B, job.Hq, job.Hkv, job.rows, p.tiles, p.nsplit);
  p.j.rec = static_cast<float*>(workspace);
  p.j.part = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + ((size_t)p.tiles * kRec * 4 + 255) / 256 * 256);
  const uint32_t qbox[3] = {64, (uint32_t)G, (uint32_t)p.qt}, kbox[3] = {64, 1, kRows};
  cudaError_t e = tensor_map_16(&p.mq, job.f16, job.q, job.T, job.Hq, job.qs_t, job.qs_h, qbox, false);
  if (e == cudaSuccess) e = tensor_map_16(&p.mk, job.f16, job.k, job.T, job.Hkv, job.ks_t, job.ks_h, kbox, false);
  if (e != cudaSuccess) return e;
  int dev = 0;
  cudaGetDevice(&dev);
  const size_t smem = sizeof(Smem) + 1024;
  void (*const kern[2][2])(ObserveParams) = {{observe_kernel<false, false>, observe_kernel<false, true>},
                                             {observe_kernel<true, false>, observe_kernel<true, true>}};
  {
    std::lock_guard<std::mutex> lock(g_observe_mu);
    for (int i = 0; i < 2; ++i)
      if (dev < 0 || dev >= 64 || !g_observe_attr[dev][2 * job.f16 + i]) {
        e = cudaFuncSetAttribute(kern[job.f16][i], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) g_observe_attr[dev][2 * job.f16 + i] = true;
      }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  const long long sm = device_sms();
  cfg.gridDim = dim3((unsigned)std::min<long long>((long long)p.tiles * p.nsplit, sm), 1, 1);
  e = cudaLaunchKernelEx(&cfg, kern[job.f16][0], p);
  if (e != cudaSuccess) return e;
  if (p.nsplit > 1) {
    cudaLaunchConfig_t jc = cfg;
    jc.gridDim = dim3((unsigned)p.tiles, 1, 1);
    jc.blockDim = dim3(kRows, 1, 1);
    jc.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&jc, join_kernel, (const float2*)p.j.part, p.j.rec, p.nsplit, p.tiles);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3((unsigned)std::min<long long>(((long long)job.T / kRows + job.B) * job.Hkv, sm), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern[job.f16][1], p);
}

}  // namespace kvq
