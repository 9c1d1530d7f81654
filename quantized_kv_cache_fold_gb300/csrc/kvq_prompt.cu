// Causal attention over packed prompts (kvq_prompt_attn, kvq_prompt_attn_sinks).
//
//   o_i = sum_j softmax_j(sm_scale q_i.k_j) v_j, j in [max(0, i - window + 1), i] of i's sequence; with first tokens that
//   stay visible (SINKS) also j < sinks.
//
// Bound by the tensor cores for all but short prompts: 4 x 128 operations per visible pair of tokens
// and query head. One persistent CTA per SM. A work item is two tiles of 128 query rows that share the key
// and value blocks (128 tokens): the same rows of two query heads of a KV head, or (the last head of an odd
// number) 256 consecutive rows of one. Two heads see the same blocks under the same mask, so neither tile
// waits for the other at an end (256 rows: the first tile ends a block early, and with a window the second
// starts one late). Both score tiles, both output tiles and (over the scores) the weights live in tensor
// memory:
//
//   S_t = Q_t K_j'           tcgen05.mma, Q and K in shared memory (K-major)
//   P_t = 2^(c S_t - base)   one thread per row, no exchange between threads; c = sm_scale log2(e)
//   O_t += P_t V_j           tcgen05.mma, P read from tensor memory, V in shared memory (MN-major)
//
// The two tiles alternate: while the warps of one turn scores into weights, the tensor cores run the
// other's products. The base of a row moves only when a score passes it by more than 8 (in powers of
// two), so P stays below 2^8 (fp16: 2^15, see kWeightRaise) and O is rescaled a few times at the start of a row, by the softmax warps
// themselves: S of a block is complete only after the products issued before it, so O is at rest then.
//
//   warps 0-3, 4-7  softmax and output of tile 0 and 1 (thread = row = tensor-memory lane)
//   warp 8          loads: Q tiles once an item, then K and V blocks into a ring (tensor-map copies)
//   warp 9          the products (one issuing thread)
//   warp 10         the schedule: the next item, while this one runs
//   warp 11         looks over the V blocks that hold masked places for some row (see below)
//
// Masked places and non-finite values: scores are masked by selection, so a key that a row does not
// see cannot reach it. A weight of exactly 0 times a NaN or infinite value would; warp 11 therefore
// replaces non-finite elements of V by 0 in the blocks at an edge of the mask (the diagonal, the
// window's start, the end of a sequence), and the rows that do see such an element get it added in the
// output step. Blocks that every row of both tiles sees are left as they are.
//
// The code of all roles together is more than the instruction caches hold, and straight-line code is fetched anew
// by every warp at every block: the softmax's loops are rolled (a half of the scores is loaded from tensor memory a
// second time instead), masks are laid over the scores in tensor memory before (24 prompts: 358 -> 341 us, window 513
// 116 -> 109). What is left at an item's end is the chain last products -> output -> first scores. Four warps for the
// output alone, with the next item's scores running meanwhile, were slower (337 -> 351 us, 109 -> 114).
//
// The products' warp is on everything's way: it takes the next item during the last block, and V's look answers for the
// next keys too, so that it waits five times a block instead of seven (329 -> 322 us). More waits (V in two halves: 337),
// polling instead of resting (347) or weights handed over whole (332) cost more than they gain.
//
// Measured (20/4 heads): one prompt of 32,768 tokens, bf16: 3.28-3.42 ms, 1.61-1.68 PFLOP/s; 24 prompts of 100-4,000
// tokens, 4.1e11 operations: 318-325 us, 1.25-1.28 PFLOP/s; 5 of 1,500-9,000, fp16, window 513: 104 us; 4 of up to 96: 10 us.
//
// First tokens that stay visible: an item's blocks are those that hold them, then its window's (where the two meet, one
// run). The blocks between are neither loaded nor multiplied. A form of its own (SINKS), so that the other keeps its code.
// 24 prompts of 100-4,000 tokens, window 513, 64 first tokens: 181 us; one of 32,768, fp16, window 4,096, 4 first tokens:
// 940-962 us, 1.34-1.37 PFLOP/s; 4 of up to 300: 13 us.
//
// Work order: items by descending row tile, so the longest run first, heads of a tile next to each other (they share
// K and V in L2); CTAs take them in turns, back and forth (c, 2n-1-c, 2n+c, ...), which evens out the descending
// lengths without a counter in memory.

#include <algorithm>
#include <mutex>

#include "kvq_internal.h"
#include "kvq_umma.cuh"

namespace kvq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;                 // rows of a tile, tokens of a block
constexpr int kItemRows = 2 * kRows;
constexpr int kTileBytes = kRows * kD * 2;  // 32 KB: two 64-dim halves of 128 rows of 128 bytes
constexpr int kRing = 4;                   // K and V blocks in flight (K in even, V in odd slots)
constexpr int kThreads = 384;
// registers a thread: 256 softmax threads and 128 others, from 168 at launch
constexpr int kRegSoftmax = 208, kRegAux = 88;
static_assert(256 * kRegSoftmax + 128 * kRegAux <= kThreads * 168, "register shares above the launch's allocation");
constexpr uint32_t kColS = 0, kColO = 256;  // tile t at + 128 t; P over the first 64 columns of S

struct PromptParams {
  CUtensorMap mq, mk, mv, mo;
  PromptJob j;
  float scale2;  // sm_scale * log2(e)
};

struct Item {
  int s, n;           // first token and length of the sequence (n < 0: no more items)
  int r0[2], hq[2];   // first row and query head of each tile (r0 >= n: no tile)
};

struct Smem {
  uint8_t q[2][kTileBytes];
  uint8_t kv[kRing][kTileBytes];
  uint8_t stage[8][2048];  // output, a softmax warp each
  uint64_t q_full, q_empty;
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t v_ok[kRing / 2];
  uint64_t s_full[2], p_half[2], p_ready[2], o_full[2];
  uint64_t item_full[2], item_empty[2];
  uint64_t fin;
  Item item[2];
  int bad[2];   // count of the last item (by parity) in whose edge blocks a value was replaced
  int failed;
  uint32_t taddr;
  int nt[KVQ_MAX_SEQS];  // row tiles of each sequence
};

// The blocks [jb, je) of tile t of an item.
struct Range {
  int jb, je;
  __device__ Range(const Item& it, int t, int window) {
    const int R = it.r0[t];
    if (R >= it.n) {
      jb = je = 0;
    } else {
      jb = window ? max(0, R - window + 1) / kRows : 0;
      je = (min(R + kRows, it.n) + kRows - 1) / kRows;
    }
  }
};

// Whether some row of the tile (rows R..R+127 of a sequence of n) misses a token of block j.
template <bool SINKS>
__device__ __forceinline__ bool edge_block(int R, int n, int j, int window, int sinks) {
  const int c = j * kRows;
  return c + kRows - 1 > R || (window && c < R + kRows - window && !(SINKS && c + kRows <= sinks));
}

// The order of blocks: without first tokens jb, jb + 1, ...; with them 0, 1, ... over the `ns` blocks that hold some, then on
// from jb. (Tiles of an item may differ in jb: the loads go by the first tile's, each tile's softmax by its own.)
template <bool SINKS>
__device__ __forceinline__ int first_block(int jb) { return SINKS ? 0 : jb; }
template <bool SINKS>
__device__ __forceinline__ int block_after(int b, int jb, int ns) { return SINKS && b + 1 >= ns && b + 1 < jb ? jb : b + 1; }
// Whether a tile takes block b.
template <bool SINKS>
__device__ __forceinline__ bool takes(const Range& r, int b, int ns) { return b < r.je && (b >= r.jb || (SINKS && b < ns)); }

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

// The items by descending row tile M, then sequence, KV head and query head: a sequence of nt tiles has at tile M < nt
// `pairs` items of two heads (all KV heads together), and `odd` of the last heads of an odd number where M is odd (256
// rows from tile M - 1 on) or the last (128 rows). Item `idx` -> M, the sequence b, and its number r among the
// sequence's at M. Items come in ascending order, so M never exceeds m_top, the last answer. Whole warp.
__device__ __forceinline__ void find_item(const int* nt, int B, int pairs, int odd, int idx, int& m_top, int& b, int& r) {
  const int lane = threadIdx.x & 31;
  auto above = [&](int m) {  // items of tiles behind m
    int v = 0;
    for (int i = lane; i < B; i += 32)
      if (nt[i] > m + 1) v += (nt[i] - m - 1) * pairs + odd * (((nt[i] + 1) >> 1) - ((m + 1) >> 1));
    return warp_sum_int(v);
  };
  int lo = 0, hi = m_top;
  while (lo < hi) {  // the smallest m with above(m) <= idx
    const int mid = (lo + hi) >> 1;
    if (above(mid) <= idx) hi = mid;
    else lo = mid + 1;
  }
  m_top = lo;
  r = idx - above(lo);
  b = 0;
  for (int i0 = 0; i0 < B; i0 += 32) {
    const int t = i0 + lane < B ? nt[i0 + lane] : 0;
    const int c = t > lo ? pairs + ((lo & 1) || lo == t - 1 ? odd : 0) : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, incl > r);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b = i0 + l;
      r -= __shfl_sync(0xffffffffu, incl - c, l);
      break;
    }
    r -= __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Offsets that go back may name rows twice: a sequence that overlaps an earlier one is skipped too (nt: row tiles of
// each, 0 where it is skipped), so that every output row has one writer.
__device__ __noinline__ void drop_overlapping(int* nt, const int32_t* cu, int B) {
  int end = 0;
  for (int b = 0; b < B; ++b) {
    if (nt[b] == 0) continue;
    if (cu[b] < end) nt[b] = 0;
    else end = cu[b + 1];
  }
}

// Of two pairs of 16-bit values: the larger of m (magnitudes) and |w|, NaN where either is.
template <bool F16>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t w) {
  uint32_t r;
  if (F16) asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %2;\n\tmax.NaN.f16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  else asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  return r;
}

template <bool F16>
__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
  constexpr uint32_t kExp = F16 ? 0x7C007C00u : 0x7F807F80u, kOne = F16 ? 0x04000400u : 0x00800080u;
  return (((w & kExp) + kOne) & 0x80008000u) != 0;
}
template <bool F16>
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
  constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
  if ((w & kExp) == kExp) w &= 0xFFFF0000u;
  if (((w >> 16) & kExp) == kExp) w &= 0x0000FFFFu;
  return w;
}
template <bool F16>
__device__ __forceinline__ float value16(uint32_t bits) {
  return F16 ? __half2float(__ushort_as_half((unsigned short)bits)) : __uint_as_float(bits << 16);
}

// The output step's slow part: adds the non-finite values of the edge blocks that this row sees to the
// row as written (the sums are infinite or NaN, so nothing is rounded twice).
template <bool F16, bool SINKS>
__device__ __noinline__ void add_nonfinite(const PromptJob& j, const Item& it, int t, int row) {
  const Range r0(it, 0, j.window), r1(it, 1, j.window);
  const int lo = j.window ? max(0, row - j.window + 1) : 0;
  const int hkv = it.hq[t] / (j.Hq / j.Hkv);
  uint16_t* o = static_cast<uint16_t*>(j.out) + (it.s + row) * j.os_t + it.hq[t] * j.os_h;
  const int ns = (j.sinks + kRows - 1) / kRows;
  for (int jb = first_block<SINKS>(r0.jb); jb < max(r0.je, r1.je); jb = block_after<SINKS>(jb, r0.jb, ns)) {  // tile 0 starts first
    bool edge = false;
    for (int u = 0; u < 2; ++u) {
      const Range& r = u ? r1 : r0;
      edge |= takes<SINKS>(r, jb, ns) && edge_block<SINKS>(it.r0[u], it.n, jb, j.window, j.sinks);
    }
    if (!edge) continue;
    for (int tok = SINKS ? jb * kRows : max(lo, jb * kRows); tok <= min(row, jb * kRows + kRows - 1); ++tok) {
      if (SINKS && tok < lo && tok >= j.sinks) continue;
      const uint16_t* v = static_cast<const uint16_t*>(j.v) + (it.s + tok) * j.vs_t + hkv * j.vs_h;
      for (int c = 0; c < kD; ++c) {
        const float x = value16<F16>(v[c]);
        if (!isfinite(x)) o[c] = (uint16_t)pack16x2<F16>(value16<F16>(o[c]) + x, 0.0f);
      }
    }
  }
}

template <bool F16, bool SINKS>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const PromptJob& j = p.j;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* failed = &sm.failed;
  const int ns = SINKS ? (j.sinks + kRows - 1) / kRows : 0;  // blocks that hold first tokens

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.v_ok[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_half[i], 4);
      mbar_init(&sm.p_ready[i], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 11);  // loads, products, V check and the 8 softmax warps
      sm.bad[i] = -1;
    }
    mbar_init(&sm.fin, 1);
    sm.failed = 0;
  }
  fence_barrier_init();
  griddep_wait();
  griddep_launch_dependents();
  bool bad = false;
  for (int b = threadIdx.x; b < j.B; b += kThreads) {
    const int s = j.cu_seqlens[b], e = j.cu_seqlens[b + 1];
    const bool ok = s >= 0 && e >= s && e <= j.T;
    if (!ok && blockIdx.x == 0) set_err(j.dev_err, KVQ_DEVERR_POS);
    sm.nt[b] = ok ? (e - s + kRows - 1) / kRows : 0;
    bad |= !ok;
  }
  if (warp == 9) tmem_alloc_512(&sm.taddr);
  tc_fence_before();
  if (__builtin_expect(__syncthreads_or(bad), 0)) {
    if (threadIdx.x == 0) drop_overlapping(sm.nt, j.cu_seqlens, j.B);
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = sm.taddr;

  if (warp >= 8) {
    reg_dealloc<kRegAux>();
    if (warp == 10) {
      // ------------------------------------------------------------ schedule
      const int G = j.Hq / j.Hkv, pairs = G / 2 * j.Hkv, odd = G & 1 ? j.Hkv : 0;
      int top = 0, items = 0;
      for (int b = lane; b < j.B; b += 32) {
        items += sm.nt[b] * pairs + (sm.nt[b] + 1) / 2 * odd;
        top = max(top, sm.nt[b] - 1);
      }
      items = warp_sum_int(items);
      top = __reduce_max_sync(0xffffffffu, top);
      const int n = gridDim.x, c = blockIdx.x;
      for (int k = 0;; ++k) {
        Item it{0, -1, {0, 0}, {0, 0}};
        const long long idx = (long long)k * n + (k & 1 ? n - 1 - c : c);
        if (idx < items) {
          int b, r;
          find_item(sm.nt, j.B, pairs, odd, (int)idx, top, b, r);
          it.s = j.cu_seqlens[b];
          it.n = j.cu_seqlens[b + 1] - it.s;
          const int per = G / 2 + (odd && ((top & 1) || top == sm.nt[b] - 1));  // items of a KV head
          const int h = r / per * G, u = r % per;
          const bool rows256 = u == G / 2;
          it.r0[0] = (rows256 ? top & ~1 : top) * kRows;
          it.r0[1] = it.r0[0] + (rows256 ? kRows : 0);
          it.hq[0] = h + 2 * u;
          it.hq[1] = it.hq[0] + (rows256 ? 0 : 1);
        }
        bool ok = k < 2 || role_wait(&sm.item_empty[k & 1], (uint32_t)(k / 2 - 1) & 1u, failed);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) {
          sm.item[k & 1] = it;
          mbar_arrive(&sm.item_full[k & 1]);
        }
        if (it.n < 0) break;
      }
    } else if (warp == 8 && lane == 0) {
      // ------------------------------------------------------------ loads
      int slot = 0, used = 0;  // next ring slot, blocks loaded so far
      auto load = [&](const CUtensorMap* map, int head, int tok) {
        if (used >= kRing && !role_wait(&sm.kv_empty[slot], (uint32_t)(used / kRing - 1) & 1u, failed)) return false;
        mbar_arrive_expect_tx(&sm.kv_full[slot], kTileBytes);
        tma_load_3d(sm.kv[slot], map, 0, head, tok, &sm.kv_full[slot]);
        tma_load_3d(sm.kv[slot] + kTileBytes / 2, map, 64, head, tok, &sm.kv_full[slot]);
        ++used;
        slot = (slot + 1) % kRing;
        return true;
      };
      bool ok = true;
      int nq = 0;
      for (int k = 0; ok; ++k) {
        if (!(ok = role_wait(&sm.item_full[k & 1], (uint32_t)(k / 2) & 1u, failed))) break;
        const Item it = sm.item[k & 1];
        mbar_arrive(&sm.item_empty[k & 1]);
        if (it.n < 0) break;
        const Range a(it, 0, j.window), b(it, 1, j.window);
        const int hkv = it.hq[0] / (j.Hq / j.Hkv);
        const int start = first_block<SINKS>(a.jb);
        if (!(ok = load(&p.mk, hkv, it.s + start * kRows))) break;  // its place is free before Q's
        if (k > 0 && !(ok = role_wait(&sm.q_empty, (uint32_t)(k - 1) & 1u, failed))) break;
        const int tiles = b.je > 0 ? 2 : 1;
        mbar_arrive_expect_tx(&sm.q_full, tiles * kTileBytes);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sm.q[t] + h * (kTileBytes / 2), &p.mq, 64 * h, it.hq[t], it.s + it.r0[t], &sm.q_full);
        ++nq;
        for (int jb = start; ok && jb < max(a.je, b.je); jb = block_after<SINKS>(jb, a.jb, ns))
          ok = (jb == start || load(&p.mk, hkv, it.s + jb * kRows)) && load(&p.mv, hkv, it.s + jb * kRows);
      }
      if (!ok) {  // no copy may be in flight when the CTA ends
        if (nq > 0) mbar_wait_bounded(&sm.q_full, (uint32_t)(nq - 1) & 1u);
        for (int u = max(0, used - kRing); u < used; ++u) mbar_wait_bounded(&sm.kv_full[u % kRing], (uint32_t)(u / kRing) & 1u);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ products
      constexpr uint32_t kIdQK = umma_idesc_16(F16, kRows, false), kIdPV = umma_idesc_16(F16, kD, true);
      const uint32_t leader = elect_one();
      const uint32_t tm = (uint32_t)uniform((int)tmem);
      const uint64_t dq0 = umma_sdesc(smem_addr(sm.q[0]), 16, 1024);
      const uint64_t dk0 = umma_sdesc(smem_addr(sm.kv[0]), 16, 1024);
      const uint64_t dv0 = umma_sdesc(smem_addr(sm.kv[0]), kTileBytes / 2, 1024);
      bool ok = true;
      int kv = 0;          // ring uses before the item: K of its block i is use kv + 2 i, V the next
      uint32_t pph0 = 0, pph1 = 0;  // phases of p_half and p_ready, tile 0 and 1
      auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(0xffffffffu, role_wait(bar, ph, failed)) != 0; };
      auto full = [&](int use) { return wait(&sm.kv_full[use % kRing], (uint32_t)(use / kRing) & 1u); };
      auto qk = [&](int t, int slot) {
        const uint64_t q = dq0 + (uint64_t)(t * (kTileBytes >> 4)), kb = dk0 + (uint64_t)(slot * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {  // 16 dims each: 32 bytes within a 64-dim half
          const uint64_t off = (uint64_t)(((kk >> 2) * (kTileBytes / 2) + (kk & 3) * 32) >> 4);
          umma_f16_by(leader, tm + kColS + 128 * t, q + off, kb + off, kIdQK, kk > 0);
        }
        umma_commit_by(leader, &sm.s_full[t]);
      };
      // 16 tokens a step: 2048 bytes of a half of V, 8 columns of P
      auto pv = [&](int t, int slot, int half, uint32_t acc) {
        const uint64_t v = dv0 + (uint64_t)(slot * (kTileBytes >> 4));
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int kk = 4 * half + k4;
          umma_f16_ts_by(leader, tm + kColO + 128 * t, tm + kColS + 128 * t + 8 * kk, v + (uint64_t)(kk * (2048 >> 4)), kIdPV, k4 > 0 ? 1u : acc);
        }
      };
      // Item k, taken while the one before is still at its last block: the switch is on the way of everything else.
      auto take = [&](int k) {
        ok = wait(&sm.item_full[k & 1], (uint32_t)(k / 2) & 1u);
        Item it = sm.item[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[k & 1]);
        it.n = ok ? uniform(it.n) : -1;
        it.r0[0] = uniform(it.r0[0]);
        it.r0[1] = uniform(it.r0[1]);
        return it;
      };
      Item it = take(0);
      for (int k = 0; ok && it.n >= 0; ++k) {
        const Range r0(it, 0, j.window), r1(it, 1, j.window);
        const int jb = first_block<SINKS>(r0.jb), je = max(r0.je, r1.je);
        ok = wait(&sm.q_full, (uint32_t)k & 1u) && full(kv);
        if (!ok) break;
        tc_fence_after();
        qk(0, kv % kRing);
        if (r1.je > 0 && (SINKS || r1.jb == jb)) qk(1, kv % kRing);
        umma_commit_by(leader, &sm.kv_empty[kv % kRing]);
        if (block_after<SINKS>(jb, r0.jb, ns) >= je) umma_commit_by(leader, &sm.q_empty);
        Item next = it;
        int uv = kv + 1;
        for (int b = jb, after; ok && b < je; b = after, uv += 2) {
          after = block_after<SINKS>(b, r0.jb, ns);
          if (after >= je) next = take(k + 1);
          const int sv = uv % kRing, sk = (uv + 1) % kRing;
          ok = ok && wait(&sm.v_ok[sv >> 1], (uint32_t)(uv / kRing) & 1u);  // V and the next K are here
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const Range& r = t ? r1 : r0;
            uint32_t& ph = t ? pph1 : pph0;
            if (takes<SINKS>(r, b, ns)) {
              // the first half of the weights may be multiplied while the second is still computed
              if (!(ok = wait(&sm.p_half[t], ph))) break;
              tc_fence_after();
              pv(t, sv, 0, b > first_block<SINKS>(r.jb));
              if (!(ok = wait(&sm.p_ready[t], ph))) break;
              ph ^= 1u;
              tc_fence_after();
              pv(t, sv, 1, 1u);
              if (b == r.je - 1) umma_commit_by(leader, &sm.o_full[t]);
            }
            if (takes<SINKS>(r, after, ns)) qk(t, sk);
          }
          if (!ok) break;
          umma_commit_by(leader, &sm.kv_empty[sv]);
          if (after < je) umma_commit_by(leader, &sm.kv_empty[sk]);
          if (after < je && block_after<SINKS>(after, r0.jb, ns) >= je) umma_commit_by(leader, &sm.q_empty);
        }
        kv = uv - 1;
        it = next;
      }
      umma_commit_by(leader, &sm.fin);  // arrives once every product issued has completed
      mbar_wait_bounded(&sm.fin, 0);
    } else if (warp == 11) {
      // ------------------------------------------------------------ V check
      int kv = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = __all_sync(0xffffffffu, role_wait(&sm.item_full[k & 1], (uint32_t)(k / 2) & 1u, failed));
        if (!ok) break;
        const Item it = sm.item[k & 1];
        __syncwarp();
        if (it.n < 0) break;
        const Range a(it, 0, j.window), b(it, 1, j.window);
        const int jb = first_block<SINKS>(a.jb), je = max(a.je, b.je);
        int use = kv + 1;
        for (int blk = jb, after; blk < je; blk = after, use += 2) {
          after = block_after<SINKS>(blk, a.jb, ns);
          const int slot = use % kRing;
          ok = __all_sync(0xffffffffu, role_wait(&sm.kv_full[slot], (uint32_t)(use / kRing) & 1u, failed));
          if (!ok) break;
          const bool edge = (takes<SINKS>(a, blk, ns) && edge_block<SINKS>(it.r0[0], it.n, blk, j.window, j.sinks)) ||
                            (takes<SINKS>(b, blk, ns) && edge_block<SINKS>(it.r0[1], it.n, blk, j.window, j.sinks));
          if (edge) {
            uint4* tile = reinterpret_cast<uint4*>(sm.kv[slot]);
            uint32_t m[4] = {0u, 0u, 0u, 0u};  // largest magnitudes, NaN above all
#pragma unroll 8
            for (int i = lane; i < kTileBytes / 16; i += 32) {
              const uint4 w = tile[i];
              m[0] = max_magnitude<F16>(m[0], w.x);
              m[1] = max_magnitude<F16>(m[1], w.y);
              m[2] = max_magnitude<F16>(m[2], w.z);
              m[3] = max_magnitude<F16>(m[3], w.w);
            }
            const bool bad = has_nonfinite<F16>(m[0]) | has_nonfinite<F16>(m[1]) | has_nonfinite<F16>(m[2]) | has_nonfinite<F16>(m[3]);
            if (__any_sync(0xffffffffu, bad)) {
              for (int i = lane; i < kTileBytes / 16; i += 32) {
                uint4 w = tile[i];
                w.x = drop_nonfinite<F16>(w.x);
                w.y = drop_nonfinite<F16>(w.y);
                w.z = drop_nonfinite<F16>(w.z);
                w.w = drop_nonfinite<F16>(w.w);
                tile[i] = w;
              }
              if (lane == 0) sm.bad[k & 1] = k;
              fence_proxy_async_shared();
            }
          }
          if (after < je) {
            ok = __all_sync(0xffffffffu, role_wait(&sm.kv_full[(use + 1) % kRing], (uint32_t)((use + 1) / kRing) & 1u, failed));
            if (!ok) break;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.v_ok[slot >> 1]);
        }
        kv = use - 1;
        if (lane == 0) mbar_arrive(&sm.item_empty[k & 1]);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax and output
    reg_alloc<kRegSoftmax>();
    const int t = warp >> 2;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_base + kColS + 128 * t, to = tmem + lane_base + kColO + 128 * t;
    const float c = p.scale2;
    uint32_t sph = 0, oph = 0;
    bool ok = true;
    auto take = [&](int k) {  // item k, taken before the output of the one before
      ok = __all_sync(0xffffffffu, role_wait(&sm.item_full[k & 1], (uint32_t)(k / 2) & 1u, failed));
      Item it = sm.item[k & 1];
      if (!ok) it.n = -1;
      return it;
    };
    Item next = take(0);
    for (int k = 0; ok && next.n >= 0; ++k) {
      const Item it = next;
      const Range rg(it, t, j.window);
      const int R = it.r0[t], row = R + 32 * (warp & 3) + lane;
      float base = -INFINITY;  // in powers of two, as the weights take it
      uint64_t l2[2] = {0ull, 0ull};
      for (int b = first_block<SINKS>(rg.jb); b < rg.je; b = block_after<SINKS>(b, rg.jb, ns)) {
        ok = __all_sync(0xffffffffu, role_wait(&sm.s_full[t], sph, failed));
        if (!ok) break;
        sph ^= 1u;
        tc_fence_after();
        if (edge_block<SINKS>(R, it.n, b, j.window, j.sinks)) {  // the mask, over the scores in tensor memory
          const int hi = row - b * kRows, lo = j.window ? hi - j.window + 1 : 0;  // seen: lo..hi
          const int first = SINKS ? j.sinks - b * kRows : 0;                      // and those before `first`, up to hi
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            uint32_t s[32];
            tmem_ld32u(ts + 32 * w, s);
            const int h = hi - 32 * w, l = lo - 32 * w;
            uint32_t m = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
            if (SINKS) {
              const int f = first - 32 * w;
              const uint32_t win = l <= 0 ? ~0u : l >= 32 ? 0u : ~0u << l, early = f <= 0 ? 0u : f >= 32 ? ~0u : (1u << f) - 1u;
              m &= win | early;
            } else if (l > 0) {
              m = l >= 32 ? 0u : m & (~0u << l);
            }
            tmem_wait_ld_all();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(m & (1u << i))) s[i] = 0xFF800000u;
            tmem_st32u(ts + 32 * w, s);
          }
          tmem_wait_st();
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        uint32_t s[64];
#pragma unroll 1
        for (int h = 1; h >= 0; --h) {  // the first half stays in registers
          tmem_ld32u(ts + 64 * h, s);
          tmem_ld32u(ts + 64 * h + 32, s + 32);
          tmem_wait_ld_all();
#pragma unroll
          for (int i = 0; i < 64; i += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = fmax3(mx[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool move = top > base + kBaseLag || (base == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, move)) {
          const float alpha = move ? fast_exp2(base - top) : 1.0f;
          if (move) base = top;
          l2[0] = mul_f2(l2[0], f2(alpha, alpha));
          l2[1] = mul_f2(l2[1], f2(alpha, alpha));
          if (b > first_block<SINKS>(rg.jb)) {  // O of the first block starts anew
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t o[32];
              tmem_ld32u(to + 32 * i, o);
              tmem_wait_ld_all();
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
              tmem_st32u(to + 32 * i, o);
            }
          }
        }
        const float neg = base == -INFINITY ? 0.0f : F16 ? kWeightRaise - base : -base;
        const uint64_t c2 = f2(c, c), n2 = f2(neg, neg);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint64_t x = fma_f2(f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, n2);
            const float e0 = fast_exp2(f2lo(x)), e1 = fast_exp2(f2hi(x));
            l2[i & 1] = add_f2(l2[i & 1], f2(e0, e1));
            pk[i] = pack16x2<F16>(e0, e1);
          }
          tmem_st32u(ts + 32 * h, pk);
          if (h == 0) {
            tmem_ld32u(ts + 64, s);
            tmem_ld32u(ts + 96, s + 32);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(h ? &sm.p_ready[t] : &sm.p_half[t]);
          if (h == 0) tmem_wait_ld_all();
        }
      }
      if (!ok) break;
      next = take(k + 1);
      if (!ok) break;
      if (rg.je > 0) {
        ok = __all_sync(0xffffffffu, role_wait(&sm.o_full[t], oph, failed));
        if (!ok) break;
        oph ^= 1u;
        tc_fence_after();
        const float l = (f2lo(l2[0]) + f2hi(l2[0])) + (f2lo(l2[1]) + f2hi(l2[1]));
        const float inv = 1.0f / l;
        // 32 dims of the warp's 32 rows at a time through shared memory. Whole ones leave by an asynchronous copy; at
        // the end of a sequence 4 lanes write 64 bytes of a row.
        uint8_t* const stage = sm.stage[warp];
        const int row0 = row - lane;
        const int have = it.n - row0;  // rows of the warp (may be 0 or fewer, or more than 32)
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32], w[16];
          tmem_ld32u(to + 32 * c, o);
          tmem_wait_ld_all();
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack16x2<F16>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
          if (lane == 0) tma_stores_read();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stage + lane * 64 + 16 * (i ^ ((lane >> 1) & 3))) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if (have >= 32) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) tma_store_3d(&p.mo, stage, 32 * c, it.hq[t], it.s + row0);
          } else {
            __syncwarp();
            const int lr = lane >> 2, lc = lane & 3;
            uint16_t* const out = static_cast<uint16_t*>(j.out) + (it.s + row0) * j.os_t + it.hq[t] * j.os_h;
#pragma unroll 1
            for (int rr = lr; rr < have; rr += 8)
              *reinterpret_cast<uint4*>(out + rr * j.os_t + 32 * c + 8 * lc) = *reinterpret_cast<const uint4*>(stage + rr * 64 + 16 * (lc ^ ((rr >> 1) & 3)));
          }
        }
        if (__builtin_expect(sm.bad[k & 1] == k, 0)) {
          // the row as written by other lanes
          if (lane == 0) tma_stores_done();
          __syncwarp();
          __threadfence();
          if (row < it.n) add_nonfinite<F16, SINKS>(j, it, t, row);
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&sm.item_empty[k & 1]);
    }
    if (lane == 0) tma_stores_read();  // no copy reads shared memory when the CTA ends
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc_512(tmem);
  if (threadIdx.x == 0 && *failed) set_err(j.dev_err, KVQ_DEVERR_TIMEOUT);
}

std::mutex g_mu;  // guards the caches below
bool g_attr[64][4] = {{false}};
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

cudaError_t encoder(EncodeTiled& f) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_encode) {
    void* sym = nullptr;
    cudaDriverEntryPointQueryResult got;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &got);
    if (e != cudaSuccess) return e;
    if (got != cudaDriverEntryPointSuccess || !sym) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeTiled>(sym);
  }
  f = g_encode;
  return cudaSuccess;
}

}  // namespace

cudaError_t tensor_map_16(void* map, bool f16, const void* base, int T, int heads, long long st, long long sh,
                          const uint32_t (&box)[3], bool swizzle64) {
  EncodeTiled f;
  const cudaError_t e = encoder(f);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {kD, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  const cuuint32_t one[3] = {1, 1, 1};
  return f(static_cast<CUtensorMap*>(map), f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
           const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           swizzle64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

cudaError_t launch_prompt(const PromptJob& job, cudaStream_t stream) {
  PromptParams p;
  p.j = job;
  p.scale2 = job.sm_scale * kLog2e;
  // the inputs: boxes of 64 dims x 1 head x 128 tokens, zeros outside (tokens from T on); the output: 32 dims x 1 head x 32
  const uint32_t in[3] = {64, 1, kRows}, out[3] = {32, 1, 32};
  cudaError_t e = tensor_map_16(&p.mq, job.f16, job.q, job.T, job.Hq, job.qs_t, job.qs_h, in, false);
  if (e == cudaSuccess) e = tensor_map_16(&p.mk, job.f16, job.k, job.T, job.Hkv, job.ks_t, job.ks_h, in, false);
  if (e == cudaSuccess) e = tensor_map_16(&p.mv, job.f16, job.v, job.T, job.Hkv, job.vs_t, job.vs_h, in, false);
  if (e == cudaSuccess) e = tensor_map_16(&p.mo, job.f16, job.out, job.T, job.Hq, job.os_t, job.os_h, out, true);
  if (e != cudaSuccess) return e;
  const bool sinks = job.window > 0 && job.sinks > 0;
  const int form = 2 * sinks + job.f16;
  const auto kern = sinks ? (job.f16 ? prompt_kernel<true, true> : prompt_kernel<false, true>)
                          : (job.f16 ? prompt_kernel<true, false> : prompt_kernel<false, false>);
  const size_t smem = sizeof(Smem) + 1024;
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (dev < 0 || dev >= 64 || !g_attr[dev][form]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) g_attr[dev][form] = true;
    }
  }
  // no more CTAs than items: T tokens in B sequences make at most T / 256 + B row blocks
  const long long most = ((long long)job.T / kItemRows + job.B) * job.Hq;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<long long>(most, device_sms()), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace kvq
