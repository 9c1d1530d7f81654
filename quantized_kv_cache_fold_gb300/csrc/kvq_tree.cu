// Attention of a tree of drafted tokens over the int4 cache or the e4m3 ring (kvq_tree_attn_*).
//
// Row i of sequence b attends to the context (the ring: to its window's part of it) and to the drafted
// tokens of its mask. The N x G query rows of a KV head share every key and value, so a page is read and
// converted once for up to 128 rows, and both products run on the tensor cores:
//
//   K, V  4-bit codes -> c s + o in fp16 (one rounding), e4m3 -> fp16 (exact), a page (64 tokens) at a time,
//         by four warps each into shared memory (K: K-major, V: MN-major, 128-byte swizzle)
//   S = Q' K^T     tcgen05.mma, 128 rows x 64 tokens, two buffers of S
//   P = 2^(c S - base + 7) in fp16 over S, one thread per row (as in kvq_prompt.cu: the base moves only
//         when a score passes it by more than 8, so P < 2^15)
//   O += P V       tcgen05.mma, P read from tensor memory
//
// Bound by the chain of a page's life, not by one unit: its copy, conversion, scores, weights and products hand over
// through one K and one V tile, so conversion waits until the page before is through (the commonest stall: its warps at
// their barrier, 4.8 per issue), with the tensor pipe 42% and the issue slots 60% busy, DRAM 27%. A page costs the same for
// 1 row as for 128 (fewer than 49 rows take kvq_attn.cu). 64 sequences of 16,384 tokens, 80 rows per KV head (581 MB,
// 1.7e11 operations): 303 us a call, of which the prologue 30 and the join 15. 8 of 32k-65k tokens, 320 rows, three
// groups that convert every page each: 301 us, 0.78 PFLOP/s. 64 windows of 513: 25.6 us.
//
// The rounding of q~, K, V and P to fp16 is what keeps both products on the tensor cores: 2^-11 each,
// against the 2^-8 of a bf16 result; sums, bases and O stay in fp32.
//
// The scores of the next page are issued before the weights of this one are ready. Two CTAs per SM, each
// with half of the tensor memory (two S of 64 columns, O 128).
//
// Work split: a segment is (sequence, KV head, group of 128 rows); the segments' pages are laid end to end
// and each CTA takes an equal contiguous part. A segment that one CTA has whole is finished there; of the
// others each CTA leaves an unnormalised partial, two at most (its first and its last piece), and
// tree_combine_kernel joins them. Short windows in large numbers are not split (launch_tree).
//
//   warps 0-3   softmax, Q', output (thread = row = tensor-memory lane)
//   warps 4-7   conversion of K (thread = token of the page and half of its dims), warps 8-11 of V
//   warp 12     copies of pages / ring blocks into shared-memory stages, K and V parts on rings of their own
//   warp 13     the products
//   warp 14     the CTA's pieces of segments, one ahead (kept out of the other roles' registers: spilled ones
//               would miss the little L1 that this much shared memory leaves)
// Groups of warps wait through one of them that watches the barrier, the others in a named barrier: with
// every warp polling, half of the instructions executed were polls.

#include <algorithm>
#include <mutex>

#include "kvq_internal.h"
#include "kvq_umma.cuh"

namespace kvq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kGroup = 128;                 // rows of a segment
constexpr int kTileBytes = kPage * kD * 2;  // fp16 tile of a page: two 64-dim halves of 64 rows of 128 bytes
constexpr int kHalf = kTileBytes / 2;
constexpr int kThreads = 512;
constexpr int kRegSoftmax = 104, kRegConv = 56, kRegAux = 40;  // from 64 at launch
static_assert(128 * (kRegSoftmax + 2 * kRegConv + kRegAux) <= kThreads * 64, "register shares above the launch's allocation");
constexpr float kKScale = 1.0f / 512.0f;  // of the int4 cache's K tiles (convert_k4)
constexpr uint32_t kColS = 0, kColO = 128;  // S of page i at + 64 (i & 1), P over its first 32 columns
constexpr int kQHalf = kGroup * 128;        // bytes of one 64-dim half of Q'
// K and V tiles. One of each, and the shared memory for copy stages instead: a second tile of K or V lets its
// conversion run ahead and take issue slots from the chain that everything waits for (64 x 16,384 x 16
// drafted: 314 us; two of V 333, two of K 350; not measured for short windows).
constexpr int kKBuf = 1, kVBuf = 1;
constexpr int kMaxTreeCtas = 320;                       // sizes the partials
constexpr int kMaxStages = 6;                           // of each ring
constexpr size_t kSmemCta = 233472 / 2 - 1024;          // two CTAs per SM (1 KB of each is the system's)
// Pages that a CTA takes at least where there are few: below this the fixed cost of a piece (Q', the partial,
// its share of the join) outweighs the shorter chain.
constexpr int kMinPages = 8;

struct TreeParams {
  TreeJob j;
  float c;         // |sm_scale| log2(e) (times k_scale), 1 where that is 0
  float qmul;      // sign of the scale (0 where it is 0), applied to q
  float vmul;      // applied to the output
  int G, R;        // query heads per KV head, rows of a KV head
  uint32_t g_inv;  // ceil(2^32 / G), 0 for G = 1
  int ng;          // row groups
  int nst;         // copy stages of each ring
  int whole;       // 1: CTA c takes the segments c, c + grid, ... as a whole; 0: equal parts of the line of pages
  float2* ml;      // partials: base and sum of each row, [2 CTAs][128]
  float* acc;      // and its 128 sums
  int* pre;        // pages of the sequences before each, [B + 1]
};

// One part (K or V) of a page in shared memory: int4 the 4096 bytes of codes, then the 256 of scales and offsets.
__host__ __device__ constexpr int part_bytes(int fmt) { return fmt == 0 ? kPage * kRec4 + kPage * 4 : kPage * kRec8; }

struct Piece {
  int b, h, g;      // segment; b < 0: no more pieces
  int j0, j1;       // its pages of this CTA, counted from page p0
  int ctx, first;   // context length, first position that some row sees
  int p0;           // page of position `first`
  int rows;         // rows of the group
  int whole, slot;  // whether these are all of the segment's pages; else the partial's slot
  int pad;
};

struct alignas(16) Smem {
  uint8_t q[2 * kQHalf];
  uint8_t k[kKBuf][kTileBytes];
  uint8_t v[kVBuf][kTileBytes];
  uint64_t raw_full[2][kMaxStages], raw_empty[2][kMaxStages];  // [K, V] part copied / read by its four warps
  uint64_t ready[2][2], freed[2][2];                           // [K, V][tile] written / its products complete
  uint64_t s_full[2], p_ready[2], o_full, q_ready, fin, pad;
  uint64_t piece_full[2], piece_empty[2];
  Piece piece[2];
  int valid[2][kMaxStages];  // the part was copied (its page lies in the pool)
  int pvalid[4];             // [page % 4] the page lies in the pool
  int failed;
  uint32_t taddr;
  // then: pre[B + 1], the rings
};

// Context length of sequence b: clamped into what the cache can hold (`bad` reports that). It and the masks are read at
// L2, not as read-only data: without new rows this is a call's first kernel, which starts before the grid ahead of it (a
// commit that writes the lengths, say) has ended.
__device__ __forceinline__ int tree_ctx(const TreeJob& j, int b, bool& bad) {
  int c = __ldcg(j.ctx + b);
  const int most = j.fmt == 0 ? j.cache.max_pages_per_seq * kPage - j.N : 1 << 30;
  if (c < 0 || c > most) {
    bad = true;
    c = max(0, min(c, most));
  }
  return c;
}
// First position that some row may see.
__device__ __forceinline__ int first_pos(const TreeJob& j, int ctx) { return j.fmt == 0 ? 0 : max(0, ctx - j.window + 1); }
__device__ __forceinline__ int num_pages(const TreeJob& j, int ctx) {
  return (ctx + j.N + kPage - 1) / kPage - first_pos(j, ctx) / kPage;
}

// pre[b] = pages of the sequences before b, by one warp (all of its lanes).
__device__ __forceinline__ void build_pre(const TreeJob& j, int* pre, bool report) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  bool bad = false;
  for (int b0 = 0; b0 < j.B; b0 += 32) {
    const int b = b0 + lane;
    int v = b < j.B ? num_pages(j, tree_ctx(j, b, bad)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (b < j.B) pre[b + 1] = sum + v;
    sum += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) pre[0] = 0;
  if (__any_sync(0xffffffffu, bad) && report && lane == 0) set_err(j.dev_err, KVQ_DEVERR_POS);
}

// The split of the line of pages: W in all, n CTAs in use, CTA c from X(c) on. n <= W, so every CTA has some.
struct Split {
  long long W;
  int n, per_seq;  // heads and groups of a sequence
  __device__ Split(const TreeParams& p, const int* pre, int ctas) {
    per_seq = p.j.Hkv * p.ng;
    W = (long long)per_seq * pre[p.j.B];
    n = (int)min((long long)ctas, max(1LL, W / kMinPages));
  }
  // (W n < 2^31 in practice: a 32-bit division takes a fifth of a 64-bit one's instructions)
  __device__ bool small() const { return W < (1 << 22); }
  __device__ long long X(int c) const { return small() ? (long long)((uint32_t)c * (uint32_t)W / (uint32_t)n) : (long long)c * W / n; }
  __device__ int owner(long long x) const {
    return small() ? (int)((((uint32_t)x + 1u) * (uint32_t)n - 1u) / (uint32_t)W) : (int)(((x + 1) * n - 1) / W);
  }
};

// The pieces of a CTA in order.
struct Pieces {
  const TreeParams& p;
  const int* pre;
  const Split& s;
  long long x, x1;
  int nb;   // pages of the piece's segment
  int seg;  // p.whole: the next segment
  __device__ Pieces(const TreeParams& p_, const int* pre_, const Split& s_, int c) : p(p_), pre(pre_), s(s_), seg(c) {
    x = c < s.n ? s.X(c) : 0;
    x1 = c < s.n ? s.X(c + 1) : 0;
  }
  __device__ bool next(Piece& o) {
    if (p.whole) {
      if (seg >= p.j.B * s.per_seq) return false;
      o.b = seg / s.per_seq;
      o.h = seg % s.per_seq / p.ng;
      o.g = seg % p.ng;
      nb = pre[o.b + 1] - pre[o.b];
      o.j0 = 0;
      o.j1 = nb;
      seg += gridDim.x;
      return true;
    }
    if (x >= x1) return false;
    int lo = 0, hi = p.j.B;  // the last b with pre[b] * per_seq <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * s.per_seq <= x) lo = mid;
      else hi = mid;
    }
    o.b = lo;
    nb = pre[lo + 1] - pre[lo];
    const long long rem = x - (long long)pre[lo] * s.per_seq;
    const int hg = (int)(rem / nb);
    o.h = hg / p.ng;
    o.g = hg % p.ng;
    o.j0 = (int)(rem - (long long)hg * nb);
    o.j1 = (int)min((long long)nb, o.j0 + (x1 - x));
    x += o.j1 - o.j0;
    return true;
  }
};

__device__ __forceinline__ int group_rows(const TreeParams& p, int g) { return min(kGroup, p.R - g * kGroup); }
// r / G (r < 4096)
__device__ __forceinline__ int div_g(const TreeParams& p, int r) { return p.g_inv ? (int)__umulhi((uint32_t)r, p.g_inv) : r; }
// Output row (of [B][N][Hq]) of row r of KV head h.
__device__ __forceinline__ size_t out_row(const TreeParams& p, int b, int h, int r) {
  const int i = div_g(p, r);
  return ((size_t)b * p.j.N + i) * p.j.Hq + h * p.G + (r - i * p.G);
}

__device__ __forceinline__ float half_lo(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
__device__ __forceinline__ float half_hi(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)(x >> 16))); }
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t both(float x) { return pack_f16x2(x, x); }


// Half of a token's K record -> its row of the K tile. Word w holds dims 8w..8w+7 in the order 0, 4, 1, 5, 2, 6, 3,
// 7 (as the nibbles pair up in 32 bits; Q' takes the same). A code is the subnormal c 2^-24 (even nibbles)
// or c 2^-20 (odd ones); the tile holds (c s + o) 2^-9, one fma a pair, so that s 2^15 fits fp16 for s < 2, which keys of
// norm sqrt(128) always have (a larger scale takes fp32). The fma rounds to fp16: off by 2^-11 of the value, or by 2^-16
// where the value is below 2^-5; o 2^-9 is exact in fp16 where |o| is 2^-5 or more and off by up to 2^-16 below. The
// scores take the 2^9 back. With a product by
// 2^15 of its own first: 64 x 16,384, 80 rows, 313 instead of 305 us.
// Places of a token's words of one half of the dims: word 8 part + 4 c + i at chunk(c) + off[i].
struct RowWords {
  uint8_t* row;     // the row in the part's half of the tile
  uint32_t off[4];  // 16 (i ^ low bits of the row)
  uint32_t hi;      // 64 where bit 2 of the row is set
  __device__ __forceinline__ RowWords(uint8_t* tile, int r, int part) : row(tile + part * kHalf + r * 128), hi((uint32_t)(r & 4) << 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = 16u * (uint32_t)(i ^ (r & 3));
  }
  __device__ __forceinline__ uint8_t* chunk(int c) const { return row + (((uint32_t)c << 6) ^ hi); }
};

template <bool WIDE>
__device__ __forceinline__ void convert_k4_as(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row, int part) {
  const int sw = k_chunk_swz(slot);
  const float s = half_lo(meta) * (16777216.0f * kKScale), o = half_hi(meta) * kKScale;
  const uint32_t s0 = both(s), s1 = both(s * 0.0625f), oo = both(o);
  const RowWords dst(tile, row, part);
  const uint4 r0 = *reinterpret_cast<const uint4*>(rec + 16 * ((2 * part) ^ sw));
  const uint4 r1 = *reinterpret_cast<const uint4*>(rec + 16 * ((2 * part + 1) ^ sw));
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint4 r = c ? r1 : r0;
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
    uint8_t* const out_c = dst.chunk(c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
      unpack8_sub(wd[i], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = e & 1 ? s * 0.0625f : s;
        if (WIDE) h[e] = pack_f16x2_sat(fmaf(half_lo(h[e]), m, o), fmaf(half_hi(h[e]), m, o));
        else h[e] = hfma2(h[e], e & 1 ? s1 : s0, oo);
      }
      *reinterpret_cast<uint4*>(out_c + dst.off[i]) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}
__device__ __noinline__ void convert_k4_wide(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row, int part) {
  convert_k4_as<true>(rec, slot, meta, tile, row, part);
}
__device__ __forceinline__ void convert_k4(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row, int part) {
  if (__builtin_expect(half_lo(meta) >= 2.0f, 0)) convert_k4_wide(rec, slot, meta, tile, row, part);
  else convert_k4_as<false>(rec, slot, meta, tile, row, part);
}

// Half of a token's V record -> its row of the V tile, dims in the same order. A code is the subnormal
// (c - 7.5) 2^(k - 23), k = 0, 4, 2, 6: times 2^15 plus 7.5 2^(k - 8) gives c 2^(k - 8) exactly, times
// s 2^(8 - k) plus o the value, rounded once. WIDE: scales from 255 on (s 2^8 would pass fp16's range) and
// offsets near it, in fp32 and saturating.
template <bool WIDE>
__device__ __forceinline__ void convert_v4_as(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row, int part) {
  const int sw = (slot >> 1) & 3;
  const uint32_t up = 0x78007800u;
  const float s = half_lo(meta), o = half_hi(meta);
  const float mul[4] = {256.0f, 16.0f, 64.0f, 4.0f};  // 2^(8 - k)
  uint32_t sc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sc[e] = both(s * mul[e]);
  const uint32_t oo = both(o);
  const RowWords dst(tile, row, part);
  const uint4 r0 = *reinterpret_cast<const uint4*>(rec + 16 * ((2 * part) ^ sw));
  const uint4 r1 = *reinterpret_cast<const uint4*>(rec + 16 * ((2 * part + 1) ^ sw));
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint4 r = c ? r1 : r0;
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
    uint8_t* const out_c = dst.chunk(c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
      unpack8_v(wd[i], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = hfma2(h[e], up, both(7.5f / mul[e]));
        if (WIDE) h[e] = pack_f16x2_sat(fmaf(half_lo(h[e]), s * mul[e], o), fmaf(half_hi(h[e]), s * mul[e], o));
        else h[e] = hfma2(h[e], sc[e], oo);
      }
      *reinterpret_cast<uint4*>(out_c + dst.off[i]) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}
__device__ __noinline__ void convert_v4_wide(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row, int part) {
  convert_v4_as<true>(rec, slot, meta, tile, row, part);
}
__device__ __forceinline__ void convert_v4(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row, int part) {
  if (__builtin_expect(half_lo(meta) >= 255.0f || fabsf(half_hi(meta)) > 60000.0f, 0)) convert_v4_wide(rec, slot, meta, tile, row, part);
  else convert_v4_as<false>(rec, slot, meta, tile, row, part);
}

// Half of a token's 128 e4m3 values -> its row of a tile, dims in order.
__device__ __forceinline__ void convert8(const uint8_t* rec, int slot, uint8_t* tile, int row, int part) {
  uint8_t* dst = tile + part * kHalf + row * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 r = *reinterpret_cast<const uint4*>(rec + 16 * ((4 * part + c) ^ (slot & 7)));
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 out;
      out.x = e4m3x2_to_f16x2(wd[2 * i]);
      out.y = e4m3x2_to_f16x2(wd[2 * i] >> 16);
      out.z = e4m3x2_to_f16x2(wd[2 * i + 1]);
      out.w = e4m3x2_to_f16x2(wd[2 * i + 1] >> 16);
      *reinterpret_cast<uint4*>(dst + 16 * ((2 * c + i) ^ (row & 7))) = out;
    }
  }
}

__device__ __forceinline__ void zero_row(uint8_t* tile, int row, int part) {
#pragma unroll 1
  for (int w = 0; w < 8; ++w) *reinterpret_cast<uint4*>(tile + part * kHalf + row * 128 + 16 * w) = make_uint4(0u, 0u, 0u, 0u);
}

// Column of dim d (0..7 of a word) in the tiles.
template <int FMT>
__device__ __forceinline__ constexpr int col_of(int d) {
  return FMT == 0 ? 2 * (d & 3) + (d >> 2) : d;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 2) tree_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const TreeJob& j = p.j;
  uint8_t* const ring = reinterpret_cast<uint8_t*>(&sm) + sizeof(Smem);  // [K, V][nst][part]
  int* const pre = reinterpret_cast<int*>(ring + 2 * p.nst * part_bytes(FMT));
  volatile int* failed = &sm.failed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int w = 0; w < 2; ++w) {
      for (int i = 0; i < kMaxStages; ++i) {
        mbar_init(&sm.raw_full[w][i], 1);
        mbar_init(&sm.raw_empty[w][i], 4);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.ready[w][i], 4);
        mbar_init(&sm.freed[w][i], 1);
      }
      mbar_init(&sm.s_full[w], 1);
      mbar_init(&sm.p_ready[w], 4);
      mbar_init(&sm.piece_full[w], 1);
      mbar_init(&sm.piece_empty[w], 14);  // copies, products, 8 conversion and 4 softmax warps
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.q_ready, 4);
    mbar_init(&sm.fin, 1);
    sm.failed = 0;
  }
  fence_barrier_init();
  // every grid before the previous one has completed, and the previous one's end waits for nothing here
  if (warp == 13) tmem_alloc_256(&sm.taddr);
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 14) {
    build_pre(j, pre, blockIdx.x == 0);
    __syncwarp();
    if (blockIdx.x == 0)  // for tree_combine_kernel
      for (int b = lane; b <= j.B; b += 32) p.pre[b] = pre[b];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.taddr;
  // Piece k as the schedule announced it; false at the end or after a wait that gave up.
  auto piece_at = [&](int k) {
    return __all_sync(0xffffffffu, role_wait(&sm.piece_full[k & 1], (uint32_t)(k >> 1) & 1u, failed)) && sm.piece[k & 1].b >= 0;
  };

  if (warp >= 12) {
    reg_dealloc<kRegAux>();
    if (warp == 14 && lane == 0) {
      // ------------------------------------------------------------ schedule
      const Split sp(p, pre, gridDim.x);
      Pieces it(p, pre, sp, blockIdx.x);
      for (int k = 0;; ++k) {
        Piece pc;
        if (it.next(pc)) {
          bool bad = false;
          pc.ctx = tree_ctx(j, pc.b, bad);
          pc.first = first_pos(j, pc.ctx);
          pc.p0 = pc.first / kPage;
          pc.rows = group_rows(p, pc.g);
          pc.whole = pc.j0 == 0 && pc.j1 == it.nb;
          pc.slot = (2 * blockIdx.x + (k > 0)) * kGroup;
        } else {
          pc.b = -1;
        }
        if (k >= 2 && !role_wait(&sm.piece_empty[k & 1], (uint32_t)(k / 2 - 1) & 1u, failed)) break;
        sm.piece[k & 1] = pc;
        mbar_arrive(&sm.piece_full[k & 1]);
        if (pc.b < 0) break;
      }
    } else if (warp == 12) {
      // ------------------------------------------------------------ copies
      const uint64_t pol = policy_evict_first();
      int issued = 0;  // pages so far
      int st = 0;      // stage of the next page
      uint32_t eph = 1;  // phase of its release (first round: none to wait for)
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!piece_at(k)) break;
        const Piece& pc = sm.piece[k & 1];
        const int pg1 = pc.p0 + pc.j1;
        for (int base = pc.p0 + pc.j0; ok && base < pg1; base += 32) {
          const uint8_t* src = nullptr;  // null: a page outside the pool
          const int pg = base + lane;
          if (pg < pg1) {
            if (FMT == 0) {
              const int phys = j.cache.block_table[(size_t)pc.b * j.cache.max_pages_per_seq + pg];
              if (phys >= 0 && phys < j.cache.num_pages) src = j.cache.pages + ((size_t)phys * j.Hkv + pc.h) * KVQ_INT4_BLOCK_BYTES;
              else set_err(j.dev_err, KVQ_DEVERR_PAGE);
            } else {
              const int nblk = j.ring.capacity / kPage;
              src = j.ring.data + (((size_t)pc.b * j.Hkv + pc.h) * nblk + pg % nblk) * (size_t)(2 * kPage * kRec8);
            }
          }
          const int n = min(32, pg1 - base);
          for (int i = 0; i < n; ++i) {
            const uint8_t* s = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i));
            if (lane == 0 && ok) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {  // K, then V
                ok = ok && (issued < p.nst || role_wait(&sm.raw_empty[w][st], eph, failed));
                if (!ok) break;
                uint64_t* full = &sm.raw_full[w][st];
                uint8_t* dst = ring + (size_t)(w * p.nst + st) * part_bytes(FMT);
                sm.valid[w][st] = s != nullptr;
                if (!s) {
                  mbar_arrive(full);
                } else if (FMT == 0) {
                  mbar_arrive_expect_tx(full, part_bytes(0));
                  bulk_g2s(dst, s + w * kPage * kRec4, kPage * kRec4, full, pol);
                  bulk_g2s(dst + kPage * kRec4, s + 2 * kPage * kRec4 + w * kPage * 4, kPage * 4, full, pol);
                } else {
                  mbar_arrive_expect_tx(full, part_bytes(1));
                  bulk_g2s(dst, s + w * kPage * kRec8, kPage * kRec8, full, pol);
                }
              }
              if (ok) {
                ++issued;
                if (++st == p.nst) {
                  st = 0;
                  eph ^= 1u;
                }
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.piece_empty[k & 1]);
      }
      if (*failed && lane == 0) {  // no copy may be in flight when the CTA ends (K of page `issued` may be under way as well)
        for (int u = max(0, issued - p.nst); u <= issued; ++u)
          for (int w = 0; w < 2; ++w)
            if (u < issued || w == 0) {
              const uint64_t t0 = globaltimer();
              while (!mbar_test(&sm.raw_full[w][u % p.nst], (uint32_t)(u / p.nst) & 1u) && globaltimer() - t0 < 20000000ull) {
              }
            }
      }
    } else if (warp == 13) {
      // ------------------------------------------------------------ products
      constexpr uint32_t kIdQK = umma_idesc_16(true, kPage, false), kIdPV = umma_idesc_16(true, kD, true);
      const uint32_t leader = elect_one();
      const uint32_t tm = (uint32_t)uniform((int)tmem);
      const uint64_t dq = umma_sdesc(smem_addr(sm.q), 16, 1024);
      const uint64_t dk = umma_sdesc(smem_addr(sm.k[0]), 16, 1024);
      const uint64_t dv = umma_sdesc(smem_addr(sm.v[0]), kHalf, 1024);
      auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(0xffffffffu, role_wait(bar, ph, failed)) != 0; };
      auto qk = [&](int c) {  // scores of page c of the CTA
        const int kb = c % kKBuf;
        if (!wait(&sm.ready[0][kb], (uint32_t)(c / kKBuf) & 1u)) return false;
        tc_fence_after();
        const uint64_t d = dk + (uint64_t)(kb * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // 16 dims each: 32 bytes within a 64-dim half
          umma_f16_by(leader, tm + kColS + 64 * (c & 1), dq + (uint64_t)(((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4),
                      d + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), kIdQK, kk > 0);
        umma_commit_by(leader, &sm.s_full[c & 1]);
        umma_commit_by(leader, &sm.freed[0][kb]);
        return true;
      };
      bool ok = true;
      int cnt = 0;  // pages so far
      for (int k = 0; ok; ++k) {
        if (!piece_at(k)) break;
        const int nb = uniform(sm.piece[k & 1].j1 - sm.piece[k & 1].j0);
        if (lane == 0) mbar_arrive(&sm.piece_empty[k & 1]);
        if (!(ok = wait(&sm.q_ready, (uint32_t)k & 1u))) break;
        if (!(ok = qk(cnt))) break;
        for (int i = 0; i < nb; ++i, ++cnt) {
          // S of the next page takes the place of the weights of the last, whose products are issued
          if (i + 1 < nb && !(ok = qk(cnt + 1))) break;
          const int vb = cnt % kVBuf;
          ok = wait(&sm.ready[1][vb], (uint32_t)(cnt / kVBuf) & 1u) && wait(&sm.p_ready[cnt & 1], (uint32_t)(cnt >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t d = dv + (uint64_t)(vb * (kTileBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 16 tokens each: 2048 bytes of a half of V, 8 columns of P
            umma_f16_ts_by(leader, tm + kColO, tm + kColS + 64 * (cnt & 1) + 8 * kk, d + (uint64_t)(kk * (2048 >> 4)), kIdPV, (kk > 0 || i > 0) ? 1u : 0u);
          umma_commit_by(leader, &sm.freed[1][vb]);
        }
        if (ok) umma_commit_by(leader, &sm.o_full);
      }
      umma_commit_by(leader, &sm.fin);  // arrives once every product issued has completed
      mbar_wait_bounded(&sm.fin, 0);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- conversion
    reg_dealloc<kRegConv>();
    const int is_v = warp >= 8;
    const bool poller = (warp & 3) == 0;
    const int slot = threadIdx.x & 63, part = (threadIdx.x >> 6) & 1;  // token, dims 64 part .. + 63
    int cnt = 0, st = 0;
    uint32_t sph = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!piece_at(k)) break;
      const Piece& pc = sm.piece[k & 1];
      const int first = pc.first, end = pc.ctx + j.N, pages = pc.j1 - pc.j0;
      int pos = (pc.p0 + pc.j0) * kPage + slot;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.piece_empty[k & 1]);
      for (int i = 0; i < pages; ++i, ++cnt, pos += kPage) {
        const int cb = is_v ? cnt % kVBuf : cnt % kKBuf, uses = is_v ? cnt / kVBuf : cnt / kKBuf;
        bool w = true;
        if (poller) {
          w = role_wait(&sm.raw_full[is_v][st], sph, failed);
          if (uses > 0) w = w && role_wait(&sm.freed[is_v][cb], (uint32_t)(uses - 1) & 1u, failed);
        }
        ok = !named_barrier_or(1 + is_v, 128, !w);
        if (!ok) break;
        const bool use = *reinterpret_cast<volatile int*>(&sm.valid[is_v][st]) != 0;
        if (slot == 0 && part == 0 && !is_v) sm.pvalid[cnt & 3] = use;
        const uint8_t* raw = ring + (size_t)(is_v * p.nst + st) * part_bytes(FMT);
        uint8_t* tile = is_v ? sm.v[cb] : sm.k[cb];
        if (!(use && pos >= first && pos < end)) {  // a token that no row may see
          zero_row(tile, slot, part);
        } else if (FMT == 0) {
          const uint32_t meta = reinterpret_cast<const uint32_t*>(raw + kPage * kRec4)[slot];
          if (is_v) convert_v4(raw + slot * kRec4, slot, meta, tile, slot, part);
          else convert_k4(raw + slot * kRec4, slot, meta, tile, slot, part);
        } else {
          convert8(raw + slot * kRec8, slot, tile, slot, part);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.ready[is_v][cb]);
          mbar_arrive(&sm.raw_empty[is_v][st]);
        }
        if (++st == p.nst) {
          st = 0;
          sph ^= 1u;
        }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax and output
    reg_alloc<kRegSoftmax>();
    const int r = threadIdx.x;  // row of the group
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    const uint32_t to = tmem + lane_base + kColO;
    const uint64_t all = j.N == 64 ? ~0ull : (1ull << j.N) - 1;
    int cnt = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!piece_at(k)) break;
      const Piece& pc = sm.piece[k & 1];
      const int ctx = pc.ctx, rows = pc.rows, r0 = pc.g * kGroup;
      const bool mine = r < rows, warp_rows = 32 * warp < rows;
      // ---- Q' of the warp's rows: 16 lanes read the 128 dims of a row, two rows at a time, sixteen in flight
      if (warp_rows) {
        const bool half_q = FMT == 1 && j.q_bf16;
        const int w = lane & 15;  // word of 8 dims
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          uint4 in[8][2];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int rr = 32 * warp + 16 * g + 2 * u + (lane >> 4);
            in[u][0] = in[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (rr < rows) {
              const size_t src = out_row(p, pc.b, pc.h, r0 + rr) * kD + 8 * w;
              if (half_q) {
                in[u][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(j.q) + src);
              } else {
                const uint4* q4 = reinterpret_cast<const uint4*>((FMT == 0 ? j.q_rot : static_cast<const float*>(j.q)) + src);
                in[u][0] = q4[0];
                in[u][1] = q4[1];
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int rr = 32 * warp + 16 * g + 2 * u + (lane >> 4);
            const uint32_t ww[8] = {in[u][0].x, in[u][0].y, in[u][0].z, in[u][0].w, in[u][1].x, in[u][1].y, in[u][1].z, in[u][1].w};
            float y[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              const float x = half_q ? bf16_bits_to_f32(d & 1 ? ww[d >> 1] >> 16 : ww[d >> 1] & 0xFFFFu) : __uint_as_float(ww[d]);
              y[col_of<FMT>(d)] = f16_query(x * p.qmul);
            }
            *reinterpret_cast<uint4*>(sm.q + (w >> 3) * kQHalf + rr * 128 + 16 * ((w & 7) ^ (rr & 7))) =
                make_uint4(pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3]), pack_f16x2(y[4], y[5]), pack_f16x2(y[6], y[7]));
          }
        }
        fence_proxy_async_shared();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_ready);
      // ---- this thread's row
      const uint64_t mask = mine ? __ldcg(reinterpret_cast<const unsigned long long*>(j.mask) + (size_t)pc.b * j.N + div_g(p, r0 + r)) & all : 0ull;
      const int lo = FMT == 0 ? 0 : max(0, ctx + max(1, __popcll(mask)) - j.window);  // first position that it sees
      float base = -INFINITY;
      uint64_t l2[2] = {0ull, 0ull};
      int pos0 = (pc.p0 + pc.j0) * kPage;
      const int pos1 = (pc.p0 + pc.j1) * kPage, pos_first = pos0;
      for (; pos0 < pos1; pos0 += kPage, ++cnt) {
        const uint32_t ts = tmem + lane_base + kColS + 64 * (cnt & 1);
        ok = group_wait(&sm.s_full[cnt & 1], (uint32_t)(cnt >> 1) & 1u, failed, warp == 0, 3, 128);
        if (!ok) break;
        tc_fence_after();
        if (warp_rows) {
          const bool pv = *reinterpret_cast<volatile int*>(&sm.pvalid[cnt & 3]) != 0;
          // pages that hold drafted tokens, lie outside the pool, or start before some row's window
          if (pos0 + kPage > ctx || !pv || (FMT == 1 && pos0 < ctx + j.N - j.window)) {
            const int cut = ctx - pos0;  // tokens from here on are drafted ones
            uint64_t m = cut <= 0 ? 0ull : cut >= 64 ? ~0ull : (1ull << cut) - 1;
            if (FMT == 1) {
              const int ll = lo - pos0;  // context tokens before this are outside the window
              if (ll > 0) m = ll >= 64 ? 0ull : m & ~((1ull << ll) - 1);
            }
            if (cut >= 0) m |= cut >= 64 ? 0ull : mask << cut;
            else if (cut > -64) m |= mask >> -cut;
            if (!pv) m = 0ull;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // rolled, over the scores in tensor memory (see kvq_prompt.cu)
              uint32_t s[32];
              tmem_ld32u(ts + 32 * h, s);
              tmem_wait_ld_all();
              const uint32_t mh = (uint32_t)(m >> (32 * h));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((mh >> i) & 1u)) s[i] = 0xFF800000u;
              tmem_st32u(ts + 32 * h, s);
            }
            tmem_wait_st();
          }
          uint32_t s[32];
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int h = 1; h >= 0; --h) {  // rolled: less code to fetch (316 -> 313 us); the first half stays in registers
            tmem_ld32u(ts + 32 * h, s);
            tmem_wait_ld_all();
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u) mx[u] = fmax3(mx[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
          const bool move = top > base + kBaseLag || (base == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, move)) {
            const float alpha = move ? fast_exp2(base - top) : 1.0f;
            if (move) base = top;
            l2[0] = mul_f2(l2[0], f2(alpha, alpha));
            l2[1] = mul_f2(l2[1], f2(alpha, alpha));
            // O of the first page starts anew; else once the product before is done
            if (pos0 > pos_first &&
                __all_sync(0xffffffffu, role_wait(&sm.freed[1][(cnt - 1) % kVBuf], (uint32_t)((cnt - 1) / kVBuf) & 1u, failed))) {
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {
                uint32_t o[16];
                tmem_ld16u(to + 16 * i, o);
                tmem_wait_ld_all();
#pragma unroll
                for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
                tmem_st16u(to + 16 * i, o);
              }
            }
          }
          const float neg = base == -INFINITY ? 0.0f : kWeightRaise - base;
          const uint64_t c2 = f2(p.c, p.c), n2 = f2(neg, neg);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t x = fma_f2(f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, n2);
              const float e0 = fast_exp2(f2lo(x)), e1 = fast_exp2(f2hi(x));
              l2[i & 1] = add_f2(l2[i & 1], f2(e0, e1));
              pk[i] = pack16x2<true>(e0, e1);
            }
            tmem_st16u(ts + 16 * h, pk);
            if (h == 0) {
              tmem_ld32u(ts + 32, s);
              tmem_wait_ld_all();
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[cnt & 1]);
      }
      if (!ok) break;
      ok = group_wait(&sm.o_full, (uint32_t)k & 1u, failed, warp == 0, 3, 128);
      if (!ok) break;
      tc_fence_after();
      // ---- end of the piece: the result, or a partial of it
      const float l = (f2lo(l2[0]) + f2hi(l2[0])) + (f2lo(l2[1]) + f2hi(l2[1]));
      const bool whole = pc.whole != 0;
      const float f = whole ? (l > 0.0f || l != l ? p.vmul / l : 0.0f) : 1.0f;
      if (!whole && mine) p.ml[(size_t)pc.slot + r] = make_float2(base, l);
      if (warp_rows) {
        // 32 dims at a time through the warp's own rows of Q' (no product reads them any more), so that 8 lanes
        // write 32 dims of a row
        const int lr = lane >> 3, lc = lane & 7;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint8_t* const stage = sm.q + (c & 1) * kQHalf + 32 * warp * 128;
          uint32_t x[32];
          tmem_ld32u(to + 32 * c, x);
          tmem_wait_ld_all();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = l == 0.0f ? 0.0f : __uint_as_float(x[i]) * f;  // nothing seen: 0
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int g8 = 8 * (i >> 1), d = 4 * (i & 1);
            *reinterpret_cast<float4*>(stage + lane * 128 + 16 * (i ^ (lane & 7))) =
                make_float4(v[g8 + col_of<FMT>(d)], v[g8 + col_of<FMT>(d + 1)], v[g8 + col_of<FMT>(d + 2)], v[g8 + col_of<FMT>(d + 3)]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + lr, dim = 32 * c + 4 * lc;
            if (32 * warp + rr >= rows) continue;
            const float4 o = *reinterpret_cast<const float4*>(stage + rr * 128 + 16 * (lc ^ (rr & 7)));
            if (!whole) {
              *reinterpret_cast<float4*>(p.acc + ((size_t)pc.slot + 32 * warp + rr) * kD + dim) = o;
            } else {
              const size_t at = out_row(p, pc.b, pc.h, r0 + 32 * warp + rr) * kD + dim;
              if (j.out_bf16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.out) + at) = make_uint2(pack16x2<false>(o.x, o.y), pack16x2<false>(o.z, o.w));
              else *reinterpret_cast<float4*>(static_cast<float*>(j.out) + at) = o;
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.piece_empty[k & 1]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc_256(tmem);
  if (threadIdx.x == 0 && *failed) set_err(j.dev_err, KVQ_DEVERR_TIMEOUT);
}

// Joins the partials of the segments that several CTAs shared, in the order of the CTAs: one block per
// segment and 8 rows of it, one warp per row, four dims a lane. A first pass (a lane per partial) takes
// the bases and sums, so that the second has its factors ready and its loads are independent.
constexpr int kCombineWarps = 8;
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const __grid_constant__ TreeParams p, int ctas) {
  const TreeJob& j = p.j;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x, g = seg % p.ng, h = seg / p.ng % j.Hkv, b = seg / p.ng / j.Hkv;
  const int r = blockIdx.y * kCombineWarps + warp;
  if (r >= group_rows(p, g)) return;
  griddep_wait();
  griddep_launch_dependents();
  const Split sp(p, p.pre, ctas);
  const int pb = p.pre[b], nb = p.pre[b + 1] - pb;
  const long long xs = (long long)pb * sp.per_seq + (long long)(h * p.ng + g) * nb;
  const int ca = sp.owner(xs), cb = sp.owner(xs + nb - 1);
  if (ca == cb) return;
  const bool second = xs > sp.X(ca);  // the segment starts within its first CTA's part
  auto slot = [&](int c) { return (size_t)(2 * c + (c == ca && second ? 1 : 0)) * kGroup + r; };
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = ca; c0 <= cb; c0 += 32) {
    const int n = min(32, cb - c0 + 1);
    const float2 ml = lane < n ? p.ml[slot(c0 + lane)] : make_float2(-INFINITY, 0.0f);
    const float mn = fmaxf(m, warp_max_all(ml.x));
    const float f0 = m == -INFINITY ? 0.0f : exp2f(m - mn), f1 = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - mn);
    float part = ml.y != ml.y ? ml.y : ml.y * f1;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) part += __shfl_xor_sync(0xffffffffu, part, s);
    l = l * f0 + part;
    o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
    m = mn;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float f = __shfl_sync(0xffffffffu, f1, i);
      const float4 a = reinterpret_cast<const float4*>(p.acc + slot(c0 + i) * kD)[lane];
      o.x = fmaf(a.x, f, o.x), o.y = fmaf(a.y, f, o.y), o.z = fmaf(a.z, f, o.z), o.w = fmaf(a.w, f, o.w);
    }
  }
  const float f = l > 0.0f || l != l ? p.vmul / l : 0.0f;
  const size_t at = out_row(p, b, h, g * kGroup + r) * kD + 4 * lane;
  if (j.out_bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.out) + at) = make_uint2(pack16x2<false>(o.x * f, o.y * f), pack16x2<false>(o.z * f, o.w * f));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(j.out) + at) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
}

std::mutex g_mu;  // guards the cache below
bool g_attr[64][2] = {{false}};

template <int FMT>
cudaError_t launch_t(TreeParams& p, long long pages_max, cudaStream_t stream) {
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (dev < 0 || dev >= 64 || !g_attr[dev][FMT]) {
      e = cudaFuncSetAttribute(tree_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemCta);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(tree_kernel<FMT>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) g_attr[dev][FMT] = true;
    }
  }
  const size_t fixed = sizeof(Smem) + 4 * ((size_t)p.j.B + 1) + 1024;  // + alignment to 1024 bytes
  p.nst = std::min<int>(kMaxStages, (int)((kSmemCta - fixed) / (2 * part_bytes(FMT))));
  const size_t smem = fixed + (size_t)p.nst * 2 * part_bytes(FMT);
  static_assert(sizeof(Smem) % 16 == 0 && kSmemCta - sizeof(Smem) - 1024 - 4 * (KVQ_MAX_SEQS + 1) >= 2 * part_bytes(1), "no room for a copy stage");
  const int sms = device_sms();
  const long long segs = (long long)p.j.B * p.j.Hkv * p.ng;
  // Windows of few pages are taken whole once there is one for every SM: a CTA then pays for Q' and the output
  // once, there are no partials, and the joining launch is saved (64 x 4 windows of 513: 46 -> 26 us).
  p.whole = FMT == 1 && segs >= sms && p.j.window + p.j.N <= 16 * kPage;
  const int ctas = (int)std::max<long long>(1, std::min<long long>(p.whole ? segs : pages_max, std::min(2 * sms, kMaxTreeCtas)));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_kernel<FMT>, p);
  if (e != cudaSuccess || p.whole) return e;
  cfg.gridDim = dim3((unsigned)segs, (unsigned)((std::min(p.R, kGroup) + kCombineWarps - 1) / kCombineWarps), 1);
  cfg.blockDim = dim3(kCombineWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel, p, ctas);
}

}  // namespace

size_t workspace_tree_partials_bytes(int B) {
  return (size_t)2 * kMaxTreeCtas * kGroup * (2 + kD) * 4 + 4 * ((size_t)B + 1);
}

cudaError_t launch_tree(const TreeJob& job, cudaStream_t stream) {
  TreeParams p{};
  p.j = job;
  const float c = job.sm_scale * kLog2e * (job.fmt == 1 ? job.k_scale : 1.0f / kKScale);
  p.qmul = c > 0.0f ? 1.0f : c < 0.0f ? -1.0f : 0.0f;
  p.c = c == 0.0f ? 1.0f : (c < 0.0f ? -c : c);
  p.vmul = job.fmt == 1 ? job.v_scale : 1.0f;
  p.G = job.Hq / job.Hkv;
  p.g_inv = p.G == 1 ? 0u : (uint32_t)(((1ull << 32) + p.G - 1) / p.G);
  p.R = job.N * p.G;
  p.ng = (p.R + kGroup - 1) / kGroup;
  p.ml = reinterpret_cast<float2*>(job.partials);
  p.acc = job.partials + (size_t)2 * 2 * kMaxTreeCtas * kGroup;
  p.pre = reinterpret_cast<int*>(p.acc + (size_t)2 * kMaxTreeCtas * kGroup * kD);
  const long long pages = job.fmt == 0 ? job.cache.max_pages_per_seq : job.ring.capacity / kPage + 1;
  const long long most = pages * job.B * job.Hkv * p.ng;
  return job.fmt == 0 ? launch_t<0>(p, most, stream) : launch_t<1>(p, most, stream);
}

}  // namespace kvq
