// Attention of a tree of drafted tokens over the int4 cache or the e4m3 ring (kvq_tree_attn_*).
//
// Row i of sequence b attends to the context (the ring: to its window's part of it) and to the drafted
// tokens of its mask. The N x G query rows of a KV head share every key and value, so the cache is read
// and converted once for up to 256 rows, and both products run on the tensor cores:
//
//   K, V  4-bit codes -> c s + o in fp16 (one rounding), e4m3 -> fp16 (exact), 128 tokens a block,
//         converted by four warps into shared memory (K: K-major, V: MN-major, 128-byte swizzle)
//   S = Q' K^T     tcgen05.mma, 128 rows x 128 tokens, accumulators in tensor memory
//   P = 2^(c S - base) in fp16 over S, one thread per row (as in kvq_prompt.cu: the base moves only
//         when a score passes it by more than 8, so P < 2^8)
//   O += P V       tcgen05.mma, P read from tensor memory
//
// The rounding of q~, K, V and P to fp16 is what keeps both products on the tensor cores: 2^-11 each,
// against the 2^-8 of a bf16 result; sums, bases and O stay in fp32.
//
// Two streams of (S, P, O) take turns, so that the tensor cores work on one while the softmax warps have
// the other: with more than 128 rows they are two row tiles over the same blocks, else two halves of the
// blocks (even, odd) over the same rows, joined at the end of a segment in tensor memory.
//
// Work split: a segment is (sequence, KV head, group of 256 rows); the segments' blocks are laid end to
// end and each CTA (one per SM) takes a contiguous part of equal weight (a block counts its row tiles). A
// segment that one CTA has whole is finished there; of the others each CTA leaves an unnormalised partial,
// two at most (its first and its last piece), and tree_combine_kernel joins them.
//
//   warps 0-3, 4-7  softmax of stream 0 and 1, Q' tiles, output (thread = row = tensor-memory lane)
//   warps 8-11      conversion of K (thread = token of the block)
//   warps 12-15     conversion of V
//   warp 16         copies of pages / ring blocks into shared-memory stages
//   warp 17         the products (one issuing thread)
//   warp 18         the CTA's pieces of segments, one ahead (kept out of the other roles' registers: spilled
//                   ones would miss the little L1 that this much shared memory leaves)

#include <algorithm>
#include <mutex>

#include "kvq_internal.h"
#include "kvq_umma.cuh"

namespace kvq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBlk = 128;                  // tokens of a block: two pages
constexpr int kGroup = 256;                // rows of a segment
constexpr int kTileBytes = kBlk * kD * 2;  // fp16 tile: two 64-dim halves of 128 rows of 128 bytes
constexpr int kHalf = kTileBytes / 2;
constexpr int kThreads = 640;
constexpr int kRegSoftmax = 120, kRegConv = 80, kRegAux = 80;  // from 96 at launch
static_assert(256 * kRegSoftmax + 256 * kRegConv + 128 * kRegAux <= kThreads * 96, "register shares above the launch's allocation");
constexpr uint32_t kColS = 0, kColO = 256;  // stream t at + 128 t; P over the first 64 columns of S
constexpr int kMaxTreeCtas = 256;           // sizes the partials
constexpr int kMaxStages = 8;
constexpr size_t kSmemMax = 227 * 1024;

struct TreeParams {
  TreeJob j;
  float c;      // |sm_scale| log2(e) (times k_scale), 1 where that is 0
  float qmul;   // sign of the scale (0 where it is 0), applied to q
  float vmul;   // applied to the output
  int G, R;     // query heads per KV head, rows of a KV head
  int ng;       // row groups
  int w_last;   // row tiles of the last group (all others: 2)
  int nst;      // copy stages
  float2* ml;   // partials: base and sum of each row, [2 CTAs][rows]
  float* acc;   // and its 128 sums
  int* pre;     // blocks of the sequences before each, [B + 1]
  int prow;     // rows of a partial slot: 128 or 256
};

__host__ __device__ constexpr int stage_bytes(int fmt) { return fmt == 0 ? KVQ_INT4_BLOCK_BYTES : 2 * kPage * kRec8; }

struct Layout {  // offsets from the 1024-byte aligned start of dynamic shared memory
  uint32_t q, k, v, raw, bars, piece, valid, bvalid, state, pre, total;
  __host__ __device__ Layout(int fmt, int qtiles, int nst, int B) {
    q = 0;
    k = q + qtiles * kTileBytes;
    v = k + 2 * kTileBytes;
    raw = v + 2 * kTileBytes;
    bars = raw + nst * stage_bytes(fmt);  // a multiple of 16
    piece = bars + 8 * 40;
    valid = piece + 2 * 64;
    bvalid = valid + 4 * kMaxStages;
    state = bvalid + 4 * 8;  // failed flag, tensor-memory address
    pre = state + 8;
    total = pre + 4 * (B + 1);
  }
};

// Context length of sequence b: clamped into what the cache can hold (`bad` reports that).
__device__ __forceinline__ int tree_ctx(const TreeJob& j, int b, bool& bad) {
  int c = __ldg(j.ctx + b);
  const int most = j.fmt == 0 ? j.cache.max_pages_per_seq * kPage - j.N : 1 << 30;
  if (c < 0 || c > most) {
    bad = true;
    c = max(0, min(c, most));
  }
  return c;
}
// First position that some row may see, and the page it lies in.
__device__ __forceinline__ int first_pos(const TreeJob& j, int ctx) { return j.fmt == 0 ? 0 : max(0, ctx - j.window + 1); }
__device__ __forceinline__ int num_blocks(const TreeJob& j, int ctx) {
  const int p0 = first_pos(j, ctx) / kPage, p1 = (ctx + j.N + kPage - 1) / kPage;
  return (p1 - p0 + 1) / 2;
}

// pre[b] = blocks of the sequences before b, by one warp (all of its lanes).
__device__ __forceinline__ void build_pre(const TreeJob& j, int* pre, bool report) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  bool bad = false;
  for (int b0 = 0; b0 < j.B; b0 += 32) {
    const int b = b0 + lane;
    int v = b < j.B ? num_blocks(j, tree_ctx(j, b, bad)) : 0;
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

// The split of the weight line: W in all, n CTAs in use, CTA c from X(c) on. A block belongs to the CTA in
// whose part its start lies; n is at most W over the largest weight, so every CTA of a segment's span has
// some of its blocks.
struct Split {
  long long W;
  int n, per_seq;  // weight of one block in all heads and groups of a sequence
  __device__ Split(const TreeParams& p, const int* pre, int ctas) {
    const int wg = 2 * (p.ng - 1) + p.w_last;
    per_seq = p.j.Hkv * wg;
    W = (long long)per_seq * pre[p.j.B];
    const int wmax = p.ng > 1 ? 2 : p.w_last;
    n = (int)min((long long)ctas, W / wmax);
  }
  __device__ long long X(int c) const { return (long long)c * W / n; }
  __device__ int owner(long long x) const { return (int)(((x + 1) * n - 1) / W); }
};

struct Piece {
  int b, h, g, w;    // segment and its row tiles; w = 0: no more pieces
  int j0, j1;        // its blocks of this CTA
  int ctx, first;    // context length, first position that some row sees
  int p0, p1;        // pages that hold positions first .. ctx + N - 1
  int rows, rows0;   // rows of the group and of its first tile
  int whole, slot;   // whether these are all of the segment's blocks; else the partial's slot
};

// The pieces of a CTA in order.
struct Pieces {
  const TreeParams& p;
  const int* pre;
  const Split& s;
  long long x, x1;
  int nb;  // blocks of the piece's segment
  __device__ Pieces(const TreeParams& p_, const int* pre_, const Split& s_, int c) : p(p_), pre(pre_), s(s_) {
    x = c < s.n ? s.X(c) : 0;
    x1 = c < s.n ? s.X(c + 1) : 0;
  }
  __device__ __noinline__ bool next(Piece& o) {
    while (x < x1) {
      int lo = 0, hi = p.j.B;  // the last b with pre[b] * per_seq <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)pre[mid] * s.per_seq <= x) lo = mid;
        else hi = mid;
      }
      o.b = lo;
      nb = pre[lo + 1] - pre[lo];
      long long rem = x - (long long)pre[lo] * s.per_seq;
      const long long per_head = (long long)nb * (s.per_seq / p.j.Hkv);
      o.h = (int)(rem / per_head);
      rem -= o.h * per_head;
      o.g = (int)min(rem / (2 * nb), (long long)(p.ng - 1));
      const long long off = rem - (long long)o.g * 2 * nb;
      o.w = o.g < p.ng - 1 ? 2 : p.w_last;
      const long long xs = x - off, xe = xs + (long long)nb * o.w;
      o.j0 = (int)((off + o.w - 1) / o.w);
      o.j1 = xe <= x1 ? nb : (int)((x1 - xs + o.w - 1) / o.w);
      x = xe;
      if (o.j0 < o.j1) return true;
    }
    return false;
  }
};

// Rows of the group, and of its first tile (two tiles: about half each, whole warps).
__device__ __forceinline__ int group_rows(const TreeParams& p, int g) { return min(kGroup, p.R - g * kGroup); }
__device__ __forceinline__ int tile0_rows(int rows, int w) { return w == 1 ? rows : min(kBlk, ((rows + 1) / 2 + 31) & ~31); }

__device__ __forceinline__ float half_lo(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
__device__ __forceinline__ float half_hi(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)(x >> 16))); }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t both(float x) { return pack_f16x2(x, x); }

// Place of 8-dim word w (0..15) of row r in an fp16 tile.
__device__ __forceinline__ uint32_t tile_offset(int r, int w) { return (w >> 3) * kHalf + r * 128 + 16 * ((w & 7) ^ (r & 7)); }

// One token's K record -> its row of the K tile. Word w holds dims 8w..8w+7 in the order 0, 4, 1, 5, 2, 6, 3,
// 7 (as the nibbles pair up in 32 bits; Q' takes the same). A code is the subnormal c 2^-24 (even nibbles)
// or c 2^-20 (odd ones): one exact product by 2^15, then c s + o rounded once.
// Places of a token's words: word 4 c + i at chunk(c) + off[i].
struct RowWords {
  uint8_t* row;
  uint32_t off[4];  // 16 (i ^ low bits of the row)
  uint32_t hi;      // 64 where bit 2 of the row is set
  __device__ __forceinline__ RowWords(uint8_t* tile, int r) : row(tile + r * 128), hi((uint32_t)(r & 4) << 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = 16u * (uint32_t)(i ^ (r & 3));
  }
  __device__ __forceinline__ uint8_t* chunk(int c) const { return row + (c >> 1) * kHalf + (((uint32_t)(c & 1) << 6) ^ hi); }
};

__device__ __forceinline__ void convert_k4(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row) {
  const int sw = k_chunk_swz(slot);
  const uint32_t up = 0x78007800u;  // 2^15
  const float s = half_lo(meta);
  const uint32_t s0 = both(s * 512.0f), s1 = both(s * 32.0f), oo = both(half_hi(meta));
  // a loop, not unrolled: the roles of the CTA together are more code than the instruction caches hold
  const RowWords dst(tile, row);
  uint4 r = *reinterpret_cast<const uint4*>(rec + 16 * sw);
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    const uint4 next = *reinterpret_cast<const uint4*>(rec + 16 * (((c + 1) & 3) ^ sw));
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
    uint8_t* const out_c = dst.chunk(c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
      unpack8_sub(wd[i], h);
      uint4 out;
      out.x = hfma2(hmul2(h[0], up), s0, oo);
      out.y = hfma2(hmul2(h[1], up), s1, oo);
      out.z = hfma2(hmul2(h[2], up), s0, oo);
      out.w = hfma2(hmul2(h[3], up), s1, oo);
      *reinterpret_cast<uint4*>(out_c + dst.off[i]) = out;
    }
    r = next;
  }
}

// One token's V record -> its row of the V tile, dims in the same order. A code is the subnormal
// (c - 7.5) 2^(k - 23), k = 0, 4, 2, 6: times 2^15 plus 7.5 2^(k - 8) gives c 2^(k - 8) exactly, times
// s 2^(8 - k) plus o the value, rounded once. WIDE: scales from 255 on (s 2^8 would pass fp16's range) and
// offsets near it, in fp32 and saturating.
template <bool WIDE>
__device__ __forceinline__ void convert_v4_as(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row) {
  const int sw = (slot >> 1) & 3;
  const uint32_t up = 0x78007800u;
  const float s = half_lo(meta), o = half_hi(meta);
  const float mul[4] = {256.0f, 16.0f, 64.0f, 4.0f};  // 2^(8 - k)
  uint32_t sc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sc[e] = both(s * mul[e]);
  const uint32_t oo = both(o);
  const RowWords dst(tile, row);
  uint4 r = *reinterpret_cast<const uint4*>(rec + 16 * sw);
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    const uint4 next = *reinterpret_cast<const uint4*>(rec + 16 * (((c + 1) & 3) ^ sw));
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
    r = next;
  }
}
__device__ __noinline__ void convert_v4_wide(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row) {
  convert_v4_as<true>(rec, slot, meta, tile, row);
}
__device__ __forceinline__ void convert_v4(const uint8_t* rec, int slot, uint32_t meta, uint8_t* tile, int row) {
  if (__builtin_expect(half_lo(meta) >= 255.0f || fabsf(half_hi(meta)) > 60000.0f, 0)) convert_v4_wide(rec, slot, meta, tile, row);
  else convert_v4_as<false>(rec, slot, meta, tile, row);
}

// One token's 128 e4m3 values -> its row of a tile, dims in order.
__device__ __forceinline__ void convert8(const uint8_t* rec, int slot, uint8_t* tile, int row) {
  uint8_t* dst = tile + row * 128;
#pragma unroll 2
  for (int c = 0; c < 8; ++c) {
    const uint4 r = *reinterpret_cast<const uint4*>(rec + 16 * (c ^ (slot & 7)));
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 out;
      out.x = e4m3x2_to_f16x2(wd[2 * i]);
      out.y = e4m3x2_to_f16x2(wd[2 * i] >> 16);
      out.z = e4m3x2_to_f16x2(wd[2 * i + 1]);
      out.w = e4m3x2_to_f16x2(wd[2 * i + 1] >> 16);
      *reinterpret_cast<uint4*>(dst + (c >> 2) * kHalf + 16 * ((2 * (c & 3) + i) ^ (row & 7))) = out;
    }
  }
}

__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll 1
  for (int w = 0; w < 16; ++w) *reinterpret_cast<uint4*>(tile + (w >> 3) * kHalf + row * 128 + 16 * (w & 7)) = make_uint4(0u, 0u, 0u, 0u);
}

// Column of dim d (0..7 of a word) in the tiles, and its inverse order for the output.
template <int FMT>
__device__ __forceinline__ constexpr int col_of(int d) {
  return FMT == 0 ? 2 * (d & 3) + (d >> 2) : d;
}

// Output row (of [B][N][Hq]) of row r of KV head h.
__device__ __forceinline__ size_t out_row(const TreeParams& p, int b, int h, int r) {
  return ((size_t)b * p.j.N + r / p.G) * p.j.Hq + h * p.G + r % p.G;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const TreeJob& j = p.j;
  const Layout L(FMT, p.prow / 128, p.nst, j.B);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* raw_full = bars;             // [8] a page copied
  uint64_t* raw_empty = bars + 8;        // [8] and read (the two K and two V warps of its tokens)
  uint64_t* k_ready = bars + 16;         // [2] K tile written
  uint64_t* v_ready = bars + 18;         // [2]
  uint64_t* k_free = bars + 20;          // [2] products over it complete
  uint64_t* v_free = bars + 22;          // [2]
  uint64_t* s_full = bars + 24;          // [2] scores of a stream complete
  uint64_t* p_ready = bars + 26;         // [2] weights written
  uint64_t* o_full = bars + 28;          // [2] a piece's last product of a stream complete
  uint64_t* q_ready = bars + 30;         // Q' of a piece written
  uint64_t* fin = bars + 31;
  uint64_t* piece_full = bars + 32;      // [2] a piece announced
  uint64_t* piece_empty = bars + 34;     // [2] and left behind by every role
  Piece* pieces = reinterpret_cast<Piece*>(smem + L.piece);
  static_assert(sizeof(Piece) <= 64, "pieces larger than their shared-memory region");
  volatile int* valid = reinterpret_cast<volatile int*>(smem + L.valid);    // [stage] the page was copied
  volatile int* bvalid = reinterpret_cast<volatile int*>(smem + L.bvalid);  // [block % 4][page] it exists in the pool
  volatile int* failed = reinterpret_cast<volatile int*>(smem + L.state);
  uint32_t* taddr = reinterpret_cast<uint32_t*>(smem + L.state + 4);
  int* pre = reinterpret_cast<int*>(smem + L.pre);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(raw_full + i, 1);
      mbar_init(raw_empty + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_ready + i, 4);
      mbar_init(v_ready + i, 4);
      mbar_init(k_free + i, 1);
      mbar_init(v_free + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + i, 4);
      mbar_init(o_full + i, 1);
      mbar_init(piece_full + i, 1);
      mbar_init(piece_empty + i, 18);  // copies, products, 8 conversion and 8 softmax warps
    }
    mbar_init(q_ready, 8);
    mbar_init(fin, 1);
    *failed = 0;
  }
  fence_barrier_init();
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) {
    build_pre(j, pre, blockIdx.x == 0);
    if (blockIdx.x == 0)  // for tree_combine_kernel
      for (int b = lane; b <= j.B; b += 32) p.pre[b] = pre[b];
  }
  if (warp == 17) tmem_alloc_512(taddr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *taddr;
  // Piece k as the schedule announced it; false at the end or after a wait that gave up.
  auto piece_at = [&](int k) {
    return role_wait(piece_full + (k & 1), (uint32_t)(k >> 1) & 1u, failed) && pieces[k & 1].w != 0;
  };

  if (warp >= 16) {
    reg_dealloc<kRegAux>();
    if (warp == 18 && lane == 0) {
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
          pc.p1 = (pc.ctx + j.N + kPage - 1) / kPage;
          pc.rows = group_rows(p, pc.g);
          pc.rows0 = tile0_rows(pc.rows, pc.w);
          pc.whole = pc.j0 == 0 && pc.j1 == it.nb;
          pc.slot = (2 * blockIdx.x + (k > 0)) * p.prow;
        } else {
          pc.w = 0;
        }
        if (k >= 2 && !role_wait(piece_empty + (k & 1), (uint32_t)(k / 2 - 1) & 1u, failed)) break;
        pieces[k & 1] = pc;
        mbar_arrive(piece_full + (k & 1));
        if (pc.w == 0) break;
      }
    } else if (warp == 16) {
      // ------------------------------------------------------------ copies
      const uint64_t pol = policy_evict_first();
      int issued = 0;  // pages so far
      int st = 0;      // stage of the next page
      uint32_t eph = 1;  // phase of its release (first round: none to wait for)
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!__all_sync(0xffffffffu, piece_at(k))) break;
        const Piece& pc = pieces[k & 1];
        const int pg1 = min(pc.p0 + 2 * pc.j1, pc.p1);
        for (int base = pc.p0 + 2 * pc.j0; ok && base < pg1; base += 32) {
          const uint8_t* src = nullptr;  // null: a page outside the pool
          const int pg = base + lane;
          if (pg < pg1) {
            if (FMT == 0) {
              const int phys = j.cache.block_table[(size_t)pc.b * j.cache.max_pages_per_seq + pg];
              if (phys >= 0 && phys < j.cache.num_pages) src = j.cache.pages + ((size_t)phys * j.Hkv + pc.h) * KVQ_INT4_BLOCK_BYTES;
              else set_err(j.dev_err, KVQ_DEVERR_PAGE);
            } else {
              const int nblk = j.ring.capacity / kPage;
              src = j.ring.data + (((size_t)pc.b * j.Hkv + pc.h) * nblk + pg % nblk) * (size_t)stage_bytes(1);
            }
          }
          const int n = min(32, pg1 - base);
          for (int i = 0; i < n; ++i) {
            const uint8_t* s = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i));
            if (lane == 0 && ok) {
              ok = issued < p.nst || role_wait(raw_empty + st, eph, failed);
              if (ok) {
                valid[st] = s != nullptr;
                if (s) {
                  mbar_arrive_expect_tx(raw_full + st, stage_bytes(FMT));
                  bulk_g2s(smem + L.raw + st * stage_bytes(FMT), s, stage_bytes(FMT), raw_full + st, pol);
                } else {
                  mbar_arrive(raw_full + st);
                }
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
        if (lane == 0) mbar_arrive(piece_empty + (k & 1));
      }
      if (*failed && lane == 0)  // no copy may be in flight when the CTA ends
        for (int u = max(0, issued - p.nst); u < issued; ++u) mbar_wait_bounded(raw_full + u % p.nst, (uint32_t)(u / p.nst) & 1u);
    } else if (warp == 17) {
      // ------------------------------------------------------------ products
      constexpr uint32_t kIdQK = umma_idesc_16(true, kBlk, false), kIdPV = umma_idesc_16(true, kD, true);
      const uint32_t leader = elect_one();
      const uint32_t tm = (uint32_t)uniform((int)tmem);
      const uint64_t dq = umma_sdesc(smem_addr(smem + L.q), 16, 1024);
      const uint64_t dk = umma_sdesc(smem_addr(smem + L.k), 16, 1024);
      const uint64_t dv = umma_sdesc(smem_addr(smem + L.v), kHalf, 1024);
      auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(0xffffffffu, role_wait(bar, ph, failed)) != 0; };
      auto wait2 = [&](uint64_t* bar, int cnt) { return wait(bar + (cnt & 1), (uint32_t)(cnt >> 1) & 1u); };
      auto qk = [&](int t, int qt, int cnt) {
        const uint64_t q = dq + (uint64_t)(qt * (kTileBytes >> 4)), kb = dk + (uint64_t)((cnt & 1) * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
          umma_f16_by(leader, tm + kColS + 128 * t, q + off, kb + off, kIdQK, kk > 0);
        }
        umma_commit_by(leader, s_full + t);
      };
      auto pv = [&](int t, int cnt, uint32_t acc) {
        const uint64_t v = dv + (uint64_t)((cnt & 1) * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_ts_by(leader, tm + kColO + 128 * t, tm + kColS + 128 * t + 8 * kk, v + (uint64_t)(kk * (2048 >> 4)), kIdPV, kk > 0 ? 1u : acc);
      };
      bool ok = true;
      int cnt = 0;  // blocks before the piece
      uint32_t pph0 = 0u, pph1 = 0u;
      for (int k = 0; ok; ++k) {
        if (!__all_sync(0xffffffffu, piece_at(k))) break;
        const int nb = uniform(pieces[k & 1].j1 - pieces[k & 1].j0), tiles = uniform(pieces[k & 1].w);
        if (lane == 0) mbar_arrive(piece_empty + (k & 1));
        if (!(ok = wait(q_ready, (uint32_t)k & 1u))) break;
        const int ahead = tiles == 2 ? 1 : 2;  // blocks whose scores are under way while one is multiplied by V
        for (int i = 0; ok && i < min(ahead, nb); ++i) {
          if (!(ok = wait2(k_ready, cnt + i))) break;
          tc_fence_after();
          qk(i, 0, cnt + i);
          if (tiles == 2) qk(1, 1, cnt + i);
          umma_commit_by(leader, k_free + ((cnt + i) & 1));
        }
        for (int i = 0; ok && i < nb; ++i) {
          if (!(ok = wait2(v_ready, cnt + i))) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t& ph = t ? pph1 : pph0;
            if (tiles == 1 && t != (i & 1)) continue;
            if (!(ok = wait(p_ready + t, ph))) break;
            ph ^= 1u;
            tc_fence_after();
            pv(t, cnt + i, i >= ahead);
            if (t == 1 || tiles == 1) umma_commit_by(leader, v_free + ((cnt + i) & 1));
            if (i + ahead >= nb) {
              umma_commit_by(leader, o_full + t);
            } else {
              if ((t == 0 || tiles == 1) && !(ok = wait2(k_ready, cnt + i + ahead))) break;
              tc_fence_after();
              qk(t, tiles == 2 ? t : 0, cnt + i + ahead);
              if (t == 1 || tiles == 1) umma_commit_by(leader, k_free + ((cnt + i + ahead) & 1));
            }
          }
        }
        cnt += nb;
      }
      umma_commit_by(leader, fin);  // arrives once every product issued has completed
      mbar_wait_bounded(fin, 0);
    }
  } else if (warp >= 8) {
    // -------------------------------------------------------------- conversion
    reg_dealloc<kRegConv>();
    const bool is_v = warp >= 12, poller = (warp & 3) == 0;
    const uint32_t gid = is_v ? 5 : 4;  // named barrier of the group
    const int tok = threadIdx.x & 127, half = tok >> 6, slot = tok & 63;
    uint64_t* ready = is_v ? v_ready : k_ready;
    uint64_t* freed = is_v ? v_free : k_free;
    uint8_t* const tile0 = smem + (is_v ? L.v : L.k);
    int cnt = 0;         // blocks so far
    int st0 = 0;         // stage and phase of the block's first page
    uint32_t sph0 = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!__all_sync(0xffffffffu, piece_at(k))) break;
      const Piece& pc = pieces[k & 1];
      const int first = pc.first, end = pc.ctx + j.N;
      const int blocks = pc.j1 - pc.j0;
      int pg = pc.p0 + 2 * pc.j0;
      const int p1 = pc.p1;
      __syncwarp();
      if (lane == 0) mbar_arrive(piece_empty + (k & 1));
      for (int i = 0; i < blocks; ++i, ++cnt, pg += 2) {
        const int cb = cnt & 1;
        const bool pair = pg + 1 < p1;  // the block has two pages
        int st1 = st0 + 1;
        uint32_t sph1 = sph0;
        if (st1 == p.nst) {
          st1 = 0;
          sph1 ^= 1u;
        }
        // one warp of the group waits for the pages and for the tile
        bool w = true;
        if (poller) {
          w = role_wait(raw_full + st0, sph0, failed);
          if (p.nst > 1 && pair) w = w && role_wait(raw_full + st1, sph1, failed);
          if (cnt >= 2) w = w && role_wait(freed + cb, (uint32_t)((cnt >> 1) - 1) & 1u, failed);
        }
        ok = !named_barrier_or(gid, 128, !w);
        if (!ok) break;
        // one stage: the second page comes into it after the first
        if (p.nst == 1 && half == 1 && pair) {
          if (!(ok = __all_sync(0xffffffffu, role_wait(raw_full, sph1, failed)))) break;
        }
        const int st = half ? st1 : st0;
        const bool use = (half == 0 || pair) && valid[st] != 0;
        if (slot == 0 && !is_v) bvalid[2 * (cnt & 3) + half] = use;
        const int pos = (pg + half) * kPage + slot;
        const bool live = use && pos >= first && pos < end;  // a token that some row may see
        const uint8_t* raw = smem + L.raw + st * stage_bytes(FMT);
        uint8_t* tile = tile0 + cb * kTileBytes;
        if (!live) {
          zero_row(tile, tok);
        } else if (FMT == 0) {
          const uint32_t meta = reinterpret_cast<const uint32_t*>(raw + 2 * kPage * kRec4)[(is_v ? kPage : 0) + slot];
          if (is_v) convert_v4(raw + kPage * kRec4 + slot * kRec4, slot, meta, tile, tok);
          else convert_k4(raw + slot * kRec4, slot, meta, tile, tok);
        } else {
          convert8(raw + (is_v ? kPage * kRec8 : 0) + slot * kRec8, slot, tile, tok);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ready + cb);
          if (half == 0 || pair) mbar_arrive(raw_empty + st);
        }
        st0 = st1;
        sph0 = sph1;
        if (pair) {
          if (++st0 == p.nst) {
            st0 = 0;
            sph0 ^= 1u;
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax and output
    reg_alloc<kRegSoftmax>();
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_base + kColS + 128 * t;
    const uint64_t all = j.N == 64 ? ~0ull : (1ull << j.N) - 1;
    uint32_t sph = 0, oph = 0;
    int cnt0 = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!__all_sync(0xffffffffu, piece_at(k))) break;
      const Piece& pc = pieces[k & 1];
      // ---- Q' rows of the tile (both groups of warps together where there is one)
      {
        const int tile = pc.w == 2 ? t : 0;
        const int nthr = pc.w == 2 ? 128 : 256, me = pc.w == 2 ? r : (int)threadIdx.x;
        const int r0 = pc.g * kGroup + tile * pc.rows0, nr = tile ? pc.rows - pc.rows0 : pc.rows0;
        // four words of 8 dims a thread in flight
        for (int e0 = me; e0 < 128 * 16; e0 += 4 * nthr) {
          uint4 in[4][2];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int e = e0 + u * nthr, row = e >> 4, w = e & 15;
            in[u][0] = in[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (row < nr) {
              const size_t src = out_row(p, pc.b, pc.h, r0 + row) * kD + 8 * w;
              if (FMT == 1 && j.q_bf16) {
                in[u][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(j.q) + src);
              } else {
                const uint4* q4 = reinterpret_cast<const uint4*>((FMT == 0 ? j.q_rot : static_cast<const float*>(j.q)) + src);
                in[u][0] = q4[0];
                in[u][1] = q4[1];
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int e = e0 + u * nthr, row = e >> 4, w = e & 15;
            const uint32_t ww[8] = {in[u][0].x, in[u][0].y, in[u][0].z, in[u][0].w, in[u][1].x, in[u][1].y, in[u][1].z, in[u][1].w};
            float y[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              const float x = FMT == 1 && j.q_bf16 ? bf16_bits_to_f32(d & 1 ? ww[d >> 1] >> 16 : ww[d >> 1] & 0xFFFFu) : __uint_as_float(ww[d]);
              y[col_of<FMT>(d)] = x * p.qmul;
            }
            *reinterpret_cast<uint4*>(smem + L.q + tile * kTileBytes + tile_offset(row, w)) =
                make_uint4(pack_f16x2_sat(y[0], y[1]), pack_f16x2_sat(y[2], y[3]), pack_f16x2_sat(y[4], y[5]), pack_f16x2_sat(y[6], y[7]));
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
      }
      // ---- this thread's row
      const int nr = pc.w == 2 && t ? pc.rows - pc.rows0 : pc.rows0;
      const int grow = pc.g * kGroup + (pc.w == 2 && t ? pc.rows0 : 0) + r;  // row of the KV head
      const bool mine = r < nr;
      const uint64_t mask = mine ? j.mask[(size_t)pc.b * j.N + grow / p.G] & all : 0ull;
      const int ctx = pc.ctx, pages0 = pc.p0 * kPage, j1 = pc.j1;
      // first position that the row sees, and whether that differs from the block range's
      const int lo = FMT == 0 ? 0 : max(0, ctx + max(1, __popcll(mask)) - j.window);
      const bool warp_rows = (r & ~31) < nr;
      float base = -INFINITY;
      uint64_t l2[2] = {0ull, 0ull};
      const int step = pc.w == 2 ? 1 : 2, jfirst = pc.j0 + (pc.w == 2 ? 0 : t);
      const int cntj = cnt0 - pc.j0;
      for (int jb = jfirst; jb < j1; jb += step) {
        ok = group_wait(s_full + t, sph, failed, (warp & 3) == 0, 2 + t, 128);
        if (!ok) break;
        sph ^= 1u;
        tc_fence_after();
        if (warp_rows) {
          const int pos0 = pages0 + 2 * kPage * jb;
          const int bi = 2 * ((cntj + jb) & 3);
          const bool pages_ok = bvalid[bi] != 0 && (bvalid[bi + 1] != 0 || pos0 + kPage >= ctx + j.N);
          // which of the block's tokens the row sees, where some may be hidden
          const bool edge = pos0 + kBlk > ctx || !pages_ok || (FMT == 1 && pos0 < ctx + j.N - j.window);
          uint64_t see[2] = {~0ull, ~0ull};
          if (edge) {
            const int cut = ctx - pos0;  // tokens from here on are drafted ones
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int cc = cut - 64 * h;
              uint64_t m = cc <= 0 ? 0ull : cc >= 64 ? ~0ull : (1ull << cc) - 1;
              if (FMT == 1) {
                const int ll = lo - pos0 - 64 * h;  // context tokens before this are outside the window
                if (ll > 0) m = ll >= 64 ? 0ull : m & ~((1ull << ll) - 1);
              }
              if (cc >= 0) m |= cc >= 64 ? 0ull : mask << cc;
              else if (cc > -64) m |= mask >> -cc;
              if (!bvalid[bi + h]) m = 0ull;
              see[h] = m;
            }
          }
          // 32 scores at a time, read once for the maximum and once for the weights
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t s[32];
          auto load = [&](int q) {
            tmem_ld32u(ts + 32 * q, s);
            tmem_wait_ld_all();
            if (edge) {
              const uint32_t m = (uint32_t)(see[q >> 1] >> (32 * (q & 1)));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((m >> i) & 1u)) s[i] = 0xFF800000u;
            }
          };
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            load(q);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u) mx[u] = fmax3(mx[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
          const bool move = top > base + 8.0f || (base == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, move)) {
            const float alpha = move ? fast_exp2(base - top) : 1.0f;
            if (move) base = top;
            l2[0] = mul_f2(l2[0], f2(alpha, alpha));
            l2[1] = mul_f2(l2[1], f2(alpha, alpha));
            if (jb > jfirst) {  // O of the first block starts anew
              const uint32_t to = tmem + lane_base + kColO + 128 * t;
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
          const float neg = base == -INFINITY ? 0.0f : -base;
          const uint64_t c2 = f2(p.c, p.c), n2 = f2(neg, neg);
          // P of 32 tokens takes 16 columns, always behind the scores still to be read
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            load(q);
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t x = fma_f2(f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, n2);
              const float e0 = fast_exp2(f2lo(x)), e1 = fast_exp2(f2hi(x));
              l2[i & 1] = add_f2(l2[i & 1], f2(e0, e1));
              pk[i] = pack16x2<true>(e0, e1);
            }
            tmem_st16u(ts + 16 * q, pk);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + t);
      }
      cnt0 += pc.j1 - pc.j0;
      if (ok && jfirst < pc.j1) {
        ok = __all_sync(0xffffffffu, role_wait(o_full + t, oph, failed));
        oph ^= 1u;
      }
      float l = (f2lo(l2[0]) + f2hi(l2[0])) + (f2lo(l2[1]) + f2hi(l2[1]));
      // ---- end of the piece: two streams over the same rows are joined, each group of warps taking half of
      // the dims. A warp that gave up takes all eight with it, so that none waits here for another.
      const bool join = pc.w == 1;
      const bool two = join && pc.j1 - pc.j0 > 1;  // the second stream had blocks
      if (join && ok) {  // base and sum for the other stream's warps, in the first columns of S (read by now)
        const float bl[4] = {base, l, 0.0f, 0.0f};
        tmem_st4(ts, bl);
        tmem_wait_st();
      }
      tc_fence_before();
      if (named_barrier_or(1, 256, !ok)) {
        ok = false;
        break;
      }
      float a0 = 1.0f, a1 = 0.0f;
      int c0 = 0, c1 = 128;
      if (join) {
        tc_fence_after();
        float other[4];
        tmem_ld4(tmem + lane_base + kColS + 128 * (1 - t), other);
        tmem_wait_ld();
        const float b0 = t == 0 ? base : other[0], b1 = t == 0 ? other[0] : base;
        const float l0 = t == 0 ? l : other[1], l1 = t == 0 ? other[1] : l;
        base = fmaxf(b0, b1);
        a0 = b0 == -INFINITY ? 0.0f : fast_exp2(b0 - base);
        a1 = b1 == -INFINITY ? 0.0f : fast_exp2(b1 - base);
        l = l0 * a0 + l1 * a1;
        if (l0 != l0 || l1 != l1) l = l0 + l1;  // NaN
        c0 = 64 * t;
        c1 = c0 + 64;
      }
      tc_fence_after();
      const bool whole = pc.whole != 0;
      const float f = whole ? (l > 0.0f || l != l ? p.vmul / l : 0.0f) : 1.0f;
      const size_t slot = (size_t)pc.slot + (join ? r : t * 128 + r);
      if (!whole && mine && (!join || t == 0)) p.ml[slot] = make_float2(base, l);
      const uint32_t to = tmem + lane_base + kColO;
      if (warp_rows) {
        // 32 rows x 32 dims at a time through 4 KB of Q' (no product reads it any more: all score products of a
        // piece are issued before the last weighted sum of either stream), so that 8 lanes write 32 dims of a row
        uint8_t* stage = smem + L.q + (pc.w == 2 ? t * kTileBytes + (warp & 3) * 4096 : warp * 4096);
        const int rbase = grow - lane;  // the warp's first row
        const int have = min(32, nr - (r & ~31));
        const int lr = lane >> 3, lc = lane & 7;
#pragma unroll 1
        for (int cc = c0; cc < c1; cc += 32) {
          uint32_t x[32];
          tmem_ld32u(to + cc + (join ? 0 : 128 * t), x);
          tmem_wait_ld_all();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(x[i]) * a0;
          if (two) {
            tmem_ld32u(to + cc + 128, x);
            tmem_wait_ld_all();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(x[i]), a1, v[i]);
          }
          if (l == 0.0f) {  // nothing seen: O holds 0, or (no product yet) anything
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 o;  // dims 4 i .. 4 i + 3 of the 32
            const int g8 = 8 * (i >> 1), d = 4 * (i & 1);
            o.x = v[g8 + col_of<FMT>(d)] * f;
            o.y = v[g8 + col_of<FMT>(d + 1)] * f;
            o.z = v[g8 + col_of<FMT>(d + 2)] * f;
            o.w = v[g8 + col_of<FMT>(d + 3)] * f;
            *reinterpret_cast<float4*>(stage + lane * 128 + 16 * (i ^ (lane & 7))) = o;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + lr;
            if (rr < have) {
              const float4 o = *reinterpret_cast<const float4*>(stage + rr * 128 + 16 * (lc ^ (rr & 7)));
              const int dim = cc + 4 * lc;
              if (!whole) {
                *reinterpret_cast<float4*>(p.acc + ((size_t)pc.slot + (join ? 0 : t * 128) + (r & ~31) + rr) * kD + dim) = o;
              } else {
                const size_t at = out_row(p, pc.b, pc.h, rbase + rr) * kD + dim;
                if (j.out_bf16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.out) + at) = make_uint2(pack16x2<false>(o.x, o.y), pack16x2<false>(o.z, o.w));
                else *reinterpret_cast<float4*>(static_cast<float*>(j.out) + at) = o;
              }
            }
          }
        }
      }
      tc_fence_before();
      if (join) named_barrier(1, 256);  // both have read both streams' O, bases and sums
      __syncwarp();
      if (lane == 0) mbar_arrive(piece_empty + (k & 1));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc_512(tmem);
  if (threadIdx.x == 0 && *failed) set_err(j.dev_err, KVQ_DEVERR_TIMEOUT);
}

// Joins the partials of the segments that several CTAs shared, in the order of the CTAs: one block per
// segment and 8 rows of it, one warp per row, four dims a lane. A first pass (a lane per partial) takes
// the bases and sums, so that the second has its factors ready and its loads are independent.
constexpr int kCombineWarps = 8;
template <int FMT>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const __grid_constant__ TreeParams p, int ctas) {
  const TreeJob& j = p.j;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x, g = seg % p.ng, h = seg / p.ng % j.Hkv, b = seg / p.ng / j.Hkv;
  const int rows = group_rows(p, g), w = g < p.ng - 1 ? 2 : p.w_last;
  const int rr = blockIdx.y * kCombineWarps + warp;
  if (rr >= rows) return;
  griddep_wait();
  griddep_launch_dependents();
  const Split sp(p, p.pre, ctas);
  const int pb = p.pre[b], nb = p.pre[b + 1] - pb;
  const long long xs = (long long)pb * sp.per_seq + (long long)h * nb * (sp.per_seq / j.Hkv) + 2LL * g * nb;
  const int ca = sp.owner(xs), cb = sp.owner(xs + (long long)(nb - 1) * w);
  if (ca == cb) return;
  const int rows0 = tile0_rows(rows, w);
  const int r = w == 2 && rr >= rows0 ? rr + 128 - rows0 : rr;
  // the segment's first block is its CTA's first one unless the block before it lies there as well
  const bool second = xs > 0 && xs - (g > 0 ? 2 : p.w_last) >= sp.X(ca);
  auto slot = [&](int c) { return (size_t)(2 * c + (c == ca && second ? 1 : 0)) * p.prow + r; };
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
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float f = __shfl_sync(0xffffffffu, f1, i);
      const float4 a = reinterpret_cast<const float4*>(p.acc + slot(c0 + i) * kD)[lane];
      o.x = fmaf(a.x, f, o.x), o.y = fmaf(a.y, f, o.y), o.z = fmaf(a.z, f, o.z), o.w = fmaf(a.w, f, o.w);
    }
  }
  const float f = l > 0.0f || l != l ? p.vmul / l : 0.0f;
  const size_t at = out_row(p, b, h, g * kGroup + rr) * kD + 4 * lane;
  if (j.out_bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.out) + at) = make_uint2(pack16x2<false>(o.x * f, o.y * f), pack16x2<false>(o.z * f, o.w * f));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(j.out) + at) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
}

std::mutex g_mu;  // guards the cache below
bool g_attr[64][2] = {{false}};

int partial_rows(int N, int Hq, int Hkv) { return N * (Hq / Hkv) <= 128 ? 128 : 256; }

template <int FMT>
cudaError_t launch_t(TreeParams& p, long long blocks_max, cudaStream_t stream) {
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (dev < 0 || dev >= 64 || !g_attr[dev][FMT]) {
      e = cudaFuncSetAttribute(tree_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) g_attr[dev][FMT] = true;
    }
  }
  const size_t fixed = Layout(FMT, p.prow / 128, 0, p.j.B).total + 1024;  // + alignment to 1024 bytes
  p.nst = std::min<int>(kMaxStages, (int)((kSmemMax - fixed) / stage_bytes(FMT)));
  if (p.nst < 1) return cudaErrorInvalidConfiguration;
  const size_t smem = fixed + (size_t)p.nst * stage_bytes(FMT);
  const int sms = device_sms();
  const int ctas = (int)std::max<long long>(1, std::min<long long>(blocks_max, std::min(sms, kMaxTreeCtas)));
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
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(p.j.B * p.j.Hkv * p.ng), (unsigned)((std::min(p.R, kGroup) + kCombineWarps - 1) / kCombineWarps), 1);
  cfg.blockDim = dim3(kCombineWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<FMT>, p, ctas);
}

}  // namespace

size_t workspace_tree_partials_bytes(int B, int N, int Hq, int Hkv) {
  return (size_t)2 * kMaxTreeCtas * partial_rows(N, Hq, Hkv) * (2 + kD) * 4 + 4 * ((size_t)B + 1);
}

cudaError_t launch_tree(const TreeJob& job, cudaStream_t stream) {
  TreeParams p{};
  p.j = job;
  float c = job.sm_scale * kLog2e * (job.fmt == 1 ? job.k_scale : 1.0f);
  p.qmul = c > 0.0f ? 1.0f : c < 0.0f ? -1.0f : 0.0f;
  p.c = c == 0.0f ? 1.0f : (c < 0.0f ? -c : c);
  p.vmul = job.fmt == 1 ? job.v_scale : 1.0f;
  p.G = job.Hq / job.Hkv;
  p.R = job.N * p.G;
  p.ng = (p.R + kGroup - 1) / kGroup;
  p.w_last = p.R - (p.ng - 1) * kGroup > 128 ? 2 : 1;
  p.prow = partial_rows(job.N, job.Hq, job.Hkv);
  p.ml = reinterpret_cast<float2*>(job.partials);
  p.acc = job.partials + (size_t)2 * 2 * kMaxTreeCtas * p.prow;
  p.pre = reinterpret_cast<int*>(p.acc + (size_t)2 * kMaxTreeCtas * p.prow * kD);
  const long long pages = job.fmt == 0 ? job.cache.max_pages_per_seq : job.ring.capacity / kPage + 1;
  const long long blocks = (pages + 1) / 2 * job.B * job.Hkv * p.ng;
  return job.fmt == 0 ? launch_t<0>(p, blocks, stream) : launch_t<1>(p, blocks, stream);
}

}  // namespace kvq
