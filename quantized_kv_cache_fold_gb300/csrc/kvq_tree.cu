// Attention of a tree of drafted tokens over the int4 cache or the e4m3 ring (kvq_tree_attn_*).
//
// Row i of sequence b attends to the context (the ring: to its window's part of it) and to the
// drafted tokens of its mask. One warp per (token, query head): every lane holds four dims.

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct TreeParams {
  TreeJob j;
  float scale2;  // sm_scale * log2(e) (* k_scale)
};

__global__ void __launch_bounds__(128) tree_rows_kernel(const TreeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const TreeJob& j = p.j;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5);  // (b, i, hq)
  if (item >= j.B * j.N * j.Hq) return;
  const int hq = item % j.Hq, i = item / j.Hq % j.N, b = item / j.Hq / j.N;
  const int hkv = hq / (j.Hq / j.Hkv);
  const uint64_t all = j.N == 64 ? ~0ull : (1ull << j.N) - 1;
  const uint64_t mask = j.mask[(size_t)b * j.N + i] & all;
  const int cap = j.fmt == 0 ? j.cache.max_pages_per_seq * kPage : j.ring.capacity;
  int ctx = j.ctx[b];
  const int most = j.fmt == 0 ? cap - j.N : 1 << 30;
  if (ctx < 0 || ctx > most) {
    if (lane == 0) set_err(j.dev_err, KVQ_DEVERR_POS);
    ctx = min(max(ctx, 0), max(most, 0));
  }
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  if (j.fmt == 0) load_row4(j.q_rot, 0, (size_t)item, lane, q);
  else load_row4(j.q, j.q_bf16, (size_t)item, lane, q);
  const int first = j.fmt == 0 ? 0 : max(0, ctx + max(1, __popcll(mask)) - j.window);
  for (int pos = first; pos < ctx + j.N && pos < (j.fmt == 0 ? cap : ctx + j.N); ++pos) {
    if (pos >= ctx && !((mask >> (pos - ctx)) & 1)) continue;
    float k[4], v[4];
    if (j.fmt == 0) {
      const int page = j.cache.block_table[(size_t)b * j.cache.max_pages_per_seq + pos / kPage];
      if (page < 0 || page >= j.cache.num_pages) {
        if (lane == 0) set_err(j.dev_err, KVQ_DEVERR_PAGE);
        continue;
      }
      const int slot = pos % kPage;
      const uint8_t* blk = j.cache.pages + ((size_t)page * j.Hkv + hkv) * KVQ_INT4_BLOCK_BYTES;
      const uint32_t* meta = reinterpret_cast<const uint32_t*>(blk + 2 * kPage * kRec4);
      const uint32_t kb = *reinterpret_cast<const uint16_t*>(blk + slot * kRec4 + 16 * ((lane >> 3) ^ k_chunk_swz(slot)) + ((2 * lane) & 15));
      const uint32_t vb = *reinterpret_cast<const uint16_t*>(blk + kPage * kRec4 + slot * kRec4 + 16 * ((lane >> 3) ^ ((slot >> 1) & 3)) + ((2 * lane) & 15));
      const uint32_t km = meta[slot], vm = meta[kPage + slot];
      const float ks = __half2float(__ushort_as_half((unsigned short)km)), ko = __half2float(__ushort_as_half((unsigned short)(km >> 16)));
      const float vs = __half2float(__ushort_as_half((unsigned short)vm)), vo = __half2float(__ushort_as_half((unsigned short)(vm >> 16)));
      const int eb[4] = {1, 4, 11, 8}, sb[4] = {15, 14, 7, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        k[c] = fmaf((float)((kb >> (4 * c)) & 15), ks, ko);
        const int e = (vb >> eb[c]) & 7;
        v[c] = fmaf((float)((vb >> sb[c]) & 1 ? 7 - e : 8 + e), vs, vo);
      }
    } else {
      const int slot = pos % cap;
      const uint8_t* blk = j.ring.data + (((size_t)b * j.Hkv + hkv) * (cap / kPage) + slot / kPage) * (2 * kPage * kRec8);
      const uint32_t kb = *reinterpret_cast<const uint32_t*>(blk + fp8_lane_offset(slot, lane));
      const uint32_t vb = *reinterpret_cast<const uint32_t*>(blk + kPage * kRec8 + fp8_lane_offset(slot, lane));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t k2 = e4m3x2_to_f16x2(kb >> (16 * c)), v2 = e4m3x2_to_f16x2(vb >> (16 * c));
        const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&k2)), vf = __half22float2(*reinterpret_cast<const __half2*>(&v2));
        k[2 * c] = kf.x, k[2 * c + 1] = kf.y;
        v[2 * c] = vf.x * j.v_scale, v[2 * c + 1] = vf.y * j.v_scale;
      }
    }
    float d = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
    const float z = d * p.scale2;
    const float mn = fmaxf(m, z);
    const float a = m == mn ? 1.0f : exp2f(m - mn);
    const float e = z == -INFINITY ? 0.0f : exp2f(z - mn);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = o[c] * a + e * v[c];
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;  // a row that attends to nothing: 0
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] *= inv;
  if (j.out_bf16) {
    uint2 u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(o[1]), "f"(o[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(o[3]), "f"(o[2]));
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.out) + (size_t)item * kD)[lane] = u;
  } else {
    reinterpret_cast<float4*>(static_cast<float*>(j.out) + (size_t)item * kD)[lane] = make_float4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace

size_t workspace_tree_partials_bytes(int B, int N, int Hq, int Hkv) { return 256; }

cudaError_t launch_tree(const TreeJob& job, cudaStream_t stream) {
  TreeParams p{job, job.sm_scale * kLog2e * (job.fmt == 1 ? job.k_scale : 1.0f)};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(((long long)job.B * job.N * job.Hq + 3) / 4), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_rows_kernel, p);
}

}  // namespace kvq
