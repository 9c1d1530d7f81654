// Causal attention over packed prompts (kvq_prompt_attn).
//
//   o_i = sum_j softmax_j(sm_scale q_i.k_j) v_j, j in [max(0, i - window + 1), i] of i's sequence.
//
// One warp per (token, query head): every lane holds four dims of q, of the running sum and of each
// key and value row; the softmax keeps a running maximum and sum in fp32.

#include <algorithm>

#include <cuda_bf16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct PromptParams {
  PromptJob j;
  float scale2;  // sm_scale * log2(e)
};

__device__ __forceinline__ void unpack4(uint2 u, bool f16, float (&x)[4]) {
  if (f16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
    x[0] = bf16_bits_to_f32(u.x & 0xFFFFu);
    x[1] = bf16_bits_to_f32(u.x >> 16);
    x[2] = bf16_bits_to_f32(u.y & 0xFFFFu);
    x[3] = bf16_bits_to_f32(u.y >> 16);
  }
}

__device__ __forceinline__ uint2 pack4(const float (&x)[4], bool f16) {
  uint2 u;
  if (f16) {
    u.x = pack_f16x2(x[0], x[1]);
    u.y = pack_f16x2(x[2], x[3]);
  } else {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(x[3]), "f"(x[2]));
  }
  return u;
}

// One row by one warp: keys first..row of the sequence that begins at token `base`.
__device__ void attend_row(const PromptParams& p, int base, int row, int hq) {
  const PromptJob& j = p.j;
  const int lane = threadIdx.x & 31;
  const int hkv = hq / (j.Hq / j.Hkv);
  auto at = [&](const void* t, long long st, long long sh, int tok, int h) {
    return reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t) + tok * st + h * sh)[lane];
  };
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  unpack4(at(j.q, j.qs_t, j.qs_h, base + row, hq), j.f16, q);
  const int first = j.window ? max(0, row - j.window + 1) : 0;
  for (int i = first; i <= row; ++i) {
    float k[4], v[4];
    unpack4(at(j.k, j.ks_t, j.ks_h, base + i, hkv), j.f16, k);
    unpack4(at(j.v, j.vs_t, j.vs_h, base + i, hkv), j.f16, v);
    float d = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
    const float z = d * p.scale2;
    const float mn = fmaxf(m, z);
    const float a = m == mn ? 1.0f : exp2f(m - mn);
    const float e = z == -INFINITY ? 0.0f : exp2f(z - mn);  // NaN stays NaN; +inf - +inf too
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = o[c] * a + e * v[c];
  }
  const float inv = 1.0f / l;
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] *= inv;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.out) + (base + row) * j.os_t + hq * j.os_h)[lane] = pack4(o, j.f16);
}

__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const PromptJob& j = p.j;
  const int hq = blockIdx.y;
  if (blockIdx.x == 0 && hq == 0)
    for (int b = threadIdx.x; b < j.B; b += blockDim.x)
      if (j.cu_seqlens[b] < 0 || j.cu_seqlens[b + 1] < j.cu_seqlens[b] || j.cu_seqlens[b + 1] > j.T) set_err(j.dev_err, KVQ_DEVERR_POS);
  for (int tok = blockIdx.x * 4 + (threadIdx.x >> 5); tok < j.T; tok += gridDim.x * 4) {
    int lo = 0, hi = j.B;  // the last b with cu_seqlens[b] <= tok
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (j.cu_seqlens[mid] <= tok) lo = mid;
      else hi = mid;
    }
    const int s = j.cu_seqlens[lo], e = j.cu_seqlens[lo + 1];
    if (s < 0 || e > j.T || tok < s || tok >= e) continue;
    attend_row(p, s, tok - s, hq);
  }
}

}  // namespace

size_t workspace_prompt_bytes(int T, int B, int Hq, int Hkv) { return 256; }

cudaError_t launch_prompt(const PromptJob& job, cudaStream_t stream) {
  PromptParams p{job, job.sm_scale * kLog2e};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min((job.T + 3) / 4, 1 << 20), (unsigned)job.Hq, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_rows_kernel, p);
}

}  // namespace kvq
