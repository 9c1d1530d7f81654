// Device pieces shared by the attention kernels with one query row per tensor-memory lane (the prompt's
// and the tree's): wide tensor-memory accesses, tensor-map copies, 16-bit packing, and the softmax
// step of a 128 x 128 block of scores.
#pragma once

#include <cuda.h>

#include "kvq_device.cuh"

namespace kvq {

// 16 consecutive 32-bit columns of this thread's lane, raw words (valid after tmem_wait_ld).
__device__ __forceinline__ void tmem_ld16u(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's lane, raw words (valid after tmem_wait_ld).
__device__ __forceinline__ void tmem_ld32u(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// The base of a row's weights follows the largest score, in powers of two: it moves when a score passes it by more than
// kBaseLag. Weights of fp16 are 2^(score - base + kWeightRaise), so the largest lies between 2^7 and 2^15 and the type's
// smallest step 2^-24 is 2^-31 of it or less: with no raise, weights below 2^-25 of the largest were lost (65,000 keys 17
// to 20 nats under one whose value is 0: the output off by 4 to 90%). The factor is the sums' as well, so it cancels.
constexpr float kBaseLag = 8.0f, kWeightRaise = 7.0f;

// Keeps values loaded by tmem_ld*u from being used before the wait after the loads.
__device__ __forceinline__ void tmem_wait_ld_all() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Box of a 3-D tensor map at (x, y, z) into shared memory, completion counted on `bar`.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Asynchronous store of a box from shared memory (written, fenced for the async proxy and synchronised before), as a
// group of its own; the groups of a thread are waited for by the thread itself.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\tcp.async.bulk.commit_group;" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
               : "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }  // sources free
__device__ __forceinline__ void tma_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }       // written

// Instruction descriptor of tcgen05.mma.kind::f16 with bf16 or f16 operands, M = 128, N columns.
__host__ __device__ constexpr uint32_t umma_idesc_16(bool f16, int n, bool b_mn) {
  return umma_idesc_f16(n, false, b_mn) | (f16 ? 0u : (1u << 7) | (1u << 10));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  uint32_t d;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The issuing warp of the products stays converged and one elected lane issues: descriptors and addresses are
// then warp-uniform values, which the instruction takes from uniform registers. (A branch on one lane
// instead costs moves to uniform registers for each product: 82 cycles to issue one that runs for 64.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void umma_f16_by(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts_by(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_commit_by(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// An arrival that orders nothing but what has completed already (the default one waits for the thread's
// outstanding global stores).
__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Bounded wait for a phase; notes a wait that gave up in *failed. (mbar_wait_bounded's suspend hint matters:
// a tight loop of plain try_waits in its place takes the 32,768-token prompt from 4.11 to 4.72 ms and the
// tree over 64 x 16,384 tokens from 355 to 370 us.)
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
  if (mbar_wait_bounded(bar, parity)) return true;
  *failed = 1;
  return false;
}

// role_wait by a group of `nthreads` threads (whole warps): the warp with `poller` set watches the mbarrier, the
// others rest in named barrier `id`, which takes no issue slots. The same answer for the whole group.
__device__ __forceinline__ bool group_wait(uint64_t* bar, uint32_t parity, volatile int* failed, bool poller, uint32_t id,
                                           uint32_t nthreads) {
  bool ok = true;
  if (poller) ok = role_wait(bar, parity, failed);
  return !named_barrier_or(id, nthreads, !ok);
}

}  // namespace kvq
