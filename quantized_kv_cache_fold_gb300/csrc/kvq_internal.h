// Internal launch interface between the C-ABI layer (kvq_api.cpp) and the kernel
// translation units. Host-side only; all arguments have been validated by the caller.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "kvq.h"

namespace kvq {

constexpr int kMaxCtas = 1024;       // cap on attention CTAs (sizes the partial-result workspace)
constexpr int kMaxRows = 48;         // S * (num_q_heads / num_kv_heads) rows per KV head and sequence
constexpr int kPartialStride = 130;  // floats per partial row: m, l, acc[128]

// Job description for the prologue/quantise kernel.
struct PrepJobs {
  // int4 append (keys rotated, values raw)
  kvq_int4_cache cache;
  const float* Mk;
  const void* k;
  const void* v;
  int kv_bf16;
  int T;                   // tokens to append (each has num_kv_heads heads)
  const int32_t* seq_ids;  // explicit mode (or null)
  const int32_t* positions;
  const int32_t* ctx_len;  // derived mode: seq = t / S, pos = ctx_len[seq] + t % S
  int S;
  // query prologue
  const float* Mq;
  const void* q;
  int q_bf16;
  int nq_rows;
  float* q_rot;      // workspace destination [nq_rows][128]
  float* q_rot_out;  // optional copy
  float eps;
  int32_t* dev_err;
  // 0: the matrix prologue (Mk, Mq are 128x128 matrices); 1: the FWHT prologue (Mk, Mq are the
  // 128 multipliers w_k = s, w_q = fp32(s g_q g_k) of kvq_fold_qk_fwht)
  int fwht;
};

cudaError_t launch_prep(const PrepJobs& jobs, cudaStream_t stream);

struct Fp8AppendJob {
  kvq_fp8_ring ring;
  const void* k;
  const void* v;
  int bf16;
  int T;
  const int32_t* seq_ids;  // explicit mode (or null)
  const int32_t* positions;
  const int32_t* pos0;     // derived mode: seq = t / S, pos = pos0[seq] + t % S
  int S;
  float k_scale, v_scale;
  int32_t* dev_err;
};

cudaError_t launch_fp8_append(const Fp8AppendJob& job, cudaStream_t stream);

// Attention over either cache format.
struct AttnJob {
  int fmt;  // 0 = int4 paged, 1 = fp8 ring
  kvq_int4_cache cache;
  kvq_fp8_ring ring;
  int window;
  float k_scale, v_scale;
  int B, S, Hq, Hkv;
  const int32_t* ctx;  // int4: ctx_len[b]; fp8: pos0[b]
  const float* q_rot;  // int4: rotated queries [B][S][Hq][128] fp32 (workspace)
  const void* q;       // fp8: queries as given
  int q_bf16;
  const void* k_new;   // fp8 cluster path: rows appended inside the attention kernel (null: none)
  const void* v_new;
  float sm_scale;
  float* out;
  // A tree of S drafted tokens in place of a verify block (null: none); int4, and rings on the cluster path.
  const uint64_t* tree_mask;
  int out_bf16;               // with tree_mask: out holds bf16
  float* partials;  // workspace
  int32_t* dev_err;
};

cudaError_t launch_attention(const AttnJob& job, cudaStream_t stream);

// FP8 window attention with one thread-block cluster per (sequence, KV head), appending
// job.k_new / job.v_new itself. swa_cluster_path() says whether a ring of this capacity, with
// this batch and these head counts, takes it; larger rings go through launch_attention (fmt 1)
// after a separate append.
bool swa_cluster_path(int capacity, int B, int S, int Hq, int Hkv);
// The chosen shape: CTAs per pair (0: split-K path), streams per CTA, stages, units per stream.
void swa_plan_shape(int capacity, int B, int S, int Hq, int Hkv, int out[4]);
cudaError_t launch_swa_cluster(const AttnJob& job, cudaStream_t stream);

// Workspace layout shared by the API and the launchers.
// Host-side argument checks of kvq_decode_attn_int4 other than the workspace (status as that
// call returns it); shared with the allocation-free entry point.
kvq_status check_decode_int4_args(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                                  kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len,
                                  const void* k_new, const void* v_new, float sm_scale, float eps, const float* out,
                                  const float* q_rot_out, const int32_t* dev_err);

// Limit of the split-K attention kernel's stage waits for later launches (kvq_set_stage_wait_limit_ns).
void set_stage_wait_limit_ns(unsigned long long ns);

// SMs of the current device (cached).
int device_sms();

// ---- prompt attention (kvq_prompt.cu)
struct PromptJob {
  const void *q, *k, *v;
  void* out;
  int f16;  // 1: fp16, 0: bf16
  int T, B, Hq, Hkv;
  long long qs_t, qs_h, ks_t, ks_h, vs_t, vs_h, os_t, os_h;  // elements
  const int32_t* cu_seqlens;
  int window;  // 0: none
  float sm_scale;
  int32_t* dev_err;
};
cudaError_t launch_prompt(const PromptJob& job, cudaStream_t stream);

// ---- tree attention (kvq_tree.cu)
struct TreeJob {
  int fmt;  // 0 = int4 paged, 1 = fp8 ring
  kvq_int4_cache cache;
  kvq_fp8_ring ring;
  int window;
  float k_scale, v_scale;
  int B, N, Hq, Hkv;
  const int32_t* ctx;
  const uint64_t* mask;
  const float* q_rot;  // int4: rotated queries (workspace)
  const void* q;       // fp8: queries as given
  int q_bf16;
  float sm_scale;
  void* out;
  int out_bf16;
  float* partials;  // workspace
  int32_t* dev_err;
};
// Trees of up to this many rows per KV head (drafted tokens x query heads per KV head) over the int4 cache take the
// verify block's kernels (launch_attention) with the mask in place of the diagonal: those multiply the codes as they are
// and scale the scores, so few rows cost little, where launch_tree first makes fp16 tiles of every token. 64 sequences of
// 16,384 tokens, 4 KV heads, verify kernels / launch_tree: 106 / 259 us with 5 rows, 164 / 262 with 15, 195 / 263 with
// 20, 258 / 284 with 45; 8 of 8,192: 21 / 35, 32 / 37, 29 / 37, 40 / 42; one of 4,096: 21-25 / 22-24 throughout; one of
// 65,536: 24 / 42, 30 / 44, 30 / 46, 37 / 44. The same with 1 and 8 KV heads (5, 15, 25, 40, 45 rows): 64 sequences (16,384;
// 8,192) 38-82 / 81-92 and 112-291 / 267-309, 8 of 8,192 17-25 / 28-34 and 26-55 / 51-61; only one of 65,536 with one KV
// head is slower from 15 rows on, 40-45 / 39-41.
constexpr int kTreeFewRows = kMaxRows;
// Over a ring, trees of up to 8 drafted tokens and 16 rows, or 24 rows while there are fewer (sequence, KV head) pairs
// than SMs, take the verify block's cluster kernel where the ring is small enough for it (swa_cluster_path): one launch
// with the append in it. Rings of 576 slots (window 513), 4 KV heads, cluster kernel / launch_tree: one sequence 6.4 /
// 18.1 us with 5 rows, 9.0 / 18.6 with 10, 13.9 / 19.0 with 20; 8 sequences 6.5 / 22.9, 9.5 / 23.2, 14.3 / 24.5; 64
// sequences 13.5 / 22.4, 20.1 / 22.4, but 30.9 / 23.2 with 20; 256 sequences 37 / 71, 51 / 72, 70 / 74. Without new rows, 1
// and 8 KV heads, 5 to 15 rows: 5-8 / 17-18 and 5-8 / 20-21 (one sequence), 6-15 / 27-28 and 23-27 / 37-38 (64), 12-17 / 22-24
// and 65-91 / 138-140 (256).
constexpr int kTreeRingRows = 16, kTreeRingRowsFewPairs = 24, kTreeRingTokens = 8;
size_t workspace_tree_partials_bytes(int B);
cudaError_t launch_tree(const TreeJob& job, cudaStream_t stream);

// ---- page pool, page copies and commits (kvq_pages.cu)
struct PoolJob {
  int32_t* page_refs;
  int num_pages;
  int32_t* block_table;
  int num_seqs, max_pages_per_seq;
  int n;
  const int32_t *a, *b, *c;  // alloc, free: ids, old and new lengths; fork: parents, children, lengths
  int32_t *copy_src, *copy_dst, *n_moves;
  int32_t* dev_err;
};
cudaError_t launch_pages_alloc(const PoolJob& job, cudaStream_t stream);
cudaError_t launch_pages_fork(const PoolJob& job, cudaStream_t stream);
cudaError_t launch_pages_free(const PoolJob& job, cudaStream_t stream);
cudaError_t launch_pages_compact(const PoolJob& job, cudaStream_t stream);

// The caches or rings of one call over several layers (a kernel parameter). Rings: max_pages is the
// number of 64-slot blocks.
struct CacheSet {
  uint8_t* pages[KVQ_MAX_CACHES];
  const int32_t* table[KVQ_MAX_CACHES];
  int32_t num_pages[KVQ_MAX_CACHES], num_seqs[KVQ_MAX_CACHES], max_pages[KVQ_MAX_CACHES];
  int32_t count, heads;
};
cudaError_t launch_pages_copy(const CacheSet& cs, int n, const int32_t* src, const int32_t* dst, const int32_t* count,
                              int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_tree_commit(int fmt, const CacheSet& cs, int B, int N, const int32_t* ctx_len, const int32_t* path,
                               const int32_t* n_accept, int32_t* ctx_out, int32_t* dev_err, cudaStream_t stream);

// Argument checks shared by the C-ABI translation units.
kvq_status check_int4_cache(const kvq_int4_cache* c);
kvq_status check_ring(const kvq_fp8_ring* r);

size_t workspace_qrot_bytes(int B, int S, int Hq);
size_t workspace_partials_bytes(int B, int S, int Hq, int Hkv);

}  // namespace kvq
