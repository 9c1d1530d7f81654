// C-ABI entry points around decoding: a prompt's attention, the attention of a tree of drafted
// tokens, the commit of its accepted branch, and the page pool. Host-side argument checks and
// dispatch only; see include/kvq.h for the contract of each call.

#include <cmath>
#include <cstdint>

#include "kvq.h"
#include "kvq_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

kvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool prompt_sizes_ok(int T, int B, int Hq, int Hkv) {
  return T >= 0 && B >= 1 && B <= KVQ_MAX_SEQS && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 &&
         (long long)T * Hq <= (1LL << 30);
}

bool tree_sizes_ok(int B, int N, int Hq, int Hkv) {
  return B >= 1 && B <= KVQ_MAX_SEQS && N >= 1 && N <= KVQ_MAX_TREE && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 &&
         Hq / Hkv <= 64 && (long long)B * N * Hq <= (1LL << 30);
}

// The checks that the int4 and ring forms of the tree's attention share.
kvq_status check_tree(int B, int N, int Hq, int Hkv, int num_seqs, kvq_dtype dtype, const void* q, const int32_t* ctx,
                      const uint64_t* mask, const void* k_new, const void* v_new, float sm_scale, const void* out,
                      kvq_dtype out_dtype, const void* workspace, size_t workspace_bytes, const int32_t* dev_err) {
  if (N < 1 || N > KVQ_MAX_TREE || Hq < 1 || Hq % Hkv || Hq / Hkv > 64) return KVQ_ERR_UNSUPPORTED;
  if (B < 1 || B > KVQ_MAX_SEQS || B > num_seqs || !tree_sizes_ok(B, N, Hq, Hkv)) return KVQ_ERR_INVALID_ARG;
  if (dtype != KVQ_F32 && dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
  if (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
  if (!q || !ctx || !mask || !out || !workspace || !dev_err) return KVQ_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return KVQ_ERR_INVALID_ARG;
  if (k_new && (!aligned(k_new, 16) || !aligned(v_new, 16))) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(mask, 8)) return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kvq_tree_workspace_bytes(B, N, Hq, Hkv)) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

kvq_status tree_int4_impl(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                          kvq_dtype dtype, int B, int N, int num_q_heads, const int32_t* ctx_len,
                          const uint64_t* tree_mask, const void* k_new, const void* v_new, float sm_scale, float eps,
                          void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                          kvq_stream_t stream, int fwht) {
  kvq_status st = kvq::check_int4_cache(cache);
  if (st != KVQ_OK) return st;
  st = check_tree(B, N, num_q_heads, cache->num_kv_heads, cache->num_seqs, dtype, q, ctx_len, tree_mask, k_new, v_new,
                  sm_scale, out, out_dtype, workspace, workspace_bytes, dev_err);
  if (st != KVQ_OK) return st;
  if ((long long)B * (cache->max_pages_per_seq + 2) > (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  if (!Mq || !aligned(Mq, 16) || (k_new && (!Mk || !aligned(Mk, 16)))) return KVQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || std::isinf(eps)) return KVQ_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  kvq::PrepJobs j{};
  j.cache = *cache;
  j.fwht = fwht;
  j.Mk = Mk;
  j.k = k_new;
  j.v = v_new;
  j.kv_bf16 = dtype == KVQ_BF16;
  j.T = k_new ? B * N : 0;
  j.ctx_len = ctx_len;
  j.S = N;
  j.Mq = Mq;
  j.q = q;
  j.q_bf16 = dtype == KVQ_BF16;
  j.nq_rows = B * N * num_q_heads;
  j.q_rot = reinterpret_cast<float*>(ws);
  j.eps = eps;
  j.dev_err = dev_err;
  if (kvq::launch_prep(j, (cudaStream_t)stream) != cudaSuccess) return KVQ_ERR_CUDA;
  if (N * (num_q_heads / cache->num_kv_heads) <= kvq::kTreeFewRows) {
    kvq::AttnJob a{};
    a.fmt = 0;
    a.cache = *cache;
    a.B = B;
    a.S = N;
    a.Hq = num_q_heads;
    a.Hkv = cache->num_kv_heads;
    a.ctx = ctx_len;
    a.q_rot = j.q_rot;
    a.sm_scale = sm_scale;
    a.out = static_cast<float*>(out);
    a.tree_mask = tree_mask;
    a.out_bf16 = out_dtype == KVQ_BF16;
    a.partials = reinterpret_cast<float*>(ws + kvq::workspace_qrot_bytes(B, N, num_q_heads));
    a.dev_err = dev_err;
    return from_cuda(kvq::launch_attention(a, (cudaStream_t)stream));
  }
  kvq::TreeJob t{};
  t.fmt = 0;
  t.cache = *cache;
  t.B = B;
  t.N = N;
  t.Hq = num_q_heads;
  t.Hkv = cache->num_kv_heads;
  t.ctx = ctx_len;
  t.mask = tree_mask;
  t.q_rot = j.q_rot;
  t.sm_scale = sm_scale;
  t.out = out;
  t.out_bf16 = out_dtype == KVQ_BF16;
  t.partials = reinterpret_cast<float*>(ws + kvq::workspace_qrot_bytes(B, N, num_q_heads));
  t.dev_err = dev_err;
  return from_cuda(kvq::launch_tree(t, (cudaStream_t)stream));
}

kvq_status check_commit(int num_caches, int B, int N, const int32_t* ctx, const int32_t* path, const int32_t* n_accept,
                        const int32_t* ctx_out, const int32_t* dev_err) {
  if (num_caches < 1 || B < 1 || B > KVQ_MAX_SEQS) return KVQ_ERR_INVALID_ARG;
  if (num_caches > KVQ_MAX_CACHES || N < 1 || N > KVQ_MAX_TREE) return KVQ_ERR_UNSUPPORTED;
  if (!ctx || !path || !n_accept || !dev_err) return KVQ_ERR_INVALID_ARG;
  // ctx_out is written by some blocks while others still read the lists
  const size_t n = 4 * (size_t)B;
  if (ctx_out && (overlap(ctx, n, ctx_out, n) || overlap(n_accept, n, ctx_out, n) || overlap(path, n * N, ctx_out, n)))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

// Whether two layers of a call are the same memory (a commit would move its records twice at once).
bool repeated(const kvq::CacheSet& cs) {
  for (int i = 1; i < cs.count; ++i)
    for (int k = 0; k < i; ++k)
      if (cs.pages[i] == cs.pages[k]) return true;
  return false;
}

// The caches of one call, checked; all of one number of KV heads.
kvq_status cache_set(const kvq_int4_cache* caches, int num_caches, kvq::CacheSet& cs) {
  if (!caches || num_caches < 1) return KVQ_ERR_INVALID_ARG;
  if (num_caches > KVQ_MAX_CACHES) return KVQ_ERR_UNSUPPORTED;
  cs.count = num_caches;
  cs.heads = caches[0].num_kv_heads;
  for (int i = 0; i < num_caches; ++i) {
    const kvq_status st = kvq::check_int4_cache(caches + i);
    if (st != KVQ_OK) return st;
    if (caches[i].num_kv_heads != cs.heads) return KVQ_ERR_INVALID_ARG;
    cs.pages[i] = caches[i].pages;
    cs.table[i] = caches[i].block_table;
    cs.num_pages[i] = caches[i].num_pages;
    cs.num_seqs[i] = caches[i].num_seqs;
    cs.max_pages[i] = caches[i].max_pages_per_seq;
  }
  return KVQ_OK;
}

kvq_status check_pool(const int32_t* refs, int num_pages, const int32_t* table, int num_seqs, int max_pages,
                      const int32_t* dev_err) {
  if (!refs || !table || !dev_err || num_pages < 1 || num_seqs < 1 || max_pages < 1) return KVQ_ERR_INVALID_ARG;
  if (max_pages > (1 << 24) || (long long)num_seqs * max_pages > (1LL << 30)) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

// alloc, fork and free: n requests of three lists each.
kvq_status pool_call(cudaError_t (*launch)(const kvq::PoolJob&, cudaStream_t), int32_t* refs, int num_pages,
                     int32_t* table, int num_seqs, int max_pages, int n, const int32_t* a, const int32_t* b,
                     const int32_t* c, int32_t* src, int32_t* dst, int32_t* dev_err, kvq_stream_t stream) {
  const kvq_status st = check_pool(refs, num_pages, table, num_seqs, max_pages, dev_err);
  if (st != KVQ_OK) return st;
  if (n < 0 || n > KVQ_MAX_SEQS) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!a || !b || !c) return KVQ_ERR_INVALID_ARG;
  if (src) {  // fork's lists are written while others still read theirs
    const size_t bytes = 4 * (size_t)n;
    if (overlap(src, bytes, dst, bytes)) return KVQ_ERR_INVALID_ARG;
    for (const int32_t* in : {a, b, c})
      if (overlap(src, bytes, in, bytes) || overlap(dst, bytes, in, bytes)) return KVQ_ERR_INVALID_ARG;
  }
  kvq::PoolJob j{refs, num_pages, table, num_seqs, max_pages, n, a, b, c, src, dst, nullptr, dev_err};
  return from_cuda(launch(j, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

size_t kvq_prompt_workspace_bytes(int T, int B, int num_q_heads, int num_kv_heads) {
  if (!prompt_sizes_ok(T, B, num_q_heads, num_kv_heads)) return 0;
  return 256;  // the kernel keeps everything on chip: the size of a valid call's workspace, nothing more
}

kvq_status kvq_prompt_attn(const void* q, const void* k, const void* v, kvq_dtype dtype, int T, int B,
                           int num_q_heads, int num_kv_heads, const int64_t* strides, const int32_t* cu_seqlens,
                           int window, float sm_scale, void* out, void* workspace, size_t workspace_bytes,
                           int32_t* dev_err, kvq_stream_t stream) {
  if (dtype == KVQ_F32) return KVQ_ERR_UNSUPPORTED;
  if (dtype != KVQ_BF16 && dtype != KVQ_F16) return KVQ_ERR_INVALID_ARG;
  if (!prompt_sizes_ok(T, B, num_q_heads, num_kv_heads)) return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.0f)) return KVQ_ERR_INVALID_ARG;
  if (T == 0) return KVQ_OK;
  if (!q || !k || !v || !cu_seqlens || !out || !workspace || !dev_err) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kvq_prompt_workspace_bytes(T, B, num_q_heads, num_kv_heads)) return KVQ_ERR_INVALID_ARG;
  const long long D = KVQ_HEAD_DIM;
  long long st[8] = {D * num_q_heads, D, D * num_kv_heads, D, D * num_kv_heads, D, D * num_q_heads, D};
  if (strides)
    for (int i = 0; i < 8; ++i) {
      if (strides[i] < 8 || strides[i] % 8 || strides[i] > (1LL << 36)) return KVQ_ERR_INVALID_ARG;
      st[i] = strides[i];
    }
  // bytes from the first to behind the last element of each tensor; the output is apart from the others
  const int heads[4] = {num_q_heads, num_kv_heads, num_kv_heads, num_q_heads};
  const void* base[4] = {q, k, v, out};
  size_t span[4];
  for (int i = 0; i < 4; ++i) span[i] = 2 * (size_t)((T - 1) * st[2 * i] + (heads[i] - 1) * st[2 * i + 1] + D);
  // (out may be interleaved with its own rows only: an out that shares a buffer with q, k or v is refused)
  for (int i = 0; i < 3; ++i)
    if (overlap(base[i], span[i], out, span[3])) return KVQ_ERR_INVALID_ARG;
  // rows of the output do not overlap one another
  if (!(st[6] >= (num_q_heads - 1) * st[7] + D && (num_q_heads == 1 || st[7] >= D)) &&
      !(st[7] >= (T - 1) * st[6] + D && (T == 1 || st[6] >= D)))
    return KVQ_ERR_INVALID_ARG;
  kvq::PromptJob j{};
  j.q = q;
  j.k = k;
  j.v = v;
  j.out = out;
  j.f16 = dtype == KVQ_F16;
  j.T = T;
  j.B = B;
  j.Hq = num_q_heads;
  j.Hkv = num_kv_heads;
  j.qs_t = st[0], j.qs_h = st[1], j.ks_t = st[2], j.ks_h = st[3];
  j.vs_t = st[4], j.vs_h = st[5], j.os_t = st[6], j.os_h = st[7];
  j.cu_seqlens = cu_seqlens;
  j.window = window > 0 ? window : 0;
  j.sm_scale = sm_scale;
  j.dev_err = dev_err;
  return from_cuda(kvq::launch_prompt(j, (cudaStream_t)stream));
}

size_t kvq_tree_workspace_bytes(int B, int N, int num_q_heads, int num_kv_heads) {
  if (!tree_sizes_ok(B, N, num_q_heads, num_kv_heads)) return 0;
  const bool few = N * (num_q_heads / num_kv_heads) <= kvq::kTreeFewRows;
  return kvq::workspace_qrot_bytes(B, N, num_q_heads) +
         std::max(kvq::workspace_tree_partials_bytes(B),
                  few ? kvq::workspace_partials_bytes(B, N, num_q_heads, num_kv_heads) : (size_t)0);
}

kvq_status kvq_tree_attn_int4(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                              kvq_dtype dtype, int B, int N, int num_q_heads, const int32_t* ctx_len,
                              const uint64_t* tree_mask, const void* k_new, const void* v_new, float sm_scale,
                              float eps, void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                              int32_t* dev_err, kvq_stream_t stream) {
  return tree_int4_impl(cache, Mq, Mk, q, dtype, B, N, num_q_heads, ctx_len, tree_mask, k_new, v_new, sm_scale, eps,
                        out, out_dtype, workspace, workspace_bytes, dev_err, stream, 0);
}

kvq_status kvq_tree_attn_int4_fwht(const kvq_int4_cache* cache, const float* wq, const float* wk, const void* q,
                                   kvq_dtype dtype, int B, int N, int num_q_heads, const int32_t* ctx_len,
                                   const uint64_t* tree_mask, const void* k_new, const void* v_new, float sm_scale,
                                   float eps, void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_err, kvq_stream_t stream) {
  return tree_int4_impl(cache, wq, wk, q, dtype, B, N, num_q_heads, ctx_len, tree_mask, k_new, v_new, sm_scale, eps,
                        out, out_dtype, workspace, workspace_bytes, dev_err, stream, 1);
}

kvq_status kvq_tree_attn_fp8_swa(const kvq_fp8_ring* ring, const void* q, kvq_dtype dtype, int B, int N,
                                 int num_q_heads, const int32_t* pos0, const uint64_t* tree_mask, int window,
                                 const void* k_new, const void* v_new, float k_scale, float v_scale, float sm_scale,
                                 void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                 int32_t* dev_err, kvq_stream_t stream) {
  kvq_status st = kvq::check_ring(ring);
  if (st != KVQ_OK) return st;
  st = check_tree(B, N, num_q_heads, ring->num_kv_heads, ring->num_seqs, dtype, q, pos0, tree_mask, k_new, v_new,
                  sm_scale, out, out_dtype, workspace, workspace_bytes, dev_err);
  if (st != KVQ_OK) return st;
  if (window < N || (long long)window + N - 1 > ring->capacity) return KVQ_ERR_INVALID_ARG;
  if (!(k_scale > 0.0f) || !(v_scale > 0.0f) || std::isinf(k_scale) || std::isinf(v_scale)) return KVQ_ERR_INVALID_ARG;
  // Rows of the output are written while other rows of q (and of k_new, v_new) are still read. A row's own query is
  // read before, so the output may take q's place exactly.
  const size_t rows = (size_t)B * N * KVQ_HEAD_DIM, in = dtype == KVQ_BF16 ? 2 : 4, res = out_dtype == KVQ_BF16 ? 2 : 4;
  if (overlap(q, rows * num_q_heads * in, out, rows * num_q_heads * res) && !(q == out && in == res)) return KVQ_ERR_INVALID_ARG;
  for (const void* x : {k_new, v_new})
    if (x && overlap(x, rows * ring->num_kv_heads * in, out, rows * num_q_heads * res)) return KVQ_ERR_INVALID_ARG;
  const bool few_pairs = (long long)B * ring->num_kv_heads < kvq::device_sms();
  if (N <= kvq::kTreeRingTokens &&
      N * (num_q_heads / ring->num_kv_heads) <= (few_pairs ? kvq::kTreeRingRowsFewPairs : kvq::kTreeRingRows) &&
      kvq::swa_cluster_path(ring->capacity, B, N, num_q_heads, ring->num_kv_heads)) {
    kvq::AttnJob a{};
    a.fmt = 1;
    a.ring = *ring;
    a.window = window;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.B = B;
    a.S = N;
    a.Hq = num_q_heads;
    a.Hkv = ring->num_kv_heads;
    a.ctx = pos0;
    a.q = q;
    a.q_bf16 = dtype == KVQ_BF16;
    a.k_new = k_new;
    a.v_new = v_new;
    a.sm_scale = sm_scale;
    a.out = static_cast<float*>(out);
    a.tree_mask = tree_mask;
    a.out_bf16 = out_dtype == KVQ_BF16;
    a.dev_err = dev_err;
    return from_cuda(kvq::launch_swa_cluster(a, (cudaStream_t)stream));
  }
  if (k_new) {
    kvq::Fp8AppendJob j{};
    j.ring = *ring;
    j.k = k_new;
    j.v = v_new;
    j.bf16 = dtype == KVQ_BF16;
    j.T = B * N;
    j.pos0 = pos0;
    j.S = N;
    j.k_scale = k_scale;
    j.v_scale = v_scale;
    j.dev_err = dev_err;
    if (kvq::launch_fp8_append(j, (cudaStream_t)stream) != cudaSuccess) return KVQ_ERR_CUDA;
  }
  kvq::TreeJob t{};
  t.fmt = 1;
  t.ring = *ring;
  t.window = window;
  t.k_scale = k_scale;
  t.v_scale = v_scale;
  t.B = B;
  t.N = N;
  t.Hq = num_q_heads;
  t.Hkv = ring->num_kv_heads;
  t.ctx = pos0;
  t.mask = tree_mask;
  t.q = q;
  t.q_bf16 = dtype == KVQ_BF16;
  t.sm_scale = sm_scale;
  t.out = out;
  t.out_bf16 = out_dtype == KVQ_BF16;
  t.partials =
      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kvq::workspace_qrot_bytes(B, N, num_q_heads));
  t.dev_err = dev_err;
  return from_cuda(kvq::launch_tree(t, (cudaStream_t)stream));
}

kvq_status kvq_tree_commit_int4(const kvq_int4_cache* caches, int num_caches, int B, int N, const int32_t* ctx_len,
                                const int32_t* path, const int32_t* n_accept, int32_t* ctx_out, int32_t* dev_err,
                                kvq_stream_t stream) {
  kvq_status st = check_commit(num_caches, B, N, ctx_len, path, n_accept, ctx_out, dev_err);
  if (st != KVQ_OK) return st;
  kvq::CacheSet cs{};
  st = cache_set(caches, num_caches, cs);
  if (st != KVQ_OK) return st;
  for (int i = 0; i < num_caches; ++i)
    if (B > caches[i].num_seqs) return KVQ_ERR_INVALID_ARG;
  if (repeated(cs)) return KVQ_ERR_INVALID_ARG;
  return from_cuda(
      kvq::launch_tree_commit(0, cs, B, N, ctx_len, path, n_accept, ctx_out, dev_err, (cudaStream_t)stream));
}

kvq_status kvq_tree_commit_fp8(const kvq_fp8_ring* rings, int num_caches, int B, int N, const int32_t* pos0,
                               const int32_t* path, const int32_t* n_accept, int32_t* ctx_out, int32_t* dev_err,
                               kvq_stream_t stream) {
  const kvq_status st = check_commit(num_caches, B, N, pos0, path, n_accept, ctx_out, dev_err);
  if (st != KVQ_OK) return st;
  if (!rings) return KVQ_ERR_INVALID_ARG;
  kvq::CacheSet cs{};
  cs.count = num_caches;
  cs.heads = rings[0].num_kv_heads;
  for (int i = 0; i < num_caches; ++i) {
    const kvq_status rs = kvq::check_ring(rings + i);
    if (rs != KVQ_OK) return rs;
    if (rings[i].num_kv_heads != cs.heads || rings[i].capacity != rings[0].capacity || B > rings[i].num_seqs)
      return KVQ_ERR_INVALID_ARG;
    cs.pages[i] = rings[i].data;
    cs.num_seqs[i] = rings[i].num_seqs;
    cs.max_pages[i] = rings[i].capacity / KVQ_PAGE_SIZE;
  }
  if (repeated(cs)) return KVQ_ERR_INVALID_ARG;
  return from_cuda(
      kvq::launch_tree_commit(1, cs, B, N, pos0, path, n_accept, ctx_out, dev_err, (cudaStream_t)stream));
}

kvq_status kvq_pages_alloc(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                           int max_pages_per_seq, int n, const int32_t* seq_ids, const int32_t* len_old,
                           const int32_t* len_new, int32_t* dev_err, kvq_stream_t stream) {
  return pool_call(kvq::launch_pages_alloc, page_refs, num_pages, block_table, num_seqs, max_pages_per_seq, n, seq_ids,
                   len_old, len_new, nullptr, nullptr, dev_err, stream);
}

kvq_status kvq_pages_fork(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                          int max_pages_per_seq, int n, const int32_t* parents, const int32_t* children,
                          const int32_t* len, int32_t* copy_src, int32_t* copy_dst, int32_t* dev_err,
                          kvq_stream_t stream) {
  if (n > 0 && (!copy_src || !copy_dst)) return KVQ_ERR_INVALID_ARG;
  return pool_call(kvq::launch_pages_fork, page_refs, num_pages, block_table, num_seqs, max_pages_per_seq, n, parents,
                   children, len, copy_src, copy_dst, dev_err, stream);
}

kvq_status kvq_pages_free(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                          int max_pages_per_seq, int n, const int32_t* seq_ids, const int32_t* len_old,
                          const int32_t* len_new, int32_t* dev_err, kvq_stream_t stream) {
  return pool_call(kvq::launch_pages_free, page_refs, num_pages, block_table, num_seqs, max_pages_per_seq, n, seq_ids,
                   len_old, len_new, nullptr, nullptr, dev_err, stream);
}

kvq_status kvq_pages_compact(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                             int max_pages_per_seq, int32_t* copy_src, int32_t* copy_dst, int32_t* n_moves,
                             int32_t* dev_err, kvq_stream_t stream) {
  const kvq_status st = check_pool(page_refs, num_pages, block_table, num_seqs, max_pages_per_seq, dev_err);
  if (st != KVQ_OK) return st;
  if (!n_moves || (num_pages > 1 && (!copy_src || !copy_dst))) return KVQ_ERR_INVALID_ARG;  // one page: empty lists
  const size_t bytes = 4 * (size_t)(num_pages / 2);
  if (overlap(copy_src, bytes, copy_dst, bytes) || overlap(copy_src, bytes, n_moves, 4) || overlap(copy_dst, bytes, n_moves, 4))
    return KVQ_ERR_INVALID_ARG;
  kvq::PoolJob j{page_refs, num_pages, block_table, num_seqs, max_pages_per_seq, 0,       nullptr,
                 nullptr,   nullptr,   copy_src,    copy_dst, n_moves,           dev_err};
  return from_cuda(kvq::launch_pages_compact(j, (cudaStream_t)stream));
}

kvq_status kvq_pages_copy(const kvq_int4_cache* caches, int num_caches, int n, const int32_t* src,
                          const int32_t* dst, const int32_t* count, int32_t* dev_err, kvq_stream_t stream) {
  kvq::CacheSet cs{};
  const kvq_status st = cache_set(caches, num_caches, cs);
  if (st != KVQ_OK) return st;
  if (n < 0 || !dev_err) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!src || !dst) return KVQ_ERR_INVALID_ARG;
  return from_cuda(kvq::launch_pages_copy(cs, n, src, dst, count, dev_err, (cudaStream_t)stream));
}

}  // extern "C"
