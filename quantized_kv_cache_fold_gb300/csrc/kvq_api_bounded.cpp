// C-ABI entry points that hold a session's cache to a size: attention under a window with first tokens, attention
// whose weights are kept. Host-side argument checks and dispatch only; see include/kvq.h for the contract of each call.

#include <algorithm>
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

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// The prologue of the queries, and the append where there are new rows; the rotated queries land at the workspace's start.
kvq_status prologue(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q, kvq_dtype dtype, int B,
                    int S, int num_q_heads, const int32_t* ctx_len, const void* k_new, const void* v_new, float eps,
                    void* workspace, int32_t* dev_err, kvq_stream_t stream, int fwht) {
  kvq::PrepJobs j{};
  j.cache = *cache;
  j.fwht = fwht;
  j.Mk = Mk;
  j.k = k_new;
  j.v = v_new;
  j.kv_bf16 = dtype == KVQ_BF16;
  j.T = k_new ? B * S : 0;
  j.ctx_len = ctx_len;
  j.S = S;
  j.Mq = Mq;
  j.q = q;
  j.q_bf16 = dtype == KVQ_BF16;
  j.nq_rows = B * S * num_q_heads;
  j.q_rot = static_cast<float*>(workspace);
  j.eps = eps;
  j.dev_err = dev_err;
  return from_cuda(kvq::launch_prep(j, (cudaStream_t)stream));
}

// What both kinds of attention over the int4 cache refuse.
kvq_status check_attn(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q, kvq_dtype dtype, int B,
                      int S, int num_q_heads, const int32_t* ctx_len, const void* k_new, const void* v_new, float sm_scale,
                      float eps, const void* out, kvq_dtype out_dtype, const void* workspace, const int32_t* dev_err) {
  const kvq_status st = kvq::check_decode_int4_args(cache, Mq, Mk, q, dtype, B, S, num_q_heads, ctx_len, k_new, v_new,
                                                    sm_scale, eps, static_cast<const float*>(out), nullptr, dev_err);
  if (st != KVQ_OK) return st;
  if (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return KVQ_ERR_INVALID_ARG;
  if ((long long)B * (cache->max_pages_per_seq + 2) > (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

kvq::AttnJob attn_job(const kvq_int4_cache* cache, int B, int S, int num_q_heads, const int32_t* ctx_len, float sm_scale,
                      void* out, kvq_dtype out_dtype, void* workspace, int32_t* dev_err) {
  kvq::AttnJob a{};
  a.fmt = 0;
  a.cache = *cache;
  a.B = B;
  a.S = S;
  a.Hq = num_q_heads;
  a.Hkv = cache->num_kv_heads;
  a.ctx = ctx_len;
  a.q_rot = static_cast<float*>(workspace);
  a.sm_scale = sm_scale;
  a.out = static_cast<float*>(out);
  a.out_bf16 = out_dtype == KVQ_BF16;
  a.partials =
      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kvq::workspace_qrot_bytes(B, S, num_q_heads));
  a.dev_err = dev_err;
  return a;
}

kvq_status window_impl(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q, kvq_dtype dtype,
                       int B, int S, int num_q_heads, const int32_t* ctx_len, int window, int sinks, const void* k_new,
                       const void* v_new, float sm_scale, float eps, void* out, kvq_dtype out_dtype, void* workspace,
                       size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream, int fwht) {
  kvq_status st = check_attn(cache, Mq, Mk, q, dtype, B, S, num_q_heads, ctx_len, k_new, v_new, sm_scale, eps, out,
                             out_dtype, workspace, dev_err);
  if (st != KVQ_OK) return st;
  if (window < 1 || sinks < 0) return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kvq_decode_workspace_bytes(B, S, num_q_heads, cache->num_kv_heads)) return KVQ_ERR_INVALID_ARG;
  st = prologue(cache, Mq, Mk, q, dtype, B, S, num_q_heads, ctx_len, k_new, v_new, eps, workspace, dev_err, stream, fwht);
  if (st != KVQ_OK) return st;
  kvq::AttnJob a = attn_job(cache, B, S, num_q_heads, ctx_len, sm_scale, out, out_dtype, workspace, dev_err);
  // positions end at 2^30: wider windows and more first tokens mean the same
  a.window = std::min(window, 1 << 30);
  a.sinks = std::min(sinks, 1 << 30);
  a.append = k_new != nullptr;
  return from_cuda(kvq::launch_attention(a, (cudaStream_t)stream));
}

kvq_status check_mass(const kvq_token_mass* m, const kvq_int4_cache* cache, int B) {
  if (!m || !m->mass || !m->ids || !aligned(m->mass, 16) || !aligned(m->ids, 4)) return KVQ_ERR_INVALID_ARG;
  if (m->num_seqs < 1 || B > m->num_seqs || m->num_kv_heads < 1 || m->max_tokens < 1 || m->max_tokens % 4) return KVQ_ERR_INVALID_ARG;
  if (cache && (m->num_kv_heads != cache->num_kv_heads ||
                m->max_tokens < (long long)cache->max_pages_per_seq * KVQ_PAGE_SIZE))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

kvq_status mass_impl(const kvq_int4_cache* cache, const kvq_token_mass* mass, const float* Mq, const float* Mk,
                     const void* q, kvq_dtype dtype, int B, int num_q_heads, const int32_t* ctx_len,
                     const int32_t* positions, const void* k_new, const void* v_new, float sm_scale, float eps, void* out,
                     kvq_dtype out_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream,
                     int fwht) {
  kvq_status st = check_attn(cache, Mq, Mk, q, dtype, B, 1, num_q_heads, ctx_len, k_new, v_new, sm_scale, eps, out,
                             out_dtype, workspace, dev_err);
  if (st != KVQ_OK) return st;
  st = check_mass(mass, cache, B);
  if (st != KVQ_OK) return st;
  if (!positions) return KVQ_ERR_INVALID_ARG;
  // mass and ids are written while other blocks still read the lists and write out
  const size_t held = 4 * (size_t)mass->num_seqs * mass->num_kv_heads * mass->max_tokens;
  const size_t rows = (size_t)B * num_q_heads * KVQ_HEAD_DIM;
  if (overlap(mass->mass, held, mass->ids, held)) return KVQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)mass->mass, (const void*)mass->ids})
    if (overlap(x, held, out, rows * (out_dtype == KVQ_BF16 ? 2 : 4)) || overlap(x, held, ctx_len, 4 * (size_t)B) ||
        overlap(x, held, positions, 4 * (size_t)B))
      return KVQ_ERR_INVALID_ARG;
  const size_t need = kvq_mass_workspace_bytes(B, num_q_heads, cache->num_kv_heads, cache->max_pages_per_seq);
  if (need == 0) return KVQ_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return KVQ_ERR_INVALID_ARG;
  st = prologue(cache, Mq, Mk, q, dtype, B, 1, num_q_heads, ctx_len, k_new, v_new, eps, workspace, dev_err, stream, fwht);
  if (st != KVQ_OK) return st;
  kvq::AttnJob a = attn_job(cache, B, 1, num_q_heads, ctx_len, sm_scale, out, out_dtype, workspace, dev_err);
  a.append = k_new != nullptr;
  a.scores = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.partials) +
                                      kvq::workspace_mass_partials_bytes(B, num_q_heads, a.Hkv));
  a.mass = mass->mass;
  a.ids = mass->ids;
  a.mass_len = mass->max_tokens;
  a.positions = positions;
  return from_cuda(kvq::launch_attention(a, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

kvq_status kvq_window_attn_int4(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                                kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len, int window,
                                int sinks, const void* k_new, const void* v_new, float sm_scale, float eps, void* out,
                                kvq_dtype out_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                kvq_stream_t stream) {
  return window_impl(cache, Mq, Mk, q, dtype, B, S, num_q_heads, ctx_len, window, sinks, k_new, v_new, sm_scale, eps, out,
                     out_dtype, workspace, workspace_bytes, dev_err, stream, 0);
}

kvq_status kvq_window_attn_int4_fwht(const kvq_int4_cache* cache, const float* wq, const float* wk, const void* q,
                                     kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len, int window,
                                     int sinks, const void* k_new, const void* v_new, float sm_scale, float eps,
                                     void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                     int32_t* dev_err, kvq_stream_t stream) {
  return window_impl(cache, wq, wk, q, dtype, B, S, num_q_heads, ctx_len, window, sinks, k_new, v_new, sm_scale, eps, out,
                     out_dtype, workspace, workspace_bytes, dev_err, stream, 1);
}

size_t kvq_mass_workspace_bytes(int B, int num_q_heads, int num_kv_heads, int max_pages_per_seq) {
  if (kvq_decode_workspace_bytes(B, 1, num_q_heads, num_kv_heads) == 0 || max_pages_per_seq < 1 || max_pages_per_seq > (1 << 24) ||
      (long long)B * num_kv_heads * max_pages_per_seq > (1LL << 31))
    return 0;
  return kvq::workspace_qrot_bytes(B, 1, num_q_heads) + kvq::workspace_mass_partials_bytes(B, num_q_heads, num_kv_heads) +
         align_up(4 * (size_t)B * num_q_heads * KVQ_PAGE_SIZE * max_pages_per_seq);
}

kvq_status kvq_mass_attn_int4(const kvq_int4_cache* cache, const kvq_token_mass* mass, const float* Mq, const float* Mk,
                              const void* q, kvq_dtype dtype, int B, int num_q_heads, const int32_t* ctx_len,
                              const int32_t* positions, const void* k_new, const void* v_new, float sm_scale, float eps,
                              void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                              kvq_stream_t stream) {
  return mass_impl(cache, mass, Mq, Mk, q, dtype, B, num_q_heads, ctx_len, positions, k_new, v_new, sm_scale, eps, out,
                   out_dtype, workspace, workspace_bytes, dev_err, stream, 0);
}

kvq_status kvq_mass_attn_int4_fwht(const kvq_int4_cache* cache, const kvq_token_mass* mass, const float* wq,
                                   const float* wk, const void* q, kvq_dtype dtype, int B, int num_q_heads,
                                   const int32_t* ctx_len, const int32_t* positions, const void* k_new,
                                   const void* v_new, float sm_scale, float eps, void* out, kvq_dtype out_dtype,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream) {
  return mass_impl(cache, mass, wq, wk, q, dtype, B, num_q_heads, ctx_len, positions, k_new, v_new, sm_scale, eps, out,
                   out_dtype, workspace, workspace_bytes, dev_err, stream, 1);
}

kvq_status kvq_mass_start(const kvq_token_mass* mass, int T, const int32_t* seq_ids, const int32_t* slots,
                          const int32_t* numbers, int fresh, int32_t* dev_err, kvq_stream_t stream) {
  const kvq_status st = check_mass(mass, nullptr, 0);
  if (st != KVQ_OK) return st;
  if (T < 0 || (long long)T * mass->num_kv_heads > (1LL << 30)) return KVQ_ERR_INVALID_ARG;
  if (T == 0) return KVQ_OK;
  if (!seq_ids || !slots || !numbers || !dev_err) return KVQ_ERR_INVALID_ARG;
  const size_t held = 4 * (size_t)mass->num_seqs * mass->num_kv_heads * mass->max_tokens, lists = 4 * (size_t)T;
  if (overlap(mass->mass, held, mass->ids, held)) return KVQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)mass->mass, (const void*)mass->ids})
    for (const int32_t* y : {seq_ids, slots, numbers})
      if (overlap(x, held, y, lists)) return KVQ_ERR_INVALID_ARG;
  return from_cuda(kvq::launch_mass_start(*mass, T, seq_ids, slots, numbers, fresh, dev_err, (cudaStream_t)stream));
}

size_t kvq_prompt_mass_workspace_bytes(int T, int B, int num_q_heads, int num_kv_heads, int rows) {
  if (T < 0 || B < 1 || B > KVQ_MAX_SEQS || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads ||
      num_q_heads / num_kv_heads > 64 || (long long)T * num_q_heads > (1LL << 30))
    return 0;
  return kvq::observe_workspace_bytes(T, B, num_q_heads, num_kv_heads, rows);
}

kvq_status kvq_prompt_mass(const void* q, const void* k, kvq_dtype dtype, int T, int B, int num_q_heads, int num_kv_heads,
                           const int64_t* strides, const int32_t* cu_seqlens, int rows, const int32_t* seq_ids,
                           float sm_scale, const kvq_token_mass* mass, void* workspace, size_t workspace_bytes,
                           int32_t* dev_err, kvq_stream_t stream) {
  if (dtype == KVQ_F32) return KVQ_ERR_UNSUPPORTED;
  if (dtype != KVQ_BF16 && dtype != KVQ_F16) return KVQ_ERR_INVALID_ARG;
  if (num_kv_heads >= 1 && num_q_heads / num_kv_heads > 64) return KVQ_ERR_UNSUPPORTED;
  const size_t need = kvq_prompt_mass_workspace_bytes(T, B, num_q_heads, num_kv_heads, rows);
  if (need == 0) return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.0f)) return KVQ_ERR_INVALID_ARG;
  if (T == 0) return KVQ_OK;
  const kvq_status st = check_mass(mass, nullptr, 0);
  if (st != KVQ_OK) return st;
  if (mass->num_kv_heads != num_kv_heads || (!seq_ids && B > mass->num_seqs)) return KVQ_ERR_INVALID_ARG;
  if (!q || !k || !cu_seqlens || !workspace || !dev_err) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(workspace, 256)) return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < need) return KVQ_ERR_INVALID_ARG;
  const long long D = KVQ_HEAD_DIM;
  long long s[4] = {D * num_q_heads, D, D * num_kv_heads, D};
  if (strides)
    for (int i = 0; i < 4; ++i) {
      if (strides[i] < 8 || strides[i] % 8 || strides[i] > (1LL << 36)) return KVQ_ERR_INVALID_ARG;
      s[i] = strides[i];
    }
  // mass and ids are written while keys and lists are still read
  const size_t held = 4 * (size_t)mass->num_seqs * num_kv_heads * mass->max_tokens;
  const size_t qb = 2 * (size_t)((T - 1) * s[0] + (num_q_heads - 1) * s[1] + D);
  const size_t kb = 2 * (size_t)((T - 1) * s[2] + (num_kv_heads - 1) * s[3] + D);
  if (overlap(mass->mass, held, mass->ids, held)) return KVQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)mass->mass, (const void*)mass->ids})
    if (overlap(x, held, q, qb) || overlap(x, held, k, kb) || overlap(x, held, cu_seqlens, 4 * (size_t)(B + 1)) ||
        (seq_ids && overlap(x, held, seq_ids, 4 * (size_t)B)) || overlap(x, held, workspace, need))
      return KVQ_ERR_INVALID_ARG;
  kvq::ObserveJob j{};
  j.q = q;
  j.k = k;
  j.f16 = dtype == KVQ_F16;
  j.T = T;
  j.B = B;
  j.Hq = num_q_heads;
  j.Hkv = num_kv_heads;
  j.qs_t = s[0], j.qs_h = s[1], j.ks_t = s[2], j.ks_h = s[3];
  j.cu_seqlens = cu_seqlens;
  j.seq_ids = seq_ids;
  j.rows = rows;
  j.sm_scale = sm_scale;
  j.mass = mass->mass;
  j.ids = mass->ids;
  j.num_seqs = mass->num_seqs;
  j.mass_len = mass->max_tokens;
  j.dev_err = dev_err;
  return from_cuda(kvq::launch_observe(j, workspace, (cudaStream_t)stream));
}

kvq_status kvq_evict_int4(const kvq_int4_cache* caches, const kvq_token_mass* masses, int num_caches, int B,
                          const int32_t* ctx_len, const int32_t* seen, int budget, int sinks, int recent,
                          int32_t* ctx_out, int32_t* dev_err, kvq_stream_t stream) {
  kvq::EvictJob j{};
  kvq_status st = kvq::cache_set(caches, num_caches, j.cs);
  if (st != KVQ_OK) return st;
  if (!masses || !ctx_len || !seen || !dev_err || B < 1 || B > KVQ_MAX_SEQS) return KVQ_ERR_INVALID_ARG;
  if (budget < 1 || sinks < 0 || recent < 0) return KVQ_ERR_INVALID_ARG;
  const size_t lens = 4 * (size_t)B;
  if (ctx_out && (overlap(ctx_len, lens, ctx_out, lens) || overlap(seen, lens, ctx_out, lens))) return KVQ_ERR_INVALID_ARG;
  for (int i = 0; i < num_caches; ++i) {
    if (B > caches[i].num_seqs) return KVQ_ERR_INVALID_ARG;
    st = check_mass(masses + i, caches + i, B);
    if (st != KVQ_OK) return st;
    if (!aligned(masses[i].ids, 16)) return KVQ_ERR_INVALID_ARG;
    j.mass[i] = masses[i].mass;
    j.ids[i] = masses[i].ids;
    j.mass_len[i] = masses[i].max_tokens;
  }
  // every list of masses and numbers is written while others are read: all apart
  if (kvq::repeated(j.cs)) return KVQ_ERR_INVALID_ARG;
  auto bytes = [&](int i) { return 4 * (size_t)masses[i].num_seqs * masses[i].num_kv_heads * masses[i].max_tokens; };
  for (int i = 0; i < num_caches; ++i) {
    for (const void* x : {(const void*)j.mass[i], (const void*)j.ids[i]}) {
      for (const int32_t* y : {ctx_len, seen, (const int32_t*)ctx_out})
        if (y && overlap(x, bytes(i), y, lens)) return KVQ_ERR_INVALID_ARG;
      for (int k = 0; k < i; ++k)
        if (overlap(x, bytes(i), j.mass[k], bytes(k)) || overlap(x, bytes(i), j.ids[k], bytes(k))) return KVQ_ERR_INVALID_ARG;
    }
    if (overlap(j.mass[i], bytes(i), j.ids[i], bytes(i))) return KVQ_ERR_INVALID_ARG;
    if ((long long)j.cs.max_pages[i] * KVQ_PAGE_SIZE > KVQ_EVICT_MAX_TOKENS) return KVQ_ERR_UNSUPPORTED;
  }
  if ((long long)num_caches * B * j.cs.heads > (1LL << 27)) return KVQ_ERR_UNSUPPORTED;
  j.B = B;
  j.ctx_len = ctx_len;
  j.seen = seen;
  j.budget = budget;
  j.sinks = sinks;
  j.recent = recent;
  j.ctx_out = ctx_out;
  j.dev_err = dev_err;
  return from_cuda(kvq::launch_evict(j, (cudaStream_t)stream));
}

}  // extern "C"
