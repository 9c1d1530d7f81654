/*
 * kvq.h -- C ABI of the rotated 4-bit KV-cache decode path (GB300, sm_103a).
 *
 * Method: "Serving Kolibri-1 with a 4-bit KV cache" (sevren.ai), section "What we do":
 * every key of a full-attention layer is rotated by a fixed randomized Hadamard matrix
 * R = H diag(s)/sqrt(128) after its RMS norm, stored as 4-bit codes with one fp16 scale
 * and one fp16 offset per token and head (4.25 bits per number); values are stored the
 * same way without rotation; queries are rotated by the same R with both QK-norm gains
 * folded in, and decode attention reads the 4-bit codes directly. The 40 sliding-window
 * layers (window 513) keep a stock FP8 e4m3 cache, read by the same kernel family.
 *
 * Conventions for every entry point:
 *  - All pointers are owned by the caller; the library allocates nothing. Pointers
 *    documented as "device" must be device-accessible memory of the current device;
 *    "host" pointers are ordinary CPU memory.
 *  - Calls taking a stream are asynchronous on that stream and never synchronise.
 *  - Host-side checks run first; on failure the call returns a non-zero kvq_status and
 *    launches nothing.
 *  - Problems only visible on the device (a block-table entry outside the page pool, a
 *    position beyond capacity, a non-finite input, an fp16 scale or offset that had to
 *    saturate, a bounded wait that gave up) are OR-ed into *dev_err as KVQ_DEVERR_* bits;
 *    the affected token-heads or pages are skipped. Kernels never trap and never spin
 *    without a time limit. The caller reads *dev_err after synchronising.
 *  - Kernels are launched with programmatic stream serialisation, so a call's first kernel
 *    may start while the previous kernel on the stream is still running. Until that kernel
 *    has completed it reads none of the call's inputs except the folded prologue weights
 *    (Mq, Mk and their FWHT multipliers), which the int4 calls stage on chip first. Those
 *    must be complete when the call is made: written by a host copy, by an ordinary kernel,
 *    or by a kernel that allows dependent launch only after writing them. Within a call each
 *    kernel waits for the one before it before reading anything that kernel writes.
 *  - Fixed geometry: head_dim 128, 64 tokens per page.
 *  - Thread-safe: no mutable global state beyond per-device attribute caches and the
 *    test-only wait limit of kvq_set_stage_wait_limit_ns.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The same type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* kvq_stream_t;

typedef enum kvq_status {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned buffer, workspace too small */
  KVQ_ERR_UNSUPPORTED = 2, /* head_dim != 128, page_size != 64, S outside 1..8, too many rows */
  KVQ_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed */
  KVQ_ERR_SCRATCH_TOO_SMALL = 4 /* kvq_decode_attn_int4_noalloc: request needs more than its fixed scratch */
} kvq_status;

/* KVQ_F16 is taken by the calls over prompts only (kvq_prompt_attn, kvq_prompt_attn_sinks, kvq_prompt_mass). */
typedef enum kvq_dtype { KVQ_F32 = 0, KVQ_BF16 = 1, KVQ_F16 = 2 } kvq_dtype;

#define KVQ_HEAD_DIM 128
#define KVQ_PAGE_SIZE 64
#define KVQ_MAX_SEQS 1024

/* bits of *dev_err */
#define KVQ_DEVERR_PAGE 0x1      /* block-table entry outside [0, num_pages) */
#define KVQ_DEVERR_POS 0x2       /* sequence id or position outside the cache */
#define KVQ_DEVERR_NONFINITE 0x4 /* NaN/Inf in a key, value or query row (row skipped) */
#define KVQ_DEVERR_RANGE 0x8     /* fp16 scale or offset saturated at +-65504 */
#define KVQ_DEVERR_TIMEOUT 0x10  /* a bounded wait on a copy gave up (results invalid) */
#define KVQ_DEVERR_POOL 0x20     /* no free page left, or a page freed more often than it is held */

/*
 * Paged int4 cache of one full-attention layer.
 * Physical layout: one contiguous 8704-byte block per (page, KV head), so that one bulk copy
 * moves a page of one head into shared memory:
 *   pages: [num_pages][num_kv_heads][8704] bytes (device, 16-byte aligned); within a block
 *     bytes    0..4095  K codes [64 tokens][64 bytes]
 *     bytes 4096..8191  V codes [64 tokens][64 bytes]
 *     bytes 8192..8447  K meta  [64 tokens] uint32
 *     bytes 8448..8703  V meta  [64 tokens] uint32
 *   A K record: byte b holds code 2b in its low nibble and code 2b+1 in its high nibble; its
 *     four 16-byte chunks are stored in XOR order: logical chunk c of token slot t at physical
 *     chunk c ^ (((t >> 1) & 1) | ((t >> 2) & 2)).
 *   A V record: 32 little-endian 16-bit elements; element l holds dims 4l..4l+3, each code c
 *     as a sign bit (c < 8) and a 3-bit magnitude e (7 - c if the sign is set, else c - 8),
 *     so that c - 7.5 = (sign ? -1 : 1) * (e + 0.5). Field bits (e, sign) per dim:
 *     dim 4l: 1-3, 15; dim 4l+1: 4-6, 14; dim 4l+2: 11-13, 7; dim 4l+3: 8-10, 0. With these
 *     positions one lop3 on the element, on it shifted left by 1, on its bytes swapped, or on
 *     those shifted left by 7, gives an f16 subnormal of (c - 7.5) times a power of two.
 *   In V records the four 16-byte chunks of token slot t (0..63)
 *   are stored in XOR order: logical chunk c at physical chunk c ^ ((t >> 1) & 3), so a
 *   transposing shared-memory read of eight consecutive tokens touches eight bank groups.
 *   A meta word: bits 0..15 the fp16 scale, bits 16..31 the fp16 offset; value = code*scale + offset.
 *   block_table: [num_seqs][max_pages_per_seq] int32 (device): physical page of logical
 *     page p of sequence q; position `pos` lives in page pos/64, slot pos%64.
 */
#define KVQ_INT4_BLOCK_BYTES 8704

typedef struct kvq_int4_cache {
  uint8_t* pages;
  const int32_t* block_table;
  int32_t num_seqs;
  int32_t max_pages_per_seq;
  int32_t num_pages;
  int32_t num_kv_heads;
  int32_t page_size; /* must be 64 */
  int32_t head_dim;  /* must be 128 */
} kvq_int4_cache;

/*
 * FP8 e4m3 ring cache of one sliding-window layer (stock format: one fp32 scale per
 * tensor). Position `pos` of sequence q, head h lives in slot pos % capacity. The ring is
 * stored in blocks of 64 slots, keys then values, one contiguous 16384-byte block each:
 *   data: [num_seqs][num_kv_heads][capacity/64][2 (K, V)][64 slots][128] bytes (device,
 *   16-byte aligned); the eight 16-byte chunks of the record in slot t are stored at
 *   physical chunk c ^ (t & 7).
 * capacity must be a multiple of 64 and at least window + S - 1 for the calls using it.
 */
typedef struct kvq_fp8_ring {
  uint8_t* data;
  int32_t num_seqs;
  int32_t num_kv_heads;
  int32_t capacity;
  int32_t head_dim; /* must be 128 */
} kvq_fp8_ring;

/* Human-readable name of a status code (static string). */
const char* kvq_status_string(kvq_status status);

/*
 * kvq_build_rotation -- section "What we do": R = H diag(s)/sqrt(128), H the Sylvester
 * Hadamard matrix, s a random sign per column: s[j] = +1 when the top bit of the j-th
 * output of splitmix64 seeded with `seed` is 0, else -1. Entries computed in fp64 and
 * rounded to fp32.
 *   s_out: host int8[head_dim] (may be NULL); R_out: host float[head_dim*head_dim], row-major.
 * Returns KVQ_ERR_UNSUPPORTED unless head_dim == 128, KVQ_ERR_INVALID_ARG if R_out is NULL.
 */
kvq_status kvq_build_rotation(uint64_t seed, int head_dim, int8_t* s_out, float* R_out);

/*
 * kvq_fold_qk -- section "What we do", QK-norm gain folding: scores depend only on q.k,
 * so g_k moves to the query side and the cache holds R n(k):
 *   M_q = R diag(g_q * g_k)  (each entry the fp64 product R[j][i]*(g_q[i]*g_k[i]) rounded
 *   once to fp32),  M_k = R.
 *   R, g_q, g_k: host inputs (row-major R); Mq_out, Mk_out: host float[128*128] outputs.
 */
kvq_status kvq_fold_qk(const float* R, const float* g_q, const float* g_k, int head_dim, float* Mq_out,
                       float* Mk_out);

/*
 * kvq_fold_qk_fwht -- the same rotation and gain fold for the fast Walsh-Hadamard prologue
 * (kvq_rotate_quant_append_fwht, kvq_decode_attn_int4_fwht). Because R = H diag(s)/sqrt(128),
 * R n = H (s n)/sqrt(128) and R diag(g_q g_k) n = H (s g_q g_k n)/sqrt(128): the folded form is
 * one multiplier per channel in front of H.
 *   s: host int8[128] of +1/-1 (from kvq_build_rotation); g_q, g_k: host float[128].
 *   wq_out[i] = s[i]*g_q[i]*g_k[i] (fp64 product rounded once to fp32); wk_out[i] = s[i].
 * Returns KVQ_ERR_INVALID_ARG for a NULL pointer or an s entry other than +1/-1.
 */
kvq_status kvq_fold_qk_fwht(const int8_t* s, const float* g_q, const float* g_k, int head_dim, float* wq_out,
                            float* wk_out);

/*
 * kvq_rotate_quant_append -- section "What we do": keys rotated (with their RMS norm) by
 * M_k and values unrotated, each quantised to 4-bit codes with fp16 scale/offset per
 * token and head, written into the page slot of (seq_ids[t], positions[t]).
 *   Mk:        device float[128*128] row-major (y = M_k n(k)).
 *   k, v:      device [T][num_kv_heads][128] of `dtype` (pre-norm keys, raw values).
 *   seq_ids, positions: device int32[T].
 * Arithmetic (bit-exact specification, fp32, IEEE operations in this order):
 *   lanes l=0..31 hold x[4l..4l+3]; t_l = fma(x3,x3,fma(x2,x2,fma(x1,x1,x0*x0)));
 *   t_l <- t_l + t_(l^o) for o = 16,8,4,2,1; inv = 1/sqrt(t/128 + eps); n = x*inv;
 *   y_j = fma chain over i=0..127 of M[j][i]*n_i;
 *   o = fp16 toward -inf of min(y); s = fp16 toward +inf of (max(y)-o)/15 (a zero o or s is
 *   stored as +0; an o below -65504 or an s above 65504 saturates there, KVQ_DEVERR_RANGE);
 *   code_i = 0 if s == 0 else clamp(round_half_even((y_i - o)/s), 0, 15).
 * Values use the same quantiser on the raw row. T == 0 is a no-op.
 */
kvq_status kvq_rotate_quant_append(const kvq_int4_cache* cache, const float* Mk, const void* k, const void* v,
                                   kvq_dtype dtype, int T, const int32_t* seq_ids, const int32_t* positions,
                                   float eps, int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_rotate_quant_append_fwht -- kvq_rotate_quant_append with the second prologue
 * specification: y = c FWHT(wk n(k)), c = fp32(1/sqrt(128)) (R n(k) up to rounding).
 *   wk: device float[128], 16-byte aligned (kvq_fold_qk_fwht's wk_out).
 * Arithmetic (bit-exact specification, fp32): n(k) as in kvq_rotate_quant_append; u_i = wk_i*n_i;
 *   for h = 1, 2, 4, ..., 64 and every i with (i & h) == 0: (u_i, u_i+h) <- (u_i + u_i+h, u_i - u_i+h);
 *   y_j = c*u_j; then the same quantiser. Values as in kvq_rotate_quant_append.
 */
kvq_status kvq_rotate_quant_append_fwht(const kvq_int4_cache* cache, const float* wk, const void* k, const void* v,
                                        kvq_dtype dtype, int T, const int32_t* seq_ids, const int32_t* positions,
                                        float eps, int32_t* dev_err, kvq_stream_t stream);

/*
 * Bytes of device workspace needed by kvq_decode_attn_int4 / kvq_decode_attn_fp8_swa for
 * B sequences, S query rows each, num_q_heads query heads over num_kv_heads KV heads.
 * Returns 0 for arguments no call would accept.
 */
size_t kvq_decode_workspace_bytes(int B, int S, int num_q_heads, int num_kv_heads);

/*
 * kvq_decode_attn_int4 -- split-K flash-decoding attention over the int4 cache (section
 * "What we do": decode reads the 4-bit codes directly, nothing is rotated back).
 *   Sequence b (0..B-1) uses block-table row b and has ctx_len[b] cached positions.
 *   Query row r (0..S-1) sits at position ctx_len[b] + r and attends causally to
 *   positions 0..ctx_len[b]+r (a speculative-decoding verify block when S > 1).
 *   q:        device [B][S][num_q_heads][128] of `dtype`, pre-norm queries; the call applies
 *             q~ = M_q n(q) with the prologue arithmetic above. Query head hq reads KV head
 *             hq / (num_q_heads/num_kv_heads).
 *   k_new, v_new: device [B][S][num_kv_heads][128] of `dtype`, or both NULL. When given, the
 *             S rows are rotated, quantised and appended at positions ctx_len[b]+r first.
 *   Mq, Mk:   device float[128*128] (Mk only read when k_new is given).
 *   sm_scale: softmax scale applied to q~.k (1/sqrt(128) for the model).
 *   out:      device float [B][S][num_q_heads][128], the normalised attention output.
 *   workspace: device, >= kvq_decode_workspace_bytes(B, S, num_q_heads, num_kv_heads),
 *             256-byte aligned; contents need no initialisation.
 *   q_rot_out: optional device float [B][S][num_q_heads][128] copy of q~ (NULL to skip).
 * Requires 1 <= B <= KVQ_MAX_SEQS, 1 <= S <= 8, S*(num_q_heads/num_kv_heads) <= 48.
 */
kvq_status kvq_decode_attn_int4(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                                kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len,
                                const void* k_new, const void* v_new, float sm_scale, float eps, float* out,
                                void* workspace, size_t workspace_bytes, float* q_rot_out, int32_t* dev_err,
                                kvq_stream_t stream);

/*
 * kvq_decode_attn_int4_fwht -- kvq_decode_attn_int4 with the FWHT prologue for the queries
 * (q~ = c FWHT(wq n(q)) in the fp32 order of kvq_rotate_quant_append_fwht) and, when
 * k_new/v_new are given, for the appended keys. The cache must have been filled with the FWHT
 * prologue too (kvq_rotate_quant_append_fwht) for the scores to match R's rotation on both sides.
 *   wq, wk: device float[128], 16-byte aligned (kvq_fold_qk_fwht); wk only read with k_new.
 * All other arguments, limits and errors as kvq_decode_attn_int4.
 */
kvq_status kvq_decode_attn_int4_fwht(const kvq_int4_cache* cache, const float* wq, const float* wk, const void* q,
                                     kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len,
                                     const void* k_new, const void* v_new, float sm_scale, float eps, float* out,
                                     void* workspace, size_t workspace_bytes, float* q_rot_out, int32_t* dev_err,
                                     kvq_stream_t stream);

/*
 * kvq_fp8_append -- stock FP8 cache write of the sliding-window layers: code =
 * e4m3(x / scale) with an IEEE fp32 division, round-to-nearest-even, saturating to +-448,
 * into slot positions[t] % capacity of sequence seq_ids[t]. Rows with a non-finite entry
 * are skipped (KVQ_DEVERR_NONFINITE).
 *   k, v: device [T][num_kv_heads][128] of `dtype`; seq_ids, positions: device int32[T].
 */
kvq_status kvq_fp8_append(const kvq_fp8_ring* ring, const void* k, const void* v, kvq_dtype dtype, int T,
                          const int32_t* seq_ids, const int32_t* positions, float k_scale, float v_scale,
                          int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_decode_attn_fp8_swa -- sliding-window attention over the FP8 ring (the stock path of
 * the 40 window-513 layers). Row r of sequence b sits at position pos0[b] + r and attends
 * to positions max(0, pos0[b]+r-window+1) .. pos0[b]+r, dequantised as e4m3(c)*k_scale and
 * e4m3(c)*v_scale. q is used as given (no prologue).
 *   q: device [B][S][num_q_heads][128] of `dtype`; out: device float [B][S][num_q_heads][128].
 *   k_new, v_new: device [B][S][num_kv_heads][128] of `dtype` or both NULL; when given they
 *     are written (kvq_fp8_append arithmetic) at positions pos0[b]+r before attending.
 *   workspace: as for kvq_decode_attn_int4.
 * Requires 1 <= B <= KVQ_MAX_SEQS, 1 <= S <= 8, window >= 1, capacity >= window + S - 1.
 */
kvq_status kvq_decode_attn_fp8_swa(const kvq_fp8_ring* ring, const void* q, kvq_dtype dtype, int B, int S,
                                   int num_q_heads, const int32_t* pos0, int window, const void* k_new,
                                   const void* v_new, float k_scale, float v_scale, float sm_scale, float* out,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                   kvq_stream_t stream);

/*
 * kvq_fp8_swa_plan -- the launch shape kvq_decode_attn_fp8_swa takes for these sizes on the
 * calling thread's current device; no launch, nothing allocated (reads device attributes and
 * the kernel's occupancy, cached per device).
 *   out[0]: CTAs per (sequence, KV head): the cluster size of the one-launch path, which
 *           appends and attends in one kernel and merges on chip; 1 also for the
 *           one-CTA-per-pair shape taken when the call has at least as many (sequence, KV head)
 *           pairs as the device has SMs; 0 where the one-launch path does not fit (rings
 *           beyond one cluster; 40 or more query rows per KV head with fewer pairs than SMs),
 *           which takes a separate append, the split-K kernel and its combine pass.
 *   out[1]: unit streams (warps per query-tile group) per CTA; out[2]: copy stages per stream;
 *   out[3]: 32-slot ring units per stream (the largest; 0 with out[0] = 0).
 * Returns KVQ_ERR_INVALID_ARG / KVQ_ERR_UNSUPPORTED under the same conditions on these
 * arguments as kvq_decode_attn_fp8_swa (capacity a positive multiple of 64).
 */
kvq_status kvq_fp8_swa_plan(int capacity, int B, int S, int num_q_heads, int num_kv_heads, int32_t out[4]);

/*
 * kvq_set_stage_wait_limit_ns -- test hook for the failure path of the bounded waits: sets, for
 * every later launch in the process, how long the split-K attention kernel of
 * kvq_decode_attn_int4 (and of the window path's split-K form) waits for a page's copy into a
 * shared-memory stage, and for a stage to be released, before it gives up, sets
 * KVQ_DEVERR_TIMEOUT and abandons the call's remaining pages (outputs then invalid). ns = 0 gives
 * up at the first unsuccessful check. The wait for copies still in flight before a CTA exits
 * always keeps the default. Default 2000000000 (2 s); the default is what a caller should run
 * with. Always returns KVQ_OK.
 */
kvq_status kvq_set_stage_wait_limit_ns(uint64_t ns);

/*
 * kvq_decode_attn_int4_noalloc -- the same computation as kvq_decode_attn_int4 for callers
 * that cannot allocate device memory at decode time (an engine that hands all free GPU
 * memory to its KV pool at start-up, a thread that must not touch the device allocator, an
 * environment where cudaMalloc or a framework allocator is unavailable). The paper has no
 * counterpart: this is a packaging variant of the workspace handling only.
 * The workspace comes from a fixed scratch array inside this library's device image, of
 * KVQ_NOALLOC_SCRATCH_BYTES. The call allocates nothing; the caller still passes every input
 * and output.
 *   - Arguments, checks and results are those of kvq_decode_attn_int4 without (workspace,
 *     workspace_bytes): the same status for the same bad argument.
 *   - Requests with valid arguments whose workspace (kvq_decode_workspace_bytes) exceeds the
 *     scratch return KVQ_ERR_SCRATCH_TOO_SMALL and launch nothing.
 *   - When the memory is taken: under lazy module loading (the CUDA default) the first call on
 *     a device loads the module holding the array, and so allocates its 16 MiB there, while
 *     looking up its device address (with that device current); under eager loading the
 *     library's load does. The device keeps it until the process exits. Make the first call on
 *     each device before reserving the memory pool the engine hands out, and before any
 *     stream capture.
 *   - Every call looks the address up again (cheap once loaded), so calls stay valid across a
 *     cudaDeviceReset.
 *   - All calls on a device share the one scratch array, which keeps the last call's
 *     contents (no call needs it zeroed). Calls whose execution overlaps on the GPU race on
 *     it: serialise them (one stream, or explicit ordering between streams and threads).
 */
#define KVQ_NOALLOC_SCRATCH_BYTES (16u << 20)

kvq_status kvq_decode_attn_int4_noalloc(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                                        kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len,
                                        const void* k_new, const void* v_new, float sm_scale, float eps, float* out,
                                        float* q_rot_out, int32_t* dev_err, kvq_stream_t stream);

/* ------------------------------------------------------------------ a prompt's attention */

/*
 * kvq_prompt_attn -- causal attention over whole prompts, packed end to end without padding.
 *   Sequence b (0..B-1) holds tokens cu_seqlens[b] .. cu_seqlens[b+1]-1 of the packed tensors; its
 *   token i attends to its tokens max(0, i-window+1)..i (window <= 0: 0..i):
 *     out_i = sum_j softmax_j(sm_scale q_i.k_j) v_j .
 *   q, k and v are used as given, as in kvq_decode_attn_fp8_swa: for a full-attention layer pass
 *   g_q*g_k*n(q) and n(k) (scores do not change under the rotation, so none is applied), and the
 *   same n(k) to kvq_rotate_quant_append (its norm leaves a normalised row as it is, up to eps).
 *   q:        device [T][num_q_heads][128] of `dtype` (KVQ_BF16 or KVQ_F16); query head hq reads
 *             KV head hq / (num_q_heads/num_kv_heads).
 *   k, v:     device [T][num_kv_heads][128] of `dtype`.
 *   strides:  host int64[8] or NULL (packed): elements between tokens and between heads of q, k, v
 *             and out, in this order (q token, q head, k token, ...). Each a positive multiple of 8;
 *             rows of 128 elements are contiguous.
 *   cu_seqlens: device int32[B+1], 0 <= cu_seqlens[0] <= ... <= cu_seqlens[B] <= T (else the
 *             sequences outside that, or that overlap one before them, are skipped,
 *             KVQ_DEVERR_POS). Empty sequences are allowed. Rows of out that no sequence has are
 *             left as they were.
 *   out:      device [T][num_q_heads][128] of `dtype`, rounded once from fp32. It must not overlap
 *             the inputs.
 *   workspace: device, >= kvq_prompt_workspace_bytes(T, B, num_q_heads, num_kv_heads), 256-byte
 *             aligned. As every attention call takes one, so does this, but its kernel keeps everything
 *             on chip: 256 bytes whatever the sizes (0 for arguments that no call accepts), neither
 *             read nor written, so any calls may share one.
 *   A row is NaN only where a key or value that it attends to makes it so: non-finite values in
 *   masked places do not reach it. Nothing is skipped for non-finite inputs.
 * Requires 1 <= B <= KVQ_MAX_SEQS, 0 <= T (T == 0 is a no-op), sm_scale > 0; q, k, v and out
 * 16-byte aligned; T*num_q_heads <= 2^30.
 */
size_t kvq_prompt_workspace_bytes(int T, int B, int num_q_heads, int num_kv_heads);
kvq_status kvq_prompt_attn(const void* q, const void* k, const void* v, kvq_dtype dtype, int T, int B,
                           int num_q_heads, int num_kv_heads, const int64_t* strides, const int32_t* cu_seqlens,
                           int window, float sm_scale, void* out, void* workspace, size_t workspace_bytes,
                           int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_prompt_attn_sinks -- kvq_prompt_attn with a window and a few first tokens that stay visible: token i attends to
 *   its tokens max(0, i-window+1)..i and to tokens 0..min(sinks, i+1)-1 (each once, where the two meet).
 *   sinks: >= 0 (0, or window <= 0: kvq_prompt_attn). All other arguments as there.
 */
kvq_status kvq_prompt_attn_sinks(const void* q, const void* k, const void* v, kvq_dtype dtype, int T, int B,
                                 int num_q_heads, int num_kv_heads, const int64_t* strides, const int32_t* cu_seqlens,
                                 int window, int sinks, float sm_scale, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream);

/* ------------------------------------------------------------------ a tree of drafted tokens */

#define KVQ_MAX_TREE 64 /* drafted tokens of one sequence's tree */
#define KVQ_MAX_CACHES 64 /* layers of one kvq_tree_commit_* or kvq_pages_copy call */

/*
 * kvq_tree_attn_int4 -- attention of a tree of drafted tokens over the int4 cache.
 *   Sequence b has ctx_len[b] cached tokens and N drafted ones, whose keys and values lie behind
 *   the context: drafted token i in the slot of position ctx_len[b] + i. Its query attends to
 *   the whole context and to the drafted tokens of its mask:
 *     tree_mask: device uint64[B][N]; bit j of word [b][i] set: token i attends to drafted token j
 *             (its own bit as well, where it attends to itself; bits from N on are ignored). A row
 *             that attends to nothing (no context, no bit) gives 0. A batch of smaller trees is
 *             padded with tokens that no mask names; their own rows may be ignored.
 *   q:        device [B][N][num_q_heads][128] of `dtype`, pre-norm: q~ = M_q n(q).
 *   k_new, v_new: device [B][N][num_kv_heads][128] of `dtype`, or both NULL: appended at positions
 *             ctx_len[b] + i first, as by kvq_rotate_quant_append.
 *   out:      device [B][N][num_q_heads][128] of out_dtype (KVQ_F32 or KVQ_BF16).
 *   workspace: device, >= kvq_tree_workspace_bytes(B, N, num_q_heads, num_kv_heads), 256-byte
 *             aligned; contents need no initialisation.
 *   The products take q~ in fp16. A row whose q~ is not finite, or has an element of magnitude
 *   65520 or more, is NaN (0 if it attends to nothing); a query that is not finite is flagged
 *   (KVQ_DEVERR_NONFINITE) as well. No other row changes.
 *   Precision: sums, maxima and the join are fp32, q~ and the weights enter the products in fp16
 *   (2^-11 of the value; weights by 2^-31 of the largest at least). With up to 48 rows per KV head
 *   (N times the query heads of one) the codes enter as they are, counted from the middle of their
 *   range, scale and offset in fp32: an element is off by 2^-11 of half its record's range; with
 *   more, keys and values are dequantised to fp16 first (2^-11 of the value, keys by 2^-15 at
 *   least). So 48 and 49 rows of the same call differ by these roundings.
 *   Other arguments, readings of positions and errors as kvq_decode_attn_int4. A position whose
 *   block-table entry is outside the pool is skipped (KVQ_DEVERR_PAGE). Slots of a page that were
 *   never written are masked, but their scales are read: a pool is zeroed before its first use.
 * Requires 1 <= B <= KVQ_MAX_SEQS, 1 <= N <= KVQ_MAX_TREE, num_q_heads/num_kv_heads <= 64,
 * B*(max_pages_per_seq+2) <= 2^31.
 */
size_t kvq_tree_workspace_bytes(int B, int N, int num_q_heads, int num_kv_heads);
kvq_status kvq_tree_attn_int4(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                              kvq_dtype dtype, int B, int N, int num_q_heads, const int32_t* ctx_len,
                              const uint64_t* tree_mask, const void* k_new, const void* v_new, float sm_scale,
                              float eps, void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                              int32_t* dev_err, kvq_stream_t stream);
/* The same with the FWHT prologue (wq, wk: device float[128], 16-byte aligned; kvq_fold_qk_fwht). */
kvq_status kvq_tree_attn_int4_fwht(const kvq_int4_cache* cache, const float* wq, const float* wk, const void* q,
                                   kvq_dtype dtype, int B, int N, int num_q_heads, const int32_t* ctx_len,
                                   const uint64_t* tree_mask, const void* k_new, const void* v_new, float sm_scale,
                                   float eps, void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_tree_attn_fp8_swa -- the same over the e4m3 ring of a sliding-window layer. Drafted token i
 *   lies in slot (pos0[b] + i) % capacity; it stands at position
 *     pos0[b] + max(1, number of drafted tokens it attends to) - 1
 *   (its depth in the tree), and its window reaches back from there: context positions above that
 *   position - window, and the drafted tokens of its mask.
 *   q is used as given and in fp16: NaN for rows as above, without a flag. workspace and out as
 *   above; out must not overlap k_new, v_new, or q but for a q of its own type in its very place
 *   (over the int4 cache it may: q, k_new and v_new are read first). Other arguments as
 *   kvq_decode_attn_fp8_swa.
 * Requires window >= N and capacity >= window + N - 1.
 */
kvq_status kvq_tree_attn_fp8_swa(const kvq_fp8_ring* ring, const void* q, kvq_dtype dtype, int B, int N,
                                 int num_q_heads, const int32_t* pos0, const uint64_t* tree_mask, int window,
                                 const void* k_new, const void* v_new, float k_scale, float v_scale, float sm_scale,
                                 void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                 int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_tree_commit_int4 / kvq_tree_commit_fp8 -- the accepted branch of each tree becomes context:
 *   the record (codes, scales, offsets) of drafted token path[b][i], at position
 *   ctx_len[b] + path[b][i], moves to position ctx_len[b] + i, for i < n_accept[b], in every one
 *   of num_caches layers in one launch. All of a sequence's records are read before any is
 *   written, so any path (also with repeated tokens) gives the records as they were before.
 *   caches / rings: host array of num_caches descriptors (1..KVQ_MAX_CACHES), of the same number of
 *             KV heads (rings: of the same capacity); each with its own block table. No layer twice,
 *             and the drafted positions' pages belong to one sequence each.
 *   path:     device int32[B][N], the accepted tokens in order; an entry outside 0..N-1 within the
 *             first n_accept[b] is skipped (KVQ_DEVERR_POS).
 *   n_accept: device int32[B], clamped to 0..N (KVQ_DEVERR_POS if it had to be).
 *   ctx_out:  device int32[B] or NULL: receives ctx_len[b] + n_accept[b]; must not overlap ctx_len,
 *             path or n_accept.
 * Requires 1 <= B <= KVQ_MAX_SEQS, 1 <= N <= KVQ_MAX_TREE.
 */
kvq_status kvq_tree_commit_int4(const kvq_int4_cache* caches, int num_caches, int B, int N, const int32_t* ctx_len,
                                const int32_t* path, const int32_t* n_accept, int32_t* ctx_out, int32_t* dev_err,
                                kvq_stream_t stream);
kvq_status kvq_tree_commit_fp8(const kvq_fp8_ring* rings, int num_caches, int B, int N, const int32_t* pos0,
                               const int32_t* path, const int32_t* n_accept, int32_t* ctx_out, int32_t* dev_err,
                               kvq_stream_t stream);

/* ------------------------------------------------------------------ the page pool */

/*
 * The pool of an int4 cache's pages is one reference count per page on the device:
 *   page_refs: device int32[num_pages]; 0: free, n: held by n block-table entries. All zero at first.
 * Layers that share a block table share the pool. Unused block-table entries hold -1. The calls
 * below change counts and tables only, in one or two launches; kvq_pages_copy moves the data of the
 * layers. New pages are always the lowest free ones, in ascending order, handed to the requests in
 * theirs, so the outcome does not depend on timing.
 *   block_table: device int32[num_seqs][max_pages_per_seq], written.
 *   n (0..KVQ_MAX_SEQS) rows are named by seq_ids (or parents / children): device int32[n]. A row
 *   outside the table, a length outside 0..64*max_pages_per_seq or the second naming of a row
 *   (the lower index counts) skips the request (KVQ_DEVERR_POS).
 * Requires 1 <= num_pages, num_seqs*max_pages_per_seq <= 2^30, max_pages_per_seq <= 2^24.
 */

/* kvq_pages_alloc -- sequence seq_ids[i] grows from len_old[i] to len_new[i] tokens: its pages
 * ceil(len_old/64) .. ceil(len_new/64)-1 get free pages (count 1). Entries for which none is left
 * are set to -1 (KVQ_DEVERR_POOL). */
kvq_status kvq_pages_alloc(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                           int max_pages_per_seq, int n, const int32_t* seq_ids, const int32_t* len_old,
                           const int32_t* len_new, int32_t* dev_err, kvq_stream_t stream);

/* kvq_pages_fork -- sequence children[i] (whose row holds no pages) becomes a copy of the first
 * len[i] tokens of parents[i]: full pages are shared (count + 1), a last page that is only partly
 * filled is replaced by a free one. copy_src[i] / copy_dst[i] (device int32[n]) receive that page of
 * the parent and of the child for kvq_pages_copy, -1 where there is none; they must not overlap one
 * another or the request's lists. A row may not be parent and child in one call (KVQ_DEVERR_POS,
 * skipped). No free page: entry -1, KVQ_DEVERR_POOL. An entry of the parent's outside the pool: entry
 * -1, KVQ_DEVERR_PAGE. */
kvq_status kvq_pages_fork(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                          int max_pages_per_seq, int n, const int32_t* parents, const int32_t* children,
                          const int32_t* len, int32_t* copy_src, int32_t* copy_dst, int32_t* dev_err,
                          kvq_stream_t stream);

/* kvq_pages_free -- sequence seq_ids[i] shrinks from len_old[i] to len_new[i] tokens: its pages
 * ceil(len_new/64) .. ceil(len_old/64)-1 are given back (count - 1; free at 0) and their entries set
 * to -1. An entry outside the pool is passed over (KVQ_DEVERR_PAGE), a count that is 0 already stays
 * (KVQ_DEVERR_POOL). */
kvq_status kvq_pages_free(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                          int max_pages_per_seq, int n, const int32_t* seq_ids, const int32_t* len_old,
                          const int32_t* len_new, int32_t* dev_err, kvq_stream_t stream);

/* kvq_pages_compact -- the L pages in use move to pages 0..L-1: those behind, in ascending order, to
 * the free ones in front, in ascending order. Counts and every entry of the table are rewritten.
 * copy_src / copy_dst (device int32[num_pages/2]) receive the moves and *n_moves (device) their
 * number (none of the three overlaps another); a page is never both source and destination. Entries
 * that name a page with count 0 stay (KVQ_DEVERR_PAGE). Every table that names pages of the pool has
 * to be rewritten: there is one. */
kvq_status kvq_pages_compact(int32_t* page_refs, int num_pages, int32_t* block_table, int num_seqs,
                             int max_pages_per_seq, int32_t* copy_src, int32_t* copy_dst, int32_t* n_moves,
                             int32_t* dev_err, kvq_stream_t stream);

/* kvq_pages_copy -- page src[i] to page dst[i], all KV heads, in every one of num_caches layers, in
 * one launch, for i < n, or i < min(n, *count) where count (device, may be NULL) is given. A pair
 * with -1 on either side is passed over; one with a page outside the pool too (KVQ_DEVERR_PAGE). A
 * page that is the destination of one pair may not be in another pair: its bytes are unspecified.
 *   caches: host array of num_caches descriptors (1..KVQ_MAX_CACHES); block tables are not read. */
kvq_status kvq_pages_copy(const kvq_int4_cache* caches, int num_caches, int n, const int32_t* src,
                          const int32_t* dst, const int32_t* count, int32_t* dev_err, kvq_stream_t stream);

/* ------------------------------------------------------------------ caches held to a size */

/*
 * kvq_window_attn_int4 -- kvq_decode_attn_int4 with a window and a few first tokens that stay visible: query row r of
 *   sequence b, at position i = ctx_len[b] + r, attends to positions max(0, i-window+1)..i and to 0..min(sinks, i+1)-1
 *   (each once, where the two meet). Pages that hold neither a first token nor one of the rows' windows are not read, and
 *   their block-table entries may be anything: a session's pages between the two may be given back (where all layers that
 *   share the block table have such windows), by kvq_pages_free with len_old = 64*floor((ctx_len-window+1)/64) of the
 *   next call (0 below 0) and len_new = sinks, or the len_old of the time before once that is more. A session that has given
 *   some back ends by two such calls, from ctx_len to that len_new and from min(sinks, ctx_len) to 0 (one from ctx_len to 0,
 *   and a fork, flag the -1 entries between), and its windows grow no wider.
 *   out:      device [B][S][num_q_heads][128] of out_dtype (KVQ_F32 or KVQ_BF16). A row that sees nothing (its pages
 *             outside the pool) gives 0.
 *   workspace: as for kvq_decode_attn_int4 (kvq_decode_workspace_bytes).
 *   The products take q~ in fp16 and weights as the tree calls of few rows do: the same precision, and the same NaN rows.
 *   Other arguments, limits and errors as kvq_decode_attn_int4.
 * Requires window >= 1, sinks >= 0, B*(max_pages_per_seq+2) <= 2^31.
 */
kvq_status kvq_window_attn_int4(const kvq_int4_cache* cache, const float* Mq, const float* Mk, const void* q,
                                kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len, int window,
                                int sinks, const void* k_new, const void* v_new, float sm_scale, float eps, void* out,
                                kvq_dtype out_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                kvq_stream_t stream);
/* The same with the FWHT prologue (wq, wk: device float[128], 16-byte aligned; kvq_fold_qk_fwht). */
kvq_status kvq_window_attn_int4_fwht(const kvq_int4_cache* cache, const float* wq, const float* wk, const void* q,
                                     kvq_dtype dtype, int B, int S, int num_q_heads, const int32_t* ctx_len, int window,
                                     int sinks, const void* k_new, const void* v_new, float sm_scale, float eps,
                                     void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                     int32_t* dev_err, kvq_stream_t stream);

/*
 * What every slot of an int4 cache of one layer has gathered, beside the cache: slot j of sequence q (position j of its
 * block-table row) and KV head h has
 *   mass[q][h][j]: the sum of the attention weights that the queries of that KV head's group have put on it,
 *   ids[q][h][j]:  the number of its token in the sequence (0, 1, ...). After an eviction the slots of different heads
 *                  hold different tokens, in no particular order.
 * mass: device float [num_seqs][num_kv_heads][max_tokens], 16-byte aligned; ids: device int32 of the same shape.
 * max_tokens: a multiple of 4, at least 64*max_pages_per_seq of the cache. The calls read and write only slots below a
 * sequence's length (a mass call: the new token's too).
 * kvq_mass_attn_int4, kvq_prompt_mass and kvq_evict_int4 keep them. Where another call puts tokens into slots
 * (kvq_rotate_quant_append, a decode, window or tree call with new rows, kvq_tree_commit_int4, kvq_pages_fork), mass and ids
 * there are the caller's to set before the next eviction, by kvq_mass_start or from those of other slots: what they held may be
 * of tokens that have left, or of a session before.
 */
typedef struct kvq_token_mass {
  float* mass;
  int32_t* ids;
  int32_t num_seqs;
  int32_t num_kv_heads;
  int32_t max_tokens;
} kvq_token_mass;

/*
 * kvq_mass_attn_int4 -- kvq_decode_attn_int4 for one new token per sequence, with its weights kept: with
 *   w_g[j] the softmax weight of query head g (of KV head h) on slot j of sequence b,
 *     mass[b][h][j] += sum_g w_g[j] for j < ctx_len[b],
 *   and the new token's slot j = ctx_len[b] is set: mass to that sum, ids to positions[b] (the tokens that the sequence
 *   has had before it; the same as ctx_len[b] until the first eviction).
 *   q:        device [B][num_q_heads][128]; k_new, v_new: device [B][num_kv_heads][128] or both NULL.
 *   positions: device int32[B].
 *   out:      device [B][num_q_heads][128] of out_dtype (KVQ_F32 or KVQ_BF16); precision as kvq_window_attn_int4.
 *   workspace: device, >= kvq_mass_workspace_bytes(B, num_q_heads, num_kv_heads, max_pages_per_seq), 256-byte aligned
 *             (4 bytes for every query head and slot: the scores of the call).
 *   Precision of the weights: q~ enters the scores in two fp16 parts (2^-22 of the value), sums are fp32, in an order that
 *   does not depend on timing. A row that is NaN (see kvq_tree_attn_int4) adds nothing; slots of a page outside the
 *   pool, and all of a sequence whose length is outside its block table (KVQ_DEVERR_POS), are left as they were.
 *   mass and ids must not overlap one another, the inputs or out. Other arguments, limits and errors as
 *   kvq_decode_attn_int4 with S = 1.
 * Requires B*num_kv_heads*max_pages_per_seq <= 2^31, B*(max_pages_per_seq+2) <= 2^31, max_pages_per_seq <= 2^24.
 */
size_t kvq_mass_workspace_bytes(int B, int num_q_heads, int num_kv_heads, int max_pages_per_seq);
kvq_status kvq_mass_attn_int4(const kvq_int4_cache* cache, const kvq_token_mass* mass, const float* Mq, const float* Mk,
                              const void* q, kvq_dtype dtype, int B, int num_q_heads, const int32_t* ctx_len,
                              const int32_t* positions, const void* k_new, const void* v_new, float sm_scale, float eps,
                              void* out, kvq_dtype out_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                              kvq_stream_t stream);
/* The same with the FWHT prologue (wq, wk: device float[128], 16-byte aligned; kvq_fold_qk_fwht). */
kvq_status kvq_mass_attn_int4_fwht(const kvq_int4_cache* cache, const kvq_token_mass* mass, const float* wq,
                                   const float* wk, const void* q, kvq_dtype dtype, int B, int num_q_heads,
                                   const int32_t* ctx_len, const int32_t* positions, const void* k_new,
                                   const void* v_new, float sm_scale, float eps, void* out, kvq_dtype out_dtype,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_mass_start -- tokens that another call has put into slots start their masses: for t < T and every KV head h, slot
 *   j = slots[t] of sequence q = seq_ids[t] gets mass[q][h][j] = 0 and ids[q][h][j] = numbers[t], unless `fresh` is 0 and ids
 *   is that number already (where a call over the prompt has set both). fresh other than 0: whatever the slots held.
 *   seq_ids, slots, numbers: device int32[T]. A token whose row or slot is outside mass is passed over (KVQ_DEVERR_POS). No
 *             slot is named twice with different numbers. mass and ids must not overlap one another or the lists.
 * Requires 0 <= T (0 is a no-op), T*num_kv_heads <= 2^30.
 */
kvq_status kvq_mass_start(const kvq_token_mass* mass, int T, const int32_t* seq_ids, const int32_t* slots,
                          const int32_t* numbers, int fresh, int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_prompt_mass -- what the tokens of packed prompts have gathered from their last rows: the mass that a cache filled with
 *   these prompts starts from. With the softmax weights w of kvq_prompt_attn (no window), for token j of sequence b:
 *     mass[seq_ids[b]][h][j] = sum over its rows i >= max(j, n - rows) and the query heads g of KV head h of w_ig[j],
 *     ids[seq_ids[b]][h][j] = j,   j < n = cu_seqlens[b+1] - cu_seqlens[b].
 *   Both are set, whatever they held; places from n on, and rows that no sequence names, are left as they were.
 *   q, k:     as kvq_prompt_attn takes them (KVQ_BF16 or KVQ_F16); strides: host int64[4] or NULL (packed), elements
 *             between tokens and between heads of q, then of k, as there.
 *   rows:     the rows that count, from the end (<= 0, or n and more: all).
 *   seq_ids:  device int32[B] or NULL (b). A row outside mass or named before, offsets as kvq_prompt_attn refuses them,
 *             or a prompt longer than max_tokens: skipped, KVQ_DEVERR_POS.
 *   workspace: device, >= kvq_prompt_mass_workspace_bytes(T, B, num_q_heads, num_kv_heads, rows), 256-byte aligned;
 *             contents need no initialisation.
 *   Precision: products of the 16-bit inputs summed in fp32, weights and sums fp32, in an order that does not depend on
 *   timing. A row whose softmax is NaN (a score that is NaN or +inf, or none above -inf) adds nothing; a score of -inf beside
 *   others is a weight of 0.
 * Requires num_q_heads/num_kv_heads <= 64 and otherwise the sizes of kvq_prompt_attn; mass and ids overlap no input.
 */
size_t kvq_prompt_mass_workspace_bytes(int T, int B, int num_q_heads, int num_kv_heads, int rows);
kvq_status kvq_prompt_mass(const void* q, const void* k, kvq_dtype dtype, int T, int B, int num_q_heads, int num_kv_heads,
                           const int64_t* strides, const int32_t* cu_seqlens, int rows, const int32_t* seq_ids,
                           float sm_scale, const kvq_token_mass* mass, void* workspace, size_t workspace_bytes,
                           int32_t* dev_err, kvq_stream_t stream);

/*
 * kvq_evict_int4 -- eviction by gathered weight: per layer, sequence b and KV head, of the n = ctx_len[b] slots
 *   min(n, budget) stay: those whose token is one of the first (ids < sinks) or one of the newest
 *   (ids >= seen[b] - recent), then those with the largest mass; among equal ones the lower slots (so too where the first
 *   and newest ones are more than the budget). A NaN mass counts less than any other.
 *   A kept slot behind the budget moves, with its record, mass and number, into a slot before it that is given up: the i-th
 *   such slot, ascending, into the i-th one given up. Nothing else changes: slots from the new length on are left as they
 *   were. What stays is the same set for any order, attention does not ask for one, and every call here that goes on
 *   with the sequence appends behind the new length. Each KV head keeps its own tokens.
 *   caches, masses: host arrays of num_caches descriptors (1..KVQ_MAX_CACHES), the layers in the same order; the same
 *             number of KV heads in all. No layer twice; no overlap of any mass or ids with another or with the lists.
 *             The pages of an evicted sequence belong to it alone (of forked sequences that share pages the copies come
 *             first).
 *   ctx_len, seen: device int32[B]: the cached tokens, and how many tokens the sequence has had in all.
 *   ctx_out:  device int32[B] or NULL: receives min(ctx_len[b], budget); must not overlap ctx_len or seen. The pages
 *             behind it can be given back by kvq_pages_free(.., ctx_len, ctx_out, ..), once all layers that share the
 *             block table have evicted.
 *   A length outside the block table is clamped (KVQ_DEVERR_POS). A move from or to a page outside the pool is passed over
 *   (KVQ_DEVERR_PAGE): its token is lost.
 * Requires 1 <= B <= KVQ_MAX_SEQS, budget >= 1, sinks, recent >= 0, 64*max_pages_per_seq <= KVQ_EVICT_MAX_TOKENS,
 * num_caches*B*num_kv_heads <= 2^27, ids 16-byte aligned.
 */
#define KVQ_EVICT_MAX_TOKENS 393216
kvq_status kvq_evict_int4(const kvq_int4_cache* caches, const kvq_token_mass* masses, int num_caches, int B,
                          const int32_t* ctx_len, const int32_t* seen, int budget, int sinks, int recent,
                          int32_t* ctx_out, int32_t* dev_err, kvq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
