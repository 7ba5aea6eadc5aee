/*
 * gqa_attn.h -- C ABI of libgqa_attn.so: causal grouped-query scaled-dot-
 * product attention, forward and backward, for bf16 tensors on an sm_103a GPU.
 *
 * The operation is the ScaledDotProductAttention / MultiHeadAttention of the
 * "Project Overview" page of llm-from-scratch (section "Core Stack: llm/",
 * llm/transformer.py) with the grouped-query heads and causal mask of the
 * microLLM-rocm README (section "Why this project exists": "Decoder-only
 * MHA/GQA ... causal attention" and the causal GQA backward), computed
 * blockwise with running softmax statistics as in the Flash Attention kernel
 * of "Project Overview", section "Performance Layer: kernel/ and parallel/":
 *
 *   S = scale * Q K^T,  key j visible to query i iff j <= i (causal != 0),
 *   LSE_i = ln sum_j exp(S_ij) over visible j,   P = exp(S - LSE),  O = P V,
 *   and for the loss L = sum(dO * O):
 *   dP = dO V^T, Delta_i = sum_d dO_id O_id, dS = P * (dP - Delta),
 *   dQ = scale * dS K,  dK = scale * dS^T Q,  dV = P^T dO,
 *   dK and dV summed over the G = Hq / Hkv query heads that share a K/V head
 *   (query head h reads K/V head h / G).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers, 16-byte aligned, densely
 *     packed (no strides, but for the token views below).  bf16 = IEEE bfloat16 stored as uint16.
 *   - Dense layout:  Q, O, dO, dQ  [B, Hq, T, D];  K, V, dK, dV  [B, Hkv, T, D];
 *                    LSE  [B, Hq, T] float32 (natural log).
 *   - Packed (varlen) layout, sequences s = 0..num_seqs-1 occupying token rows
 *     [cu_seqlens[s], cu_seqlens[s+1]):  Q, O, dO, dQ  [total, Hq, D];
 *     K, V, dK, dV  [total, Hkv, D];  LSE  [Hq, total] float32.  cu_seqlens
 *     is a DEVICE int32 array of num_seqs + 1 entries, cu_seqlens[0] = 0,
 *     non-decreasing, cu_seqlens[num_seqs] = total_tokens.  The mask is causal
 *     within each sequence; sequences never see each other.
 *   - D (head dim) is 64 or 128; Hq % Hkv == 0.
 *   - stream is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Calls are asynchronous on that stream; errors found on the host are
 *     returned before anything is launched; errors found on the device (a
 *     bounded wait that timed out, invalid cu_seqlens contents) are recorded
 *     in a per-device status word read by attn_get_device_status().
 *   - Ownership: the caller allocates every buffer; the library allocates no
 *     device memory and never frees caller memory.  Outputs are fully
 *     overwritten (no zero-initialisation needed).  Inputs are read-only.
 *   - Sizes of zero (B, T, num_seqs or total_tokens) are no-ops returning
 *     ATTN_OK.
 */
#ifndef GQA_ATTN_H_
#define GQA_ATTN_H_

#include <stddef.h>

#if defined(__GNUC__)
#define GQA_ATTN_API __attribute__((visibility("default")))
#else
#define GQA_ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_NULL = 1,       /* a required pointer is NULL */
    ATTN_ERR_SHAPE = 2,      /* negative size, Hq % Hkv != 0, Hq/Hkv < 1, size too large */
    ATTN_ERR_HEADDIM = 3,    /* D not 64 or 128 */
    ATTN_ERR_ALIGN = 4,      /* a pointer is not 16-byte aligned */
    ATTN_ERR_SEQLENS = 5,    /* cu_seqlens / cache_lens invalid (device-detected: status word) */
    ATTN_ERR_WORKSPACE = 6,  /* workspace NULL or smaller than the *_workspace_size() value */
    ATTN_ERR_ARCH = 7,       /* current device is not compute capability 10.3 */
    ATTN_ERR_CUDA = 8,       /* a CUDA runtime call failed (launch, tensor map, attribute) */
    ATTN_ERR_TIMEOUT = 9,    /* device-detected: a bounded in-kernel wait expired */
    ATTN_ERR_SCRATCH_LIMIT = 10, /* attn_bwd_noalloc: sizes need more than its built-in scratch */
    ATTN_ERR_PAGES = 11,     /* device-detected: a block-table entry names no page of the pool */
    ATTN_ERR_CHECK = 12,     /* device-detected, debug build only: a bounds check of a computed index failed */
    ATTN_ERR_RANGE = 13      /* device-detected: a rotated q or k value is not finite or does not fit f16 */
} attn_status;

/* Forward, dense layout.  Writes O (bf16) and LSE (float32). */
GQA_ATTN_API attn_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int Hq, int Hkv, int T, int D, int causal, float scale, void* stream);

/* Bytes of device workspace attn_bwd needs for these sizes (0 if invalid). */
GQA_ATTN_API size_t attn_bwd_workspace_size(int B, int Hq, int Hkv, int T, int D);

/* Backward, dense layout.  Reads Q, K, V, the forward's O and LSE, and dO;
 * writes dQ, dK, dV (bf16).  workspace: device memory of at least
 * attn_bwd_workspace_size() bytes, 256-byte aligned, owned by the caller; it
 * holds Delta and LSE*log2(e) per query row and the dQ kernel's tile counter,
 * and needs no initialisation (the call writes all of it first); two calls
 * in flight at once need two workspaces.  dK and dV come from a
 * key/value-stationary kernel, dQ from a persistent query-stationary one
 * that takes its tiles from that counter; each tile's gradient is summed in
 * a fixed order inside one CTA, so the results are bit-reproducible. */
GQA_ATTN_API attn_status attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                     const void* dout, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                     int B, int Hq, int Hkv, int T, int D, int causal, float scale, void* stream);

/* Backward, dense layout, without a caller-provided workspace and without
 * allocating anything.  (No counterpart in the pages: an operational
 * variant of attn_bwd.)  It is for callers that cannot hand the library
 * device memory or let it allocate: code running where allocation is not
 * allowed or not available -- e.g. a host framework that has reserved every
 * byte of the device for its own pool, a plugin that only ever receives the
 * tensors it must read and write, or a stream that is being captured into a
 * CUDA graph, during which cudaMalloc is not permitted.
 * The scratch is a static device array of attn_bwd_noalloc_scratch_bytes()
 * bytes (16 MiB: 8 bytes per query row, so up to 2^21 rows B*Hq*T, T rounded
 * up to 128) inside the library; every GPU that loads the library holds it
 * until the process exits.  Sizes whose attn_bwd_workspace_size() exceeds
 * it return ATTN_ERR_SCRATCH_LIMIT before anything is launched.  The first
 * call on a device looks up the array's device address (once per device,
 * with that device current), so make that first call before any stream
 * capture.  All calls share the one array and the kernels re-initialise
 * everything they read from it, but calls whose work overlaps on the GPU
 * (other streams, other host threads) race on it: serialise them.
 * The looked-up address (like the device status word's) stays cached for the
 * life of the process: after cudaDeviceReset() or anything else that
 * destroys the device's primary context, do not call this library on that
 * device again in the same process.
 * Otherwise identical to attn_bwd (same arguments minus the workspace, same
 * results bit for bit). */
GQA_ATTN_API attn_status attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                                          const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                          int B, int Hq, int Hkv, int T, int D, int causal, float scale,
                                          void* stream);

/* Size in bytes of attn_bwd_noalloc's built-in scratch array. */
GQA_ATTN_API size_t attn_bwd_noalloc_scratch_bytes(void);

/* Forward, packed variable-length layout.  max_seqlen must be >= every
 * sequence's length (it sizes the launch grid). */
GQA_ATTN_API attn_status attn_varlen_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                            const int* cu_seqlens, int num_seqs, int total_tokens, int max_seqlen,
                            int Hq, int Hkv, int D, int causal, float scale, void* stream);

GQA_ATTN_API size_t attn_varlen_bwd_workspace_size(int num_seqs, int total_tokens, int Hq, int Hkv, int D);

/* Forward with rotary queries and keys (RoPE of MultiHeadAttentionWithRoPE,
 * llm-from-scratch "Project Overview"; positions-aware RoPE of the
 * microLLM-rocm README, section "Why this project exists"): the dense layout
 * of attn_fwd; q and k of every row are rotated at their positions
 * 0..T-1 before the attention, with the rotary table of attn_decode_fwd
 * (rope_cos_sin: DEVICE float32 [rope_positions, D], 16-byte aligned,
 * rope_positions >= T; row p holds cos(p*theta_i) for i < D/2, then
 * sin(p*theta_i); feature i pairs with feature i + D/2).  The rotated q and
 * k are written as f16 (11 significant bits) into the workspace and the
 * score MMA takes them as f16; P V and everything else is as attn_fwd.
 * A rotated value that is not finite or has |value| >= 65520 (beyond f16;
 * it becomes infinite there) is recorded in the device status word as
 * ATTN_ERR_RANGE; the call still completes, and its outputs for the rows
 * that meet that value are then not meaningful.  The rotary backward
 * (attn_bwd_rope, attn_varlen_bwd_rope) reports the same way.
 * workspace: DEVICE, 256-byte aligned, >= attn_fwd_rope_workspace_size()
 * bytes (the two rotated copies), no initialisation; errors as attn_fwd,
 * plus ATTN_ERR_WORKSPACE. */
GQA_ATTN_API size_t attn_fwd_rope_workspace_size(int B, int Hq, int Hkv, int T, int D);
GQA_ATTN_API attn_status attn_fwd_rope(const void* q, const void* k, const void* v, void* o, float* lse,
                                       void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int T,
                                       int D, int causal, float scale, const float* rope_cos_sin,
                                       int rope_positions, void* stream);

/* attn_fwd_rope for the packed variable-length layout of attn_varlen_fwd:
 * every sequence's tokens are at positions 0..len-1 (the offset from
 * cu_seqlens[s]); rope_positions >= max_seqlen.  A cu_seqlens whose
 * positions fall outside the table is reported through the device status
 * word (ATTN_ERR_SEQLENS), as attn_varlen_fwd reports it.
 * workspace: DEVICE, 256-byte aligned, >= attn_varlen_fwd_rope_workspace_size()
 * bytes. */
GQA_ATTN_API size_t attn_varlen_fwd_rope_workspace_size(int total_tokens, int Hq, int Hkv, int D);
GQA_ATTN_API attn_status attn_varlen_fwd_rope(const void* q, const void* k, const void* v, void* o, float* lse,
                                              const int* cu_seqlens, int num_seqs, int total_tokens,
                                              int max_seqlen, int Hq, int Hkv, int D, int causal, float scale,
                                              const float* rope_cos_sin, int rope_positions, void* workspace,
                                              size_t workspace_bytes, void* stream);

/* Backward of attn_fwd_rope (rotary queries and keys; RoPE of
 * MultiHeadAttentionWithRoPE, llm-from-scratch "Project Overview";
 * positions-aware RoPE of the microLLM-rocm README, section "Why this project
 * exists"): the gradients of L = sum(dO * O) with respect to the UNROTATED
 * q and k (and v).  Arguments as attn_bwd, plus the rotary table of
 * attn_fwd_rope (rope_cos_sin DEVICE float32 [rope_positions, D], 16-byte
 * aligned, rope_positions >= T); o and lse are attn_fwd_rope's outputs.
 * The kernels rotate q and k at positions 0..T-1 into f16 copies (as the
 * forward does), run the backward with f16 Q/K operands and an f16 dS, and
 * take dQ and dK back through the rotation (x -> R^T x at each row's
 * position) before rounding them to bf16.
 * workspace: DEVICE, 256-byte aligned, >= attn_bwd_rope_workspace_size()
 * bytes (the rotated copies and attn_bwd's workspace), no initialisation. */
GQA_ATTN_API size_t attn_bwd_rope_workspace_size(int B, int Hq, int Hkv, int T, int D);
GQA_ATTN_API attn_status attn_bwd_rope(const void* q, const void* k, const void* v, const void* o,
                                       const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                       void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int T,
                                       int D, int causal, float scale, const float* rope_cos_sin,
                                       int rope_positions, void* stream);

/* attn_bwd_rope for the packed variable-length layout (attn_varlen_bwd's
 * arguments plus the table; positions 0..len-1 in every sequence,
 * rope_positions >= max_seqlen).  workspace >=
 * attn_varlen_bwd_rope_workspace_size() bytes. */
GQA_ATTN_API size_t attn_varlen_bwd_rope_workspace_size(int num_seqs, int total_tokens, int Hq, int Hkv, int D);
GQA_ATTN_API attn_status attn_varlen_bwd_rope(const void* q, const void* k, const void* v, const void* o,
                                              const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                              void* workspace, size_t workspace_bytes, const int* cu_seqlens,
                                              int num_seqs, int total_tokens, int max_seqlen, int Hq, int Hkv, int D,
                                              int causal, float scale, const float* rope_cos_sin,
                                              int rope_positions, void* stream);

/* Backward, packed variable-length layout (arguments as attn_bwd plus the
 * sequence description of attn_varlen_fwd). */
GQA_ATTN_API attn_status attn_varlen_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                            const void* dout, void* dq, void* dk, void* dv, void* workspace,
                            size_t workspace_bytes, const int* cu_seqlens, int num_seqs, int total_tokens,
                            int max_seqlen, int Hq, int Hkv, int D, int causal, float scale, void* stream);

/* Cached (decode) attention: the newest Tq positions of each batch row
 * attend to that row's KV cache -- the cached GQA / per-row-prefix cached
 * attention and KV-cache decode of the microLLM-rocm README (section "Why
 * this project exists"), with the forward's mathematics above restricted to
 * Tq query rows per sequence:
 *
 *   row b holds n_b = cache_lens[b] keys (the Tq new ones included); query
 *   t (0 <= t < Tq) of row b is position n_b - Tq + t and sees the keys
 *   j <= n_b - Tq + t of its own row (the causal mask aligned to the end of
 *   the cache); query head h reads K/V head h / (Hq / Hkv).
 *
 * Layouts (device pointers, 16-byte aligned, densely packed):
 *   q, o      bf16 [B, Hq, Tq, D]     (the new queries, the output)
 *   k_cache,
 *   v_cache   bf16 [B, Hkv, S, D]     (S = cache capacity; rows past n_b are
 *                                      never used and may hold anything)
 *   lse       float32 [B, Hq, Tq]     (natural log)
 *   cache_lens DEVICE int32 [B], Tq <= cache_lens[b] <= S.  A row outside
 *             that range is reported through the device status word
 *             (ATTN_ERR_SEQLENS) and its outputs are left unwritten.
 * workspace: attn_decode_workspace_size() bytes, 256-byte aligned, no
 * initialisation needed; the size is 0 (workspace may be NULL) when the
 * key range is not split.  Limits: Tq <= S; B*Hq*Tq < 2^31. */
GQA_ATTN_API size_t attn_decode_workspace_size(int B, int Hq, int Hkv, int Tq, int S, int D);

/* Rotary queries (positions-aware RoPE of the microLLM-rocm README, section
 * "Why this project exists"; RoPE / MultiHeadAttentionWithRoPE of the
 * llm-from-scratch "Project Overview"), for both decode entry points:
 * rope_cos_sin NULL = none; otherwise a DEVICE float32 table
 * [rope_positions, D], 16-byte aligned, rope_positions >= the cache capacity
 * (S, or max_pages * page_size): row p holds cos(p*theta_i) for i < D/2, then
 * sin(p*theta_i).  Each query t of row b is rotated at its position
 * p = cache_lens[b] - Tq + t before the scores: feature i pairs with feature
 * i + D/2, x'_i = x_i cos - x_{i+D/2} sin, x'_{i+D/2} = x_{i+D/2} cos + x_i sin,
 * computed in f32 and carried into the score MMA to about 2^-16 of each
 * element (a bf16 value plus a bf16 remainder; E4M3 caches: the three E4M3
 * parts below).  The cache must hold keys already rotated at their
 * positions (as appending them rotated leaves them). */
GQA_ATTN_API attn_status attn_decode_fwd(const void* q, const void* k_cache, const void* v_cache,
                                         const int* cache_lens, void* o, float* lse, void* workspace,
                                         size_t workspace_bytes, int B, int Hq, int Hkv, int Tq, int S, int D,
                                         float scale, const float* rope_cos_sin, int rope_positions, void* stream);

/* Cached attention over a PAGED KV cache (the paged KV-cache management of
 * the RoseLLM README, section "Inference and serving").  Same queries, mask
 * and outputs as attn_decode_fwd; the cache is a pool of pages:
 *   k_pages, v_pages  bf16 [num_pages, Hkv, page_size, D]: a page holds
 *                     page_size consecutive positions of one batch row,
 *                     every K/V head (each (page, head) block contiguous)
 *   block_table       DEVICE int32 [B, max_pages]: key position j of row b
 *                     is row j % page_size of page block_table[b*max_pages + j/page_size];
 *                     only the entries of pages that hold one of the row's
 *                     cache_lens[b] keys are read
 *   cache_lens        DEVICE int32 [B], Tq <= cache_lens[b] <= max_pages * page_size
 * page_size: 16, 32, 64 or a multiple of 128.  workspace: as attn_decode_fwd
 * with S = max_pages * page_size (attn_decode_workspace_size).  An entry
 * outside [0, num_pages) is reported through the device status word
 * (ATTN_ERR_PAGES) and the page is read as zeros (the row's result is then
 * meaningless, no memory outside the pool is touched). */
GQA_ATTN_API attn_status attn_decode_paged_fwd(const void* q, const void* k_pages, const void* v_pages,
                                               const int* block_table, const int* cache_lens, void* o, float* lse,
                                               void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                                               int Tq, int page_size, int num_pages, int max_pages, int D,
                                               float scale, const float* rope_cos_sin, int rope_positions,
                                               void* stream);

/* Cached attention over FP8 K/V caches (the FP8 E4M3 quantize/dequantize
 * and KV-cache decode of the microLLM-rocm README, section "Why this project
 * exists"): same queries, mask and outputs as attn_decode_fwd /
 * attn_decode_paged_fwd, with the caches stored as E4M3 codes (1 byte each:
 * sign, 4 exponent bits with bias 7, 3 mantissa bits, no infinities) and one
 * scale per cache: K = e4m3(k8) * k_scale, V = e4m3(v8) * v_scale.
 *   k8, v8           uint8 [B, Hkv, S, D]  (contiguous), or
 *   k8_pages, v8_pages uint8 [num_pages, Hkv, page_size, D]  (paged, as
 *                    attn_decode_paged_fwd)
 * The scores are taken on the K codes as stored: each query row q (after
 * rotation, if any) is split into three E4M3 parts with one f32 scale per
 * row, q = s (h0 + h1 + h2), s = max|q| / 448, which holds q to about 2^-12
 * of each element (2^-19 of the row's largest for elements below E4M3's
 * normal range); the products accumulate in f32.  V is widened exactly to
 * f16 and P is rounded to f16 for the P V product (f32 accumulation).  NaN
 * codes at visible keys give NaN where the definition does; codes past
 * cache_lens[b] are never used.  Workspace, rotary table and errors as
 * attn_decode_fwd. */
GQA_ATTN_API attn_status attn_decode_fp8_fwd(const void* q, const void* k8, const void* v8, float k_scale,
                                             float v_scale, const int* cache_lens, void* o, float* lse,
                                             void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Tq,
                                             int S, int D, float scale, const float* rope_cos_sin,
                                             int rope_positions, void* stream);

GQA_ATTN_API attn_status attn_decode_paged_fp8_fwd(const void* q, const void* k8_pages, const void* v8_pages,
                                                   float k_scale, float v_scale, const int* block_table,
                                                   const int* cache_lens, void* o, float* lse, void* workspace,
                                                   size_t workspace_bytes, int B, int Hq, int Hkv, int Tq,
                                                   int page_size, int num_pages, int max_pages, int D, float scale,
                                                   const float* rope_cos_sin, int rope_positions, void* stream);

/* ---------------------------------------------------------------------------
 * The KV cache of a serving step: where its tokens go (attn_cache_plan), rotary
 * positions (attn_rope*), writing keys and values (attn_cache_append*), and
 * attention over a cache held in 4 bits (attn_decode_q4_fwd and its paged
 * form).  These belong to the paged KV-cache management of the RoseLLM README
 * (section "Inference and serving") and the positions-aware RoPE and KV-cache
 * decode of the microLLM-rocm README (section "Why this project exists").
 *
 * Cache slots.  A cache is [num_pages, Hkv, page_size, ...]: slot
 * p * page_size + r is row r of page p, in every K/V head.  A contiguous
 * cache [B, Hkv, S, ...] is the case num_pages = B, page_size = S, where
 * position j of batch row b is slot b * S + j.
 *
 * Token views.  q, k and v here are [B, T, H, D] bf16 with strides of their
 * own: element (b, t, h, d) lies at b*s_b + t*s_t + h*s_h + d (strides in
 * elements, multiples of 8, none negative), so the views of one fused
 * projection's output and both layouts above ([B,H,T,D] and [total,H,D] as
 * B = 1, T = total) need no copy.  Strides are passed as HOST arrays of three
 * (s_b, s_t, s_h) per tensor, read before the call returns.  Token (b, t) is
 * number b*T + t of slots.  Outputs whose rows overlap give undefined values.
 *
 * Rotary positions.  rope_cos_sin is float32 [rope_positions, rotary_dim]
 * (DEVICE, 16-byte aligned), row p holding the rotary_dim/2 cosines, then the
 * sines.  The first rotary_dim features of each head are rotated (a multiple
 * of 16, <= D), the others kept: pair i is features (i, i + rotary_dim/2), or
 * with interleaved != 0 features (2i, 2i+1):
 *   y_first = x_first c - x_second s,   y_second = x_second c + x_first s.
 * positions: DEVICE int32.  A position outside the table is reported through
 * the device status word (ATTN_ERR_SEQLENS). */

/* Block table, slots and positions of a step's new tokens, from the request
 * lengths, in one launch (graph-capturable: nothing depends on the lengths on
 * the host).  Request b holds cache_lens[b] keys in the first
 * ceil(cache_lens[b] / page_size) entries of block_table row b and adds
 * new_lens[b] tokens.  It gets the pages it lacks from free_pages, in request
 * order from index cursor[0] on (NULL: 0), and they are written into its
 * block-table row (the only entries changed).  Written as well:
 *   slots, positions  [total_tokens]  of the new tokens, packed in request
 *                     order; entries past the last token are -1 and 0
 *   cu_seqlens        [B + 1]  each request's first packed token
 *   lens_out          [B]      cache_lens + new_lens
 *   cursor_out        [1]      index of the first page still free
 * (DEVICE int32; none of them may overlap an input or block_table.)
 * Tokens are packed: a request with new_lens[b] = 0 has no entry in slots and
 * positions.  Where k and v keep a row for every request, idle ones too (a
 * captured step of one token each), row b's slot is entry cu_seqlens[b] if
 * cu_seqlens[b + 1] > cu_seqlens[b], else -1; its position likewise.
 * Positions count the row's keys: cache_lens[b] and on.  They are those of the
 * text only where the row holds its whole text.  Behind a shared prefix of m keys
 * they are m further on, and in a row that was cut (attn_cache_evict) further by
 * the keys it lost: there the program keeps each row's next position and takes
 * the slots alone from here.
 * A request with a negative length, or whose new length exceeds
 * max_pages * page_size, is refused: it gets no pages, its tokens (none if
 * new_lens[b] < 0) get slot -1 and its length stays (ATTN_ERR_SEQLENS).  So
 * are the first request whose tokens exceed total_tokens (ATTN_ERR_SEQLENS;
 * cu_seqlens stops at total_tokens) or whose pages exceed free_pages
 * (ATTN_ERR_PAGES) and every valid one after it.  A negative page in
 * block_table or free_pages gives slot -1 (ATTN_ERR_PAGES).
 * 0 <= B <= 8192; page_size >= 1; B * max_pages and max_pages * page_size
 * below 2^31. */
GQA_ATTN_API attn_status attn_cache_plan(const int* cache_lens, const int* new_lens, int* block_table,
                                         const int* free_pages, const int* cursor, int* slots, int* positions,
                                         int* cu_seqlens, int* lens_out, int* cursor_out, int B, int page_size,
                                         int max_pages, int num_free, int total_tokens, void* stream);

/* Rotary table of positions 0..n-1 (rope_cos_sin float32 [n, rotary_dim], as
 * above), with frequencies theta_i = base^(-2i/rotary_dim) scaled for contexts
 * longer than the trained one:
 *   original_positions = 0: theta_i / factor (position interpolation; factor 1: none);
 *   otherwise by parts: with t_i = original_positions * theta_i / (2 pi) turns
 *   over the original context and g = clamp((t_i - low_turns) /
 *   (high_turns - low_turns), 0, 1), theta_i g + (theta_i / factor) (1 - g).
 * (The ramp is over turns.  Where a model's table was made with a ramp over the
 * pair index, between two bounds found from the turns and rounded to whole
 * pairs, this one differs for the pairs between the bounds: such a model needs
 * its own table, which every operator here takes.)
 * Cosines and sines are multiplied by mscale.  The angle of a position is
 * taken in fixed point (64 bits of a turn from a frequency in double), so that
 * far positions lose little; sine and cosine of what is left are f32
 * polynomials (within 2^-23), multiplied by mscale in f32: entries whose angle
 * is below 2^24 are within 2^-22 |mscale| of the exact ones (an f32 rounding
 * alone would be within 2^-25).  rotary_dim: a multiple of 16, at most
 * 512.  base > 1, factor > 0, low_turns < high_turns, all finite, and so are
 * 1 / factor and mscale in float32. */
GQA_ATTN_API attn_status attn_rope_table(float* rope_cos_sin, int n, int rotary_dim, double base, double factor,
                                         int original_positions, double low_turns, double high_turns, double mscale,
                                         void* stream);

/* Rotates q [B,T,Hq,D] and k [B,T,Hkv,D] (k, k_out NULL with Hkv = 0: q alone)
 * at positions[b * positions_stride + t] (positions_stride: T, or 0 for the
 * same positions in every batch row), in f32, rounded once to bf16.
 * strides: HOST, 12 entries: q, k, q_out, k_out, three each.  An output may be
 * its input (same pointer and strides).  A row whose position is outside the
 * table is written as zeros.  D: a multiple of 16, at most 512. */
GQA_ATTN_API attn_status attn_rope(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
                                   int positions_stride, const float* rope_cos_sin, int rope_positions, int B, int T,
                                   int Hq, int Hkv, int D, int rotary_dim, int interleaved, const long long* strides,
                                   void* stream);

/* Backward of attn_rope: the gradients of its inputs from those of its outputs
 * (the transposed rotation; with a table of mscale m, m^2 times the inverse's
 * input).  Arguments as attn_rope. */
GQA_ATTN_API attn_status attn_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk,
                                       const int* positions, int positions_stride, const float* rope_cos_sin,
                                       int rope_positions, int B, int T, int Hq, int Hkv, int D, int rotary_dim,
                                       int interleaved, const long long* strides, void* stream);

/* Writes k and v [B,T,Hkv,D] into the cache slots slots[b*T + t] (DEVICE
 * int32).  Slot -1 writes nothing (padded tokens); any other slot outside
 * [0, num_pages * page_size) is reported (ATTN_ERR_PAGES) and writes nothing.
 * The slots of one call must differ from one another: a slot named twice
 * holds a mixture of its tokens.  k and v must not overlap the caches.  rope_cos_sin (NULL: none) rotates k in f32
 * at positions[b*T + t] on the way; a token whose position is outside the
 * table is reported and not written.  strides: HOST, 6 entries: k, v.
 *   attn_cache_append      bf16 caches [num_pages, Hkv, page_size, D]
 *   attn_cache_append_fp8  E4M3 caches: code = e4m3(x * (1 / scale)), nearest
 *                          even, saturating at +-448 (infinities too), NaN
 *                          kept; 1 / scale rounded to f32
 *   attn_cache_append_q4   4-bit caches (below)
 * D: 64 or 128. */
GQA_ATTN_API attn_status attn_cache_append(const void* k, const void* v, const int* slots, const int* positions,
                                           const float* rope_cos_sin, int rope_positions, int rotary_dim,
                                           int interleaved, void* k_cache, void* v_cache, int B, int T, int Hkv,
                                           int D, int page_size, int num_pages, const long long* strides,
                                           void* stream);
GQA_ATTN_API attn_status attn_cache_append_fp8(const void* k, const void* v, const int* slots, const int* positions,
                                               const float* rope_cos_sin, int rope_positions, int rotary_dim,
                                               int interleaved, void* k8, void* v8, float k_scale, float v_scale,
                                               int B, int T, int Hkv, int D, int page_size, int num_pages,
                                               const long long* strides, void* stream);

/* The 4-bit cache format: E2M1 codes (sign, 2 exponent bits, 1 mantissa bit:
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one E4M3 scale for 16 consecutive features
 * and one f32 scale for the cache; 4.5 bits per element.
 *   k4, v4        uint8 [num_pages, Hkv, page_size, D/2]: features 2i (low
 *                 half) and 2i + 1 of a row in byte i
 *   k4_sf, v4_sf  uint8 [num_pages, Hkv, page_size, D/16]: E4M3 codes
 *   value = e2m1(code) * e4m3(sf) * k_scale (v_scale).
 * Appending takes, in f32 and rounded as elementary operations are,
 *   sf = e4m3(min(max_16 |x| * (1 / (6 scale)), 448)),
 *   code = e2m1(x * (1 / (e4m3(sf) * scale))), nearest even, saturating at 6;
 * a block with a NaN or an infinity stores the NaN scale and reads as NaN, one
 * whose sf rounds to 0 stores zeros.  Scales: 1e-20 <= scale <= 1e20. */
GQA_ATTN_API attn_status attn_cache_append_q4(const void* k, const void* v, const int* slots, const int* positions,
                                              const float* rope_cos_sin, int rope_positions, int rotary_dim,
                                              int interleaved, void* k4, void* k4_sf, void* v4, void* v4_sf,
                                              float k_scale, float v_scale, int B, int T, int Hkv, int D,
                                              int page_size, int num_pages, const long long* strides, void* stream);

/* Reads cache slots back as values: k, v bf16 [tokens, Hkv, D] (dense), the
 * 4-bit values above rounded to bf16 -- what a later prompt chunk or a shared
 * prefix attends to through attn_fwd.  Slot -1 (and, reported as
 * ATTN_ERR_PAGES, any other outside the cache) gives zeros. */
GQA_ATTN_API attn_status attn_cache_gather_q4(const int* slots, const void* k4, const void* k4_sf, const void* v4,
                                              const void* v4_sf, float k_scale, float v_scale, void* k, void* v,
                                              int tokens, int Hkv, int D, int page_size, int num_pages, void* stream);

/* Cached attention over 4-bit caches: the queries, mask, rotary table and
 * outputs of attn_decode_fwd over k4, k4_sf, v4, v4_sf [B, Hkv, S, ...] as
 * above.  Any 0 <= cache_lens[b] <= S is a valid length: a query at a
 * negative position (cache_lens[b] < Tq) sees no key and gets O = 0, LSE =
 * -infinity, so a batch slot without a request is a row of length 0.  A row
 * outside that range is reported (ATTN_ERR_SEQLENS), its outputs unwritten.
 * e2m1 * e4m3 is exact in f16; the query rows (after rotation in f32, if any)
 * are scaled by a power of two per row and carried in f16, value and remainder
 * when rotated.  A plain query's feature is exact down to 2^-31 of its row's
 * largest, and below that off by at most 2^-39 of it; a rotated one is off by
 * at most 2^-22 of itself and 2^-39 of the largest.  Else the scores' only
 * roundings are the f32 accumulation's.  P is rounded to f16 for the P V
 * product (f32 accumulation).  The quotient and the logarithm of a row whose
 * pieces met between CTAs are taken to 2 ulp of f32, those of other rows as the
 * language's functions give them.  How a row is cut into pieces follows from the sizes and the lengths: the same call
 * gives the same bits, another capacity may give other last bits.
 * workspace: attn_decode_q4_workspace_size() bytes, 256-byte aligned, no
 * initialisation; calls in flight at once need one each.  Errors as
 * attn_decode_fwd; the cache tensors must be 16-byte aligned.  S (paged:
 * max_pages * page_size) is at most 2^31 - 33; scale * k_scale * log2(e) is
 * finite in float32. */
GQA_ATTN_API size_t attn_decode_q4_workspace_size(int B, int Hq, int Hkv, int Tq, int S, int D);
GQA_ATTN_API attn_status attn_decode_q4_fwd(const void* q, const void* k4, const void* k4_sf, const void* v4,
                                            const void* v4_sf, float k_scale, float v_scale, const int* cache_lens,
                                            void* o, float* lse, void* workspace, size_t workspace_bytes, int B,
                                            int Hq, int Hkv, int Tq, int S, int D, float scale,
                                            const float* rope_cos_sin, int rope_positions, void* stream);

/* The same over paged 4-bit caches [num_pages, Hkv, page_size, ...] through a
 * block table (both as attn_decode_paged_fwd; a table entry outside the pool
 * is reported as ATTN_ERR_PAGES and its keys read as zeros). */
GQA_ATTN_API attn_status attn_decode_paged_q4_fwd(const void* q, const void* k4_pages, const void* k4_sf_pages,
                                                  const void* v4_pages, const void* v4_sf_pages, float k_scale,
                                                  float v_scale, const int* block_table, const int* cache_lens,
                                                  void* o, float* lse, void* workspace, size_t workspace_bytes, int B,
                                                  int Hq, int Hkv, int Tq, int page_size, int num_pages, int max_pages,
                                                  int D, float scale, const float* rope_cos_sin, int rope_positions,
                                                  void* stream);

/* ---------------------------------------------------------------------------
 * Attention of rows that share prefixes (the paged KV-cache management of the
 * RoseLLM README, section "Inference and serving"; per-row-prefix cached
 * attention of the microLLM-rocm README, section "Why this project exists"):
 * one system prompt or document behind a batch, or several samples of each
 * prompt.  The keys and values of a prefix are read once for all of its rows.
 *
 *   prefix p (0 <= p < P) belongs to the W = B / P rows p*W .. p*W + W - 1 and
 *   holds m_p = prefix_lens[p] keys; row b holds n_b = cache_lens[b] keys of its
 *   own behind them (the Tq new ones included).  Query t of row b has own
 *   position n_b - Tq + t; it sees every key of its prefix and the own keys up
 *   to that position.  A query at a negative own position (n_b < Tq; a batch
 *   slot without a request has n_b = 0) sees nothing: O = 0, LSE = -infinity.
 *
 *   q, o                  bf16 [B, Hq, Tq, D];  lse float32 [B, Hq, Tq]
 *   k_prefix, v_prefix    bf16 [P, Hkv, Sp, D]   (rows past m_p are not used)
 *   k_cache, v_cache      bf16 [B, Hkv, S, D]    (rows past n_b are not used)
 *   prefix_lens           DEVICE int32 [P], 0 <= m_p <= Sp
 *   cache_lens            DEVICE int32 [B], 0 <= n_b <= S
 * A length outside its range is reported (ATTN_ERR_SEQLENS); the outputs of the
 * rows it concerns are left unwritten.  B is a multiple of P; Tq <= S; Sp may
 * be 0 (k_prefix, v_prefix NULL).  Queries and keys are taken as they are: with
 * rotary positions, rotated before (attn_rope, attn_cache_append), an own key's
 * position following the prefix's.  P is rounded to bf16 for the P V product;
 * everything else is f32.  Rows of a cache that no query of a (row, K/V head)
 * sees may hold anything; a V that is infinite or NaN at an own position that
 * one of the Tq queries sees may make NaN of the others too.  A NaN score makes
 * NaN of O and LSE of the query that has it (LSE is -infinity only where a query
 * sees nothing, or scores of -infinity alone).  How a row's keys are cut into pieces follows from
 * the sizes and the lengths: the same call gives the same bits.
 * workspace: attn_decode_prefix_workspace_size() bytes, 256-byte aligned, no
 * initialisation; calls in flight at once need one each. */
GQA_ATTN_API size_t attn_decode_prefix_workspace_size(int B, int Hq, int Hkv, int Tq, int P, int Sp, int S, int D);
GQA_ATTN_API attn_status attn_decode_prefix_fwd(const void* q, const void* k_prefix, const void* v_prefix,
                                                const int* prefix_lens, const void* k_cache, const void* v_cache,
                                                const int* cache_lens, void* o, float* lse, void* workspace,
                                                size_t workspace_bytes, int B, int Hq, int Hkv, int Tq, int P, int Sp,
                                                int S, int D, float scale, void* stream);

/* The same over one pool of pages [num_pages, Hkv, page_size, D] (page sizes of
 * attn_decode_paged_fwd): key j of prefix p is row j % page_size of page
 * prefix_table[p*max_prefix_pages + j/page_size], own key j of row b that of
 * page block_table[b*max_pages + j/page_size]; own keys begin with a page of
 * their own wherever the prefix ends.  An entry outside [0, num_pages) is
 * reported (ATTN_ERR_PAGES) and its keys read as zeros.  workspace: as above
 * with Sp = max_prefix_pages * page_size, S = max_pages * page_size. */
GQA_ATTN_API attn_status attn_decode_paged_prefix_fwd(const void* q, const void* k_pages, const void* v_pages,
                                                      const int* prefix_table, const int* prefix_lens,
                                                      const int* block_table, const int* cache_lens, void* o, float* lse,
                                                      void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                                                      int Tq, int P, int page_size, int num_pages, int max_prefix_pages,
                                                      int max_pages, int D, float scale, void* stream);

/* Attention weight of cached keys (for evicting those that receive little; the
 * KV-cache management of the RoseLLM README, section "Inference and serving"):
 *   weights[j] += sum over the Hq/Hkv query heads of j's K/V head and the
 *   queries t that see j (j <= cache_lens[b] - Tq + t) of
 *   exp(scale q . k_j - lse)
 * where the entries of the row's last Tq positions, the step's new keys, are set
 * to the sum instead (whatever their slots held before), with q bf16
 * [B, Hq, Tq, D] and the lse float32 [B, Hq, Tq] that the step's
 * attention returned (-infinity, a query that saw no key: adds nothing; NaN:
 * makes NaN of what it sees).  Behind
 * a shared prefix that lse counts the prefix's keys too, and so do the weights.
 *   weights  float32 [num_pages, Hkv, page_size], an entry beside each key
 *            (slots as above); entries of positions past a row's length stay
 *   keys     bf16 [num_pages, Hkv, page_size, D], E4M3 codes of the same shape
 *            (key = e4m3 * k_scale), or 4-bit codes and block scales
 *   cache_lens DEVICE int32 [B], 0 <= cache_lens[b] <= the capacity: otherwise
 *            reported (ATTN_ERR_SEQLENS) and the row's weights stay
 *   block_table DEVICE int32 [B, max_pages], any page size; NULL: contiguous
 *            caches, num_pages = B, page_size = S, max_pages unused.  An entry
 *            outside the pool is reported (ATTN_ERR_PAGES), its keys skipped.
 * No two (row, position) of a call may be the same slot: an entry that two rows
 * name gets one of their sums.  Scores and sums are f32, in a fixed order; for
 * E4M3 and 4-bit keys the queries are carried in f16, scaled by a power of two a
 * row: exact down to 2^-31 of a row's largest feature, below that off by at
 * most 2^-39 of it. */
GQA_ATTN_API attn_status attn_cache_weights(const void* q, const void* k_cache, const float* lse, const int* block_table,
                                            const int* cache_lens, float* weights, int B, int Hq, int Hkv, int Tq,
                                            int page_size, int num_pages, int max_pages, int D, float scale,
                                            void* stream);
GQA_ATTN_API attn_status attn_cache_weights_fp8(const void* q, const void* k8, float k_scale, const float* lse,
                                                const int* block_table, const int* cache_lens, float* weights, int B,
                                                int Hq, int Hkv, int Tq, int page_size, int num_pages, int max_pages,
                                                int D, float scale, void* stream);
GQA_ATTN_API attn_status attn_cache_weights_q4(const void* q, const void* k4, const void* k4_sf, float k_scale,
                                               const float* lse, const int* block_table, const int* cache_lens,
                                               float* weights, int B, int Hq, int Hkv, int Tq, int page_size,
                                               int num_pages, int max_pages, int D, float scale, void* stream);

/* Eviction: each row of more than `budget` keys is cut down to `budget`, in
 * place, each K/V head by itself.  Positions below `first` and the last `recent`
 * ones stay; of the others those with the largest weights do (of equal weights
 * the lower position; -0 equals 0, a NaN counts as the largest).  The kept
 * rows of `weights` and of the num_planes <= 8 planes move to positions
 * 0 .. budget-1 in their order, bit for bit; the entries behind stay as they
 * were.  A row of at most `budget` keys is not touched.  (Keys that were
 * rotated keep their rotation, so a later token's rotary position is the one it
 * has in the text, not the row's new length, which is what attn_cache_plan gives:
 * the program keeps it.  A paged row needs only its first
 * ceil(budget / page_size) pages afterwards.)
 *   planes     HOST array of DEVICE pointers, plane i [num_pages, Hkv, page_size]
 *              rows of row_bytes[i] (HOST; a multiple of 4, at most 4096)
 *   weights    float32 [num_pages, Hkv, page_size]
 *   kept       DEVICE int32 [B, Hkv, budget]: the positions kept, ascending; of
 *              a shorter row all its positions, then -1
 *   lens_out   DEVICE int32 [B]: min(cache_lens[b], budget)
 *   block_table, cache_lens as attn_cache_weights; a row whose length is out of
 *              range is reported, left alone, its kept all -1 and its lens_out its
 *              cache_lens.  Positions in a page outside the pool are reported
 *              (ATTN_ERR_PAGES), count as the smallest weight and are not moved.
 * No two (row, position) may be the same slot; no output may overlap another
 * buffer of the call (ATTN_ERR_SHAPE).  first + recent <= budget, budget >= 1. */
GQA_ATTN_API attn_status attn_cache_evict(float* weights, void* const* planes, const int* row_bytes, int num_planes,
                                          const int* block_table, const int* cache_lens, int budget, int recent,
                                          int first, int* kept, int* lens_out, int B, int Hkv, int page_size,
                                          int num_pages, int max_pages, void* stream);

/* Static description of a status code. */
GQA_ATTN_API const char* attn_status_string(attn_status status);

/* Synchronises `stream`, then reads the current device's status word into
 * *out (ATTN_OK or the first device-detected error since it was last
 * cleared); clears it when clear != 0.  Returns ATTN_ERR_CUDA if the copy
 * fails (e.g. a sticky CUDA error), else ATTN_OK. */
GQA_ATTN_API attn_status attn_get_device_status(void* stream, int* out, int clear);

/* Debug build (libgqa_attn_debug.so, compiled with -DGQA_DEBUG; no
 * counterpart in the pages): the kernels check every computed tensor-map
 * coordinate, global row offset, workspace row and rotary-table row against
 * its bounds before the access; a failed check skips the access, records
 * ATTN_ERR_CHECK in the status word and its source line in a second word.
 * attn_get_check_line synchronises `stream` and reads (and clears when
 * clear != 0) that line: 0 when no check failed, always 0 in the release
 * build.  attn_is_debug_build returns 1 in the debug build, 0 otherwise. */
GQA_ATTN_API attn_status attn_get_check_line(void* stream, int* out, int clear);
GQA_ATTN_API int attn_is_debug_build(void);

/* Failure-path self-test (no counterpart in the pages).  Launches one small
 * kernel that waits, through the library's bounded in-kernel wait, on a
 * barrier that nothing ever completes, with a limit of limit_ms milliseconds
 * (1..5000).  The wait expires, ATTN_ERR_TIMEOUT is recorded in the device
 * status word and the kernel returns normally: the GPU is neither hung nor
 * faulted, and attn_get_device_status() then reports the timeout. */
GQA_ATTN_API attn_status attn_selftest_wait_timeout(int limit_ms, void* stream);

/* Failure-path test of the production kernels (no counterpart in the pages;
 * not thread-safe).  Arms one injected failure for the next launch of one
 * kernel: 1 the forward (attn_fwd and attn_fwd_rope), 2 the backward's dK/dV
 * kernel, 3 the backward's dQ kernel (attn_bwd and its variants); 0 disarms.
 * In that launch every bounded wait gives up after limit_ms (1..5000) instead
 * of the usual 2 s, and one CTA's TMA producer stops before the loads of
 * its second step (the forward's and the dK/dV kernel's first CTA; for the
 * persistent dQ kernel, the CTA that takes its first tile), so one of that
 * CTA's waits expires.  The kernel then
 * records ATTN_ERR_TIMEOUT in the device status word, its other roles see
 * the CTA's abort flag and stop, the issued copies and MMAs are drained,
 * TMEM is freed and the kernel returns: the GPU is neither hung nor faulted
 * and the next call runs normally.  The failing CTA's outputs are left
 * unwritten or partial; every other CTA completes.  The injection is
 * consumed by the launch that takes it. */
GQA_ATTN_API attn_status attn_test_inject_timeout(int kernel, int limit_ms);

/* Kernel timing (instrumentation; not thread-safe).  While enabled, every
 * kernel launch is bracketed by a CUDA event pair recorded on the caller's
 * stream.  attn_profile_read synchronises those events and returns, for one
 * kernel kind (0 forward, 1 backward preprocess, 2 backward dK/dV kernel,
 * 3 unused, 4 decode partial, 5 decode split merge, 6 backward dQ kernel,
 * 7 cache plan, 8 rotary rows, 9 rotary table, 10 cache append, 11 cache
 * gather, 12 shared prefix, 13 its merge, 14 attention weights of cached keys,
 * 15 eviction, 16 a shared prefix's own keys), the number of launches and their summed device
 * time in milliseconds since the last attn_profile_reset.  At most 65536
 * launches are recorded between resets.  Off by default. */
GQA_ATTN_API attn_status attn_profile_enable(int enable);
GQA_ATTN_API attn_status attn_profile_reset(void);
GQA_ATTN_API attn_status attn_profile_read(int kind, int* launches, double* total_ms);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ATTN_H_ */
