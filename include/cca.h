/*
 * libcca: CCA-Attention (Core Context Aware attention) on NVIDIA B200
 * (sm_100a), as a C ABI.
 *
 * The method is the one described in the write-up "ICML 2025 | 全局池化+局部
 * 保留，CCA-Attention为LLM长文本建模带来突破性进展" of the paper "Core Context
 * Aware Transformers for Long Context Language Modeling":
 *
 *  - globally-aware pooling (section 全局感知池化): the sequence is cut into
 *    non-overlapping groups of g tokens; the query of each group's last
 *    token scores the group's keys, softmax(q . k / sqrt(d)), and those
 *    weights average the group's keys and values into one core key/value;
 *  - locality-preserving module (section 局部保留模块): every token also sees
 *    the raw keys/values of a window of at least w preceding tokens, aligned
 *    to the group size;
 *  - global-local fusion (section 全局-局部模块可微融合): one softmax over the
 *    concatenation of the core and the raw keys;
 *  - KV-cache support for decoding (section 基于 Triton 的底层加速).
 *
 * Definitions used by every call (r = Hq / Hkv; query head hq reads
 * key/value head hq / r):
 *   m          = floor(T / g) complete groups; group j = tokens jg..jg+g-1
 *   ws(t)      = g * floor(max(t - w, 0) / g), start of t's local window
 *   query t attends to core keys/values of groups j < ws(t) / g and to raw
 *   keys/values ws(t)..t, all scaled by 1/sqrt(d), under one softmax.
 *   Grouped-query attention (r > 1): each key/value head gets one core
 *   key/value per group, weighted by the mean of its r query heads' softmax
 *   vectors.
 *
 * Data: Q, K, V and raw cache rows are bf16; core keys/values (Kc, Vc and
 * the cache's core slots) are fp16, whose 11 significant bits keep the
 * error of the pooled rows of large keys well inside the attention's error
 * budget.  All tensors are row-major and contiguous, layout [B, H, T, d]
 * ("head-major"); d is 64 or 128.  Arithmetic is fp32 (scores, softmax,
 * accumulation) with bf16 (raw keys) or fp16 (core keys) tensor-core
 * operands.  Because core rows and the query copy used against them are
 * fp16, input magnitudes must stay below 65504; larger values are clamped
 * and reported as CCA_ERR_RANGE by cca_device_status().
 *
 * Memory: every pointer is a device pointer owned by the caller and
 * borrowed for the call; the library allocates nothing.  Calls are
 * asynchronous on the given stream (the CUDA runtime's cudaStream_t; 0 is
 * the legacy default stream).  Outputs must not alias inputs.  Pointers
 * must be 16-byte aligned (the per-row length arrays: 8-byte).
 *
 * Errors: argument checks run on the host before any launch; a call that
 * fails them returns a nonzero status and writes nothing.  CCA_ERR_CUDA
 * reports a launch error.  Device-side waits are bounded: a wait that runs
 * out records a timeout in a device status word and the kernel returns
 * early; cca_device_status() reads and clears it (and the fp16 range and
 * per-row capacity flags).
 */
#ifndef CCA_H
#define CCA_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CCA_OK = 0,
    CCA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size or shape */
    CCA_ERR_UNSUPPORTED = 2, /* d not 64/128, g or w beyond the limits     */
    CCA_ERR_CAPACITY = 3,    /* cache has no room for the request          */
    CCA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed          */
    CCA_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out         */
    CCA_ERR_RANGE = 6,       /* a value beyond the fp16 range was clamped  */
    CCA_ERR_SCRATCH = 7,     /* request exceeds the library's fixed scratch */
    CCA_ERR_SEQLENS = 8,     /* packed sequence offsets that do not ascend
                                within the packed rows                      */
    CCA_ERR_PAGE = 9         /* a page table entry, row number or parent
                                outside the paged cache                     */
} cca_status;

/* Element type of an output that may be written in either precision. */
typedef enum { CCA_BF16 = 0, CCA_F32 = 1 } cca_dtype;

/* Largest group size the kernels accept. */
#define CCA_MAX_G 256

/*
 * Decode cache (section 基于 Triton 的底层加速 says the kernel supports a KV
 * cache; section 计算和存储效率对比 that it shrinks it).  It holds the core
 * key/value of every completed group and the newest raw tokens in a ring:
 *   k_core, v_core: fp16 [B, Hkv, core_cap, d]; slot j = group j
 *   k_tail, v_tail: bf16 [B, Hkv, tail_cap, d]; token p in slot p % tail_cap
 * tail_cap >= w + g keeps the whole local window of the newest token.
 * All batch rows share one length `len` (tokens appended so far), which the
 * host keeps in this struct.  The buffers belong to the caller.
 */
typedef struct {
    void *k_core, *v_core;
    void *k_tail, *v_tail;
    int B, Hq, Hkv, d, g, w;
    int64_t core_cap, tail_cap;
    int64_t len;
} cca_cache;

/*
 * Globally-aware pooling (section 全局感知池化).
 *   Q [B, Hq, T, d], K and V [B, Hkv, T, d]  (bf16, read)
 *   Kc, Vc [B, Hkv, m, d], m = floor(T / g)  (fp16, written)
 * For each (b, kv head h, group j) the scores of the group's last query
 * against the group's keys are soft-maxed (per query head, averaged over
 * the r query heads of h) and pool that group's keys and values.  A trailing
 * partial group is not pooled.  1 <= g <= CCA_MAX_G.
 */
cca_status cca_pool(const void *Q, const void *K, const void *V, void *Kc,
                    void *Vc, int B, int Hq, int Hkv, int64_t T, int d, int g,
                    cudaStream_t stream);

/*
 * Fused core + local attention for a whole sequence (sections 局部保留模块
 * and 全局-局部模块可微融合).
 *   Q [B, Hq, T, d], K, V [B, Hkv, T, d] (bf16), Kc, Vc [B, Hkv, m, d]
 *   (fp16, from cca_pool), O [B, Hq, T, d] written in o_dtype (bf16 or
 *   fp32), 32-byte aligned (CCA_ERR_INVALID_ARG otherwise).
 * O[t] = softmax over { q_t . Kc[j] / sqrt(d) : j < ws(t)/g } and
 * { q_t . K[i] / sqrt(d) : ws(t) <= i <= t } applied to [Vc ; V].
 * Runs on tcgen05 tensor cores with TMA-staged tiles.
 */
cca_status cca_attn_prefill(const void *Q, const void *K, const void *V,
                            const void *Kc, const void *Vc, void *O,
                            cca_dtype o_dtype, int B, int Hq, int Hkv,
                            int64_t T, int d, int g, int w,
                            cudaStream_t stream);

/*
 * Training: the forward attention of cca_attn_prefill that also writes
 * each row's log-sum-exp, lse [B, Hq, T] (fp32, device memory, log2 units:
 * lse[t] = log2 of the sum over t's keys of 2^(q_t . key * log2(e) /
 * sqrt(d))), which cca_attn_backward reads.  Other arguments, results and
 * errors as cca_attn_prefill.
 */
cca_status cca_attn_prefill_lse(const void *Q, const void *K, const void *V, const void *Kc,
                                const void *Vc, void *O, cca_dtype o_dtype, float *lse, int B,
                                int Hq, int Hkv, int64_t T, int d, int g, int w,
                                cudaStream_t stream);

/* Bytes of device workspace cca_attn_backward needs for these shapes
 * (0 for an invalid shape). */
size_t cca_attn_backward_workspace_bytes(int B, int Hq, int Hkv, int64_t T, int d, int g);

/*
 * Backward pass for training (the write-up's section 全局-局部模块可微融合
 * calls the global-local fusion differentiable, and its section 基于 Triton
 * 的底层加速 says the fused operator serves training): for an upstream
 * gradient dO of the attention output, the gradients of
 * L = sum(dO * O) with respect to Q, K and V, through the fused attention
 * (queries, raw window keys/values, pooled core keys/values) and through
 * the pooling (section 全局感知池化: each group's weights come from its last
 * query and its keys).
 *   Q, K, V, Kc, Vc as for cca_attn_prefill; O and lse from
 *   cca_attn_prefill_lse on the same inputs (O in o_dtype); dO [B, Hq, T, d]
 *   bf16.  dQ [B, Hq, T, d], dK, dV [B, Hkv, T, d]: fp32, written, each
 *   32-byte aligned (CCA_ERR_INVALID_ARG otherwise).
 *   workspace: cca_attn_backward_workspace_bytes bytes of device memory,
 *   256-byte aligned (fp16 copies of Q and dO, per-row sums, fp32 core
 *   gradients; the call clears what it accumulates).  r = Hq / Hkv <= 32.
 * Runs as four launches on `stream` (per-row sums; dQ on tcgen05 tensor
 * cores, persistent CTAs taking one 128-row query tile at a time; dK, dV on
 * tcgen05, persistent CTAs taking one 128-key tile at a time; the pooling's
 * chain rule, one warp per group).  Errors as
 * cca_attn_prefill; values beyond the fp16 range in Q or dO are clamped in
 * the core stream's copies and reported as CCA_ERR_RANGE.
 */
cca_status cca_attn_backward(const void *Q, const void *K, const void *V, const void *Kc,
                             const void *Vc, const void *O, cca_dtype o_dtype,
                             const float *lse, const void *dO, float *dQ, float *dK,
                             float *dV, int B, int Hq, int Hkv, int64_t T, int d, int g,
                             int w, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream);

/*
 * Fill a cache from a prefix of T tokens (Q, K, V as for cca_pool).  The
 * write-up's section 基于 Triton 的底层加速 gives the operator KV-cache
 * support for prefill and decode; section 计算和存储效率对比 measures the
 * cache's size against full attention.  This call pools every complete
 * group into its core slot (section 全局感知池化) and copies the last
 * min(T, tail_cap) raw tokens into their ring slots (the window of
 * section 局部保留模块); it sets c->len = T.
 * CCA_ERR_CAPACITY if floor((T - 1) / g) >= core_cap.  The cache's shape
 * fields (B, Hq, Hkv, d, g, w, core_cap, tail_cap) must be set.
 */
cca_status cca_cache_prefill(cca_cache *c, const void *Q, const void *K,
                             const void *V, int64_t T, cudaStream_t stream);

/*
 * Append one token t = c->len per batch row (KV-cache support, section
 * 基于 Triton 的底层加速; pooling of a completed group, section
 * 全局感知池化): q_t [B, Hq, d], k_t, v_t [B, Hkv, d] (bf16).  k_t, v_t
 * go to ring slot t % tail_cap; if the token completes group j = t / g
 * ((t + 1) % g == 0), that group is pooled from the ring with the token's
 * own queries (it is the group's last token) into core slot j.  On success c->len becomes t + 1.  CCA_ERR_CAPACITY (nothing
 * written) if t / g >= core_cap.
 */
cca_status cca_cache_append(cca_cache *c, const void *q_t, const void *k_t,
                            const void *v_t, cudaStream_t stream);

/* Bytes of device workspace cca_attn_decode needs for this cache (for its
 * current and any smaller length). */
size_t cca_decode_workspace_bytes(const cca_cache *c);

/*
 * Attention of the newest token t = c->len - 1 over the cache: core slots
 * j < ws(t)/g and ring slots of tokens ws(t)..t, one softmax (the fused
 * core + local attention of sections 局部保留模块 and 全局-局部模块可微融合,
 * for one query, from the cache of section 基于 Triton 的底层加速).
 *   q_t [B, Hq, d] (bf16), o_t [B, Hq, d] written in o_dtype.
 * Split over key ranges; partial results go to `workspace` (device memory
 * of at least cca_decode_workspace_bytes(c) bytes, 256-byte aligned, its
 * contents need no initialisation: the call clears the few counters it
 * uses with cudaMemsetAsync on `stream`).  The last block of each (batch,
 * kv head) to finish combines the partials, in the same kernel.
 */
cca_status cca_attn_decode(const cca_cache *c, const void *q_t, void *o_t,
                           cca_dtype o_dtype, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/*
 * One decode step in one launch: cca_cache_append of token t = c->len
 * followed by cca_attn_decode of that token, fused into a single kernel
 * (the write-up's section 基于 Triton 的底层加速 describes one
 * cache-friendly operator with native KV-cache support; sections
 * 全局感知池化, 局部保留模块 and 全局-局部模块可微融合 define what it
 * computes).  Arguments as for the two calls: q_t [B, Hq, d], k_t, v_t
 * [B, Hkv, d] (bf16), o_t [B, Hq, d] in o_dtype.  The results, and the
 * cache contents afterwards, equal those of the two separate calls.  On
 * success c->len becomes t + 1; CCA_ERR_CAPACITY (nothing launched) if
 * t / g >= core_cap.
 * Workspace: as for cca_attn_decode (cca_decode_workspace_bytes(c) bytes,
 * 256-byte aligned), but this call does not clear the completion counters
 * it keeps there: zero-fill a workspace once before its first use with a
 * cache (e.g. cudaMemsetAsync(ws, 0, bytes, stream)).  Every decode call of
 * this library (this one, cca_attn_decode, cca_attn_decode_rows) leaves the
 * counters at zero when it completes, so the workspace stays ready for the
 * next call on the same cache.  Calls sharing a workspace must not overlap
 * on the GPU.
 */
cca_status cca_decode_step(cca_cache *c, const void *q_t, const void *k_t, const void *v_t,
                           void *o_t, cca_dtype o_dtype, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/*
 * Per-row lengths in device memory (the same cache append and decode
 * attention as above, sections 基于 Triton 的底层加速, 全局感知池化,
 * 局部保留模块 and 全局-局部模块可微融合).  These two calls read each batch
 * row's length from `lens` (device memory, B entries of long long, 8-byte
 * aligned) instead of c->len, so rows may have different lengths and a
 * sequence of decode steps can be captured once in a CUDA graph and
 * replayed (nothing the host must know changes from step to step).
 * c->len is neither read nor written.  lens[b] must be the number of tokens
 * row b holds: as set when the row was filled (cca_cache_prefill of that
 * row) and advanced by cca_cache_append_rows.  The library cannot tell a
 * larger value from a real length: a row whose lens[b] runs ahead of what
 * was appended is decoded from stale ring and core slots, and only a length
 * beyond the cache's capacity is reported.
 *
 * cca_cache_append_rows: row b appends its token t = lens[b] exactly as
 * cca_cache_append does (ring slot t % tail_cap, pooling of group t / g when
 * the token completes it), then sets lens[b] = t + 1, all on the device.  A
 * row whose token would not fit (t / g >= core_cap) is left unchanged and
 * cca_device_status() reports CCA_ERR_CAPACITY.  Requires Hkv <= 32 (one
 * warp per key/value head in one block per row): CCA_ERR_UNSUPPORTED
 * otherwise.
 */
cca_status cca_cache_append_rows(const cca_cache *c, long long *lens, const void *q_t,
                                 const void *k_t, const void *v_t, cudaStream_t stream);

/*
 * cca_attn_decode_rows (sections 局部保留模块 and 全局-局部模块可微融合 for
 * one query per row): cca_attn_decode for token t_b = lens[b] - 1 of every
 * row b, each over its own core slots and ring window.  The workspace
 * is the same as cca_attn_decode's.  A row with lens[b] == 0 gets a zero
 * output; a row longer than the cache gets a zero output and
 * cca_device_status() reports CCA_ERR_CAPACITY.
 */
cca_status cca_attn_decode_rows(const cca_cache *c, const long long *lens, const void *q_t,
                                void *o_t, cca_dtype o_dtype, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/* Size of the library's fixed decode scratch (bytes): the largest
 * cca_decode_workspace_bytes() that cca_attn_decode_noalloc can serve. */
#define CCA_NOALLOC_SCRATCH_BYTES (4u << 20)

/*
 * cca_attn_decode without a caller-provided workspace.  The paper has no
 * counterpart: this is a service for callers that cannot allocate device
 * memory, such as runtimes that plan all device memory up front and forbid
 * other allocations, plug-in hosts that only pass input and output pointers,
 * or latency-critical loops that cannot afford cudaMalloc (which may
 * synchronise the device).  It computes exactly what cca_attn_decode
 * computes, with the split-K partials in a fixed array of
 * CCA_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it is loaded
 * on until the process exits; it allocates nothing.
 *   Returns CCA_ERR_SCRATCH (nothing launched) if the cache needs more
 *   workspace than that array; other errors as cca_attn_decode.
 *   The first call in each CUDA context (once per device for the runtime's
 *   primary contexts, and again after a context is re-created, e.g. after
 *   cudaDeviceReset) looks up the array's device address with that context
 *   current, so make it before any stream capture begins.
 *   All calls share the array: calls whose kernels may overlap on the GPU
 *   (e.g. on unordered streams) race.  Nothing in it needs clearing.
 */
cca_status cca_attn_decode_noalloc(const cca_cache *c, const void *q_t, void *o_t,
                                   cca_dtype o_dtype, cudaStream_t stream);

/*
 * The LCA variant (page "Latent-Condensed Transformer for Efficient Long
 * Context Modeling", section 2 方法论, 核心设计思想): a later method by the
 * authors of CCA that condenses each group differently and keeps the same
 * core + local attention.  Per group of g tokens and key/value head:
 *   - semantic condensation (语义凝聚): every query head's average query
 *     over the group's own g query rows scores the group's keys,
 *     q_bar . k / sqrt(d); softmax per query head, mean over the r query
 *     heads of the key/value head; the weights pool the value and the
 *     content part of the key (entries [0, d - d_rope));
 *   - positional anchoring (位置锚定): the positional part of the key (the
 *     last d_rope entries: the rotary key of latent attention) is not mixed
 *     but copied from the group's highest-weight token (the first one on a
 *     tie).
 * d_rope: 0 <= d_rope <= d, a multiple of 8 (CCA_ERR_INVALID_ARG
 * otherwise).  The condensed rows (fp16, range clamp as for cca_pool) feed
 * cca_attn_prefill and cca_attn_decode unchanged: the local window and the
 * single softmax over [core ; raw] (section 局部上下文保留 and 推理流程 of
 * that page) are CCA's.
 */

/* Condensation of every complete group: arguments, layout and errors as
 * cca_pool, plus d_rope.  Reads every query row (the group averages), not
 * only each group's last. */
cca_status cca_lca_pool(const void *Q, const void *K, const void *V, void *Kc, void *Vc, int B,
                        int Hq, int Hkv, int64_t T, int d, int g, int d_rope,
                        cudaStream_t stream);

/*
 * Decode cache for the LCA variant (推理流程 of that page: the cache keeps
 * the condensed rows and the newest w tokens, and condenses each group as
 * it completes).  q_sum [B, Hq, d] (fp32, device memory, 16-byte aligned,
 * caller-owned) holds per query head the sum of the query rows of the open
 * (incomplete) group: a completed group needs its average query, and a
 * query row is not kept once its token is appended.
 *
 * cca_lca_cache_prefill: as cca_cache_prefill, with cca_lca_pool's
 * condensation; sets q_sum to the sums of the trailing partial group's
 * query rows (zero if T is a multiple of g) and c->len = T.
 *
 * cca_lca_cache_append: as cca_cache_append for token t = c->len (ring slot
 * t % tail_cap); adds q_t to q_sum, or, if t completes group j = t / g,
 * condenses group j from the ring with average queries (q_sum + q_t) / g
 * into core slot j and zeroes q_sum.  c->len becomes t + 1.
 * CCA_ERR_CAPACITY (nothing written) if t / g >= core_cap.
 *
 * The same q_sum and d_rope must serve every call on one cache.  Decode
 * attention is cca_attn_decode on the same cache.
 */
cca_status cca_lca_cache_prefill(cca_cache *c, float *q_sum, const void *Q, const void *K,
                                 const void *V, int64_t T, int d_rope, cudaStream_t stream);
cca_status cca_lca_cache_append(cca_cache *c, float *q_sum, const void *q_t, const void *k_t,
                                const void *v_t, int d_rope, cudaStream_t stream);

/*
 * Packed prompts: S sequences of different lengths, one behind the other,
 * without padding (sections 全局感知池化, 局部保留模块 and
 * 全局-局部模块可微融合 for a whole sequence, each by itself).
 * cu [S + 1] (int32, device memory, 4-byte aligned): sequence s is rows
 * cu[s] .. cu[s + 1] - 1; 0 <= cu[0], ascending (equal neighbours are an
 * empty sequence), cu[S] <= total.  Offsets that break this make the calls
 * write nothing and are reported by cca_device_status (CCA_ERR_SEQLENS).
 * Rows that no sequence owns (before cu[0], behind cu[S]) are never read
 * into a result, whatever they hold, and their outputs stay as they were.
 * 1 <= S <= CCA_MAX_SEQS.
 *
 * A packed tensor is `heads` x `total` rows of d contiguous elements; row t
 * of head h starts head * h + row * t elements behind `data`.  Both memory
 * orders that occur are so described: [heads, total, d] and
 * [total, heads, d], with or without gaps.  data: 16-byte aligned; row and
 * head: at least d and multiples of 8 (the stride of an extent of 1 is not
 * read).  For outputs: 32-byte aligned, multiples of 16, and rows that do
 * not overlap.
 */
typedef struct {
    void *data;
    int64_t row, head; /* strides in elements */
} cca_rows;

#define CCA_MAX_SEQS 8192

/*
 * cca_pool for packed prompts: Q [Hq], K, V [Hkv] packed bf16 tensors.
 * Kc, Vc (fp16, written): contiguous [Hkv, total / g, d]; the core row of
 * group j of sequence s is row cu[s] / g + j (division rounding down), so
 * that sequences never share a row; rows that hold no group become zero.
 */
cca_status cca_pool_packed(const cca_rows *Q, const cca_rows *K, const cca_rows *V,
                           const int32_t *cu, void *Kc, void *Vc, int S, int Hq, int Hkv,
                           int64_t total, int d, int g, cudaStream_t stream);

/* Bytes of device workspace cca_attn_prefill_packed needs, for the order in
 * which it takes the sequences' query blocks (0 for up to 64 sequences with up
 * to 256 blocks, total / 256 + S, and for an invalid shape). */
size_t cca_packed_workspace_bytes(int S, int64_t total);

/*
 * cca_attn_prefill for packed prompts: O [Hq] (o_dtype) gets each
 * sequence's causal attention over its own core rows (Kc, Vc from
 * cca_pool_packed) and its own window.  w >= total is plain causal
 * attention: no core row is seen, Kc and Vc may be NULL.
 * workspace: cca_packed_workspace_bytes(S, total) bytes, 256-byte aligned
 * (may be NULL for 0); its contents need no initialisation.  Calls sharing a
 * workspace must not overlap on the GPU.
 * Sequences are isolated from one another whatever they hold.  Within one,
 * as in cca_attn_prefill, a value row that is not finite may reach the
 * outputs of earlier rows whose 128-key tile it lies in.
 */
cca_status cca_attn_prefill_packed(const cca_rows *Q, const cca_rows *K, const cca_rows *V,
                                   const void *Kc, const void *Vc, const int32_t *cu,
                                   const cca_rows *O, cca_dtype o_dtype, int S, int Hq, int Hkv,
                                   int64_t total, int d, int g, int w, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/*
 * Paged decode cache: the cache of section 基于 Triton 的底层加速 (core rows
 * of completed groups, raw rows of the window) for B rows of any lengths
 * that share their memory in pages.  A page holds `page` rows of every
 * key/value head; core rows and raw rows have a pool each, the same for
 * every layer of a model (page p of each layer's pool belongs to the same
 * tokens):
 *   k_core, v_core: fp16 [layers, core_pages, Hkv, page, d]
 *   k_raw, v_raw:   bf16 [layers, raw_pages, Hkv, page, d]
 * Row b holds lens[b] tokens (0: the row is free).  Its core row j is row
 * j % page of page core_table[b, j / page], its token p is row p % page of
 * page raw_table[b, p / page].  An entry is -1 where the row has no page:
 * behind its end, and in raw_table before the window of its newest token.
 * core_ref[p], raw_ref[p] count the entries that name page p; a page of
 * count 0 is free.  A full page may belong to several rows
 * (cca_paged_fork); the page a row writes next is its own.
 * page: a power of two, 16 .. 1024.  Hq / Hkv <= 16.  B <= 4096.
 * raw_cols * page <= 2^31 - 256.
 * core_cols and core_pages may both be 0: a cache of plain causal
 * attention, for w >= raw_cols * page (no window ever ends).
 * The buffers belong to the caller; lens is 8-byte, pools 16-byte aligned.
 * Rows of a page that hold no token, and free pages, may hold anything.
 * A new cache: tables filled with -1, counts and lens with 0.
 *
 * The calls below read lens and tables on the device: a sequence of them can
 * be captured in a CUDA graph.  Their workspace (cca_paged_workspace_bytes
 * bytes, 256-byte aligned) is zero-filled once before its first use with a
 * cache, and every call leaves it ready for the next; calls sharing a
 * workspace must not overlap on the GPU.
 */
typedef struct {
    void *k_core, *v_core, *k_raw, *v_raw;
    int32_t *core_table, *raw_table; /* [B, core_cols], [B, raw_cols] */
    int32_t *core_ref, *raw_ref;     /* [core_pages], [raw_pages] */
    long long *lens;                 /* [B] */
    int layers, B, Hq, Hkv, d, g, w, page;
    int core_cols, raw_cols, core_pages, raw_pages;
} cca_paged_cache;

size_t cca_paged_workspace_bytes(const cca_paged_cache *c);

/*
 * Room for more tokens: row b is lengthened by n_new[b] >= 0 tokens
 * (device memory, B entries; NULL: by n, every row that is not free), as
 * prompt or as the next token of a step, for all layers at once.  lens[b]
 * grows and the row gets the pages that the longer row needs: raw pages
 * for the window of its new last token and everything behind, core pages
 * for its complete groups.  The free pages of lowest number are taken, rows
 * in order, a row's columns in order; then the raw pages that lie wholly
 * before the new window are given back.  The new tokens' contents are
 * written by cca_paged_fill (the whole sequence) or cca_paged_step (the newest
 * token).  So a row that holds tokens and is given more than one, a further
 * prompt for instance, has to be filled again from its first token before
 * anything reads it: its pages' new rows hold anything until then, and no
 * call can tell.  (For that all its pages have to be its own, as after a
 * prompt and its steps.)  A row that does not fit (its
 * table's columns; or the pages that it and the rows before it need exceed
 * the free ones of a pool) keeps its length and pages and is reported by
 * cca_device_status (CCA_ERR_CAPACITY).
 */
cca_status cca_paged_reserve(const cca_paged_cache *c, const long long *n_new, long long n,
                             cudaStream_t stream);

/*
 * cca_paged_reserve for a loop of steps: also notes in the workspace which
 * rows it refused.  Such a row is held: cca_paged_step with the same
 * workspace leaves it as it is (zero output, nothing written), so that its
 * last token is not written over, until a later call gives it room.  A row
 * that is given nothing because it asked for nothing stays what it was.
 * cca_paged_fork with this workspace hands the note on with the row.  A
 * workspace that holds notes serves one cache only, until it is zero-filled
 * again.
 */
cca_status cca_paged_reserve_held(const cca_paged_cache *c, const long long *n_new, long long n,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Fill one layer's pages from packed prompts: sequence s becomes row
 * rows[s] (int32, device memory) of the cache, which cca_paged_reserve has
 * given the length of the sequence.  K, V: packed bf16 tensors [Hkv]; Kc,
 * Vc: their core rows from cca_pool_packed (NULL for a cache without core
 * pages).  Copied are the rows of the last token's window and the core rows
 * of all complete groups.  A sequence whose row is out of range, not of its
 * length, or named by a later sequence too is left out; so are token and
 * core rows whose page is missing or belongs to another row as well.  Both
 * are reported (CCA_ERR_PAGE).
 */
cca_status cca_paged_fill(const cca_paged_cache *c, int layer, const cca_rows *K,
                          const cca_rows *V, const void *Kc, const void *Vc, const int32_t *cu,
                          const int32_t *rows, int S, int64_t total, cudaStream_t stream);

/*
 * Attention of the newest token t = lens[b] - 1 of every row over one
 * layer of the cache: q_t [B, Hq, d] (bf16) -> o_t [B, Hq, d] (o_dtype).
 * A free row gets a zero output; so does a row longer than its table, which
 * is reported (CCA_ERR_CAPACITY).  The same call on the same cache gives the
 * same bits; how a row's keys are shared out among the SMs depends on the
 * whole batch, so in another batch its output may differ by roundings.  Keys whose page is missing are left out
 * and reported (CCA_ERR_PAGE).
 */
cca_status cca_attn_decode_paged(const cca_paged_cache *c, int layer, const void *q_t, void *o_t,
                                 cca_dtype o_dtype, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/*
 * One decode step of one layer in one launch: writes the newest token t =
 * lens[b] - 1 of every row (k_t, v_t [B, Hkv, d], for which
 * cca_paged_reserve has made room) to its page, pools the group it completes
 * into its core row, and computes cca_attn_decode_paged of it.  lens is not
 * changed, so that the layers of a model take their steps one after the
 * other.  A row that cca_paged_reserve_held refused is left as it is and gets
 * a zero output.  (After cca_paged_reserve, which leaves no note, a row
 * without new room still ends in the token before, and its step writes that
 * one again.)  A token or core row whose page
 * is missing or belongs to another row as well is not written, and is
 * reported (CCA_ERR_PAGE).
 */
cca_status cca_paged_step(const cca_paged_cache *c, int layer, const void *q_t, const void *k_t,
                          const void *v_t, void *o_t, cca_dtype o_dtype, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/*
 * Rows take over other rows: afterwards row b holds what row parent[b]
 * (int32, device memory, B entries) held before the call; parent[b] = b
 * keeps a row, -1 frees it.  One call so forks a prompt into several samples,
 * reorders the beams of a search and frees finished rows, for all layers.
 * Full pages are shared; a partly filled last page (raw or core) stays with
 * the parent itself if it keeps its row, else with the lowest row that
 * takes it over, and the others get a copy in the free page of lowest number
 * (rows in order, pages freed by this call included).  A row for
 * whose copies no page is left is freed and reported (CCA_ERR_CAPACITY).  A
 * parent out of range keeps its row and is reported (CCA_ERR_PAGE).
 * Called between steps: the tokens that rows hold have been written, and
 * those of the next step are reserved afterwards (a page that a reserved
 * token fills up would be shared, and not be written).
 */
cca_status cca_paged_fork(const cca_paged_cache *c, const int32_t *parent, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/*
 * Compact the pools: the pages in use of the highest numbers move, for all
 * layers, to the free ones of the lowest numbers (both in ascending order),
 * until the pages in use are 0 .. live - 1; tables and counts follow.
 * live [2] (device memory, 8-byte aligned, written): pages in use of the
 * core and of the raw pool, to which the pools can be cut.
 */
cca_status cca_paged_compact(const cca_paged_cache *c, long long *live, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/*
 * Synchronise `stream`, then report CCA_ERR_CUDA if a CUDA error is
 * pending, CCA_ERR_TIMEOUT if any kernel of this library recorded a
 * timed-out wait since the last call, CCA_ERR_CAPACITY if a per-row call
 * met a row longer than its cache or a paged cache had no page for a row,
 * CCA_ERR_PAGE or CCA_ERR_SEQLENS if a call met such data in device memory,
 * CCA_ERR_RANGE if one clamped a value to the fp16 range, else CCA_OK.  The
 * records are cleared.
 */
cca_status cca_device_status(cudaStream_t stream);

/*
 * Failure-path self-test: launch on `stream` one small kernel that waits,
 * with the library's bounded wait and a limit of `limit_us` microseconds
 * (1 .. 2000000), on a barrier that nothing completes.  The wait runs out
 * and the kernel records a timeout, so a later cca_device_status(stream)
 * returns CCA_ERR_TIMEOUT, and the context stays usable (no fault, trap or
 * hang).  The pages define no such step; it lets callers and tests check
 * how the library reports a stuck kernel.  CCA_ERR_INVALID_ARG for a limit
 * outside the range (nothing launched), CCA_ERR_CUDA on a launch error.
 */
cca_status cca_selftest_wait_timeout(unsigned int limit_us, cudaStream_t stream);

/* Human-readable name of a status. */
const char *cca_status_string(cca_status s);

/* Library version, "major.minor.patch". */
const char *cca_version(void);

/* Text of the CUDA error behind the calling thread's last CCA_ERR_CUDA
 * ("no error" if there was none).  The string is static. */
const char *cca_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* CCA_H */
