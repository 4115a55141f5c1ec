/*
 * na.h -- C ABI of the GB300 (sm_103a) library for RoPE-rotated causal
 * grouped-query attention over a per-sequence KV cache.
 *
 * The operation comes from two docs.rs source pages:
 *   [cortiq]  cortiq-engine 0.5.39 src/attention.rs
 *   [needle]  needle-core 0.3.1 src/v2/batch.rs
 *
 * Conventions shared by every entry point
 *   - bf16 means IEEE bfloat16 stored as 16-bit words, little-endian.
 *   - Token-packed tensors hold the new tokens of all sequences back to back
 *     (varlen packing): token t belongs to sequence b when
 *     cu_seqlens[b] <= t < cu_seqlens[b+1].
 *   - The KV cache is head-major, one slot per absolute position:
 *     k[b][kv_head][slot][head_dim] (same for v), slot = position
 *     (position % capacity with NA_RING_CACHE).
 *   - Every pointer argument is DEVICE memory unless its comment says HOST.
 *     Configuration structs are HOST memory and are read only during the call.
 *   - Ownership: the caller allocates and frees every buffer (including the
 *     workspace).  The library allocates no device memory, never synchronises
 *     the host with the device, and enqueues all work on `stream`
 *     (a cudaStream_t; NULL is the legacy default stream).
 *   - Threads: calls may come from several host threads at once, each with its
 *     own buffers, workspace and stream (na_attn_decode_static_ws excepted: its
 *     calls share one scratch array).  Work goes to the calling thread's current
 *     device, whose primary context the library makes current on that thread.
 *   - Errors: a negative na_status is returned when host-side validation fails;
 *     nothing is enqueued in that case.  Conditions only the device can see
 *     (a position past the cache capacity, an internal wait that timed out) are
 *     reported by writing a nonzero na_status value into *status (a device
 *     int32, may be NULL to skip reporting); the affected tile is skipped and the
 *     kernel returns normally.  The library never clears *status: the caller
 *     zeroes it and reads it when convenient.
 *   - Alignment: q, k, v, q_out, gate, out and the cache base pointers must be
 *     16-byte aligned, contiguous, with head_dim a multiple of 8.
 */
#ifndef NA_H
#define NA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum na_status {
    NA_OK = 0,
    NA_ERR_INVALID_ARG = -1,   /* null pointer, bad size, num_heads % num_kv_heads != 0, ... */
    NA_ERR_UNSUPPORTED = -2,   /* a shape or option this build does not implement */
    NA_ERR_CAPACITY = -3,      /* a position does not fit the cache / probability stride */
    NA_ERR_WORKSPACE = -4,     /* workspace missing or smaller than required */
    NA_ERR_CUDA = -5,          /* a CUDA runtime call (launch, attribute) failed */
    NA_ERR_DEVICE_TIMEOUT = -6, /* device only: a bounded wait inside a kernel gave up */
    NA_ERR_PAGE = -7           /* device only: a page index outside the paged cache */
} na_status;

/* Option flags (na_attn_cfg.flags). */
#define NA_QK_NORM 1u                 /* per-head RMSNorm of q and k before RoPE [cortiq fn rmsnorm_head] */
#define NA_QK_NORM_ZERO_CENTERED 2u   /* with NA_QK_NORM: multiply by (1 + w) instead of w */
#define NA_V_NORM 4u                  /* scale-less RMS of v before it enters the cache [cortiq fn vnorm_head] */
#define NA_OUT_GATE 8u                /* out *= sigmoid(gate) after attention [cortiq fn apply_gate] */
#define NA_RING_CACHE 16u             /* the cache is a ring: position pos lives in slot pos % capacity
                                         (needle-core batch.rs, the per-position write-and-attend loop:
                                         a ring of kv_window positions).  Needs window > 0.  The pages'
                                         ring holds exactly the window, so writes and attends must
                                         alternate; here the ring holds at least window + (new tokens
                                         per sequence) - 1 positions, so a whole chunk is written first
                                         without overwriting a key any of its rows still reads.
                                         Prefill needs capacity % 128 == 0 and capacity >= window +
                                         max_new_len - 1; decode needs capacity >= window and
                                         capacity % 64 == 0 (NA_ERR_UNSUPPORTED otherwise). */

/* One attention layer [cortiq struct QwenAttnCfg, the in-scope fields]. */
typedef struct na_attn_cfg {
    int32_t num_heads;     /* H query heads */
    int32_t num_kv_heads;  /* KV heads; H % KV == 0; query head h reads kv head h / (H / KV) */
    int32_t head_dim;      /* d: 64 or 128 */
    int32_t rotary_dim;    /* rd: even, 0 <= rd <= d; RoPE turns dims [0, rd) only */
    float sm_scale;        /* score scale; <= 0 selects 1 / sqrt(head_dim) */
    float rms_eps;         /* epsilon of the qk-norm and v-norm */
    uint32_t flags;        /* NA_* option bits */
    float softcap;         /* > 0: each scaled score s becomes softcap * tanh(s / softcap)
                              ahead of the softmax (cortiq QwenAttnCfg.softcap, the Gemma-2
                              soft cap on attention logits); 0: off */
    int32_t window;        /* > 0: a query at pos attends only keys pos - window + 1 .. pos
                              (cortiq QwenAttnCfg.window, sliding window); 0: full context */
} na_attn_cfg;

/* RoPE frequencies [cortiq fns rope_inv_freq, yarn_inv_freq, rope_rotate_scaled]. */
typedef struct na_rope_params {
    double base;          /* inv_freq[i] = base^(-2 i / rd) */
    int32_t yarn;         /* 0: plain RoPE; 1: YaRN ramp between extrapolation and interpolation */
    double factor;        /* YaRN context extension factor (> 0) */
    int32_t orig_max_pos; /* YaRN original_max_position_embeddings (> 0 when yarn) */
    double beta_fast;     /* YaRN ramp bounds in rotations */
    double beta_slow;
    double attn_factor;   /* multiplier on cos and sin; <= 0 selects 1 without YaRN and
                             0.1 ln(factor) + 1 with YaRN */
} na_rope_params;

/* Caller-owned per-sequence cache: k, v bf16 [batch][num_kv_heads][capacity][head_dim]. */
typedef struct na_kv_cache {
    void *k;
    void *v;
    int32_t batch;
    int32_t capacity;
} na_kv_cache;

/* Element type of a paged cache (na_paged_kv_cache.dtype). */
#define NA_KV_BF16 0
#define NA_KV_E4M3 1 /* 8-bit floating point (4 exponent, 3 fraction bits, largest 448) with one
                        scale per (page, kv head): a stored byte b stands for b * 2^(s - 127),
                        s the E8M0 scale byte (0 .. 254).  The attention calls take V's scales
                        down to 2^-40 exactly (values of smaller ones are rounded to multiples of
                        2^-64) and report one above 2^47 as NA_ERR_UNSUPPORTED. */

/*
 * Caller-owned paged cache: a pool of pages and a page table.  Position pos of
 * sequence b lives in slot pos % page_size of page
 * page_table[b * pages_per_seq + pos / page_size].
 * (An addition of this library; the pages have no counterpart.)
 *
 *   - Pages that hold no position that the call reads or writes may have any
 *     table entry (past a sequence's end, before a sliding window).  Any other
 *     entry outside [0, num_pages) is reported as NA_ERR_PAGE: an append skips
 *     its tokens, an attention call's outputs of that sequence are unspecified.
 *   - Sequences may share pages that they only read (a common prompt).  Pages
 *     that a call appends to belong to one sequence.
 *   - Slots that hold no position of the sequence may hold any bits.  Queries and
 *     the keys and values of the sequence have to be finite: a NaN or infinity of
 *     V reaches every query row of its tile, masked or not.
 *   - Sizes: page_size 16, 32, 64 or 128; num_pages * kv heads * page_size
 *     <= 2^31 - 1 (NA_ERR_UNSUPPORTED otherwise).  The capacity of a sequence is
 *     pages_per_seq * page_size.  NA_RING_CACHE is NA_ERR_UNSUPPORTED: a window
 *     needs no ring here, its past pages can be given away.
 */
typedef struct na_paged_kv_cache {
    void *k;                   /* [num_pages][num_kv_heads][page_size][head_dim], 16-byte aligned */
    void *v;
    uint8_t *k_scale;          /* NA_KV_E4M3: [num_pages][num_kv_heads] E8M0 bytes, else ignored */
    uint8_t *v_scale;
    const int32_t *page_table; /* int32 [batch][pages_per_seq] */
    int32_t num_pages;
    int32_t page_size;
    int32_t batch;
    int32_t pages_per_seq;
    int32_t dtype;             /* NA_KV_BF16 or NA_KV_E4M3 */
} na_paged_kv_cache;

/*
 * Fused qk-norm + RoPE + cache append for a chunk of new tokens.
 * [cortiq fn finish_projection (norms before RoPE, partial rotary) and
 *  fn rope_rotate_scaled; needle module doc "What has to stay sequential":
 *  the chunk's K/V are written before any of its positions attends.]
 *
 * For new token t of sequence b, pos = cache_lens[b] + (t - cu_seqlens[b]):
 *   q_out[t][h]            = RoPE(norm_q(q[t][h]), pos)         for every h
 *   cache.k[b][g][pos]     = RoPE(norm_k(k[t][g]), pos)         for every g
 *   cache.v[b][g][pos]     = vnorm(v[t][g])  (or v unchanged)
 * (slot pos % capacity instead of pos with NA_RING_CACHE).
 * RoPE turns pairs (x[i], x[i + rd/2]), i < rd/2, by pos * inv_freq[i] and
 * multiplies both outputs by the attention factor.
 * Accuracy: each stored rotated or normed value is within one bf16 ulp of the
 * exact result: the correctly rounded value unless the exact one lies within
 * ~2^-23 (relative) of a bf16 rounding boundary (about 7 values in a million);
 * V without V-norm is stored bit for bit.
 *
 *   cfg, rope     HOST structs.
 *   batch         number of sequences (>= 1, <= cache->batch).
 *   cu_seqlens    int32 [batch + 1], non-decreasing, cu_seqlens[0] == 0.
 *   cache_lens    int32 [batch]: tokens already cached (prior length).
 *   total_tokens  HOST copy of cu_seqlens[batch]; 0 is a no-op returning NA_OK.
 *   q             bf16 [total_tokens][H][d];  k, v bf16 [total_tokens][KV][d].
 *   q_norm_w, k_norm_w  bf16 [d] (shared by all heads), 16-byte aligned, required with
 *              NA_QK_NORM, else ignored.
 *   q_out         bf16 [total_tokens][H][d]: rotated queries (may not alias q).
 *   status        device int32 or NULL; a token whose pos >= capacity is skipped and
 *                 NA_ERR_CAPACITY is written.
 * The caller advances cache_lens afterwards.
 */
int na_rope_append_kv(const na_attn_cfg *cfg, const na_rope_params *rope, int32_t batch,
                      const int32_t *cu_seqlens, const int32_t *cache_lens,
                      int32_t total_tokens, const void *q, const void *k, const void *v,
                      const void *q_norm_w, const void *k_norm_w, void *q_out,
                      const na_kv_cache *cache, int32_t *status, void *stream);

/*
 * Causal GQA attention of a chunk of new tokens against the cache.
 * [cortiq fn qwen_attention_batch, portable batched attend: query bi of the
 *  chunk sees keys 0 .. s0 + bi; fn attention_head: softmax(q.k * scale) . V;
 *  fn apply_gate; needle fn batch_attention.]
 *
 * The chunk's keys must already be in the cache (na_rope_append_kv first).
 * New token t of sequence b at pos = cache_lens[b] + (t - cu_seqlens[b]) and
 * query head h attends keys 0 .. pos of kv head h / (H / KV):
 *   out[t][h] = sum_j softmax_j(scale * q_rot[t][h] . k_j) v_j   (* sigmoid(gate[t][h]))
 * With cfg->window > 0 only keys pos - window + 1 .. pos are attended; with
 * cfg->softcap > 0 each scaled score is capped before the softmax.  Chunks of a
 * few tokens per sequence (the drafted tokens of a speculative verify) are
 * valid chunks: each attends the cache plus its own earlier tokens.
 * Arithmetic: Q.K and P.V on bf16 tensor cores with fp32 accumulation, the
 * softmax in fp32 with P rounded to bf16 for the P.V product; with unit-scale
 * inputs the output is within 2e-2 (max-abs) and 5e-3 (relative L2) of the
 * exact result.
 *
 *   cu_seqlens    int32 [batch + 1], non-decreasing, cu_seqlens[0] == 0.
 *   cache_lens    int32 [batch]: prior lengths (the same values given to na_rope_append_kv).
 *   total_tokens  HOST copy of cu_seqlens[batch]; 0 is a no-op returning NA_OK.
 *   max_new_len   HOST upper bound of cu_seqlens[b+1] - cu_seqlens[b].
 *   max_total_len HOST upper bound of cache_lens[b] + new length; <= capacity unless
 *                 NA_RING_CACHE (then positions wrap; see that flag for its capacity rules).
 *   q_rot         bf16 [total_tokens][H][d] (q_out of na_rope_append_kv).
 *   gate          bf16 [total_tokens][H][d], required with NA_OUT_GATE, else ignored.
 *   out           bf16 [total_tokens][H][d].
 *   workspace     device scratch of at least na_prefill_workspace_size() bytes
 *                 (NULL allowed when that size is 0).
 *   status        device int32 or NULL: NA_ERR_INVALID_ARG when a new length exceeds
 *                 max_new_len or cu_seqlens[0] != 0, NA_ERR_CAPACITY when a position
 *                 reaches max_total_len or the capacity (those rows are not written).
 * Errors (before anything is enqueued): NA_ERR_INVALID_ARG for null or misaligned
 * buffers and negative sizes, NA_ERR_UNSUPPORTED for a ring whose capacity is not
 * a multiple of 128, a cache of more than 2^31 - 1 rows (batch x kv heads x
 * capacity) or bounds so loose that the tiles of query rows (batch x heads x
 * max_new_len / rows of a tile) do not fit a grid, NA_ERR_CAPACITY when the ring
 * cannot hold a window plus a chunk, NA_ERR_WORKSPACE for a missing or short
 * workspace.
 */
int na_attn_prefill_chunk(const na_attn_cfg *cfg, int32_t batch, const int32_t *cu_seqlens,
                          const int32_t *cache_lens, int32_t total_tokens, int32_t max_new_len,
                          int32_t max_total_len, const void *q_rot, const na_kv_cache *cache,
                          const void *gate, void *out, void *workspace, size_t ws_bytes,
                          int32_t *status, void *stream);

/*
 * Single-token decode with optional per-key probabilities.
 * [cortiq fn attention_head (returns the per-key probabilities that feed
 *  eviction scoring), fns qwen_attention_core and attend_all_heads: the current
 *  token is appended first, then each group's K/V are streamed once for all its
 *  query heads.]
 * Arithmetic: bf16 MMAs with fp32 accumulation, softmax and probabilities in
 * fp32; with unit-scale inputs the output is within 2e-2 (max-abs) of the exact
 * result and each probability within 1e-4 (measured ~1.5e-6 of its own value).
 *
 *   q_rot      bf16 [batch][H][d], already rotated (one query per sequence).
 *   kv_lens    int32 [batch]: keys to attend, current token included (0 gives a zero
 *              output and writes no probabilities).
 *   max_kv_len HOST upper bound of kv_lens; <= capacity and <= probs_stride.
 *   gate       bf16 [batch][H][d] with NA_OUT_GATE, else ignored.
 *   out        bf16 [batch][H][d].
 *   probs      fp32 [batch][H][probs_stride] or NULL: probs[b][h][j] = p_j for
 *              j < kv_lens[b]; entries past kv_lens[b] are not written.
 *   num_splits granularity of the key split (0 = automatic).  The keys of all
 *              sequences are cut into one equal slice per CTA of the split pass
 *              (two CTAs per SM); num_splits > 0 makes every slice at least
 *              ceil(max_kv_len / num_splits) keys long, so the longest sequence
 *              is merged from at most num_splits + 1 partial results.
 *   workspace  at least na_decode_workspace_size() bytes: partial results of
 *              every slice piece plus 8 bytes per (sequence, kv head, head
 *              chunk); its size depends on the batch and the head layout, not on
 *              the lengths.  Not read before the call writes it (any contents
 *              will do, also after a call that timed out).
 *   status     device int32 or NULL: NA_ERR_CAPACITY for a length past the
 *              capacity or max_kv_len (zero output), NA_ERR_DEVICE_TIMEOUT when
 *              a wait of the split pass gave up (the affected heads get a zero
 *              output and no probabilities).
 * Errors (before anything is enqueued): NA_ERR_INVALID_ARG for null or
 * misaligned buffers, NA_ERR_CAPACITY when max_kv_len (or, with a ring, the
 * window) exceeds the capacity or a stride, NA_ERR_UNSUPPORTED for a ring whose
 * capacity is not a multiple of 64 (keys are read in aligned 64-key tiles) or a
 * cache of more than 2^31 - 1 rows (batch x kv heads x capacity: the tensor-map
 * row coordinate is 32-bit), NA_ERR_WORKSPACE for a missing or short workspace.
 */
int na_attn_decode(const na_attn_cfg *cfg, int32_t batch, const void *q_rot,
                   const na_kv_cache *cache, const int32_t *kv_lens, int32_t max_kv_len,
                   const void *gate, void *out, float *probs, int32_t probs_stride,
                   int32_t num_splits, void *workspace, size_t ws_bytes, int32_t *status,
                   void *stream);

/*
 * na_attn_decode for callers that cannot supply a workspace.
 * (An addition of this library; the pages have no counterpart.)
 *
 * Some callers have no way to allocate device memory for the workspace: a
 * plugin inside another runtime that owns all device memory and exposes no
 * allocator, or a serving loop that may not allocate once it is running.  This
 * entry point takes the same arguments as na_attn_decode minus the workspace
 * and keeps the split partials in a fixed 20 MiB device array inside the
 * library, so the call allocates nothing.  That array exists on every GPU that
 * loads the library, for as long as the library stays loaded.
 *
 *   - Sizes whose na_decode_workspace_size() exceeds 20 MiB are rejected with
 *     NA_ERR_WORKSPACE before anything is enqueued (for 32 query heads and
 *     head_dim 128: a batch of up to about 1200 sequences, of any length).
 *   - The first call on a device looks up the array's device address (with that
 *     device current) and keeps it; make that first call before any stream
 *     capture.  A cudaDeviceReset() of the device invalidates the kept address:
 *     do not call this entry point on a device after resetting it.
 *   - All calls share the array and it keeps the last call's contents; the
 *     decode needs nothing in it to start at zero (the split pass writes every
 *     partial result and piece span the merge pass reads, in the same call,
 *     and a piece whose wait gave up is written as a marker that the merge
 *     pass reports as NA_ERR_DEVICE_TIMEOUT, with a zero output, instead of
 *     merging).  Calls whose kernels overlap on the GPU (other streams, other
 *     host threads) race on the array: order them on one stream.
 */
int na_attn_decode_static_ws(const na_attn_cfg *cfg, int32_t batch, const void *q_rot,
                             const na_kv_cache *cache, const int32_t *kv_lens, int32_t max_kv_len,
                             const void *gate, void *out, float *probs, int32_t probs_stride,
                             int32_t num_splits, int32_t *status, void *stream);

/*
 * Born-rule importance of a decode step: the probability mass that reads each key.
 * [cortiq fn qwen_attention_core: each head's per-key probabilities are summed into
 *  `imp`, which cache.accumulate_imp adds to the position's running importance for
 *  importance-aware eviction; fn attend_all_heads returns the same sum.]
 *
 *   imp[b][j] = sum over the H query heads of probs[b][h][j]     for j < kv_lens[b]
 * or, with accumulate != 0, imp[b][j] += that sum.  Keys past kv_lens[b] are not
 * touched.  The sum is fp32 and deterministic: the heads are cut into four
 * consecutive groups, each summed in index order, and the group sums are added
 * in group order.  Both strides a multiple of 4 with 16-byte-aligned probs and
 * imp give 16-byte accesses (the fast layout); any stride is correct.
 *
 *   probs       fp32 [batch][H][probs_stride]: the probabilities na_attn_decode wrote.
 *   kv_lens     int32 [batch] (device), the same lengths given to na_attn_decode.
 *   max_kv_len  HOST upper bound of kv_lens; <= probs_stride and <= imp_stride.
 *   imp         fp32 [batch][imp_stride] (device), caller-owned.
 *   status      device int32 or NULL: NA_ERR_CAPACITY for a length past max_kv_len
 *               (that sequence is skipped).
 * Errors: NA_ERR_INVALID_ARG for null buffers or a non-positive batch,
 * NA_ERR_CAPACITY when max_kv_len exceeds a stride.
 */
int na_decode_importance(const na_attn_cfg *cfg, int32_t batch, const float *probs,
                         int32_t probs_stride, const int32_t *kv_lens, int32_t max_kv_len,
                         float *imp, int32_t imp_stride, int32_t accumulate, int32_t *status,
                         void *stream);

/*
 * na_rope_append_kv into a paged cache.
 *
 * As na_rope_append_kv, K and V rows going to their pages.  With NA_KV_BF16 pages
 * the values are the same bit for bit.  With NA_KV_E4M3 the normed and rotated
 * fp32 value x (within ~2^-20 of the page's largest) is rounded once, to nearest
 * even, to the byte of x * 2^-e, where 2^e is the page's scale for this kv head
 * and K or V: the smallest power of two with max |x| <= 448 * 2^e over the
 * page's tokens.  A page that already holds tokens of the sequence (the chunk
 * starts inside it) keeps its scale unless the new tokens need a larger one;
 * then its earlier tokens are rounded to the larger one.  The scale of a page
 * whose first token is appended depends on the new tokens alone, whatever the
 * page held before.  q_out is bf16 in both cases.
 *
 *   total_tokens  HOST upper bound of cu_seqlens[batch] (a padded batch): rows of
 *                 q_out past cu_seqlens[batch] are left as they were.
 *   status  NA_ERR_CAPACITY for a token whose position is not below
 *           pages_per_seq * page_size, NA_ERR_PAGE for one whose table entry
 *           lies outside the cache, NA_ERR_INVALID_ARG (NA_KV_E4M3) for a
 *           sequence outside the call's tokens; such tokens are skipped (with
 *           NA_KV_E4M3 their q_out may still be written).
 */
int na_rope_append_kv_paged(const na_attn_cfg *cfg, const na_rope_params *rope, int32_t batch,
                            const int32_t *cu_seqlens, const int32_t *cache_lens,
                            int32_t total_tokens, const void *q, const void *k, const void *v,
                            const void *q_norm_w, const void *k_norm_w, void *q_out,
                            const na_paged_kv_cache *cache, int32_t *status, void *stream);

/*
 * na_attn_decode over a paged cache: one query per sequence, the same arithmetic
 * (E4M3 values are f16 numbers exactly; so is a query scaled by a power of two, for
 * elements down to 2^-26 of its largest, and within 2^-33 of that below; K's scale is
 * applied to the scores in fp32, V's in the exponent of the weights, which are
 * rounded to f16), the same outputs and probabilities.
 *
 *   max_kv_len  HOST upper bound of kv_lens; <= pages_per_seq * page_size.
 *   num_splits, workspace, probs, gate, status: as in na_attn_decode (the split
 *               pass has three CTAs per SM over E4M3 pages), with
 *               na_decode_paged_workspace_size() bytes of workspace.  With
 *               num_splits 0 sequences of few keys are not cut over the grid: up to
 *               8 CTAs share a sequence's kv head, without partial results.
 */
int na_attn_decode_paged(const na_attn_cfg *cfg, int32_t batch, const void *q_rot,
                         const na_paged_kv_cache *cache, const int32_t *kv_lens,
                         int32_t max_kv_len, const void *gate, void *out, float *probs,
                         int32_t probs_stride, int32_t num_splits, void *workspace,
                         size_t ws_bytes, int32_t *status, void *stream);

/*
 * na_attn_prefill_chunk over a paged cache: the same arithmetic and outputs.  With
 * E4M3 pages K is multiplied as it is stored, a query element as the sum of two
 * E4M3 numbers (exact down to 2^-10 of the row's largest magnitude, within 2^-17
 * of that below), V as the f16 number that it exactly is, by weights rounded to
 * f16 with V's scale in their exponent.
 *
 *   max_total_len  HOST upper bound of cache_lens[b] + new length;
 *                  <= pages_per_seq * page_size.
 *   total_tokens   HOST upper bound of cu_seqlens[batch] (a padded batch): rows of
 *                  out past cu_seqlens[batch] are left as they were.
 *   workspace      na_prefill_paged_workspace_size() bytes (NULL allowed when that is 0).
 *   Everything else as in na_attn_prefill_chunk.
 */
int na_attn_prefill_chunk_paged(const na_attn_cfg *cfg, int32_t batch, const int32_t *cu_seqlens,
                                const int32_t *cache_lens, int32_t total_tokens,
                                int32_t max_new_len, int32_t max_total_len, const void *q_rot,
                                const na_paged_kv_cache *cache, const void *gate, void *out,
                                void *workspace, size_t ws_bytes, int32_t *status, void *stream);

/* Workspace bytes (HOST out-parameter) that na_attn_prefill_chunk_paged needs for these bounds. */
int na_prefill_paged_workspace_size(const na_attn_cfg *cfg, int32_t batch, int32_t total_tokens,
                                    int32_t max_new_len, int32_t max_total_len, size_t *bytes);

/* Workspace bytes (HOST out-parameter) that na_attn_decode_paged needs for these bounds. */
int na_decode_paged_workspace_size(const na_attn_cfg *cfg, int32_t batch, int32_t max_kv_len,
                                   int32_t num_splits, size_t *bytes);

/* Workspace bytes (HOST out-parameter) that na_attn_prefill_chunk needs for these bounds. */
int na_prefill_workspace_size(const na_attn_cfg *cfg, int32_t batch, int32_t total_tokens,
                              int32_t max_new_len, int32_t max_total_len, size_t *bytes);

/* Workspace bytes (HOST out-parameter) that na_attn_decode needs for these bounds. */
int na_decode_workspace_size(const na_attn_cfg *cfg, int32_t batch, int32_t max_kv_len,
                             int32_t num_splits, size_t *bytes);

/*
 * Self-test of the device-side failure detection (an addition of this
 * library).  Every wait of the library's kernels for a copy or a tensor-core
 * operation gives up after about a second (2^31 SM cycles) and writes
 * NA_ERR_DEVICE_TIMEOUT into the caller's status word instead of hanging.  (The
 * CTAs of a cluster in na_attn_decode_paged also meet in hardware barriers, which
 * every thread reaches whatever its own waits said.)  This call runs that same bounded wait, in a
 * one-CTA kernel, on a barrier that nothing ever completes: after about a
 * second *status holds NA_ERR_DEVICE_TIMEOUT (unless it already held an error),
 * the kernel returns normally and the context stays usable.
 *
 *   status  device int32, required.
 * Errors: NA_ERR_INVALID_ARG for a NULL status; NA_ERR_CUDA if the launch fails.
 */
int na_selftest_wait_timeout(int32_t *status, void *stream);

/* Static description of a status code (HOST string, never NULL). */
const char *na_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* NA_H */
