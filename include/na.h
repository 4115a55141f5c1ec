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

#define NA_ROPE_INTERLEAVED 2u /* RoPE turns pairs (x[2 i], x[2 i + 1]) instead of (x[i], x[i + rd/2]) */

/* ------------------------------------------------------- pages of a cache --
 *
 * The page tables of a serving batch, its forks and evictions.  (Additions of
 * this library; the pages have no counterpart.)  One table serves every layer
 * of a model, so na_pages_fork is called once a step, and na_pages_copy and
 * na_pages_compact once per layer.  A latent cache (below) has one kv head of
 * head_dim = kv_rank + rope_dim and v NULL.
 */

/*
 * One step of a batch's page tables: which sequences go on, from which, and
 * how many positions they need.
 *
 * The old batch is table [old_batch][pages_per_seq]: row p holds the pages of its
 * sequence, lens[p] tokens, its entries up to the first negative one.  Sequence b
 * of the new batch continues parents[b] (an old sequence, many may share one), or
 * starts empty (parents[b] < 0); an old sequence that is nobody's parent ends.
 * With n = lens[parents[b]] (or 0) tokens:
 *   - new_table[b] gets the parent's n / page_size full pages, shared.  The child
 *     with the lowest b gets all of the parent's other pages too (a part-filled one,
 *     and those reserved behind it).  For any other child of a parent whose last
 *     page is part-filled a page is taken, and the copy that it needs is
 *     copy_src[b] -> copy_dst[b] (-1 where there is none): na_pages_copy.
 *   - pages are taken until the row has room for n + grow[b] tokens (grow NULL: 0).
 *   - ref[page] counts the rows that hold a page, of this batch and of others (a
 *     prefix that is kept, a second table).  new_ref is ref without the old rows'
 *     and with the new ones'; a page with count 0 is free.  Pages are taken in
 *     index order from those free after that, for b in order and positions in order.
 * The other entries of new_table are -1.  All results are functions of the
 * inputs alone, in whatever order the device works.
 *
 *   batch, old_batch  1 .. 4096 sequences.
 *   parents, grow     int32 [batch] (grow may be NULL);  lens int32 [old_batch].
 *   table             int32 [old_batch][pages_per_seq];  ref int32 [num_pages].
 *   new_table         int32 [batch][pages_per_seq];  new_ref int32 [num_pages];
 *   new_lens, copy_src, copy_dst  int32 [batch].  No output may overlap an input or
 *                     another output (callers keep two tables and take turns).
 *   status  NA_ERR_INVALID_ARG for a parent >= old_batch (taken as none) or a
 *           negative grow (taken as 0), NA_ERR_PAGE for an entry >= num_pages (which
 *           ends its row) or a row with fewer pages than lens needs (the missing ones
 *           are taken), NA_ERR_CAPACITY when no page is free or a row would need more
 *           than pages_per_seq (the entries that are missing are -1, a copy
 *           without a page -1 -> -1).
 * Errors: NA_ERR_INVALID_ARG for null pointers (status and grow may be NULL) and
 * sizes below 1, NA_ERR_UNSUPPORTED for a page size other than 16, 32, 64, 128,
 * more than 4096 sequences or a new table of more than 2^31 - 1 entries.
 */
int na_pages_fork(int32_t batch, int32_t old_batch, const int32_t *parents, const int32_t *grow,
                  const int32_t *lens, const int32_t *table, int32_t pages_per_seq,
                  int32_t page_size, const int32_t *ref, int32_t num_pages, int32_t *new_table,
                  int32_t *new_ref, int32_t *new_lens, int32_t *copy_src, int32_t *copy_dst,
                  int32_t *status, void *stream);

/*
 * Whole pages (K, V and their scales, every kv head) from src[i] to dst[i], i < n;
 * a pair with a negative src or dst is skipped.  The pairs have to be independent:
 * no page may be the dst of two, or the dst of one and the src of another.
 *
 *   cache   its page_table, batch and pages_per_seq are not looked at.
 *   n       pairs; 0 is a no-op.   src, dst  int32 [n].
 *   status  NA_ERR_PAGE for a page >= num_pages (that pair is skipped).
 * Errors: as for a paged cache; head_dim has to be a multiple of 8 (NA_KV_E4M3: 16)
 * and at most 1024 (NA_ERR_UNSUPPORTED).
 */
int na_pages_copy(int32_t num_kv_heads, int32_t head_dim, const na_paged_kv_cache *cache, int32_t n,
                  const int32_t *src, const int32_t *dst, int32_t *status, void *stream);

/*
 * The kept tokens of each sequence, in a cache's pages, to the front of others: row
 * j < keep_lens[b] of sequence b in `to` becomes the row at position keep[b][j]
 * (j itself with keep NULL) of sequence b in `from`.  With rope, K's dimensions
 * [rotary_start, rotary_start + rotary_dim) are turned by (j - keep[b][j]) positions,
 * so that a key stands as if it had been appended at its new position (cos and sin
 * are not multiplied by an attention factor again).  This is what eviction by
 * na_decode_importance needs: positions then follow from the new lengths, in the
 * attention calls and for the tokens to come.  With keep NULL, no rope and a
 * contiguous `to` it gathers sequences out of their pages.
 * bf16: an unturned row is moved bit for bit; a turned value is rounded once to
 * bf16 (within one ulp, correctly but for 2^-22 of its pair next to a rounding border).
 * E4M3: a new page's scale is the smallest power of two 2^e, -127 <= e <= 127, with
 * max |x| <= 448 * 2^e over the rows moved into it, x the stored values turned in fp32
 * (within 2^-20 of the row's largest), and every x is rounded once to x * 2^-e.  (Other
 * slots of such a page keep their bytes, a page into which no row is moved its scale too.)
 *
 *   from, to   caches of one dtype; their page sizes may differ, and they may be
 *              the same pools.  No page that `to` writes may be one that `from`
 *              reads, or belong to two sequences.  Slots of `to` behind a sequence's
 *              rows are left as they were.
 *   rope       HOST, or NULL: nothing is turned.  rotary_dim even, rotary_start +
 *              rotary_dim <= head_dim.  flags: 0 or NA_ROPE_INTERLEAVED.
 *   max_keep   HOST upper bound of keep_lens, and keep's row stride; 0 is a no-op.
 *   status     NA_ERR_CAPACITY for a length above max_keep or `to`'s positions or a
 *              kept position outside `from`'s (the row is skipped, a sequence
 *              altogether for its length), NA_ERR_PAGE for a table entry outside its
 *              pool (its rows are skipped), NA_ERR_UNSUPPORTED for an E8M0 byte 255
 *              (taken as 2^127).
 * Errors: as for paged caches; NA_ERR_UNSUPPORTED for a head_dim that is no multiple
 * of 8 (E4M3: 16) or above 1024 (E4M3: 128) or a rotary_dim above 128.
 */
int na_pages_compact(int32_t num_kv_heads, int32_t head_dim, int32_t batch,
                     const na_paged_kv_cache *from, const na_paged_kv_cache *to, const int32_t *keep,
                     const int32_t *keep_lens, int32_t max_keep, const na_rope_params *rope,
                     int32_t rotary_start, int32_t rotary_dim, uint32_t flags, int32_t *status,
                     void *stream);

/* -------------------------------------------------------- latent attention --
 *
 * Attention whose keys and values come from one latent vector a token.  (An
 * addition of this library; the pages have no counterpart.)  A token's row is
 * [c, r]: c its kv_rank latent numbers, r a rotated key part of rope_dim that all
 * heads share.  With the maps U_h (nope_dim x kv_rank) and W_h (v_dim x kv_rank) of
 * head h its key is [U_h c, r] and its value W_h c, so with a query [a, s]
 *     score = scale * (a . U_h c + s . r) = scale * ([U_h^T a, s] . [c, r]),
 *     out   = sum_j p_j W_h c_j           = W_h (sum_j p_j c_j).
 * Absorbed form (na_attn_latent_paged): queries [U_h^T a, s] against the cached rows,
 * the sum of the latents out; a row is read once for all heads, which suits single
 * tokens and short chunks.  Expanded form (na_attn_latent_expanded): [U_h c, W_h c]
 * made first, then attention of nope_dim + rope_dim and v_dim, with fewer products
 * per query and key: for long chunks.  The maps themselves are matrix products of
 * the caller's.
 */
#define NA_LATENT_NORM 1u         /* RMS norm of the latent part before it enters the cache */

typedef struct na_latent_cfg {
    int32_t num_heads; /* H, any number */
    int32_t kv_rank;   /* R: 128, 256 or 512 */
    int32_t rope_dim;  /* rd: 16, 32, 48 or 64 */
    int32_t nope_dim;  /* 64 or 128: expanded keys; with rope_dim the default score scale */
    int32_t v_dim;     /* 64 or 128: expanded values */
    float sm_scale;    /* score scale; <= 0 selects 1 / sqrt(nope_dim + rope_dim) */
    float rms_eps;     /* epsilon of the latent norm */
    uint32_t flags;    /* NA_LATENT_NORM, NA_ROPE_INTERLEAVED */
} na_latent_cfg;

/* Caller-owned pages of latent rows; the rules of na_paged_kv_cache, one row for all heads. */
typedef struct na_paged_latent_cache {
    void *kv;                  /* bf16 [num_pages][page_size][kv_rank + rope_dim], 16-byte aligned */
    const int32_t *page_table; /* int32 [batch][pages_per_seq] */
    int32_t num_pages;         /* num_pages * page_size <= 2^31 - 1 */
    int32_t page_size;         /* 16, 32, 64 or 128 */
    int32_t batch;
    int32_t pages_per_seq;
} na_paged_latent_cache;

/*
 * New tokens' latent rows into their pages, and the queries' rotated parts.
 *
 * For new token t of sequence b at pos = cache_lens[b] + (t - cu_seqlens[b]):
 *   row[:R]        = norm(kv[t][:R])  (unchanged without NA_LATENT_NORM)
 *   row[R:]        = RoPE(kv[t][R:], pos)
 *   q_out[t][h][:] = RoPE(q[t][h][:], pos)     rope_dim elements, every h
 * Accuracy: as na_rope_append_kv (a normed value within one bf16 ulp, correctly
 * rounded but for ~2^-21 next to a rounding border).
 *
 *   kv        bf16 [total_tokens] rows of R + rd elements, kv_stride elements apart.
 *   q, q_out  bf16: rope_dim elements of token t and head h start q_stride * (t H + h)
 *             elements after q (q_out_stride after q_out): the rotated part of wider
 *             query rows.  q_out may be q, with the same stride; otherwise they may not
 *             overlap.  Both NULL: no queries.
 *   kv_norm_w bf16 [R], required with NA_LATENT_NORM, else ignored.
 *   total_tokens  HOST upper bound of cu_seqlens[batch]; rows past it are left alone.
 *   status    as na_rope_append_kv_paged (NA_ERR_CAPACITY, NA_ERR_PAGE; such a token's
 *             row is skipped, with NA_ERR_CAPACITY its queries too).
 * Errors: NA_ERR_INVALID_ARG for pointers that are null or not 16-byte aligned, strides
 * that are no multiple of 8 elements or smaller than a row.
 */
int na_latent_append_paged(const na_latent_cfg *cfg, const na_rope_params *rope, int32_t batch,
                           const int32_t *cu_seqlens, const int32_t *cache_lens,
                           int32_t total_tokens, const void *kv, int64_t kv_stride, const void *q,
                           int64_t q_stride, void *q_out, int64_t q_out_stride,
                           const void *kv_norm_w, const na_paged_latent_cache *cache,
                           int32_t *status, void *stream);

/*
 * Absorbed latent attention of new tokens, whose rows are in the pages already:
 *   out[t][h] = sum_j softmax_j(scale * q_lat[t][h] . row_j) row_j[:R],  j <= pos of t.
 * One token per sequence (a decode step) and chunks are the same call.
 * Arithmetic: bf16 tensor cores with fp32 accumulation, the softmax in fp32, weights
 * rounded to bf16 for the second product; with unit-scale inputs within 2e-2 (max-abs)
 * and 5e-3 (relative L2) of the exact result.
 *
 *   q_lat      bf16 [total_tokens][H][R + rd];  out bf16 [total_tokens][H][R].
 *   total_tokens, max_new_len, max_total_len  HOST upper bounds, as in
 *              na_attn_prefill_chunk_paged; rows of out past cu_seqlens[batch] are left
 *              as they were.
 *   workspace  na_latent_paged_workspace_size() bytes.  Any contents will do.
 *   status     as na_attn_prefill_chunk_paged; a sequence with a bad length is skipped.
 */
int na_attn_latent_paged(const na_latent_cfg *cfg, int32_t batch, const int32_t *cu_seqlens,
                         const int32_t *cache_lens, int32_t total_tokens, int32_t max_new_len,
                         int32_t max_total_len, const void *q_lat,
                         const na_paged_latent_cache *cache, void *out, void *workspace,
                         size_t ws_bytes, int32_t *status, void *stream);

/* Workspace bytes (HOST out-parameter) that na_attn_latent_paged needs for these bounds; enough for
 * every call of this configuration with smaller ones. */
int na_latent_paged_workspace_size(const na_latent_cfg *cfg, int32_t batch, int32_t total_tokens,
                                   int32_t max_new_len, int32_t max_total_len, size_t *bytes);

/*
 * Expanded latent attention, causal: with n new tokens and key_lens[b] keys sequence b's
 * i-th token sees its first key_lens[b] - n + 1 + i keys (none: a row of zeros).
 *   out[t][h] = sum_j softmax_j(scale * (q[t][h][:dn] . kv[j][h][:dn] + q[t][h][dn:] . k_pe[j]))
 *               kv[j][h][dn:]
 * over its keys, rows key_starts[b] .. key_starts[b] + key_lens[b] - 1 of kv and k_pe.
 * Arithmetic and accuracy as na_attn_prefill_chunk.
 *
 *   key_starts, key_lens  int32 [batch].  Sequences may share keys.
 *   max_new_len, max_key_len  HOST upper bounds.
 *   q     bf16 [total_tokens][H][dn + rd].
 *   kv    bf16 [total_keys][H][dn + dv]: keys and values as the expanding product writes them.
 *   k_pe  bf16, rd elements a key, k_pe_stride elements apart (a multiple of 8): the rotated
 *         part of latent rows.
 *   out   bf16 [total_tokens][H][dv].
 *   total_keys  at least 1 where there are tokens (NA_ERR_INVALID_ARG).
 *   status  NA_ERR_INVALID_ARG for a new length above max_new_len or outside the call's
 *           tokens, NA_ERR_CAPACITY for keys above max_key_len or outside the total_keys
 *           rows; such a sequence is skipped.
 * Keys and values of the sequences have to be finite; other rows of kv may hold any bits.
 */
int na_attn_latent_expanded(const na_latent_cfg *cfg, int32_t batch, const int32_t *cu_seqlens,
                            const int32_t *key_starts, const int32_t *key_lens,
                            int32_t total_tokens, int32_t total_keys, int32_t max_new_len,
                            int32_t max_key_len, const void *q, const void *kv, const void *k_pe,
                            int64_t k_pe_stride, void *out, int32_t *status, void *stream);

/*
 * Self-test of the device-side failure detection (an addition of this
 * library).  Every wait of the library's kernels for a copy or a tensor-core
 * operation gives up after about a second (2^31 SM cycles) and writes
 * NA_ERR_DEVICE_TIMEOUT into the caller's status word instead of hanging.  (The
 * CTAs of a cluster in na_attn_decode_paged, the latent attention calls and na_pages_fork
 * also meet in hardware barriers, which every thread reaches whatever its own waits said.)  This call runs that same bounded wait, in a
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
