// latent_api.cu -- C ABI of latent attention: argument validation, launch planning and
// kernel launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "latent.cuh"
#include "na_host.cuh"


namespace {

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

int check_cfg(const na_latent_cfg *c)
{
    if (!c || c->num_heads <= 0)
        return NA_ERR_INVALID_ARG;
    if (c->flags & ~(NA_LATENT_NORM | NA_ROPE_INTERLEAVED))
        return NA_ERR_INVALID_ARG;
    if (!(c->rms_eps >= 0.f) || !std::isfinite(c->sm_scale))
        return NA_ERR_INVALID_ARG;
    if ((c->kv_rank != 128 && c->kv_rank != 256 && c->kv_rank != 512) ||
        (c->nope_dim != 64 && c->nope_dim != 128) || (c->v_dim != 64 && c->v_dim != 128))
        return NA_ERR_UNSUPPORTED;
    if (c->rope_dim < 16 || c->rope_dim > 64 || c->rope_dim % 16 != 0)
        return NA_ERR_UNSUPPORTED;
    return NA_OK;
}

float score_scale_log2(const na_latent_cfg *c)
{
    const double s = c->sm_scale > 0.f ? (double)c->sm_scale
                                       : 1.0 / sqrt((double)(c->nope_dim + c->rope_dim));
    return (float)(s * 1.4426950408889634);
}

int check_cache(const na_paged_latent_cache *c, int batch, PagedView *view)
{
    if (!c || !c->kv || !c->page_table || c->num_pages <= 0 || c->pages_per_seq <= 0 ||
        c->batch < batch || !aligned16(c->kv))
        return NA_ERR_INVALID_ARG;
    const int log = page_size_log(c->page_size);
    if (log < 0 || c->num_pages > (0x7fffffff >> log) || c->pages_per_seq > (0x7fffffff >> log))
        return NA_ERR_UNSUPPORTED;
    *view = PagedView{c->page_table, c->pages_per_seq, c->num_pages, log, nullptr, nullptr};
    return NA_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? NA_OK : NA_ERR_CUDA; }

// How a call's work is cut into runs, and what of its results the workspace holds.
struct LatentRuns {
    int grid, unit_rows, most;  // `most`: runs that the device has at a time
    double tiles;
    bool cut_by_sequence;
    size_t slot_rows;           // partial rows
    size_t ws_bytes;
};

// The size of the workspace goes by these bounds alone, new lengths no longer than the call, and
// never falls when one of them grows, so that one buffer serves every smaller step: partial rows
// for as many runs of 64 rows as there are SMs (pairs of CTAs have half as many of 128), or for all
// tiles where there are fewer, and an entry per SM whatever a unit's rows are.
LatentRuns plan_runs(const na_latent_cfg *c, int batch, int total_tokens, int max_new_len, int max_total_len)
{
    LatentRuns r{};
    const long long rows = (long long)std::min(max_new_len, total_tokens) * c->num_heads;
    r.unit_rows = latent_unit_rows(rows, c->kv_rank);
    r.tiles = (double)batch * ceil_div(rows, r.unit_rows) * ceil_div(max_total_len, kLatentKeys);
    r.most = r.unit_rows > 64 ? std::max(sm_count() / 2, 1) : sm_count();
    r.grid = (int)std::max(1.0, std::min((double)r.most, r.tiles));
    r.cut_by_sequence = rows <= r.unit_rows && batch <= r.grid;
    const double runs = std::max(sm_count(), 2) * (double)std::min(r.unit_rows, 64);
    r.slot_rows = 2 * (size_t)std::min(runs, std::max(r.tiles, 1.0) * r.unit_rows);
    r.ws_bytes = r.slot_rows * (c->kv_rank + 2) * sizeof(float) + sm_count() * sizeof(int4);
    return r;
}

struct LatentPlan : LatentRuns {
    int joined_grid, pieces;  // pieces > 0: units of their own clusters instead of runs
};

// Runs: one CTA or pair of CTAs per SM, fewer where the bounds allow no more tiles than that, and
// a second pass.  Units joined in their own clusters need neither the search for a run's
// beginning nor the pass, which is 2.5 to 3 us less, worth some 3 tiles of 512 latent
// numbers or 5 of fewer; but a cluster has 8 CTAs at most and none helps another (4
// heads, 333 keys of 128: 9.9 us by runs, 6.7; 16 heads, 512 numbers, 1000 keys: 13.9 and 12.2,
// 4000 keys: 15.6 and 20.7).  The lengths are bounds: batches are taken for 0.6 of them.
LatentPlan plan_latent(const na_latent_cfg *c, int batch, int total_tokens, int max_new_len,
                       int max_total_len)
{
    LatentPlan pl{plan_runs(c, batch, total_tokens, max_new_len, max_total_len), 0, 0};
    const long long rows = (long long)std::min(max_new_len, total_tokens) * c->num_heads;
    const int joined_rows = rows <= 32 ? 32 : 64;
    const double units = (double)batch * ceil_div(rows, joined_rows);
    const int longest = (int)ceil_div(max_total_len, kLatentKeys);
    int pieces = std::min(kLatentMaxPieces, longest);
    while (pieces > 1 && units > sm_clusters(pieces))
        pieces--;
    const double by_runs = pl.tiles * (batch > 1 ? 0.6 : 1.0) / pl.most + (c->kv_rank == 512 ? 3 : 5);
    if (pieces > 0 && units <= sm_count() && ceil_div(longest, pieces) <= by_runs) {
        pl.pieces = pieces;
        pl.joined_grid = (int)units;
    }
    return pl;
}

// Which kernel an expanded call takes, and what it cuts.  Tall units (256 rows, one CTA per SM) carry
// more products per byte of shared memory, 128-row units on two CTAs per SM begin and end behind
// one another; a tall unit may be cut into pieces of its keys, a cluster of up to 8 CTAs.
//   - Fewer tall units than SMs: all are cut (128 tokens after 4096, 8 heads: 53.2 us on 128-row
//     units, 57.2 on tall ones, 20.1 in eight pieces).  A piece costs its CTA ~8 us
//     besides its keys, hence 256 of them at least.  Ragged batches only have bounds: a sequence
//     counts for half a unit beside its tokens, and a few clusters that wait do no harm.
//   - Batches of equal lengths: the units left over after the last whole wave of SMs, in a launch of
//     their own, which from 4096 keys on gains more than it costs (2048 tokens after 16384, 40
//     heads: 746 us uncut, 625; after 1024: 109 and 128).
//   - Where all units have about as many keys, CTAs take them in turn, the next one's beginning beside
//     the end of the last (4 prompts of 1024 tokens after 16384, 40 heads: 1167 us by a CTA
//     per unit, 1082; 8 of 256 after 4096: 183 and 179); where they differ more the hardware's order,
//     a CTA for each, balances them better (8 prompts of 100 .. 1000 after 1536, 8 heads: 78 and 91).
//   - Below 1024 keys a row on average the 128-row units are faster (1024 tokens of one prompt, 8
//     heads: 16.3 us against 19.2; 16 prompts of 1 .. 512 tokens, 32 heads: 86 against
//     107 in tiles of 128 keys), and so they are for sequences of few tokens, whose tall units are mostly empty (64 of
//     1 .. 60 tokens after 1000 .. 2000: 366 against 452).
int plan_expanded(ExpandedParams &p)
{
    const int sms = sm_count(), keys = std::min(p.max_key_len, p.total_keys);
    const bool equal = (long long)p.batch * p.max_new_len == p.total_tokens;
    const double per_tile = (double)p.H * p.batch;
    const double tall_units = per_tile * ceil_div(p.max_new_len, 2 * kExpandedRows);
    const double short_units = per_tile * ceil_div(p.max_new_len, kExpandedRows);
    if (short_units > INT_MAX / 8)
        return NA_ERR_UNSUPPORTED;
    const double busy = equal ? tall_units
                              : std::min(tall_units, p.H * (p.total_tokens / (2.0 * kExpandedRows) +
                                                            p.batch / 2.0));
    const double most = equal ? 1.0 : 1.15;
    int pieces = kExpandedMaxPieces;
    while (pieces > 1 && (busy > most * sm_clusters(pieces) || keys / pieces < 256))
        pieces--;
    int cut = pieces > 1 ? (int)tall_units : 0;
    const int keys_per_row = (cut ? keys : std::min(keys, p.total_keys / p.batch)) - p.max_new_len / 2;
    p.tall = keys_per_row >= 1024 && (cut || p.total_tokens >= 96ll * p.batch);
    if (p.tall && !cut && equal && keys >= 4096) {
        const int rest = (int)tall_units % sms;
        pieces = rest ? kExpandedMaxPieces : 1;
        while (pieces > 1 && rest > sm_clusters(pieces))
            pieces--;
        cut = pieces > 1 ? rest : 0;
    }
    p.units = (int)(p.tall ? tall_units : short_units);
    p.sms = sms;
    p.in_turn = equal && 2ll * p.max_new_len <= keys;
    p.pieces = pieces;
    p.cut_units = cut;
    return NA_OK;
}

}  // namespace

extern "C" {

int na_latent_append_paged(const na_latent_cfg *cfg, const na_rope_params *rope, int32_t batch,
                           const int32_t *cu_seqlens, const int32_t *cache_lens,
                           int32_t total_tokens, const void *kv, int64_t kv_stride, const void *q,
                           int64_t q_stride, void *q_out, int64_t q_out_stride,
                           const void *kv_norm_w, const na_paged_latent_cache *cache,
                           int32_t *status, void *stream)
{
    int rc = check_cfg(cfg);
    if (rc != NA_OK)
        return rc;
    if ((rc = check_rope(rope)) != NA_OK)
        return rc;
    if (batch <= 0 || total_tokens < 0)
        return NA_ERR_INVALID_ARG;
    PagedView pg;
    if ((rc = check_cache(cache, batch, &pg)) != NA_OK)
        return rc;
    if (total_tokens == 0)
        return NA_OK;
    if (!cu_seqlens || !cache_lens || !kv || !aligned16(kv) || !q != !q_out || !aligned16(q) ||
        !aligned16(q_out))
        return NA_ERR_INVALID_ARG;
    if (kv_stride % 8 != 0 || kv_stride < cfg->kv_rank + cfg->rope_dim)
        return NA_ERR_INVALID_ARG;
    if (q && (q_stride % 8 != 0 || q_stride < cfg->rope_dim || q_out_stride % 8 != 0 ||
              q_out_stride < cfg->rope_dim || (q == q_out && q_stride != q_out_stride)))
        return NA_ERR_INVALID_ARG;
    const bool normed = (cfg->flags & NA_LATENT_NORM) != 0;
    if (normed && (!kv_norm_w || !aligned16(kv_norm_w)))
        return NA_ERR_INVALID_ARG;
    const RopeTable &table = rope_table(rope, cfg->rope_dim);
    LatentAppendParams p{};
    p.H = cfg->num_heads;
    p.R = cfg->kv_rank;
    p.rd = cfg->rope_dim;
    p.batch = batch;
    p.capacity = cache->pages_per_seq * cache->page_size;
    p.total_tokens = total_tokens;
    p.normed = normed;
    p.interleaved = (cfg->flags & NA_ROPE_INTERLEAVED) != 0;
    p.eps = cfg->rms_eps;
    p.rope_scale = table.scale;
    p.cu_seqlens = cu_seqlens;
    p.cache_lens = cache_lens;
    p.kv = static_cast<const bf16 *>(kv);
    p.q = static_cast<const bf16 *>(q);
    p.norm_w = static_cast<const bf16 *>(kv_norm_w);
    p.q_out = static_cast<bf16 *>(q_out);
    p.cache = static_cast<bf16 *>(cache->kv);
    p.kv_stride = kv_stride;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.status = status;
    return done(launch_latent_append(p, pg, table.turns, static_cast<cudaStream_t>(stream)));
}

int na_latent_paged_workspace_size(const na_latent_cfg *cfg, int32_t batch, int32_t total_tokens,
                                   int32_t max_new_len, int32_t max_total_len, size_t *bytes)
{
    const int rc = check_cfg(cfg);
    if (rc != NA_OK)
        return rc;
    if (!bytes || batch <= 0 || total_tokens < 0 || max_new_len < 0 || max_total_len < 0)
        return NA_ERR_INVALID_ARG;
    *bytes = plan_runs(cfg, batch, total_tokens, max_new_len, max_total_len).ws_bytes;
    return NA_OK;
}

int na_attn_latent_paged(const na_latent_cfg *cfg, int32_t batch, const int32_t *cu_seqlens,
                         const int32_t *cache_lens, int32_t total_tokens, int32_t max_new_len,
                         int32_t max_total_len, const void *q_lat,
                         const na_paged_latent_cache *cache, void *out, void *workspace,
                         size_t ws_bytes, int32_t *status, void *stream)
{
    int rc = check_cfg(cfg);
    if (rc != NA_OK)
        return rc;
    if (batch <= 0 || total_tokens < 0 || max_new_len < 0 || max_total_len < 0)
        return NA_ERR_INVALID_ARG;
    PagedView pg;
    if ((rc = check_cache(cache, batch, &pg)) != NA_OK)
        return rc;
    if (total_tokens == 0)
        return NA_OK;
    if (!cu_seqlens || !cache_lens || !q_lat || !out || max_new_len <= 0 || !aligned16(q_lat) ||
        !aligned16(out))
        return NA_ERR_INVALID_ARG;
    const int capacity = cache->pages_per_seq * cache->page_size;
    if (max_total_len > capacity)
        return NA_ERR_CAPACITY;
    // query rows are addressed by 32-bit tensor-map coordinates
    if ((long long)total_tokens * cfg->num_heads > INT_MAX - 256)
        return NA_ERR_UNSUPPORTED;
    const LatentPlan pl = plan_latent(cfg, batch, total_tokens, max_new_len, max_total_len);
    if (!workspace || ws_bytes < pl.ws_bytes || !aligned16(workspace))
        return NA_ERR_WORKSPACE;
    LatentParams p{};
    p.H = cfg->num_heads;
    p.R = cfg->kv_rank;
    p.rd = cfg->rope_dim;
    p.batch = batch;
    p.capacity = capacity;
    p.scale_log2 = score_scale_log2(cfg);
    p.total_tokens = total_tokens;
    p.max_new_len = std::min(max_new_len, total_tokens);  // (no sequence has more)
    p.max_total_len = max_total_len;
    p.unit_rows = pl.pieces ? std::min(pl.unit_rows, 64) : pl.unit_rows;
    p.grid = pl.pieces ? pl.joined_grid : pl.grid;
    p.pieces = pl.pieces;
    p.cut_by_sequence = pl.cut_by_sequence;
    p.cu_seqlens = cu_seqlens;
    p.cache_lens = cache_lens;
    p.q = static_cast<const bf16 *>(q_lat);
    p.cache = static_cast<const bf16 *>(cache->kv);
    p.out = static_cast<bf16 *>(out);
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = p.part_o + pl.slot_rows * cfg->kv_rank;
    p.cut = reinterpret_cast<int4 *>(p.part_ml + pl.slot_rows * 2);
    p.status = status;
    if ((rc = bind_context()) != NA_OK)
        return rc;
    return done(launch_latent(p, pg, static_cast<cudaStream_t>(stream)));
}

int na_attn_latent_expanded(const na_latent_cfg *cfg, int32_t batch, const int32_t *cu_seqlens,
                            const int32_t *key_starts, const int32_t *key_lens,
                            int32_t total_tokens, int32_t total_keys, int32_t max_new_len,
                            int32_t max_key_len, const void *q, const void *kv, const void *k_pe,
                            int64_t k_pe_stride, void *out, int32_t *status, void *stream)
{
    int rc = check_cfg(cfg);
    if (rc != NA_OK)
        return rc;
    if (batch <= 0 || total_tokens < 0 || total_keys < 0 || max_new_len < 0 || max_key_len < 0)
        return NA_ERR_INVALID_ARG;
    if (total_tokens == 0)
        return NA_OK;
    if (!cu_seqlens || !key_starts || !key_lens || !q || !kv || !k_pe || !out || max_new_len <= 0 ||
        total_keys == 0)
        return NA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(kv) || !aligned16(k_pe) || !aligned16(out) ||
        k_pe_stride % 8 != 0 || k_pe_stride < cfg->rope_dim)
        return NA_ERR_INVALID_ARG;
    if ((long long)k_pe_stride >= (1ll << 32) ||
        (long long)std::max(total_tokens, total_keys) * cfg->num_heads >= (1ll << 40))
        return NA_ERR_UNSUPPORTED;
    max_new_len = std::min(max_new_len, total_tokens);
    ExpandedParams p{};
    p.H = cfg->num_heads;
    p.dn = cfg->nope_dim;
    p.rd = cfg->rope_dim;
    p.dv = cfg->v_dim;
    p.batch = batch;
    p.scale_log2 = score_scale_log2(cfg);
    p.total_tokens = total_tokens;
    p.total_keys = total_keys;
    p.max_new_len = max_new_len;
    p.max_key_len = max_key_len;
    p.cu_seqlens = cu_seqlens;
    p.key_starts = key_starts;
    p.key_lens = key_lens;
    p.q = static_cast<const bf16 *>(q);
    p.kv = static_cast<const bf16 *>(kv);
    p.k_pe = static_cast<const bf16 *>(k_pe);
    p.k_pe_stride = k_pe_stride;
    p.out = static_cast<bf16 *>(out);
    p.status = status;
    if ((rc = plan_expanded(p)) != NA_OK)
        return rc;
    if ((rc = bind_context()) != NA_OK)
        return rc;
    return done(launch_latent_expanded(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
