// pages_api.cu -- C ABI of the page operations: argument validation and launches.
#include <climits>

#include "na_host.cuh"
#include "pages.cuh"

namespace {

// A cache of any row width whose pages are copied or moved, checked.  `table`: its page
// table is used; without v it holds latent rows.
int check_pages(int kv_heads, int head_dim, const na_paged_kv_cache *c, int batch, bool table,
                PagedView *view)
{
    if (!c || !c->k || c->num_pages <= 0 || kv_heads <= 0 || head_dim <= 0)
        return NA_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v))
        return NA_ERR_INVALID_ARG;
    if (c->dtype != NA_KV_BF16 && c->dtype != NA_KV_E4M3)
        return NA_ERR_INVALID_ARG;
    const bool e4m3 = c->dtype == NA_KV_E4M3;
    if (e4m3 && (!c->v || !c->k_scale || !c->v_scale))
        return NA_ERR_INVALID_ARG;
    if (table && (!c->page_table || c->pages_per_seq <= 0 || c->batch < batch))
        return NA_ERR_INVALID_ARG;
    const int log = page_size_log(c->page_size);
    if (log < 0 || head_dim % (e4m3 ? 16 : 8) != 0 || head_dim > 1024)
        return NA_ERR_UNSUPPORTED;
    if ((long long)c->num_pages * kv_heads > (0x7fffffffLL >> log) ||
        (table && (long long)c->pages_per_seq > (0x7fffffffLL >> log)))
        return NA_ERR_UNSUPPORTED;
    *view = PagedView{c->page_table, c->pages_per_seq, c->num_pages, log,
                      e4m3 ? c->k_scale : nullptr, e4m3 ? c->v_scale : nullptr};
    return NA_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? NA_OK : NA_ERR_CUDA; }

}  // namespace

extern "C" {

int na_pages_fork(int32_t batch, int32_t old_batch, const int32_t *parents, const int32_t *grow,
                  const int32_t *lens, const int32_t *table, int32_t pages_per_seq,
                  int32_t page_size, const int32_t *ref, int32_t num_pages, int32_t *new_table,
                  int32_t *new_ref, int32_t *new_lens, int32_t *copy_src, int32_t *copy_dst,
                  int32_t *status, void *stream)
{
    if (batch <= 0 || old_batch <= 0 || pages_per_seq <= 0 || num_pages <= 0)
        return NA_ERR_INVALID_ARG;
    if (!parents || !lens || !table || !ref || !new_table || !new_ref || !new_lens || !copy_src ||
        !copy_dst)
        return NA_ERR_INVALID_ARG;
    const int log = page_size_log(page_size);
    if (log < 0 || batch > kMaxForkBatch || old_batch > kMaxForkBatch ||
        (long long)pages_per_seq > (0x7fffffffLL >> log) || num_pages > (0x7fffffff >> log))
        return NA_ERR_UNSUPPORTED;
    // the entries that a step has to fill are counted, and ranked, in 32 bits
    if ((long long)batch * pages_per_seq > INT_MAX)
        return NA_ERR_UNSUPPORTED;
    return done(launch_pages_fork(ForkParams{batch, old_batch, pages_per_seq, log, num_pages, parents,
                                             grow, lens, table, ref, new_table, new_ref, new_lens,
                                             copy_src, copy_dst, status},
                                  static_cast<cudaStream_t>(stream)));
}

int na_pages_copy(int32_t num_kv_heads, int32_t head_dim, const na_paged_kv_cache *cache, int32_t n,
                  const int32_t *src, const int32_t *dst, int32_t *status, void *stream)
{
    PagedView view;
    const int rc = check_pages(num_kv_heads, head_dim, cache, 0, false, &view);
    if (rc != NA_OK)
        return rc;
    if (n < 0)
        return NA_ERR_INVALID_ARG;
    if (n == 0)
        return NA_OK;
    if (!src || !dst)
        return NA_ERR_INVALID_ARG;
    const bool e4m3 = cache->dtype == NA_KV_E4M3;
    PageCopyParams p{};
    p.n = n;
    p.num_pages = cache->num_pages;
    p.kv_heads = num_kv_heads;
    p.page_bytes = (long long)num_kv_heads * cache->page_size * head_dim * (e4m3 ? 1 : 2);
    p.k = static_cast<uint8_t *>(cache->k);
    p.v = static_cast<uint8_t *>(cache->v);
    p.k_scale = e4m3 ? cache->k_scale : nullptr;
    p.v_scale = e4m3 ? cache->v_scale : nullptr;
    p.src = src;
    p.dst = dst;
    p.status = status;
    return done(launch_pages_copy(p, static_cast<cudaStream_t>(stream)));
}

int na_pages_compact(int32_t num_kv_heads, int32_t head_dim, int32_t batch,
                     const na_paged_kv_cache *from, const na_paged_kv_cache *to, const int32_t *keep,
                     const int32_t *keep_lens, int32_t max_keep, const na_rope_params *rope,
                     int32_t rotary_start, int32_t rotary_dim, uint32_t flags, int32_t *status,
                     void *stream)
{
    CompactParams p{};
    int rc;
    if (batch <= 0 || max_keep < 0)
        return NA_ERR_INVALID_ARG;
    if ((rc = check_pages(num_kv_heads, head_dim, from, batch, true, &p.from)) != NA_OK ||
        (rc = check_pages(num_kv_heads, head_dim, to, batch, true, &p.to)) != NA_OK)
        return rc;
    if (from->dtype != to->dtype || !from->v != !to->v || (flags & ~NA_ROPE_INTERLEAVED))
        return NA_ERR_INVALID_ARG;
    const bool e4m3 = from->dtype == NA_KV_E4M3;
    if (e4m3 && (head_dim > 128 || num_kv_heads > 32767))
        return NA_ERR_UNSUPPORTED;
    if (rope) {
        if ((rc = check_rope(rope)) != NA_OK)
            return rc;
        if (rotary_start < 0 || rotary_dim < 0 || (rotary_dim & 1) || rotary_start > head_dim ||
            rotary_dim > head_dim - rotary_start)
            return NA_ERR_INVALID_ARG;
        if (rotary_dim > 128)
            return NA_ERR_UNSUPPORTED;
    }
    if (max_keep == 0)
        return NA_OK;
    if (!keep_lens)
        return NA_ERR_INVALID_ARG;
    p.KV = num_kv_heads;
    p.d = head_dim;
    p.batch = batch;
    p.max_keep = max_keep;
    p.turn = rope && rotary_dim > 0;
    p.rot_start = p.turn ? rotary_start : 0;
    p.rd = p.turn ? rotary_dim : 0;
    p.interleaved = (flags & NA_ROPE_INTERLEAVED) != 0;
    p.keep = keep;
    p.keep_lens = keep_lens;
    p.from_k = static_cast<const uint8_t *>(from->k);
    p.from_v = static_cast<const uint8_t *>(from->v);
    p.to_k = static_cast<uint8_t *>(to->k);
    p.to_v = static_cast<uint8_t *>(to->v);
    p.to_positions = to->pages_per_seq * to->page_size;
    p.to_k_scale = to->k_scale;
    p.to_v_scale = to->v_scale;
    p.status = status;
    static const RopeTurns none{};
    return done(launch_pages_compact(p, e4m3, p.turn ? rope_table(rope, rotary_dim).turns : none,
                                     static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
