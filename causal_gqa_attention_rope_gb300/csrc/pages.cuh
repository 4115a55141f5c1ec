// pages.cuh -- parameters of the page kernels (pages.cu), filled in by the C ABI
// (pages_api.cu).
#pragma once

#include "na_internal.cuh"

constexpr int kMaxForkBatch = 4096;

struct ForkParams {
    int batch, old_batch, pages_per_seq, page_log, num_pages;
    const int32_t *parents, *grow, *lens, *table, *ref;
    int32_t *new_table, *new_ref, *new_lens, *copy_src, *copy_dst;
    int32_t *status;
};

struct PageCopyParams {
    int n, num_pages, kv_heads;
    long long page_bytes;      // of K or V in one page, all kv heads: a multiple of 16
    int chunks;                // CTAs per pair for K, and as many for V
    uint8_t *k, *v, *k_scale, *v_scale;  // v and the scales may be null
    const int32_t *src, *dst;
    int32_t *status;
};

struct CompactParams {
    int KV, d, batch, max_keep;
    int turn;                  // K is turned
    int rot_start, rd;         // the turned dimensions of K
    int interleaved;
    const int32_t *keep, *keep_lens;
    const uint8_t *from_k, *from_v;      // v may be null (latent rows)
    uint8_t *to_k, *to_v;
    PagedView from, to;
    int to_positions;          // positions of a sequence in `to`
    uint8_t *to_k_scale, *to_v_scale;    // E4M3
    int32_t *status;
};

cudaError_t launch_pages_fork(const ForkParams &p, cudaStream_t stream);
cudaError_t launch_pages_copy(const PageCopyParams &p, cudaStream_t stream);
cudaError_t launch_pages_compact(const CompactParams &p, bool e4m3, const RopeTurns &turns,
                                 cudaStream_t stream);
