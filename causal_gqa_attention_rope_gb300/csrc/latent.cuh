// latent.cuh -- parameters of the latent attention kernels, filled in by the C ABI
// (latent_api.cu).
#pragma once

#include "na_internal.cuh"

struct LatentAppendParams {
    int H, R, rd, batch, capacity, total_tokens;
    int normed, interleaved;
    float eps, rope_scale;
    const int32_t *cu_seqlens, *cache_lens;
    const bf16 *kv, *q, *norm_w;
    bf16 *q_out, *cache;
    long long kv_stride, q_stride, q_out_stride;  // elements
    int32_t *status;
};

struct LatentParams {
    int H, R, rd, batch, capacity;
    float scale_log2;          // score scale * log2(e)
    int total_tokens, max_new_len, max_total_len;
    int unit_rows;             // 32, 64 or 128 (R > 128)
    int grid;                  // CTAs (pairs of them for 128 rows), each with an equal run of key tiles
    int cut_by_sequence;       // one unit a sequence: cut[b], else by run
    int pieces;                // > 0: no runs; `grid` units (of all sequences, with the longest
                               // one's each), a cluster of that many CTAs each, 32 or 64 rows
    const int32_t *cu_seqlens, *cache_lens;
    const bf16 *q, *cache;
    bf16 *out;
    float *part_o;             // [2 grid][unit_rows][R]: rows of a cut unit, run c's first piece at 2 c
    float *part_ml;            // [2 grid][unit_rows][2]: (max, sum), log2 domain
    int4 *cut;                 // [grid]: first row, rows, first and last run of a unit (last -1: not cut);
                               // by sequence, written only where a unit's first piece is done
    int32_t *status;
};

struct ExpandedParams {
    int H, dn, rd, dv, batch;
    float scale_log2;
    int total_tokens, total_keys, max_new_len, max_key_len;
    int tall;                  // units of 256 rows, else of 128
    int units;                 // of all sequences, with the longest one's tiles each
    int sms, in_turn;          // tall: CTAs that run at a time, and whether each takes units in turn
    int cut_units, pieces;     // tall: the last units, cut into pieces of their keys (a cluster each)
    const int32_t *cu_seqlens, *key_starts, *key_lens;
    const bf16 *q, *kv, *k_pe;
    long long k_pe_stride;     // elements
    bf16 *out;
    int32_t *status;
};

// Query rows (token, head) of a unit: enough for those of any sequence, 128 (64 in each of a
// pair of CTAs) at most, 64 with 128 latent numbers, which pairs do not split.
inline int latent_unit_rows(long long most_rows, int kv_rank)
{
    return most_rows <= 32 ? 32 : (most_rows <= 64 || kv_rank == 128 ? 64 : 128);
}
// Whether an entry of `cut` names runs of the call.  One whose kernel gave a wait up (and reported it)
// was not written: it is whatever the workspace held, and nothing may be addressed by it.
__host__ __device__ inline bool names_runs(const int4 &cut, int grid)
{
    return cut.z >= 0 && cut.z <= cut.w && cut.w < grid;
}
constexpr int kLatentKeys = 64;  // keys of a tile
constexpr int kLatentMaxPieces = 8;  // CTAs of a cluster
constexpr int kExpandedMaxPieces = 8;  // CTAs of a cluster
constexpr int kExpandedRows = 128;  // query tokens of an expanded tile; a tall unit has two

cudaError_t launch_latent_append(const LatentAppendParams &p, const PagedView &pg,
                                 const RopeTurns &turns, cudaStream_t stream);
cudaError_t launch_latent(const LatentParams &p, const PagedView &pg, cudaStream_t stream);
// Clusters of that many CTAs, one per SM, that the device runs at a time.
int sm_clusters(int ctas);
// Absorbed attention in units of 128 rows, kv_rank 256 and 512, without the second pass.
cudaError_t launch_latent_pair(const LatentParams &p, const PagedView &pg, cudaStream_t stream);
cudaError_t launch_latent_expanded(const ExpandedParams &p, cudaStream_t stream);
