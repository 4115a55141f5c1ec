// latent_append.cu -- new tokens' latent rows into their pages, and the rotated parts
// of their queries (na_latent_append_paged).
//
// A CTA per token.  A few hundred bytes to a few KB a token, with three dependent
// rounds of loads (bounds, page id, rows): bound by latency, so every thread
// requests its first elements before it looks for the token's sequence.  The first
// warps turn units of 16 elements (8 pairs) of the H + 1 rotated rows, by one cos and
// sin per pair and token that the first of them leaves in shared memory; the last
// warp norms the latent part, its sum of squares in fp32.  Up to four warps turn, as many as
// there are units for them (8192 tokens of 4 heads: 18.2 us by four, 12.9 by one); up to eight
// where all tokens are on their SMs at once (64 tokens of 32 heads: 3.3 us, 2.8; 1024 of 40
// heads 6.0 by four and 7.2 by six).
#include "latent.cuh"
#include "rope_math.cuh"

namespace {

using namespace rope;

constexpr int MAX_UNIT_THREADS = 256;
constexpr int MANY_TOKENS = 256, MANY_UNIT_THREADS = 128;

template <int R>
__global__ void __launch_bounds__(MAX_UNIT_THREADS + 32)
    latent_append_kernel(const __grid_constant__ LatentAppendParams p,
                         const __grid_constant__ PagedView pg,
                         const __grid_constant__ RopeTurns turns)
{
    __shared__ float4 cos_sin[32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, unit_threads = blockDim.x - 32;
    const int per_row = p.rd / 16, half = p.rd / 2;
    const int units = (p.q ? p.H + 1 : 1) * per_row;
    const bf16 *token = p.kv + t * p.kv_stride;
    // Row 0 is the key's part, row h + 1 head h's.
    auto source = [&](int row) {
        return row == 0 ? token + R : p.q + ((size_t)t * p.H + row - 1) * p.q_stride;
    };
    auto places = [&](int i, int &row, int &e0, int &e1) {
        row = i / per_row;
        const int u = i - row * per_row;
        e0 = p.interleaved ? 16 * u : 8 * u;
        e1 = p.interleaved ? e0 + 8 : e0 + half;
    };
    const bool norm_warp = tid >= unit_threads;
    constexpr int LATENT = R / 32;  // elements per lane: 4, 8 or 16
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    int row = 0, e0 = 0, e1 = 0;
    if (norm_warp) {
        if constexpr (LATENT == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(token + lane * 4));
            x0.x = u.x;
            x0.y = u.y;
        } else {
            x0 = ldg_early(token + lane * 8);
            if constexpr (LATENT == 16)
                x1 = ldg_early(token + 256 + lane * 8);
        }
    } else if (tid < units) {
        places(tid, row, e0, e1);
        const bf16 *src = source(row);
        x0 = *reinterpret_cast<const uint4 *>(src + e0);
        x1 = *reinterpret_cast<const uint4 *>(src + e1);
    }

    RopeAppendParams bounds{};  // what owner_of looks at
    bounds.batch = p.batch;
    bounds.cu_seqlens = p.cu_seqlens;
    bounds.cache_lens = p.cache_lens;
    const int end = __ldg(p.cu_seqlens + p.batch);
    int b, pos;
    owner_of(bounds, t, lane, b, pos);
    if (t >= end)
        return;  // padding behind the last sequence
    if (pos < 0 || pos >= p.capacity) {
        if (tid == 0)
            na_report(p.status, NA_ERR_CAPACITY);
        return;
    }
    const int page = __ldg(pg.table + (size_t)b * pg.pages_per_seq + (pos >> pg.page_log));
    const bool there = (unsigned)page < (unsigned)pg.num_pages;
    bf16 *out = p.cache + (((size_t)max(page, 0) << pg.page_log) +
                           (pos & ((1 << pg.page_log) - 1))) * (R + p.rd);
    if (tid < half)
        cos_sin[tid] = cos_sin_turns((unsigned)pos, turns.hi[tid], turns.lo[tid], kTrig.e);
    if (!there && tid == 0)
        na_report(p.status, NA_ERR_PAGE);
    __syncthreads();

    if (norm_warp) {
        if (!there)
            return;
        if (p.normed) {
            float x[16] = {}, w[16] = {};
            bf16x8_to_f32(x0, x);
            if constexpr (LATENT == 16)
                bf16x8_to_f32(x1, x + 8);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < LATENT; i++)
                sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = 1.0f / sqrtf(sum / R + p.eps);
            if constexpr (LATENT == 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p.norm_w + lane * 4));
                bf16x8_to_f32(make_uint4(u.x, u.y, 0, 0), w);
            } else {
                bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.norm_w + lane * 8)), w);
                if constexpr (LATENT == 16)
                    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.norm_w + 256 + lane * 8)), w + 8);
            }
#pragma unroll
            for (int i = 0; i < LATENT; i++)
                x[i] = x[i] * inv * w[i];
            x0 = f32_to_bf16x8(x);
            x1 = f32_to_bf16x8(x + 8);
        }
        if constexpr (LATENT == 4) {
            *reinterpret_cast<uint2 *>(out + lane * 4) = make_uint2(x0.x, x0.y);
        } else {
            *reinterpret_cast<uint4 *>(out + lane * 8) = x0;
            if constexpr (LATENT == 16)
                *reinterpret_cast<uint4 *>(out + 256 + lane * 8) = x1;
        }
        return;
    }
    for (int i = tid; i < units; i += unit_threads) {
        if (i != tid) {
            places(i, row, e0, e1);
            const bf16 *src = source(row);
            x0 = *reinterpret_cast<const uint4 *>(src + e0);
            x1 = *reinterpret_cast<const uint4 *>(src + e1);
        }
        const float4 *cs = cos_sin + (p.interleaved ? e0 / 2 : e0);
        float a[16], y[16];
        bf16x8_to_f32(x0, a);
        bf16x8_to_f32(x1, a + 8);
        if (p.interleaved) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                rotate_exact(a[2 * k], a[2 * k + 1], cs[k], p.rope_scale, y[2 * k], y[2 * k + 1]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++)
                rotate_exact(a[k], a[8 + k], cs[k], p.rope_scale, y[k], y[8 + k]);
        }
        if (row == 0 && !there)
            continue;
        bf16 *dst = row == 0 ? out + R : p.q_out + ((size_t)t * p.H + row - 1) * p.q_out_stride;
        *reinterpret_cast<uint4 *>(dst + e0) = f32_to_bf16x8(y);
        *reinterpret_cast<uint4 *>(dst + e1) = f32_to_bf16x8(y + 8);
    }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams &p, const PagedView &pg,
                                 const RopeTurns &turns, cudaStream_t stream)
{
    const auto kernel = p.R == 512   ? latent_append_kernel<512>
                        : p.R == 256 ? latent_append_kernel<256>
                                     : latent_append_kernel<128>;
    const int units = (p.q ? p.H + 1 : 1) * (p.rd / 16);
    const int most = p.total_tokens > MANY_TOKENS ? MANY_UNIT_THREADS : MAX_UNIT_THREADS;
    const int unit_threads = units < most ? (units + 31) / 32 * 32 : most;
    return launch_kernel(kernel, dim3(p.total_tokens), dim3(unit_threads + 32), 0, stream, p, pg, turns);
}
