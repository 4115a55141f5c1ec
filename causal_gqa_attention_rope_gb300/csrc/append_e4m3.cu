// append_e4m3.cu -- keys and values of a chunk into E4M3 pages with one
// power-of-two scale per (page, kv head) (na_rope_append_kv_paged).
//
// A page's scale is 2^e with the smallest e such that max |x| <= 448 * 2^e
// over its tokens (448 is E4M3's largest value), so it is known only when all
// of the page's tokens are: one CTA takes one page that the call touches, one
// kv head, and K or V.  Its threads hold the page's new rows in registers --
// normed and rotated in fp32, 16 elements of a row per thread -- agree on the
// largest magnitude, and round once to E4M3.  When the page holds earlier
// tokens of the sequence its scale never shrinks, and when it grows those
// tokens are rounded to the new one: a power of two, so only values that leave
// E4M3's normal range (2^-15 of the page's largest, and below) change.
//
// The kernel moves 3 bytes per element and is bound by latency: bounds, page id
// and rows are one dependent load apart each, so the rows are requested before
// the page id is looked at.
//
// Grid slots.  Sequence b touches at most new_b / page + 2 pages; it owns the
// slots [F(b), F(b + 1)) with F(b) = cu_seqlens[b] / page + 2 b, which hold that
// many, and a CTA finds its sequence by a 32-way search for the last b with
// F(b) <= slot (one round of loads up to 32 sequences, two up to 1024).
#include <cuda_fp16.h>

#include "na_internal.cuh"

namespace {

// cos and sin of 2 pi pos f, f in turns as a 64-bit fraction: the phase is
// exact modulo one turn to 2^-32, its cosine and sine are within ~2e-7, far
// below the 2^-4 of the rounding to E4M3.
__device__ __forceinline__ void cos_sin_phase(int pos, unsigned long long f, float &c, float &s)
{
    const int phase = (int)(((unsigned long long)(unsigned)pos * f) >> 32);
    sincospif((float)phase * 0x1p-31f, &s, &c);
}

// Two fp32 values to E4M3, round to nearest even, saturating; lo in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(const float *y, float mul)
{
    return pack_e4m3x2(y[0] * mul, y[1] * mul) | (pack_e4m3x2(y[2] * mul, y[3] * mul) << 16);
}

// Four E4M3 bytes times `mul`, rounded again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float mul)
{
    uint32_t lo, hi;
    e4m3x4_to_f16(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    const float y[4] = {a.x, a.y, b.x, b.y};
    return pack_e4m3x4(y, mul);
}

// E8M0 byte of the smallest power of two 2^e with amax <= 448 * 2^e
// (448 = 1.75 * 2^8); 0 for a zero or tiny amax.
__device__ __forceinline__ int scale_byte(float amax)
{
    const uint32_t u = __float_as_uint(fminf(amax, 3.4028235e38f));
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, 0);
}

// The page of one CTA: tokens [tok0, tok0 + rows) at positions pos0 ..
struct PageWork {
    int b, page, tok0, pos0, rows;
};

// Finds this slot's work; every warp does so by itself.  False: nothing to do
// (errors reported by one thread of the grid row).
__device__ __forceinline__ bool find_page(const RopeAppendParams &p, const PagedView &pg, int slot,
                                          bool reporter, PageWork &w)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.batch, step;
    int c0 = 0, c1 = 0, prior = 0;
    do {
        step = (n + 31) / 32;
        const int off = lane * step;
        int a0 = 0, a1 = 0, pl = 0;
        bool below = false;
        if (off < n) {
            a0 = __ldg(p.cu_seqlens + lo + off);
            a1 = __ldg(p.cu_seqlens + lo + off + 1);
            pl = __ldg(p.cache_lens + lo + off);
            below = (a0 >> pg.page_log) + 2 * (lo + off) <= slot;
        }
        const unsigned m = __ballot_sync(0xffffffffu, below);
        const int src = m ? 31 - __clz(m) : 0;
        c0 = __shfl_sync(0xffffffffu, a0, src);
        c1 = __shfl_sync(0xffffffffu, a1, src);
        prior = __shfl_sync(0xffffffffu, pl, src);
        lo += src * step;
        n = min(step, n - src * step);
    } while (step > 1);
    const int j = slot - ((c0 >> pg.page_log) + 2 * lo);  // page ordinal within the sequence
    if (c1 <= c0 || j < 0)
        return false;
    if (c0 < 0 || c1 > p.total_tokens) {  // a sequence outside the call's tokens
        if (reporter)
            na_report(p.status, NA_ERR_INVALID_ARG);
        return false;
    }
    if (prior < 0) {
        if (reporter)
            na_report(p.status, NA_ERR_CAPACITY);
        return false;
    }
    const long long page = (prior >> pg.page_log) + (long long)j;
    const long long first = max((long long)prior, page << pg.page_log);
    const long long last = min((long long)prior + (c1 - c0), (page + 1) << pg.page_log);
    if (first >= last)
        return false;
    if (page >= pg.pages_per_seq) {
        if (reporter)
            na_report(p.status, NA_ERR_CAPACITY);
        return false;
    }
    w.b = lo;
    w.page = (int)page;
    w.pos0 = (int)first;
    w.rows = (int)(last - first);
    w.tok0 = c0 + (int)(first - prior);
    return true;
}

// R rows' units of 16 elements per thread: R * NT / (D / 16) rows >= the page.
// Unit k of a rotated row holds the eight pairs 8k .. 8k + 7, then the tail two
// elements per pair slot; GENERIC is the same with rotary_dim not a multiple of
// 16, element by element.
template <int D, int R, int NT, bool GENERIC>
__global__ void __launch_bounds__(NT) kv_append_e4m3_kernel(const RopeAppendParams p,
                                                            const PagedView pg,
                                                            const RopeTurns turns)
{
    constexpr int UPR = D / 16;  // units per row: the row's lanes, aligned in a warp
    __shared__ float warp_max[NT / 32];
    const bool is_v = blockIdx.z != 0;
    const int g = blockIdx.y;
    const int half = p.rd / 2;
    const int k = threadIdx.x % UPR, row0 = threadIdx.x / UPR;
    const bool normed = (p.flags & (is_v ? NA_V_NORM : NA_QK_NORM)) != 0;
    // element of pair slot i: its first and its second
    auto first_of = [&](int i) { return is_v || i >= half ? (is_v ? 2 * i : p.rd + 2 * (i - half)) : i; };
    auto second_of = [&](int i) { return !is_v && i < half ? i + half : first_of(i) + 1; };
    const bool rot = !is_v && 8 * k < half;  // (GENERIC: some slots of the unit may not be)
    unsigned long long f[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        f[i] = rot ? turns.hi[8 * k + i] : 0ull;
    grid_dependency_wait();
    grid_dependents_launch();
    PageWork w;
    if (!find_page(p, pg, blockIdx.x, threadIdx.x == 0 && g == 0 && !is_v, w))
        return;

    // The rows first, then the page id: both loads in flight together.
    const bf16 *src = (is_v ? p.v : p.k) + ((size_t)w.tok0 * p.KV + g) * D;
    const size_t src_stride = (size_t)p.KV * D;
    // two 8-element chunks of a unit (not GENERIC)
    const int ca = rot ? k : 2 * k, cb = rot ? half / 8 + k : 2 * k + 1;
    uint4 xa[R], xb[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = row0 + r * (NT / UPR);
        xa[r] = xb[r] = make_uint4(0, 0, 0, 0);
        if (row < w.rows) {
            const bf16 *x = src + row * src_stride;
            if constexpr (GENERIC) {
                uint16_t h[16];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    h[i] = reinterpret_cast<const uint16_t *>(x)[first_of(8 * k + i)];
                    h[8 + i] = reinterpret_cast<const uint16_t *>(x)[second_of(8 * k + i)];
                }
                auto two = [&](int i) { return (uint32_t)h[i] | ((uint32_t)h[i + 1] << 16); };
                xa[r] = make_uint4(two(0), two(2), two(4), two(6));
                xb[r] = make_uint4(two(8), two(10), two(12), two(14));
            } else {
                xa[r] = __ldg(reinterpret_cast<const uint4 *>(x) + ca);
                xb[r] = __ldg(reinterpret_cast<const uint4 *>(x) + cb);
            }
        }
    }
    const int id = __ldcg(pg.table + (size_t)w.b * pg.pages_per_seq + w.page);
    float wa[8], wb[8];  // norm weights of the unit (K)
    if (!is_v && normed) {
        if constexpr (GENERIC) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                wa[i] = __bfloat162float(p.kw[first_of(8 * k + i)]);
                wb[i] = __bfloat162float(p.kw[second_of(8 * k + i)]);
            }
        } else {
            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.kw) + ca), wa);
            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.kw) + cb), wb);
        }
        if (p.flags & NA_QK_NORM_ZERO_CENTERED) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                wa[i] += 1.0f;
                wb[i] += 1.0f;
            }
        }
    }
    if ((unsigned)id >= (unsigned)pg.num_pages) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_PAGE);
        return;
    }
    uint8_t *scale = const_cast<uint8_t *>(is_v ? pg.v_scale : pg.k_scale) + (size_t)id * p.KV + g;
    const int held = w.pos0 & ((1 << pg.page_log) - 1);  // earlier tokens of the page
    const int old = held ? (int)__ldcg(scale) : 0;

    float ya[R][8], yb[R][8];
    float amax = 0.f;
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = row0 + r * (NT / UPR);
        if (r * (NT / UPR) >= w.rows)  // uniform: no thread has a row left
            break;
        bf16x8_to_f32(xa[r], ya[r]);
        bf16x8_to_f32(xb[r], yb[r]);
        float fr = 1.0f;
        if (normed) {  // every lane shuffles; rows are aligned to UPR lanes
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++)
                ss = fmaf(ya[r][i], ya[r][i], fmaf(yb[r][i], yb[r][i], ss));
#pragma unroll
            for (int o = UPR / 2; o; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            fr = 1.0f / sqrtf(ss / (float)D + p.eps);
            if (!is_v) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    ya[r][i] *= wa[i];
                    yb[r][i] *= wb[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float a = ya[r][i] * fr, b = yb[r][i] * fr;
            if (rot && (!GENERIC || 8 * k + i < half)) {
                float c, s;
                cos_sin_phase(w.pos0 + row, f[i], c, s);
                const float a0 = a, b0 = b;
                a = (a0 * c - b0 * s) * p.rope_scale;
                b = (a0 * s + b0 * c) * p.rope_scale;
            }
            ya[r][i] = a;
            yb[r][i] = b;
            amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));  // rows past the page's: zeros
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0)
        warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; i++)
        amax = fmaxf(amax, warp_max[i]);
    const int now = max(old, scale_byte(amax));

    uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? p.cache_v : p.cache_k);
    uint8_t *page = pool + (((size_t)id * p.KV + g) << pg.page_log) * D;
    if (held && now > old) {
        const int e = 127 + old - now;
        const float shrink = e > 0 ? __uint_as_float((uint32_t)e << 23) : 0.f;
        uint4 *rows = reinterpret_cast<uint4 *>(page);
        for (int i = threadIdx.x; i < held * D / 16; i += NT) {
            uint4 u = __ldcg(rows + i);
            u.x = rescale_e4m3x4(u.x, shrink);
            u.y = rescale_e4m3x4(u.y, shrink);
            u.z = rescale_e4m3x4(u.z, shrink);
            u.w = rescale_e4m3x4(u.w, shrink);
            rows[i] = u;
        }
    }
    const float mul = e8m0_value(254 - now);  // 2^-e
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = row0 + r * (NT / UPR);
        if (row >= w.rows)
            break;
        uint8_t *dst = page + (size_t)(held + row) * D;
        const uint2 a = make_uint2(pack_e4m3x4(ya[r], mul), pack_e4m3x4(ya[r] + 4, mul));
        const uint2 b = make_uint2(pack_e4m3x4(yb[r], mul), pack_e4m3x4(yb[r] + 4, mul));
        if constexpr (GENERIC) {
            const uint32_t q[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int i = 0; i < 8; i++) {
                dst[first_of(8 * k + i)] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
                dst[second_of(8 * k + i)] = (uint8_t)(q[2 + i / 4] >> (8 * (i % 4)));
            }
        } else {
            *reinterpret_cast<uint2 *>(dst + 8 * ca) = a;
            *reinterpret_cast<uint2 *>(dst + 8 * cb) = b;
        }
    }
    if (threadIdx.x == 0)
        *scale = (uint8_t)now;
}

template <int D, int R, int NT>
cudaError_t launch_pages(const RopeAppendParams &p, const PagedView &pg, const RopeTurns &turns,
                         cudaStream_t stream)
{
    const long long slots = (p.total_tokens >> pg.page_log) + 2ll * p.batch;
    const dim3 grid((unsigned)slots, p.KV, 2);
    if (p.rd % 16 == 0)
        return launch_kernel(kv_append_e4m3_kernel<D, R, NT, false>, grid, dim3(NT), 0, stream, p,
                             pg, turns);
    return launch_kernel(kv_append_e4m3_kernel<D, R, NT, true>, grid, dim3(NT), 0, stream, p, pg,
                         turns);
}

}  // namespace

cudaError_t launch_kv_append_e4m3(const RopeAppendParams &p, const PagedView &pg,
                                  const RopeTurns &turns, cudaStream_t stream)
{
    if (p.d == 128) {
        switch (pg.page_log) {
        case 4: return launch_pages<128, 1, 128>(p, pg, turns, stream);
        case 5: return launch_pages<128, 2, 128>(p, pg, turns, stream);
        case 6: return launch_pages<128, 4, 128>(p, pg, turns, stream);
        default: return launch_pages<128, 4, 256>(p, pg, turns, stream);
        }
    }
    switch (pg.page_log) {
    case 4: return launch_pages<64, 1, 64>(p, pg, turns, stream);
    case 5: return launch_pages<64, 1, 128>(p, pg, turns, stream);
    case 6: return launch_pages<64, 2, 128>(p, pg, turns, stream);
    default: return launch_pages<64, 4, 128>(p, pg, turns, stream);
    }
}
