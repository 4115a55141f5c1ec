// append_paged.cu -- a chunk's queries, keys and values into a paged cache, in
// one launch (na_rope_append_kv_paged).  Two kinds of CTA share the grid.
//
// Rows: q (and with bf16 pages k and v), arithmetic as in rope_append.cu.  A CTA
// takes NT / 64 tokens: its threads request 16 elements of up to P rows each
// before anything else, find the tokens' sequences and pages, compute one cos
// and sin each (all pairs of all tokens of the CTA) into shared memory, and
// rotate.  The rows of a token are then served by one cos and sin per pair
// instead of one per pair and 8 rows, and the loads of P rows are in flight at
// once.  Few tokens take P = 1 and one token per CTA, for more CTAs.
// (2048 tokens of 40 query heads, d 128: 15.1 us with the E4M3 pages of 8
// kv heads, against 17.7 + 9.1 us as two launches with 64-thread CTAs per row
// group.)
//
// E4M3 pages.  A page's scale is 2^e with the smallest e such that max |x| <=
// 448 * 2^e over its tokens (448 is E4M3's largest value), so it is known only
// when all of the page's tokens are: one CTA takes one page that the call
// touches, one kv head, and K or V.  Its threads norm and rotate the page's new
// rows in fp32, 16 elements of a row per thread, leave them in shared memory, agree
// on the largest magnitude, and round once to E4M3.  (In a call of a token or two
// per sequence a warp does this, its rows in registers.)  When the page holds
// earlier tokens of the sequence its scale never shrinks, and when it grows
// those tokens are rounded to the new one: a power of two, so only values that
// leave E4M3's normal range (2^-15 of the page's largest, and below) change.
//
// Both move a few bytes per element and are bound by latency: bounds, page id
// and rows are one dependent load apart each, so the rows are requested before
// the others are looked at.
//
// Page slots.  Sequence b touches at most new_b / page + 2 pages; it owns the
// slots [F(b), F(b + 1)) with F(b) = cu_seqlens[b] / page + 2 b, which hold that
// many, and a CTA finds its sequence by a 32-way search for the last b with
// F(b) <= slot (one round of loads up to 32 sequences, two up to 1024).
#include <cuda_fp16.h>

#include "na_internal.cuh"
#include "rope_math.cuh"

namespace {

using namespace rope;

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

__device__ __forceinline__ uint32_t pack_e4m3x4(float4 y, float mul)
{
    return pack_e4m3x2(y.x * mul, y.y * mul) | (pack_e4m3x2(y.z * mul, y.w * mul) << 16);
}

// Four E4M3 bytes times `mul`, rounded again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float mul)
{
    uint32_t lo, hi;
    e4m3x4_to_f16(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack_e4m3x4(make_float4(a.x, a.y, b.x, b.y), mul);
}

// E8M0 byte of the smallest power of two 2^e with amax <= 448 * 2^e
// (448 = 1.75 * 2^8); 0 for a zero or tiny amax.
__device__ __forceinline__ int scale_byte(float amax)
{
    const uint32_t u = __float_as_uint(fminf(amax, 3.4028235e38f));
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, 0);
}

// Rows of a GENERIC call (rotary_dim no multiple of 16) pass through shared memory
// between the 16 consecutive elements that a lane loads or stores and the eight
// pairs, rd / 2 apart, that it rotates: a row's UPR lanes sit in one warp, and a
// row is an odd number of words, so that the four rows of a warp miss each other's
// banks.  (2048 tokens of 40/8 heads, E4M3 pages, rotary_dim 34: 23 us; 48 with
// the queries staged by rope_append.cu and the pages element by element from global
// memory; rotary_dim 64 takes 15.)
template <int D, int NT>
struct RowStage {
    uint32_t words[NT / (D / 16)][D / 2 + 1];
};

// Element of pair slot i, its first and its second: (i, i + half) of the rotated
// ones, then the tail two by two.
__device__ __forceinline__ int slot_first(int i, int half) { return i < half ? i : 2 * i; }
__device__ __forceinline__ int slot_second(int i, int half) { return i < half ? i + half : 2 * i + 1; }

// A lane's chunks 2 k and 2 k + 1 in, its eight slots out (called by whole warps).
__device__ __forceinline__ void stage_in(uint32_t *row, int k, int half, uint4 xa, uint4 xb,
                                         float (&a)[8], float (&c)[8])
{
    __syncwarp();  // the reads of what was here
    const uint32_t x[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
    for (int j = 0; j < 8; j++)
        row[8 * k + j] = x[j];
    __syncwarp();
    const bf16 *el = reinterpret_cast<const bf16 *>(row);
#pragma unroll
    for (int e = 0; e < 8; e++) {
        a[e] = __bfloat162float(el[slot_first(8 * k + e, half)]);
        c[e] = __bfloat162float(el[slot_second(8 * k + e, half)]);
    }
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

// One unit of a row at position pos, normed and rotated in place; its largest
// magnitude.  The row's other lanes run with it.  (GENERIC: the unit's first `pairs`
// slots are rotated.)
template <int D, bool GENERIC>
__device__ __forceinline__ float unit_values(const RopeAppendParams &p, float (&ya)[8], float (&yb)[8],
                                             const float (&wa)[8], const float (&wb)[8],
                                             const unsigned long long (&f)[8], int pos, bool is_v,
                                             bool normed, bool rot, int pairs)
{
    float fr = 1.0f, amax = 0.f;
    if (normed) {  // every lane shuffles; rows are aligned to their lanes
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++)
            ss = fmaf(ya[i], ya[i], fmaf(yb[i], yb[i], ss));
#pragma unroll
        for (int o = D / 32; o; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        fr = 1.0f / sqrtf(ss / (float)D + p.eps);
        if (!is_v) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                ya[i] *= wa[i];
                yb[i] *= wb[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float a = ya[i] * fr, b = yb[i] * fr;
        if (rot && (!GENERIC || i < pairs)) {
            float c, s;
            cos_sin_phase(pos, f[i], c, s);
            const float a0 = a, b0 = b;
            a = (a0 * c - b0 * s) * p.rope_scale;
            b = (a0 * s + b0 * c) * p.rope_scale;
        }
        ya[i] = a;
        yb[i] = b;
        amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
    }
    return amax;
}

// Earlier tokens of a page, rounded to its new scale: 16 bytes a thread.
__device__ __forceinline__ void rescale_held(uint8_t *page, int bytes, int old, int now, int thread,
                                             int threads)
{
    const int e = 127 + old - now;
    const float shrink = e > 0 ? __uint_as_float((uint32_t)e << 23) : 0.f;
    uint4 *rows = reinterpret_cast<uint4 *>(page);
    for (int i = thread; i < bytes / 16; i += threads) {
        uint4 u = __ldcg(rows + i);
        u.x = rescale_e4m3x4(u.x, shrink);
        u.y = rescale_e4m3x4(u.y, shrink);
        u.z = rescale_e4m3x4(u.z, shrink);
        u.w = rescale_e4m3x4(u.w, shrink);
        rows[i] = u;
    }
}

// The work of a page CTA (below) by one warp, for calls of a token or two per
// sequence: four pages to a CTA instead of one CTA of which one row's lanes have
// work (64 single tokens, 8 kv heads, d 128, pages of 64: 4.4 us, 8.5 by CTAs).  The
// first 32 / (D / 16) rows stay in registers; should a page get more they are
// computed twice, for the scale and for the bytes.
template <int D>
__device__ __forceinline__ void append_page_warp(const RopeAppendParams &p, const PagedView &pg,
                                                 const RopeTurns &turns, int slot, int g, bool is_v)
{
    constexpr int UPR = D / 16, RP = 32 / UPR;
    const int lane = threadIdx.x & 31, half = p.rd / 2;
    const int k = lane % UPR, row0 = lane / UPR;
    const bool normed = (p.flags & (is_v ? NA_V_NORM : NA_QK_NORM)) != 0;
    const bool rot = !is_v && 8 * k < half;
    unsigned long long f[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        f[i] = rot ? turns.hi[8 * k + i] : 0ull;
    grid_dependency_wait();
    grid_dependents_launch();
    PageWork w;
    if (!find_page(p, pg, slot, lane == 0 && g == 0 && !is_v, w))
        return;
    const bf16 *src = (is_v ? p.v : p.k) + ((size_t)w.tok0 * p.KV + g) * D;
    const int ca = rot ? k : 2 * k, cb = rot ? half / 8 + k : 2 * k + 1;
    auto load = [&](int row, float (&ya)[8], float (&yb)[8]) {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (row < w.rows) {
            const uint4 *x = reinterpret_cast<const uint4 *>(src + (size_t)row * p.KV * D);
            a = __ldg(x + ca);
            b = __ldg(x + cb);
        }
        bf16x8_to_f32(a, ya);
        bf16x8_to_f32(b, yb);
    };
    const int id = __ldcg(pg.table + (size_t)w.b * pg.pages_per_seq + w.page);
    float ya[8], yb[8], wa[8], wb[8];
    load(row0, ya, yb);
    if (!is_v && normed) {
        bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.kw) + ca), wa);
        bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.kw) + cb), wb);
        if (p.flags & NA_QK_NORM_ZERO_CENTERED) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                wa[i] += 1.0f;
                wb[i] += 1.0f;
            }
        }
    }
    if ((unsigned)id >= (unsigned)pg.num_pages) {
        if (lane == 0)
            na_report(p.status, NA_ERR_PAGE);
        return;
    }
    uint8_t *scale = const_cast<uint8_t *>(is_v ? pg.v_scale : pg.k_scale) + (size_t)id * p.KV + g;
    const int held = w.pos0 & ((1 << pg.page_log) - 1);  // earlier tokens of the page
    const int old = held ? (int)__ldcg(scale) : 0;
    auto values = [&](int row, float (&a)[8], float (&b)[8]) {
        return unit_values<D, false>(p, a, b, wa, wb, f, w.pos0 + row, is_v, normed, rot, 8);
    };
    float amax = values(row0, ya, yb);
    for (int r = RP; r < w.rows; r += RP) {
        float ta[8], tb[8];
        load(r + row0, ta, tb);
        amax = fmaxf(amax, values(r + row0, ta, tb));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int now = max(old, scale_byte(amax));
    uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? p.cache_v : p.cache_k);
    uint8_t *page = pool + (((size_t)id * p.KV + g) << pg.page_log) * D;
    if (held && now > old)
        rescale_held(page, held * D, old, now, lane, 32);
    const float mul = e8m0_value(254 - now);  // 2^-e
    auto store = [&](int row, const float (&a)[8], const float (&b)[8]) {
        if (row >= w.rows)
            return;
        uint8_t *dst = page + (size_t)(held + row) * D;
        *reinterpret_cast<uint2 *>(dst + 8 * ca) =
            make_uint2(pack_e4m3x4(make_float4(a[0], a[1], a[2], a[3]), mul),
                       pack_e4m3x4(make_float4(a[4], a[5], a[6], a[7]), mul));
        *reinterpret_cast<uint2 *>(dst + 8 * cb) =
            make_uint2(pack_e4m3x4(make_float4(b[0], b[1], b[2], b[3]), mul),
                       pack_e4m3x4(make_float4(b[4], b[5], b[6], b[7]), mul));
    };
    store(row0, ya, yb);
    for (int r = RP; r < w.rows; r += RP) {
        float ta[8], tb[8];
        load(r + row0, ta, tb);
        values(r + row0, ta, tb);
        store(r + row0, ta, tb);
    }
    if (lane == 0)
        *scale = (uint8_t)now;
}

// R rows' units of 16 elements per thread: R * NT / (D / 16) rows >= the page.
// Unit k of a rotated row holds the eight pairs 8k .. 8k + 7, then the tail two
// elements per pair slot.
template <int D, int R, int NT, bool GENERIC>
__device__ __forceinline__ void append_page(const RopeAppendParams &p, const PagedView &pg,
                                            const RopeTurns &turns, RowStage<D, NT> *stage,
                                            int slot, int g, bool is_v)
{
    constexpr int UPR = D / 16;  // units per row: the row's lanes, aligned in a warp
    __shared__ float warp_max[NT / 32];
    const int half = p.rd / 2;
    const int k = threadIdx.x % UPR, row0 = threadIdx.x / UPR;
    const bool normed = (p.flags & (is_v ? NA_V_NORM : NA_QK_NORM)) != 0;
    const int pairs = is_v ? 0 : half;  // a V row's slots are all tail
    const bool rot = !is_v && 8 * k < half;  // (GENERIC: some slots of the unit may not be)
    unsigned long long f[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        f[i] = rot ? turns.hi[8 * k + i] : 0ull;
    grid_dependency_wait();
    grid_dependents_launch();
    PageWork w;
    if (!find_page(p, pg, slot, threadIdx.x == 0 && g == 0 && !is_v, w))
        return;

    // The rows first, then the page id: both loads in flight together.
    const bf16 *src = (is_v ? p.v : p.k) + ((size_t)w.tok0 * p.KV + g) * D;
    const size_t src_stride = (size_t)p.KV * D;
    // two 8-element chunks of a unit
    const int ca = rot && !GENERIC ? k : 2 * k, cb = rot && !GENERIC ? half / 8 + k : 2 * k + 1;
    uint4 xa[R], xb[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = row0 + r * (NT / UPR);
        xa[r] = xb[r] = make_uint4(0, 0, 0, 0);
        if (row < w.rows) {
            const bf16 *x = src + row * src_stride;
            xa[r] = __ldg(reinterpret_cast<const uint4 *>(x) + ca);
            xb[r] = __ldg(reinterpret_cast<const uint4 *>(x) + cb);
        }
    }
    const int id = __ldcg(pg.table + (size_t)w.b * pg.pages_per_seq + w.page);
    float wa[8], wb[8];  // norm weights of the unit (K)
    if (!is_v && normed) {
        if constexpr (GENERIC) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                wa[i] = __bfloat162float(p.kw[slot_first(8 * k + i, half)]);
                wb[i] = __bfloat162float(p.kw[slot_second(8 * k + i, half)]);
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

    // The values wait in shared memory for the page's scale (in registers they
    // would cost the row CTAs of the launch their occupancy): [unit's quad][thread].
    extern __shared__ float4 vals[];
    auto at = [&](int r, int q) -> float4 & { return vals[(r * 4 + q) * NT + threadIdx.x]; };
    float amax = 0.f;
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = row0 + r * (NT / UPR);
        if (r * (NT / UPR) >= w.rows)  // uniform: no thread has a row left
            break;
        float ya[8], yb[8];
        if constexpr (GENERIC) {
            stage_in(stage->words[row0], k, pairs, xa[r], xb[r], ya, yb);
        } else {
            bf16x8_to_f32(xa[r], ya);
            bf16x8_to_f32(xb[r], yb);
        }
        amax = fmaxf(amax, unit_values<D, GENERIC>(p, ya, yb, wa, wb, f, w.pos0 + row, is_v, normed, rot,
                                                  half - 8 * k));
        at(r, 0) = make_float4(ya[0], ya[1], ya[2], ya[3]);
        at(r, 1) = make_float4(ya[4], ya[5], ya[6], ya[7]);
        at(r, 2) = make_float4(yb[0], yb[1], yb[2], yb[3]);
        at(r, 3) = make_float4(yb[4], yb[5], yb[6], yb[7]);
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
    if (held && now > old)
        rescale_held(page, held * D, old, now, threadIdx.x, NT);
    const float mul = e8m0_value(254 - now);  // 2^-e
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int row = row0 + r * (NT / UPR);
        if (GENERIC ? r * (NT / UPR) >= w.rows : row >= w.rows)  // (GENERIC: whole warps go on)
            break;
        uint8_t *dst = page + (size_t)(held + row) * D;
        const uint2 a = make_uint2(pack_e4m3x4(at(r, 0), mul), pack_e4m3x4(at(r, 1), mul));
        const uint2 b = make_uint2(pack_e4m3x4(at(r, 2), mul), pack_e4m3x4(at(r, 3), mul));
        if constexpr (GENERIC) {
            __syncwarp();
            uint32_t *words = stage->words[row0];
            uint8_t *bytes = reinterpret_cast<uint8_t *>(words);
            const uint32_t q[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int i = 0; i < 8; i++) {
                bytes[slot_first(8 * k + i, pairs)] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
                bytes[slot_second(8 * k + i, pairs)] = (uint8_t)(q[2 + i / 4] >> (8 * (i % 4)));
            }
            __syncwarp();
            if (row < w.rows)
                *reinterpret_cast<uint4 *>(dst + 16 * k) =
                    make_uint4(words[4 * k], words[4 * k + 1], words[4 * k + 2], words[4 * k + 3]);
        } else {
            *reinterpret_cast<uint2 *>(dst + 8 * ca) = a;
            *reinterpret_cast<uint2 *>(dst + 8 * cb) = b;
        }
    }
    if (threadIdx.x == 0)
        *scale = (uint8_t)now;
}

constexpr int kManyRowCtas = 608;  // four per SM

// Page CTAs of a call: (slot, kv head, K or V).
long long page_ctas(const RopeAppendParams &p, const PagedView &pg)
{
    return ((p.total_tokens >> pg.page_log) + 2ll * p.batch) * p.KV * 2;
}

template <int D, int R, int NT, bool GENERIC>
__device__ __forceinline__ void append_page_cta(const RopeAppendParams &p, const PagedView &pg,
                                                const RopeTurns &turns, RowStage<D, NT> *stage,
                                                int i)
{
    const int per = 2 * p.KV, slot = i / per, rest = i - slot * per;
    append_page<D, R, NT, GENERIC>(p, pg, turns, stage, slot, rest >> 1, rest & 1);
}

// Where a token's rows go.
struct RowPlace {
    int pos;        // < 0: the token is skipped
    int id, slot;   // bf16 pages: its page and slot there
};

// rotate_exact (rope_math.cuh) of two pairs at a time on packed fp32 operations:
// the same products, sums and roundings, -a1 standing in for the subtractions.
// c: cos hi, hi, lo, lo of the two pairs; s: sin likewise.
__device__ __forceinline__ void rotate_exact2(float2 a0, float2 a1, float4 c, float4 s, float2 fr,
                                              float2 &y0, float2 &y1)
{
    const float2 na1 = make_float2(-a1.x, -a1.y);
    const float2 ch = make_float2(c.x, c.y), cl = make_float2(c.z, c.w);
    const float2 sh = make_float2(s.x, s.y), sl = make_float2(s.z, s.w);
    {
        const float2 t = __fmul2_rn(a1, sh), nt = __fmul2_rn(na1, sh);
        const float2 ne = __ffma2_rn(na1, sh, t);  // minus the rounding error of t
        const float2 h = __ffma2_rn(a0, ch, nt);
        const float2 lo = __fadd2_rn(__ffma2_rn(a0, cl, __fmul2_rn(na1, sl)), ne);
        y0 = __ffma2_rn(h, fr, __fmul2_rn(lo, fr));
    }
    {
        const float2 t = __fmul2_rn(a1, ch), nt = __fmul2_rn(na1, ch);
        const float2 e = __ffma2_rn(a1, ch, nt);
        const float2 h = __ffma2_rn(a0, sh, t);
        const float2 lo = __fadd2_rn(__ffma2_rn(a0, sl, __fmul2_rn(a1, cl)), e);
        y1 = __ffma2_rn(h, fr, __fmul2_rn(lo, fr));
    }
}

// The rows of TK tokens from token t0 on: P of them per thread group from row
// slot first on (row slots run token after token).
template <int D, int NT, int P, int TK, bool E4M3, bool GENERIC>
__device__ __forceinline__ void append_rows(const RopeAppendParams &p, const PagedView &pg,
                                            const RopeTurns &turns, RowStage<D, NT> *stage, int t0,
                                            int first)
{
    constexpr int UPR = D / 16, RP = NT / UPR;  // 32-byte units per row, rows per pass
    // cos (and sin) hi, hi, lo, lo of pairs 8 k + 2 j and the next: [2 j (+ 1)][k]
    __shared__ float4 cs[TK][64];
    __shared__ RowPlace place[TK];
    const int H = p.H, KV = E4M3 ? 0 : p.KV, rows = H + 2 * KV;
    const int half = p.rd / 2, lane = threadIdx.x & 31;
    const int k = threadIdx.x % UPR;
    // GENERIC rows of bf16 pages come without norms (launch_rope_append_paged sends those
    // with norms to the staged kernel)
    constexpr bool NORMS = !GENERIC || E4M3;
    const bool qk_norm = NORMS && (p.flags & NA_QK_NORM) != 0;
    const bool zero_centered = (p.flags & NA_QK_NORM_ZERO_CENTERED) != 0;
    const bool v_norm = NORMS && !E4M3 && (p.flags & NA_V_NORM) != 0;
    const int ntok = min(TK, p.total_tokens - t0);
    const bool rot = GENERIC ? 8 * k < half : k < p.rd / 16;
    // 16-byte chunks of a unit: of a rotated row, and of a V row
    const int qa = rot && !GENERIC ? k : 2 * k, qb = rot && !GENERIC ? half / 8 + k : 2 * k + 1;

    // this thread's cos and sin: pair `pair` of token `tk`
    const int tk = TK == 1 ? 0 : threadIdx.x / 64, pair = threadIdx.x & 63;
    const bool trig = (TK > 1 || threadIdx.x < 64) && pair < half;
    const unsigned long long fhi = trig ? turns.hi[pair] : 0ull;
    const unsigned int flo = trig ? turns.lo[pair] : 0u;
    grid_dependency_wait();
    grid_dependents_launch();

    // Row slot first + i RP + thread / UPR: its token (of the CTA) and row.
    auto row_at = [&](int i, int &t, int &r) {
        r = first + i * RP + threadIdx.x / UPR;
        t = 0;
#pragma unroll
        for (int u = 1; u < TK; u++)
            if (r >= rows) {
                r -= rows;
                t = u;
            }
        return t < ntok && r < rows;
    };
    uint4 xa[P], xb[P];
#pragma unroll
    for (int i = 0; i < P; i++) {
        int t, r;
        xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
        if (row_at(i, t, r)) {
            const size_t tok = (size_t)(t0 + t);
            const bf16 *src;
            const bool is_v = !E4M3 && r >= H + KV;
            if (E4M3 || r < H)
                src = p.q + (tok * H + r) * D;
            else
                src = is_v ? p.v + (tok * KV + (r - H - KV)) * D : p.k + (tok * KV + (r - H)) * D;
            xa[i] = ldg_early(reinterpret_cast<const uint4 *>(src) + (is_v ? 2 * k : qa));
            xb[i] = ldg_early(reinterpret_cast<const uint4 *>(src) + (is_v ? 2 * k + 1 : qb));
        }
    }
    int pos = -1;
    if (tk < ntok) {  // a warp's threads share tk
        const int end = __ldg(p.cu_seqlens + p.batch);  // rows behind it are left alone
        int b;
        owner_of(p, t0 + tk, lane, b, pos);
        int id = 0;
        if (t0 + tk >= end) {
            pos = -1;
        } else if (pos < 0 || pos >= p.capacity) {
            if (lane == 0)
                na_report(p.status, NA_ERR_CAPACITY);
            pos = -1;
        } else if constexpr (!E4M3) {
            id = __ldcg(pg.table + (size_t)b * pg.pages_per_seq + (pos >> pg.page_log));
            if ((unsigned)id >= (unsigned)pg.num_pages) {
                if (lane == 0)
                    na_report(p.status, NA_ERR_PAGE);
                pos = -1;
            }
        }
        if (pair == 0)
            place[tk] = RowPlace{pos, id, pos & ((1 << pg.page_log) - 1)};
        if (trig && pos >= 0) {
            const float4 x = cos_sin_turns((unsigned)pos, fhi, flo, kTrig.e);
            float *c = reinterpret_cast<float *>(&cs[tk][(pair & 6) * 8 + (pair >> 3)]) + (pair & 1);
            c[0] = x.x;
            c[2] = x.y;
            c[32] = x.z;
            c[34] = x.w;
        }
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < P; i++) {
        int t, r;
        const bool active = row_at(i, t, r);
        const bool is_v = !E4M3 && r >= H + KV;
        float a[8], c[8];
        if constexpr (GENERIC) {
            stage_in(stage->words[threadIdx.x / UPR], k, is_v ? 0 : half, xa[i], xb[i], a, c);
        } else {
            bf16x8_to_f32(xa[i], a);
            bf16x8_to_f32(xb[i], c);
        }
        // (GENERIC: a rotated unit's slots from `half` on are plain)
        auto turned = [&](int e) { return rot && (!GENERIC || 8 * k + e < half); };
        float f = 1.0f;
        if (qk_norm || v_norm) {  // every lane shuffles; rows are aligned to UPR lanes
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e++)
                ss = fmaf(a[e], a[e], fmaf(c[e], c[e], ss));
#pragma unroll
            for (int o = UPR / 2; o; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (is_v ? v_norm : qk_norm)
                f = 1.0f / sqrtf(ss / (float)D + p.eps);
        }
        const RowPlace pl = place[t];
        const bool written = active && pl.pos >= 0;
        if (!GENERIC && !written)
            continue;  // (GENERIC: whole warps go on)
        float ya[8], yb[8];
        if (is_v) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                ya[e] = a[e] * f;
                yb[e] = c[e] * f;
            }
        } else {
            const float4 *trig_row = cs[t] + k;
            const float fr = f * p.rope_scale;  // the attention factor scales rotated dims only
            float wa[8], wb[8];
            if (qk_norm) {
                const uint4 *w = reinterpret_cast<const uint4 *>(E4M3 || r < H ? p.qw : p.kw);
                if constexpr (GENERIC) {
                    const bf16 *el = reinterpret_cast<const bf16 *>(w);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        wa[e] = __bfloat162float(el[slot_first(8 * k + e, half)]);
                        wb[e] = __bfloat162float(el[slot_second(8 * k + e, half)]);
                    }
                } else {
                    bf16x8_to_f32(__ldg(w + qa), wa);
                    bf16x8_to_f32(__ldg(w + qb), wb);
                }
            }
            // (rows that never have norms take this way too, without weights: it has the bits
            // of the contiguous call's staged rows)
            if ((qk_norm && zero_centered) || !NORMS) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    F2 x0{a[e], 0.f}, x1{c[e], 0.f};
                    if (qk_norm) {
                        x0 = weighted(a[e], wa[e], zero_centered);
                        x1 = weighted(c[e], wb[e], zero_centered);
                    }
                    if (turned(e)) {
                        const float *tr = reinterpret_cast<const float *>(trig_row + (e & 6) * 8) + (e & 1);
                        rotate(x0, x1, make_float4(tr[0], tr[2], tr[32], tr[34]), fr, ya[e], yb[e]);
                    } else {
                        ya[e] = fmaf(x0.hi, f, x0.lo * f);
                        yb[e] = fmaf(x1.hi, f, x1.lo * f);
                    }
                }
            } else {
                if (qk_norm) {  // x * w of two bf16 values is exact in fp32
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        a[e] *= wa[e];
                        c[e] *= wb[e];
                    }
                }
                if (rot) {
                    const float2 fr2 = make_float2(fr, fr);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        float2 y0, y1;
                        rotate_exact2(make_float2(a[e], a[e + 1]), make_float2(c[e], c[e + 1]),
                                      trig_row[e * 8], trig_row[e * 8 + 8], fr2, y0, y1);
                        ya[e] = turned(e) ? y0.x : a[e] * f;
                        ya[e + 1] = turned(e + 1) ? y0.y : a[e + 1] * f;
                        yb[e] = turned(e) ? y1.x : c[e] * f;
                        yb[e + 1] = turned(e + 1) ? y1.y : c[e + 1] * f;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        ya[e] = a[e] * f;
                        yb[e] = c[e] * f;
                    }
                }
            }
        }
        bf16 *dst;
        if (E4M3 || r < H)
            dst = p.q_out + ((size_t)(t0 + t) * H + r) * D;
        else
            dst = (is_v ? p.cache_v : p.cache_k) +
                  ((((size_t)pl.id * KV + (is_v ? r - H - KV : r - H)) << pg.page_log) + pl.slot) * D;
        if constexpr (GENERIC) {
            __syncwarp();
            uint32_t *words = stage->words[threadIdx.x / UPR];
            bf16 *el = reinterpret_cast<bf16 *>(words);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                el[slot_first(8 * k + e, is_v ? 0 : half)] = __float2bfloat16_rn(ya[e]);
                el[slot_second(8 * k + e, is_v ? 0 : half)] = __float2bfloat16_rn(yb[e]);
            }
            __syncwarp();
            const uint32_t *x = words + 8 * k;
            if (written) {
                reinterpret_cast<uint4 *>(dst)[2 * k] = make_uint4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<uint4 *>(dst)[2 * k + 1] = make_uint4(x[4], x[5], x[6], x[7]);
            }
        } else {
            reinterpret_cast<uint4 *>(dst)[is_v ? 2 * k : qa] = f32_to_bf16x8(ya);
            reinterpret_cast<uint4 *>(dst)[is_v ? 2 * k + 1 : qb] = f32_to_bf16x8(yb);
        }
    }
}

// Page CTAs first (E4M3): theirs is the longer chain of dependent loads.
// FEW: a warp each.
// 768 threads per SM hold a thread to 80 registers, where the instances with most to
// hold spill (-Xptxas -v, bytes of stores / loads): R = 4 page rows 52 / 172 with
// P = 2 row units, 72 / 184 with four; P = 4 alone 16 / 20 to 24 / 28; a warp per page
// 64 / 72; GENERIC up to 20 / 68; R and P up to two, and bf16 pages up to P = 2, none.
template <int D, bool E4M3, int R, int NT, int P, bool GENERIC, bool FEW>
__global__ void __launch_bounds__(NT, 768 / NT) append_paged_kernel(const RopeAppendParams p,
                                                          const PagedView pg, const RopeTurns turns,
                                                          const int n_page_ctas,
                                                          const int ctas_per_group)
{
    constexpr int TK = P == 1 ? 1 : NT / 64, RP = NT / (D / 16);
    int i = blockIdx.x;
    RowStage<D, NT> *stage = nullptr;
    if constexpr (GENERIC) {
        __shared__ RowStage<D, NT> rows;
        stage = &rows;
    }
    if constexpr (E4M3) {
        if (i < n_page_ctas) {
            if constexpr (FEW) {
                const int per = 2 * p.KV, item = i * (NT / 32) + threadIdx.x / 32;
                const int slot = item / per, rest = item - slot * per;
                append_page_warp<D>(p, pg, turns, slot, rest >> 1, rest & 1);
            } else {
                append_page_cta<D, R, NT, GENERIC>(p, pg, turns, stage, i);
            }
            return;
        }
        i -= n_page_ctas;
    }
    const int group = i / ctas_per_group, part = i - group * ctas_per_group;
    append_rows<D, NT, P, TK, E4M3, GENERIC>(p, pg, turns, stage, group * TK, part * P * RP);
}

// Shared memory of the page CTAs, granted to `kernel` once per device where it
// is more than the default.
template <int R, int NT, typename Kernel>
cudaError_t grant_smem(Kernel kernel, std::atomic<unsigned long long> &done)
{
    constexpr int bytes = R * NT * 64;
    if (bytes <= 48 * 1024)
        return cudaSuccess;
    return once_per_device(done, [kernel] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
}

template <int D, bool E4M3, int R, int NT, int P, bool GENERIC, bool FEW = false>
cudaError_t launch_fused(const RopeAppendParams &p, const PagedView &pg, const RopeTurns &turns,
                         cudaStream_t stream)
{
    constexpr int TK = P == 1 ? 1 : NT / 64, RP = NT / (D / 16);
    const int rows = p.H + (E4M3 ? 0 : 2 * p.KV);
    const long long groups = (p.total_tokens + TK - 1) / TK;
    const int per = (TK * rows + P * RP - 1) / (P * RP);
    long long pages = E4M3 ? page_ctas(p, pg) : 0;
    if (FEW)  // (a last warp without a slot finds no work)
        pages = (pages + NT / 32 - 1) / (NT / 32);
    if (pages + groups * per > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    static std::atomic<unsigned long long> granted{0};
    const size_t smem = E4M3 && !FEW ? R * NT * 64 : 0;
    const cudaError_t e = grant_smem<E4M3 && !FEW ? R : 0, NT>(append_paged_kernel<D, E4M3, R, NT, P, GENERIC, FEW>, granted);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(append_paged_kernel<D, E4M3, R, NT, P, GENERIC, FEW>, dim3((unsigned)(pages + groups * per)),
                         dim3(NT), smem, stream, p, pg, turns, (int)pages, per);
}

// P row units per thread while that still gives every SM a few CTAs: 4 where the
// rows of a CTA's tokens come out even, else 2.  (16 sequences of 1 .. 512 tokens, 32
// query heads, E4M3 pages of 16: 23.8 us at 2, 22.0 at 4; 2048 tokens of 40 heads,
// where 4 leaves three of eight slots empty: 18.5 at 2, 20.9 at 4.)
// E4M3 pages of a call of two tokens per sequence or fewer, on the average, get a
// warp each (what the host knows of the lengths; a long sequence among many without
// new tokens is right but walks its pages by single warps, twice).
template <int D, bool E4M3, int R, int NT>
cudaError_t launch_p(const RopeAppendParams &p, const PagedView &pg, const RopeTurns &turns,
                     cudaStream_t stream)
{
    const int rows = p.H + (E4M3 ? 0 : 2 * p.KV);
    const long long units = (long long)p.total_tokens * rows * (D / 16);
    if (p.rd % 16 != 0)
        return units >= 2ll * NT * kManyRowCtas ? launch_fused<D, E4M3, R, NT, 2, true>(p, pg, turns, stream)
                                                : launch_fused<D, E4M3, R, NT, 1, true>(p, pg, turns, stream);
    if constexpr (E4M3) {
        if (p.total_tokens <= 2ll * p.batch && units < 2ll * NT * kManyRowCtas)
            return launch_fused<D, true, 1, 128, 1, false, true>(p, pg, turns, stream);
    }
    if (units >= 4ll * NT * kManyRowCtas && NT / 64 * rows % (4 * NT / (D / 16)) == 0)
        return launch_fused<D, E4M3, R, NT, 4, false>(p, pg, turns, stream);
    if (units >= 2ll * NT * kManyRowCtas)
        return launch_fused<D, E4M3, R, NT, 2, false>(p, pg, turns, stream);
    return launch_fused<D, E4M3, R, NT, 1, false>(p, pg, turns, stream);
}

}  // namespace

cudaError_t launch_append_paged(const RopeAppendParams &p, const PagedView &pg, bool e4m3,
                                const RopeTurns &turns, cudaStream_t stream)
{
    if (p.d == 128) {
        if (!e4m3)
            return launch_p<128, false, 1, 128>(p, pg, turns, stream);
        switch (pg.page_log) {
        case 4: return launch_p<128, true, 1, 128>(p, pg, turns, stream);
        case 5: return launch_p<128, true, 2, 128>(p, pg, turns, stream);
        case 6: return launch_p<128, true, 4, 128>(p, pg, turns, stream);
        default: return launch_p<128, true, 4, 256>(p, pg, turns, stream);
        }
    }
    if (!e4m3)
        return launch_p<64, false, 1, 128>(p, pg, turns, stream);
    switch (pg.page_log) {
    case 4:
    case 5: return launch_p<64, true, 1, 128>(p, pg, turns, stream);
    case 6: return launch_p<64, true, 2, 128>(p, pg, turns, stream);
    default: return launch_p<64, true, 4, 128>(p, pg, turns, stream);
    }
}
