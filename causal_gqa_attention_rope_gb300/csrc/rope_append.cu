// rope_append.cu -- fused qk-RMSNorm, V-norm, RoPE and KV-cache append.
//
// Computes, per new token t of sequence b at pos = cache_lens[b] + (t - cu_seqlens[b]):
//   q_out[t][h]        = RoPE(norm_q(q[t][h]), pos)
//   cache_k[b][g][pos] = RoPE(norm_k(k[t][g]), pos)
//   cache_v[b][g][pos] = vnorm(v[t][g])
// following cortiq-engine src/attention.rs, fns finish_projection (norms before
// RoPE, partial rotary over the first rd dims), rmsnorm_head, vnorm_head and
// rope_rotate_scaled (half-split pairs (x[i], x[i + rd/2]), both outputs scaled
// by the attention factor).
//
// The kernel moves 2 * (H + 2 KV) * d * 2 bytes per token and is bound by the
// latency of its one round trip, so everything a thread needs is requested
// first, the work between the loads and the stores is short and free of double
// precision, and many small CTAs share an SM to overlap their round trips:
//   - rope_append_kernel (rotary_dim a multiple of 16): a CTA of 64 threads
//     takes 64 / (d / 16) rows of one token (grid: tokens x row groups); each
//     thread owns one 32-byte unit of a row -- chunks [8k, 8k + 8) and
//     [rd/2 + 8k, ...) of the rotated part (eight rotation pairs), two
//     consecutive chunks of the non-rotated tail, or of a V row -- loads it
//     with two 16-byte loads, takes the row's sum of squares with shuffles
//     among the row's lanes, rotates in registers and stores it with two
//     16-byte stores.  The only shared data are the cos/sin of the rd/2 pair
//     indices, computed by the CTA (one 256-entry table lookup each, read
//     through the cache).  One CTA per token of all rows left one CTA per SM
//     and measured ~39 us per 2048-token chunk of 56 rows.
//   - rope_append_staged_kernel (any even rotary_dim): the rows are staged in
//     shared memory and every thread works on independent (row, pair) slots.
//
// Precision.  Before its final rounding to bf16 a rotated value differs from
// the exact rotation by at most ~2^-23 of its own magnitude (plus ~2^-43 of
// its inputs), so the stored bf16 is the correctly rounded value unless the
// exact one lies that close to a bf16 rounding boundary; then it may be the
// neighbour, one ulp off (measured: about 7 in a million rotated values):
//   - The angle is taken in turns: pos * inv_freq / (2 pi) is formed exactly
//     modulo 1 in 64-bit fixed point (inv_freq / (2 pi) is passed as a 96-bit
//     fixed-point fraction, from a double-double division on the host; the
//     product needs only integer multiplies).  Its top 8 bits select cos and sin
//     of a multiple of 2 pi / 256 from a table built at compile time; the rest,
//     |r| <= pi / 256, goes through the Taylor series of cos and sin evaluated
//     in fp32 pairs (hi + lo, fmaf residuals for the leading products), and the
//     two are combined with the angle-sum formulas.  Absolute error of cos and
//     sin below 2^-43 (the rounding of the ~3e-7 low parts).
//   - The rotation keeps every rounding relative to its own result: one of the
//     two leading products is split exactly (its error recovered by an fmaf),
//     the other enters an fmaf unrounded (inputs carried as fp32 pairs use
//     error-free products and sums instead); the norm weight enters as the
//     exact product x * w of two bf16 values (for the zero-centred style,
//     x + x * w is kept as an fp32 hi + lo pair); the row factors (1 / rms,
//     and the attention factor on the rotated dims) are applied last as one
//     relative rounding.
#include "na_internal.cuh"
#include "rope_math.cuh"

namespace {

using namespace rope;

constexpr int kStagedThreads = 256;

__device__ __forceinline__ const bf16 *row_src(const RopeAppendParams &p, int t, int r)
{
    if (r < p.H)
        return p.q + ((size_t)t * p.H + r) * p.d;
    if (r < p.H + p.KV)
        return p.k + ((size_t)t * p.KV + (r - p.H)) * p.d;
    return p.v + ((size_t)t * p.KV + (r - p.H - p.KV)) * p.d;
}

// Slab b of the cache holds `cap` slots per kv head: a sequence's whole cache,
// or one page.
__device__ __forceinline__ bf16 *row_dst(const RopeAppendParams &p, int t, int r, int b, int slot,
                                         size_t cap)
{
    if (r < p.H)
        return p.q_out + ((size_t)t * p.H + r) * p.d;
    if (r < p.H + p.KV)
        return p.cache_k + (((size_t)b * p.KV + (r - p.H)) * cap + slot) * p.d;
    return p.cache_v + (((size_t)b * p.KV + (r - p.H - p.KV)) * cap + slot) * p.d;
}

// The slab, slot and slots per slab of position pos of sequence b: its page
// with a paged cache.  False when the page index lies outside the cache.
template <bool PAGED>
__device__ __forceinline__ bool cache_place(const RopeAppendParams &p, const PagedView &pg, int pos,
                                            int &b, int &slot, size_t &cap)
{
    if constexpr (PAGED) {
        const int id = __ldcg(pg.table + (size_t)b * pg.pages_per_seq + (pos >> pg.page_log));
        b = id;
        slot = pos & ((1 << pg.page_log) - 1);
        cap = (size_t)1 << pg.page_log;
        return (unsigned)id < (unsigned)pg.num_pages;
    }
    slot = (p.flags & NA_RING_CACHE) ? pos % p.capacity : pos;
    cap = (size_t)p.capacity;
    return true;
}

// ------------------------------------------------------ register path --

constexpr int kAppendThreads = 64;  // one 32-byte row unit each: 4 rows of d = 128, 8 of d = 64

template <int D>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const RopeAppendParams p,
                                                                const RopeTurns turns)
{
    constexpr int UPR = D / 16;  // 32-byte units per row
    __shared__ float4 cs[64];
    const int t = blockIdx.x;
    const int H = p.H, KV = p.KV, rows = H + 2 * KV;
    const int row0 = blockIdx.y * (kAppendThreads / UPR);  // the CTA's first row
    const int half = p.rd / 2;
    const int lane = threadIdx.x & 31;
    const bool qk_norm = (p.flags & NA_QK_NORM) != 0;
    const bool zero_centered = (p.flags & NA_QK_NORM_ZERO_CENTERED) != 0;
    const bool v_norm = (p.flags & NA_V_NORM) != 0;

    // This thread's unit: row r, 8-element chunks starting at e0 and e1.
    const int unit = threadIdx.x;
    const int r = row0 + unit / UPR, k = unit % UPR;
    const bool active = r < rows;
    const bool is_v = r >= H + KV;
    const bool rot = !is_v && k < p.rd / 16;
    int e0, e1;
    if (is_v) {
        e0 = 16 * k;
        e1 = e0 + 8;
    } else if (rot) {
        e0 = 8 * k;
        e1 = half + 8 * k;
    } else {
        e0 = p.rd + 16 * (k - p.rd / 16);
        e1 = e0 + 8;
    }

    // Kernel parameters go before the wait: this thread's frequency (a
    // dynamically indexed parameter).
    unsigned long long fhi = 0;
    unsigned int flo = 0;
    if ((int)threadIdx.x < half) {
        fhi = turns.hi[threadIdx.x];
        flo = turns.lo[threadIdx.x];
    }
    grid_dependency_wait();
    grid_dependents_launch();

    // Everything the token needs is requested first.
    uint4 xa = make_uint4(0, 0, 0, 0), xb = xa, wa = xa, wb = xa;
    if (active) {
        const uint4 *src = reinterpret_cast<const uint4 *>(row_src(p, t, r));
        xa = ldg_early(src + e0 / 8);
        xb = ldg_early(src + e1 / 8);
        if (qk_norm && !is_v) {
            const uint4 *w = reinterpret_cast<const uint4 *>(r < H ? p.qw : p.kw);
            wa = ldg_early(w + e0 / 8);
            wb = ldg_early(w + e1 / 8);
        }
    }
    int b, pos;
    owner_of(p, t, lane, b, pos);
    const bool ring = (p.flags & NA_RING_CACHE) != 0;  // slot = pos % capacity
    if (pos < 0 || (!ring && pos >= p.capacity)) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_CAPACITY);
        return;
    }
    const int slot = ring ? pos % p.capacity : pos;
    __syncthreads();
    if ((int)threadIdx.x < half)  // stored [i][k] for pair 8k + i: a row's lanes read adjacent entries
        cs[(threadIdx.x & 7) * 8 + (threadIdx.x >> 3)] = cos_sin_turns((unsigned)pos, fhi, flo, kTrig.e);
    __syncthreads();

    float a[8], c[8];
    bf16x8_to_f32(xa, a);
    bf16x8_to_f32(xb, c);
    const bool normed = is_v ? v_norm : qk_norm;
    float f = 1.0f;
    if (qk_norm || v_norm) {  // every lane shuffles; rows are aligned to UPR lanes
        float ss = 0.f;      // squares of bf16 values are exact in fp32
#pragma unroll
        for (int i = 0; i < 8; i++)
            ss = fmaf(a[i], a[i], fmaf(c[i], c[i], ss));
#pragma unroll
        for (int o = UPR / 2; o; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (normed)
            f = 1.0f / sqrtf(ss / (float)D + p.eps);
    }
    if (!active)
        return;

    float ya[8], yb[8];
    if (is_v) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            ya[i] = a[i] * f;
            yb[i] = c[i] * f;
        }
    } else {
        F2 xa2[8], xb2[8];
        if (qk_norm) {
            float wfa[8], wfb[8];
            bf16x8_to_f32(wa, wfa);
            bf16x8_to_f32(wb, wfb);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                xa2[i] = weighted(a[i], wfa[i], zero_centered);
                xb2[i] = weighted(c[i], wfb[i], zero_centered);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                xa2[i] = F2{a[i], 0.f};
                xb2[i] = F2{c[i], 0.f};
            }
        }
        if (rot) {
            const float fr = f * p.rope_scale;  // the attention factor scales rotated dims only
            if (qk_norm && zero_centered) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    rotate(xa2[i], xb2[i], cs[i * 8 + k], fr, ya[i], yb[i]);
            } else if (qk_norm) {
                // x * w of two bf16 values is exact in fp32 (its low part is 0):
                // the exact-input rotation gives the same value with fewer terms
#pragma unroll
                for (int i = 0; i < 8; i++)
                    rotate_exact(xa2[i].hi, xb2[i].hi, cs[i * 8 + k], fr, ya[i], yb[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    rotate_exact(a[i], c[i], cs[i * 8 + k], fr, ya[i], yb[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                ya[i] = fmaf(xa2[i].hi, f, xa2[i].lo * f);
                yb[i] = fmaf(xb2[i].hi, f, xb2[i].lo * f);
            }
        }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(row_dst(p, t, r, b, slot, (size_t)p.capacity));
    dst[e0 / 8] = f32_to_bf16x8(ya);
    dst[e1 / 8] = f32_to_bf16x8(yb);
}

// -------------------------------------------------------- staged path --

// PAGED: keys and values go to pages, and rows behind the last sequence are left
// alone.
template <bool PAGED>
__global__ void __launch_bounds__(kStagedThreads) rope_append_staged_kernel(const RopeAppendParams p,
                                                                           const PagedView pg,
                                                                           const RopeTurns turns)
{
    extern __shared__ float smem_f[];
    const int t = blockIdx.x;
    const int H = p.H, KV = p.KV, d = p.d, rows = H + 2 * KV;
    const int half = p.rd / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool qk_norm = (p.flags & NA_QK_NORM) != 0;
    const bool zero_centered = (p.flags & NA_QK_NORM_ZERO_CENTERED) != 0;
    const bool v_norm = (p.flags & NA_V_NORM) != 0;

    float *xs = smem_f;                                          // [rows][d]
    float4 *cs = reinterpret_cast<float4 *>(xs + rows * d);      // [64] (cos hi, lo, sin hi, lo)
    TrigEntry *trig = reinterpret_cast<TrigEntry *>(cs + 64);    // [256]
    float *wq = reinterpret_cast<float *>(trig + 256);           // [d] q norm weights
    float *wk = wq + d;                                          // [d] k norm weights
    float *rf = wk + d;                                          // [rows] 1 / rms per row

    const int cpr = d / 8;  // 16-byte chunks per row
    const int chunks = rows * cpr;
    for (int i = threadIdx.x; i < 256; i += kStagedThreads)
        reinterpret_cast<uint4 *>(trig)[i] = __ldg(reinterpret_cast<const uint4 *>(&kTrig) + i);
    grid_dependency_wait();
    grid_dependents_launch();
    if (PAGED && t >= __ldg(p.cu_seqlens + p.batch))
        return;
    int b, pos;
    owner_of(p, t, lane, b, pos);
    const bool ring = (p.flags & NA_RING_CACHE) != 0;  // slot = pos % capacity
    if (pos < 0 || (!ring && pos >= p.capacity)) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_CAPACITY);
        return;
    }
    int slot;
    size_t cap;
    if (!cache_place<PAGED>(p, pg, pos, b, slot, cap)) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_PAGE);
        return;
    }
    if (qk_norm) {
        for (int i = threadIdx.x; i < 2 * d; i += kStagedThreads)
            wq[i] = __bfloat162float(i < d ? p.qw[i] : p.kw[i - d]);
    }
    for (int c = threadIdx.x; c < chunks; c += kStagedThreads) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row_src(p, t, c / cpr)) + (c % cpr));
        float f[8];
        bf16x8_to_f32(u, f);
        float4 *dst = reinterpret_cast<float4 *>(xs + c * 8);
        dst[0] = make_float4(f[0], f[1], f[2], f[3]);
        dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
    __syncthreads();

    // cos/sin per pair index (two warps) while the other warps take row norms.
    if (threadIdx.x < 64) {
        if ((int)threadIdx.x < half)
            cs[threadIdx.x] = cos_sin_turns((unsigned)pos, turns.hi[threadIdx.x],
                                            turns.lo[threadIdx.x], trig);
    } else if (qk_norm || v_norm) {
        for (int r = warp - 2; r < rows; r += kStagedThreads / 32 - 2) {
            const bool is_v = r >= H + KV;
            float f = 1.0f;
            if (is_v ? v_norm : qk_norm) {
                const float *x = xs + r * d;
                float ss = 0.f;
                for (int i = lane; i < d; i += 32)
                    ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                f = 1.0f / sqrtf(ss / (float)d + p.eps);
            }
            if (lane == 0)
                rf[r] = f;
        }
    }
    __syncthreads();

    // Every row has d/2 slots.  Q and K rows: slot i < half is the pair
    // (i, i + half), the rest cover the non-rotated tail two elements at a
    // time; V rows: elements (2i, 2i + 1).
    const int slots = d / 2;
    const int items = rows * slots;
    const bool any_norm = qk_norm || v_norm;
    for (int it = threadIdx.x; it < items; it += kStagedThreads) {
        const int r = it / slots, i = it - r * slots;
        float *x = xs + r * d;
        const float f = any_norm ? rf[r] : 1.0f;
        if (r >= H + KV) {
            if (v_norm) {
                x[2 * i] *= f;
                x[2 * i + 1] *= f;
            }
            continue;
        }
        const float *w = qk_norm ? (r < H ? wq : wk) : nullptr;
        auto a_of = [&](int e) -> F2 {
            if (!w)
                return {x[e], 0.f};
            return weighted(x[e], w[e], zero_centered);
        };
        if (i < half) {
            float y0, y1;
            rotate(a_of(i), a_of(i + half), cs[i], f * p.rope_scale, y0, y1);
            x[i] = y0;
            x[i + half] = y1;
        } else {
            const int e0 = p.rd + 2 * (i - half);
            const F2 a0 = a_of(e0), a1 = a_of(e0 + 1);
            x[e0] = fmaf(a0.hi, f, a0.lo * f);
            x[e0 + 1] = fmaf(a1.hi, f, a1.lo * f);
        }
    }
    __syncthreads();

    for (int c = threadIdx.x; c < chunks; c += kStagedThreads) {
        const int r = c / cpr, j = c - r * cpr;
        reinterpret_cast<uint4 *>(row_dst(p, t, r, b, slot, cap))[j] = f32_to_bf16x8(xs + r * d + j * 8);
    }
}

// inv_freq / (2 pi) as a 96-bit fixed-point fraction.  The quotient is formed
// as a double-double (error ~2^-104 relative), then each part is converted to
// fixed point exactly.
void turns_fixed_point(double inv_freq, unsigned long long &hi, unsigned int &lo)
{
    const double bh = 2.0 * kPiHi, bl = 2.0 * kPiLo;
    const double q1 = inv_freq / bh;
    const double p = q1 * bh;
    const double pe = fma(q1, bh, -p);
    const double rsd = ((inv_freq - p) - pe) - q1 * bl;
    const double q2 = rsd / bh;
    const __int128 x = (__int128)ldexp(q1, 96) + (__int128)nearbyint(ldexp(q2, 96));
    hi = (unsigned long long)(x >> 32);
    lo = (unsigned int)(x & 0xffffffff);
}

template <bool PAGED>
cudaError_t launch_staged(const RopeAppendParams &p, const PagedView &pg, const RopeTurns &turns,
                          cudaStream_t stream)
{
    const size_t smem = rope_append_smem_bytes(p.H, p.KV, p.d, p.rd);
    // the largest dynamic shared memory granted so far, per device
    static std::atomic<size_t> configured[kMaxDevices];
    const int dev = current_device_index();
    if (smem > 48 * 1024 && (dev < 0 || smem > configured[dev].load(std::memory_order_acquire))) {
        cudaError_t e = cudaFuncSetAttribute(rope_append_staged_kernel<PAGED>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess)
            return e;
        if (dev >= 0) {
            size_t cur = configured[dev].load(std::memory_order_relaxed);
            while (cur < smem && !configured[dev].compare_exchange_weak(cur, smem))
                ;
        }
    }
    return launch_kernel(rope_append_staged_kernel<PAGED>, dim3(p.total_tokens),
                         dim3(kStagedThreads), smem, stream, p, pg, turns);
}

}  // namespace

RopeTurns rope_turns_of(const double *inv_freq, int half)
{
    RopeTurns turns{};
    for (int i = 0; i < half && i < 64; i++)
        turns_fixed_point(inv_freq[i], turns.hi[i], turns.lo[i]);
    return turns;
}

cudaError_t launch_rope_append(const RopeAppendParams &p, const RopeTurns &turns,
                               cudaStream_t stream)
{
    if (p.rd % 16 == 0) {
        const int rows_per_cta = kAppendThreads / (p.d / 16);
        const dim3 grid(p.total_tokens, (p.H + 2 * p.KV + rows_per_cta - 1) / rows_per_cta);
        if (p.d == 128)
            return launch_kernel(rope_append_kernel<128>, grid, dim3(kAppendThreads), 0, stream, p,
                                 turns);
        return launch_kernel(rope_append_kernel<64>, grid, dim3(kAppendThreads), 0, stream, p, turns);
    }
    return launch_staged<false>(p, PagedView{}, turns, stream);
}

// Into pages.  The staged rows stay for bf16 pages with norms at a rotary dimension
// that is no multiple of 16: their sums run in another order than the register
// kernels', and bf16 pages hold the bits of the contiguous call.
cudaError_t launch_rope_append_paged(const RopeAppendParams &p, const PagedView &pg, bool e4m3,
                                     const RopeTurns &turns, cudaStream_t stream)
{
    if (p.rd % 16 != 0 && !e4m3 && (p.flags & (NA_QK_NORM | NA_V_NORM)))
        return launch_staged<true>(p, pg, turns, stream);
    return launch_append_paged(p, pg, e4m3, turns, stream);
}

size_t rope_append_smem_bytes(int H, int KV, int d, int rd)
{
    (void)rd;
    const size_t rows = (size_t)(H + 2 * KV);
    return (rows * d + 64 * 4 + 256 * 4 + 2 * (size_t)d + rows) * sizeof(float);
}
