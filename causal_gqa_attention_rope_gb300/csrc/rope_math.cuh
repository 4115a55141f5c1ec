// rope_math.cuh -- the rotation's arithmetic, shared by the append kernels
// (rope_append.cu explains its precision): cos and sin of a position's turns as
// fp32 pairs, the rotation of exact and of paired inputs, and how a token finds
// its sequence.
#pragma once

#include "na_internal.cuh"

namespace rope {

// pi as an unevaluated sum of two doubles (the high part is pi rounded to
// double, the low part the next 53 bits).
constexpr double kPiHi = 3.141592653589793116;
constexpr double kPiLo = 1.2246467991473532e-16;
constexpr double kStep = kPiHi / 128.0;  // 2 pi / 256

// ------------------------------------------------- compile-time table --

// Taylor series about 0, used by the table builder for |x| <= pi / 4 where
// the terms fall below 1e-30 long before the loop ends.
constexpr double series_sin(double x)
{
    double term = x, sum = x;
    for (int n = 1; n < 20; ++n) {
        term *= -x * x / ((2.0 * n) * (2.0 * n + 1.0));
        sum += term;
    }
    return sum;
}

constexpr double series_cos(double x)
{
    double term = 1.0, sum = 1.0;
    for (int n = 1; n < 20; ++n) {
        term *= -x * x / ((2.0 * n - 1.0) * (2.0 * n));
        sum += term;
    }
    return sum;
}

struct alignas(16) TrigEntry {
    float ch, cl, sh, sl;  // cos and sin of 2 pi j / 256 as fp32 hi + lo pairs
};
struct TrigTable {
    TrigEntry e[256];
};

// cos and sin of 2 pi j / 256: the angle is written as a quarter turn q plus
// an offset within +-pi/4, whose series is evaluated; the quarter turn is
// applied by exact swaps and sign changes.
constexpr TrigTable make_trig_table()
{
    TrigTable t{};
    for (int j = 0; j < 256; ++j) {
        const int q = ((j + 32) / 64) % 4;
        const int off = j - 64 * ((j + 32) / 64);  // in [-32, 32)
        const double x = off * kStep;
        const double c0 = series_cos(x), s0 = series_sin(x);
        double c = c0, s = s0;
        if (q == 1) {
            c = -s0;
            s = c0;
        } else if (q == 2) {
            c = -c0;
            s = -s0;
        } else if (q == 3) {
            c = s0;
            s = -c0;
        }
        const float ch = (float)c, sh = (float)s;
        t.e[j] = TrigEntry{ch, (float)(c - (double)ch), sh, (float)(s - (double)sh)};
    }
    return t;
}

__device__ const TrigTable kTrig = make_trig_table();

// 2 pi as an fp32 pair.
constexpr float kTwoPiHi = (float)(2.0 * kPiHi);
constexpr float kTwoPiLo = (float)((2.0 * kPiHi - (double)kTwoPiHi) + 2.0 * kPiLo);

// ----------------------------------------------- fp32 pair arithmetic --

struct F2 {
    float hi, lo;  // unevaluated sum
};

// a * b + c * d of two pairs' products as a pair: leading products exact, their
// sum error-free, cross terms rounded once.
__host__ __device__ __forceinline__ F2 prod_sum(F2 a, F2 b, F2 c, F2 d)
{
    const float p0 = a.hi * b.hi;
    const float e0 = fmaf(a.hi, b.hi, -p0);
    const float p1 = c.hi * d.hi;
    const float e1 = fmaf(c.hi, d.hi, -p1);
    const float s = p0 + p1;
    const float bb = s - p0;
    const float t = (p0 - (s - bb)) + (p1 - bb);
    const float cross = fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, fmaf(c.hi, d.lo, c.lo * d.hi)));
    return {s, t + (e0 + e1) + cross};
}

// cos and sin of 2 pi * pos * (fhi 2^-64 + flo 2^-96) as fp32 pairs
// (cos hi, cos lo, sin hi, sin lo).
__host__ __device__ __forceinline__ float4 cos_sin_turns(unsigned int pos, unsigned long long fhi,
                                                         unsigned int flo, const TrigEntry *tab)
{
    // Fraction of a turn in units of 2^-64 (exact but for the dropped bits
    // below 2^-64), rounded to the nearest 1/256 turn j plus a remainder.
    unsigned long long u = (unsigned long long)pos * fhi + (((unsigned long long)pos * flo) >> 32);
    u += 1ull << 55;
    const int j = (int)(u >> 56);
    const long long rem = (long long)(u & ((1ull << 56) - 1)) - (1ll << 55);  // |rem| <= 2^55
    // rem * 2^-64 as an fp32 pair: three exactly representable pieces.
    const int a_part = (int)(rem >> 32);  // |.| <= 2^23
    const unsigned int b_part = (unsigned int)(rem & 0xffffffffll);
    const float t1 = (float)a_part * 0x1p-32f;
    const float t2 = (float)(b_part >> 8) * 0x1p-56f;
    const float t3 = (float)(b_part & 255u) * 0x1p-64f;
    const float rh0 = t1 + t2;
    const float bb = rh0 - t1;
    const float rl0 = ((t1 - (rh0 - bb)) + (t2 - bb)) + t3;
    // r = 2 pi * remainder, radians, |r| <= pi / 256
    const float dh = rh0 * kTwoPiHi;
    const float dl = fmaf(rh0, kTwoPiHi, -dh) + fmaf(rh0, kTwoPiLo, rl0 * kTwoPiHi);

    // Series of the remainder.
    const float z = dh * dh;
    const float ze = fmaf(dh, dh, -z);
    // sin r = dh - dh^3/6 + dh^5/120 + dl (1 - dh^2/2)
    const float p3 = dh * z;
    const float p3e = fmaf(dh, z, -p3) + dh * ze;
    const float sin_lo = dl * fmaf(z, -0.5f, 1.0f) - (p3 * (1.0f / 6.0f) + p3e * (1.0f / 6.0f)) +
                         p3 * z * (1.0f / 120.0f);
    const F2 sn = {dh, sin_lo};
    // cos r = 1 - r^2/2 + r^4/24 - r^6/720, with r^2 = z + ze + 2 dh dl
    const float half_z = 0.5f * z;
    const float c0 = 1.0f - half_z;
    const float c0e = (1.0f - c0) - half_z;
    const float z2 = z * z;
    const float cos_lo = c0e - 0.5f * ze - dh * dl + z2 * (1.0f / 24.0f) - z2 * z * (1.0f / 720.0f);
    const F2 cs = {c0, cos_lo};

    const TrigEntry e = tab[j];
    const F2 tc = {e.ch, e.cl}, ts = {e.sh, e.sl};
    const F2 nts = {-e.sh, -e.sl};
    const F2 c = prod_sum(tc, cs, nts, sn);  // cos(t + r) = cos t cos r - sin t sin r
    const F2 s = prod_sum(ts, cs, tc, sn);   // sin(t + r) = sin t cos r + cos t sin r
    return make_float4(c.hi, c.lo, s.hi, s.lo);
}

// a = x * w as an unevaluated fp32 sum hi + lo (exact).
__device__ __forceinline__ F2 weighted(float x, float w, bool zero_centered)
{
    const float p = x * w;
    const float pe = fmaf(x, w, -p);  // exact residual of the product
    if (!zero_centered)
        return {p, pe};
    // x * (1 + w) = x + x * w: error-free sum of x and p, residuals folded into lo
    const float s = x + p;
    const float bb = s - x;
    const float se = (x - (s - bb)) + (p - bb);
    return {s, se + pe};
}

// Rotated pair (y0, y1) = (a0 cos - a1 sin, a0 sin + a1 cos) * fr.
__device__ __forceinline__ void rotate(F2 a0, F2 a1, float4 c, float fr, float &y0, float &y1)
{
    const F2 r0 = prod_sum(a0, F2{c.x, c.y}, F2{-a1.hi, -a1.lo}, F2{c.z, c.w});
    const F2 r1 = prod_sum(a0, F2{c.z, c.w}, a1, F2{c.x, c.y});
    y0 = fmaf(r0.hi, fr, r0.lo * fr);
    y1 = fmaf(r1.hi, fr, r1.lo * fr);
}

// The same for exact inputs (no low parts).  Of the two leading products one
// is split exactly -- t = a1 sin_hi rounded, e its error from an fma -- and
// the other enters an fma unrounded, so h = a0 cos_hi - t carries a single
// rounding relative to itself; e and the low parts of cos and sin are added
// once.  Before the final rounding to bf16 the result is within ~2^-23 of
// itself (plus ~2^-48 of the inputs).
__device__ __forceinline__ void rotate_exact(float a0, float a1, float4 c, float fr, float &y0,
                                             float &y1)
{
    {
        const float t = a1 * c.z;
        const float e = fmaf(a1, c.z, -t);
        const float h = fmaf(a0, c.x, -t);
        const float lo = fmaf(a0, c.y, -a1 * c.w) - e;
        y0 = fmaf(h, fr, lo * fr);
    }
    {
        const float t = a1 * c.x;
        const float e = fmaf(a1, c.x, -t);
        const float h = fmaf(a0, c.z, t);
        const float lo = fmaf(a0, c.w, a1 * c.y) + e;
        y1 = fmaf(h, fr, lo * fr);
    }
}

// Owner sequence b of token t (the last b with cu_seqlens[b] <= t, empty
// sequences skipped) and the token's position, a warp at a time: cu_seqlens
// and cache_lens are read in the same round.
__device__ __forceinline__ void owner_of(const RopeAppendParams &p, int t, int lane, int &b,
                                         int &pos)
{
    b = 0;
    pos = -1;
    for (int base = 0; base < p.batch; base += 32) {
        const int i = base + lane;
        int cu = 0x7fffffff, cl = 0;
        if (i < p.batch) {
            cu = __ldg(p.cu_seqlens + i);
            cl = __ldg(p.cache_lens + i);
        }
        const unsigned m = __ballot_sync(0xffffffffu, cu <= t);
        if (m) {
            const int src = 31 - __clz(m);
            b = base + src;
            pos = __shfl_sync(0xffffffffu, cl, src) + (t - __shfl_sync(0xffffffffu, cu, src));
        }
        if (m != 0xffffffffu)
            break;
    }
}

// 16-byte read-only load kept where it is written (the compiler may not sink
// it past the barriers that follow, so its latency overlaps theirs).
__device__ __forceinline__ uint4 ldg_early(const void *p)
{
    uint4 u;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}

}  // namespace rope
