// decode_shared.cuh -- what the split passes of the single-token decode share:
// the cut of the concatenated key streams into one equal slice per CTA, the
// walk over a slice's pieces, and the warp-level bf16 MMA with its fragment
// loads.  The contiguous cache (decode.cu) and the paged cache
// (decode_paged.cu) differ in how a tile of keys reaches shared memory and
// registers, not in these.
#pragma once

#include "na_internal.cuh"

namespace dec {

constexpr float kRescaleThreshold = 8.0f;  // log2 units

// Keys of sequence b that are attended -- the last `window` of its length, or
// all of them without a window -- with *first the index of the first one; 0
// for a length past the cache capacity or the host bound (skipped here,
// reported by the combine pass).
__device__ __forceinline__ int attended_keys(const DecodeParams &p, int b, int &first)
{
    const int n = __ldg(p.kv_lens + b);
    const bool ring = (p.flags & NA_RING_CACHE) != 0;  // positions wrap at the capacity
    if (n < 0 || (!ring && n > p.capacity) || n > p.max_kv_len) {
        first = 0;
        return 0;
    }
    const int len = (p.window > 0 && n > p.window) ? p.window : n;
    first = n - len;
    return len;
}

__device__ __forceinline__ int valid_len(const DecodeParams &p, int b)
{
    int first;
    return attended_keys(p, b, first);
}

// What a stream counts for in the cut into equal slices: its keys, and COST more
// ahead of them for the time that a CTA spends on a piece besides its keys.
template <int COST>
__device__ __forceinline__ int stream_weight(int n)
{
    return n > 0 ? n + COST : 0;
}

// Where this CTA's key slice starts: computed by one full warp, then shared.
struct Slice {
    long long start, end;  // [start, end) in the concatenation of all streams
    long long off;         // offset of the stream holding `start`
    int b, si;             // its sequence and stream index within the sequence
    int empty;
};

// One piece: the keys [k0, k1) of stream (b, kvh, hc) that this CTA reads.
struct Piece {
    int b, kvh, hc, k0, k1, id;
    int kf;            // cache index of the stream's first attended key
    bool first, last;  // holds the stream's first / last key
};

template <int COST = 0>
__device__ __forceinline__ void locate_slice(const DecodeParams &p, int lane, Slice &out)
{
    const unsigned FULL = 0xffffffffu;
    const int spb = p.KV * p.head_chunks;  // streams per sequence
    long long t = 0;
    for (int b = lane; b < p.batch; b += 32)
        t += stream_weight<COST>(valid_len(p, b));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        t += __shfl_xor_sync(FULL, t, m);
    const long long total = t * spb;
    const long long grid = gridDim.x;
    long long P = (total + grid - 1) / grid;
    if (P < p.min_slice)
        P = p.min_slice;
    Slice sl{};
    sl.start = (long long)blockIdx.x * P;
    sl.end = min(sl.start + P, total);
    sl.empty = sl.start >= total;
    if (!sl.empty) {
        // First sequence whose streams extend past `start`.
        long long base = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            const int b = b0 + lane;
            const int n = b < p.batch ? stream_weight<COST>(valid_len(p, b)) : 0;
            const long long w = (long long)n * spb;
            long long incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(FULL, incl, o);
                if (lane >= o)
                    incl += y;
            }
            const long long excl = base + incl - w;
            const unsigned hit = __ballot_sync(FULL, w > 0 && sl.start < excl + w && sl.start >= excl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                sl.b = b0 + src;
                const long long off_b = __shfl_sync(FULL, excl, src);
                const int nb = __shfl_sync(FULL, n, src);
                sl.si = (int)((sl.start - off_b) / nb);
                sl.off = off_b + (long long)sl.si * nb;
                break;
            }
            base += __shfl_sync(FULL, incl, 31);
        }
    }
    if (lane == 0)
        out = sl;
}

// Walks this CTA's pieces in order; every thread of the CTA walks the same way.
template <int COST = 0>
struct Walker {
    long long start, end, off;
    int b, si, len, kfirst, spb, c;
    bool done;

    __device__ __forceinline__ void init(const Slice &sl, const DecodeParams &p)
    {
        start = sl.start;
        end = sl.end;
        off = sl.off;
        b = sl.b;
        si = sl.si;
        spb = p.KV * p.head_chunks;
        c = blockIdx.x;
        done = sl.empty != 0;
        kfirst = 0;
        len = done ? 0 : attended_keys(p, b, kfirst);
    }

    __device__ __forceinline__ bool next(const DecodeParams &p, Piece &pc)
    {
        while (!done && b < p.batch && off < end) {
            const long long s_off = off;
            const int n = len, sb = b, ssi = si, kfs = kfirst;
            off += stream_weight<COST>(n);
            if (++si == spb) {
                si = 0;
                if (++b < p.batch)
                    len = attended_keys(p, b, kfirst);
            }
            const long long k_off = s_off + COST;  // of the stream's first key
            const long long lo = start > k_off ? start - k_off : 0;
            const long long hi = end - k_off < n ? end - k_off : n;
            if (lo < hi) {
                pc.b = sb;
                pc.kvh = ssi / p.head_chunks;
                pc.hc = ssi - pc.kvh * p.head_chunks;
                pc.k0 = (int)lo;
                pc.k1 = (int)hi;
                pc.id = sb * spb + ssi + c;
                pc.kf = kfs;
                pc.first = lo == 0;
                pc.last = hi == n;
                return true;
            }
        }
        return false;
    }
};

// ------------------------------------------------ warp-level bf16 MMA --
// mma.sync m16n8k16 (bf16 in, fp32 accumulate) and its fragment loads.  For a
// 16x16 A tile, lane l holds rows l/4 and l/4 + 8 at columns 2(l%4), +1 and
// 2(l%4) + 8, +9; for a 16x8 B tile, rows 2(l%4), +1 and +8, +9 of column l/4;
// the 16x8 accumulator holds rows l/4 and l/4 + 8 at columns 2(l%4), +1.

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// The transpose of an 8x8 b16 matrix held one 32-bit pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x on the MUFU unit (approximate, flushes subnormal results to zero).
__device__ __forceinline__ float ex2_mufu(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace dec
