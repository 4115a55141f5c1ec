// latent_runs.cuh -- how the kernels of absorbed latent attention share out their work: units of query
// rows of one sequence, and the key tiles of all units, one after the other, cut into one
// equal run per CTA or pair of CTAs, whatever the lengths; a unit counts for UNIT_STEPS more, about
// what its Q and its results hold a CTA up.
#pragma once

#include "latent.cuh"

namespace {

constexpr int KT = kLatentKeys;
constexpr int UNIT_STEPS = 1;

struct Sequence {
    int tok0, n, prior;
};

// Sequence b; n = 0 where it breaks the call's bounds (`code` says how).
__device__ __forceinline__ Sequence sequence_of(const LatentParams &p, int b, int &code)
{
    Sequence s;
    s.tok0 = __ldg(p.cu_seqlens + b);
    s.n = __ldg(p.cu_seqlens + b + 1) - s.tok0;
    s.prior = __ldg(p.cache_lens + b);
    code = NA_OK;
    if (s.n > p.max_new_len || s.tok0 < 0 || (b == 0 && s.tok0 != 0) ||
        (long long)s.tok0 + s.n > p.total_tokens)
        code = NA_ERR_INVALID_ARG;
    else if (s.n > 0 && (s.prior < 0 || (long long)s.prior + s.n > min(p.capacity, p.max_total_len)))
        code = NA_ERR_CAPACITY;
    if (code != NA_OK || s.n < 0)
        s.n = 0;
    return s;
}

template <int UR>
__device__ __forceinline__ int units_of(const LatentParams &p, const Sequence &s)
{
    return (s.n * p.H + UR - 1) / UR;
}

// Keys that the rows of unit t see.
template <int UR>
__device__ __forceinline__ int keys_of(const LatentParams &p, const Sequence &s, int t)
{
    return s.prior + (min(t * UR + UR, s.n * p.H) - 1) / p.H + 1;
}

// What the unit counts for in a run: steps.
template <int UR>
__device__ __forceinline__ int steps_of(const LatentParams &p, const Sequence &s, int t)
{
    return (keys_of<UR>(p, s, t) + KT - 1) / KT + UNIT_STEPS;
}

// Steps of the sequences 32 `chunk` + lane, a warp at a time: each lane its own, or, where
// one of them has many units, all lanes together one sequence after the other.
template <int UR>
__device__ __forceinline__ long long chunk_steps(const LatentParams &p, int chunk, int lane)
{
    const int b = chunk * 32 + lane;
    Sequence s{0, 0, 0};
    int code = NA_OK;
    if (b < p.batch)
        s = sequence_of(p, b, code);
    if (code != NA_OK && blockIdx.x == 0)
        na_report(p.status, code);
    const int units = units_of<UR>(p, s);
    long long sum = 0;
    if (!__any_sync(0xffffffffu, units > 16)) {
        for (int t = 0; t < units; t++)
            sum += steps_of<UR>(p, s, t);
        return sum;
    }
    for (int i = 0; i < 32; i++) {
        const Sequence o{0, __shfl_sync(0xffffffffu, s.n, i), __shfl_sync(0xffffffffu, s.prior, i)};
        long long x = 0;
        for (int t = lane; t < units_of<UR>(p, o); t += 32)
            x += steps_of<UR>(p, o, t);
#pragma unroll
        for (int k = 16; k; k >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, k);
        if (lane == i)
            sum = x;
    }
    return sum;
}

__device__ __forceinline__ long long inclusive_sum(long long x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    return x;
}

// Runs that have work (all others are empty), and the first step of run c; the runs of
// `total` steps are as equal as can be, none of them empty.
__device__ __forceinline__ long long busy_runs(const LatentParams &p, long long total)
{
    return min((long long)p.grid, total);
}

__device__ __forceinline__ long long run_begin(const LatentParams &p, long long total, int c)
{
    const long long busy = busy_runs(p, total);
    return c >= busy ? total : total * c / busy;
}

// The run that holds the step before `end`: the last c with total c / busy < end.
__device__ __forceinline__ int run_of(const LatentParams &p, long long total, long long end)
{
    return (int)((end * busy_runs(p, total) + total - 1) / total) - 1;
}

// Run `run`: sm.total, sm.begin and the unit and step of it that it begins with.  Each warp
// sums a range of sequences; the one whose range holds the beginning looks it up.
template <int UR, int WARPS, class Smem>
__device__ __forceinline__ void find_run(const LatentParams &p, Smem &sm, int run, int warp, int lane)
{
    const int chunks = (p.batch + 31) / 32, per = (chunks + WARPS - 1) / WARPS;
    const int c0 = min(warp * per, chunks), c1 = min(c0 + per, chunks);
    long long mine = 0, chunk_sum = 0;  // (a single chunk's sums are kept)
    for (int c = c0; c < c1; c++) {
        chunk_sum = chunk_steps<UR>(p, c, lane);
        mine += chunk_sum;
    }
#pragma unroll
    for (int k = 16; k; k >>= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, k);
    if (lane == 0)
        sm.warp_steps[warp] = mine;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
        before += w < warp ? sm.warp_steps[w] : 0;
        total += sm.warp_steps[w];
    }
    const long long begin = run_begin(p, total, run);
    if (threadIdx.x == 0) {
        sm.total = total;
        sm.begin = begin;
    }
    if (begin >= before && begin < before + mine) {
        for (int c = c0; c < c1; c++) {
            if (per > 1)
                chunk_sum = chunk_steps<UR>(p, c, lane);
            const long long upto = inclusive_sum(chunk_sum, lane);
            const unsigned past = __ballot_sync(0xffffffffu, before + upto > begin);
            if (past) {
                const int i = __ffs(past) - 1, b = c * 32 + i;
                before += __shfl_sync(0xffffffffu, upto - chunk_sum, i);
                int code;
                const Sequence s = sequence_of(p, b, code);
                for (int t = 0;; t += 32) {
                    const long long x = t + lane < units_of<UR>(p, s) ? steps_of<UR>(p, s, t + lane) : 0;
                    const long long y = inclusive_sum(x, lane);
                    const unsigned m = __ballot_sync(0xffffffffu, before + y > begin);
                    if (m) {
                        const int k = __ffs(m) - 1;
                        if (lane == k) {
                            sm.b0 = b;
                            sm.t0 = t + k;
                            sm.step0 = (int)(begin - (before + y - x));
                        }
                        break;
                    }
                    before += __shfl_sync(0xffffffffu, y, 31);
                }
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    __syncthreads();
}

// One after the other, the pieces of a run.  Every warp role walks them for itself.
template <int UR>
struct Walk {
    int b, t, step;       // next: sequence, unit, step of it
    long long left;       // steps of the run from there
    Sequence s;
    bool have;

    // the piece: tiles [lo, hi) of `tiles` of unit `unit` of sequence `seq`, which has `keys`
    int seq, unit, lo, hi, tiles, keys;

    template <class Smem>
    __device__ __forceinline__ Walk(const LatentParams &p, const Smem &sm, int run)
        : b(sm.b0), t(sm.t0), step(sm.step0), left(run_begin(p, sm.total, run + 1) - sm.begin),
          have(false)
    {
    }

    // Piece `piece` of p.pieces of a unit of its own (none where the sequence has fewer units).
    __device__ __forceinline__ Walk(const LatentParams &p, int index, int piece) : left(0), have(false)
    {
        const int units = (p.max_new_len * p.H + UR - 1) / UR;  // of the longest sequence
        b = index / units;
        t = index % units;
        int code;
        s = sequence_of(p, b, code);
        if (code != NA_OK && t == 0 && piece == 0 && threadIdx.x == 0)
            na_report(p.status, code);
        if (t >= units_of<UR>(p, s))
            return;
        const int all = (keys_of<UR>(p, s, t) + KT - 1) / KT;
        const int from = (int)((long long)all * piece / p.pieces);
        step = from + UNIT_STEPS;
        left = (int)((long long)all * (piece + 1) / p.pieces) - from;
        have = true;
    }

    __device__ __forceinline__ bool next(const LatentParams &p)
    {
        if (left <= 0)
            return false;
        int code;
        while (!have) {
            s = sequence_of(p, b, code);
            have = t < units_of<UR>(p, s);
            if (!have) {
                b++;
                t = 0;
            }
        }
        seq = b;
        unit = t;
        keys = keys_of<UR>(p, s, t);
        tiles = (keys + KT - 1) / KT;
        const int end = (int)min((long long)tiles + UNIT_STEPS, step + left);
        lo = max(step - UNIT_STEPS, 0);
        hi = max(end - UNIT_STEPS, 0);
        left -= end - step;
        step = 0;
        t++;
        have = t < units_of<UR>(p, s);
        if (!have) {
            b++;
            t = 0;
        }
        return hi > lo;  // (none: the run ends within the unit's first steps)
    }

    // rows of the unit from `at` on, `most` at most, and the first one among the call's
    __device__ __forceinline__ int rows(const LatentParams &p, int at, int most) const
    {
        return max(min(most, s.n * p.H - unit * UR - at), 0);
    }
    __device__ __forceinline__ long long row0(const LatentParams &p) const
    {
        return (long long)s.tok0 * p.H + unit * UR;
    }
};

// Named barrier that also says whether any thread's `x` holds.
__device__ __forceinline__ bool any_of(bool x, int id, int threads)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}

// `at`'s place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t place_in_cta(const void *at, int rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(at)), "r"(rank));
    return a;
}

}  // namespace
