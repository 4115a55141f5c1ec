// prefill.cu -- causal GQA attention of a chunk of new tokens against the
// per-sequence KV cache, on the sm_100-family tensor cores (tcgen05 + TMEM +
// TMA).  Semantics: cortiq-engine src/attention.rs, fn qwen_attention_batch
// (query bi of a chunk sees keys 0 .. s0 + bi: all history and the earlier
// keys of its own chunk), fn attention_head (softmax(q.k * scale) . V per row)
// and fn apply_gate (sigmoid gate on the output).
//
// One CTA owns 128 query rows of one (sequence, query head) -- the 128 lanes
// of tensor memory -- and walks the 128-key tiles of kv head h / (H / KV) that
// those rows can see (tiles wholly above the diagonal are never loaded).
// Warp roles (8 warps):
//   warp 0     TMA producer: the Q tile once, then K and V tiles into a
//              3-stage ring (128-byte swizzled, as the MMA descriptors expect);
//              the Q tile and the first three stages are issued by the thread
//              that initialises the barriers, before the CTA-wide barrier;
//   warp 1     allocates tensor memory; one lane issues S_j = Q K_j^T (SS, both
//              K-major) into one of three S buffers in tensor memory;
//   warp 2     one lane issues O += P_j V_j (TS: P read from tensor memory over
//              S_j, V MN-major).  Two issuing threads, because one thread cannot
//              keep the tensor core busy with M = N = 128 instructions (each
//              takes ~116 SM cycles to issue, measured on GB300, against ~64
//              cycles of math);
//   warps 4-7  softmax, one query row per thread (its TMEM lane): load S_j,
//              mask, online max in the log2 domain (the reference max is raised
//              only when it grows by more than 2^8, and only then is the O row
//              rescaled in tensor memory), exponentiate on the MUFU unit
//              (measured faster than moving part of the exponentials to a
//              polynomial on the FMA pipe), write P_j as bf16 over S_j, and
//              finally normalise O and stage it through the idle K ring;
//   all warps  then gate and store 16 of the staged rows each, a whole row per
//              instruction (coalesced) instead of one 16-byte piece of 32
//              different rows; warps 0-3 prefetch their gate rows at the start.
// With three S buffers the tensor core computes S_{j+1} and S_{j+2} while the
// softmax works on tile j, and PV_j runs while it prepares P_{j+1}.
//
// A paged cache (na_attn_prefill_chunk_paged) differs in how a K or V tile gets
// there.  bf16 pages: the producer warp keeps the page ids of the next 64 pages
// in registers, one per lane and batch, and each lane issues one box (a page's
// rows by 64 columns) straight into the tile.
//
// E4M3 pages.  K's bytes go to the tensor cores as they are (kind::f8f6f4, twice
// the rate of bf16): a bf16 query has 8 significand bits and an E4M3 number 4,
// so a query row, scaled by a power of two, is the sum of two E4M3 numbers per
// element, and S = Q_hi K^T + Q_lo K^T costs what the bf16 product costs.  (The
// sum is exact for elements down to 2^-10 of the row's largest and within 2^-17
// of that below.)  The row's and K's powers of two multiply the scores in the
// softmax, 16 keys at a time sharing a page.  V's boxes land as bytes in a raw
// ring, and four more warps (the last ones) turn them into the swizzled f16 tile, two
// conversions a word; V's scale enters the weights (na_internal.cuh), which are
// f16 here.  A 2048-token chunk over 28672 keys, 40/8 heads, takes 1004 us (0.66
// of the bf16 peak).  With one softmax group and V converted to bf16, ten integer
// instructions a word, it took 1595 us, with K converted the same way too 2217 us;
// with the tiles left unconverted it would take 920 us, and without the softmax
// 762 us.
//
// Two softmax groups (PAIR: E4M3, REP = 1).  Without the softmax a tile of the
// E4M3 kernel takes 0.78 us, with one warp per 32 rows 1.04: ~1900 cycles of
// waiting, loading, taking maxima, exponentiating and storing, one after the
// other, of which the exponentials' unit is busy 512.  Warps 4-7 take columns
// 0 .. 63 of a tile and warps 8-11 the same rows' columns 64 .. 127.  The two warps
// of a row swap their maxima through shared memory and one barrier of 64 threads
// per tile (which also keeps the second's weights off columns that the first has
// yet to load), so that both hold the same reference; sums stay apart until the
// end.  A mixed step of 16 prompts takes 463 us so, 490 with one group; a long
// context 1004 against 1016.  What stays is the exponentials' phase, 1036 cycles
// for the two warps together, with the tensor cores on the same tensor memory.
// (Groups that alternate tiles, half a tile apart: 608 and 1292 us, and with
// accumulators and references of their own 615 and 1336: both load scores again
// or in smaller pieces to stay within 128 registers.)
//
// Few rows (REP = 4).  A tile of a paged call with at most 32 rows -- drafted
// tokens, single tokens of a mixed batch -- is loaded four times over, so that
// each softmax warp has all the rows in its 32 lanes and takes a quarter of the
// keys: it exponentiates 32 columns instead of 128 and writes zeros for the
// others, and the four partial rows of a query are merged at the end like split
// pieces.  With one warp working on every key and three on padding the softmax
// held the tile loop up (64 sequences of 512 .. 8192 keys, 2 .. 8 tokens: 156 us
// against 126 us).
#include <climits>
#include <cuda.h>
#include <cuda_fp16.h>
#include <mutex>
#include <type_traits>

#include "na_internal.cuh"
#include "tc_primitives.cuh"
#include "tile_waits.cuh"

namespace {

constexpr int BM = 128;      // query rows per CTA (tensor-memory lanes)
constexpr int BN = 128;      // keys per tile
constexpr int STAGES = 3;    // K/V shared-memory ring depth (bf16 caches)
constexpr int NUM_S = 3;     // S/P buffers in tensor memory
constexpr int THREADS = 256; // 8 warps: producer, S issuer, PV issuer, idle, 4 softmax

// Threads of a CTA: E4M3 pages have four more warps that convert, and, unless the
// rows are laid over the lanes, a second softmax group.
constexpr int cta_threads(bool e4m3, int rep)
{
    return THREADS + (e4m3 ? 128 : 0) + (e4m3 && rep == 1 ? 128 : 0);
}
constexpr int E4M3_K_STAGES = 4;  // K tiles in bytes
constexpr int E4M3_V_STAGES = 2;  // f16 V tiles behind a raw ring ...
constexpr int RAW_STAGES = 3;     // ... of this many in bytes
constexpr int SCALE_SLOTS = 8;    // K scales outlive their tile until its softmax (at most 7 tiles)
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL0 = 128;  // S buffer i at columns 128 (i + 1); O at column 0

// Where K and V come from.
enum KvSource { KV_CONTIGUOUS, KV_PAGED, KV_PAGED_E4M3 };

template <int D, KvSource SRC>
struct __align__(1024) TcSmem {
    static constexpr int KB = D / 64;  // 64-wide column blocks of a row
    static constexpr int KST = STAGES, VST = STAGES;
    bf16 q[KB][BM * 64];
    bf16 k[KST][KB][BN * 64];
    bf16 v[VST][KB][BN * 64];
    uint64_t q_full;
    uint64_t k_full[KST], k_empty[KST], v_full[VST], v_empty[VST];
    uint64_t s_full[NUM_S], s_free[NUM_S], p_full[NUM_S];
    uint64_t o_done[NUM_S], drain[2];  // o_done[b]: the PVs of tiles b, b + NUM_S, ...
    uint32_t tmem_base;
    int abort_flag;
};

template <int D>
struct __align__(1024) TcSmem<D, KV_PAGED_E4M3> {
    static constexpr int KB = D / 64;
    static constexpr int KST = E4M3_K_STAGES, VST = E4M3_V_STAGES;
    uint8_t q8[2][BM * D];           // high and low parts of Q, rows of D bytes, swizzled
    uint8_t k[KST][BN * D];          // the same layout
    uint8_t raw[RAW_STAGES][BN * D]; // V's bytes, rows of D (swizzled with D = 128)
    bf16 v[VST][KB][BN * 64];        // (the first holds the bf16 Q tile at the start)
    // for 32 keys of a tile, 16 and 16: K's scales, V's exponents in the weights, 2^-those
    float4 mul_off[SCALE_SLOTS][4];
    float2 v_inv[SCALE_SLOTS][4];
    uint8_t v_scale[RAW_STAGES][8];  // V's E8M0 bytes
    float pair_max[2][2][BM];        // the softmax groups' row maxima, by tile parity
    int pair_failed[4];              // a wait of one of the row quarter's two warps gave up
    uint64_t raw_full[RAW_STAGES], raw_empty[RAW_STAGES];
    uint64_t q_full, q_split;
    uint64_t k_full[KST], k_empty[KST], v_full[VST], v_empty[VST];
    uint64_t s_full[NUM_S], s_free[NUM_S], p_full[NUM_S];
    uint64_t o_done[NUM_S], drain[2];
    uint32_t tmem_base;
    int abort_flag;
};

template <int D, KvSource SRC>
constexpr size_t tc_smem_bytes()
{
    // at least ~116 KB so that a single CTA owns the SM (and its tensor memory)
    return (sizeof(TcSmem<D, SRC>) + 1024) > (116u << 10) ? sizeof(TcSmem<D, SRC>) + 1024
                                                          : (116u << 10);
}

// A raw E4M3 tile (BN rows of D bytes) into a 128-byte-swizzled f16 tile, by the
// four converting warps; `w` is the warp's index among them.  A thread turns 16
// bytes into two 16-byte chunks at a time, and eight consecutive lanes have to
// read and write all eight bank groups.  D = 64: two whole rows, their chunks
// 2 c of opposite parity once swizzled.  D = 128: half of row r and of row
// r ^ 5, whose swizzles send chunks 0 .. 3 to different halves on the raw side
// and chunks 2 c to different parities on the f16 side.
// EDGE: rows outside [lo, hi) hold no visible key and become zero, and V scales
// beyond the weights' range are multiplied in.
template <int D, bool EDGE>
__device__ __forceinline__ void convert_rows(const uint8_t *raw, const uint8_t *scale, uint8_t *tile,
                                             int w, int lane, int lo, int hi)
{
    constexpr int RPI = 512 / D;         // rows per warp instruction
    constexpr int ITERS = BN / 4 / RPI;  // a warp takes 32 consecutive rows
    const int ch = D == 128 ? ((lane >> 3) & 1) * 4 + (lane & 3) : lane & 3;
    auto row_of = [&](int i) {
        if constexpr (D == 128) {
            const int pair = (i & 1) * 2 + (lane >> 4);
            return w * 32 + (i >> 1) * 8 + ((lane & 4) ? pair ^ 5 : pair);
        }
        return w * 32 + i * RPI + (lane >> 2);
    };
    uint8_t *out = tile + (ch / 4) * (BN * 128);
    const int c0 = 2 * (ch % 4);
    uint4 u[ITERS];
#pragma unroll
    for (int i = 0; i < ITERS; i++) {
        const int r = row_of(i);
        u[i] = *reinterpret_cast<const uint4 *>(raw + r * D + ((D == 128 ? ch ^ (r & 7) : ch) << 4));
    }
#pragma unroll
    for (int i = 0; i < ITERS; i++) {
        const int r = row_of(i);
        uint32_t o[8];
        e4m3x4_to_f16(u[i].x, o[0], o[1]);
        e4m3x4_to_f16(u[i].y, o[2], o[3]);
        e4m3x4_to_f16(u[i].z, o[4], o[5]);
        e4m3x4_to_f16(u[i].w, o[6], o[7]);
        if constexpr (EDGE) {
            const uint32_t rest = v_rest_f16x2(scale[r >> 4]);
            const uint32_t rest2 = v_rest_f16x2_second(scale[r >> 4]);
            const bool seen = r >= lo && r < hi;
#pragma unroll
            for (int q = 0; q < 8; q++)
                o[q] = seen ? mul_f16x2(mul_f16x2(o[q], rest), rest2) : 0u;
        }
        uint8_t *row = out + r * 128;
        *reinterpret_cast<uint4 *>(row + ((c0 ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(row + (((c0 + 1) ^ (r & 7)) << 4)) =
            make_uint4(o[4], o[5], o[6], o[7]);
    }
}

template <int D>
__device__ __forceinline__ void convert_tile(const uint8_t *raw, const uint8_t *scale, bf16 *tile,
                                             int w, int lane, int lo, int hi)
{
    uint8_t *out = reinterpret_cast<uint8_t *>(tile);
    const bool extreme = __any_sync(0xffffffffu, abs((int)scale[lane & 7] - 127) > kMaxVExp);
    if (extreme || lo > 0 || hi < BN)
        convert_rows<D, true>(raw, scale, out, w, lane, lo, hi);
    else
        convert_rows<D, false>(raw, scale, out, w, lane, lo, hi);
}

// 16-byte chunk c of row r of a D-byte-row tile, 128- or 64-byte swizzled.
template <int D>
__device__ __forceinline__ uint32_t byte_chunk_off(int r, int c)
{
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4))
                    : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Two fp32 values as E4M3 (x0 in the low byte) and what is left of them.
__device__ __forceinline__ uint32_t e4m3x2_split(float &x0, float &x1)
{
    uint16_t h;
    uint32_t f;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(x1), "f"(x0));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&f));
    x0 -= y.x;
    x1 -= y.y;
    return h;
}

// Row r of the staged bf16 Q tile as high and low E4M3 parts of row * 2^a, with
// 2^a putting the row's largest magnitude into [128, 256); returns 2^-a.  PARTS
// threads share a row, each writing its part (and COPIES of it, one tile of BM /
// COPIES rows behind the other): the first scores wait for it (a chunk of 128
// tokens over 2176 keys, 32/8 heads: 16.5 us with one thread per row, 16.0 with two).
template <int D, int PARTS, int COPIES>
__device__ __forceinline__ float split_q_row(const bf16 *staged, uint8_t *hi, uint8_t *lo, int r,
                                             int part)
{
    auto chunk = [&](int c) {  // eight elements
        return *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(staged) +
                                                (c >> 3) * (BM * 128) + r * 128 +
                                                (((c & 7) ^ (r & 7)) << 4));
    };
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < D / 8; c++) {
        float x[8];
        bf16x8_to_f32(chunk(c), x);
#pragma unroll
        for (int i = 0; i < 8; i++)
            amax = fmaxf(amax, fabsf(x[i]));
    }
    const int e = min(261 - (int)(__float_as_uint(amax) >> 23), 254);  // 2^a = 2^(e - 127)
    const float up = __uint_as_float((uint32_t)e << 23);
#pragma unroll 2
    for (int i0 = 0; i0 < D / 16 / PARTS; i0++) {
        const int c = part * (D / 16 / PARTS) + i0;
        uint32_t h[4], l[4];
#pragma unroll
        for (int half = 0; half < 2; half++) {
            float x[8];
            bf16x8_to_f32(chunk(2 * c + half), x);
            uint32_t hh[4], ll[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float x0 = x[2 * i] * up, x1 = x[2 * i + 1] * up;
                hh[i] = e4m3x2_split(x0, x1);
                ll[i] = e4m3x2_split(x0, x1);
            }
            h[2 * half] = hh[0] | (hh[1] << 16);
            h[2 * half + 1] = hh[2] | (hh[3] << 16);
            l[2 * half] = ll[0] | (ll[1] << 16);
            l[2 * half + 1] = ll[2] | (ll[3] << 16);
        }
        const uint32_t at = byte_chunk_off<D>(r, c);
#pragma unroll
        for (int i = 0; i < COPIES; i++) {
            const uint32_t to = at + i * (BM / COPIES) * D;
            *reinterpret_cast<uint4 *>(hi + to) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(lo + to) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
    return e8m0_value((uint32_t)(254 - e));
}

// Up to kRankBatch sequences of a paged call go to the slots in order of
// decreasing end position, as up to 32 do by shuffles: one thread per sequence
// counts those ahead of it.  (64 sequences of 512 .. 8192 keys, 512 units on 152
// SMs: 197 us in table order, 156 us so.)  Called by all threads of a CTA
// of at least 256; every thread gets the sequence of `slot`.
constexpr int kRankBatch = 256;

struct RankScratch {
    int4 keys[kRankBatch / 4];
    int4 found;
};

__device__ __forceinline__ void rank_sequences(const PrefillParams &p, RankScratch &sc, int slot,
                                               int &b, int &tok0, int &n_new, int &prior)
{
    const int t = threadIdx.x;
    int c0 = 0, c1 = 0, pl = 0, key = INT_MIN;
    if (t < kRankBatch) {
        if (t < p.batch) {
            c0 = __ldg(p.cu_seqlens + t);
            c1 = __ldg(p.cu_seqlens + t + 1);
            pl = __ldg(p.cache_lens + t);
            key = pl + (c1 - c0);
        }
        reinterpret_cast<int *>(sc.keys)[t] = key;
    }
    __syncthreads();
    if (t < p.batch) {
        int rank = 0;
        for (int j = 0; j < p.batch; j += 4) {  // entries past the batch are INT_MIN
            const int4 k = sc.keys[j / 4];
            rank += (k.x > key) || (k.x == key && j < t);
            rank += (k.y > key) || (k.y == key && j + 1 < t);
            rank += (k.z > key) || (k.z == key && j + 2 < t);
            rank += (k.w > key) || (k.w == key && j + 3 < t);
        }
        if (rank == slot)
            sc.found = make_int4(t, c0, c1 - c0, pl);
    }
    __syncthreads();
    // through a shuffle: the compiler then knows them the same across the warp
    // (without, the tile loop ran 17% slower)
    const int4 f = sc.found;
    b = __shfl_sync(0xffffffffu, f.x, 0);
    tok0 = __shfl_sync(0xffffffffu, f.y, 0);
    n_new = __shfl_sync(0xffffffffu, f.z, 0);
    prior = __shfl_sync(0xffffffffu, f.w, 0);
}

// The work of a CTA.  REP: the tile's rows fill 128 / REP lanes, REP times over
// (paged calls).
template <int D, bool CAPPED, KvSource SRC, int REP>
__device__ __forceinline__ void prefill_tile(const PrefillParams &p, const PagedView &pg,
                                             const CUtensorMap &map_q, const CUtensorMap &map_k,
                                             const CUtensorMap &map_v)
{
    typedef TcSmem<D, SRC> Smem;
    constexpr int KB = D / 64;
    constexpr int KST = Smem::KST, VST = Smem::VST;
    constexpr bool PAGED = SRC != KV_CONTIGUOUS, E4M3 = SRC == KV_PAGED_E4M3;
    constexpr bool PAIR = E4M3 && REP == 1;   // two softmax groups
    constexpr int CONVERT0 = PAIR ? 12 : 8;   // first of the converting warps
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~uintptr_t(1023));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Prologue that reads no global memory: descriptor prefetch, barriers and
    // tensor memory; it may overlap the end of the previous kernel.
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
        mbar_init(&sm.q_full, 1);
        for (int s = 0; s < KST; s++) {
            mbar_init(&sm.k_full[s], 1);
            mbar_init(&sm.k_empty[s], 1);
        }
        for (int s = 0; s < VST; s++) {  // filled by copies, or by the converting warps
            mbar_init(&sm.v_full[s], E4M3 ? 4 : 1);
            mbar_init(&sm.v_empty[s], 1);
        }
        if constexpr (E4M3) {
            mbar_init(&sm.q_split, PAIR ? 8 : 4);
            for (int s = 0; s < RAW_STAGES; s++) {
                mbar_init(&sm.raw_full[s], 1);
                mbar_init(&sm.raw_empty[s], 4);
            }
        }
        for (int s = 0; s < NUM_S; s++) {
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.s_free[s], 1);
            mbar_init(&sm.p_full[s], PAIR ? 8 : 4);
        }
        for (int s = 0; s < NUM_S; s++)
            mbar_init(&sm.o_done[s], 1);
        mbar_init(&sm.drain[0], 1);
        mbar_init(&sm.drain[1], 1);
        sm.abort_flag = 0;
        if constexpr (PAIR)
            for (int i = 0; i < 4; i++)
                sm.pair_failed[i] = 0;
        fence_barrier_init();
    }
    // The block's unit: CTAs 0 .. full_units - 1 take whole units, the rest one
    // of num_splits key ranges of a tail unit.  Units run in the order
    // (query tile, head group, sequence slot), heaviest query tiles first.
    const int idx = blockIdx.x;
    const bool in_tail = idx >= p.full_units;
    const int nsplit = in_tail ? p.num_splits : 1;
    const int tail_unit = in_tail ? (idx - p.full_units) / p.num_splits : 0;
    const int split = in_tail ? (idx - p.full_units) - tail_unit * p.num_splits : 0;
    const int unit = in_tail ? p.full_units + tail_unit : idx;
    const int hg = (unit / p.q_tiles) % p.HG;
    const int slot = unit / (p.q_tiles * p.HG);
    const int qt = p.q_tiles - 1 - (unit % p.q_tiles);  // heaviest (latest) query tiles first
    // A tile that certainly has rows -- a sequence's first, or with a single
    // sequence any tile below the host-known token count -- takes the tensor
    // memory before the wait and issues its first copies speculatively.
    // Other tiles may be empty padding; they check first and leave at once.
    const bool eager = !PAGED && p.batch == 1 && p.window == 0 &&
                       qt * p.tile_tokens < p.total_tokens;
    if (eager && warp == 1)
        tc::tmem_alloc(&sm.tmem_base, TMEM_COLS);
    grid_dependency_wait();
    grid_dependents_launch();

    // ------------------------------------------------------------ the tile --
    // The 128 rows are tile_tokens tokens x pack query heads of one kv group,
    // token-major: row r is token r >> pack_shift, head h0 + (r & (pack - 1)).
    // (Paged calls pack groups that are no power of two as well.)
    const int pack_shift = __ffs(p.pack) - 1;
    auto tok_of = [&](int r) { return PAGED ? (r * p.pack_inv) >> 16 : r >> pack_shift; };
    auto head_of = [&](int r) { return PAGED ? r - tok_of(r) * p.pack : r & (p.pack - 1); };
    const int h0 = hg * p.pack;
    const int kvh = h0 / p.group;
    const int r0 = qt * p.tile_tokens;  // first token of the tile within the sequence
    const int split_off = nsplit > 1 ? split * p.split_len : 0;
    // The sequence this block serves.  With several sequences (up to 32) the
    // slots go to sequences in order of decreasing end position (prior + new
    // tokens), so the longest tiles start first (list scheduling of this
    // one-CTA-per-SM grid: measured ~10% shorter on mixed lengths).  The
    // bounds of every sequence come in the same round of loads.
    int b = slot, tok0, n_new, prior;
    if (PAGED && p.batch > 32 && p.batch <= kRankBatch) {
        // in the K ring, which is loaded only after the CTA's next barrier
        rank_sequences(p, *reinterpret_cast<RankScratch *>(&sm.k[0]), slot, b, tok0, n_new, prior);
        tc::fence_proxy_async_smem();
    } else if (p.batch > 1 && p.batch <= 32) {
        int c0 = 0, c1 = 0, pl = 0, key = -1;
        if (lane < p.batch) {
            c0 = __ldg(p.cu_seqlens + lane);
            c1 = __ldg(p.cu_seqlens + lane + 1);
            pl = __ldg(p.cache_lens + lane);
            key = pl + (c1 - c0);
        }
        int rank = 0;
        for (int j = 0; j < p.batch; j++) {
            const int kj = __shfl_sync(0xffffffffu, key, j);
            rank += (kj > key) || (kj == key && j < lane);
        }
        const unsigned m = __ballot_sync(0xffffffffu, lane < p.batch && rank == slot);
        const int src = __ffs(m) - 1;  // ranks are a permutation of 0 .. batch - 1
        b = src;
        tok0 = __shfl_sync(0xffffffffu, c0, src);
        n_new = __shfl_sync(0xffffffffu, c1, src) - tok0;
        prior = __shfl_sync(0xffffffffu, pl, src);
    }
    const int spec_row = (b * p.KV + kvh) * p.capacity + split_off;  // tile 0 without a window
    // K/V tiles that no other CTA of the call reads (one query tile holding
    // every query head of its kv group) are loaded first in line for L2
    // eviction, so streaming them does not push out lines worth keeping.
    const bool read_once = p.kv_read_once != 0;
    const uint64_t kv_policy = l2_policy_evict_first();
    auto load_kv = [&](void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
        if (read_once)
            tc::tma_load_2d_hint(dst, map, x, y, bar, kv_policy);
        else
            tc::tma_load_2d(dst, map, x, y, bar);
    };
    // With a single sequence the first K and V tiles depend only on the block,
    // and its tokens start at row 0: those copies are issued before the
    // sequence bounds arrive, overlapping that round trip (a CTA that turns out
    // to have no work waits for them before it exits).
    const bool early_q = eager;
    if constexpr (!PAGED) {
        if (eager && threadIdx.x == 0) {
            mbar_arrive_expect_tx(&sm.q_full, KB * BM * 128);
            for (int kb = 0; kb < KB; kb++)
                tc::tma_load_3d(sm.q[kb], &map_q, kb * 64, h0, r0, &sm.q_full);
            mbar_arrive_expect_tx(&sm.k_full[0], KB * BN * 128);
            for (int kb = 0; kb < KB; kb++)
                load_kv(sm.k[0][kb], &map_k, kb * 64, spec_row, &sm.k_full[0]);
            mbar_arrive_expect_tx(&sm.v_full[0], KB * BN * 128);
            for (int kb = 0; kb < KB; kb++)
                load_kv(sm.v[0][kb], &map_v, kb * 64, spec_row, &sm.v_full[0]);
        }
    }
    if (!(p.batch > 1 && p.batch <= (PAGED ? kRankBatch : 32))) {
        tok0 = __ldg(p.cu_seqlens + b);
        n_new = __ldg(p.cu_seqlens + b + 1) - tok0;
        prior = __ldg(p.cache_lens + b);
    }
    const int rows_tok = min(p.tile_tokens, n_new - r0);
    const int rows = PAGED ? rows_tok * p.pack : rows_tok << pack_shift;  // valid tensor-memory rows
    const int pos_lo = prior + r0, pos_hi = prior + r0 + rows_tok - 1;
    // Keys the tile can see: from the key tile holding the first row's window
    // start (0 without a window) to the last row; splits cut that range.
    const int win_tile = p.window > 0 ? max(0, pos_lo - p.window + 1) / BN * BN : 0;
    const int k_begin = win_tile + split_off;
    // Cache row of key tile j: with a ring the key position wraps at the
    // capacity (a multiple of the key tile, so a tile never straddles the end).
    const bool ring = (p.flags & NA_RING_CACHE) != 0;
    const int kv_row0 = (b * p.KV + kvh) * p.capacity;
    auto tile_row = [&](int j) {
        const int k = k_begin + j * BN;
        return kv_row0 + (ring ? k % p.capacity : k);
    };
    int k_end = pos_hi + 1;
    if (nsplit > 1)
        k_end = min(k_end, k_begin + p.split_len);
    bool run = true;  // uniform over the CTA
    // A sequence must lie inside the call's tokens (cu_seqlens within
    // [0, total_tokens]): its rows are read from Q and written to out.
    if (n_new > p.max_new_len || (b == 0 && tok0 != 0) || tok0 < 0 ||
        (long long)tok0 + n_new > p.total_tokens) {
        if (qt == 0 && hg == 0 && split == 0 && threadIdx.x == 0)
            na_report(p.status, NA_ERR_INVALID_ARG);
        run = false;
    } else if (r0 >= n_new) {
        run = false;
    } else if (prior < 0 || (!ring && pos_hi >= p.capacity) || pos_hi >= p.max_total_len) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_CAPACITY);
        run = false;
    } else if (k_begin >= k_end) {
        run = false;
    }
    if (!run) {
        if (eager) {  // let the early copies land, give the tensor memory back
            if (threadIdx.x == 0) {
                if (early_q)
                    drain_wait(&sm.q_full, 0, p.status);
                drain_wait(&sm.k_full[0], 0, p.status);
                drain_wait(&sm.v_full[0], 0, p.status);
            }
            tc::fence_before_sync();
            __syncthreads();
            if (warp == 1) {
                tc::fence_after_sync();
                tc::tmem_dealloc(sm.tmem_base, TMEM_COLS);
            }
        }
        return;
    }
    if (!eager && warp == 1)
        tc::tmem_alloc(&sm.tmem_base, TMEM_COLS);
    const int n_tiles = (k_end - k_begin + BN - 1) / BN;
    // tiles loaded before the barrier (of pages none: their ids come first)
    const int pre = n_tiles < STAGES ? n_tiles : STAGES;
    // first key that any row sees: pages before it may be gone
    const int vis_lo = p.window > 0 ? max(k_begin, pos_lo - p.window + 1) : k_begin;

    if (threadIdx.x == 0) {
        // The Q tile (unless already issued) and the remaining first ring
        // stages go out before the CTA-wide barrier (fresh stages need no
        // wait), so these copies overlap the tensor-memory allocation and the
        // barrier itself.
        if (!early_q) {
            // (a paged box holds tile_tokens x pack rows, 128 / REP of them at most)
            mbar_arrive_expect_tx(&sm.q_full,
                                  PAGED ? REP * KB * p.pack * p.tile_tokens * 128 : KB * BM * 128);
            for (int kb = 0; kb < KB; kb++) {
                bf16 *dst;
                if constexpr (E4M3)
                    dst = sm.v[0][kb];
                else
                    dst = sm.q[kb];
                for (int i = 0; i < REP; i++)
                    tc::tma_load_3d(dst + i * (BM / REP) * 64, &map_q, kb * 64, h0, tok0 + r0,
                                    &sm.q_full);
            }
        }
        if constexpr (!PAGED) {
            for (int j = eager ? 1 : 0; j < pre; j++) {
                mbar_arrive_expect_tx(&sm.k_full[j], KB * BN * 128);
                for (int kb = 0; kb < KB; kb++)
                    load_kv(sm.k[j][kb], &map_k, kb * 64, tile_row(j), &sm.k_full[j]);
                mbar_arrive_expect_tx(&sm.v_full[j], KB * BN * 128);
                for (int kb = 0; kb < KB; kb++)
                    load_kv(sm.v[j][kb], &map_v, kb * 64, tile_row(j), &sm.v_full[j]);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;

    // Output rows are staged in shared memory by the softmax warps (they hold
    // the tensor-memory lanes) and then stored by all eight warps, SR rows
    // each: one warp per sub-partition storing 32 rows back to back was
    // latency-bound (~1.5 us per CTA, 3.3 us with the gate).  A warp's gate
    // words for its rows are requested early -- warps 0-3 now, the softmax
    // warps after their last tile.
    constexpr int LDS = D + 4;   // staged row stride (floats): conflict-free row writes
    constexpr int EPL = D / 32;  // elements per lane in the row stores
    constexpr int GW = D / 64;   // 32-bit words of gate per lane and row
    constexpr int SW = PAIR ? 16 : 8;  // storing warps
    constexpr int SR = BM / REP / SW;  // rows stored per warp
    float *stage = reinterpret_cast<float *>(&sm.k[0]);  // the K ring (and what follows), idle by then
    const bool split_out = nsplit > 1;
    // rows of this piece in the workspace: [tail unit][split][row]
    const size_t piece_row0 = ((size_t)tail_unit * p.num_splits + split) * BM;
    const bool gated_out = !split_out && (p.flags & NA_OUT_GATE) && p.gate;
    uint32_t gq[SR][GW];
    auto load_gate = [&]() {
#pragma unroll
        for (int i = 0; i < SR; i++) {
            const int rr = warp * SR + i;
            const size_t off = ((size_t)(tok0 + r0 + tok_of(rr)) * p.H + h0 + head_of(rr)) * D +
                               lane * 2 * GW;
            gq[i][0] = 0;
            if constexpr (GW == 2)
                gq[i][1] = 0;
            if (rr < rows) {
                if constexpr (GW == 2) {
                    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p.gate + off));
                    gq[i][0] = u.x;
                    gq[i][1] = u.y;
                } else {
                    gq[i][0] = __ldg(reinterpret_cast<const unsigned int *>(p.gate + off));
                }
            }
        }
    };
    if (!E4M3 && warp < 4 && gated_out)  // (E4M3: the registers are needed, all load at the end)
        load_gate();

    auto softmax = [&]() {
        // ------------------------------------------------------- softmax --
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;  // TMEM lane
        const int rq = r & (BM / REP - 1);  // its query row
        const int row_pos = pos_lo + tok_of(rq);
        // the 32-column blocks of a score tile that this warp takes
        constexpr int NC = PAIR ? 2 : 4 / REP;
        const int group = PAIR ? (warp - 4) >> 2 : 0;
        const int c0 = PAIR ? 2 * group : (REP == 1 ? 0 : quarter / (4 / REP) * NC);
        const int row_lo = p.window > 0 ? row_pos - p.window + 1 : INT_MIN;  // first visible key
        constexpr bool capped = CAPPED;
        // soft-capped scores, kept in the raw score's units so the rest of the
        // softmax is unchanged: s' = (c / scale) tanh(s scale / c), with
        // tanh(y) = 1 - 2 / (e^(2y) + 1)
        const float cap_in = capped ? 2.0f * p.scale_log2 / p.softcap : 0.f;
        const float cap_out = capped ? p.softcap * NA_LOG2E / p.scale_log2 : 0.f;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t o_t = tmem + lane_off;
        float sl2 = p.scale_log2;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        if constexpr (E4M3) {
            ok = warp_wait(&sm.q_full, 0, &sm.abort_flag);
            if (ok) {  // the row by two threads, or (REP) each of its four copies a part of it
                if constexpr (PAIR)
                    sl2 *= split_q_row<D, 2, 1>(sm.v[0][0], sm.q8[0], sm.q8[1], r, group);
                else
                    sl2 *= split_q_row<D, REP, REP>(sm.v[0][0], sm.q8[0], sm.q8[1], rq, quarter);
                tc::fence_proxy_async_smem();  // before the tensor core's reads
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.q_split);
            }
        }
        for (int j = 0; (PAIR || ok) && j < n_tiles; j++) {
            const int sb = j % NUM_S;
            const int j0 = k_begin + j * BN;
            const uint32_t s_t = tmem + S_COL0 * (sb + 1) + lane_off;
            // (PAIR: a failed wait is told at the tile's barrier, and both warps leave)
            if (!(ok && warp_wait(&sm.s_full[sb], (j / NUM_S) & 1, &sm.abort_flag))) {
                ok = false;
                if constexpr (PAIR) {
                    if (lane == 0) {
                        *(volatile int *)&sm.pair_failed[quarter] = 1;
                        set_abort(&sm.abort_flag, p.status);
                    }
                    __syncwarp();
                    named_barrier_sync(2 + quarter, 64);
                }
                break;
            }
            tc::fence_after_sync();
            uint32_t sr[NC][32];
#pragma unroll
            for (int c = 0; c < NC; c++)
                tc::tmem_ld32(s_t + (c0 + c) * 32, sr[c]);
            // E4M3: what turns a raw score of 16 keys into the log2 domain (the soft
            // cap leaves it there), V's exponents in the weights, and 2^-those;
            // requested with the scores, since shared memory answers late while the
            // tensor cores read it.
            float4 mul_off[NC];
            float2 v_inv[NC];
            if constexpr (E4M3) {
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(mul_off[c].x), "=f"(mul_off[c].y), "=f"(mul_off[c].z),
                                   "=f"(mul_off[c].w)
                                 : "r"(smem_addr(&sm.mul_off[j % SCALE_SLOTS][c0 + c])));
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                                 : "=f"(v_inv[c].x), "=f"(v_inv[c].y)
                                 : "r"(smem_addr(&sm.v_inv[j % SCALE_SLOTS][c0 + c])));
                    // positive: masked scores are -inf
                    mul_off[c].x = fmaxf(mul_off[c].x * sl2, 1.2e-38f);
                    mul_off[c].y = fmaxf(mul_off[c].y * sl2, 1.2e-38f);
                }
            }
            tc::tmem_wait_ld();

            if constexpr (capped && E4M3) {
                const float in = 2.0f / p.softcap, out = p.softcap * NA_LOG2E;
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const float4 mo = mul_off[c];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const float e = ex2_mufu(__uint_as_float(sr[c][i]) * (i < 16 ? mo.x : mo.y) * in);
                        sr[c][i] = __float_as_uint(out * (1.0f - __fdividef(2.0f, e + 1.0f)));
                    }
                }
            } else if constexpr (capped) {
#pragma unroll
                for (int c = 0; c < NC; c++)
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const float e = ex2_mufu(__uint_as_float(sr[c][i]) * cap_in);
                        sr[c][i] = __float_as_uint(cap_out * (1.0f - __fdividef(2.0f, e + 1.0f)));
                    }
            }
            const bool need_mask = (j0 + BN - 1 > pos_lo) || (j0 + BN > k_end) || (j0 < row_lo);
            if (need_mask) {
#pragma unroll
                for (int c = 0; c < NC; c++)
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const int key = j0 + (c0 + c) * 32 + i;
                        if (key > row_pos || key >= k_end || key < row_lo)
                            sr[c][i] = __float_as_uint(-INFINITY);
                    }
            }
            // row maximum: four independent chains of 3-input max (E4M3: two per 32
            // keys, of score + V's exponent)
            float mxs;
            if constexpr (E4M3) {
                float mg[2 * NC];
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const float4 mo = mul_off[c];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t *x = &sr[c][16 * h];
                        float m0 = max3f(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
                        float m1 = max3f(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
                        m0 = max3f(m0, __uint_as_float(x[6]), __uint_as_float(x[7]));
                        m1 = max3f(m1, __uint_as_float(x[8]), __uint_as_float(x[9]));
                        m0 = max3f(m0, __uint_as_float(x[10]), __uint_as_float(x[11]));
                        m1 = max3f(m1, __uint_as_float(x[12]), __uint_as_float(x[13]));
                        m0 = max3f(m0, __uint_as_float(x[14]), __uint_as_float(x[15]));
                        const float mul = capped ? 1.0f : (h ? mo.y : mo.x);
                        mg[2 * c + h] = fmaf(fmaxf(m0, m1), mul, h ? mo.w : mo.z);
                    }
                }
                mxs = fmaxf(mg[0], mg[1]);
#pragma unroll
                for (int c = 1; c < NC; c++)
                    mxs = max3f(mxs, mg[2 * c], mg[2 * c + 1]);
            } else {
            float mxa = -INFINITY, mxb = -INFINITY, mxc = -INFINITY, mxd = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    mxa = max3f(mxa, __uint_as_float(sr[c][i]), __uint_as_float(sr[c][i + 1]));
                    mxb = max3f(mxb, __uint_as_float(sr[c][i + 2]), __uint_as_float(sr[c][i + 3]));
                    mxc = max3f(mxc, __uint_as_float(sr[c][i + 4]), __uint_as_float(sr[c][i + 5]));
                    mxd = max3f(mxd, __uint_as_float(sr[c][i + 6]), __uint_as_float(sr[c][i + 7]));
                }
            const float mx = max3f(mxa, mxb, fmaxf(mxc, mxd));
            mxs = mx * sl2;
            }
            if constexpr (PAIR) {  // the other half of the row
                sm.pair_max[j & 1][group][r] = mxs;
                named_barrier_sync(2 + quarter, 64);
                if (*(volatile int *)&sm.pair_failed[quarter]) {
                    ok = false;
                    break;
                }
                mxs = fmaxf(mxs, sm.pair_max[j & 1][group ^ 1][r]);
            }
            float alpha = 1.f;
            bool corr = false;
            constexpr float TOP = E4M3 ? kF16Top : 0.f, LIMIT = E4M3 ? kF16Limit : 8.0f;
            if (mxs > m_ref + LIMIT) {
                alpha = (m_ref == -INFINITY) ? 0.f : ex2_mufu(m_ref - (mxs - TOP));
                corr = (m_ref != -INFINITY);
                m_ref = mxs - TOP;
            }
            const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < NC; c++) {
                uint32_t pk[16];
                float4 mo = mul_off[c];
                const float2 inv = v_inv[c];
                if constexpr (E4M3 && capped)
                    mo.x = mo.y = 1.0f;
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const float sc = E4M3 ? (i < 8 ? mo.x : mo.y) : sl2;
                    const float nm = E4M3 ? neg_m + (i < 8 ? mo.z : mo.w) : neg_m;
                    const float2 x = __ffma2_rn(
                        make_float2(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1])),
                        make_float2(sc, sc), make_float2(nm, nm));
                    const float2 pp = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
                    if constexpr (E4M3) {
                        const float w = i < 8 ? inv.x : inv.y;
                        acc[i & 3] = __ffma2_rn(pp, make_float2(w, w), acc[i & 3]);
                        pk[i] = pack_f16x2(pp.x, pp.y);
                    } else {
                        acc[i & 3] = __fadd2_rn(acc[i & 3], pp);
                        pk[i] = pack_bf16x2(pp.x, pp.y);
                    }
                }
                tc::tmem_st16(s_t + (c0 + c) * 16, pk);
            }
            const float2 acc01 = __fadd2_rn(acc[0], acc[1]), acc23 = __fadd2_rn(acc[2], acc[3]);
            const float rs = (acc01.x + acc01.y) + (acc23.x + acc23.y);
            if constexpr (REP > 1) {  // the other warps' keys weigh nothing in these lanes
                const uint32_t none[16] = {};
#pragma unroll
                for (int c = 1; c < REP; c++)
                    tc::tmem_st16(s_t + ((c0 + c * NC) & 3) * 16, none);
                static_assert(NC == 1, "one column block per warp");
            }
            tc::tmem_wait_st();

            if (!E4M3 && (j0 + BN > k_end || (PAGED && j0 < vis_lo))) {
                // Key rows past the valid range hold whatever the cache has there
                // (and with pages so do those before the window: their page may
                // be gone); zero them so P * V sees no non-finite values.  (E4M3:
                // the converting warps do.)
                const int st = j % VST;
                if (!warp_wait(&sm.v_full[st], (j / VST) & 1, &sm.abort_flag)) {
                    ok = false;
                    break;
                }
                if (r >= k_end - j0 || (PAGED && r < vis_lo - j0)) {
#pragma unroll
                    for (int kb = 0; kb < KB; kb++) {
                        uint4 *row = reinterpret_cast<uint4 *>(sm.v[st][kb] + r * 64);
#pragma unroll
                        for (int c = 0; c < 8; c++)
                            row[c] = make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_proxy_async_smem();
            }
            // O is touched here only to rescale it (rare), and then PV(j-1) must
            // have landed.  PV(j) commits to o_done[j % NUM_S], so a wait there is
            // exact however rarely the softmax looks: the barrier's previous
            // phase, PV(j-1-NUM_S), completed before S(j-1) could be issued (its
            // S buffer had to be free), and its next one, PV(j-1+NUM_S), needs a
            // P this warp has not written yet.  Waiting for PV(j-1) on every tile
            // kept PV(j) from being queued behind it.
            if (j >= 1 && group == 0 && __any_sync(0xffffffffu, corr)) {
                if (!warp_wait(&sm.o_done[(j - 1) % NUM_S], ((j - 1) / NUM_S) & 1, &sm.abort_flag)) {
                    ok = false;
                    if constexpr (PAIR)
                        continue;  // to the next tile's barrier
                    break;
                }
                // rescale this warp's O rows (PV(j-1) has landed)
                tc::fence_after_sync();
                const float a = corr ? alpha : 1.f;
#pragma unroll
                for (int c = 0; c < D / 32; c++) {
                    uint32_t o[32];
                    tc::tmem_ld32(o_t + c * 32, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                    tc::tmem_st32(o_t + c * 32, o);
                }
                tc::tmem_wait_st();
            }
            l = l * alpha + rs;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.p_full[sb]);
        }
        // This warp's gate rows, requested now so their latency overlaps the
        // last P V product.
        if (!E4M3 && ok && gated_out)
            load_gate();
        const bool done = ok && warp_wait(&sm.o_done[(n_tiles - 1) % NUM_S],
                                          ((n_tiles - 1) / NUM_S) & 1, &sm.abort_flag);
        float2 *ml = reinterpret_cast<float2 *>(stage + BM * LDS);  // REP: (reference, sum) per lane
        if constexpr (REP > 1) {  // joined by every softmax warp, whatever became of its waits
            ml[r] = make_float2(m_ref, l);
            named_barrier_sync(1, BM);
        }
        if constexpr (PAIR) {  // the row's two sums (one reference)
            sm.pair_max[0][group][r] = l;
            named_barrier_sync(1, 2 * BM);
            l += sm.pair_max[0][group ^ 1][r];
        }
        if (done) {
            // ---------------------------------------------------- epilogue --
            // Each thread writes its O row (normalised unless this is a split
            // partial) into the idle K ring, rows padded by 16 bytes so the
            // row-per-thread writes are bank-conflict free; then each warp
            // stores its 32 rows one row per instruction, coalesced.
            tc::fence_after_sync();
            float scale = split_out ? 1.0f : (l > 0.f ? 1.0f / l : 0.f);
            if constexpr (REP > 1) {  // the row's partials: their weights against each other
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int i = 0; i < REP; i++)
                    M = fmaxf(M, ml[rq + i * (BM / REP)].x);
#pragma unroll
                for (int i = 0; i < REP; i++) {
                    const float2 x = ml[rq + i * (BM / REP)];
                    if (x.x != -INFINITY)
                        L = fmaf(x.y, ex2_mufu(x.x - M), L);
                }
                scale = m_ref == -INFINITY ? 0.f : ex2_mufu(m_ref - M);
                if (!split_out)
                    scale *= L > 0.f ? 1.0f / L : 0.f;
                m_ref = M;
                l = L;
            }
            {
                constexpr int OC = PAIR ? D / 64 : D / 32;  // column blocks of O (PAIR: half each)
                const int oc0 = group * OC;
                uint32_t o[OC][32];  // in one round of loads
#pragma unroll
                for (int c = 0; c < OC; c++)
                    tc::tmem_ld32(o_t + (oc0 + c) * 32, o[c]);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < OC; c++) {
                    float4 *row4 = reinterpret_cast<float4 *>(stage + r * LDS + (oc0 + c) * 32);
#pragma unroll
                    for (int q = 0; q < 8; q++)
                        row4[q] = make_float4(__uint_as_float(o[c][4 * q]) * scale,
                                              __uint_as_float(o[c][4 * q + 1]) * scale,
                                              __uint_as_float(o[c][4 * q + 2]) * scale,
                                              __uint_as_float(o[c][4 * q + 3]) * scale);
                }
            }
            if (split_out && group == 0 && r < rows) {
                p.part_ml[(piece_row0 + r) * 2] = m_ref;
                p.part_ml[(piece_row0 + r) * 2 + 1] = l;
            }
        } else if (lane == 0) {
            set_abort(&sm.abort_flag, p.status);
        }
    };
    // (The order of the roles is measured, for each source its own: drafted tokens over
    // E4M3 pages take 124.0 us so and 125.5 in the contiguous order; the other way round
    // below.)
    if (!PAGED || warp < 4) {
        if (PAGED && warp == 0) {
            // ------------------------------------------------ producer, pages --
            const int page_log = pg.page_log, nbox = BN >> page_log;  // 8 .. 1 boxes of rows per tile
            constexpr int COLS = E4M3 ? 1 : KB;
            constexpr uint32_t BOX_ROW = E4M3 ? D : 128;
            const int bi = lane & (nbox - 1), bc = lane / nbox;  // this lane's box: rows, columns
            const int p_lo = vis_lo >> page_log, p_hi = (k_end - 1) >> page_log;
            const int32_t *row = pg.table + (size_t)b * pg.pages_per_seq;
            struct Entry {
                int id;
                uint32_t scales;  // K's byte | V's byte << 8
            };
            auto entry = [&](int i) {
                Entry e{-1, 0x7f7fu};
                if (i >= p_lo && i <= p_hi) {
                    e.id = __ldcg(row + i);
                    if ((unsigned)e.id >= (unsigned)pg.num_pages) {  // reported; page 0 is read instead
                        na_report(p.status, NA_ERR_PAGE);
                        e.id = 0;
                    }
                    if constexpr (E4M3) {
                        const size_t at = (size_t)e.id * p.KV + kvh;
                        const uint32_t vs = __ldcg(pg.v_scale + at);
                        if ((int)vs - 127 > kTopVExp)
                            na_report(p.status, NA_ERR_UNSUPPORTED);
                        e.scales = (uint32_t)__ldcg(pg.k_scale + at) | (vs << 8);
                    }
                }
                return e;
            };
            int wb = k_begin >> page_log;  // page of lane 0's current entry
            Entry cur = entry(wb + lane), nxt = entry(wb + 32 + lane);
            bool ok = true;
            auto wait_all = [&](uint64_t *bar, uint32_t parity) {
                const bool got = mbar_wait_bounded(bar, parity) && !aborted(&sm.abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    if (lane == 0)
                        set_abort(&sm.abort_flag, p.status);
                    return false;
                }
                return true;
            };
            // One tile's boxes into dst, completing on bar.
            auto load_tile = [&](const CUtensorMap *map, int id, int n, uint8_t *dst, uint64_t *bar) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, n * (BOX_ROW << page_log));
                __syncwarp();
                if (id >= 0)
                    load_kv(dst + bc * (BN * 128) + (bi << page_log) * BOX_ROW, map, bc * 64,
                            (id * p.KV + kvh) << page_log, bar);
            };
            int k_issued = 0, v_issued = 0;
            for (int j = 0; ok && j < n_tiles; j++) {
                const int j0 = k_begin + j * BN;
                if ((j0 >> page_log) - wb >= 32) {
                    cur = nxt;
                    wb += 32;
                    nxt = entry(wb + 32 + lane);
                }
                int id = __shfl_sync(0xffffffffu, cur.id, ((j0 >> page_log) - wb + bi) & 31);
                if (bc >= COLS)
                    id = -1;
                const int n = __popc(__ballot_sync(0xffffffffu, id >= 0));
                const uint32_t scales = __shfl_sync(0xffffffffu, cur.scales,
                                                    (((j0 + 16 * (lane & 7)) >> page_log) - wb) & 31);
                const int ks = j % KST;
                if (!(ok = wait_all(&sm.k_empty[ks], ((j / KST) & 1) ^ 1)))
                    break;
                if constexpr (E4M3) {
                    if (lane < 8) {
                        const int slot = j % SCALE_SLOTS, e = v_weight_exp(scales >> 8);
                        float *mo = reinterpret_cast<float *>(&sm.mul_off[slot][lane >> 1]);
                        mo[lane & 1] = e8m0_value(scales & 255u);
                        mo[2 + (lane & 1)] = (float)e;
                        reinterpret_cast<float *>(&sm.v_inv[slot][lane >> 1])[lane & 1] = exp2i(-e);
                    }
                }
                load_tile(&map_k, id, n, reinterpret_cast<uint8_t *>(sm.k[ks]), &sm.k_full[ks]);
                k_issued = j + 1;
                if constexpr (E4M3) {
                    const int rs = j % RAW_STAGES;
                    if (!(ok = wait_all(&sm.raw_empty[rs], ((j / RAW_STAGES) & 1) ^ 1)))
                        break;
                    if (lane < 8)
                        sm.v_scale[rs][lane] = (uint8_t)(scales >> 8);
                    load_tile(&map_v, id, n, sm.raw[rs], &sm.raw_full[rs]);
                } else {
                    const int vs = j % VST;
                    if (!(ok = wait_all(&sm.v_empty[vs], ((j / VST) & 1) ^ 1)))
                        break;
                    load_tile(&map_v, id, n, reinterpret_cast<uint8_t *>(sm.v[vs]), &sm.v_full[vs]);
                }
                v_issued = j + 1;
            }
            // every copy issued lands before the CTA can exit
            if (lane == 0) {
                drain_wait(&sm.q_full, 0, p.status);
                for (int j = k_issued - 1; j >= 0 && j >= k_issued - KST; j--)
                    drain_wait(&sm.k_full[j % KST], (j / KST) & 1, p.status);
                constexpr int VR = E4M3 ? RAW_STAGES : VST;
                for (int j = v_issued - 1; j >= 0 && j >= v_issued - VR; j--) {
                    uint64_t *bar;
                    if constexpr (E4M3)
                        bar = &sm.raw_full[j % VR];
                    else
                        bar = &sm.v_full[j % VR];
                    drain_wait(bar, (j / VR) & 1, p.status);
                }
            }
        } else if (warp == 0) {
            // ------------------------------------------------------ producer --
            if constexpr (!PAGED) {
                if (lane == 0) {
                    int issued = pre;
                    for (int j = pre; j < n_tiles; j++) {
                        const int st = j % STAGES;
                        const uint32_t par = ((j / STAGES) & 1) ^ 1;
                        if (!mbar_wait_bounded(&sm.k_empty[st], par) || aborted(&sm.abort_flag)) {
                            set_abort(&sm.abort_flag, p.status);
                            break;
                        }
                        mbar_arrive_expect_tx(&sm.k_full[st], KB * BN * 128);
                        for (int kb = 0; kb < KB; kb++)
                            load_kv(sm.k[st][kb], &map_k, kb * 64, tile_row(j), &sm.k_full[st]);
                        if (!mbar_wait_bounded(&sm.v_empty[st], par) || aborted(&sm.abort_flag)) {
                            set_abort(&sm.abort_flag, p.status);
                            drain_wait(&sm.k_full[st], (j / STAGES) & 1, p.status);
                            break;
                        }
                        mbar_arrive_expect_tx(&sm.v_full[st], KB * BN * 128);
                        for (int kb = 0; kb < KB; kb++)
                            load_kv(sm.v[st][kb], &map_v, kb * 64, tile_row(j), &sm.v_full[st]);
                        issued = j + 1;
                    }
                    // every copy issued lands before the CTA can exit
                    drain_wait(&sm.q_full, 0, p.status);
                    for (int j = issued - 1; j >= 0 && j >= issued - STAGES; j--) {
                        drain_wait(&sm.k_full[j % STAGES], (j / STAGES) & 1, p.status);
                        drain_wait(&sm.v_full[j % STAGES], (j / STAGES) & 1, p.status);
                    }
                }
            }
        } else if (warp == 1) {
            // ---------------------------------------------------- S = Q K^T issue --
            if (lane == 0) {
                constexpr uint32_t idesc_s = E4M3 ? tc::idesc_e4m3_f32(BM, BN)
                                                  : tc::idesc_bf16_f32(BM, BN, false, false);
                // Descriptors of the Q tile and of K stage 0; a 64-wide column block
                // (BM = BN rows of 128 B) is BLK16 16-byte units, a K stage K_STAGE16.
                constexpr uint32_t BLK16 = (BM * 128) >> 4;
                constexpr uint32_t K_STAGE16 = (E4M3 ? BN * D : KB * BN * 128) >> 4;
                constexpr uint32_t Q_PART16 = (BM * D) >> 4;  // from the high to the low part (E4M3)
                static_assert(BM == BN, "one column-block stride for Q and K");
                uint64_t qd0, kd0;
                bool ok;
                if constexpr (E4M3) {
                    qd0 = tc::desc_kmajor_bytes<D>(smem_addr(sm.q8[0]));
                    kd0 = tc::desc_kmajor_bytes<D>(smem_addr(sm.k[0]));
                    ok = mbar_wait_bounded(&sm.q_split, 0);
                } else {
                    qd0 = tc::desc_kmajor_sw128(smem_addr(sm.q[0]));
                    kd0 = tc::desc_kmajor_sw128(smem_addr(sm.k[0][0]));
                    ok = mbar_wait_bounded(&sm.q_full, 0);
                }
                bool any = false;
                for (int j = 0; ok && j < n_tiles; j++) {
                    const int st = j % KST, sb = j % NUM_S;
                    ok = mbar_wait_bounded(&sm.k_full[st], (j / KST) & 1);
                    if (ok && j >= NUM_S)
                        ok = mbar_wait_bounded(&sm.s_free[sb], ((j / NUM_S) - 1) & 1);
                    if (!ok || aborted(&sm.abort_flag))
                        break;
                    tc::fence_after_sync();
                    const uint32_t s_t = tmem + S_COL0 * (sb + 1);
                    const uint64_t kd = kd0 + (uint64_t)(st * K_STAGE16);
                    if constexpr (E4M3) {
#pragma unroll
                        for (int k = 0; k < D / 32; k++)  // 32 bytes of d per step
                            tc::mma_ss_bytes(s_t, qd0 + k * 2, kd + k * 2, idesc_s, k > 0);
#pragma unroll
                        for (int k = 0; k < D / 32; k++)
                            tc::mma_ss_bytes(s_t, qd0 + Q_PART16 + k * 2, kd + k * 2, idesc_s, true);
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 16; k++) {  // descriptor start addresses advance in 16-byte units
                            const uint32_t off = (k >> 2) * BLK16 + (k & 3) * 2;
                            tc::mma_ss(s_t, qd0 + off, kd + off, idesc_s, k > 0);
                        }
                    }
                    tc::mma_commit(&sm.s_full[sb]);
                    tc::mma_commit(&sm.k_empty[st]);
                    any = true;
                }
                if (!ok)
                    set_abort(&sm.abort_flag, p.status);
                if (any) {  // all issued MMAs complete before tensor memory is released
                    tc::mma_commit(&sm.drain[0]);
                    drain_wait(&sm.drain[0], 0, p.status);
                }
            }
        } else if (warp == 2) {
            // --------------------------------------------------- O += P V issue --
            if (lane == 0) {
                constexpr uint32_t idesc_o = E4M3 ? tc::idesc_f16_f32(BM, D, false, true)
                                                  : tc::idesc_bf16_f32(BM, D, false, true);
                constexpr uint32_t V_STAGE16 = (KB * BN * 128) >> 4;  // a V stage in 16-byte units
                const uint64_t vd0 = tc::desc_mnmajor_sw128(smem_addr(sm.v[0][0]), BN * 128);
                bool ok = true, any = false;
                for (int j = 0; ok && j < n_tiles; j++) {
                    const int st = j % VST, sb = j % NUM_S;
                    ok = mbar_wait_bounded(&sm.p_full[sb], (j / NUM_S) & 1);
                    if (ok)
                        ok = mbar_wait_bounded(&sm.v_full[st], (j / VST) & 1);
                    if (!ok || aborted(&sm.abort_flag))
                        break;
                    tc::fence_after_sync();
                    const uint32_t p_t = tmem + S_COL0 * (sb + 1);
                    const uint64_t vd = vd0 + (uint64_t)(st * V_STAGE16);
#pragma unroll
                    for (int k = 0; k < BN / 16; k++)  // 16 keys = 16 rows of 128 B per step
                        tc::mma_ts(tmem, p_t + k * 8, vd + (uint64_t)(k * 128), idesc_o, j > 0 || k > 0);
                    tc::mma_commit(&sm.s_free[sb]);
                    tc::mma_commit(&sm.v_empty[st]);
                    tc::mma_commit(&sm.o_done[sb]);
                    any = true;
                }
                if (!ok)
                    set_abort(&sm.abort_flag, p.status);
                if (any) {
                    tc::mma_commit(&sm.drain[1]);
                    drain_wait(&sm.drain[1], 0, p.status);
                }
            }
        } else if (warp >= 4) {
            if constexpr (!PAGED)
                softmax();
        }
    } else if (E4M3 && warp >= CONVERT0) {
        // -------------------------------------- E4M3 V tiles to f16 tiles --
        if constexpr (E4M3) {
            for (int j = 0; j < n_tiles; j++) {
                const int rs = j % RAW_STAGES, st = j % VST;
                bool ok = warp_wait(&sm.raw_full[rs], (j / RAW_STAGES) & 1, &sm.abort_flag);
                if (ok && j == 0)  // the first V stage holds Q until it is split
                    ok = warp_wait(&sm.q_split, 0, &sm.abort_flag);
                if (ok)
                    ok = warp_wait(&sm.v_empty[st], ((j / VST) & 1) ^ 1, &sm.abort_flag);
                if (!ok) {
                    if (lane == 0)
                        set_abort(&sm.abort_flag, p.status);
                    break;
                }
                const int j0 = k_begin + j * BN;
                convert_tile<D>(sm.raw[rs], sm.v_scale[rs], sm.v[st][0], warp - CONVERT0, lane,
                                vis_lo - j0, k_end - j0);
                tc::fence_proxy_async_smem();  // before the tensor core's reads
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.v_full[st]);
                    mbar_arrive(&sm.raw_empty[rs]);
                }
            }
        }
    } else {
        if constexpr (PAGED)
            softmax();
    }
    if (E4M3 && warp < SW && gated_out)
        load_gate();

    tc::fence_before_sync();
    __syncthreads();  // the staged rows are complete (unless a wait gave up)
    if (!aborted(&sm.abort_flag) && warp < SW) {
        // Lanes across a row, one row per step, this warp's SR rows.
#pragma unroll
        for (int i = 0; i < SR; i++) {
            const int rr = warp * SR + i;
            if (rr >= rows)
                break;
            const float *src = stage + rr * LDS + lane * EPL;
            float v[EPL];
            if constexpr (EPL == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(src);
                v[0] = x.x;
                v[1] = x.y;
                v[2] = x.z;
                v[3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(src);
                v[0] = x.x;
                v[1] = x.y;
            }
            if constexpr (REP > 1) {  // the row's weighted partials
#pragma unroll
                for (int u = 1; u < REP; u++)
#pragma unroll
                    for (int e = 0; e < EPL; e++)
                        v[e] += src[u * (BM / REP) * LDS + e];
            }
            if (split_out) {
                float *dst = p.part_o + (piece_row0 + rr) * D + lane * EPL;
                if constexpr (EPL == 4)
                    *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                else
                    *reinterpret_cast<float2 *>(dst) = make_float2(v[0], v[1]);
                continue;
            }
            if (gated_out) {
#pragma unroll
                for (int e = 0; e < EPL; e += 2) {
                    const float g0 = __uint_as_float(gq[i][e / 2] << 16);
                    const float g1 = __uint_as_float(gq[i][e / 2] & 0xffff0000u);
                    v[e] *= __fdividef(1.0f, 1.0f + __expf(-g0));
                    v[e + 1] *= __fdividef(1.0f, 1.0f + __expf(-g1));
                }
            }
            uint32_t pk[EPL / 2];
#pragma unroll
            for (int e = 0; e < EPL; e += 2)
                pk[e / 2] = pack_bf16x2(v[e], v[e + 1]);
            const size_t tok = (size_t)(tok0 + r0 + tok_of(rr));
            const int h = h0 + head_of(rr);
            const size_t off = (tok * p.H + h) * D + lane * EPL;
            if constexpr (EPL == 4)
                *reinterpret_cast<uint2 *>(p.out + off) = make_uint2(pk[0], pk[1]);
            else
                *reinterpret_cast<uint32_t *>(p.out + off) = pk[0];
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// A contiguous cache's kernel has no page view among its parameters, and its roles
// in an order of their own: 16 chunks of 2048 tokens, 40/8 heads, with their appends
// take 7.51 ms, and took 7.64 as one more instance of the paged kernel (7.57 before
// there was one).  Registers and arithmetic are the same.
template <int D, bool CAPPED>
__global__ void __launch_bounds__(THREADS, 1)
    prefill_tc_kernel(const __grid_constant__ PrefillParams p,
                      const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v)
{
    prefill_tile<D, CAPPED, KV_CONTIGUOUS, 1>(p, PagedView{}, map_q, map_k, map_v);
}

template <int D, bool CAPPED, KvSource SRC, int REP>
__global__ void __launch_bounds__(cta_threads(SRC == KV_PAGED_E4M3, REP), 1)
    prefill_tc_paged_kernel(const __grid_constant__ PrefillParams p,
                            const __grid_constant__ PagedView pg,
                            const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v)
{
    prefill_tile<D, CAPPED, SRC, REP>(p, pg, map_q, map_k, map_v);
}

// The sequence that grid slot `slot` serves, and its bounds: with 2 to 32
// sequences the slots go to sequences in order of decreasing end position
// (prior + new tokens), as in the attention pass; otherwise slot b is
// sequence b.  Called by a full warp; every lane gets the same values.
__device__ __forceinline__ void slot_sequence(const PrefillParams &p, int slot, int lane, int &b,
                                              int &tok0, int &n_new, int &prior)
{
    if (p.batch > 1 && p.batch <= 32) {
        int c0 = 0, c1 = 0, pl = 0, key = -1;
        if (lane < p.batch) {
            c0 = __ldg(p.cu_seqlens + lane);
            c1 = __ldg(p.cu_seqlens + lane + 1);
            pl = __ldg(p.cache_lens + lane);
            key = pl + (c1 - c0);
        }
        int rank = 0;
        for (int j = 0; j < p.batch; j++) {
            const int kj = __shfl_sync(0xffffffffu, key, j);
            rank += (kj > key) || (kj == key && j < lane);
        }
        const unsigned m = __ballot_sync(0xffffffffu, lane < p.batch && rank == slot);
        const int src = __ffs(m) - 1;
        b = src;
        tok0 = __shfl_sync(0xffffffffu, c0, src);
        n_new = __shfl_sync(0xffffffffu, c1, src) - tok0;
        prior = __shfl_sync(0xffffffffu, pl, src);
        return;
    }
    b = slot;
    tok0 = __ldg(p.cu_seqlens + b);
    n_new = __ldg(p.cu_seqlens + b + 1) - tok0;
    prior = __ldg(p.cache_lens + b);
}

// Merge pass of the cut (tail) units: CTA (u, g) merges rows 8 g .. 8 g + 7
// of tail unit u, one warp per row.  Lane s loads piece s's (max, sum) (one
// round), the row's M and L come from warp reductions, then each lane loads
// its D/32 output elements of every piece's row, four pieces in flight at a
// time, weights them by 2^(m_s - M) in piece order, normalises and gates.
constexpr int kMergeRows = 8;

template <int D, bool PAGED>
__global__ void __launch_bounds__(256) prefill_combine_kernel(const PrefillParams p)
{
    constexpr int EPL = D / 32;  // output elements per lane
    grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned FULL = 0xffffffffu;
    const int tu = blockIdx.x;
    const int r = blockIdx.y * kMergeRows + warp;            // the warp's row of the unit
    const size_t row0 = (size_t)tu * p.num_splits * BM + r;  // piece s at row0 + s BM
    // The pieces' (max, sum) (lane s: piece s) and rows of the first four
    // pieces are requested at once, in parallel with the sequence bounds: one
    // round trip instead of three dependent ones.  Pieces past the row's last
    // one are read but never used (their slots hold other calls' rows).
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml);
    float2 ml_pre = make_float2(-INFINITY, 0.f);
    if (lane < p.num_splits)
        ml_pre = ml[row0 + (size_t)lane * BM];
    auto load_row = [&](int s, float (&v)[EPL]) {
        const float *src = p.part_o + (row0 + (size_t)s * BM) * D + lane * EPL;
        if constexpr (EPL == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(src);
            v[0] = x.x;
            v[1] = x.y;
            v[2] = x.z;
            v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(src);
            v[0] = x.x;
            v[1] = x.y;
        }
    };
    float pre[4][EPL];
#pragma unroll
    for (int u = 0; u < 4; u++)
        if (u < p.num_splits)
            load_row(u, pre[u]);
    const int unit = p.full_units + tu;
    const int hg = (unit / p.q_tiles) % p.HG;
    const int slot = unit / (p.q_tiles * p.HG);
    const int qt = p.q_tiles - 1 - (unit % p.q_tiles);
    int b, tok0, n_new, prior;
    __shared__ RankScratch rank_scratch;
    if (PAGED && p.batch > 32 && p.batch <= kRankBatch)
        rank_sequences(p, rank_scratch, slot, b, tok0, n_new, prior);
    else
        slot_sequence(p, slot, lane, b, tok0, n_new, prior);
    const int r0 = qt * p.tile_tokens;
    const bool ring = (p.flags & NA_RING_CACHE) != 0;
    if (n_new > p.max_new_len || (b == 0 && tok0 != 0) || tok0 < 0 ||
        (long long)tok0 + n_new > p.total_tokens || r0 >= n_new)
        return;  // invalid bounds were reported by the attention pass
    const int rows_tok = min(p.tile_tokens, n_new - r0);
    const int pos_lo = prior + r0, pos_hi = pos_lo + rows_tok - 1;
    if (prior < 0 || (!ring && pos_hi >= p.capacity) || pos_hi >= p.max_total_len)
        return;
    const int pack_shift = __ffs(p.pack) - 1;
    if (r >= (PAGED ? rows_tok * p.pack : rows_tok << pack_shift))
        return;
    const int tok = PAGED ? (r * p.pack_inv) >> 16 : r >> pack_shift;
    const size_t out_row = (size_t)(tok0 + r0 + tok) * p.H + hg * p.pack +
                           (PAGED ? r - tok * p.pack : r & (p.pack - 1));
    uint32_t gw[EPL / 2];  // gate words, requested before the merge arithmetic
    const bool gated = (p.flags & NA_OUT_GATE) && p.gate;
    if (gated) {
        const bf16 *gt = p.gate + out_row * D + lane * EPL;
        if constexpr (EPL == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(gt));
            gw[0] = u.x;
            gw[1] = u.y;
        } else {
            gw[0] = __ldg(reinterpret_cast<const unsigned int *>(gt));
        }
    }
    // pieces with keys: the splits start at the key tile holding the first
    // row's window start (0 without a window), split_len keys apart
    const int win_tile = p.window > 0 ? max(0, pos_lo - p.window + 1) / BN * BN : 0;
    const int ns = min(p.num_splits, (pos_hi - win_tile) / p.split_len + 1);
    float M = -INFINITY;
    for (int s0 = 0; s0 < ns; s0 += 32)
        if (s0 + lane < ns)
            M = fmaxf(M, s0 == 0 ? ml_pre.x : ml[row0 + (size_t)(s0 + lane) * BM].x);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    float acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; e++)
        acc[e] = 0.f;
    float L = 0.f;
    for (int s0 = 0; s0 < ns; s0 += 32) {
        float w = 0.f;  // this lane's piece weight 2^(m - M)
        if (s0 + lane < ns) {
            const float2 v = s0 == 0 ? ml_pre : ml[row0 + (size_t)(s0 + lane) * BM];
            if (v.x != -INFINITY) {
                w = exp2f(v.x - M);
                L = fmaf(v.y, w, L);
            }
        }
        const int n = min(32, ns - s0);
        for (int s = 0; s < n; s += 4) {
            float v[4][EPL];
#pragma unroll
            for (int u = 0; u < 4; u++) {
                if (s0 + s == 0) {
#pragma unroll
                    for (int e = 0; e < EPL; e++)
                        v[u][e] = pre[u][e];
                } else if (s + u < n) {
                    load_row(s0 + s + u, v[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const float ws = __shfl_sync(FULL, w, min(s + u, n - 1));
                if (s + u < n) {
#pragma unroll
                    for (int e = 0; e < EPL; e++)
                        acc[e] = fmaf(v[u][e], ws, acc[e]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        L += __shfl_xor_sync(FULL, L, o);
    const float inv = L > 0.f ? 1.0f / L : 0.f;
    bf16 *dst = p.out + out_row * D + lane * EPL;
    float g[EPL];
#pragma unroll
    for (int e = 0; e < EPL; e++)
        g[e] = 1.0f;
    if (gated) {
#pragma unroll
        for (int e = 0; e < EPL; e += 2) {
            g[e] = __fdividef(1.0f, 1.0f + __expf(-__uint_as_float(gw[e / 2] << 16)));
            g[e + 1] = __fdividef(1.0f, 1.0f + __expf(-__uint_as_float(gw[e / 2] & 0xffff0000u)));
        }
    }
    uint32_t packed[EPL / 2];
#pragma unroll
    for (int e = 0; e < EPL; e += 2)
        packed[e / 2] = pack_bf16x2(acc[e] * inv * g[e], acc[e + 1] * inv * g[e + 1]);
    if constexpr (EPL == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(packed[0], packed[1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = packed[0];
}

template <int D, KvSource SRC, int REP = 1>
cudaError_t launch_prefill_t(const PrefillParams &p, const PagedView &pg, int total_tokens,
                             int cache_batch, cudaStream_t stream)
{
    CUtensorMap mq, mk, mv;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.H, (cuuint64_t)total_tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.H * D * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)p.pack, (cuuint32_t)p.tile_tokens};
        if (!make_bf16_tile_map(&mq, p.q, 3, dims, strides, box))
            return cudaErrorInvalidValue;
    }
    if constexpr (SRC == KV_CONTIGUOUS) {
        const cuuint64_t rows = (cuuint64_t)cache_batch * p.KV * p.capacity;
        const cuuint64_t dims[2] = {(cuuint64_t)D, rows};
        const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
        const cuuint32_t box[2] = {64, BN};
        if (!make_bf16_tile_map(&mk, p.cache_k, 2, dims, strides, box) ||
            !make_bf16_tile_map(&mv, p.cache_v, 2, dims, strides, box))
            return cudaErrorInvalidValue;
    } else {  // rows (page, kv head, slot), boxes of a page's rows
        constexpr bool e4m3 = SRC == KV_PAGED_E4M3;
        const cuuint64_t rows = ((cuuint64_t)pg.num_pages * p.KV) << pg.page_log;
        const cuuint64_t dims[2] = {(cuuint64_t)D, rows};
        const cuuint64_t strides[1] = {(cuuint64_t)D * (e4m3 ? 1 : 2)};
        const cuuint32_t box[2] = {(cuuint32_t)(e4m3 ? D : 64), 1u << pg.page_log};
        const bool ok = e4m3 ? make_u8_tile_map(&mk, p.cache_k, 2, dims, strides, box, true) &&
                                   make_u8_tile_map(&mv, p.cache_v, 2, dims, strides, box, D == 128)
                             : make_bf16_tile_map(&mk, p.cache_k, 2, dims, strides, box) &&
                                   make_bf16_tile_map(&mv, p.cache_v, 2, dims, strides, box);
        if (!ok)
            return cudaErrorInvalidValue;
    }
    const size_t smem = tc_smem_bytes<D, SRC>();
    static std::atomic<unsigned long long> configured{0};
    auto kernel_of = [](auto capped) {
        constexpr bool CAPPED = decltype(capped)::value;
        if constexpr (SRC == KV_CONTIGUOUS)
            return prefill_tc_kernel<D, CAPPED>;
        else
            return prefill_tc_paged_kernel<D, CAPPED, SRC, REP>;
    };
    const auto plain = kernel_of(std::false_type()), capped = kernel_of(std::true_type());
    cudaError_t e = once_per_device(configured, [=] {
        cudaError_t r = cudaFuncSetAttribute(plain, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(capped, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return r;
    });
    if (e != cudaSuccess)
        return e;
    const dim3 grid(p.full_units + p.tail_units * p.num_splits);
    const dim3 block(cta_threads(SRC == KV_PAGED_E4M3, REP));
    const auto kernel = p.softcap > 0.f ? capped : plain;
    if constexpr (SRC == KV_CONTIGUOUS)
        e = launch_kernel(kernel, grid, block, smem, stream, p, mq, mk, mv);
    else
        e = launch_kernel(kernel, grid, block, smem, stream, p, pg, mq, mk, mv);
    if (e != cudaSuccess || p.num_splits == 1)
        return e;
    return launch_kernel(prefill_combine_kernel<D, SRC != KV_CONTIGUOUS>, dim3(p.tail_units, BM / kMergeRows), dim3(256),
                         0, stream, p);
}

// A paged call, by whether its tiles have few rows.
template <int D, KvSource SRC>
cudaError_t launch_paged_t(const PrefillParams &p, const PagedView &pg, int total_tokens,
                           cudaStream_t stream)
{
    return p.rep == 1 ? launch_prefill_t<D, SRC, 1>(p, pg, total_tokens, 0, stream)
                      : launch_prefill_t<D, SRC, kPrefillRep>(p, pg, total_tokens, 0, stream);
}

}  // namespace

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// bf16 tensor map with 64-element (128-byte) inner boxes and 128-byte swizzle.
bool make_bf16_tile_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
              const cuuint64_t *strides_bytes, const cuuint32_t *box)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base),
              dims, strides_bytes, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_u8_tile_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
                      const cuuint64_t *strides_bytes, const cuuint32_t *box, bool swizzle)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(base), dims,
              strides_bytes, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                       : (box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B),
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int prefill_key_tile() { return BN; }
int prefill_q_tile() { return BM; }

cudaError_t launch_prefill(const PrefillParams &p, int d, int total_tokens, int cache_batch,
                           cudaStream_t stream)
{
    const PagedView none{};
    if (d == 128)
        return launch_prefill_t<128, KV_CONTIGUOUS>(p, none, total_tokens, cache_batch, stream);
    return launch_prefill_t<64, KV_CONTIGUOUS>(p, none, total_tokens, cache_batch, stream);
}

cudaError_t launch_prefill_paged(const PrefillParams &p, const PagedView &pg, bool e4m3, int d,
                                 int total_tokens, cudaStream_t stream)
{
    if (d == 128)
        return e4m3 ? launch_paged_t<128, KV_PAGED_E4M3>(p, pg, total_tokens, stream)
                    : launch_paged_t<128, KV_PAGED>(p, pg, total_tokens, stream);
    return e4m3 ? launch_paged_t<64, KV_PAGED_E4M3>(p, pg, total_tokens, stream)
                : launch_paged_t<64, KV_PAGED>(p, pg, total_tokens, stream);
}
