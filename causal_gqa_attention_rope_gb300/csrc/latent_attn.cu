// latent_attn.cu -- absorbed latent attention over pages (na_attn_latent_paged), on
// the sm_100-family tensor cores (tcgen05 + TMEM + TMA).
//
// A unit is 64 query rows (32 where a sequence has no more) -- (token, head) pairs of one
// sequence, token-major -- and the key tiles of 64 cached rows that they see.  For each
// tile
//     S   [64 rows x 64 keys]  = Q K^T      M = 64, K = R + 64 (rope part padded by TMA's
//                                           zeros to a whole column block)
//     O^T [R dims x 64 rows]  += V^T P^T    M = 128 per block of dims, K = 64 keys
// where V is the first R columns of the K tile in shared memory: K-major as K, M-major
// as V^T.  With the rows along N the accumulators of R = 512 take 256 columns of
// tensor memory, where rows along M would take all 512 and leave none to S, and M =
// 128 runs at the full rate.  A row's bytes come from memory once for all heads.
//
// A tile lies in shared memory as its rope block and R / 128 pairs of column blocks, each
// kind in a ring of its own.  S starts on a pair when it has landed and PV gives a
// pair back when its 128 dims are done, so that loading runs on through both: with
// whole tiles handed over, two of them deep, a tile took 3750 cycles of which its
// load was 3000, and 64 sequences of 512 .. 8192 keys 76.6 us.  32 query rows leave
// room for half a tile more.
//
// Warps: 0 producer (TMA: Q of a unit, then its tiles, a box per page and 64 columns),
// 1 issues S into one of two buffers, 2 issues O^T, 4 .. 7 softmax, 16 rows each
// (M = 64 puts row r into lane 32 (r / 16) + r % 16), four lanes to a row, each 16
// of a tile's keys.  Max and sum are kept per row in fp32; the reference maximum is
// raised only when a score exceeds it by more than 2^8, and then all four warps
// rescale the columns of O^T by the factors in shared memory.
//
// Work: by runs (latent_runs.cuh), one per CTA, one CTA per SM.  A unit that a cut goes through is
// left in pieces (unnormalised rows with maximum and sum) which a second pass joins.  Run c
// has at most two: the end of a unit that an earlier one began (slot 2 c) and the beginning of one
// that others finish (slot 2 c + 1).  Short contexts instead take a cluster of up to 8 CTAs per unit
// (JOINED), which join its pieces out of one another's shared memory: no search for the run's
// beginning, no second pass, and the sequence's first pages asked for beside its lengths.
//
// Sequences of more than 64 rows (chunks, drafted tokens, many heads) take units of 128 rows in
// pairs of CTAs: latent_pair.cu.  With 128 latent numbers, which that kernel does not split, they
// take units of 64 rows here, each of which loads its tiles, from L2 where another has had them (64
// sequences of 512 .. 8192 keys, 2 .. 8 tokens of 32 heads: 98 us).
#include <algorithm>
#include <climits>

#include "latent_runs.cuh"
#include "na_host.cuh"
#include "tc_primitives.cuh"
#include "tile_waits.cuh"

namespace {

constexpr int MAX_ROWS = 64;               // M of S, whatever a unit's rows are
constexpr int THREADS = 256;
constexpr uint32_t BLOCK_BYTES = KT * 128;  // 64 keys of 64 bf16: a column block of a tile

// QR: rows of a unit.  With 32 the products' rows 32 .. 63 are whatever lies behind a block of
// Q, and nobody looks at them.
template <int R, int QR>
struct __align__(1024) LatentSmem {
    static constexpr int CB = R / 64 + 1;   // column blocks of a row
    static constexpr int DB = R / 128;      // pairs of them in V: blocks of 128 dims
    static constexpr int PAIRS = R == 512 ? (QR == 32 ? 10 : 8) : (R == 256 ? 8 : 6);
    static constexpr int ROPES = R == 512 ? (QR == 32 ? 3 : 2) : (R == 256 ? 4 : 6);
    bf16 q[CB][QR * 64];
    bf16 pair[PAIRS][2][KT * 64];
    bf16 rope[ROPES][KT * 64];
    bf16 p[QR * 64];
    float factor[2][MAX_ROWS]; // a tile's corrections by row, by tile parity
    float inv[MAX_ROWS];       // at a piece's end: 1 / sum, or 1
    uint64_t q_full, q_empty, pair_full[PAIRS], pair_empty[PAIRS], rope_full[ROPES],
        rope_empty[ROPES], s_full[2], s_empty[2], p_full, pv_done, o_empty, drain[2];
    float2 ml[MAX_ROWS];       // at a joined piece's end: the rows' (max, sum)
    long long warp_steps[THREADS / 32];
    long long total, begin;
    int b0, t0, step0;         // where the CTA's run begins
    uint32_t tmem_base;
    int abort_flag;
};

// 16 lanes x 64 columns of tensor memory: thread l gets columns 8 i + 2 (l % 4) + {0, 1}
// of lane l / 4 in r[4 i], r[4 i + 1] and of lane l / 4 + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

// What is at `at`'s place in CTA `rank` of the cluster.
__device__ __forceinline__ float4 load_cluster_4(const void *at, int rank)
{
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(place_in_cta(at, rank))
                 : "memory");
    return x;
}

__device__ __forceinline__ float2 load_cluster_2(const void *at, int rank)
{
    float2 x;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(x.x), "=f"(x.y)
                 : "r"(place_in_cta(at, rank))
                 : "memory");
    return x;
}

// The rows of a unit whose pieces P CTAs of a cluster hold, each unnormalised in `stage` (rows of
// R + 4) with their maxima and sums in `ml`: CTA `piece` joins every P-th row.  Other CTAs'
// shared memory gives some 14 bytes a cycle (64 rows of 512 in pieces: 4 us), so that
// nothing is asked for twice, and the own piece not through the cluster; P is known to the compiler,
// because loads behind a branch were waited for one by one.
template <int R, int P>
__device__ __forceinline__ void join_rows_of(const LatentParams &p, const float *stage, const float2 *ml,
                                             float (*weight)[MAX_ROWS], int piece, int rows, long long row0)
{
    constexpr int AT_ONCE = THREADS / (R / 4);
    if (threadIdx.x < rows) {
        float2 of[P];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int c = 0; c < P; c++)
            of[c] = load_cluster_2(ml + threadIdx.x, c);
#pragma unroll
        for (int c = 0; c < P; c++)
            m = fmaxf(m, of[c].x);
#pragma unroll
        for (int c = 0; c < P; c++) {
            of[c].x = of[c].x == -INFINITY ? 0.f : exp2f(of[c].x - m);
            l = fmaf(of[c].x, of[c].y, l);
        }
        const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
        for (int c = 0; c < P; c++)
            weight[c][threadIdx.x] = of[c].x * inv;
    }
    __syncthreads();
    // (a few rows at a time where a row has few pieces; the last stands for those behind it)
    constexpr int ROWS = P == 1 ? 4 : (P <= 3 ? 2 : 1), STEP = P * AT_ONCE;
    const int x = threadIdx.x % (R / 4) * 4;
    for (int r0 = piece + P * (threadIdx.x / (R / 4)); r0 < rows; r0 += ROWS * STEP) {
        float4 v[ROWS][P];
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
            const float *row = stage + min(r0 + i * STEP, rows - 1) * (R + 4) + x;
            v[i][0] = *reinterpret_cast<const float4 *>(row);
#pragma unroll
            for (int k = 1; k < P; k++)
                v[i][k] = load_cluster_4(row, piece + k < P ? piece + k : piece + k - P);
        }
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
            const int r = r0 + i * STEP;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < P; k++) {
                const float w = weight[piece + k < P ? piece + k : piece + k - P][min(r, rows - 1)];
                if (w != 0.f)  // (a piece without keys holds whatever was there)
                    o = make_float4(fmaf(w, v[i][k].x, o.x), fmaf(w, v[i][k].y, o.y),
                                    fmaf(w, v[i][k].z, o.z), fmaf(w, v[i][k].w, o.w));
            }
            if (r < rows)
                *reinterpret_cast<uint2 *>(p.out + (row0 + r) * R + x) =
                    make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        }
    }
}

template <int R>
__device__ __forceinline__ void join_rows(const LatentParams &p, const float *stage, const float2 *ml,
                                          float (*weight)[MAX_ROWS], int piece, int rows, long long row0)
{
    static_assert(kLatentMaxPieces == 8, "cases");
    switch (p.pieces) {
    case 1: return join_rows_of<R, 1>(p, stage, ml, weight, piece, rows, row0);
    case 2: return join_rows_of<R, 2>(p, stage, ml, weight, piece, rows, row0);
    case 3: return join_rows_of<R, 3>(p, stage, ml, weight, piece, rows, row0);
    case 4: return join_rows_of<R, 4>(p, stage, ml, weight, piece, rows, row0);
    case 5: return join_rows_of<R, 5>(p, stage, ml, weight, piece, rows, row0);
    case 6: return join_rows_of<R, 6>(p, stage, ml, weight, piece, rows, row0);
    case 7: return join_rows_of<R, 7>(p, stage, ml, weight, piece, rows, row0);
    default: return join_rows_of<R, 8>(p, stage, ml, weight, piece, rows, row0);
    }
}

// JOINED: a cluster of p.pieces CTAs per unit, a piece of its keys each, instead of runs.
template <int R, int QR, bool JOINED>
__global__ void __launch_bounds__(THREADS, 1)
    latent_attn_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ PagedView pg,
                       const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_kv)
{
    typedef LatentSmem<R, QR> Smem;
    constexpr int CB = Smem::CB, DB = Smem::DB, PAIRS = Smem::PAIRS, ROPES = Smem::ROPES;
    constexpr uint32_t S_COL = DB * QR;                // O^T block d at column QR d, then S
    constexpr uint32_t TMEM_COLS = S_COL + 128 <= 256 ? 256 : 512;
    constexpr uint32_t BLOCK16 = BLOCK_BYTES >> 4;
    const int group = JOINED ? p.pieces : 1;
    const int run = blockIdx.x / group;
    const int piece = JOINED ? blockIdx.x % group : 0;
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_kv);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < PAIRS; i++) {
            mbar_init(&sm.pair_full[i], 1);
            mbar_init(&sm.pair_empty[i], 1);
        }
        for (int i = 0; i < ROPES; i++) {
            mbar_init(&sm.rope_full[i], 1);
            mbar_init(&sm.rope_empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 4);
            mbar_init(&sm.drain[i], 1);
        }
        mbar_init(&sm.p_full, 4);
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.o_empty, 4);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1)
        tc::tmem_alloc(&sm.tmem_base, TMEM_COLS);
    grid_dependency_wait();
    grid_dependents_launch();
    tc::fence_before_sync();
    if constexpr (JOINED)
        __syncthreads();
    else
        find_run<QR, THREADS / 32>(p, sm, run, warp, lane);
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    auto begin_walk = [&] {
        if constexpr (JOINED)
            return Walk<QR>(p, run, piece);
        else
            return Walk<QR>(p, sm, run);
    };
    // The sequence's first pages, asked for beside its lengths.
    int early = -1;
    if constexpr (JOINED) {
        const int b = run / ((p.max_new_len * p.H + QR - 1) / QR);
        if (warp == 0 && lane < pg.pages_per_seq)
            early = __ldg(pg.table + (size_t)b * pg.pages_per_seq + lane);
    }
    Walk<QR> w = begin_walk();
    int join_count = 0;          // rows of the unit, for all threads
    long long join_row0 = 0;
    if constexpr (JOINED) {
        if (w.have) {
            join_row0 = (long long)w.s.tok0 * p.H + (long long)w.t * QR;
            join_count = min(QR, w.s.n * p.H - w.t * QR);
        }
    }
    float *stage = reinterpret_cast<float *>(&sm.pair[0]);  // idle when a piece's rows are done
    static_assert(!JOINED || sizeof(float) * QR * (R + 4) <= sizeof(sm.pair) + sizeof(sm.rope), "staged rows");

    if (warp == 0) {
        // ------------------------------------------------------------ producer --
        const int box_log = min(pg.page_log, 6), boxes = KT >> box_log;
        const int in_page = (1 << pg.page_log) - 1;
        const uint64_t policy = l2_policy_evict_first();
        const bool read_once = (long long)p.max_new_len * p.H <= QR;  // one unit a sequence
        int g = 0, pairs = 0, pieces = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t *bar, uint32_t parity) {
            if (!warp_wait(bar, parity, &sm.abort_flag)) {
                if (lane == 0)
                    set_abort(&sm.abort_flag, p.status);
                ok = false;
            }
            return ok;
        };
        for (; ok && w.next(p); pieces++) {
            const int32_t *row = pg.table + (size_t)w.seq * pg.pages_per_seq;
            // This lane's page of a tile (boxes of them): its table entry, asked for two tiles ahead and
            // not looked at before the tile's turn (800 cycles a tile otherwise), then checked; -1
            // where there is none.
            auto has_page = [&](int j) {
                return lane < boxes && j < w.hi && j * KT + (lane << box_log) < w.keys;
            };
            auto ask = [&](int j) {
                const int entry = (j * KT + (lane << box_log)) >> pg.page_log;
                int id = JOINED ? __shfl_sync(0xffffffffu, early, entry & 31) : 0;
                if (has_page(j) && (!JOINED || entry >= 32))
                    id = __ldg(row + entry);
                return id;
            };
            auto checked = [&](int j, int id) {
                if (!has_page(j))
                    return -1;
                if ((unsigned)id >= (unsigned)pg.num_pages) {  // reported; page 0 is read instead
                    na_report(p.status, NA_ERR_PAGE);
                    id = 0;
                }
                return id;
            };
            int asked = ask(w.lo), asked_next = ask(w.lo + 1);
            if (pieces > 0 && !wait_all(&sm.q_empty, (pieces - 1) & 1))
                break;
            if (lane == 0)
                mbar_arrive_expect_tx(&sm.q_full, CB * QR * 128);
            __syncwarp();
            if (lane < CB)
                tc::tma_load_2d(sm.q[lane], &map_q, lane * 64, (int)w.row0(p), &sm.q_full);
            for (int j = w.lo; ok && j < w.hi; j++) {
                const int id = checked(j, asked);
                asked = asked_next;
                asked_next = ask(j + 2);
                const int n = __popc(__ballot_sync(0xffffffffu, id >= 0));
                const int first = (id << pg.page_log) + (pg.page_log > 6 ? (j * KT) & in_page : 0);
                const int box = lane & (boxes - 1), block = lane / boxes;
                const int from = __shfl_sync(0xffffffffu, first, box);
                // `blocks` column blocks from column x on, a box of a page's rows per lane
                auto load = [&](bf16 *dst, int x, int blocks, uint64_t *bar) {
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar, n * blocks * (128u << box_log));
                    __syncwarp();
                    if (box < n && block < blocks) {
                        bf16 *to = dst + block * (KT * 64) + (box << box_log) * 64;
                        if (read_once)
                            tc::tma_load_2d_hint(to, &map_kv, x + block * 64, from, bar, policy);
                        else
                            tc::tma_load_2d(to, &map_kv, x + block * 64, from, bar);
                    }
                };
                const int rs = g % ROPES;
                if (!wait_all(&sm.rope_empty[rs], ((g / ROPES) & 1) ^ 1))
                    break;
                load(sm.rope[rs], R, 1, &sm.rope_full[rs]);
                g++;
                for (int c = 0; c < DB; c++, pairs++) {
                    const int ps = pairs % PAIRS;
                    if (!wait_all(&sm.pair_empty[ps], ((pairs / PAIRS) & 1) ^ 1))
                        break;
                    load(sm.pair[ps][0], c * 128, 2, &sm.pair_full[ps]);
                }
            }
        }
        // every copy issued lands before the CTA can exit
        if (lane == 0) {
            if (pieces > 0)
                drain_wait(&sm.q_full, (pieces - 1) & 1, p.status);
            for (int i = g - 1; i >= 0 && i >= g - ROPES; i--)
                drain_wait(&sm.rope_full[i % ROPES], (i / ROPES) & 1, p.status);
            for (int i = pairs - 1; i >= 0 && i >= pairs - PAIRS; i--)
                drain_wait(&sm.pair_full[i % PAIRS], (i / PAIRS) & 1, p.status);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- S = Q K^T issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(MAX_ROWS, KT, false, false);
            constexpr uint32_t Q16 = (QR * 128) >> 4;  // a column block of Q
            const uint64_t qd = tc::desc_kmajor_sw128(smem_addr(sm.q[0]));
            const uint64_t rd0 = tc::desc_kmajor_sw128(smem_addr(sm.rope[0]));
            const uint64_t kd0 = tc::desc_kmajor_sw128(smem_addr(sm.pair[0][0]));
            bool ok = true;
            bool issued = false;
            int g = 0, pairs = 0;
            for (int piece = 0; ok && w.next(p); piece++) {
                ok = mbar_wait_bounded(&sm.q_full, piece & 1);
                for (int j = w.lo; ok && j < w.hi; j++, g++) {
                    const int sb = g & 1, rs = g % ROPES;
                    ok = mbar_wait_bounded(&sm.rope_full[rs], (g / ROPES) & 1);
                    if (ok && g >= 2)
                        ok = mbar_wait_bounded(&sm.s_empty[sb], ((g >> 1) - 1) & 1);
                    if (!ok || aborted(&sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t s_t = tmem + S_COL + sb * KT;
                    // 16 columns, 32 bytes of a block's rows, per instruction
                    const uint64_t rd = rd0 + (uint64_t)(rs * BLOCK16);
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        tc::mma_ss(s_t, qd + (CB - 1) * Q16 + k * 2, rd + k * 2, idesc, k > 0);
                    issued = true;
                    tc::mma_commit(&sm.rope_empty[rs]);
#pragma unroll
                    for (int c = 0; c < DB; c++, pairs++) {
                        const int ps = pairs % PAIRS;
                        ok = ok && mbar_wait_bounded(&sm.pair_full[ps], (pairs / PAIRS) & 1);
                        if (!ok)
                            continue;
                        tc::fence_after_sync();
                        const uint64_t kd = kd0 + (uint64_t)(ps * 2 * BLOCK16);
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            tc::mma_ss(s_t, qd + (2 * c + (k >> 2)) * Q16 + (k & 3) * 2,
                                       kd + (k >> 2) * BLOCK16 + (k & 3) * 2, idesc, true);
                    }
                    if (!ok)
                        break;
                    tc::mma_commit(&sm.s_full[sb]);
                    if (j == w.hi - 1)
                        tc::mma_commit(&sm.q_empty);
                }
            }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            if (issued) {  // all issued MMAs complete before tensor memory is released
                tc::mma_commit(&sm.drain[0]);
                drain_wait(&sm.drain[0], 0, p.status);
            }
        }
    } else if (warp == 2) {
        // ----------------------------------------------------- O^T += V^T P^T issue --
        if (elect_one()) {
            const uint64_t vd0 = tc::desc_mnmajor_sw128(smem_addr(sm.pair[0][0]), BLOCK_BYTES);
            const uint64_t pd = tc::desc_kmajor_sw128(smem_addr(sm.p));
            bool ok = true;
            int g = 0, pairs = 0;
            for (int piece = 0; ok && w.next(p); piece++) {
                // the rows' columns in whole sixteens
                const uint32_t idesc = tc::idesc_bf16_f32(128, (w.rows(p, 0, QR) + 15) / 16 * 16, true, false);
                if (piece > 0)
                    ok = mbar_wait_bounded(&sm.o_empty, (piece - 1) & 1);
                for (int j = w.lo; ok && j < w.hi; j++, g++) {
                    ok = mbar_wait_bounded(&sm.p_full, g & 1);
#pragma unroll
                    for (int d = 0; d < DB; d++)  // (long complete: S has read the tile)
                        ok = ok && mbar_wait_bounded(&sm.pair_full[(pairs + d) % PAIRS],
                                                     ((pairs + d) / PAIRS) & 1);
                    if (!ok || aborted(&sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
#pragma unroll
                    for (int d = 0; d < DB; d++, pairs++) {
                        const int ps = pairs % PAIRS;
                        const uint64_t vd = vd0 + (uint64_t)(ps * 2 * BLOCK16);
#pragma unroll
                        for (int k = 0; k < KT / 16; k++)  // 16 keys: rows of 128 B of V, 32 B of a row of P
                            tc::mma_ss(tmem + d * QR, vd + (uint64_t)(k * 128), pd + (uint64_t)(k * 2), idesc,
                                       j > w.lo || k > 0);
                        tc::mma_commit(&sm.pair_empty[ps]);
                    }
                    tc::mma_commit(&sm.pv_done);
                }
            }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            if (g > 0) {
                tc::mma_commit(&sm.drain[1]);
                drain_wait(&sm.drain[1], 0, p.status);
            }
        }
    } else if (warp >= 4) {
        // -------------------------------------------------------------- softmax --
        const int quarter = warp & 3, tid = threadIdx.x - 128;
        const int ra = quarter * 16 + (lane >> 2);  // this thread's rows: ra and ra + 8
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float sl2 = p.scale_log2;
        bool ok = true;
        int g = 0;
        // Where a unit that begins here is told to the second pass: by sequence where each has one
        // unit, else by run.
        const bool leader = tid == 0;
        if (!JOINED && leader && !p.cut_by_sequence)
            p.cut[run] = make_int4(0, 0, 0, -1);
        if (JOINED && tid < MAX_ROWS)
            sm.ml[tid] = make_float2(-INFINITY, 0.f);  // until there are keys
        while (ok && w.next(p)) {
            const int rows = w.rows(p, 0, QR);
            int lim[2];  // keys that the rows see
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = ra + 8 * h;
                lim[h] = r < rows ? w.s.prior + (w.unit * QR + r) / p.H + 1 : 0;
            }
            float m_ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
            for (int j = w.lo; j < w.hi; j++, g++) {
                const int j0 = j * KT, sb = g & 1;
                ok = ok && warp_wait(&sm.s_full[sb], (g >> 1) & 1, &sm.abort_flag);
                uint32_t s[32];
                if (ok) {
                    tc::fence_after_sync();
                    tmem_ld_16x64(tmem + S_COL + sb * KT + lane_off, s);
                    tc::tmem_wait_ld();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm.s_empty[sb]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        s[i] = 0;
                }
                if (j0 + KT > min(lim[0], lim[1])) {
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const int key = j0 + (i >> 2) * 8 + (lane & 3) * 2 + (i & 1);
                        if (key >= lim[(i >> 1) & 1])
                            s[i] = __float_as_uint(-INFINITY);
                    }
                }
                float alpha[2];
                bool raise = false;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        mx = max3f(mx, __uint_as_float(s[4 * i + 2 * h]),
                                   __uint_as_float(s[4 * i + 2 * h + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2;
                    alpha[h] = 1.f;
                    if (mx > m_ref[h] + 8.0f) {
                        alpha[h] = m_ref[h] == -INFINITY ? 0.f : ex2_mufu(m_ref[h] - mx);
                        raise = raise || m_ref[h] != -INFINITY;
                        m_ref[h] = mx;
                    }
                    if ((lane & 3) == 0)
                        sm.factor[g & 1][ra + 8 * h] = alpha[h];
                }
                // (a warp whose wait gave up still comes here, so that the others go on to see it)
                const bool rescale = any_of(raise || !ok, 1, 128);
                if (aborted(&sm.abort_flag))
                    ok = false;
                uint32_t pk[16];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float neg_m = m_ref[h] == -INFINITY ? 0.f : -m_ref[h];
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float2 x = __ffma2_rn(
                            make_float2(__uint_as_float(s[4 * i + 2 * h]),
                                        __uint_as_float(s[4 * i + 2 * h + 1])),
                            make_float2(sl2, sl2), make_float2(neg_m, neg_m));
                        const float2 e = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
                        acc = __fadd2_rn(acc, e);
                        pk[2 * i + h] = pack_bf16x2(e.x, e.y);
                    }
                    sum[h] = fmaf(sum[h], alpha[h], acc.x + acc.y);
                }
                // P and O^T are free once the last tile's product is done
                if (ok && g > 0)
                    ok = warp_wait(&sm.pv_done, (g - 1) & 1, &sm.abort_flag);
                if (ok && rescale && j > w.lo) {
                    tc::fence_after_sync();
                    const float *f = sm.factor[g & 1];
#pragma unroll 1
                    for (int c = 0; c < DB * QR; c += 32) {
                        uint32_t o[32];
                        tc::tmem_ld32(tmem + lane_off + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f[(c & (QR - 1)) + i]);
                        tc::tmem_st32(tmem + lane_off + c, o);
                    }
                    tc::tmem_wait_st();
                }
                if (ok && j0 + KT > w.keys)
                    for (int c = 0; c < DB; c++)
                        ok = ok && warp_wait(&sm.pair_full[(g * DB + c) % PAIRS],
                                             ((g * DB + c) / PAIRS) & 1, &sm.abort_flag);
                if (ok) {
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        const int r = ra + 8 * (i & 1);
                        if (QR < MAX_ROWS && r >= QR)
                            continue;
                        *reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(sm.p) + r * 128 +
                                                      (((i >> 1) ^ (r & 7)) << 4) + (lane & 3) * 4) = pk[i];
                    }
                    if (j0 + KT > w.keys) {
                        // Rows behind the last key hold whatever was there: zeros, so that no
                        // weight of 0 meets a NaN.  (S of this tile has been read off.)
                        const int from = w.keys - j0;
                        const int per = (KT - from) * 8;
                        for (int i = tid; i < per * 2 * DB; i += 128) {
                            const int cb = i / per, k = i - cb * per;
                            uint4 *v = reinterpret_cast<uint4 *>(
                                sm.pair[(g * DB + (cb >> 1)) % PAIRS][cb & 1]);
                            v[from * 8 + k] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    tc::fence_proxy_async_smem();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm.p_full);
                }
            }
            // ------------------------------------------------------- a piece's rows --
            ok = ok && warp_wait(&sm.pv_done, (g - 1) & 1, &sm.abort_flag);
            const bool whole = !JOINED && w.lo == 0 && w.hi == w.tiles;
            const size_t slot_row = (size_t)(2 * run + (w.lo == 0 ? 1 : 0)) * QR;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
                sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
                if ((lane & 3) == 0) {
                    sm.inv[ra + 8 * h] = whole ? (sum[h] > 0.f ? 1.0f / sum[h] : 0.f) : 1.f;
                    if (JOINED && ra + 8 * h < rows)
                        sm.ml[ra + 8 * h] = make_float2(m_ref[h], sum[h]);
                    else if (!whole && ok && ra + 8 * h < rows)
                        reinterpret_cast<float2 *>(p.part_ml)[slot_row + ra + 8 * h] =
                            make_float2(m_ref[h], sum[h]);
                }
            }
            if (any_of(!ok, 1, 128)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const long long row0 = w.row0(p);
#pragma unroll 1
            for (int c = 0; c < DB * QR; c += 32) {
                const int r0 = c & (QR - 1), dim = (c / QR) * 128 + quarter * 32 + lane;
                if (r0 >= rows)
                    continue;
                uint32_t o[32];
                tc::tmem_ld32(tmem + lane_off + c, o);
                tc::tmem_wait_ld();
                if constexpr (JOINED) {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (r0 + i < rows)
                            stage[(r0 + i) * (R + 4) + dim] = __uint_as_float(o[i]);
                } else if (whole) {
                    bf16 *dst = p.out + (row0 + r0) * R + dim;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (r0 + i < rows)
                            dst[(size_t)i * R] = __float2bfloat16_rn(__uint_as_float(o[i]) * sm.inv[r0 + i]);
                } else {
                    float *dst = p.part_o + (slot_row + r0) * R + dim;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (r0 + i < rows)
                            dst[(size_t)i * R] = __uint_as_float(o[i]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.o_empty);
            if (!JOINED && w.lo == 0 && leader) {
                // the unit ends (tiles - hi) behind the end of this run
                const long long end = run_begin(p, sm.total, run + 1) + (w.tiles - w.hi);
                if (!whole || p.cut_by_sequence)
                    p.cut[p.cut_by_sequence ? w.seq : run] = make_int4(
                        (int)w.row0(p), rows, run, whole ? -1 : run_of(p, sm.total, end));
            }
        }
        if (!ok && lane == 0)
            set_abort(&sm.abort_flag, p.status);
    }
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (JOINED) {  // (a CTA whose waits gave up has reported it: what there is gets joined)
        if (p.pieces > 1)
            cluster_sync();
        // (the weights lie over P, which is done with)
        static_assert(sizeof(float) * kLatentMaxPieces * MAX_ROWS <= sizeof(sm.p), "weights");
        join_rows<R>(p, stage, sm.ml, reinterpret_cast<float(*)[MAX_ROWS]>(sm.p), piece, join_count,
                     join_row0);
        if (p.pieces > 1)
            cluster_sync();  // until then the others read this one's rows
    }
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the pieces of a cut unit.  R / 4 threads take a row's pieces, 8 in flight; with GROUPS
// = 4 as many groups take a quarter of them each and are added up at the end.
constexpr int MERGE_THREADS_PER_DIM = 4;  // rows or groups of a CTA

template <int R, int UR, int GROUPS>
__global__ void __launch_bounds__(R / 4 * MERGE_THREADS_PER_DIM)
    latent_merge_kernel(const __grid_constant__ LatentParams p)
{
    constexpr int ROWS = MERGE_THREADS_PER_DIM / GROUPS;
    __shared__ float4 sums[GROUPS > 1 ? GROUPS - 1 : 1][R / 4];
    grid_dependency_wait();
    grid_dependents_launch();
    int4 cut = p.cut[blockIdx.x];
    if (p.cut_by_sequence) {  // a sequence without a unit has no entry, any other's rows are its own
        int code;
        const Sequence s = sequence_of(p, blockIdx.x, code);
        cut.x = s.tok0 * p.H;
        cut.y = s.n * p.H;
    }
    const int part = threadIdx.x / (R / 4), x = threadIdx.x % (R / 4), lane = threadIdx.x & 31;
    const int r = blockIdx.y * ROWS + (GROUPS > 1 ? 0 : part), group = GROUPS > 1 ? part : 0;
    if (!names_runs(cut, p.grid) || r >= cut.y)
        return;
    const int pieces = cut.w - cut.z + 1;
    // piece i in slot 2 c + 1 of the first run, 2 c of those after it
    auto slot = [&](int i) { return (size_t)(2 * (cut.z + i) + (i == 0 ? 1 : 0)) * UR + r; };
    auto load = [&](int i) { return reinterpret_cast<const float4 *>(p.part_o + slot(i) * R)[x]; };
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml);
    // the group's first 8 pieces, and 32 pieces' maxima and sums, asked for together
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; k++)
        if (group + k * GROUPS < pieces)
            v[k] = load(group + k * GROUPS);
    const float2 mine = lane < pieces ? ml[slot(lane)] : make_float2(-INFINITY, 0.f);
    float M = mine.x;
    for (int i = lane + 32; i < pieces; i += 32)
        M = fmaxf(M, ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int i0 = 0; i0 < pieces; i0 += 32) {
        float weight = 0.f;
        if (i0 + lane < pieces) {
            const float2 m = i0 == 0 ? mine : ml[slot(i0 + lane)];
            if (m.x != -INFINITY) {
                weight = exp2f(m.x - M);
                L = fmaf(m.y, weight, L);
            }
        }
        const int n = min(32, pieces - i0);
        for (int i = group; i < n; i += 8 * GROUPS) {
            if (i0 + i != group) {
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (i + k * GROUPS < n)
                        v[k] = load(i0 + i + k * GROUPS);
            }
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float wk = __shfl_sync(0xffffffffu, weight, min(i + k * GROUPS, 31));
                if (i + k * GROUPS < n) {
                    acc.x = fmaf(v[k].x, wk, acc.x);
                    acc.y = fmaf(v[k].y, wk, acc.y);
                    acc.z = fmaf(v[k].z, wk, acc.z);
                    acc.w = fmaf(v[k].w, wk, acc.w);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        L += __shfl_xor_sync(0xffffffffu, L, o);
    if constexpr (GROUPS > 1) {
        if (group > 0)
            sums[group - 1][x] = acc;
        __syncthreads();
        if (group > 0)
            return;
#pragma unroll
        for (int k = 0; k < GROUPS - 1; k++) {
            const float4 a = sums[k][x];
            acc.x += a.x;
            acc.y += a.y;
            acc.z += a.z;
            acc.w += a.w;
        }
    }
    const float inv = L > 0.f ? 1.0f / L : 0.f;
    uint2 u;
    u.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    u.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2 *>(p.out + ((size_t)cut.x + r) * R)[x] = u;
}

// Second pass: the units that runs left in pieces.
template <int R, int UR>
cudaError_t launch_merge(const LatentParams &p, cudaStream_t stream)
{
    if (p.grid == 1)
        return cudaSuccess;
    const int rows = (int)std::min((long long)p.max_new_len * p.H, (long long)UR);
    const dim3 block(R / 4 * MERGE_THREADS_PER_DIM);
    const int entries = p.cut_by_sequence ? p.batch : p.grid;
    // Few units have many pieces each (4 long contexts of 16 heads: the pass took 10 us with a
    // thread per dim and row, every entry of every run looked at).
    if ((long long)entries * rows <= 2 * sm_count())
        return launch_kernel(latent_merge_kernel<R, UR, 4>, dim3(entries, rows), block, 0, stream, p);
    return launch_kernel(latent_merge_kernel<R, UR, 1>,
                         dim3(entries, (rows + MERGE_THREADS_PER_DIM - 1) / MERGE_THREADS_PER_DIM),
                         block, 0, stream, p);
}

template <int R, int QR, bool JOINED>
cudaError_t launch_latent_t(const LatentParams &p, const PagedView &pg, cudaStream_t stream)
{
    CUtensorMap mq, mkv;
    const cuuint64_t wide = R + p.rd;
    const cuuint64_t q_dims[2] = {wide, (cuuint64_t)p.total_tokens * p.H};
    const cuuint64_t kv_dims[2] = {wide, (cuuint64_t)pg.num_pages << pg.page_log};
    const cuuint64_t strides[1] = {wide * 2};
    const cuuint32_t q_box[2] = {64, QR}, kv_box[2] = {64, 1u << (pg.page_log < 6 ? pg.page_log : 6)};
    if (!make_bf16_tile_map(&mq, p.q, 2, q_dims, strides, q_box) ||
        !make_bf16_tile_map(&mkv, p.cache, 2, kv_dims, strides, kv_box))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(LatentSmem<R, QR>) + 1024;
    // one CTA per SM, so that its tensor memory is its own
    static_assert(smem > (116u << 10) && smem <= 232448, "shared memory of one CTA per SM");
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = once_per_device(configured, [] {
        return cudaFuncSetAttribute(latent_attn_kernel<R, QR, JOINED>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    const int cluster = JOINED ? p.pieces : 1;
    e = launch_kernel_cluster(latent_attn_kernel<R, QR, JOINED>, dim3(p.grid * cluster), dim3(THREADS),
                              smem, cluster > 1 ? cluster : 0, stream, p, pg, mq, mkv);
    if (JOINED || e != cudaSuccess)
        return e;
    return launch_merge<R, QR>(p, stream);
}

template <int R>
cudaError_t launch_latent_rows(const LatentParams &p, const PagedView &pg, cudaStream_t stream)
{
    if (p.pieces > 0)
        return p.unit_rows == 32 ? launch_latent_t<R, 32, true>(p, pg, stream)
                                 : launch_latent_t<R, 64, true>(p, pg, stream);
    if (p.unit_rows == 32)
        return launch_latent_t<R, 32, false>(p, pg, stream);
    if constexpr (R > 128)
        if (p.unit_rows > 64) {
            const cudaError_t e = launch_latent_pair(p, pg, stream);
            return e != cudaSuccess ? e : launch_merge<R, 128>(p, stream);
        }
    return launch_latent_t<R, 64, false>(p, pg, stream);
}

}  // namespace

cudaError_t launch_latent(const LatentParams &p, const PagedView &pg, cudaStream_t stream)
{
    switch (p.R) {
    case 512: return launch_latent_rows<512>(p, pg, stream);
    case 256: return launch_latent_rows<256>(p, pg, stream);
    default: return launch_latent_rows<128>(p, pg, stream);
    }
}
