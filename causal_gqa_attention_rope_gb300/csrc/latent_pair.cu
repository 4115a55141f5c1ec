// latent_pair.cu -- absorbed latent attention (na_attn_latent_paged) in units of 128 query rows, for
// sequences that have more than 64 (chunks, drafted tokens, many heads): two CTAs as a pair
// (cta_group::2), by runs of key tiles as in latent_attn.cu.
//
// Each CTA has 64 of the rows, Q in shared memory.  For a tile of 64 keys
//     S   [128 rows x 64 keys]  = Q K^T      M = 128: a CTA has its rows and the tile's keys
//                                            32 rank .. + 31, all columns
//     O^T [R dims x 128 rows]  += V^T P^T    M = 256 per two blocks of 128 dims, one of each
//                                            CTA's: it has all keys of its dims, and P of its rows
// K's bytes are thus read from shared memory for 128 rows at a time, half in each CTA, and V's for
// all rows.  With 64 rows a CTA by itself the same products took its shared memory 1960
// cycles per tile (S 36 x 33, O^T 16 x 49) and the tensor cores 1660, tiles written not
// counted; here 1440 (36 x 26, 8 x 65).  The quarter of a tile that a CTA needs for both
// comes twice, once into K's ring and once into V's, and that pays: K is free as soon as S
// is done, where a tile that served both was held until the softmax and O^T were through, two
// deep, and that bounded the loop (3190 cycles a tile).
//
// O^T has the rows along its columns and the dims in both CTAs, so each of them rescales and
// normalises all 128 rows: the factors go to both by st.async, whose barrier
// also says that they are there.  K's and Q's copies of both CTAs complete on the first one's
// barriers.  That the second one's weights are written, its S read and its V landed its warps tell by
// arriving there too.  All that they speak of is in their own CTA's shared memory or in
// registers, so the release before the arrival is one of shared memory alone: one of all
// memory took some 900 cycles a tile (drafted tokens 191 us, 144 so).
//
// Warps: 0 loads Q and K, 3 V; of the first CTA 1 issues S, 2 issues O^T, of the second 1 tells
// that V has landed; 4 .. 7 and 8 .. 11 softmax of the even and the odd tiles (one group of
// four warps took 1500 cycles a tile, most of them latencies of its many meetings: drafted
// tokens 159 us, 145 with two groups): thread (32 q +
// lane) has row 32 (q % 2) + lane and half of a tile's keys.  The reference maximum goes from
// group to group as soon as a tile's maximum is known.
#include <climits>

#include "latent_runs.cuh"
#include "tc_primitives.cuh"
#include "tile_waits.cuh"

namespace {

constexpr int QR = 64, UR = 2 * QR;
constexpr int THREADS = 384;
constexpr int NUM_S = 4;
constexpr uint32_t Q_BLOCK = QR * 128, K_BLOCK = KT / 2 * 128, V_BLOCK = KT * 128;  // of 64 columns

template <int R>
struct __align__(1024) PairSmem {
    static constexpr int CB = R / 64 + 1;   // column blocks of a row
    static constexpr int DB = R / 256;      // blocks of 128 dims per CTA
    static constexpr int ST = R == 512 ? 2 : 4;
    bf16 q[CB][QR * 64];
    bf16 k[ST][CB][KT / 2 * 64];
    bf16 v[ST][2 * DB][KT * 64];
    bf16 p[2][QR * 64];
    float factor[2][UR];       // of all rows, from both CTAs
    float halves[2][2][QR];    // by group: maxima of a row's two threads; at a piece's end their sums
    float m_ref[2][QR];        // reference maxima after even and odd tiles
    uint64_t q_full, q_empty, k_full[ST], k_empty[ST], v_full[ST], v_empty[ST];
    uint64_t s_full[NUM_S], s_read[NUM_S], m_done[2], p_full[2], pv_done[2], f_full[2], sums_full,
        o_empty, drain[2];
    uint64_t v_other[ST];      // of the first CTA: the second one's V has landed
    long long warp_steps[THREADS / 32];
    long long total, begin;
    int b0, t0, step0;         // where the pair's run begins
    uint32_t tmem_base;
    int abort_flag;
};

// x into the word at `at`'s place in CTA `rank`, counted as 4 bytes on the barrier at `bar`'s there.
__device__ __forceinline__ void store_async(const float *at, const uint64_t *bar, int rank, float x)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                     place_in_cta(at, rank)),
                 "r"(__float_as_uint(x)), "r"(place_in_cta(bar, rank))
                 : "memory");
}

// One arrival on the barrier at `bar`'s place in the first CTA.  A thread there that waits with
// mbar_wait_cluster sees what is in this CTA's shared memory by now, this thread's writes and
// those that it has seen.
__device__ __forceinline__ void arrive_in_first(const uint64_t *bar)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(place_in_cta(bar, 0))
                 : "memory");
}

template <int R>
__global__ void __launch_bounds__(THREADS, 1)
    latent_pair_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ PagedView pg,
                       const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v)
{
    typedef PairSmem<R> Smem;
    constexpr int CB = Smem::CB, DB = Smem::DB, ST = Smem::ST;
    constexpr uint32_t S_COL = DB * UR;                // O^T block d at column 128 d, then S
    constexpr uint32_t TMEM_COLS = S_COL + NUM_S * KT / 2 <= 256 ? 256 : 512;
    const int run = blockIdx.x / 2, rank = blockIdx.x % 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < ST; i++) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
            mbar_init(&sm.v_other[i], 1);
        }
        for (int i = 0; i < NUM_S; i++) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_read[i], 8);  // a group's warps of both CTAs
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sm.m_done[i], 4);
            mbar_init(&sm.p_full[i], 8);
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.f_full[i], 1);
            mbar_init(&sm.drain[i], 1);
        }
        mbar_init(&sm.sums_full, 1);
        mbar_init(&sm.o_empty, 16);  // the softmax warps of both CTAs
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1)
        tc::tmem_alloc_pair(&sm.tmem_base, TMEM_COLS);
    grid_dependency_wait();
    grid_dependents_launch();
    tc::fence_before_sync();
    find_run<UR, THREADS / 32>(p, sm, run, warp, lane);
    cluster_sync();  // the other CTA's barriers and tensor memory are there
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    Walk<UR> w(p, sm, run);

    if (warp == 0 || warp == 3) {
        // ----------------------------------------------------------- producers --
        const bool is_k = warp == 0;
        const int box_log = min(pg.page_log, 6), boxes = KT >> box_log;  // rows of one page in a tile
        const int in_page = (1 << pg.page_log) - 1;
        uint64_t *full = is_k ? sm.k_full : sm.v_full, *empty = is_k ? sm.k_empty : sm.v_empty;
        int g = 0, pieces = 0;
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
            // not looked at before the tile's turn, then checked; -1 where there is none.
            auto has_page = [&](int j) {
                return lane < boxes && j < w.hi && j * KT + (lane << box_log) < w.keys;
            };
            auto ask = [&](int j) {
                return has_page(j) ? __ldg(row + ((j * KT + (lane << box_log)) >> pg.page_log)) : 0;
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
            if (is_k) {
                if (pieces > 0 && !wait_all(&sm.q_empty, (pieces - 1) & 1))
                    break;
                if (lane == 0 && rank == 0)
                    mbar_arrive_expect_tx(&sm.q_full, 2 * CB * Q_BLOCK);
                __syncwarp();
                if (lane < CB)
                    tc::tma_load_2d_pair(sm.q[lane], &map_q, lane * 64, (int)w.row0(p) + rank * QR,
                                         place_in_cta(&sm.q_full, 0));
            }
            for (int j = w.lo; ok && j < w.hi; j++, g++) {
                const int id = checked(j, asked), st = g % ST;
                asked = asked_next;
                asked_next = ask(j + 2);
                const unsigned there = __ballot_sync(0xffffffffu, id >= 0);
                if (!wait_all(&empty[st], ((g / ST) & 1) ^ 1))
                    break;
                // K: this CTA's 32 keys, 1 or 2 boxes; V: all keys, 1, 2 or 4
                const int log = is_k ? min(box_log, 5) : box_log;
                const int count = is_k ? KT / 2 >> log : boxes, blocks = is_k ? CB : 2 * DB;
                const int box = lane & (count - 1), block = lane / count;
                const int key = (is_k ? rank * (KT / 2) : 0) + (box << log);  // in the tile
                const int page = __shfl_sync(0xffffffffu, id, key >> box_log);
                const bool mine = block < blocks && (there >> (key >> box_log) & 1);
                // (the first CTA's barrier is told of K's bytes in both)
                const unsigned of_tile = __ballot_sync(
                    0xffffffffu, lane < (KT >> log) && (there >> (lane << log >> box_log) & 1));
                if (lane == 0 && (!is_k || rank == 0))
                    mbar_arrive_expect_tx(&full[st], __popc(of_tile) * blocks * (128u << log));
                __syncwarp();
                if (mine) {
                    const int y = (page << pg.page_log) + ((j * KT + key) & in_page);
                    if (is_k)
                        tc::tma_load_2d_pair(sm.k[st][block] + (box << log) * 64, &map_k, block * 64, y,
                                             place_in_cta(&full[st], 0));
                    else  // column blocks 2 i and 2 i + 1: dims (2 i + rank) 128 .. + 127
                        tc::tma_load_2d(sm.v[st][block] + (box << log) * 64, &map_v,
                                        (2 * (block >> 1) + rank) * 128 + (block & 1) * 64, y, &full[st]);
                }
            }
        }
        // every copy issued lands before the CTA can exit (K's and Q's of the second: the first waits)
        if (lane == 0 && (!is_k || rank == 0)) {
            if (is_k && pieces > 0)
                drain_wait(&sm.q_full, (pieces - 1) & 1, p.status);
            for (int i = g - 1; i >= 0 && i >= g - ST; i--)
                drain_wait(&full[i % ST], (i / ST) & 1, p.status);
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------- S = Q K^T issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(UR, KT, false, false);
            const uint64_t qd = tc::desc_kmajor_sw128(smem_addr(sm.q[0]));
            const uint64_t kd0 = tc::desc_kmajor_sw128(smem_addr(sm.k[0][0]));
            bool ok = true, issued = false;
            int g = 0;
            for (int piece = 0; ok && w.next(p); piece++) {
                ok = mbar_wait_bounded(&sm.q_full, piece & 1);
                for (int j = w.lo; ok && j < w.hi; j++, g++) {
                    const int sb = g % NUM_S, st = g % ST;
                    ok = mbar_wait_bounded(&sm.k_full[st], (g / ST) & 1);
                    if (ok && g >= NUM_S)
                        ok = mbar_wait_cluster(&sm.s_read[sb], (g / NUM_S - 1) & 1);
                    if (!ok || aborted(&sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t s_t = tmem + S_COL + sb * (KT / 2);
                    const uint64_t kd = kd0 + (uint64_t)(st * CB * (K_BLOCK >> 4));
#pragma unroll
                    for (int k = 0; k < CB * 4; k++)  // 16 columns, 32 bytes of a block's rows
                        tc::mma_ss_pair(s_t, qd + (k >> 2) * (Q_BLOCK >> 4) + (k & 3) * 2,
                                        kd + (k >> 2) * (K_BLOCK >> 4) + (k & 3) * 2, idesc, k > 0);
                    issued = true;
                    tc::mma_commit_pair(&sm.s_full[sb]);
                    tc::mma_commit_pair(&sm.k_empty[st]);
                    if (j == w.hi - 1)
                        tc::mma_commit_pair(&sm.q_empty);
                }
            }
            for (int i = max(g - NUM_S, 0); ok && i < g; i++)  // no arrival is under way at the end
                ok = mbar_wait_cluster(&sm.s_read[i % NUM_S], (i / NUM_S) & 1);
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            if (issued) {  // all issued MMAs complete before tensor memory is released
                tc::mma_commit_pair(&sm.drain[0]);
                drain_wait(&sm.drain[0], 0, p.status);
            }
        }
    } else if (warp == 2 && rank == 0) {
        // ----------------------------------------------------- O^T += V^T P^T issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(256, UR, true, false);
            const uint64_t vd0 = tc::desc_mnmajor_sw128(smem_addr(sm.v[0][0]), V_BLOCK);
            const uint64_t pd0 = tc::desc_kmajor_sw128(smem_addr(sm.p[0]));
            bool ok = true;
            int g = 0;
            for (int piece = 0; ok && w.next(p); piece++) {
                if (piece > 0)
                    ok = mbar_wait_cluster(&sm.o_empty, (piece - 1) & 1);
                for (int j = w.lo; ok && j < w.hi; j++, g++) {
                    const int st = g % ST;
                    ok = mbar_wait_bounded(&sm.v_full[st], (g / ST) & 1) &&
                         mbar_wait_cluster(&sm.v_other[st], (g / ST) & 1) &&
                         mbar_wait_cluster(&sm.p_full[g & 1], (g >> 1) & 1);
                    if (!ok || aborted(&sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint64_t pd = pd0 + (uint64_t)((g & 1) * (Q_BLOCK >> 4));
#pragma unroll
                    for (int d = 0; d < DB; d++) {
                        const uint64_t vd = vd0 + (uint64_t)((st * 2 * DB + 2 * d) * (V_BLOCK >> 4));
#pragma unroll
                        for (int k = 0; k < KT / 16; k++)  // 16 keys: rows of 128 B of V, 32 B of a row of P
                            tc::mma_ss_pair(tmem + d * UR, vd + (uint64_t)(k * 128), pd + (uint64_t)(k * 2),
                                            idesc, j > w.lo || k > 0);
                    }
                    tc::mma_commit_pair(&sm.v_empty[st]);
                    tc::mma_commit_pair(&sm.pv_done[g & 1]);
                }
            }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            if (g > 0) {
                tc::mma_commit_pair(&sm.drain[1]);
                drain_wait(&sm.drain[1], 0, p.status);
            }
        }
    } else if (warp == 1) {
        // ------------------------- of the second CTA: tells the first that V has landed --
        if (lane == 0) {
            bool ok = true;
            for (int g = 0; ok && w.next(p);)
                for (int j = w.lo; ok && j < w.hi; j++, g++) {
                    ok = mbar_wait_bounded(&sm.v_full[g % ST], (g / ST) & 1) && !aborted(&sm.abort_flag);
                    if (ok)
                        arrive_in_first(&sm.v_other[g % ST]);
                }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
        }
    } else if (warp >= 4) {
        // -------------------------------------------------------------- softmax --
        const int group = warp >= 8, quarter = warp & 3, tid = threadIdx.x & 127;
        const int r = (quarter & 1) * 32 + lane, half = quarter >> 1;  // row, and keys 32 half .. + 31
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float sl2 = p.scale_log2;
        bool ok = true;
        int g = 0;  // tiles, those of group g & 1
        // x of this CTA's rows to both CTAs, into `to` (of all rows) ...
        auto send = [&](float *to, uint64_t *bar, float x) {
            if (half == 0)
#pragma unroll
                for (int c = 0; c < 2; c++)
                    store_async(to + rank * QR + r, bar, c, x);
            if (tid == 0)
                mbar_arrive_expect_tx(bar, UR * 4);
        };
        // ... where they are when this has returned true.
        auto received = [&](uint64_t *bar, uint32_t parity) {
            const bool done = mbar_wait_cluster(bar, parity) && !aborted(&sm.abort_flag);
            return __all_sync(0xffffffffu, done) != 0;
        };
        // An arrival of this warp in the first CTA.
        auto tell = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) {
                if (rank == 0)
                    mbar_arrive(bar);
                else
                    arrive_in_first(bar);
            }
        };
        const bool leader = threadIdx.x == 128 && rank == 0;
        if (leader && !p.cut_by_sequence)
            p.cut[run] = make_int4(0, 0, 0, -1);
        for (int piece = 0; ok && w.next(p); piece++) {
            const int rows = w.rows(p, 0, UR), mine = w.rows(p, rank * QR, QR);
            // keys that the row sees
            const int lim = r < mine ? w.s.prior + (w.unit * UR + rank * QR + r) / p.H + 1 : 0;
            const int g0 = g, g_end = g + w.hi - w.lo;
            float m_own = -INFINITY, sum = 0.f;  // of this group's tiles
            for (g += (g ^ group) & 1; g < g_end; g += 2) {
                const int j0 = (w.lo + g - g0) * KT, sb = g % NUM_S, st = g % ST;
                ok = ok && warp_wait(&sm.s_full[sb], (g / NUM_S) & 1, &sm.abort_flag);
                uint32_t s[32];
                if (ok) {
                    tc::fence_after_sync();
                    tc::tmem_ld32(tmem + S_COL + sb * (KT / 2) + lane_off, s);
                    tc::tmem_wait_ld();
                    tc::fence_before_sync();
                    tell(&sm.s_read[sb]);
                    // The product before the last is done: its P, and all that the group had for
                    // it here and in the other CTA, may be written over.
                    if (g >= 2)
                        ok = warp_wait(&sm.pv_done[group], ((g >> 1) - 1) & 1, &sm.abort_flag);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        s[i] = 0;
                }
                if (j0 + KT > lim) {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (j0 + half * 32 + i >= lim)
                            s[i] = __float_as_uint(-INFINITY);
                }
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; i++)
                    mx = max3f(mx, __uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
                sm.halves[group][half][r] = mx;
                // (a warp whose wait gave up still comes here, so that the others go on to see it)
                if (any_of(!ok, 1 + group, 128)) {
                    ok = false;
                    break;
                }
                mx = fmaxf(mx, sm.halves[group][half ^ 1][r]) * sl2;
                // the reference after the tile before, which the other group had
                float m_ref = -INFINITY, alpha = 1.f;  // (1 as well where there is nothing to rescale yet)
                if (g > g0) {
                    ok = warp_wait(&sm.m_done[group ^ 1], ((g - 1) >> 1) & 1, &sm.abort_flag);
                    m_ref = sm.m_ref[group ^ 1][r];
                }
                if (mx > m_ref + 8.0f) {
                    if (m_ref != -INFINITY)
                        alpha = ex2_mufu(m_ref - mx);
                    m_ref = mx;
                }
                if (half == 0)
                    sm.m_ref[group][r] = m_ref;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.m_done[group]);
                send(sm.factor[group], &sm.f_full[group], alpha);
                const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
                float2 acc = make_float2(0.f, 0.f);
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const float2 x = __ffma2_rn(
                        make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                        make_float2(sl2, sl2), make_float2(neg_m, neg_m));
                    const float2 e = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
                    acc = __fadd2_rn(acc, e);
                    pk[i] = pack_bf16x2(e.x, e.y);
                }
                if (m_own != m_ref) {
                    sum *= m_own == -INFINITY ? 0.f : ex2_mufu(m_own - m_ref);
                    m_own = m_ref;
                }
                sum += acc.x + acc.y;
#pragma unroll
                for (int c = 0; c < 4; c++)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(sm.p[group]) + r * 128 +
                                               (((half * 4 + c) ^ (r & 7)) << 4)) =
                        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                if (ok && j0 + KT > w.keys) {
                    // Rows behind the last key hold whatever was there: zeros, so that no weight of 0
                    // meets a NaN.
                    ok = warp_wait(&sm.v_full[st], (g / ST) & 1, &sm.abort_flag);
                    const int from = w.keys - j0, per = (KT - from) * 8;
                    for (int i = tid; ok && i < per * 2 * DB; i += 128)
                        reinterpret_cast<uint4 *>(sm.v[st][i / per])[from * 8 + i % per] =
                            make_uint4(0, 0, 0, 0);
                }
                ok = received(&sm.f_full[group], (g >> 1) & 1) && ok;
                const float4 fs = reinterpret_cast<const float4 *>(sm.factor[group])[lane];
                if (__any_sync(0xffffffffu, fs.x != 1.f || fs.y != 1.f || fs.z != 1.f || fs.w != 1.f) && ok) {
                    // O^T is touched only to rescale it, when the last product has landed
                    ok = warp_wait(&sm.pv_done[group ^ 1], ((g - 1) >> 1) & 1, &sm.abort_flag);
                    if (ok) {
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < DB * UR; c += 32) {
                            uint32_t o[32];
                            tc::tmem_ld32(tmem + lane_off + c, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) *
                                                       sm.factor[group][(c & (UR - 1)) + i]);
                            tc::tmem_st32(tmem + lane_off + c, o);
                        }
                        tc::tmem_wait_st();
                    }
                }
                if (ok) {
                    tc::fence_proxy_async_smem();
                    tc::fence_before_sync();
                    tell(&sm.p_full[group]);
                }
            }
            // ------------------------------------------------------- a piece's rows --
            g = g_end;
            if (ok)  // (the last product; all before it are done then)
                ok = warp_wait(&sm.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &sm.abort_flag);
            if (any_of(!ok, 3, 256)) {
                ok = false;
                break;
            }
            const float m_ref = sm.m_ref[(g - 1) & 1][r];
            if (m_own != m_ref)
                sum *= m_own == -INFINITY ? 0.f : ex2_mufu(m_own - m_ref);
            sm.halves[group][half][r] = sum;
            named_barrier_sync(3, 256);
            sum = (sm.halves[0][0][r] + sm.halves[0][1][r]) + (sm.halves[1][0][r] + sm.halves[1][1][r]);
            const bool whole = w.lo == 0 && w.hi == w.tiles;
            const size_t slot_row = (size_t)(2 * run + (w.lo == 0 ? 1 : 0)) * UR;
            if (!whole && group == 0 && half == 0 && r < mine)
                reinterpret_cast<float2 *>(p.part_ml)[slot_row + rank * QR + r] = make_float2(m_ref, sum);
            float *inv = reinterpret_cast<float *>(sm.p[0]);  // (P is done with here and in the other CTA)
            if (group == 0)
                send(inv, &sm.sums_full, whole ? (sum > 0.f ? 1.0f / sum : 0.f) : 1.f);
            ok = received(&sm.sums_full, piece & 1);
            tc::fence_after_sync();
            const long long row0 = w.row0(p);
#pragma unroll 1
            for (int c = group * 32; ok && c < DB * UR; c += 64) {
                const int r0 = c & (UR - 1), dim = (2 * (c / UR) + rank) * 128 + quarter * 32 + lane;
                if (r0 >= rows)
                    continue;
                uint32_t o[32];
                tc::tmem_ld32(tmem + lane_off + c, o);
                tc::tmem_wait_ld();
                if (whole) {
                    bf16 *dst = p.out + (row0 + r0) * R + dim;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (r0 + i < rows)
                            dst[(size_t)i * R] =
                                __float2bfloat16_rn(__uint_as_float(o[i]) * inv[r0 + i]);
                } else {
                    float *dst = p.part_o + (slot_row + r0) * R + dim;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (r0 + i < rows)
                            dst[(size_t)i * R] = __uint_as_float(o[i]);
                }
            }
            if (any_of(!ok, 3, 256)) {  // (and the sums and maxima have been read)
                ok = false;
                break;
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(&sm.o_empty, 0);
            if (w.lo == 0 && leader) {
                // the unit ends (tiles - hi) behind the end of this run
                const long long end = run_begin(p, sm.total, run + 1) + (w.tiles - w.hi);
                if (!whole || p.cut_by_sequence)
                    p.cut[p.cut_by_sequence ? w.seq : run] =
                        make_int4((int)w.row0(p), rows, run, whole ? -1 : run_of(p, sm.total, end));
            }
        }
        if (!ok && lane == 0)
            set_abort(&sm.abort_flag, p.status);
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // the other CTA's products read this one's memory, and it arrives in it
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

template <int R>
cudaError_t launch_pair_t(const LatentParams &p, const PagedView &pg, cudaStream_t stream)
{
    CUtensorMap mq, mk, mv;
    const cuuint64_t wide = R + p.rd;
    const cuuint64_t q_dims[2] = {wide, (cuuint64_t)p.total_tokens * p.H};
    const cuuint64_t kv_dims[2] = {wide, (cuuint64_t)pg.num_pages << pg.page_log};
    const cuuint64_t strides[1] = {wide * 2};
    const cuuint32_t q_box[2] = {64, QR}, k_box[2] = {64, 1u << (pg.page_log < 5 ? pg.page_log : 5)},
                     v_box[2] = {64, 1u << (pg.page_log < 6 ? pg.page_log : 6)};
    if (!make_bf16_tile_map(&mq, p.q, 2, q_dims, strides, q_box) ||
        !make_bf16_tile_map(&mk, p.cache, 2, kv_dims, strides, k_box) ||
        !make_bf16_tile_map(&mv, p.cache, 2, kv_dims, strides, v_box))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(PairSmem<R>);
    // one CTA per SM, so that its tensor memory is its own
    static_assert(smem > (116u << 10) && smem <= 232448, "shared memory of one CTA per SM");
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = once_per_device(configured, [] {
        return cudaFuncSetAttribute(latent_pair_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(latent_pair_kernel<R>, dim3(2 * p.grid), dim3(THREADS), smem, 2, stream, p,
                                 pg, mq, mk, mv);
}

}  // namespace

cudaError_t launch_latent_pair(const LatentParams &p, const PagedView &pg, cudaStream_t stream)
{
    return p.R == 512 ? launch_pair_t<512>(p, pg, stream) : launch_pair_t<256>(p, pg, stream);
}
