// latent_expanded.cu -- expanded latent attention (na_attn_latent_expanded): causal
// attention of nope_dim + rope_dim and v_dim, on the sm_100-family tensor cores
// (tcgen05 + TMEM + TMA).
//
// Query tokens of one head against the key tiles that they see: S = Q K^T with K of dn + 64
// columns -- the head's own dn out of kv's rows and the rotated part that all heads share,
// padded by TMA's zeros to a column block -- then O += P V, P over its S in tensor
// memory, a softmax thread per row, the reference maximum raised only when a score exceeds
// it by more than 2^8.  Keys and values are read where the expanding product left them,
// so nothing is concatenated.  Two kernels; plan_expanded() in latent_api.cu says which when:
//
// latent_expanded_kernel: 128 rows, tiles of 64 keys, two CTAs per SM, one at its products while
// the other begins, ends or waits: for short prompts.  16 of 1 .. 512 tokens, 32 heads: 86 us,
// and 107 with one CTA per SM and tiles of 128 keys.
//
// latent_expanded_tall_kernel: 256 rows as two tiles that take turns, the products of one beside the
// softmax of the other, with one CTA per SM and 128 keys at a time.  K of 192 columns costs
// shared memory as much time as the tensor cores (per 128 rows and keys Q, K and V are
// read for the products, 128 KB, and K and V written, 80 KB: 1625 cycles at 128 bytes,
// against 1280 of products); two tiles write K and V once for both.  8 waves of full CTAs run
// at 1580 TFLOP/s (0.92 of what the tensor cores sustain), with one tile per CTA and three
// buffers of S 1494.  One thread issues the products of both tiles, so that S needs one
// buffer per tile, and K and V come through a ring of column blocks, because a whole tile
// of either would have to wait for all of the one before.
// A unit can be cut into pieces of its keys: the CTAs of a cluster take one each and join their rows
// out of one another's shared memory.  That fills the SMs where units are few, and the last wave:
// 2048 tokens after 28672, 40 heads, are 320 units on 152 SMs: 1033 us, with the last 16 in six
// pieces, and the others in turn, 944 .. 997 from run to run (1650 .. 1560 TFLOP/s).
#include <algorithm>
#include <climits>

#include "latent.cuh"
#include "tc_primitives.cuh"
#include "tile_waits.cuh"

namespace {

constexpr int BM = kExpandedRows;
constexpr uint32_t S_COL0 = 128;  // O at column 0, S buffer i at column S_COL0 + BN i
constexpr uint32_t Q_BLOCK = BM * 128;  // a column block: rows of 64 bf16

// ------------------------------------------------------------------- the unit --

// What a CTA works on: UR query rows of a head and sequence, and what they see.
struct Unit {
    int head, tok0, n, start;
    int r0, rows;       // its first row within the sequence and how many (1 .. UR) it has
    int pos_lo, k_end;  // position of row 0 (may be negative), keys that the last row sees
    bool run;           // there are rows, and they are sound (a bad sequence is reported)
};

// Units run with the last query tiles, which see most keys, first; up to 32 sequences in order
// of decreasing keys, so that the longest units start first.
template <int UR>
__device__ __forceinline__ Unit find_unit(const ExpandedParams &p, int index, int lane, bool reporter)
{
    Unit u;
    const int units = (p.max_new_len + UR - 1) / UR;  // of a sequence and head
    u.r0 = (units - 1 - index % units) * UR;
    u.head = index / units % p.H;
    int b = index / units / p.H;
    if (p.batch > 1 && p.batch <= 32) {
        const int key = lane < p.batch ? __ldg(p.key_lens + lane) : INT_MIN;
        int order = 0;
        for (int i = 0; i < p.batch; i++) {
            const int other = __shfl_sync(0xffffffffu, key, i);
            order += other > key || (other == key && i < lane);
        }
        b = __ffs(__ballot_sync(0xffffffffu, lane < p.batch && order == b)) - 1;
    }
    u.tok0 = __ldg(p.cu_seqlens + b);
    u.n = __ldg(p.cu_seqlens + b + 1) - u.tok0;
    u.start = __ldg(p.key_starts + b);
    const int keys = __ldg(p.key_lens + b);
    u.rows = min(UR, u.n - u.r0);
    u.pos_lo = keys - u.n + u.r0;
    u.k_end = u.pos_lo + u.rows;
    u.run = false;
    if (u.n > p.max_new_len || u.tok0 < 0 || (b == 0 && u.tok0 != 0) ||
        (long long)u.tok0 + u.n > p.total_tokens) {
        if (u.r0 == 0 && u.head == 0 && reporter)
            na_report(p.status, NA_ERR_INVALID_ARG);
    } else if (u.rows <= 0) {
        // padding: the sequence has fewer tiles
    } else if (keys < 0 || u.start < 0 || keys > p.max_key_len ||
               (long long)u.start + keys > p.total_keys) {
        if (reporter)
            na_report(p.status, NA_ERR_CAPACITY);
    } else {
        u.run = true;
    }
    return u;
}

template <int DV>
__device__ __forceinline__ bf16 *rows_out(const ExpandedParams &p, const Unit &u)
{
    return p.out + ((size_t)(u.tok0 + u.r0) * p.H + u.head) * DV;
}

// Rows that see no key.
template <int DV>
__device__ __forceinline__ void store_zeros(const ExpandedParams &p, const Unit &u, int tid, int threads)
{
    bf16 *out = rows_out<DV>(p, u);
    for (int i = tid; i < u.rows * (DV / 8); i += threads)
        *reinterpret_cast<uint4 *>(out + (size_t)(i / (DV / 8)) * p.H * DV + i % (DV / 8) * 8) =
            make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ the softmax --

// A softmax thread's row: reference maximum (log2 domain) and sum.
struct RowState {
    float m_ref = -INFINITY, l = 0.f;
};

// Scores of a tile, NB x 32 keys from j0 on, in tensor memory at s_t: masked, exponentiated, the
// weights written over them as bf16.  `alpha`, the factor of what was summed before, is to
// be applied to O where the result is true.
template <int NB>
__device__ __forceinline__ bool weigh_tile(uint32_t s_t, int j0, int pos_lo, int row_pos, int k_end,
                                           float sl2, RowState &st, float &alpha)
{
    uint32_t sr[NB][32];
#pragma unroll
    for (int c = 0; c < NB; c++)
        tc::tmem_ld32(s_t + c * 32, sr[c]);
    tc::tmem_wait_ld();
    if (j0 + NB * 32 - 1 > pos_lo) {  // (rows see keys up to their position, < k_end)
#pragma unroll
        for (int c = 0; c < NB; c++)
#pragma unroll
            for (int i = 0; i < 32; i++) {
                const int key = j0 + c * 32 + i;
                if (key > row_pos || key >= k_end)
                    sr[c][i] = __float_as_uint(-INFINITY);
            }
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < NB; c++)
#pragma unroll
        for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int k = 0; k < 4; k++)
                mx[k] = max3f(mx[k], __uint_as_float(sr[c][i + 2 * k]),
                              __uint_as_float(sr[c][i + 2 * k + 1]));
    const float mxs = max3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * sl2;
    alpha = 1.f;
    bool corr = false;
    if (mxs > st.m_ref + 8.0f) {
        alpha = st.m_ref == -INFINITY ? 0.f : ex2_mufu(st.m_ref - mxs);
        corr = st.m_ref != -INFINITY;
        st.m_ref = mxs;
    }
    const float neg_m = st.m_ref == -INFINITY ? 0.f : -st.m_ref;
    float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                     make_float2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < NB; c++) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1])),
                make_float2(sl2, sl2), make_float2(neg_m, neg_m));
            const float2 e = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
            acc[i & 3] = __fadd2_rn(acc[i & 3], e);
            pk[i] = pack_bf16x2(e.x, e.y);
        }
        tc::tmem_st16(s_t + c * 16, pk);
    }
    const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
    st.l = fmaf(st.l, alpha, (a01.x + a01.y) + (a23.x + a23.y));
    tc::tmem_wait_st();
    return corr;
}

// This warp's rows of O times `a`.
template <int DV>
__device__ __forceinline__ void rescale_rows(uint32_t o_t, float a)
{
#pragma unroll
    for (int c = 0; c < DV / 32; c++) {
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

// Key row r of a V tile's column blocks: zeros, so that no weight of 0 meets a NaN.
__device__ __forceinline__ void zero_row(bf16 *block, int r)
{
    uint4 *row = reinterpret_cast<uint4 *>(block + r * 64);
#pragma unroll
    for (int i = 0; i < 8; i++)
        row[i] = make_uint4(0, 0, 0, 0);
}

// The normalised rows, a thread each, into `stage`, whose rows are padded by 16 bytes so that
// this meets no bank conflicts ...
template <int DV>
__device__ __forceinline__ void stage_row(uint32_t o_t, float scale, float *stage, int r)
{
#pragma unroll
    for (int c = 0; c < DV / 32; c++) {
        uint32_t o[32];
        tc::tmem_ld32(o_t + c * 32, o);
        tc::tmem_wait_ld();
        float4 *row = reinterpret_cast<float4 *>(stage + r * (DV + 4) + c * 32);
#pragma unroll
        for (int i = 0; i < 8; i++)
            row[i] = make_float4(__uint_as_float(o[4 * i]) * scale, __uint_as_float(o[4 * i + 1]) * scale,
                                 __uint_as_float(o[4 * i + 2]) * scale,
                                 __uint_as_float(o[4 * i + 3]) * scale);
    }
}

// ... and from there to the output, a row per warp and instruction.
template <int DV>
__device__ __forceinline__ void store_rows(const ExpandedParams &p, const Unit &u, const float *stage,
                                           int warp, int lane)
{
    constexpr int EPL = DV / 32;  // elements per lane
    bf16 *out = rows_out<DV>(p, u);
    for (int r = warp; r < u.rows; r += blockDim.x / 32) {
        const float *src = stage + r * (DV + 4) + lane * EPL;
        bf16 *dst = out + (size_t)r * p.H * DV + lane * EPL;
        if constexpr (EPL == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(src);
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(src);
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(x.x, x.y);
        }
    }
}

// ------------------------------------------------------- 128 rows: two CTAs per SM --
//
// Warps: 0 producer, 1 issues S, 2 issues O, 4 .. 7 softmax; all eight store the rows.

namespace two {
constexpr int THREADS = 256;
constexpr int BN = 64;
constexpr int NUM_S = 2;
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t KV_BLOCK = BN * 128;
}  // namespace two

template <int DN, int DV>
struct __align__(1024) ExpandedSmem {
    static constexpr int QB = DN / 64 + 1, VB = DV / 64;  // column blocks
    static constexpr int KST = 2, VST = 1;
    bf16 q[QB][BM * 64];
    bf16 k[KST][QB][two::BN * 64];
    bf16 v[VST][VB][two::BN * 64];
    uint64_t q_full, k_full[KST], k_empty[KST], v_full[VST], v_empty[VST];
    uint64_t s_full[two::NUM_S], s_free[two::NUM_S], p_full[two::NUM_S], o_done[two::NUM_S], drain[2];
    uint32_t tmem_base;
    int abort_flag;
};

template <int DN, int DV>
__global__ void __launch_bounds__(two::THREADS, 2)
    latent_expanded_kernel(const __grid_constant__ ExpandedParams p,
                           const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_kv,
                           const __grid_constant__ CUtensorMap map_pe)
{
    using namespace two;
    typedef ExpandedSmem<DN, DV> Smem;
    constexpr int QB = Smem::QB, VB = Smem::VB, KST = Smem::KST, VST = Smem::VST;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_kv);
        tc::prefetch_tmap(&map_pe);
        mbar_init(&sm.q_full, 1);
        for (int i = 0; i < KST; i++) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < VST; i++) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int i = 0; i < NUM_S; i++) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_done[i], 1);
        }
        mbar_init(&sm.drain[0], 1);
        mbar_init(&sm.drain[1], 1);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    grid_dependents_launch();

    const Unit u = find_unit<BM>(p, blockIdx.x, lane, threadIdx.x == 0);
    if (!u.run)
        return;
    if (u.k_end <= 0) {
        store_zeros<DV>(p, u, threadIdx.x, THREADS);
        return;
    }
    const int n_tiles = (u.k_end + BN - 1) / BN;
    auto load_k = [&](int j) {
        const int st = j % KST;
        mbar_arrive_expect_tx(&sm.k_full[st], QB * KV_BLOCK);
        for (int c = 0; c < QB - 1; c++)
            tc::tma_load_3d(sm.k[st][c], &map_kv, c * 64, u.head, u.start + j * BN, &sm.k_full[st]);
        tc::tma_load_2d(sm.k[st][QB - 1], &map_pe, 0, u.start + j * BN, &sm.k_full[st]);
    };
    auto load_v = [&](int j) {
        const int st = j % VST;
        mbar_arrive_expect_tx(&sm.v_full[st], VB * KV_BLOCK);
        for (int c = 0; c < VB; c++)
            tc::tma_load_3d(sm.v[st][c], &map_kv, DN + c * 64, u.head, u.start + j * BN, &sm.v_full[st]);
    };
    const int k_pre = min(n_tiles, KST), v_pre = min(n_tiles, VST);
    if (threadIdx.x == 0) {  // (fresh stages need no wait)
        mbar_arrive_expect_tx(&sm.q_full, QB * Q_BLOCK);
        for (int c = 0; c < QB; c++)
            tc::tma_load_3d(sm.q[c], &map_q, c * 64, u.head, u.tok0 + u.r0, &sm.q_full);
        for (int j = 0; j < k_pre; j++)
            load_k(j);
        for (int j = 0; j < v_pre; j++)
            load_v(j);
    }
    if (warp == 1)
        tc::tmem_alloc(&sm.tmem_base, TMEM_COLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;

    static_assert(sizeof(float) * BM * (DV + 4) <= sizeof(sm.q) + sizeof(sm.k) + sizeof(sm.v),
                  "the rows are staged over Q, K and V, idle by then");
    float *stage = reinterpret_cast<float *>(&sm.q[0]);

    if (warp == 0) {
        // ------------------------------------------------------------ producer --
        if (lane == 0) {
            int k_issued = k_pre, v_issued = v_pre;
            bool ok = true;
            while (ok && (k_issued < n_tiles || v_issued < n_tiles)) {
                // in the order of their use: K of a tile two tiles ahead of V's
                if (k_issued < n_tiles && k_issued - v_issued <= KST - VST) {
                    ok = mbar_wait_bounded(&sm.k_empty[k_issued % KST], ((k_issued / KST) & 1) ^ 1) &&
                         !aborted(&sm.abort_flag);
                    if (ok)
                        load_k(k_issued++);
                } else {
                    ok = mbar_wait_bounded(&sm.v_empty[v_issued % VST], ((v_issued / VST) & 1) ^ 1) &&
                         !aborted(&sm.abort_flag);
                    if (ok)
                        load_v(v_issued++);
                }
            }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            // every copy issued lands before the CTA can exit
            drain_wait(&sm.q_full, 0, p.status);
            for (int j = k_issued - 1; j >= 0 && j >= k_issued - KST; j--)
                drain_wait(&sm.k_full[j % KST], (j / KST) & 1, p.status);
            for (int j = v_issued - 1; j >= 0 && j >= v_issued - VST; j--)
                drain_wait(&sm.v_full[j % VST], (j / VST) & 1, p.status);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- S = Q K^T issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(BM, BN, false, false);
            constexpr uint32_t Q16 = Q_BLOCK >> 4, K16 = KV_BLOCK >> 4;
            const uint64_t qd = tc::desc_kmajor_sw128(smem_addr(sm.q[0]));
            const uint64_t kd0 = tc::desc_kmajor_sw128(smem_addr(sm.k[0][0]));
            bool ok = mbar_wait_bounded(&sm.q_full, 0), any = false;
            for (int j = 0; ok && j < n_tiles; j++) {
                const int st = j % KST, sb = j % NUM_S;
                ok = mbar_wait_bounded(&sm.k_full[st], (j / KST) & 1);
                if (ok && j >= NUM_S)
                    ok = mbar_wait_bounded(&sm.s_free[sb], ((j / NUM_S) - 1) & 1);
                if (!ok || aborted(&sm.abort_flag))
                    break;
                tc::fence_after_sync();
                const uint32_t s_t = tmem + S_COL0 + sb * BN;
                const uint64_t kd = kd0 + (uint64_t)(st * QB * K16);
#pragma unroll
                for (int k = 0; k < QB * 4; k++)
                    tc::mma_ss(s_t, qd + (k >> 2) * Q16 + (k & 3) * 2, kd + (k >> 2) * K16 + (k & 3) * 2,
                               idesc, k > 0);
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
        // --------------------------------------------------------- O += P V issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(BM, DV, false, true);
            constexpr uint32_t V16 = KV_BLOCK >> 4;
            const uint64_t vd0 = tc::desc_mnmajor_sw128(smem_addr(sm.v[0][0]), KV_BLOCK);
            bool ok = true, any = false;
            for (int j = 0; ok && j < n_tiles; j++) {
                const int st = j % VST, sb = j % NUM_S;
                ok = mbar_wait_bounded(&sm.p_full[sb], (j / NUM_S) & 1) &&
                     mbar_wait_bounded(&sm.v_full[st], (j / VST) & 1);
                if (!ok || aborted(&sm.abort_flag))
                    break;
                tc::fence_after_sync();
                const uint32_t p_t = tmem + S_COL0 + sb * BN;
                const uint64_t vd = vd0 + (uint64_t)(st * VB * V16);
#pragma unroll
                for (int k = 0; k < BN / 16; k++)  // 16 keys = 16 rows of 128 B per step
                    tc::mma_ts(tmem, p_t + k * 8, vd + (uint64_t)(k * 128), idesc, j > 0 || k > 0);
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
        // -------------------------------------------------------------- softmax --
        const int quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16, o_t = tmem + lane_off;
        RowState st;
        bool ok = true;
        for (int j = 0; ok && j < n_tiles; j++) {
            const int sb = j % NUM_S, j0 = j * BN;
            if (!(ok = warp_wait(&sm.s_full[sb], (j / NUM_S) & 1, &sm.abort_flag)))
                break;
            tc::fence_after_sync();
            float alpha;
            const bool corr = weigh_tile<BN / 32>(tmem + S_COL0 + sb * BN + lane_off, j0, u.pos_lo,
                                                  u.pos_lo + r, u.k_end, p.scale_log2, st, alpha);
            if (j0 + BN > u.k_end) {  // rows behind the last visible key may hold any bits
                // (V's barrier only tells the phases of two tiles apart: V of the tile before has
                // landed when its product is done)
                const int vs = j % VST;
                if (j >= 1 &&
                    !(ok = warp_wait(&sm.o_done[(j - 1) % NUM_S], ((j - 1) / NUM_S) & 1, &sm.abort_flag)))
                    break;
                if (!(ok = warp_wait(&sm.v_full[vs], (j / VST) & 1, &sm.abort_flag)))
                    break;
                if (r < BN && r >= u.k_end - j0)
                    for (int c = 0; c < VB; c++)
                        zero_row(sm.v[vs][c], r);
                tc::fence_proxy_async_smem();
            }
            if (j >= 1 && __any_sync(0xffffffffu, corr)) {
                // O is touched only to rescale it, and then PV(j - 1) has to have landed (its
                // barrier's phase is exact however rarely it is looked at: S(j) could not be
                // issued before PV(j - NUM_S), and PV(j - 1 + NUM_S) needs a P not yet written)
                if (!(ok = warp_wait(&sm.o_done[(j - 1) % NUM_S], ((j - 1) / NUM_S) & 1, &sm.abort_flag)))
                    break;
                tc::fence_after_sync();
                rescale_rows<DV>(o_t, corr ? alpha : 1.f);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.p_full[sb]);
        }
        if (ok && warp_wait(&sm.o_done[(n_tiles - 1) % NUM_S], ((n_tiles - 1) / NUM_S) & 1,
                            &sm.abort_flag)) {
            tc::fence_after_sync();
            stage_row<DV>(o_t, st.l > 0.f ? 1.0f / st.l : 0.f, stage, r);
        } else if (lane == 0) {
            set_abort(&sm.abort_flag, p.status);
        }
    }
    tc::fence_before_sync();
    __syncthreads();  // the staged rows are complete (unless a wait gave up)
    if (!aborted(&sm.abort_flag))
        store_rows<DV>(p, u, stage, warp, lane);
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ---------------------------------------------------- 256 rows, in pieces of their keys --
//
// Warps: 0 .. 7 softmax, a row of the two tiles per thread, 8 producer, 9 issues all products, 10
// finds the next units.  Where plan_expanded() lets a CTA take units in turn, the roles go on to the
// next as soon as they are done with one: its keys and queries are on their way while the
// last products run, and its first scores are behind them while the rows are stored (2048 tokens
// after 4096, 40 heads: 216 us by a CTA per unit, 191).

namespace tall {
constexpr int THREADS = 384;
constexpr int TILES = 2;         // query tiles of a CTA
constexpr int UR = TILES * BM;
constexpr int BN = 128;
constexpr uint32_t O_COL0 = 256;  // S of tile t at column 128 t, O behind them
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t BLOCK = BN * 128;  // a column block: 128 rows of 64 bf16
}  // namespace tall

// K and V of the key tiles pass through one ring of column blocks, in the order of their use:
// K of tile 0, its V, K of tile 1 ...
template <int DN, int DV>
struct __align__(1024) TallSmem {
    static constexpr int QB = DN / 64 + 1, VB = DV / 64;  // column blocks
    static constexpr int PER = QB + VB;                   // of a key tile
    static constexpr int SLOTS = 14 - tall::TILES * QB;
    bf16 q[tall::TILES][QB][BM * 64];
    bf16 ring[SLOTS][tall::BN * 64];
    uint64_t q_full[tall::TILES], q_empty[tall::TILES], full[SLOTS], empty[SLOTS];
    uint64_t s_full[tall::TILES], p_full[tall::TILES], o_done[tall::TILES], o_empty[tall::TILES], drain;
    uint64_t unit_full[2], unit_empty[2];
    Unit unit[2];              // the next ones, handed to all roles; rows 0: no more
    uint32_t tmem_base;
    int abort_flag;
};

// A place in the ring.
template <int SLOTS>
struct RingAt {
    int slot;
    uint32_t parity;  // of its `full` barrier
    __device__ __forceinline__ explicit RingAt(int item) : slot(item % SLOTS), parity((item / SLOTS) & 1) {}
};

// `at`'s place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t place_in_cta(const void *at, int rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(at)), "r"(rank));
    return a;
}

__device__ __forceinline__ float4 load_cluster(uint32_t a)
{
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(a)
                 : "memory");
    return x;
}

__device__ __forceinline__ int load_cluster_word(uint32_t a)
{
    int x;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}

// A unit's rows from the P pieces of its keys, a CTA of the cluster each: those of 1 / P of the
// warps here, staged unnormalised with their maxima and sums by every CTA.  Other CTAs' shared
// memory gives some 14 bytes a cycle (5 us for a unit), so that nothing is asked for
// twice, and the own piece not through the cluster; P is known to the compiler, because loads
// behind a branch were waited for one by one.
template <int DV, int P>
__device__ __forceinline__ void join_rows_of(const ExpandedParams &p, const Unit &u, const float *stage,
                                             const int *abort_flag, int piece, int warp, int lane)
{
    int bad = 0;
#pragma unroll
    for (int c = 0; c < P; c++)
        bad |= load_cluster_word(place_in_cta(abort_flag, c));
    if (bad)
        return;
    bf16 *out = rows_out<DV>(p, u);
    const int x = min(lane * 4, DV - 4);
    for (int r = piece + P * warp; r < u.rows; r += P * (tall::THREADS / 32)) {
        const float *row = stage + r * (DV + 4);
        // lane k has the maximum and sum of the k-th piece from this one on
        const int at = piece + min(lane, P - 1);
        const float4 ml = load_cluster(place_in_cta(row + DV, at < P ? at : at - P));
        float4 v[P];
        v[0] = *reinterpret_cast<const float4 *>(row + x);
#pragma unroll
        for (int k = 1; k < P; k++)
            v[k] = load_cluster(place_in_cta(row + x, piece + k < P ? piece + k : piece + k - P));
        float m = ml.x;
#pragma unroll
        for (int k = 1; k < kExpandedMaxPieces; k *= 2)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        m = __shfl_sync(0xffffffffu, m, 0);
        const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; k++) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            l = fmaf(wk, __shfl_sync(0xffffffffu, ml.y, k), l);
            o = make_float4(fmaf(wk, v[k].x, o.x), fmaf(wk, v[k].y, o.y), fmaf(wk, v[k].z, o.z),
                            fmaf(wk, v[k].w, o.w));
        }
        const float inv = l > 0.f ? 1.0f / l : 0.f;
        if (lane * 4 < DV)
            *reinterpret_cast<uint2 *>(out + (size_t)r * p.H * DV + x) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
}

template <int DV>
__device__ __forceinline__ void join_rows(const ExpandedParams &p, const Unit &u, const float *stage,
                                          const int *abort_flag, int piece, int pieces, int warp, int lane)
{
    static_assert(kExpandedMaxPieces == 8, "cases, and lanes with a piece");
    switch (pieces) {
    case 2: return join_rows_of<DV, 2>(p, u, stage, abort_flag, piece, warp, lane);
    case 3: return join_rows_of<DV, 3>(p, u, stage, abort_flag, piece, warp, lane);
    case 4: return join_rows_of<DV, 4>(p, u, stage, abort_flag, piece, warp, lane);
    case 5: return join_rows_of<DV, 5>(p, u, stage, abort_flag, piece, warp, lane);
    case 6: return join_rows_of<DV, 6>(p, u, stage, abort_flag, piece, warp, lane);
    case 7: return join_rows_of<DV, 7>(p, u, stage, abort_flag, piece, warp, lane);
    default: return join_rows_of<DV, 8>(p, u, stage, abort_flag, piece, warp, lane);
    }
}

// Units are handed out in rounds of one per CTA, every other round in reverse, since they come in
// order of decreasing keys.
__device__ __forceinline__ int unit_of_round(int round)
{
    const int at = round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    return round * gridDim.x + at;
}

template <int DN, int DV>
__global__ void __launch_bounds__(tall::THREADS, 1)
    latent_expanded_tall_kernel(const __grid_constant__ ExpandedParams p, const int first_unit,
                                const int units, const int pieces,
                                const __grid_constant__ CUtensorMap map_q,
                                const __grid_constant__ CUtensorMap map_kv,
                                const __grid_constant__ CUtensorMap map_pe)
{
    using namespace tall;
    typedef TallSmem<DN, DV> Smem;
    constexpr int QB = Smem::QB, VB = Smem::VB, PER = Smem::PER, SLOTS = Smem::SLOTS;
    typedef RingAt<SLOTS> At;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 8 * 32) {  // (the producer)
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_kv);
        tc::prefetch_tmap(&map_pe);
        for (int t = 0; t < TILES; t++) {
            mbar_init(&sm.q_full[t], 1);
            mbar_init(&sm.q_empty[t], 1);
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.p_full[t], 4);
            mbar_init(&sm.o_done[t], 1);
            mbar_init(&sm.o_empty[t], 4);
        }
        for (int i = 0; i < SLOTS; i++) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sm.unit_full[i], 1);
            mbar_init(&sm.unit_empty[i], 10);  // the producer, the issuer and the softmax warps
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    grid_dependents_launch();
    const int piece = blockIdx.x % pieces;  // (with pieces a CTA has one unit)
    auto index_of = [&](int round) { return pieces > 1 ? blockIdx.x / pieces : unit_of_round(round); };
    const bool single = pieces > 1 || units <= (int)gridDim.x;  // the CTA has no other unit
    const Unit found = find_unit<UR>(p, first_unit + index_of(0), lane, threadIdx.x == 0);
    const bool begun = found.run && found.k_end > 0;
    if (found.run && !begun && piece == 0)
        store_zeros<DV>(p, found, threadIdx.x, THREADS);
    if (single && !begun)  // (all CTAs of a cluster)
        return;

    // What a piece has of a unit.
    struct Span {
        int first, tiles;  // key tiles; there may be none
        int qt;            // query tiles
        __device__ __forceinline__ Span(const Unit &u, int piece, int pieces)
        {
            const int all = (u.k_end + BN - 1) / BN;
            first = (int)((long long)all * piece / pieces);
            tiles = (int)((long long)all * (piece + 1) / pieces) - first;
            qt = u.rows > BM ? 2 : 1;
        }
    };

    // Column block i of a unit's keys, Q behind the first keys: `item` of the ring.
    auto load_block = [&](const Unit &u, const Span &sp, int i, int item) {
        const At at(item);
        const int c = i % PER, y = u.start + (sp.first + i / PER) * BN;
        uint64_t *bar = &sm.full[at.slot];
        mbar_arrive_expect_tx(bar, BLOCK);
        if (c < QB - 1) {
            tc::tma_load_3d(sm.ring[at.slot], &map_kv, c * 64, u.head, y, bar);
        } else if (c == QB - 1) {
            tc::tma_load_2d(sm.ring[at.slot], &map_pe, 0, y, bar);
        } else {
            // V's blocks at ascending places: where the ring ends between them the first slot
            // takes the first dims
            const bool swapped = VB == 2 && (item - (c - QB)) % SLOTS == SLOTS - 1;
            tc::tma_load_3d(sm.ring[at.slot], &map_kv, DN + (swapped ? 1 - (c - QB) : c - QB) * 64, u.head,
                            y, bar);
        }
    };
    auto load_q = [&](const Unit &u, int t) {
        mbar_arrive_expect_tx(&sm.q_full[t], QB * Q_BLOCK);
        for (int c = 0; c < QB; c++)
            tc::tma_load_3d(sm.q[t][c], &map_q, c * 64, u.head, u.tok0 + u.r0 + t * BM, &sm.q_full[t]);
    };
    // The first unit's: fresh slots need no wait.
    const Span sp0(found, piece, pieces);
    const int early = begun ? min(sp0.tiles * PER, SLOTS) : 0;
    if (threadIdx.x == 8 * 32)
        for (int i = 0; i < early; i++) {
            if (i == QB)
                for (int t = 0; t < sp0.qt; t++)
                    load_q(found, t);
            load_block(found, sp0, i, i);
        }
    if (warp == 9)
        tc::tmem_alloc(&sm.tmem_base, TMEM_COLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    // The CTA's k-th unit: the one found first, then those handed out, if `wait` says they are there.
    // `ok` falls with a wait that gave up; false when there is no other.
    auto next_unit = [&](int k, Unit &u, bool &ok, auto &&wait, bool arrive) {
        if (begun && k == 0) {
            u = found;
            return true;
        }
        if (single)
            return false;
        const int h = k - begun;
        ok = wait(&sm.unit_full[h & 1], (h >> 1) & 1);
        if (!ok)
            return false;
        u = sm.unit[h & 1];
        if (arrive)
            mbar_arrive(&sm.unit_empty[h & 1]);
        return u.rows > 0;
    };
    auto bounded = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_bounded(bar, parity); };

    static_assert(sizeof(float) * UR * (DV + 4) <= sizeof(sm.q) + sizeof(sm.ring),
                  "the rows of a piece are staged over Q, K and V, idle by then");
    float *stage = reinterpret_cast<float *>(&sm.q[0]);

    if (warp == 10 && !single) {
        // --------------------------------------------------------------- units --
        int handed = 0;
        bool ok = true;
        auto hand = [&](const Unit &u) {
            const int i = handed & 1;
            ok = warp_wait(&sm.unit_empty[i], ((handed >> 1) & 1) ^ 1, &sm.abort_flag);
            if (ok && lane == 0) {
                sm.unit[i] = u;
                mbar_arrive(&sm.unit_full[i]);
            }
            handed++;
        };
        for (int round = 1; ok && round * (int)gridDim.x < units; round++) {
            const int index = index_of(round);
            if (index >= units)
                continue;
            const Unit u = find_unit<UR>(p, first_unit + index, lane, lane == 0);
            if (!u.run)
                continue;
            if (u.k_end <= 0) {
                store_zeros<DV>(p, u, lane, 32);
                continue;
            }
            hand(u);
        }
        Unit none{};
        if (ok)
            hand(none);
        if (!ok && lane == 0)
            set_abort(&sm.abort_flag, p.status);
    } else if (warp == 8) {
        // ------------------------------------------------------------ producer --
        if (lane == 0) {
            // loaded so far: column blocks, and Q of the two tiles
            int item = early, queries[2] = {early > 0, early > 0 && sp0.qt > 1};
            bool ok = true;
            Unit u;
            for (int n = 0; ok && next_unit(n, u, ok, bounded, true); n++) {
                const Span sp(u, piece, pieces);
                for (int i = n == 0 ? early : 0; ok && i < sp.tiles * PER; i++, item++) {
                    if (i == QB)
#pragma unroll
                        for (int t = 0; t < TILES; t++)
                            if (t < sp.qt && ok) {
                                ok = mbar_wait_bounded(&sm.q_empty[t], (queries[t] & 1) ^ 1) &&
                                     !aborted(&sm.abort_flag);
                                if (ok) {
                                    load_q(u, t);
                                    queries[t]++;
                                }
                            }
                    const At at(item);
                    ok = ok && mbar_wait_bounded(&sm.empty[at.slot], at.parity ^ 1) && !aborted(&sm.abort_flag);
                    if (!ok)
                        break;
                    load_block(u, sp, i, item);
                }
            }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            // every copy issued lands before the CTA can exit
            for (int t = 0; t < TILES; t++)
                if (queries[t] > 0)
                    drain_wait(&sm.q_full[t], (queries[t] - 1) & 1, p.status);
            for (int i = max(item - SLOTS, 0); i < item; i++)
                drain_wait(&sm.full[At(i).slot], At(i).parity, p.status);
        }
    } else if (warp == 9) {
        // ------------------------------------------------ S = Q K^T and O += P V --
        // One thread issues all products, and the tensor cores take them in that order: S of a
        // tile is written over weights that the product before it has read, and what S's
        // commit tells is also true of that product.
        if (elect_one()) {
            constexpr uint32_t idesc_s = tc::idesc_bf16_f32(BM, BN, false, false);
            constexpr uint32_t idesc_o = tc::idesc_bf16_f32(BM, DV, false, true);
            constexpr uint32_t B16 = BLOCK >> 4;
            const uint64_t qd0 = tc::desc_kmajor_sw128(smem_addr(sm.q[0][0]));
            const uint64_t kd0 = tc::desc_kmajor_sw128(smem_addr(sm.ring[0]));
            bool ok = true, issued = false;
            int base = 0;                        // the unit's first column block in the ring
            int had[2] = {0, 0}, weighed[2] = {0, 0};  // by query tile: units, and products with V
            Unit u;
            for (int n = 0; ok && next_unit(n, u, ok, bounded, true); n++) {
                const Span sp(u, piece, pieces);
                auto scores = [&](int j, int t) {
                    const uint64_t qd = qd0 + (uint64_t)(t * QB * B16);
                    if (j == 0)
                        ok = ok && mbar_wait_bounded(&sm.q_full[t], had[t] & 1);
#pragma unroll
                    for (int c = 0; c < QB; c++) {
                        const At at(base + j * PER + c);
                        if (t == 0)
                            ok = ok && mbar_wait_bounded(&sm.full[at.slot], at.parity);
                        if (!ok)
                            return;
                        if (t == 0 || c == 0)
                            tc::fence_after_sync();
                        const uint64_t kd = kd0 + (uint64_t)(at.slot * B16);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            tc::mma_ss(tmem + t * BN, qd + c * B16 + i * 2, kd + i * 2, idesc_s,
                                       c > 0 || i > 0);
                    }
                    issued = true;
                    tc::mma_commit(&sm.s_full[t]);
                    if (t == sp.qt - 1)
                        for (int c = 0; c < QB; c++)
                            tc::mma_commit(&sm.empty[At(base + j * PER + c).slot]);
                    if (j == sp.tiles - 1)
                        tc::mma_commit(&sm.q_empty[t]);
                };
                for (int t = 0; t < sp.qt && sp.tiles > 0; t++)
                    scores(0, t);
                for (int j = 0; j < sp.tiles && ok; j++) {
                    const At v0(base + j * PER + QB), v1(base + j * PER + PER - 1);
                    const int lo = min(v0.slot, v1.slot), hi = max(v0.slot, v1.slot);
                    const uint64_t vd = tc::desc_mnmajor_sw128(smem_addr(sm.ring[lo]), (hi - lo) * BLOCK);
#pragma unroll
                    for (int t = 0; t < TILES; t++) {
                        if (t >= sp.qt || !ok)
                            break;
                        ok = mbar_wait_bounded(&sm.p_full[t], weighed[t]++ & 1) &&
                             mbar_wait_bounded(&sm.full[v0.slot], v0.parity) &&
                             mbar_wait_bounded(&sm.full[v1.slot], v1.parity);
                        if (ok && j == 0 && had[t] > 0)  // the last unit's rows are out of O
                            ok = mbar_wait_bounded(&sm.o_empty[t], (had[t] - 1) & 1);
                        if (!ok || aborted(&sm.abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
#pragma unroll
                        for (int i = 0; i < BN / 16; i++)  // 16 keys = 16 rows of 128 B per step
                            tc::mma_ts(tmem + O_COL0 + t * DV, tmem + t * BN + i * 8,
                                       vd + (uint64_t)(i * 128), idesc_o, j > 0 || i > 0);
                        if (t == sp.qt - 1)
                            for (int c = 0; c < VB; c++)
                                tc::mma_commit(&sm.empty[At(base + j * PER + QB + c).slot]);
                        if (j + 1 < sp.tiles)
                            scores(j + 1, t);
                        else
                            tc::mma_commit(&sm.o_done[t]);
                    }
                }
                base += sp.tiles * PER;
                if (sp.tiles > 0)
#pragma unroll
                    for (int t = 0; t < TILES; t++)
                        had[t] += t < sp.qt;
            }
            if (!ok)
                set_abort(&sm.abort_flag, p.status);
            if (issued) {  // all issued MMAs complete before tensor memory is released
                tc::mma_commit(&sm.drain);
                drain_wait(&sm.drain, 0, p.status);
            }
        }
    } else if (warp < 8) {
        // -------------------------------------------------------------- softmax --
        const int t = warp / 4, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16, o_t = tmem + O_COL0 + t * DV + lane_off;
        bool ok = true;
        int base = 0, had = 0, weighed = 0;  // as the issuing thread counts them
        auto by_warp = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, &sm.abort_flag); };
        Unit u;
        for (int n = 0; ok && next_unit(n, u, ok, by_warp, false); n++) {
            __syncwarp();
            if (lane == 0 && n >= begun)
                mbar_arrive(&sm.unit_empty[(n - begun) & 1]);
            const Span sp(u, piece, pieces);
            if (t < sp.qt) {
                const int pos_lo = u.pos_lo + t * BM, k_end = min(u.k_end, pos_lo + BM);
                RowState st;
                for (int j = 0; ok && j < sp.tiles; j++) {
                    const int j0 = (sp.first + j) * BN;
                    if (!(ok = warp_wait(&sm.s_full[t], weighed++ & 1, &sm.abort_flag)))
                        break;
                    tc::fence_after_sync();
                    float alpha;
                    const bool corr = weigh_tile<BN / 32>(tmem + t * BN + lane_off, j0, pos_lo, pos_lo + r,
                                                          k_end, p.scale_log2, st, alpha);
                    if (t == 0 && j0 + BN > u.k_end) {  // rows behind the last visible key may hold any bits
                        for (int c = 0; c < VB; c++) {
                            const At at(base + j * PER + QB + c);
                            ok = ok && warp_wait(&sm.full[at.slot], at.parity, &sm.abort_flag);
                            if (ok && r >= u.k_end - j0)
                                zero_row(sm.ring[at.slot], r);
                        }
                        if (!ok)
                            break;
                        tc::fence_proxy_async_smem();
                    }
                    if (__any_sync(0xffffffffu, corr))  // (O holds all of the tiles before)
                        rescale_rows<DV>(o_t, corr ? alpha : 1.f);
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm.p_full[t]);
                }
                if (pieces == 1) {
                    if (!ok || !(ok = warp_wait(&sm.o_done[t], had & 1, &sm.abort_flag)))
                        break;
                    tc::fence_after_sync();
                    uint32_t o[DV / 32][32];
#pragma unroll
                    for (int c = 0; c < DV / 32; c++)
                        tc::tmem_ld32(o_t + c * 32, o[c]);
                    tc::tmem_wait_ld();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm.o_empty[t]);
                    if (t * BM + r < u.rows) {
                        const float inv = st.l > 0.f ? 1.0f / st.l : 0.f;
                        uint4 *row = reinterpret_cast<uint4 *>(rows_out<DV>(p, u) + (size_t)(t * BM + r) * p.H * DV);
#pragma unroll
                        for (int c = 0; c < DV / 8; c++) {
                            const uint32_t *x = &o[c / 4][c % 4 * 8];
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                w[i] = pack_bf16x2(__uint_as_float(x[2 * i]) * inv,
                                                   __uint_as_float(x[2 * i + 1]) * inv);
                            row[c] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                } else {
                    // the row unnormalised, its maximum and sum in the padding
                    float *rows = stage + t * BM * (DV + 4);
                    if (sp.tiles == 0) {
                        for (int c = 0; c < DV; c += 4)
                            *reinterpret_cast<float4 *>(rows + r * (DV + 4) + c) =
                                make_float4(0.f, 0.f, 0.f, 0.f);
                    } else {
                        for (int i = 0; i < sp.qt; i++)  // all products are done with what lies there
                            ok = ok && warp_wait(&sm.o_done[i], 0, &sm.abort_flag);
                        if (!ok)
                            break;
                        tc::fence_after_sync();
                        stage_row<DV>(o_t, 1.f, rows, r);
                    }
                    *reinterpret_cast<float2 *>(rows + r * (DV + 4) + DV) = make_float2(st.m_ref, st.l);
                }
                had++;
            }
            base += sp.tiles * PER;
        }
        if (!ok && lane == 0)
            set_abort(&sm.abort_flag, p.status);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (pieces > 1) {
        cluster_sync();
        join_rows<DV>(p, found, stage, &sm.abort_flag, piece, pieces, warp, lane);
        cluster_sync();  // until then the other CTAs read this one's rows
    }
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------------- launches --

// Tensor maps of the queries, of kv's rows (boxes of 64 columns, `keys` rows of one head) and of
// the shared part.
bool make_maps(const ExpandedParams &p, int keys, CUtensorMap *mq, CUtensorMap *mkv, CUtensorMap *mpe)
{
    const cuuint64_t qw = p.dn + p.rd, kw = p.dn + p.dv, H = p.H;
    const cuuint64_t q_dims[3] = {qw, H, (cuuint64_t)p.total_tokens};
    const cuuint64_t q_strides[2] = {qw * 2, H * qw * 2};
    const cuuint64_t kv_dims[3] = {kw, H, (cuuint64_t)p.total_keys};
    const cuuint64_t kv_strides[2] = {kw * 2, H * kw * 2};
    const cuuint64_t pe_dims[2] = {(cuuint64_t)p.rd, (cuuint64_t)p.total_keys};
    const cuuint64_t pe_strides[1] = {(cuuint64_t)p.k_pe_stride * 2};
    const cuuint32_t rows = (cuuint32_t)keys;
    const cuuint32_t q_box[3] = {64, 1, BM}, kv_box[3] = {64, 1, rows}, pe_box[2] = {64, rows};
    return make_bf16_tile_map(mq, p.q, 3, q_dims, q_strides, q_box) &&
           make_bf16_tile_map(mkv, p.kv, 3, kv_dims, kv_strides, kv_box) &&
           make_bf16_tile_map(mpe, p.k_pe, 2, pe_dims, pe_strides, pe_box);
}

template <int DN, int DV>
cudaError_t launch_expanded_t(const ExpandedParams &p, cudaStream_t stream)
{
    CUtensorMap mq, mkv, mpe;
    if (!make_maps(p, two::BN, &mq, &mkv, &mpe))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(ExpandedSmem<DN, DV>);
    static_assert(2 * (smem + 1024) <= 233472, "shared memory of two CTAs per SM");
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = once_per_device(configured, [] {
        return cudaFuncSetAttribute(latent_expanded_kernel<DN, DV>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    return launch_kernel(latent_expanded_kernel<DN, DV>, dim3((unsigned)p.units),
                         dim3(two::THREADS), smem, stream, p, mq, mkv, mpe);
}

template <int DN, int DV>
cudaError_t configure_tall()
{
    constexpr size_t smem = sizeof(TallSmem<DN, DV>);
    static_assert(smem > (116u << 10) && smem <= 232448, "shared memory of one CTA per SM");
    static std::atomic<unsigned long long> configured{0};
    return once_per_device(configured, [] {
        return cudaFuncSetAttribute(latent_expanded_tall_kernel<DN, DV>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
}

template <int DN, int DV>
cudaError_t launch_tall_t(const ExpandedParams &p, cudaStream_t stream)
{
    using namespace tall;
    CUtensorMap mq, mkv, mpe;
    if (!make_maps(p, BN, &mq, &mkv, &mpe))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(TallSmem<DN, DV>);
    cudaError_t e = configure_tall<DN, DV>();
    if (e != cudaSuccess)
        return e;
    const int whole = p.units - p.cut_units;
    if (whole > 0) {
        e = launch_kernel(latent_expanded_tall_kernel<DN, DV>, dim3((unsigned)(p.in_turn ? std::min(whole, p.sms) : whole)),
                          dim3(THREADS), smem, stream, p, 0, whole, 1, mq, mkv, mpe);
        if (e != cudaSuccess)
            return e;
    }
    if (p.cut_units > 0)
        e = launch_kernel_cluster(latent_expanded_tall_kernel<DN, DV>, dim3((unsigned)(p.cut_units * p.pieces)),
                                  dim3(THREADS), smem, p.pieces, stream, p, whole, p.cut_units, p.pieces, mq, mkv,
                                  mpe);
    return e;
}

}  // namespace

int sm_clusters(int ctas)
{
    // (any kernel with one CTA per SM will do)
    static std::atomic<int> cached[kMaxDevices][kExpandedMaxPieces + 1];
    const int dev = current_device_index();
    int n = dev >= 0 ? cached[dev][ctas].load(std::memory_order_relaxed) : 0;
    if (n > 0)
        return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * 64));
    cfg.blockDim = dim3(tall::THREADS);
    cfg.dynamicSmemBytes = sizeof(TallSmem<128, 128>);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (configure_tall<128, 128>() != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, latent_expanded_tall_kernel<128, 128>, &cfg) != cudaSuccess)
        return 0;  // (nothing is cut then)
    if (dev >= 0)
        cached[dev][ctas].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_latent_expanded(const ExpandedParams &p, cudaStream_t stream)
{
    if (p.tall) {
        if (p.dn == 128)
            return p.dv == 128 ? launch_tall_t<128, 128>(p, stream) : launch_tall_t<128, 64>(p, stream);
        return p.dv == 128 ? launch_tall_t<64, 128>(p, stream) : launch_tall_t<64, 64>(p, stream);
    }
    if (p.dn == 128)
        return p.dv == 128 ? launch_expanded_t<128, 128>(p, stream) : launch_expanded_t<128, 64>(p, stream);
    return p.dv == 128 ? launch_expanded_t<64, 128>(p, stream) : launch_expanded_t<64, 64>(p, stream);
}
