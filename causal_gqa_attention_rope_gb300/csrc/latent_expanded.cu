// latent_expanded.cu -- expanded latent attention (na_attn_latent_expanded): causal
// attention of nope_dim + rope_dim and v_dim, on the sm_100-family tensor cores
// (tcgen05 + TMEM + TMA).
//
// The pipeline of prefill.cu with other operands.  A CTA owns 128 query tokens of one
// head and walks the 128-key tiles that they see: S = Q K^T with K of dn + 64
// columns -- the head's own dn out of kv's rows and the rotated part that all heads
// share, padded by TMA's zeros to a column block -- then O += P V.  Keys and values
// are read where the expanding product left them, so nothing is concatenated.
//
// Warps: 0 producer, 1 issues S into one of three buffers, 2 issues O (P in tensor
// memory, over its S), 4 .. 7 softmax, a row per thread; all eight store the rows.
#include <climits>

#include "latent.cuh"
#include "tc_primitives.cuh"
#include "tile_waits.cuh"

namespace {

constexpr int BM = kExpandedRows, BN = 128;
constexpr int THREADS = 256;
constexpr int NUM_S = 3;
constexpr uint32_t S_COL0 = 128;  // S buffer i at columns 128 (i + 1); O at column 0
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t BLOCK_BYTES = 128 * 128;  // 128 rows of 64 bf16

template <int DN, int DV>
struct __align__(1024) ExpandedSmem {
    static constexpr int QB = DN / 64 + 1, VB = DV / 64;  // column blocks
    static constexpr int STAGES = DN + DV == 128 ? 3 : 2;
    bf16 q[QB][BM * 64];
    bf16 k[STAGES][QB][BN * 64];
    bf16 v[STAGES][VB][BN * 64];
    uint64_t q_full, k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
    uint64_t s_full[NUM_S], s_free[NUM_S], p_full[NUM_S], o_done[NUM_S], drain[2];
    uint32_t tmem_base;
    int abort_flag;
};

template <int DN, int DV>
__global__ void __launch_bounds__(THREADS, 1)
    latent_expanded_kernel(const __grid_constant__ ExpandedParams p,
                           const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_kv,
                           const __grid_constant__ CUtensorMap map_pe)
{
    typedef ExpandedSmem<DN, DV> Smem;
    constexpr int QB = Smem::QB, VB = Smem::VB, STAGES = Smem::STAGES;
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_kv);
        tc::prefetch_tmap(&map_pe);
        mbar_init(&sm.q_full, 1);
        for (int i = 0; i < STAGES; i++) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
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

    // Unit: query tile (the last ones, which see most keys, first), head, sequence; up to
    // 32 sequences in order of decreasing keys, so that the longest units start first.
    const int unit = blockIdx.x;
    const int qt = p.q_tiles - 1 - unit % p.q_tiles;
    const int head = unit / p.q_tiles % p.H;
    int b = unit / (p.q_tiles * p.H);
    if (p.batch > 1 && p.batch <= 32) {
        const int key = lane < p.batch ? __ldg(p.key_lens + lane) : INT_MIN;
        int rank = 0;
        for (int i = 0; i < p.batch; i++) {
            const int other = __shfl_sync(0xffffffffu, key, i);
            rank += other > key || (other == key && i < lane);
        }
        b = __ffs(__ballot_sync(0xffffffffu, lane < p.batch && rank == b)) - 1;
    }
    const int tok0 = __ldg(p.cu_seqlens + b), n = __ldg(p.cu_seqlens + b + 1) - tok0;
    const int start = __ldg(p.key_starts + b), keys = __ldg(p.key_lens + b);
    const int r0 = qt * BM;
    if (n > p.max_new_len || tok0 < 0 || (b == 0 && tok0 != 0) || (long long)tok0 + n > p.total_tokens) {
        if (qt == 0 && head == 0 && threadIdx.x == 0)
            na_report(p.status, NA_ERR_INVALID_ARG);
        return;
    }
    if (r0 >= n)
        return;
    if (keys < 0 || start < 0 || keys > p.max_key_len || (long long)start + keys > p.total_keys) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_CAPACITY);
        return;
    }
    const int rows = min(BM, n - r0);
    const int pos_lo = keys - n + r0;          // position of row 0; may be negative
    const int k_end = pos_lo + rows;           // keys that the last row sees
    bf16 *out = p.out + ((size_t)(tok0 + r0) * p.H + head) * DV;
    if (k_end <= 0) {                          // no row sees a key
        for (int i = threadIdx.x; i < rows * (DV / 8); i += THREADS)
            *reinterpret_cast<uint4 *>(out + (size_t)(i / (DV / 8)) * p.H * DV + i % (DV / 8) * 8) =
                make_uint4(0, 0, 0, 0);
        return;
    }
    const int n_tiles = (k_end + BN - 1) / BN;
    auto load_k = [&](int j) {
        const int st = j % STAGES;
        mbar_arrive_expect_tx(&sm.k_full[st], QB * BLOCK_BYTES);
        for (int c = 0; c < QB - 1; c++)
            tc::tma_load_3d(sm.k[st][c], &map_kv, c * 64, head, start + j * BN, &sm.k_full[st]);
        tc::tma_load_2d(sm.k[st][QB - 1], &map_pe, 0, start + j * BN, &sm.k_full[st]);
    };
    auto load_v = [&](int j) {
        const int st = j % STAGES;
        mbar_arrive_expect_tx(&sm.v_full[st], VB * BLOCK_BYTES);
        for (int c = 0; c < VB; c++)
            tc::tma_load_3d(sm.v[st][c], &map_kv, DN + c * 64, head, start + j * BN, &sm.v_full[st]);
    };
    const int pre = min(n_tiles, STAGES);
    if (threadIdx.x == 0) {  // (fresh stages need no wait)
        mbar_arrive_expect_tx(&sm.q_full, QB * BLOCK_BYTES);
        for (int c = 0; c < QB; c++)
            tc::tma_load_3d(sm.q[c], &map_q, c * 64, head, tok0 + r0, &sm.q_full);
        for (int j = 0; j < pre; j++) {
            load_k(j);
            load_v(j);
        }
    }
    if (warp == 1)
        tc::tmem_alloc(&sm.tmem_base, TMEM_COLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;

    constexpr int LDS = DV + 4;  // staged row stride (floats): conflict-free row writes
    static_assert(sizeof(float) * BM * LDS <= sizeof(sm.k) + sizeof(sm.v),
                  "the rows are staged in the K ring and what follows, idle by then");
    float *stage = reinterpret_cast<float *>(&sm.k[0]);

    if (warp == 0) {
        // ------------------------------------------------------------ producer --
        if (lane == 0) {
            int issued = pre;
            for (int j = pre; j < n_tiles; j++) {
                const int st = j % STAGES;
                const uint32_t par = ((j / STAGES) & 1) ^ 1;
                if (!mbar_wait_bounded(&sm.k_empty[st], par) || aborted(&sm.abort_flag)) {
                    set_abort(&sm.abort_flag, p.status);
                    break;
                }
                load_k(j);
                if (!mbar_wait_bounded(&sm.v_empty[st], par) || aborted(&sm.abort_flag)) {
                    set_abort(&sm.abort_flag, p.status);
                    drain_wait(&sm.k_full[st], (j / STAGES) & 1, p.status);
                    break;
                }
                load_v(j);
                issued = j + 1;
            }
            // every copy issued lands before the CTA can exit
            drain_wait(&sm.q_full, 0, p.status);
            for (int j = issued - 1; j >= 0 && j >= issued - STAGES; j--) {
                drain_wait(&sm.k_full[j % STAGES], (j / STAGES) & 1, p.status);
                drain_wait(&sm.v_full[j % STAGES], (j / STAGES) & 1, p.status);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- S = Q K^T issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(BM, BN, false, false);
            constexpr uint32_t BLOCK16 = BLOCK_BYTES >> 4;
            const uint64_t qd = tc::desc_kmajor_sw128(smem_addr(sm.q[0]));
            const uint64_t kd0 = tc::desc_kmajor_sw128(smem_addr(sm.k[0][0]));
            bool ok = mbar_wait_bounded(&sm.q_full, 0), any = false;
            for (int j = 0; ok && j < n_tiles; j++) {
                const int st = j % STAGES, sb = j % NUM_S;
                ok = mbar_wait_bounded(&sm.k_full[st], (j / STAGES) & 1);
                if (ok && j >= NUM_S)
                    ok = mbar_wait_bounded(&sm.s_free[sb], ((j / NUM_S) - 1) & 1);
                if (!ok || aborted(&sm.abort_flag))
                    break;
                tc::fence_after_sync();
                const uint32_t s_t = tmem + S_COL0 * (sb + 1);
                const uint64_t kd = kd0 + (uint64_t)(st * QB * BLOCK16);
#pragma unroll
                for (int k = 0; k < QB * 4; k++) {
                    const uint32_t off = (k >> 2) * BLOCK16 + (k & 3) * 2;
                    tc::mma_ss(s_t, qd + off, kd + off, idesc, k > 0);
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
        // --------------------------------------------------------- O += P V issue --
        if (elect_one()) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(BM, DV, false, true);
            constexpr uint32_t BLOCK16 = BLOCK_BYTES >> 4;
            const uint64_t vd0 = tc::desc_mnmajor_sw128(smem_addr(sm.v[0][0]), BLOCK_BYTES);
            bool ok = true, any = false;
            for (int j = 0; ok && j < n_tiles; j++) {
                const int st = j % STAGES, sb = j % NUM_S;
                ok = mbar_wait_bounded(&sm.p_full[sb], (j / NUM_S) & 1) &&
                     mbar_wait_bounded(&sm.v_full[st], (j / STAGES) & 1);
                if (!ok || aborted(&sm.abort_flag))
                    break;
                tc::fence_after_sync();
                const uint32_t p_t = tmem + S_COL0 * (sb + 1);
                const uint64_t vd = vd0 + (uint64_t)(st * VB * BLOCK16);
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
        const int row_pos = pos_lo + r;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16, o_t = tmem + lane_off;
        const float sl2 = p.scale_log2;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; ok && j < n_tiles; j++) {
            const int sb = j % NUM_S, j0 = j * BN;
            const uint32_t s_t = tmem + S_COL0 * (sb + 1) + lane_off;
            if (!(ok = warp_wait(&sm.s_full[sb], (j / NUM_S) & 1, &sm.abort_flag)))
                break;
            tc::fence_after_sync();
            uint32_t sr[4][32];
#pragma unroll
            for (int c = 0; c < 4; c++)
                tc::tmem_ld32(s_t + c * 32, sr[c]);
            tc::tmem_wait_ld();
            if (j0 + BN - 1 > pos_lo) {  // (rows see keys up to their position, < k_end)
#pragma unroll
                for (int c = 0; c < 4; c++)
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const int key = j0 + c * 32 + i;
                        if (key > row_pos || key >= k_end)
                            sr[c][i] = __float_as_uint(-INFINITY);
                    }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; c++)
#pragma unroll
                for (int i = 0; i < 32; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        mx[k] = max3f(mx[k], __uint_as_float(sr[c][i + 2 * k]),
                                      __uint_as_float(sr[c][i + 2 * k + 1]));
            const float mxs = max3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * sl2;
            float alpha = 1.f;
            bool corr = false;
            if (mxs > m_ref + 8.0f) {
                alpha = m_ref == -INFINITY ? 0.f : ex2_mufu(m_ref - mxs);
                corr = m_ref != -INFINITY;
                m_ref = mxs;
            }
            const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; c++) {
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
            const float rs = (a01.x + a01.y) + (a23.x + a23.y);
            tc::tmem_wait_st();
            if (j0 + BN > k_end) {
                // Rows behind the last visible key may hold any bits: zeros, so that no weight of
                // 0 meets a NaN.
                const int st = j % STAGES;
                if (!(ok = warp_wait(&sm.v_full[st], (j / STAGES) & 1, &sm.abort_flag)))
                    break;
                if (r >= k_end - j0) {
#pragma unroll
                    for (int c = 0; c < VB; c++) {
                        uint4 *row = reinterpret_cast<uint4 *>(sm.v[st][c] + r * 64);
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            row[i] = make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_proxy_async_smem();
            }
            if (j >= 1 && __any_sync(0xffffffffu, corr)) {
                // O is touched only to rescale it, and then PV(j - 1) has to have landed (its
                // barrier's phase is exact however rarely it is looked at: S(j) could not be
                // issued before PV(j - NUM_S), and PV(j - 1 + NUM_S) needs a P not yet written)
                if (!(ok = warp_wait(&sm.o_done[(j - 1) % NUM_S], ((j - 1) / NUM_S) & 1, &sm.abort_flag)))
                    break;
                tc::fence_after_sync();
                const float a = corr ? alpha : 1.f;
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
            l = l * alpha + rs;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.p_full[sb]);
        }
        if (ok && warp_wait(&sm.o_done[(n_tiles - 1) % NUM_S], ((n_tiles - 1) / NUM_S) & 1,
                            &sm.abort_flag)) {
            tc::fence_after_sync();
            const float scale = l > 0.f ? 1.0f / l : 0.f;
            uint32_t o[DV / 32][32];
#pragma unroll
            for (int c = 0; c < DV / 32; c++)
                tc::tmem_ld32(o_t + c * 32, o[c]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < DV / 32; c++) {
                float4 *row = reinterpret_cast<float4 *>(stage + r * LDS + c * 32);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    row[i] = make_float4(__uint_as_float(o[c][4 * i]) * scale,
                                         __uint_as_float(o[c][4 * i + 1]) * scale,
                                         __uint_as_float(o[c][4 * i + 2]) * scale,
                                         __uint_as_float(o[c][4 * i + 3]) * scale);
            }
        } else if (lane == 0) {
            set_abort(&sm.abort_flag, p.status);
        }
    }
    tc::fence_before_sync();
    __syncthreads();  // the staged rows are complete (unless a wait gave up)
    if (!aborted(&sm.abort_flag)) {
        constexpr int EPL = DV / 32;  // elements per lane, a row per instruction
        for (int r = warp; r < rows; r += THREADS / 32) {
            const float *src = stage + r * LDS + lane * EPL;
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
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int DN, int DV>
cudaError_t launch_expanded_t(const ExpandedParams &p, cudaStream_t stream)
{
    CUtensorMap mq, mkv, mpe;
    const cuuint64_t qw = DN + p.rd, kw = DN + DV, H = p.H;
    const cuuint64_t q_dims[3] = {qw, H, (cuuint64_t)p.total_tokens};
    const cuuint64_t q_strides[2] = {qw * 2, H * qw * 2};
    const cuuint64_t kv_dims[3] = {kw, H, (cuuint64_t)p.total_keys};
    const cuuint64_t kv_strides[2] = {kw * 2, H * kw * 2};
    const cuuint64_t pe_dims[2] = {(cuuint64_t)p.rd, (cuuint64_t)p.total_keys};
    const cuuint64_t pe_strides[1] = {(cuuint64_t)p.k_pe_stride * 2};
    const cuuint32_t box3[3] = {64, 1, 128}, box2[2] = {64, 128};
    if (!make_bf16_tile_map(&mq, p.q, 3, q_dims, q_strides, box3) ||
        !make_bf16_tile_map(&mkv, p.kv, 3, kv_dims, kv_strides, box3) ||
        !make_bf16_tile_map(&mpe, p.k_pe, 2, pe_dims, pe_strides, box2))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(ExpandedSmem<DN, DV>) + 1024;
    static_assert(smem > (116u << 10) && smem <= 232448, "shared memory of one CTA per SM");
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = once_per_device(configured, [] {
        return cudaFuncSetAttribute(latent_expanded_kernel<DN, DV>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    return launch_kernel(latent_expanded_kernel<DN, DV>, dim3((unsigned)(p.q_tiles * p.H * p.batch)),
                         dim3(THREADS), smem, stream, p, mq, mkv, mpe);
}

}  // namespace

cudaError_t launch_latent_expanded(const ExpandedParams &p, cudaStream_t stream)
{
    if (p.dn == 128)
        return p.dv == 128 ? launch_expanded_t<128, 128>(p, stream) : launch_expanded_t<128, 64>(p, stream);
    return p.dv == 128 ? launch_expanded_t<64, 128>(p, stream) : launch_expanded_t<64, 64>(p, stream);
}
