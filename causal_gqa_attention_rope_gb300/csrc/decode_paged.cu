// decode_paged.cu -- the split pass of the single-token decode over a paged
// cache (na_attn_decode_paged).  The arithmetic, the cut of the keys into equal
// slices and the merge pass are those of the contiguous cache (decode.cu,
// decode_shared.cuh); here a tile of keys is gathered from pages, and pages may
// hold E4M3 with one power-of-two scale per (page, kv head).
//
// Per key a kv head reads 2 d s bytes (s = 1 or 2) for 4 HPC d multiply-adds,
// HPC <= 8 query heads at a time: the pass is bound by HBM, and what it has to
// avoid is spending more time on instructions than the bytes take.
//
// The producer warp keeps the page ids (and scales) of 32 pages at a time in
// registers, one page per lane, the next windows' loading meanwhile; each lane
// then issues one box of a tile: a page's rows, or 64 of them, by 128 bytes.  A
// tile is 64 keys aligned to 64 positions, so a box never leaves its page and the
// 16 keys of a consumer warp always share one page, hence one scale pair, which
// the producer hands over with the tile.
//
// E4M3 pages: the bytes become exact f16 values in registers (two conversions a
// word; as bf16 they take nine integer instructions: 171 us for 64 sequences of
// 512 .. 8192 keys, 32/8 heads, d 128, against 167 us at that step), and both
// products run on f16 MMAs.  A word holds four consecutive d of one key
// (K) or two d of two keys (V, loaded transposed as 16-bit pairs), so its f16
// pairs are two d of one key: for the scores they are taken as they are, Q
// permuted to match; for V two byte permutes ahead of the conversion pair the
// keys, and the output rows come out as even and odd d.  A query is scaled by
// a power of two to f16's range (exact for every element that matters: down to
// 2^-26 of the largest, within 2^-33 of it below); K's scale multiplies the
// scores in fp32 and V's enters the weights (na_internal.cuh), which have f16's
// 11 significand bits.
#include <type_traits>

#include "decode_shared.cuh"
#include "na_internal.cuh"
#include "tc_primitives.cuh"

namespace {

using namespace dec;

constexpr int TILE = 64;   // keys per tile: CWARPS warps x 16 keys
constexpr int CWARPS = 4;  // consumer warps
constexpr int THREADS = (CWARPS + 1) * 32;
constexpr int MAX_HPC = 8;
constexpr int MAX_CLUSTER = 8;  // CTAs of a cluster, at most (the portable size)

// Tiles in flight and CTAs per SM.  An E4M3 tile is half as large, and what its
// pass lacks first is warps (64 sequences of 512 .. 8192 keys, 32/8 heads: two
// CTAs of four or six tiles 106 us, three of three 100 us).
constexpr int kStages = 3;
template <bool E4M3>
constexpr int kCtasPerSm = E4M3 ? 3 : 2;

// What a piece costs a CTA besides its keys -- its queries, the merge of the warps
// -- in keys: a slice of many short streams gets that much less of them.  (64
// sequences of 512 .. 8192 keys, 32/8 heads: E4M3 with probabilities 119.8 us at 0,
// 114.2 at 128, 113.8 at 256, 114.5 at 384; bf16 171.1 at 0, 169.1 at 64, 168.1 at
// 128 and at 256.)
template <bool E4M3>
constexpr int kPieceCost = E4M3 ? 256 : 128;

template <int D, bool E4M3>
struct __align__(1024) PagedSmem {
    static constexpr int ST = kStages;
    static constexpr uint32_t ROW = D * (E4M3 ? 1 : 2);           // bytes of a row
    static constexpr uint32_t BOX = ROW < 128 ? ROW : 128;        // of a row in one box
    static constexpr uint32_t TILE_BYTES = TILE * ROW;
    uint8_t k[ST][TILE_BYTES];
    uint8_t v[ST][TILE_BYTES];
    // partial results on their way to another warp: [output quads, (max, sum)][lane]
    float4 merge[CWARPS - 1][D / 16 + 1][32];
    uint16_t scales[ST][CWARPS];  // a warp's K | V << 8 scale bytes in each stage (E4M3)
    uint64_t full[ST];
    uint64_t empty[ST];
    float2 fin[MAX_HPC];  // a finished stream's reference and 1 / sum, per head
    Slice slice;
    int abort_flag, cluster_bad;
};

// Byte offset, within a tile of K or V, of 16-byte chunk c of row r, as the
// swizzled boxes leave it: 128-byte box rows (chunk ^ row % 8), or 64-byte ones
// (chunk ^ (row / 2) % 4).
template <uint32_t ROW>
__device__ __forceinline__ uint32_t chunk_off(int r, int c)
{
    if constexpr (ROW == 64)
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    else
        return (uint32_t)((c >> 3) * (TILE * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The page windows that the producer walks: 32 consecutive pages of a piece,
// one per lane, piece after piece.  A second walker runs ahead of the tiles, so
// that a window's ids are requested two windows early and its scales one: the
// producer never waits for a load it has just issued, but at its start.
struct WindowIds {
    int id;       // this lane's page, as the table has it (in flight)
    bool wanted;  // the page holds keys of the piece
    int wb, kvh;  // the window's first page; the piece's kv head
};

struct Window {
    int id;           // this lane's page (-1: not wanted)
    uint32_t ks, vs;  // the scale bytes of its K and V (in flight at first)
    int wb;
};

template <int COST>
struct WindowIter {
    Walker<COST> walk;
    Piece pc;
    int wb, p_lo, p_hi;  // the window's first page, the piece's first and last
    bool valid;

    __device__ __forceinline__ void start(const Slice &sl, const DecodeParams &p)
    {
        walk.init(sl, p);
        wb = 0;
        p_hi = -1;
        valid = true;
    }

    template <int TILE>
    __device__ __forceinline__ WindowIds next(const DecodeParams &p, const PagedView &pg, int lane)
    {
        wb += 32;
        if (valid && wb > p_hi && (valid = walk.next(p, pc))) {
            const int lo = pc.kf + pc.k0;
            wb = (lo / TILE * TILE) >> pg.page_log;
            p_lo = lo >> pg.page_log;
            p_hi = (pc.kf + pc.k1 - 1) >> pg.page_log;
        }
        const int i = wb + lane;
        WindowIds w{0, valid && i >= p_lo && i <= p_hi, wb, pc.kvh};
        if (w.wanted)
            w.id = __ldcg(pg.table + (size_t)pc.b * pg.pages_per_seq + i);
        return w;
    }
};

// A window's ids checked (one outside the cache is reported, and page 0 read
// instead) and its scales requested.
template <bool E4M3>
__device__ __forceinline__ Window open_window(const DecodeParams &p, const PagedView &pg,
                                              const WindowIds &ids)
{
    Window w{-1, 127u, 127u, ids.wb};
    if (ids.wanted) {
        w.id = ids.id;
        if ((unsigned)w.id >= (unsigned)pg.num_pages) {
            na_report(p.status, NA_ERR_PAGE);
            w.id = 0;
        }
        if constexpr (E4M3) {
            w.ks = __ldcg(pg.k_scale + (size_t)w.id * p.KV + ids.kvh);
            w.vs = __ldcg(pg.v_scale + (size_t)w.id * p.KV + ids.kvh);
        }
    }
    return w;
}

// This thread's lane of a partial in CTA `rank` of the cluster.
__device__ __forceinline__ float4 cluster_load(const float4 *p, int rank)
{
    uint32_t a;
    float4 x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(a)
                 : "memory");
    return x;
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A stream that a cluster of C CTAs (one, or up to MAX_CLUSTER) has read whole, by
// the NT consumer threads of each: warp 0 holds the merged rows' d-blocks s = rank
// mod C and writes them (gated); then the raw scores of this CTA's keys become
// probabilities.  `bad`: a wait gave up; the rows are zero.
template <int D, bool E4M3, int NT>
__device__ __forceinline__ void finish_stream(const DecodeParams &p, const Piece &pc, float2 *fin,
                                              int head0, int hpc, const float (&acc)[D / 16][4],
                                              const float (&m_ref)[2], const float (&l_sum)[2],
                                              bool bad, int rank, int C)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const size_t row0 = (size_t)pc.b * p.H + head0;
    if (threadIdx.x < 32) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int h = 2 * t + i;
            if (h >= hpc)
                break;
            const float inv = l_sum[i] > 0.f && !bad ? 1.0f / l_sum[i] : 0.f;
            if (g == 0)
                fin[h] = make_float2(m_ref[i], inv);
            const bf16 *gate = p.gate ? p.gate + (row0 + h) * D : nullptr;
            bf16 *out = p.out + (row0 + h) * D;
            auto value = [&](float o, int e) {
                o = bad ? 0.f : o * inv;
                return gate ? o * (1.0f / (1.0f + __expf(-__bfloat162float(gate[e])))) : o;
            };
#pragma unroll
            for (int s = 0; s < D / 16; s++) {
                if ((s & (C - 1)) != rank)
                    continue;
                if constexpr (E4M3) {
                    const int e = 16 * s + 2 * g;
                    *reinterpret_cast<uint32_t *>(out + e) =
                        pack_bf16x2(value(acc[s][i], e), value(acc[s][2 + i], e + 1));
                } else {
                    const int e = 16 * s + g;
                    out[e] = __float2bfloat16_rn(value(acc[s][i], e));
                    out[e + 8] = __float2bfloat16_rn(value(acc[s][2 + i], e + 8));
                }
            }
        }
    }
    if (!p.probs)
        return;
    named_barrier_sync(1, NT);
    if (bad)
        return;
    // keys before the window (none without one) get 0, from the first CTA
    const int j0 = rank == 0 ? 0 : pc.kf + pc.k0, n = pc.kf + pc.k1;
    for (int h = 0; h < hpc; h++) {
        float *row = p.probs + (row0 + h) * p.probs_stride;
        const float2 f = fin[h];
        for (int j = j0 + threadIdx.x; j < n; j += NT)
            row[j] = j < pc.kf ? 0.f : ex2_mufu(row[j] - f.x) * f.y;
    }
}

// Short streams are not cut over the whole grid: SPLIT is the slice of the
// concatenation and a merge pass behind it, DIRECT one CTA per stream, CLUSTER
// p.direct CTAs per stream, neighbouring tiles each, whose partials meet through
// shared memory: no partial results in the workspace and no merge pass.
enum Mode { SPLIT, DIRECT, CLUSTER };

template <int D, bool E4M3, bool CAPPED, Mode MODE>
__global__ void __launch_bounds__(THREADS, kCtasPerSm<E4M3>)
    decode_paged_kernel(const DecodeParams p, const PagedView pg,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v)
{
    typedef PagedSmem<D, E4M3> Smem;
    constexpr int ST = Smem::ST;
    constexpr int KS = D / 16;  // k-steps of the score MMA, d-blocks of the PV MMA
    constexpr uint32_t ROW = Smem::ROW, STAGE_BYTES = Smem::TILE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned FULL = 0xffffffffu;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], CWARPS);
        }
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == CWARPS && lane == 0) {
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
    }
    grid_dependency_wait();
    grid_dependents_launch();
    const int C = MODE == CLUSTER ? p.direct : 1;  // CTAs of a stream, and this one's number
    const int rank = blockIdx.x & (C - 1);
    if constexpr (MODE != SPLIT) {  // this CTA's stream, all of it or its share of the tiles
        if (threadIdx.x == 0) {
            const int spb = p.KV * p.head_chunks, st = blockIdx.x / C, b = st / spb;
            int kf;
            const int len = attended_keys(p, b, kf);
            long long start = 0, end = len;
            if constexpr (MODE == CLUSTER) {
                const int t0 = kf / TILE, share = (kf + len - t0 * TILE + TILE * C - 1) / (TILE * C);
                const int lo = (t0 + rank * share) * TILE - kf;
                start = max(0, lo);
                end = min(len, lo + share * TILE);
            }
            constexpr int COST = kPieceCost<E4M3>;
            sm.slice = Slice{start + COST, end + COST, 0, b, st - b * spb, start >= end};
        }
    } else if (warp == CWARPS) {
        locate_slice<kPieceCost<E4M3>>(p, lane, sm.slice);
    }
    __syncthreads();
    Walker<kPieceCost<E4M3>> walk;
    walk.init(sm.slice, p);
    Piece pc;

    // A piece's keys are positions [kf + k0, kf + k1); its tiles are the
    // TILE-aligned position ranges covering them, and keys of a tile outside
    // the piece are masked.
    if (warp == CWARPS) {
        // ---------------------------------------------------------- producer --
        const uint64_t policy = l2_policy_evict_first();  // K/V lines are read once
        const int page = 1 << pg.page_log;
        const int box_log = min(pg.page_log, 6), nbox = TILE >> box_log;
        constexpr int COLS = (int)(ROW / Smem::BOX);  // boxes side by side in a row
        // this lane's box of a tile: rows [bi << box_log, ...), column block bc, of K or of V
        const int bi = lane & (nbox - 1), bc = (lane / nbox) % COLS, bt = lane / (nbox * COLS);
        const uint32_t box_bytes = Smem::BOX << box_log;
        WindowIter<kPieceCost<E4M3>> iter;
        iter.start(sm.slice, p);
        WindowIds ids = iter.next<TILE>(p, pg, lane);
        WindowIds ids1 = iter.next<TILE>(p, pg, lane);
        Window nxt = open_window<E4M3>(p, pg, ids), cur = nxt;
        ids = ids1;
        ids1 = iter.next<TILE>(p, pg, lane);
        auto advance = [&]() {
            cur = nxt;
            nxt = open_window<E4M3>(p, pg, ids);
            ids = ids1;
            ids1 = iter.next<TILE>(p, pg, lane);
            if (E4M3 && (int)cur.vs - 127 > kTopVExp)
                na_report(p.status, NA_ERR_UNSUPPORTED);
        };
        uint32_t it = 0;
        bool ok = true;
        while (ok && walk.next(p, pc)) {
            const int lo = pc.kf + pc.k0, hi = pc.kf + pc.k1;
            advance();
            for (int t0 = lo / TILE * TILE; t0 < hi; t0 += TILE, it++) {
                const int stage = it % ST;
                if ((t0 >> pg.page_log) - cur.wb >= 32)
                    advance();
                const bool free = mbar_wait_bounded(&sm.empty[stage], ((it / ST) & 1) ^ 1) &&
                                  !*(volatile int *)&sm.abort_flag;
                if (!__all_sync(FULL, free)) {
                    if (lane == 0) {
                        na_report(p.status, NA_ERR_DEVICE_TIMEOUT);
                        *(volatile int *)&sm.abort_flag = 1;
                    }
                    ok = false;
                    break;
                }
                const int pos = t0 + (bi << box_log);
                const int id = __shfl_sync(FULL, cur.id, ((pos >> pg.page_log) - cur.wb) & 31);
                const bool mine = bt < 2 && id >= 0;
                const uint32_t n = __popc(__ballot_sync(FULL, mine));
                if constexpr (E4M3) {
                    const int kp = t0 + 16 * (lane & 3);
                    const uint32_t sc = __shfl_sync(FULL, cur.ks | (cur.vs << 8),
                                                    ((kp >> pg.page_log) - cur.wb) & 31);
                    if (lane < CWARPS)
                        sm.scales[stage][lane] = (uint16_t)sc;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(&sm.full[stage], n * box_bytes);
                __syncwarp();
                if (mine) {
                    uint8_t *dst = (bt ? sm.v[stage] : sm.k[stage]) + bc * (TILE * 128) +
                                   (bi << box_log) * Smem::BOX;
                    const int y = ((id * p.KV + pc.kvh) << pg.page_log) + (pos & (page - 1));
                    tc::tma_load_2d_hint(dst, bt ? &map_v : &map_k, bc * 64, y, &sm.full[stage],
                                         policy);
                }
            }
        }
        // Every copy issued lands before the CTA can exit.
        for (int s = 0; s < ST; s++) {
            if ((int)it - 1 - s < 0)
                break;
            const uint32_t last = it - 1 - s;
            if (!mbar_wait_bounded(&sm.full[last % ST], (last / ST) & 1))
                na_report(p.status, NA_ERR_DEVICE_TIMEOUT);
        }
        return;
    }

    // ------------------------------------------------------------ consumers --
    // As in the contiguous pass: warp w scores keys 16 w .. 16 w + 15 of each
    // tile with S^T = K Q^T, lane l ends up with keys l/4 and l/4 + 8 of heads
    // 2(l%4) and 2(l%4) + 1, and their probabilities, transposed in registers,
    // are the B operand of O^T += V^T P^T.
    const int hpc = p.group / p.head_chunks;
    if constexpr (MODE != SPLIT) {  // a stream without keys: zero rows, as the merge pass gives
        if (walk.done) {
            const Slice sl = sm.slice;
            const int n = __ldg(p.kv_lens + sl.b);
            if (threadIdx.x == 0 && (n < 0 || n > p.capacity || n > p.max_kv_len))
                na_report(p.status, NA_ERR_CAPACITY);
        }
    }
    if constexpr (MODE == DIRECT) {
        if (walk.done) {
            const Slice sl = sm.slice;
            const int kvh = sl.si / p.head_chunks, hc = sl.si - kvh * p.head_chunks;
            uint32_t *out = reinterpret_cast<uint32_t *>(
                p.out + ((size_t)sl.b * p.H + kvh * p.group + hc * hpc) * D);
            for (int e = threadIdx.x; e < hpc * D / 2; e += CWARPS * 32)
                out[e] = 0u;
            return;
        }
    }
    const int g = lane >> 2, t = lane & 3;
    const int h0 = 2 * t, h1 = 2 * t + 1;  // this lane's heads (columns)
    const bool v0 = h0 < hpc, v1 = h1 < hpc;
    const uint32_t k_base = smem_addr(sm.k[0]), v_base = smem_addr(sm.v[0]);
    // ldmatrix row addresses: lane l feeds row l % 8 of 8x8 matrix l / 8.  K's
    // matrices (rows +0/+8, chunks +0/+1) come in the order (0,0) (8,0) (0,1)
    // (8,1); V's (transposed) the same with E4M3, (0,0) (0,1) (8,0) (8,1) with bf16.
    const int mi = lane >> 3, mr = lane & 7;
    const int ka_row = warp * 16 + (mi & 1) * 8 + mr, ka_col = mi >> 1;
    const int va_row = E4M3 ? ka_row : warp * 16 + (mi >> 1) * 8 + mr;
    const int va_col = E4M3 ? ka_col : mi & 1;
    uint32_t it = 0;
    // A warp whose wait timed out keeps walking the pieces so that every warp
    // joins the same named barriers, but does no more waits or writes.
    bool aborted = false;
    // A cluster's CTAs all take part in the merge, those without keys too.
    bool once = true;
    auto next_piece = [&]() {
        const bool more = walk.next(p, pc);
        if constexpr (MODE == CLUSTER) {
            if (!more && once) {
                const Slice sl = sm.slice;
                pc.b = sl.b;
                pc.kvh = sl.si / p.head_chunks;
                pc.hc = sl.si - pc.kvh * p.head_chunks;
                pc.k0 = pc.k1 = pc.kf = 0;
            }
            const bool go = once;
            once = false;
            return go;
        }
        return more;
    };

    while (next_piece()) {
        const int lo = pc.kf + pc.k0, hi = pc.kf + pc.k1;
        if (*(volatile int *)&sm.abort_flag)
            aborted = true;
        const int head0 = pc.kvh * p.group + pc.hc * hpc;

        // Q as the B operand: column g is head g (zero past hpc), rows are d --
        // with E4M3, k-step s takes d = 16 s + 4 t + {0, 1} and {2, 3}, in f16 with
        // the row's largest magnitude in [2^8, 2^9).
        uint32_t qf[KS][2];
        float mul0 = p.scale_log2, mul1 = p.scale_log2;  // raw score to log2 domain, heads h0, h1
        {
            const bf16 *qrow = p.q + ((size_t)pc.b * p.H + head0 + min(g, hpc - 1)) * D;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                if constexpr (E4M3) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(qrow + 16 * s + 4 * t);
                    qf[s][0] = u.x;
                    qf[s][1] = u.y;
                } else {
                    const uint32_t w0 = *reinterpret_cast<const uint32_t *>(qrow + 16 * s + 2 * t);
                    const uint32_t w1 = *reinterpret_cast<const uint32_t *>(qrow + 16 * s + 2 * t + 8);
                    qf[s][0] = g < hpc ? w0 : 0u;
                    qf[s][1] = g < hpc ? w1 : 0u;
                }
            }
            if constexpr (E4M3) {
                uint32_t amax = 0;  // bits of the largest magnitude, bf16
#pragma unroll
                for (int s = 0; s < KS; s++)
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        amax = max(amax, max(qf[s][i] & 0x7fffu, (qf[s][i] >> 16) & 0x7fffu));
                amax = max(amax, __shfl_xor_sync(FULL, amax, 1));
                amax = max(amax, __shfl_xor_sync(FULL, amax, 2));
                const int e = min(262 - (int)(amax >> 7), 254);  // 2^(e - 127) scales the row
                const float up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
                for (int s = 0; s < KS; s++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint32_t w = qf[s][i];
                        qf[s][i] = g < hpc ? pack_f16x2(__uint_as_float(w << 16) * up,
                                                        __uint_as_float(w & 0xffff0000u) * up)
                                           : 0u;
                    }
                const float down = e8m0_value((uint32_t)(254 - e));
                mul0 *= __shfl_sync(FULL, down, 8 * t);  // the lane with g = h0
                mul1 *= __shfl_sync(FULL, down, 8 * t + 4);
            }
        }
        float acc[KS][4];
#pragma unroll
        for (int s = 0; s < KS; s++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                acc[s][i] = 0.f;
        float m_ref[2] = {-INFINITY, -INFINITY};
        float l_sum[2] = {0.f, 0.f};
        float *prow0 = (p.probs && v0) ? p.probs + ((size_t)pc.b * p.H + head0 + h0) * p.probs_stride
                                        : nullptr;
        float *prow1 = (p.probs && v1) ? p.probs + ((size_t)pc.b * p.H + head0 + h1) * p.probs_stride
                                        : nullptr;

        for (int t0 = lo / TILE * TILE; t0 < hi && !aborted; t0 += TILE, it++) {
            const int stage = it % ST;
            const bool got = mbar_wait_bounded(&sm.full[stage], (it / ST) & 1);
            if (!__all_sync(FULL, got)) {  // warp-uniform before the .sync.aligned MMAs
                if (lane == 0) {
                    na_report(p.status, NA_ERR_DEVICE_TIMEOUT);
                    *(volatile int *)&sm.abort_flag = 1;
                }
                aborted = true;
                break;
            }
            const uint32_t kst = k_base + stage * STAGE_BYTES;
            const uint32_t vst = v_base + stage * STAGE_BYTES;
            const bool partial = t0 < lo || t0 + TILE > hi;  // the same in every warp
            if (partial) {
                // V rows of masked keys are zeroed: they meet a zero probability
                // in the PV MMA and must not be NaN.
                constexpr int CPR = ROW / 16;  // chunks per row
                for (int c = lane; c < 16 * CPR; c += 32) {
                    const int r = warp * 16 + c / CPR, ch = c % CPR;
                    const int pos = t0 + r;
                    if (pos < lo || pos >= hi)
                        *reinterpret_cast<uint4 *>(sm.v[stage] + chunk_off<ROW>(r, ch)) =
                            make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }

            // S^T = K Q^T for this warp's 16 keys.
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
            float sm0 = mul0, sm1 = mul1, v_off = 0.f, v_inv = 1.f;
            uint32_t v_byte = 127;
            if constexpr (E4M3) {
                const uint32_t bytes = sm.scales[stage][warp];
                const float kv = e8m0_value(bytes & 255u);
                sm0 *= kv;
                sm1 *= kv;
                v_byte = bytes >> 8;
                const int e = v_weight_exp(v_byte);
                v_off = (float)e;
                v_inv = exp2i(-e);
#pragma unroll
                for (int s = 0; s < KS / 2; s++) {
                    uint32_t w[4], a0[4], a1[4];
                    ldsm_x4(kst + chunk_off<ROW>(ka_row, 2 * s + ka_col), w);
                    e4m3x4_to_f16(w[0], a0[0], a0[2]);
                    e4m3x4_to_f16(w[1], a0[1], a0[3]);
                    e4m3x4_to_f16(w[2], a1[0], a1[2]);
                    e4m3x4_to_f16(w[3], a1[1], a1[3]);
                    mma_f16_16816(sc, a0, qf[2 * s][0], qf[2 * s][1]);
                    mma_f16_16816(sc, a1, qf[2 * s + 1][0], qf[2 * s + 1][1]);
                }
            } else {
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    uint32_t a[4];
                    ldsm_x4(kst + chunk_off<ROW>(ka_row, 2 * s + ka_col), a);
                    mma_bf16_16816(sc, a, qf[s][0], qf[s][1]);
                }
            }
            // Scores (log2 domain), masked outside the piece and for the padding
            // heads; recorded for the combine pass.
            const int pa = t0 + warp * 16 + g, pb = pa + 8;  // this lane's key positions
            const bool ina = pa >= lo && pa < hi, inb = pb >= lo && pb < hi;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float x = sc[i] * ((i & 1) ? sm1 : sm0);
                if constexpr (CAPPED) {  // c tanh(s / c) in the log2 domain, tanh(y) = 1 - 2 / (e^2y + 1)
                    const float e = exp2f(x * p.cap_in);
                    x = p.cap_out * (1.0f - __fdividef(2.0f, e + 1.0f));
                }
                const bool ok = ((i & 2) ? inb : ina) && ((i & 1) ? v1 : v0);
                sc[i] = ok ? x : -INFINITY;
            }
            if (prow0) {
                if (ina)
                    prow0[pa] = sc[0];
                if (inb)
                    prow0[pb] = sc[2];
            }
            if (prow1) {
                if (ina)
                    prow1[pa] = sc[1];
                if (inb)
                    prow1[pb] = sc[3];
            }
            // When a score exceeds its head's reference by too much (rarely) the
            // reference is raised to the tile's maximum, over the 8 lanes sharing the
            // column.  E4M3: of score + V's exponent, and the reference stays kF16Top
            // below it.
            constexpr float TOP = E4M3 ? kF16Top : 0.f, LIMIT = E4M3 ? kF16Limit : kRescaleThreshold;
            float mx0 = fmaxf(sc[0], sc[2]) + v_off, mx1 = fmaxf(sc[1], sc[3]) + v_off;
            if (__any_sync(FULL, mx0 > m_ref[0] + LIMIT || mx1 > m_ref[1] + LIMIT)) {
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(FULL, mx0, m));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(FULL, mx1, m));
                }
                const float n0 = fmaxf(m_ref[0], mx0 - TOP), n1 = fmaxf(m_ref[1], mx1 - TOP);
                const float a0 = (m_ref[0] == -INFINITY) ? 0.f : exp2f(m_ref[0] - n0);
                const float a1 = (m_ref[1] == -INFINITY) ? 0.f : exp2f(m_ref[1] - n1);
                m_ref[0] = n0;
                m_ref[1] = n1;
                l_sum[0] *= a0;
                l_sum[1] *= a1;
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    acc[s][0] *= a0;
                    acc[s][1] *= a1;
                    acc[s][2] *= a0;
                    acc[s][3] *= a1;
                }
            }
            float pr[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if constexpr (E4M3) {  // a column without a key yet: m_ref is -inf too
                    pr[i] = (sc[i] == -INFINITY) ? 0.f : ex2_mufu(sc[i] + (v_off - m_ref[i & 1]));
                    l_sum[i & 1] = fmaf(pr[i], v_inv, l_sum[i & 1]);
                } else {
                    pr[i] = (sc[i] == -INFINITY) ? 0.f : exp2f(sc[i] - m_ref[i & 1]);
                    l_sum[i & 1] += pr[i];
                }
            }
            // P^T as the B operand: keys 2(l%4).. of head l/4.
            const uint32_t b0 = movmatrix_trans(E4M3 ? pack_f16x2(pr[0], pr[1]) : pack_bf16x2(pr[0], pr[1]));
            const uint32_t b1 = movmatrix_trans(E4M3 ? pack_f16x2(pr[2], pr[3]) : pack_bf16x2(pr[2], pr[3]));
            // O^T += V^T P^T, one 16-row block of d at a time.
            if constexpr (E4M3) {
                const bool extreme = abs((int)v_byte - 127) > kMaxVExp;  // warp-uniform
                const uint32_t rest = v_rest_f16x2(v_byte), rest2 = v_rest_f16x2_second(v_byte);
#pragma unroll
                for (int s = 0; s < KS / 2; s++) {
                    uint32_t w[4], a0[4], a1[4];
                    ldsm_x4_trans(vst + chunk_off<ROW>(va_row, 2 * s + va_col), w);
#pragma unroll
                    for (int i = 0; i < 4; i++)  // (key 0, key 1) of the even d, then of the odd
                        w[i] = __byte_perm(w[i], 0u, 0x3120);
                    e4m3x4_to_f16(w[0], a0[0], a0[1]);
                    e4m3x4_to_f16(w[1], a0[2], a0[3]);
                    e4m3x4_to_f16(w[2], a1[0], a1[1]);
                    e4m3x4_to_f16(w[3], a1[2], a1[3]);
                    if (extreme) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            a0[i] = mul_f16x2(mul_f16x2(a0[i], rest), rest2);
                            a1[i] = mul_f16x2(mul_f16x2(a1[i], rest), rest2);
                        }
                    }
                    mma_f16_16816(acc[2 * s], a0, b0, b1);
                    mma_f16_16816(acc[2 * s + 1], a1, b0, b1);
                }
            } else {
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    uint32_t a[4];
                    ldsm_x4_trans(vst + chunk_off<ROW>(va_row, 2 * s + va_col), a);
                    mma_bf16_16816(acc[s], a, b0, b1);
                }
            }
            if (partial)
                tc::fence_proxy_async_smem();  // the zeroed rows before the stage's next copy
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.empty[stage]);
        }
        // Sums over the 8 lanes of each column; then the warps' partials are merged
        // pairwise, 1 into 0 and 3 into 2, 2 into 0.  Lane l of every warp holds the
        // same heads and d, so a partial crosses as one float4 per lane and step,
        // and the order of the additions is fixed.  (Adding warp after warp into
        // one buffer of rows, as the contiguous pass does: 154 us against 110 us
        // for 64 sequences of 512 .. 8192 keys, 32/8 heads.)
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
            l_sum[0] += __shfl_xor_sync(FULL, l_sum[0], m);
            l_sum[1] += __shfl_xor_sync(FULL, l_sum[1], m);
        }
        auto give = [&](float4 (*buf)[32]) {
#pragma unroll
            for (int s = 0; s < KS; s++)
                buf[s][lane] = make_float4(acc[s][0], acc[s][1], acc[s][2], acc[s][3]);
            buf[KS][lane] = make_float4(m_ref[0], m_ref[1], l_sum[0], l_sum[1]);
        };
        auto take = [&](const float4 (*buf)[32]) {
            const float4 o = buf[KS][lane];
            const float om[2] = {o.x, o.y}, ol[2] = {o.z, o.w};
            float fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float m = fmaxf(m_ref[i], om[i]);
                fa[i] = m_ref[i] == -INFINITY ? 0.f : exp2f(m_ref[i] - m);
                fb[i] = om[i] == -INFINITY ? 0.f : exp2f(om[i] - m);
                m_ref[i] = m;
                l_sum[i] = l_sum[i] * fa[i] + ol[i] * fb[i];
            }
#pragma unroll
            for (int s = 0; s < KS; s++) {
                const float4 x = buf[s][lane];
                acc[s][0] = acc[s][0] * fa[0] + x.x * fb[0];
                acc[s][1] = acc[s][1] * fa[1] + x.y * fb[1];
                acc[s][2] = acc[s][2] * fa[0] + x.z * fb[0];
                acc[s][3] = acc[s][3] * fa[1] + x.w * fb[1];
            }
        };
        if (warp & 1)
            give(sm.merge[warp >> 1]);
        named_barrier_sync(1, CWARPS * 32);
        if (!(warp & 1))
            take(sm.merge[warp >> 1]);
        if (warp == 2)
            give(sm.merge[2]);
        named_barrier_sync(1, CWARPS * 32);
        // (Warps 1 and 3 write again after this barrier, which the readers of their
        // buffers have passed; warp 2 after the next piece's first one.)
        if (warp == 0)
            take(sm.merge[2]);
        if constexpr (MODE == CLUSTER) {
            // The CTAs' partials: warp 0 of each offers its own (merge[0], which it has
            // read), takes every CTA's maximum and sum, and the d-blocks that it writes,
            // in the order of the ranks.  All consumer threads meet in both barriers
            // whatever happened before; the second lets no CTA go whose partial is
            // still being read.
            bool bad = *(volatile int *)&sm.abort_flag != 0;
            if (warp == 0) {
                give(sm.merge[0]);
                if (bad)
                    sm.merge[0][KS][lane] = make_float4(-INFINITY, -INFINITY, -1.f, -1.f);
            }
            cluster_arrive();
            cluster_wait();
            if (warp == 0) {
                float4 ml[MAX_CLUSTER];
#pragma unroll
                for (int c = 0; c < MAX_CLUSTER; c++)
                    ml[c] = c < C ? cluster_load(&sm.merge[0][KS][lane], c)
                                  : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
                m_ref[0] = m_ref[1] = -INFINITY;
#pragma unroll
                for (int c = 0; c < MAX_CLUSTER; c++) {
                    bad = bad || ml[c].z < 0.f;
                    m_ref[0] = fmaxf(m_ref[0], ml[c].x);
                    m_ref[1] = fmaxf(m_ref[1], ml[c].y);
                }
                l_sum[0] = l_sum[1] = 0.f;
#pragma unroll
                for (int c = 0; c < MAX_CLUSTER; c++) {  // the factors replace the maxima
                    ml[c].x = ml[c].x == -INFINITY ? 0.f : exp2f(ml[c].x - m_ref[0]);
                    ml[c].y = ml[c].y == -INFINITY ? 0.f : exp2f(ml[c].y - m_ref[1]);
                    l_sum[0] += ml[c].z * ml[c].x;
                    l_sum[1] += ml[c].w * ml[c].y;
                }
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    if ((s & (C - 1)) != rank)
                        continue;
                    float4 x[MAX_CLUSTER];
#pragma unroll
                    for (int c = 0; c < MAX_CLUSTER; c++)
                        x[c] = c < C ? cluster_load(&sm.merge[0][s][lane], c)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                    acc[s][0] = acc[s][1] = acc[s][2] = acc[s][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < MAX_CLUSTER; c++) {
                        acc[s][0] += x[c].x * ml[c].x;
                        acc[s][1] += x[c].y * ml[c].y;
                        acc[s][2] += x[c].z * ml[c].x;
                        acc[s][3] += x[c].w * ml[c].y;
                    }
                }
                if (lane == 0)
                    sm.cluster_bad = bad;
            }
            __syncwarp();
            cluster_arrive();
            named_barrier_sync(1, THREADS - 32);  // cluster_bad
            finish_stream<D, E4M3, THREADS - 32>(p, pc, sm.fin, head0, hpc, acc, m_ref, l_sum,
                                                 sm.cluster_bad != 0, rank, C);
            __syncwarp();
            cluster_wait();
            continue;
        }
        if constexpr (MODE == DIRECT) {  // the whole stream: its rows and probabilities
            finish_stream<D, E4M3, THREADS - 32>(p, pc, sm.fin, head0, hpc, acc, m_ref, l_sum,
                                                 *(volatile int *)&sm.abort_flag != 0, 0, 1);
            continue;
        }
        if (warp != 0)
            continue;
        // Every consumer warp has finished this piece's tiles (or given up): the
        // abort flag is final for the piece, and a piece of a CTA whose wait gave
        // up is written as the marker (max -inf, sum -1) that the merge pass reports.
        const bool bad = *(volatile int *)&sm.abort_flag != 0;
        // acc row l/4 is d = 16 s + l/4 and row l/4 + 8 is 8 further on (bf16),
        // or d = 16 s + 2 (l/4) and the next one (E4M3).
        float *po = p.part_o + (size_t)pc.id * hpc * D;
        float *ml = p.part_ml + (size_t)pc.id * hpc * 2;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int h = h0 + i;
            if (h >= hpc)
                break;
            if (!bad) {
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    float *o = po + h * D + 16 * s + (E4M3 ? 2 * g : g);
                    if constexpr (E4M3) {
                        *reinterpret_cast<float2 *>(o) = make_float2(acc[s][i], acc[s][2 + i]);
                    } else {
                        o[0] = acc[s][i];
                        o[8] = acc[s][2 + i];
                    }
                }
            }
            if (g == 0)
                *reinterpret_cast<float2 *>(ml + 2 * h) =
                    bad ? make_float2(-INFINITY, -1.0f) : make_float2(m_ref[i], l_sum[i]);
        }
        if (threadIdx.x == 0) {  // the span follows from the slicing alone: always written
            const int stream = pc.id - blockIdx.x;
            if (pc.first)
                p.piece_span[2 * stream] = pc.id;
            if (pc.last)
                p.piece_span[2 * stream + 1] = pc.id;
        }
    }
}

template <int D, bool E4M3, bool CAPPED, Mode MODE>
cudaError_t launch_paged_split(const DecodeParams &p, const PagedView &pg, cudaStream_t stream)
{
    typedef PagedSmem<D, E4M3> Smem;
    // K and V as 2-D tensors of cache rows ((page, kv head, slot) x D), read in
    // boxes of a page's rows, or 64 of them, by 128 bytes (E4M3 with d = 64: 64).
    CUtensorMap mk, mv;
    const cuuint64_t rows = ((cuuint64_t)pg.num_pages * p.KV) << pg.page_log;
    const cuuint64_t dims[2] = {(cuuint64_t)D, rows};
    const cuuint64_t strides[1] = {(cuuint64_t)Smem::ROW};
    const cuuint32_t box[2] = {(cuuint32_t)(E4M3 ? Smem::BOX : Smem::BOX / 2),
                               1u << (pg.page_log < 6 ? pg.page_log : 6)};
    const bool ok = E4M3 ? make_u8_tile_map(&mk, p.cache_k, 2, dims, strides, box, true) &&
                               make_u8_tile_map(&mv, p.cache_v, 2, dims, strides, box, true)
                         : make_bf16_tile_map(&mk, p.cache_k, 2, dims, strides, box) &&
                               make_bf16_tile_map(&mv, p.cache_v, 2, dims, strides, box);
    if (!ok)
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(Smem) + 1024;  // + alignment slack
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = once_per_device(configured, [smem] {
        cudaError_t r = cudaFuncSetAttribute(decode_paged_kernel<D, E4M3, CAPPED, MODE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(decode_paged_kernel<D, E4M3, CAPPED, MODE>,
                                     cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        return r;
    });
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(decode_paged_kernel<D, E4M3, CAPPED, MODE>, dim3(p.grid),
                                 dim3(THREADS), smem, MODE == CLUSTER ? p.direct : 0, stream, p, pg,
                                 mk, mv);
}

template <int D, bool E4M3>
cudaError_t launch_paged_t(const DecodeParams &p, const PagedView &pg, cudaStream_t stream)
{
    auto split = [&](auto capped) {
        constexpr bool CAP = decltype(capped)::value;
        if (p.direct > 1)
            return launch_paged_split<D, E4M3, CAP, CLUSTER>(p, pg, stream);
        if (p.direct)
            return launch_paged_split<D, E4M3, CAP, DIRECT>(p, pg, stream);
        const cudaError_t e = launch_paged_split<D, E4M3, CAP, SPLIT>(p, pg, stream);
        return e != cudaSuccess ? e : launch_decode_combine(p, D, stream);
    };
    return p.cap_out > 0.f ? split(std::true_type()) : split(std::false_type());
}

}  // namespace

int decode_paged_ctas_per_sm(bool e4m3) { return e4m3 ? kCtasPerSm<true> : kCtasPerSm<false>; }

// CTAs per stream of a call that is not cut over the whole grid, or 0.  A tile
// takes a CTA 0.45 us (bf16) or 0.6 us (E4M3), the meeting in shared memory 1 us,
// the merge pass 3 us: 128 keys per CTA while every CTA has an SM of its own, then
// 256 while all are resident, and the whole grid once that leaves a CTA more than
// 512 (or 256 with so few streams that the grid cuts them finer).  Measured, d 128,
// one kv head per stream, split against this, bf16 / E4M3 in us: 16 streams of 1024
// keys 8.3 / 9.1 against 8.2 / 8.7, of 2048 11.0 / 11.3 against 9.1 / 9.9; 64 of 2048
// 16.3 / 15.8 against 12.0 / 14.1; 16 of 512 8.7 / 10.0 with one CTA each, 7.7 / 8.1
// with four.  Beyond: 2 streams of 4096 keys 9.7 / 10.8 against 10.3 / 11.6; 128 of 512
// with two CTAs each, two per SM, 10.1 / 11.1 against 9.3 / 10.6 with one.
int decode_paged_cluster(bool e4m3, int sms, long long streams, int max_kv_len)
{
    int C = 1;
    if (max_kv_len > 256)
        while (C < MAX_CLUSTER && max_kv_len > 128 * C && streams * 2 * C <= sms)
            C *= 2;
    if (max_kv_len > 512)
        while (C < MAX_CLUSTER && max_kv_len > 256 * C &&
               streams * 2 * C <= (long long)sms * decode_paged_ctas_per_sm(e4m3))
            C *= 2;
    return max_kv_len <= (streams < 8 ? 256 : 512) * C ? C : 0;
}

cudaError_t launch_decode_paged(const DecodeParams &p, const PagedView &pg, bool e4m3, int d,
                                cudaStream_t stream)
{
    if (d == 128)
        return e4m3 ? launch_paged_t<128, true>(p, pg, stream) : launch_paged_t<128, false>(p, pg, stream);
    return e4m3 ? launch_paged_t<64, true>(p, pg, stream) : launch_paged_t<64, false>(p, pg, stream);
}
