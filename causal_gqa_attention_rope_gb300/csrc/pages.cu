// pages.cu -- the pages of a cache between attention calls: a step of the page
// tables (na_pages_fork), whole pages copied (na_pages_copy), kept tokens moved to
// the front of new pages (na_pages_compact).
#include <climits>
#include <cuda_fp16.h>

#include "pages.cuh"
#include "rope_math.cuh"
#include "tile_waits.cuh"

namespace {

using namespace rope;

// ------------------------------------------------------------------- fork --
//
// A cluster of FORK_CTAS: a step's tables are a few thousand entries, and every phase
// needs what the phase before found about all sequences, so the CTAs meet in between and
// leave what all of them need in everybody's shared memory.  A warp takes a new row, which
// it copies from its parent's, or an old row without a child.  Counts of references change
// by atomics on integers, whose order does not show, and only for parents that have not
// exactly one child (kids - 1 for a shared page, -1 for an ended sequence's).  Free pages
// are then found in index order by a scan, page rank k going to the sequence whose range of
// missing pages holds k, and a copy to the one that gets its sequence's first.  Bound by latency:
// 256 sequences in 8750 pages take 8.4 us by itself, 9.9 where 95 of them get a copy of a page
// (11 with the launch that copies them); one CTA took 26, 17 of them for the rows.

constexpr int FORK_CTAS = 8;
constexpr int FORK_AHEAD = 4;  // entries per lane and round of a row
constexpr int FORK_PAGES = 2;  // pages per thread and round of the scan

// Exclusive prefix sums of N values per thread over the CTA; `total` gets the sums.
template <int THREADS, int N>
__device__ __forceinline__ void block_prefix(int (&v)[N], int (*warp_sums)[THREADS / 32], int (&total)[N])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x[N], before[N];
#pragma unroll
    for (int n = 0; n < N; n++)
        x[n] = v[n];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < N; n++) {
            const int y = __shfl_up_sync(0xffffffffu, x[n], o);
            if (lane >= o)
                x[n] += y;
        }
    __syncthreads();  // the sums of an earlier call have been read
    if (lane == 31)
#pragma unroll
        for (int n = 0; n < N; n++)
            warp_sums[n][warp] = x[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; n++) {
        total[n] = lane < THREADS / 32 ? warp_sums[n][lane] : 0;
        before[n] = lane < warp ? total[n] : 0;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; n++) {
            before[n] += __shfl_xor_sync(0xffffffffu, before[n], o);
            total[n] += __shfl_xor_sync(0xffffffffu, total[n], o);
        }
#pragma unroll
    for (int n = 0; n < N; n++)
        v[n] = before[n] + x[n] - v[n];
}

// x into the word at `at`'s place in CTA `rank` of the cluster.
__device__ __forceinline__ void store_in_cta(int *at, int rank, int x)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(at)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) pages_fork_kernel(const ForkParams p)
{
    extern __shared__ int fork_smem[];
    int *kids = fork_smem;               // [old_batch]
    int *first = kids + p.old_batch;     // [old_batch]  lowest child
    int *lens = first + p.old_batch;     // [old_batch]
    int *parents = lens + p.old_batch;   // [batch]
    int *start = parents + p.batch;      // [batch]  first missing entry
    int *offs = start + p.batch;         // [batch]  missing entries before sequence b
    int *copied = offs + p.batch;        // [batch]  page whose copy is the first missing entry, or -1
    __shared__ int warp_sums[2][THREADS / 32], free_of[FORK_CTAS];
    grid_dependency_wait();
    grid_dependents_launch();
    const int rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.pages_per_seq;

    // (what the first round needs is asked for together)
    const int page0 = rank * THREADS + tid;
    const int len0 = tid < p.old_batch ? __ldg(p.lens + tid) : 0;
    const int parent0 = tid < p.batch ? __ldg(p.parents + tid) : 0;
    const int ref0 = page0 < p.num_pages ? __ldg(p.ref + page0) : 0;
    for (int i = tid; i < p.old_batch; i += THREADS) {
        kids[i] = 0;
        first[i] = INT_MAX;
        lens[i] = max(i == tid ? len0 : __ldg(p.lens + i), 0);
    }
    for (int b = tid; b < p.batch; b += THREADS) {
        int par = b == tid ? parent0 : __ldg(p.parents + b);
        if (par >= p.old_batch) {
            na_report(p.status, NA_ERR_INVALID_ARG);
            par = -1;
        }
        parents[b] = max(par, -1);
    }
    for (int i = page0; i < p.num_pages; i += FORK_CTAS * THREADS)
        p.new_ref[i] = i == page0 ? ref0 : __ldg(p.ref + i);
    __syncthreads();
    for (int b = tid; b < p.batch; b += THREADS)
        if (parents[b] >= 0) {
            atomicAdd(&kids[parents[b]], 1);
            atomicMin(&first[parents[b]], b);
        }
    cluster_sync();  // (and every thread of the CTA)

    // Items: new rows, then old rows (of which those without a child).
    for (int i = rank * (THREADS / 32) + warp; i < p.batch + p.old_batch;
         i += FORK_CTAS * (THREADS / 32)) {
        const bool fresh = i < p.batch;
        const int row = fresh ? parents[i] : (kids[i - p.batch] == 0 ? i - p.batch : -1);
        if (!fresh && row < 0)
            continue;
        int grow = fresh && p.grow ? __ldg(p.grow + i) : 0;
        const int n = row >= 0 ? lens[row] : 0, full = n >> p.page_log;
        // the row's counts change: once for each page, by the lowest child or without one
        const bool elder = row >= 0 && (!fresh || first[row] == i);
        const int shared = row >= 0 ? kids[row] - 1 : 0;
        const int32_t *from = p.table + (size_t)max(row, 0) * P;
        int32_t *to = p.new_table + (size_t)i * P;
        int held = P, part_filled = -1;  // entry `full`, in one of the lanes
        bool end = false;
        for (int base = 0; base < P; base += 32 * FORK_AHEAD) {
            int e[FORK_AHEAD];
#pragma unroll
            for (int k = 0; k < FORK_AHEAD; k++) {
                const int j = base + k * 32 + lane;
                e[k] = row >= 0 && j < P && !end ? __ldg(from + j) : -1;
            }
#pragma unroll
            for (int k = 0; k < FORK_AHEAD; k++) {
                const int j0 = base + k * 32, j = j0 + lane;
                if (j0 >= P)
                    break;
                const bool is_page = !end && (unsigned)e[k] < (unsigned)p.num_pages;
                const unsigned bad = __ballot_sync(0xffffffffu, !is_page);
                const int good = bad ? __ffs(bad) - 1 : 32;  // 0 behind the row's end
                if (bad && !end) {
                    end = true;
                    held = min(j0 + good, P);
                    if (elder && lane == good && e[k] >= 0)
                        na_report(p.status, NA_ERR_PAGE);
                }
                const int delta = fresh && j >= full ? 0 : shared;
                if (elder && lane < good && delta != 0)
                    atomicAdd(p.new_ref + e[k], delta);
                if (fresh && j < P)
                    to[j] = lane < good && (elder || j < full) ? e[k] : -1;
                if (j == full)
                    part_filled = e[k];
            }
            if (end && !fresh)
                break;
        }
        if (!fresh)
            continue;
        held = row >= 0 ? held : 0;
        const int mine = elder ? held : min(full, held);
        const long long pages = ((long long)n + max(grow, 0) + (1 << p.page_log) - 1) >> p.page_log;
        // a part-filled page that is there is copied for all children but the first
        const bool copies = row >= 0 && !elder && (n & ((1 << p.page_log) - 1)) && full < held;
        const int page = __shfl_sync(0xffffffffu, part_filled, full & 31);
        const int copy = copies ? page : -1;
        if (lane < FORK_CTAS) {
            store_in_cta(start + i, lane, mine);
            store_in_cta(copied + i, lane, copy);
            store_in_cta(offs + i, lane, max((int)min(pages, (long long)P) - mine, 0));
        }
        if (lane == 0) {
            if (grow < 0)
                na_report(p.status, NA_ERR_INVALID_ARG);
            if (((long long)held << p.page_log) < n)
                na_report(p.status, NA_ERR_PAGE);
            if (pages > P)
                na_report(p.status, NA_ERR_CAPACITY);
            p.new_lens[i] = n;
            p.copy_src[i] = -1;  // until a page is found
            p.copy_dst[i] = -1;
        }
    }
    cluster_sync();

    // Missing pages before each sequence's, in every CTA, and free pages in order: a CTA's run of
    // pages, counted, then ranked behind the runs before.
    constexpr int ROUND = THREADS * FORK_PAGES;
    const int run = (p.num_pages + FORK_CTAS - 1) / FORK_CTAS;
    const int p0 = min(rank * run, p.num_pages), p1 = min(p0 + run, p.num_pages);
    auto free_at = [&](int at) {  // which of FORK_PAGES pages are free
        unsigned free = 0;
#pragma unroll
        for (int i = 0; i < FORK_PAGES; i++)
            if (at + i < p1 && __ldcg(p.new_ref + at + i) == 0)
                free |= 1u << i;
        return free;
    };
    const unsigned free0 = free_at(p0 + FORK_PAGES * tid);  // the first round's
    int count = __popc(free0);
    for (int at = p0 + ROUND + FORK_PAGES * tid; at < p1; at += ROUND)
        count += __popc(free_at(at));
    int missing = 0, total = 0;
    for (int base = 0; base < p.batch; base += THREADS) {
        const int b = base + tid;
        int v[2] = {b < p.batch ? offs[b] : 0, base == 0 ? count : 0}, sum[2];
        block_prefix<THREADS>(v, warp_sums, sum);
        if (b < p.batch)
            offs[b] = missing + v[0];
        missing += sum[0];
        total += sum[1];
    }
    if (tid < FORK_CTAS)
        store_in_cta(free_of + rank, tid, total);
    cluster_sync();
    int found = 0, all = 0;
#pragma unroll
    for (int c = 0; c < FORK_CTAS; c++) {
        found += c < rank ? free_of[c] : 0;
        all += free_of[c];
    }
    for (int base = p0; base < p1 && found < missing; base += ROUND) {
        const int at = base + FORK_PAGES * tid;
        const unsigned free = base == p0 ? free0 : free_at(at);
        int v[1] = {__popc(free)}, sum[1];
        block_prefix<THREADS>(v, warp_sums, sum);
        int k = found + v[0];
        found += sum[0];
        if (!free || k >= missing)
            continue;
        int lo = 0, hi = p.batch - 1;  // the last b with offs[b] <= k
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (offs[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
#pragma unroll
        for (int i = 0; i < FORK_PAGES; i++) {
            if (!(free >> i & 1) || k >= missing)
                continue;
            while (lo + 1 < p.batch && offs[lo + 1] <= k)
                lo++;
            p.new_table[(size_t)lo * P + start[lo] + (k - offs[lo])] = at + i;
            p.new_ref[at + i] = 1;
            if (k == offs[lo] && copied[lo] >= 0) {
                p.copy_src[lo] = copied[lo];
                p.copy_dst[lo] = at + i;
            }
            k++;
        }
    }
    if (all < missing && rank == 0 && tid == 0)
        na_report(p.status, NA_ERR_CAPACITY);
}

// ------------------------------------------------------------------- copy --
//
// Bound by memory: a CTA moves COPY_BYTES of one page, every thread's four
// 16-byte loads in flight before its first store.

constexpr int COPY_THREADS = 256;
constexpr int COPY_BYTES = COPY_THREADS * 16 * 4;

__global__ void __launch_bounds__(COPY_THREADS) pages_copy_kernel(const PageCopyParams p)
{
    grid_dependency_wait();
    grid_dependents_launch();
    const int per = p.v ? 2 * p.chunks : p.chunks;
    const int pair = blockIdx.x / per, part = blockIdx.x - pair * per;
    const int src = __ldg(p.src + pair), dst = __ldg(p.dst + pair);
    if (src < 0 || dst < 0)
        return;
    if (src >= p.num_pages || dst >= p.num_pages) {
        if (part == 0 && threadIdx.x == 0)
            na_report(p.status, NA_ERR_PAGE);
        return;
    }
    const bool is_v = part >= p.chunks;
    uint8_t *pool = is_v ? p.v : p.k;
    const long long at = (long long)(is_v ? part - p.chunks : part) * COPY_BYTES + threadIdx.x * 16;
    const uint8_t *from = pool + src * p.page_bytes;
    uint8_t *to = pool + dst * p.page_bytes;
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const long long x = at + i * COPY_THREADS * 16;
        if (x < p.page_bytes)
            u[i] = *reinterpret_cast<const uint4 *>(from + x);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const long long x = at + i * COPY_THREADS * 16;
        if (x < p.page_bytes)
            *reinterpret_cast<uint4 *>(to + x) = u[i];
    }
    if (p.k_scale && (part == 0 || part == p.chunks)) {
        uint8_t *scale = is_v ? p.v_scale : p.k_scale;
        for (int g = threadIdx.x; g < p.kv_heads; g += COPY_THREADS)
            scale[(size_t)dst * p.kv_heads + g] = scale[(size_t)src * p.kv_heads + g];
    }
}

// ---------------------------------------------------------------- compact --
//
// A row's elements in units of W (8, one 16-byte word of bf16, or 1 where the
// turned dimensions have no such multiple): units of W pairs that turn together,
// then the others.

// Elements e0 .. and e1 .. (both W long) of pair unit u: the two halves, or with
// interleaved pairs 2 W consecutive elements.
template <int W>
__device__ __forceinline__ void pair_unit(const CompactParams &p, int u, int &e0, int &e1)
{
    e0 = p.rot_start + (p.interleaved ? 2 * u * W : u * W);
    e1 = e0 + (p.interleaved ? W : p.rd / 2);
}

// Element of unit u of those that do not turn.
template <int W>
__device__ __forceinline__ int plain_unit(const CompactParams &p, int u)
{
    const int e = u * W;
    return e >= p.rot_start ? e + p.rd : e;
}

// Where row j of sequence b comes from and goes to: rows of one kv head's pages as
// (page, slot); false (with a report) where there is no such place.
struct Move {
    int src, src_slot, dst, dst_slot, shift;  // shift: old position - new position
};

__device__ __forceinline__ bool find_move(const CompactParams &p, int b, int j, Move &m)
{
    const int old = p.keep ? __ldg(p.keep + (size_t)b * p.max_keep + j) : j;
    const int old_page = old >> p.from.page_log, new_page = j >> p.to.page_log;
    if (old < 0 || old_page >= p.from.pages_per_seq) {
        na_report(p.status, NA_ERR_CAPACITY);
        return false;
    }
    m.src = __ldg(p.from.table + (size_t)b * p.from.pages_per_seq + old_page);
    m.dst = __ldg(p.to.table + (size_t)b * p.to.pages_per_seq + new_page);
    if ((unsigned)m.src >= (unsigned)p.from.num_pages || (unsigned)m.dst >= (unsigned)p.to.num_pages) {
        na_report(p.status, NA_ERR_PAGE);
        return false;
    }
    m.src_slot = old & ((1 << p.from.page_log) - 1);
    m.dst_slot = j & ((1 << p.to.page_log) - 1);
    m.shift = old - j;
    return true;
}

// Rows to move of sequence b (0, with a report, for a length that has no room).
__device__ __forceinline__ int kept_rows(const CompactParams &p, int b)
{
    const int n = __ldg(p.keep_lens + b);
    if (n > p.max_keep || n > p.to_positions) {
        if (threadIdx.x == 0)
            na_report(p.status, NA_ERR_CAPACITY);
        return 0;
    }
    return n;
}

// cos and sin of pair i turned back by `shift` positions (forward for a negative one), each
// within 2^-24: the phase in 2^-32 of a turn, split into the nearest 1 / 256 turn (a table)
// and a remainder |r| <= pi / 256, whose series are cut where the next term is below 2^-37.
__device__ __forceinline__ float2 turn_back(const RopeTurns &t, int i, int shift)
{
    const uint32_t u = (uint32_t)(((unsigned long long)(unsigned)abs(shift) * t.hi[i]) >> 32) + (1u << 23);
    const TrigEntry e = kTrig.e[u >> 24];
    const float r = (float)((int)(u & 0xffffffu) - (1 << 23)) * (kTwoPiHi * 0x1p-32f);
    const float z = r * r;
    const float c1 = z * fmaf(z, 1.0f / 24.0f, -0.5f);     // cos r - 1
    const float sr = fmaf(r * z, -1.0f / 6.0f, r);         // sin r
    const float c = e.ch + fmaf(e.ch, c1, fmaf(-e.sh, sr, e.cl));
    const float s = e.sh + fmaf(e.sh, c1, fmaf(e.ch, sr, e.sl));
    return make_float2(c, shift > 0 ? -s : s);
}

template <int W>
struct Words;
template <>
struct Words<8> {
    typedef uint4 T;
    static __device__ __forceinline__ void widen(const uint4 &u, float *f) { bf16x8_to_f32(u, f); }
    static __device__ __forceinline__ uint4 round(const float *f) { return f32_to_bf16x8(f); }
};
template <>
struct Words<1> {
    typedef uint16_t T;
    static __device__ __forceinline__ void widen(uint16_t u, float *f)
    {
        f[0] = __uint_as_float((uint32_t)u << 16);
    }
    static __device__ __forceinline__ uint16_t round(const float *f)
    {
        return (uint16_t)(pack_bf16x2(f[0], 0.f) & 0xffffu);
    }
};

constexpr int COMPACT_THREADS = 256;
constexpr int COMPACT_ROWS = 16;
constexpr int COMPACT_LOADS = 4;       // units whose loads a thread has in flight
constexpr int COMPACT_TURN_LOADS = 2;  // the same of those that turn

// The first of `units` that this thread takes and the first row it does so for; the next row
// is `apart` further.  Rows that are narrower than the CTA are taken side by side.
__device__ __forceinline__ int first_unit(int units, int &row, int &apart)
{
    apart = max(COMPACT_THREADS / max(units, 1), 1);
    if (units >= COMPACT_THREADS) {
        row = 0;
        return threadIdx.x;
    }
    row = threadIdx.x / max(units, 1);
    return row < apart ? (int)threadIdx.x - row * units : units;
}

// bf16: a CTA moves COMPACT_ROWS rows of one sequence, all kv heads of K and V: where they
// come from and go to, and cos and sin of their shifts, are found once and left in shared
// memory.  Then units of 16 bytes (pairs of them where K turns), consecutive lanes along a
// row, a thread the same one of several rows: COMPACT_LOADS loads ahead of the stores, and
// one division for all of them.  64 sequences of 512 .. 8192 tokens, 8 kv heads, a quarter
// kept: 101 us, 0.80 of the copy bandwidth; 86 us where nothing turns, which is what rows of
// 256 bytes out of four times as many cost.  Turning is bound by instructions: with cos and
// sin as pairs of fp32 numbers and a division per unit it took 141 us.
template <int W>
__global__ void __launch_bounds__(COMPACT_THREADS, 5)
    pages_compact_kernel(const __grid_constant__ CompactParams p,
                         const __grid_constant__ RopeTurns turns, int row_blocks)
{
    typedef typename Words<W>::T Word;
    extern __shared__ float2 cos_sin[];  // [row][W][pairs / W]: without bank conflicts between units
    __shared__ long long src_at[COMPACT_ROWS], dst_at[COMPACT_ROWS];  // element of head 0; -1: no place
    __shared__ int shift_of[COMPACT_ROWS];
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.x / row_blocks, j0 = (blockIdx.x - b * row_blocks) * COMPACT_ROWS;
    const int n = min(kept_rows(p, b) - j0, COMPACT_ROWS);
    if (n <= 0)
        return;
    const int half = p.turn ? p.rd / 2 : 0;
    if (threadIdx.x < n) {
        Move m;
        const bool there = find_move(p, b, j0 + threadIdx.x, m);
        src_at[threadIdx.x] =
            there ? (((long long)m.src * p.KV << p.from.page_log) + m.src_slot) * p.d : -1;
        dst_at[threadIdx.x] = there ? (((long long)m.dst * p.KV << p.to.page_log) + m.dst_slot) * p.d : -1;
        shift_of[threadIdx.x] = there ? m.shift : 0;
    }
    __syncthreads();
    const long long src_head = (long long)p.d << p.from.page_log, dst_head = (long long)p.d << p.to.page_log;

    // What does not turn: V, and K's other dimensions.
    const int k_plain = (p.d - 2 * half) / W, units = k_plain + (p.to_v ? p.d / W : 0);
    int r0, rows_apart;
    for (int y = first_unit(units * p.KV, r0, rows_apart); y < units * p.KV; y += COMPACT_THREADS) {
        const int g = y / units;
        int u = y - g * units;
        const bool is_v = u >= k_plain;
        if (is_v)
            u -= k_plain;
        const int e = is_v || !p.turn ? u * W : plain_unit<W>(p, u);
        const bf16 *from = reinterpret_cast<const bf16 *>(is_v ? p.from_v : p.from_k) + g * src_head + e;
        bf16 *to = reinterpret_cast<bf16 *>(is_v ? p.to_v : p.to_k) + g * dst_head + e;
        for (int ra = r0; ra < n; ra += rows_apart * COMPACT_LOADS) {
            Word x[COMPACT_LOADS];
#pragma unroll
            for (int k = 0; k < COMPACT_LOADS; k++) {
                const int r = ra + k * rows_apart;
                if (r < n && src_at[r] >= 0)
                    x[k] = *reinterpret_cast<const Word *>(from + src_at[r]);
            }
#pragma unroll
            for (int k = 0; k < COMPACT_LOADS; k++) {
                const int r = ra + k * rows_apart;
                if (r < n && src_at[r] >= 0)
                    *reinterpret_cast<Word *>(to + dst_at[r]) = x[k];
            }
        }
    }
    if (half == 0)
        return;

    for (int i = threadIdx.x; i < n * half; i += COMPACT_THREADS) {
        const int r = i / half, u = i - r * half;
        cos_sin[r * half + u % W * (half / W) + u / W] = turn_back(turns, u, shift_of[r]);
    }
    __syncthreads();
    const int pairs = half / W;
    for (int y = first_unit(pairs * p.KV, r0, rows_apart); y < pairs * p.KV; y += COMPACT_THREADS) {
        const int g = y / pairs, u = y - g * pairs;
        int e0, e1;
        pair_unit<W>(p, u, e0, e1);
        const bf16 *from = reinterpret_cast<const bf16 *>(p.from_k) + g * src_head;
        bf16 *to = reinterpret_cast<bf16 *>(p.to_k) + g * dst_head;
        for (int ra = r0; ra < n; ra += rows_apart * COMPACT_TURN_LOADS) {
            Word x0[COMPACT_TURN_LOADS], x1[COMPACT_TURN_LOADS];
#pragma unroll
            for (int k = 0; k < COMPACT_TURN_LOADS; k++) {
                const int r = ra + k * rows_apart;
                if (r < n && src_at[r] >= 0) {
                    x0[k] = *reinterpret_cast<const Word *>(from + src_at[r] + e0);
                    x1[k] = *reinterpret_cast<const Word *>(from + src_at[r] + e1);
                }
            }
#pragma unroll
            for (int k = 0; k < COMPACT_TURN_LOADS; k++) {
                const int r = ra + k * rows_apart;
                if (r >= n || src_at[r] < 0)
                    continue;
                if (shift_of[r] != 0) {  // (a row that stays keeps its bits, NaN's too)
                    const float2 *cs = cos_sin + r * half + u;
                    float a[2 * W], z[2 * W], lo[W], hi[W];
                    Words<W>::widen(x0[k], a);
                    Words<W>::widen(x1[k], a + W);
#pragma unroll
                    for (int w = 0; w < W; w++) {  // z: the pairs one after the other
                        const float2 c = cs[w * pairs];
                        const float a0 = p.interleaved ? a[2 * w] : a[w];
                        const float a1 = p.interleaved ? a[2 * w + 1] : a[W + w];
                        z[2 * w] = fmaf(a0, c.x, -a1 * c.y);
                        z[2 * w + 1] = fmaf(a1, c.x, a0 * c.y);
                    }
#pragma unroll
                    for (int w = 0; w < W; w++) {
                        lo[w] = p.interleaved ? z[w] : z[2 * w];
                        hi[w] = p.interleaved ? z[W + w] : z[2 * w + 1];
                    }
                    x0[k] = Words<W>::round(lo);
                    x1[k] = Words<W>::round(hi);
                }
                *reinterpret_cast<Word *>(to + dst_at[r] + e0) = x0[k];
                *reinterpret_cast<Word *>(to + dst_at[r] + e1) = x1[k];
            }
        }
    }
}

// E4M3: a CTA fills one page of one kv head, of K or V: the rows in fp32 into shared
// memory, their largest magnitude, then the bytes.
__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    uint32_t lo, hi;
    e4m3x4_to_f16(byte, lo, hi);
    return __half2float(__ushort_as_half((unsigned short)(lo & 0xffffu)));
}

__device__ __forceinline__ uint32_t e4m3x4_of(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// E8M0 byte of the smallest 2^e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), e >= -127.
__device__ __forceinline__ int scale_byte(float amax)
{
    const uint32_t x = __float_as_uint(amax);
    return max((int)(x >> 23) - 8 + ((x & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
}

template <int W>
__global__ void __launch_bounds__(COMPACT_THREADS)
    pages_compact_e4m3_kernel(const __grid_constant__ CompactParams p,
                              const __grid_constant__ RopeTurns turns, int page_blocks)
{
    extern __shared__ float rows[];  // [page][d]
    __shared__ float amax_of[COMPACT_THREADS / 32];
    __shared__ int moved[128];       // row r of the page is among those to write
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.x / page_blocks, pg = blockIdx.x - b * page_blocks;
    const bool is_v = blockIdx.y >= p.KV;
    const int g = is_v ? blockIdx.y - p.KV : blockIdx.y;
    const int j0 = pg << p.to.page_log;
    const int n = min(kept_rows(p, b) - j0, 1 << p.to.page_log);
    if (n <= 0)
        return;
    const int32_t dst = __ldg(p.to.table + (size_t)b * p.to.pages_per_seq + pg);
    const bool turn = p.turn && !is_v;
    const int pairs = turn ? p.rd / 2 / W : 0;
    const int units = pairs + (p.d - (turn ? p.rd : 0)) / W;
    // The rows times 2^-down: 0, then 16 where a value exceeds fp32, whose largest is then infinite
    // (scales of 2^119 and more; what that loses at the other end is far below the page's
    // smallest step).
    float amax;
    int down = 0;
    for (;; down = 16) {
        amax = -1.f;  // no row is moved
        for (int i = threadIdx.x; i < n * units; i += COMPACT_THREADS) {
            const int r = i / units, u = i - r * units;
            Move m;
            const bool there = find_move(p, b, j0 + r, m);
            if (u == 0)
                moved[r] = there;
            if (!there)
                continue;
            amax = fmaxf(amax, 0.f);
            const uint8_t *from = (is_v ? p.from_v : p.from_k) +
                                  ((((size_t)m.src * p.KV + g) << p.from.page_log) + m.src_slot) * p.d;
            uint32_t s = __ldg((is_v ? p.from.v_scale : p.from.k_scale) + (size_t)m.src * p.KV + g);
            if (s == 255) {
                na_report(p.status, NA_ERR_UNSUPPORTED);
                s = 254;
            }
            const float mul = e8m0_value(s) * exp2i(-down);
            float *row = rows + r * p.d;
            auto load = [&](int e, float (&x)[W]) {
                if constexpr (W == 8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(from + e);
                    uint32_t h[4];
                    e4m3x4_to_f16(w.x, h[0], h[1]);
                    e4m3x4_to_f16(w.y, h[2], h[3]);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                        x[2 * k] = f.x * mul;
                        x[2 * k + 1] = f.y * mul;
                    }
                } else {
                    x[0] = e4m3_value(from[e]) * mul;
                }
            };
            if (u >= pairs) {
                const int e = turn ? plain_unit<W>(p, u - pairs) : u * W;
                float x[W];
                load(e, x);
#pragma unroll
                for (int w = 0; w < W; w++) {
                    row[e + w] = x[w];
                    amax = fmaxf(amax, fabsf(x[w]));
                }
                continue;
            }
            int e0, e1;
            pair_unit<W>(p, u, e0, e1);
            float x[2][W];
            load(e0, x[0]);
            load(e1, x[1]);
#pragma unroll
            for (int w = 0; w < W; w++) {
                const float2 c = turn_back(turns, u * W + w, m.shift);
                // the pair's places: its halves, or two neighbours of the 2 W elements
                const int i0 = p.interleaved ? 2 * w : w, i1 = p.interleaved ? 2 * w + 1 : W + w;
                const float a0 = x[i0 / W][i0 % W], a1 = x[i1 / W][i1 % W];
                const float y0 = fmaf(a0, c.x, -a1 * c.y), y1 = fmaf(a1, c.x, a0 * c.y);
                row[(i0 < W ? e0 : e1) + i0 % W] = y0;
                row[(i1 < W ? e0 : e1) + i1 % W] = y1;
                amax = fmaxf(amax, fmaxf(fabsf(y0), fabsf(y1)));
                if (fmaxf(fabsf(a0), fabsf(a1)) == INFINITY)
                    amax = INFINITY;  // (what is turned may be infinity less infinity)
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((threadIdx.x & 31) == 0)
            amax_of[threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < COMPACT_THREADS / 32; w++)
            amax = fmaxf(amax, amax_of[w]);
        if (amax != INFINITY || down)
            break;
        __syncthreads();  // all have read the page's largest
    }
    if (amax < 0.f)
        return;  // reported with the rows; the page keeps its bytes and what they stand for
    const int s = min(scale_byte(amax) + down, 254);
    // 2^(127 - s + down) in two factors: the first of a small scale alone exceeds fp32
    const int up = 127 - s + down, half = up / 2;
    const float m0 = exp2i(half), m1 = exp2i(up - half);
    const size_t page = (size_t)dst * p.KV + g;
    uint8_t *to = (is_v ? p.to_v : p.to_k) + (page << p.to.page_log) * p.d;
    if (threadIdx.x == 0)
        (is_v ? p.to_v_scale : p.to_k_scale)[page] = (uint8_t)s;
    for (int i = threadIdx.x; i < n * (p.d / 4); i += COMPACT_THREADS) {
        const int r = i / (p.d / 4);
        if (!moved[r])
            continue;
        const float4 x = *reinterpret_cast<const float4 *>(rows + 4 * i);
        reinterpret_cast<uint32_t *>(to)[i] =
            e4m3x4_of(x.x * m0 * m1, x.y * m0 * m1, x.z * m0 * m1, x.w * m0 * m1);
    }
}

}  // namespace

namespace {

template <int THREADS>
cudaError_t launch_fork_t(const ForkParams &p, cudaStream_t stream)
{
    const size_t smem = (3 * (size_t)p.old_batch + 4 * (size_t)p.batch) * sizeof(int);
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = once_per_device(configured, [] {
        return cudaFuncSetAttribute(pages_fork_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    7 * kMaxForkBatch * (int)sizeof(int));
    });
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(pages_fork_kernel<THREADS>, dim3(FORK_CTAS), dim3(THREADS), smem, FORK_CTAS,
                                 stream, p);
}

}  // namespace

// A warp per row, new or old, as far as a CTA has them: fewer threads meet faster (32 sequences with
// the launch that copies: 8.2 us by 1024 threads, 6.8 by 256), more rows at a time are worth that
// (256 so: 10.7 and 14.7).
cudaError_t launch_pages_fork(const ForkParams &p, cudaStream_t stream)
{
    const int warps = (p.batch + p.old_batch + FORK_CTAS - 1) / FORK_CTAS;
    return warps <= 8    ? launch_fork_t<256>(p, stream)
           : warps <= 16 ? launch_fork_t<512>(p, stream)
                         : launch_fork_t<1024>(p, stream);
}

cudaError_t launch_pages_copy(const PageCopyParams &p, cudaStream_t stream)
{
    PageCopyParams q = p;
    q.chunks = (int)((p.page_bytes + COPY_BYTES - 1) / COPY_BYTES);
    const long long grid = (long long)p.n * q.chunks * (p.v ? 2 : 1);
    if (grid > INT_MAX)
        return cudaErrorInvalidConfiguration;
    return launch_kernel(pages_copy_kernel, dim3((unsigned)grid), dim3(COPY_THREADS), 0, stream, q);
}

cudaError_t launch_pages_compact(const CompactParams &p, bool e4m3, const RopeTurns &turns,
                                 cudaStream_t stream)
{
    // rows that a sequence can have: a loose bound costs no CTAs
    const long long rows = p.max_keep < p.to_positions ? p.max_keep : p.to_positions;
    // words of 8 elements where pairs, their start and the rest come in such
    const int unit = p.turn ? (p.rd | 2 * p.rot_start) & 15 : 0;
    if (e4m3) {
        const int page = 1 << p.to.page_log;
        const int blocks = (int)((rows + page - 1) / page);
        if ((long long)blocks * p.batch > INT_MAX)
            return cudaErrorInvalidConfiguration;
        const dim3 grid((unsigned)(blocks * p.batch), 2 * p.KV);
        const size_t smem = (size_t)page * p.d * sizeof(float);
        const auto kernel = unit ? pages_compact_e4m3_kernel<1> : pages_compact_e4m3_kernel<8>;
        static std::atomic<unsigned long long> configured{0};
        const cudaError_t e = once_per_device(configured, [] {
            const int most = 128 * 128 * sizeof(float);
            const cudaError_t r = cudaFuncSetAttribute(
                pages_compact_e4m3_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            return r != cudaSuccess ? r
                                    : cudaFuncSetAttribute(pages_compact_e4m3_kernel<1>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           most);
        });
        if (e != cudaSuccess)
            return e;
        return launch_kernel(kernel, grid, dim3(COMPACT_THREADS), smem, stream, p, turns, blocks);
    }
    const int blocks = (int)((rows + COMPACT_ROWS - 1) / COMPACT_ROWS);
    if ((long long)blocks * p.batch > INT_MAX)
        return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)COMPACT_ROWS * (p.turn ? p.rd / 2 : 0) * sizeof(float2);  // 8 KB at most
    return launch_kernel(unit ? pages_compact_kernel<1> : pages_compact_kernel<8>,
                         dim3((unsigned)(blocks * p.batch)), dim3(COMPACT_THREADS), smem, stream, p,
                         turns, blocks);
}
