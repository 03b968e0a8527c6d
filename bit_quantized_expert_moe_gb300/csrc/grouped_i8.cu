// Products of 8-bit expert weights with ragged segments of 8-bit rows, on the
// 5th-generation tensor cores (tcgen05, TMEM accumulators, TMA):
//   y[r][n] = sx[r] sw[e][n] sum_k x[r][k] W[e][n][k]     for the rows r of segment e
//
// The integer rate of the tensor cores here is 1/11 of the 16-bit one (153 against
// 1900 T), and an 8-bit code is a 16-bit float exactly: the products run in fp16,
// with fp32 sums, which are exact while they are within 2^24.  The weights stay 8-bit in memory and in
// shared memory and are widened into tensor memory, from where the MMA takes its A
// operand.  The rows' codes are widened once, in memory (every block of 256 weight rows
// reads them again), by warps of the same kernel, ahead of the tiles that need them, or
// where they are few by a kernel before.
//
// Tiles of 256 weight rows x (at most) 192 rows r by CTA pairs (2-SM clusters,
// cta_group::2), each CTA with its 128 weight rows and half of the rows r.  192 and
// not 256: two accumulators and two stages of A share the 512 columns of tensor memory.
//
// What bounds it: with many rows an expert the MMAs (one expert, 7296 rows, 4096 x 4096
// 130 us, 1888 TFLOP/s of the 1968 of a 16-bit library product); with few the weights'
// stream and their widening, whose chain of loads, arithmetic and stores a stage is as
// long as its copy (512 tokens over 256 experts of 7168 x 2048 640 us, 6.0 TB/s; 570 without
// the widening).  4096 Zipf-skewed tokens, 128 experts of 1536 x 2048: 167 us, 197 with the
// rows widened by a kernel before.  Tried: 16 widening warps 174 and 711 us (skewed,
// large); two sets of four that take every second stage 196 and 679 for 192 and 671;
// four stages of A for tiles of 128 columns: no change.
//
// Warp roles (576 threads a CTA): 0 TMA producer, 1 TMEM owner and (even CTA) MMA
// issuer, 4-11 widen the weights (warp w: TMEM lanes 32 (w % 4) .. + 31, either half
// of a stage's 128 k), 12-15 epilogue (the same lanes), 2, 3, 16 and 17 widen rows.
// Rows: units of 16 KB of a tile's rows, in the order of the tiles, taken from a counter by
// CTAs that run already (a tile's copies wait for its units, and these for no CTA that
// may not have started: another kernel may hold its SM).  A unit done is counted for
// its tile; the counters are cleared by a kernel before.
// Barriers: wfull[s] a CTA's own weights have landed; xfull[s] (even CTA) both CTAs'
// rows have; afull[a] (even CTA) both CTAs' warps have widened a stage; empty[s],
// aempty[a] and accfull[b] are signalled to both CTAs by the MMAs' completion, which
// follows the widening; accempty[b] (even CTA) counts both epilogues' warps.  Every
// waiter waits for every round of a barrier that it uses, in order.  Every wait is
// bounded in time: one that gives up sets the error word and every role leaves its loop.
#include "device_value.h"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int BM = 128;      // weight rows of a CTA (256 a pair)
constexpr int BN = 192;      // most rows r of a tile
constexpr int BL = 128;      // k of a stage: one 128-byte swizzle row of codes, two of fp16
constexpr int W_BYTES = BM * BL;
constexpr int OUT_BYTES = 32 * 80;  // an epilogue warp's block on its way out: 32 rows of 32 columns, 16 bytes apart
constexpr int THREADS = 576;
constexpr int ROW_WARPS = 4;
constexpr int WIDEN_WARP0 = 4, WIDEN_WARPS = 8, EP_WARP0 = 12, EP_WARPS = 4;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t A_COL = 2 * BN, A_COLS = BL / 2;  // two stages of A behind the accumulators
static_assert(A_COL + 2 * A_COLS <= TMEM_COLS, "tensor memory");
// Tiles of up to COLS rows r: the ring's stages are deeper where those are few and the
// weights' stream is all that counts (two stages are being widened or multiplied: at five
// no more than 48 KB of weights would be under way).
template <int COLS>
struct Ring {
    static constexpr int X_BYTES = COLS / 2 * 64 * 2;  // 64 k of a CTA's rows
    static constexpr int STAGE_BYTES = W_BYTES + 2 * X_BYTES, STAGES = COLS > 64 ? 5 : 8;
    static constexpr int BYTES = STAGES * STAGE_BYTES + EP_WARPS * OUT_BYTES;
    static constexpr int NBAR = 3 * STAGES + 8, OFF_SUMS = 8 * NBAR + 8;
    static constexpr int BAR_BYTES = OFF_SUMS + 4 * (THREADS / 32) + 8;  // and the unit taken
    static size_t smem(int E) { return 1024 + (size_t)BYTES + BAR_BYTES + 4 * ((size_t)E + 1); }
};

struct Params {
    int R, E, N, K;
    const int32_t* offsets;
    const float *x_scale, *w_scale;
    uint16_t* y;
    bool bf16;
    int tile_cols;  // most rows r of a tile
    uint32_t* err;
    const int8_t* x;
    uint16_t* x16;
    int* counts;    // units taken; units done of every row tile; null: the rows are there
    int unit_rows;  // rows of a unit
};

__device__ __forceinline__ bool segment(const Params& p, int e, int& r0, int& cnt) {
    const int i = __ldg(p.offsets + e), j = __ldg(p.offsets + e + 1);
    const bool ok = i >= 0 && i <= j && j <= p.R;
    r0 = ok ? i : 0;
    cnt = ok ? j - i : 0;
    return ok;
}

// One tile of the output: rows c0 .. c0 + ncols - 1, weight rows from m0.
struct Item {
    int e, m0, c0, ncols;
};
struct Work {
    int mb, items;
    const int* tile_pre;  // row tiles before each expert, [E + 1]
    __device__ int tiles(const Params& p) const { return tile_pre[p.E]; }
    __device__ Item item(const Params& p, int i) const {
        Item t;
        const int tile = i / mb;
        t.m0 = (i - tile * mb) * 2 * BM;
        int lo = 0, hi = p.E - 1;  // the expert whose row tiles include `tile`
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tile_pre[mid + 1] <= tile) lo = mid + 1;
            else hi = mid;
        }
        t.e = lo;
        int r0, cnt;
        segment(p, t.e, r0, cnt);
        // the segment's units of 16 rows are spread evenly over its tiles
        const int nt = tile_pre[lo + 1] - tile_pre[lo], k = tile - tile_pre[lo];
        const int units = (cnt + 15) >> 4, each = units / nt, more = units - each * nt;
        const int u0 = k * each + min(k, more);
        t.c0 = r0 + 16 * u0;
        t.ncols = min(16 * (each + (k < more)), cnt - 16 * u0);
        return t;
    }
};
__device__ __forceinline__ int mma_cols(const Item& t) { return (t.ncols + 15) & ~15; }

// Four codes as two pairs of fp16: a byte c + 128 in the mantissa of 1024 is
// 1152 + c, exactly.
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
    c ^= 0x80808080u;
    lo = hsub2_u32(__byte_perm(c, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_u32(__byte_perm(c, 0x64646464u, 0x4342), 0x64806480u);
}

// Rows that other CTAs have widened with ordinary stores, about to be copied by TMA.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ int units_done(const int* count) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
    return v;
}
__device__ __forceinline__ bool wait_units(const int* count, int units, volatile int* abort_flag, uint32_t* err) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1; units_done(count) < units; ++it)
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > tc::WAIT_LIMIT_NS) {
                *abort_flag = 1;
                set_error(err, ERRBIT_TIMEOUT);
                return false;
            }
        }
    return true;
}

__device__ __forceinline__ void widen16(const uint4& w, uint4* out) {
    uint4 a, b;
    widen4(w.x, a.x, a.y);
    widen4(w.y, a.z, a.w);
    widen4(w.z, b.x, b.y);
    widen4(w.w, b.z, b.w);
    out[0] = a;
    out[1] = b;
}

constexpr int BOXES = BN / 32;  // a CTA's half of a tile is 8 .. 96 rows; map i has boxes of 16 (i + 1) rows
struct Maps {
    CUtensorMap w, x[BOXES];
};

template <int COLS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    grouped_i8_tc_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Ring<COLS>;
    constexpr int STAGES = L::STAGES, STAGE_BYTES = L::STAGE_BYTES, X_BYTES = L::X_BYTES;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + L::BYTES;
    const uint32_t bar_wfull = bars, bar_xfull = bars + 8 * STAGES, bar_empty = bars + 16 * STAGES;
    const uint32_t bar_afull = bars + 24 * STAGES, bar_aempty = bar_afull + 16;
    const uint32_t bar_accfull = bar_afull + 32, bar_accempty = bar_afull + 48;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + L::BYTES + 8 * L::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* warp_sums = reinterpret_cast<int*>(gbase + L::BYTES + L::OFF_SUMS);
    int* tile_pre = reinterpret_cast<int*>(gbase + L::BYTES + L::BAR_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    grid_dependency_launch();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(bar_wfull + 8 * s, 1);
            tc::mbar_init(bar_xfull + 8 * s, 1);
            tc::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(bar_afull + 8 * b, 2 * WIDEN_WARPS);
            tc::mbar_init(bar_aempty + 8 * b, 1);
            tc::mbar_init(bar_accfull + 8 * b, 1);
            tc::mbar_init(bar_accempty + 8 * b, 2 * EP_WARPS);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    // the maps that the tiles may use (see launch)
    if (warp == 3 && lane <= p.tile_cols / 32) tc::tma_prefetch_desc(lane ? &maps.x[lane - 1] : &maps.w);
    if (warp == 1) {
        tc::tmem_alloc_pair(smem_u32((const void*)tmem_slot), TMEM_COLS);
        tc::tmem_relinquish_pair();
    }
    // both CTAs' barriers are initialised and the tensor memory allocated
    // before either CTA signals the other
    tc::tc_fence_before();
    __syncwarp();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the kernels before this one in the stream are complete: from here on
    // global memory is read and written
    grid_dependency_wait();
    // the segments, two experts a thread: row tiles before each expert; with one out
    // of place there is nothing to do (overlapping ones could add up to any number)
    constexpr int PER = 2;
    static_assert(PER * THREADS >= 1024, "too few threads for the experts");
    const int e0 = threadIdx.x * PER;
    int cnt[PER], sum = 0;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        int r0 = 0;
        cnt[k] = 0;
        if (e0 + k < p.E) bad |= !segment(p, e0 + k, r0, cnt[k]);
        cnt[k] = (cnt[k] + p.tile_cols - 1) / p.tile_cols;
        sum += cnt[k];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) warp_sums[warp] = before;
    bad = __syncthreads_or(bad);
    before -= sum;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) before += w < warp ? warp_sums[w] : 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (e0 + k < p.E) tile_pre[e0 + k] = before;
        before += cnt[k];
        if (e0 + k == p.E - 1) tile_pre[p.E] = before;
    }
    if (threadIdx.x == 0 && blockIdx.x == 0 && bad) set_error(p.err, ERRBIT_RANGE);
    __syncthreads();
    Work work;
    work.mb = ceil_div(p.N, 2 * BM);
    work.tile_pre = tile_pre;
    work.items = bad ? 0 : tile_pre[p.E] * work.mb;
    const int blocks = ceil_div(p.K, BL);  // stages of a tile

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (tc::elect_one()) {
            const uint32_t xfull_lead = tc::mapa_shared(bar_xfull, 0);
            int s = 0, g = 0;  // stage, stages issued so far
            uint32_t phase = 1;
            bool ok = true;
            // The next tile is looked up while the ring is full, not between two tiles
            // (offsets, a search and a look at its rows: 0.7 us of a tile's 6).
            Item t{}, to{};
            bool there = !p.counts;  // the tile's rows
            if (pair < work.items) t = work.item(p, pair);
            for (int i = pair; ok && i < work.items; i += npairs, t = to) {
                if (!there) ok = wait_units(p.counts + 1 + i / work.mb, ceil_div(t.ncols, p.unit_rows), abort_flag, p.err);
                if (!ok) break;
                if (p.counts) fence_proxy_async_global();
                there = !p.counts;
                const int half = mma_cols(t) >> 1, bi = (half + 15) / 16 - 1, xbytes = (bi + 1) * 16 * 128;
                const int m = t.m0 + (int)rank * BM, c = t.c0 + (int)rank * half;
                for (int j = 0; j < blocks; ++j, ++g) {
                    ok = tc::mbar_wait(bar_empty + 8 * s, phase, abort_flag, p.err);
                    if (!ok) break;
                    const uint32_t sw = base + s * STAGE_BYTES, sx = sw + W_BYTES;
                    const bool two = BL * j + 64 < p.K;
                    tc::mbar_arrive_expect_tx(bar_wfull + 8 * s, W_BYTES);
                    tc::tma_load_3d(sw, &maps.w, bar_wfull + 8 * s, BL * j, m, t.e);
                    if (rank == 0) tc::mbar_arrive_expect_tx(bar_xfull + 8 * s, (two ? 4 : 2) * xbytes);
                    tc::tma_load_2d_pair(sx, &maps.x[bi], xfull_lead + 8 * s, BL * j, c);
                    if (two) tc::tma_load_2d_pair(sx + X_BYTES, &maps.x[bi], xfull_lead + 8 * s, BL * j + 64, c);
                    if (j == min(STAGES, blocks) - 1 && i + npairs < work.items) {
                        to = work.item(p, i + npairs);
                        if (p.counts) there = units_done(p.counts + 1 + (i + npairs) / work.mb) >= ceil_div(to.ncols, p.unit_rows);
                    }
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the MMAs have read every stage, so every copy has landed
            for (int k = max(0, g - STAGES); ok && k < g; ++k)
                ok = tc::mbar_wait(bar_empty + 8 * (k % STAGES), (uint32_t)(k / STAGES) & 1u, abort_flag, p.err);
        }
    } else if (warp == 1) {
        // -------------------------------------- MMA issuer (even CTA of the pair)
        if (rank == 0 && tc::elect_one()) {
            int s = 0, ic = 0, g = 0;
            uint32_t phase = 0;
            bool ok = true;
            int cols = pair < work.items ? mma_cols(work.item(p, pair)) : 0;  // (the next tile's: as above)
            for (int i = pair; ok && i < work.items; i += npairs, ++ic) {
                const uint32_t idesc = tc::idesc_16_f32(2 * BM, cols, 0, false, false);
                const int b = ic & 1;
                // both CTAs' epilogues have read the accumulator
                ok = tc::mbar_wait_cluster(bar_accempty + 8 * b, ((uint32_t)(ic >> 1) & 1u) ^ 1u, abort_flag, p.err);
                if (!ok) break;
                const uint32_t d = tmem_base + (uint32_t)(BN * b);
                for (int j = 0; j < blocks; ++j, ++g) {
                    const int a = g & 1;
                    ok = tc::mbar_wait_cluster(bar_xfull + 8 * s, phase, abort_flag, p.err) &&
                         tc::mbar_wait_cluster(bar_afull + 8 * a, (uint32_t)(g >> 1) & 1u, abort_flag, p.err);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t sx = base + s * STAGE_BYTES + W_BYTES, da = tmem_base + A_COL + A_COLS * a;
                    const uint64_t db0 = tc::sw128_kmajor_desc(sx), db1 = tc::sw128_kmajor_desc(sx + X_BYTES);
                    const int left = p.K - BL * j;
#pragma unroll
                    for (int k = 0; k < BL / 16; ++k)
                        if (k == 0 || 16 * k < left)
                            tc::mma_f16_tmem_a_pair(d, da + 8 * k, (k < 4 ? db0 : db1) + 2 * (k & 3), idesc, k > 0 || j > 0);
                    tc::mma_commit_pair(bar_empty + 8 * s);
                    tc::mma_commit_pair(bar_aempty + 8 * a);
                    if (j == blocks - 1) tc::mma_commit_pair(bar_accfull + 8 * b);
                    if (j == 0 && i + npairs < work.items) cols = mma_cols(work.item(p, i + npairs));
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= WIDEN_WARP0 && warp < EP_WARP0) {
        // --------------------------------------- weights into tensor memory
        const int q = warp & 3, half = (warp - WIDEN_WARP0) >> 2;  // lanes; k 64 half .. + 63
        const uint32_t afull_lead = tc::mapa_shared(bar_afull, 0);
        const uint32_t row = (uint32_t)(32 * q + lane);
        const uint32_t t_a = tmem_base + A_COL + 32u * half + ((uint32_t)(32 * q) << 16);
        int s = 0, g = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = pair; ok && i < work.items; i += npairs) {
            for (int j = 0; j < blocks; ++j, ++g) {
                const int a = g & 1;
                ok = tc::mbar_wait(bar_wfull + 8 * s, phase, abort_flag, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // 64 codes of this thread's row: 16-byte piece c lies at c ^ (row % 8)
                const uint32_t src = base + s * STAGE_BYTES + row * 128;
                uint4 w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w[c].x), "=r"(w[c].y), "=r"(w[c].z), "=r"(w[c].w)
                                 : "r"(src + (((uint32_t)(4 * half + c) ^ (row & 7)) << 4)) : "memory");
                uint32_t v[2][16];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t(&o)[16] = v[c >> 1];
                    const int k = 8 * (c & 1);
                    widen4(w[c].x, o[k], o[k + 1]);
                    widen4(w[c].y, o[k + 2], o[k + 3]);
                    widen4(w[c].z, o[k + 4], o[k + 5]);
                    widen4(w[c].w, o[k + 6], o[k + 7]);
                }
                ok = tc::mbar_wait(bar_aempty + 8 * a, ((uint32_t)(g >> 1) & 1u) ^ 1u, abort_flag, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::tc_fence_after();
                tc::tmem_st_32x32b_x16(t_a + A_COLS * a, v[0]);
                tc::tmem_st_32x32b_x16(t_a + A_COLS * a + 16, v[1]);
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(afull_lead + 8 * a);
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp < WIDEN_WARP0 || warp >= EP_WARP0 + EP_WARPS) {
        // ------------------------------------------------------- rows, in memory
        volatile int* taken = reinterpret_cast<volatile int*>(warp_sums + THREADS / 32);
        const int tid = 32 * (warp < WIDEN_WARP0 ? warp - 2 : warp - (EP_WARP0 + EP_WARPS) + 2) + lane;
        const int per = ceil_div(p.tile_cols, p.unit_rows), units = p.counts && work.items ? work.tiles(p) * per : 0;
        // One thread takes units, the next while one is under way (and no more after a
        // wait that gave up: the others may see the flag at another time).
        int next = units;
        if (tid == 0 && units) next = atomicAdd(p.counts, 1);
        for (;;) {
            if (tid == 0) *taken = next;
            asm volatile("bar.sync 1, %0;" :: "n"(32 * ROW_WARPS) : "memory");
            const int u = *taken;
            if (u >= units) break;
            if (tid == 0) next = *abort_flag ? units : atomicAdd(p.counts, 1);
            const int tile = u / per;
            const Item t = work.item(p, tile * work.mb);
            const int r0 = (u - tile * per) * p.unit_rows, rows = min(p.unit_rows, t.ncols - r0);
            if (rows > 0) {
                constexpr int AHEAD = 8, STEP = 32 * ROW_WARPS;
                const size_t first = (size_t)(t.c0 + r0) * p.K / 16;  // pieces of 16 codes
                const uint4* src = reinterpret_cast<const uint4*>(p.x) + first;
                uint4* dst = reinterpret_cast<uint4*>(p.x16) + 2 * first;
                const int n = rows * (p.K / 16);
                for (int i = tid; i < n; i += AHEAD * STEP) {
                    uint4 w[AHEAD];
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k)
                        if (i + k * STEP < n) w[k] = __ldg(src + i + k * STEP);
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k)
                        if (i + k * STEP < n) widen16(w[k], dst + 2 * (i + k * STEP));
                }
                fence_proxy_async_global();
            }
            // all of the unit is written, and `taken` read
            asm volatile("bar.sync 1, %0;" :: "n"(32 * ROW_WARPS) : "memory");
            if (tid == 0 && rows > 0)
                asm volatile("red.release.gpu.global.add.s32 [%0], 1;" :: "l"(p.counts + 1 + tile) : "memory");
        }
    } else if (warp >= EP_WARP0) {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3;
        const uint32_t accempty_lead = tc::mapa_shared(bar_accempty, 0);
        const uint32_t t_lane = (uint32_t)(32 * q) << 16;
        const uint32_t buf = base + STAGES * STAGE_BYTES + (warp - EP_WARP0) * OUT_BYTES;
        int ic = 0;
        for (int i = pair; i < work.items; i += npairs, ++ic) {
            const Item t = work.item(p, i);
            const int m = t.m0 + (int)rank * BM + 32 * q + lane;  // this thread's weight row
            const int b = ic & 1;
            const float sw = m < p.N ? __ldg(p.w_scale + (size_t)t.e * p.N + m) : 0.f;
            const bool ok = tc::mbar_wait(bar_accfull + 8 * b, (uint32_t)(ic >> 1) & 1u, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc::tc_fence_after();
            const int cols = ceil_div(t.ncols, 32);
            for (int cb = 0; cb < cols; ++cb) {
                const int n = min(32, t.ncols - 32 * cb);
                const float sx = lane < n ? __ldg(p.x_scale + t.c0 + 32 * cb + lane) : 0.f;
                uint32_t v[32];
                tc::tmem_ld_32x32b_x32(tmem_base + (uint32_t)(BN * b) + 32u * cb + t_lane, v);
                tc::tmem_ld_wait();
                // D holds the output transposed: this thread's column m of 32 rows.
                // Through shared memory into 64 bytes of a row by 4 lanes.
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float f = __uint_as_float(v[j]) * sw * __shfl_sync(0xffffffffu, sx, j);
                    asm volatile("st.shared.b16 [%0], %1;"
                                 :: "r"(buf + 80 * j + 2 * lane), "h"(p.bf16 ? float_to_bf16_bits(f) : float_to_f16_bits(f)) : "memory");
                }
                __syncwarp();
                const int mc = m - lane + 8 * (lane & 3);  // this lane's 8 columns
                uint16_t* o = p.y + (size_t)(t.c0 + 32 * cb) * p.N + mc;
                const int rows = mc < p.N ? n : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 8 * j + (lane >> 2);
                    if (r < rows) {
                        uint4 w;
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(buf + 80 * r + 16 * (lane & 3)) : "memory");
                        *reinterpret_cast<uint4*>(o + (size_t)r * p.N) = w;
                    }
                }
                __syncwarp();
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(accempty_lead + 8 * b);
        }
    }

    // A wait that gave up: copies and MMAs that were issued finish well inside
    // this time.  Otherwise nothing is in flight here.
    __syncwarp();
    if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {}
    }
    // neither CTA frees its tensor memory or exits while the other may still
    // signal its barriers or use its memory
    __syncwarp();
    tc::tc_fence_before();
    tc::cluster_sync();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// The rows' codes as fp16, 16 a thread and step, before the product's kernel.
__global__ void __launch_bounds__(256) widen_rows_kernel(const int8_t* __restrict__ x, uint16_t* __restrict__ out, size_t n16) {
    grid_dependency_launch();
    grid_dependency_wait();
    const size_t step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16; i += step)
        widen16(__ldg(reinterpret_cast<const uint4*>(x) + i), reinterpret_cast<uint4*>(out) + 2 * i);
}

__global__ void __launch_bounds__(256) clear_counts_kernel(int* counts, int n) {
    grid_dependency_launch();
    grid_dependency_wait();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) counts[i] = 0;
}

int sm_pairs() { return std::max(1, num_sms() / 2); }

// Tiles of `cols` rows r when all experts have the same rows, or the most that there can be.
int tile_count(const GroupedI8Shape& g, int cols, bool even) {
    const int used = std::min(g.R, g.E);  // experts with rows
    const long long tiles = even ? (long long)used * ceil_div(ceil_div(g.R, used), cols) : g.R / cols + used;
    return (int)std::min<long long>(INT32_MAX, tiles * ceil_div(g.N, 2 * BM));
}
// Rows r of a tile: 192, 128 or 64, by the rounds of tiles times what a pair receives
// for one (256 bytes of codes and two for each row r).
int tile_columns(const GroupedI8Shape& g, int pairs) {
    int best = BN;
    long long least = INT64_MAX;
    for (int cols = BN; cols >= 64; cols -= 64) {
        const int all = ceil_div(g.R, std::min(g.R, g.E)), width = ceil_div(all, ceil_div(all, cols));
        const long long cost = (long long)ceil_div(tile_count(g, cols, true), pairs) * (BM + width);
        if (cost < least || (cols == 64 && all <= 64)) {
            least = cost;
            best = cols;
        }
    }
    return best;
}

// Most row tiles; the counters lie behind the widened rows.
int row_tiles(const GroupedI8Shape& g, int cols) { return g.R / cols + std::min(g.R, g.E); }
int* counts_of(const GroupedI8Shape& g) { return reinterpret_cast<int*>(g.x16 + (size_t)g.R * g.K); }

template <int COLS>
cudaError_t launch_tc(const GroupedI8Shape& g, const GroupedI8Data& d, int cols, bool first, cudaStream_t s) {
    Maps maps;
    const uint64_t wd[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E}, ws[2] = {(uint64_t)g.K, (uint64_t)g.N * g.K};
    const uint32_t wb[3] = {BL, BM, 1};
    bool ok = make_tensor_map_8(&maps.w, d.w, 3, wd, ws, wb);
    const uint64_t xd[2] = {(uint64_t)g.K, (uint64_t)g.R}, xs[1] = {(uint64_t)g.K * 2};
    for (int i = 0; i < cols / 32 && ok; ++i) {
        const uint32_t xb[2] = {64, (uint32_t)(i + 1) * 16};
        ok = make_tensor_map_16(&maps.x[i], false, g.x16, 2, xd, xs, xb);
    }
    if (!ok) return cudaErrorInvalidValue;
    static DeviceValue pairs;  // CTA pairs that the GPU holds at once
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int max_pairs = pairs.get(dev, [] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() & ~1));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = Ring<COLS>::smem(1024);
        int nc = 0;
        if (allow_smem<grouped_i8_tc_kernel<COLS>>() != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&nc, grouped_i8_tc_kernel<COLS>, &cfg) != cudaSuccess || nc < 1) {
            (void)cudaGetLastError();
            nc = sm_pairs();
        }
        return nc;
    });
    const Params p{g.R, g.E, g.N, g.K, g.offsets, d.x_scale, d.w_scale, static_cast<uint16_t*>(d.y),
                   g.out == MOE_DT_BF16, cols, g.err, d.x, g.x16, first ? nullptr : counts_of(g), std::max(1, std::min(32, 16384 / g.K))};
    const int grid = 2 * std::max(1, std::min(max_pairs, tile_count(g, cols, false)));
    return launch_overlapped<grouped_i8_tc_kernel<COLS>>(dim3(grid), dim3(THREADS), Ring<COLS>::smem(g.E), s, maps, p);
}
cudaError_t launch_tc(const GroupedI8Shape& g, const GroupedI8Data& d, cudaStream_t s) {
    const int cols = tile_columns(g, sm_pairs()), n = 1 + row_tiles(g, cols);
    // Few rows are widened by a kernel before, which takes less than the first tiles' wait
    // for their units; many by the same kernel.  Either way (us), by pieces of 16 codes:
    // 2^14.4 1238 rows, 8 experts of 520 x 272 6.9, 8.5; 2^15 512 rows, 16 of 2048 x 1024 12.3,
    // 14.0; 2^16 512 rows, 128 of 1536 x 2048 76.6, 75.6; 2^17.6 12000 rows, 8 of 520 x 272 19.0,
    // 19.5; 2^17.8 512 rows, 256 of 2048 x 7168 527, 516; 2^18 4096 rows, 16 of 2048 x 1024 24.6,
    // 25.0, 2048 rows, 128 of 1536 x 2048 83.0, 80.4; 2^19 4096 of these 85.9, 83.1, 8192 rows,
    // 16 of 2048 x 1024 43.0, 41.9.  From 2^16 to 2^18 many experts lose up to 3 % by it, few
    // gain as much.
    const size_t n16 = (size_t)g.R * g.K / 16;
    const bool first = n16 <= (1 << 18);
    const cudaError_t e = first ? launch_overlapped(widen_rows_kernel, std::max(1, ceil_div((int)n16, 256)), 256, 0, s, d.x, g.x16, n16)
                                : launch_overlapped(clear_counts_kernel, std::min(ceil_div(n, 256), 16), 256, 0, s, counts_of(g), n);
    if (e != cudaSuccess) return e;
    return cols > 64 ? launch_tc<BN>(g, d, cols, first, s) : launch_tc<64>(g, d, cols, first, s);
}

}  // namespace

// Up to 32 rows, or 128 where they are no more than the experts, go to the kernel for few
// rows.  Spread by chance over 128 experts of 1536 x 2048, 128 rows take 41.8 us there and 129
// by this kernel 52.9; all at one expert 14.6 and 11.5, which the sizes do not tell.
static bool takes_few(int R, int E) { return R <= 32 || (R <= 128 && R <= E); }

size_t grouped_i8_halves(int R, int E, int N, int K) {
    (void)N;
    return R <= 32 ? 0 : (size_t)R * K + 2 * (1 + (size_t)R / 64 + std::min(R, E));
}
cudaError_t launch_grouped_i8(const GroupedI8Shape& g, const GroupedI8Data& d, cudaStream_t s) {
    return takes_few(g.R, g.E) ? launch_grouped_i8_few(g, d, s) : launch_tc(g, d, s);
}

}  // namespace moe
