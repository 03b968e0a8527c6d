// Products of 16-bit expert weights with ragged row segments, on the
// 5th-generation tensor cores (tcgen05, TMEM accumulators, TMA).
//
// Segment e is rows offsets[e] .. offsets[e+1]-1.
//   Y    y[r][n]     = sum_k x[r][k] W[e][n][k]
//   DX   dx[r][k]    = sum_n dy[r][n] W[e][n][k]
//   DW   dW[e][n][k] = sum_{r in e} dy[r][n] x[r][k]
//
// The three are one kernel: D[m][c] = sum_l A[m][l] B[c][l] in tiles of 256 x
// (at most) 256, by CTA pairs (2-SM clusters, cta_group::2): each CTA holds its
// 128 rows of A and half of B, so an SM receives 32 KB for 64 l instead of the
// 48 KB that one CTA alone would need for the same 2 x 128 x 256 products.
//         m            c           l                 A            B
//   Y     weight row n row r       k                 W   K-major  x   K-major
//   DX    weight col k row r       n                 W   MN-major dy  K-major
//   DW    n            k           row r of segment  dy  MN-major x   MN-major
// MN-major operands are read by the tensor core from the rows as TMA brings
// them (descriptor with the transpose bit): nothing is transposed in memory.
// The weights are M in Y and DX, so that a tile of few rows costs an MMA of
// few columns (a multiple of 16) and not an M of 128 that is mostly padding:
// with 16 rows an expert the weights' bytes are all that counts.
// Widths that are no multiple of a tile: TMA fills zeros out of bounds.  Rows
// behind a segment belong to the next expert: in Y and DX they are columns of
// D that are not stored; in DW they would be summed, so the rows up to the next
// multiple of 16 are set to zero in shared memory and no MMA reads further.
//
// Warp roles (384 threads a CTA): 0 TMA producer, 1 TMEM owner and (even CTA)
// MMA issuer, 2 (DW) ragged ends, 4-11 epilogue (warp w: TMEM lanes
// 32 (w % 4) .. + 31, every second block of columns).  Two accumulators: the
// epilogue of a tile runs beside the MMAs of the next.
// Barriers: both CTAs' copies complete on the even CTA's full[s].  DW: where a
// segment ends inside 16 rows, the copies complete on each CTA's own tail[s]
// instead; its warp 2 clears the rows and both arrive on full[s], which counts
// two arrivals (otherwise both by the even CTA's producer).  empty[s] and
// accfull[b] are signalled to both CTAs by the MMAs' completion, accempty[b] of
// the even CTA counts both epilogues' warps.  A wait names a round of its barrier
// by the round's parity, so every waiter waits for every round of a barrier that
// it uses, in order.  Every wait is bounded in time: one that gives up sets the
// error word and every role leaves its loop.
#include "device_value.h"
#include "internal.h"
#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace moe {
namespace {

enum class Product { Y, DX, DW };

constexpr int BM = 128;             // A rows of a CTA (256 a pair)
constexpr int BN = 256;             // most columns of a tile
constexpr int BL = 64;              // l of a stage: one 128-byte swizzle row
constexpr int A_BYTES = BM * BL * 2;
constexpr int B_BYTES = BN / 2 * BL * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int ATOM64 = 64 * BL * 2;  // MN-major: 64 l rows of 64 elements
constexpr int STAGES = 6;
// DW: clearing the rows behind a segment takes longer than the ring is ahead
// of the MMAs, so a tile's ragged end is loaded first and used after this many of
// the tile's other stages (less than STAGES - 1: its stage is given back before
// the ring needs it).  Loaded and used last, 4096 tokens took 227 us.
constexpr int END_DEFER = 3;
// An epilogue warp's block on its way out: DW 32 rows of 64 columns; Y, DX 32 rows
// r of 32 columns, 16 bytes apart so that neighbouring rows use other banks.
template <Product PR>
constexpr int OUT_BYTES = PR == Product::DW ? 32 * 128 : 32 * 80;
constexpr int THREADS = 384;
constexpr int EP_WARP0 = 4, EP_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512;  // two accumulators of 256 columns
constexpr int NBAR = 3 * STAGES + 4;
constexpr size_t BAR_BYTES = 256;
static_assert(8 * NBAR + 8 <= 192 && 192 + THREADS / 8 <= BAR_BYTES, "barrier area too small");

template <Product PR>
constexpr int RING_BYTES = STAGES * STAGE_BYTES + EP_WARPS * OUT_BYTES<PR>;
// Y, DX: and the row tiles before each expert.
template <Product PR>
size_t smem_bytes(int E) {
    return 1024 + (size_t)RING_BYTES<PR> + BAR_BYTES + (PR == Product::DW ? 0 : 4 * ((size_t)E + 1));
}

struct GroupedParams {
    int R, E, N, K;
    const int32_t* offsets;
    void* out;
    uint32_t type;  // 0 fp16, 1 bf16
    int tile_cols;  // most columns of a tile
    int splits;     // shares of the summed index, each a tile of its own (SPLIT)
    float* part;    // [splits][R or E][...]: the output of every share in fp32
    uint32_t* err;
};

// Rows of segment e; false if it is not inside [0, R].
__device__ __forceinline__ bool segment(const GroupedParams& p, int e, int& r0, int& cnt) {
    const int i = __ldg(p.offsets + e), j = __ldg(p.offsets + e + 1);
    const bool ok = i >= 0 && i <= j && j <= p.R;
    r0 = ok ? i : 0;
    cnt = ok ? j - i : 0;
    return ok;
}

// One tile of the output.
struct Item {
    int e;
    int m0;        // first of the pair's 256 A rows
    int c0, ncols; // first column and how many (Y, DX: rows r; DW: k)
    int l0, nl;    // the summed index: first (DW: row) and how many
    int split;
};

template <Product PR, bool SPLIT>
struct Work {
    int mb;     // blocks of 256 A rows
    int cb;     // DW: blocks of 256 columns
    int items;
    const int* tile_pre;  // Y, DX: row tiles before each expert, [E + 1]

    __device__ Work(const GroupedParams& p, const int* pre, bool bad) : tile_pre(pre) {
        mb = ceil_div(PR == Product::DX ? p.K : p.N, 2 * BM);
        cb = ceil_div(p.K, p.tile_cols);
        items = bad ? 0 : PR == Product::DW ? p.E * mb * cb : pre[p.E] * mb;
        if (SPLIT) items *= p.splits;
    }
    __device__ Item item(const GroupedParams& p, int i) const {
        Item t;
        t.split = SPLIT ? i % p.splits : 0;
        if (SPLIT) i /= p.splits;
        if (PR == Product::DW) {
            const int per = mb * cb;
            t.e = i / per;
            i -= t.e * per;
            t.m0 = i / cb * 2 * BM;
            t.c0 = i % cb * p.tile_cols;
            t.ncols = min(p.tile_cols, p.K - t.c0);
            segment(p, t.e, t.l0, t.nl);
        } else {
            const int tile = i / mb;
            t.m0 = (i - tile * mb) * 2 * BM;
            // the expert whose row tiles include `tile`
            int lo = 0, hi = p.E - 1;
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
            t.l0 = 0;
            t.nl = PR == Product::DX ? p.N : p.K;
        }
        if (SPLIT) {  // shares of whole stages; the last ones may be empty
            const int share = ceil_div(ceil_div(t.nl, BL), p.splits) * BL, from = min(t.nl, t.split * share);
            t.l0 += from;
            t.nl = min(share, t.nl - from);
        }
        return t;
    }
};

// DW: whether `left` rows of a segment end inside 16 rows of a stage, which an
// MMA sums together.
__device__ __forceinline__ bool ragged_end(int left) { return left < BL && (left & 15); }

__device__ __forceinline__ int mma_cols(const Item& t) { return (t.ncols + 15) & ~15; }

// Boxes of B rows (Y, DX): a CTA's half of a tile is 8 .. 128 rows; map i has
// boxes of 16 (i + 1) rows.
constexpr int BOXES = 8;
struct Maps {
    CUtensorMap a, b[BOXES];  // DW: b[0], and b[1] the output
};

// SPLIT: where a few tiles sum long rows, their shares go to pairs that would
// have nothing to do, and grouped_sum_kernel adds the shares up.
template <Product PR, bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    grouped_tc_kernel(const __grid_constant__ Maps maps, const GroupedParams p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + RING_BYTES<PR>;
    const uint32_t bar_full = bars, bar_empty = bars + 8 * STAGES, bar_tail = bars + 16 * STAGES;
    const uint32_t bar_accfull = bars + 24 * STAGES, bar_accempty = bar_accfull + 16;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + RING_BYTES<PR> + 8 * NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* warp_sums = reinterpret_cast<int*>(gbase + RING_BYTES<PR> + 192);
    int* tile_pre = reinterpret_cast<int*>(gbase + RING_BYTES<PR> + BAR_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    grid_dependency_launch();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(bar_full + 8 * s, PR == Product::DW ? 2 : 1);
            tc::mbar_init(bar_empty + 8 * s, 1);
            tc::mbar_init(bar_tail + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(bar_accfull + 8 * b, 1);
            tc::mbar_init(bar_accempty + 8 * b, 2 * EP_WARPS);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    // the maps that the tiles may use (see launch)
    if (warp == 2 && lane <= p.tile_cols / 32) tc::tma_prefetch_desc(lane ? &maps.b[lane - 1] : &maps.a);
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
    // the segments, three experts a thread; with one out of place there is
    // nothing to do (overlapping ones could add up to any number of tiles)
    constexpr int PER = 3;
    static_assert(PER * THREADS >= 1024, "too few threads for the experts");
    const int e0 = threadIdx.x * PER;
    int cnt[PER];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        int r0 = 0;
        cnt[k] = 0;
        if (e0 + k < p.E) bad |= !segment(p, e0 + k, r0, cnt[k]);
    }
    if (PR == Product::DW) {
        bad = __syncthreads_or(bad);
    } else {
        // row tiles before each expert
        int sum = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
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
    }
    if (threadIdx.x == 0 && blockIdx.x == 0) {
        if (bad) set_error(p.err, ERRBIT_RANGE);
        if (SPLIT) p.err[WS_NO_SHARES_WORD] = bad;
    }
    __syncthreads();
    const Work<PR, SPLIT> work(p, tile_pre, bad);

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (tc::elect_one()) {
            const uint32_t full_lead = tc::mapa_shared(bar_full, 0);
            int s = 0, g = 0;  // stage, stages issued so far
            uint32_t phase = 1;
            bool ok = true;
            for (int i = pair; ok && i < work.items; i += npairs) {
                const Item t = work.item(p, i);
                const int half = mma_cols(t) >> 1;
                const int bi = PR == Product::DW ? 0 : (half + 15) / 16 - 1, box = (bi + 1) * 16;
                const CUtensorMap* mb = &maps.b[bi];
                const uint32_t bytes = 2 * (A_BYTES + (PR == Product::DW ? (half > 64 ? 2 : 1) * ATOM64 : box * BL * 2));
                const int m = t.m0 + (int)rank * BM, c = t.c0 + (int)rank * half;
                const int blocks = ceil_div(t.nl, BL);
                const bool end_first = PR == Product::DW && ragged_end(t.nl - BL * (blocks - 1));
                for (int j = 0; j < blocks; ++j, ++g) {
                    const int l = BL * (!end_first ? j : j == 0 ? blocks - 1 : j - 1);
                    ok = tc::mbar_wait(bar_empty + 8 * s, phase, abort_flag, p.err);
                    if (!ok) break;
                    const uint32_t sa = base + s * STAGE_BYTES, sb = sa + A_BYTES;
                    const uint32_t fl = full_lead + 8 * s, f = bar_full + 8 * s;
                    if (PR == Product::DW) {
                        uint32_t to = fl;
                        if (end_first && j == 0) {
                            to = tc::mapa_shared(bar_tail + 8 * s, rank);
                            tc::mbar_arrive_expect_tx(bar_tail + 8 * s, bytes >> 1);
                        } else if (rank == 0) {
                            tc::mbar_arrive_expect_tx(f, bytes);
                            tc::mbar_arrive(f);
                        }
                        tc::tma_load_2d_pair(sa, &maps.a, to, m, t.l0 + l);
                        tc::tma_load_2d_pair(sa + ATOM64, &maps.a, to, m + 64, t.l0 + l);
                        tc::tma_load_2d_pair(sb, mb, to, c, t.l0 + l);
                        if (half > 64) tc::tma_load_2d_pair(sb + ATOM64, mb, to, c + 64, t.l0 + l);
                    } else {
                        if (rank == 0) tc::mbar_arrive_expect_tx(f, bytes);
                        if (PR == Product::Y) {
                            tc::tma_load_3d_pair(sa, &maps.a, fl, t.l0 + l, m, t.e);
                        } else {
                            tc::tma_load_3d_pair(sa, &maps.a, fl, m, t.l0 + l, t.e);
                            tc::tma_load_3d_pair(sa + ATOM64, &maps.a, fl, m + 64, t.l0 + l, t.e);
                        }
                        tc::tma_load_2d_pair(sb, mb, fl, t.l0 + l, c);
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
            int s0 = 0, ic = 0;   // the tile's first stage
            uint32_t phase0 = 0;  // and its round's parity
            bool ok = true;
            for (int i = pair; ok && i < work.items; i += npairs) {
                const Item t = work.item(p, i);
                if (t.nl == 0) continue;
                const uint32_t idesc = tc::idesc_16_f32(2 * BM, mma_cols(t), p.type, PR != Product::Y, PR == Product::DW);
                const int b = ic & 1;
                // both CTAs' epilogues have read the accumulator
                ok = tc::mbar_wait_cluster(bar_accempty + 8 * b, ((uint32_t)(ic >> 1) & 1u) ^ 1u, abort_flag, p.err);
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t d = tmem_base + 256u * b;
                const int blocks = ceil_div(t.nl, BL), last = t.nl - BL * (blocks - 1);
                // a ragged end is the tile's first stage in the ring and its
                // (defer + 1)-th here
                const int defer = PR == Product::DW && ragged_end(last) ? min(blocks - 1, END_DEFER) : 0;
                int next = s0;
                uint32_t next_phase = phase0;
                auto advance = [&] {
                    if (++next == STAGES) {
                        next = 0;
                        next_phase ^= 1u;
                    }
                };
                if (defer) advance();
                for (int j = 0; j < blocks; ++j) {
                    const bool end = defer && j == defer;
                    const int s = end ? s0 : next;
                    const uint32_t phase = end ? phase0 : next_phase;
                    if (!end) advance();
                    ok = tc::mbar_wait_cluster(bar_full + 8 * s, phase, abort_flag, p.err);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t sa = base + s * STAGE_BYTES, sb = sa + A_BYTES;
                    constexpr uint32_t SA = PR == Product::Y ? 32 : 2048, SB = PR == Product::DW ? 2048 : 32;
                    const uint64_t da = PR == Product::Y ? tc::sw128_kmajor_desc(sa) : tc::sw128_mnmajor_desc(sa, ATOM64);
                    const uint64_t db = PR == Product::DW ? tc::sw128_mnmajor_desc(sb, ATOM64) : tc::sw128_kmajor_desc(sb);
                    const int left = end || (!defer && j == blocks - 1) ? last : BL;
                    // 16 l further: the start address, in units of 16 bytes
#pragma unroll
                    for (int k = 0; k < BL / 16; ++k)
                        if (k == 0 || 16 * k < left)
                            tc::mma_f16_pair(d, da + k * (SA >> 4), db + k * (SB >> 4), idesc, k > 0 || j > 0);
                    tc::mma_commit_pair(bar_empty + 8 * s);
                    if (j == blocks - 1) tc::mma_commit_pair(bar_accfull + 8 * b);
                }
                s0 = next;
                phase0 = next_phase;
                ++ic;
            }
        }
    } else if (PR == Product::DW && warp == 2) {
        // ------------------------- ragged ends: clears the rows behind a segment
        const uint32_t full_lead = tc::mapa_shared(bar_full, 0);
        int s = 0;            // the tile's first stage
        uint32_t phases = 0;  // of the tail barriers, which are not used in every round
        bool ok = true;
        for (int i = pair; ok && i < work.items; i += npairs) {
            const Item t = work.item(p, i);
            if (t.nl == 0) continue;
            const int blocks = ceil_div(t.nl, BL), left = t.nl - BL * (blocks - 1), end = (left + 15) & ~15;
            if (ragged_end(left)) {
                ok = tc::mbar_wait(bar_tail + 8 * s, (phases >> s) & 1u, abort_flag, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                phases ^= 1u << s;
                // rows left .. end-1 of the four blocks of 64 rows x 128 B
                unsigned char* st = gbase + s * STAGE_BYTES + (lane >> 3) * ATOM64 + (lane & 7) * 16;
                for (int row = left; row < end; ++row) *reinterpret_cast<uint4*>(st + row * 128) = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster_release(full_lead + 8 * s);
            }
            s = (s + blocks) % STAGES;
        }
    } else if (warp >= EP_WARP0) {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3, eh = (warp - EP_WARP0) >> 2;
        const uint32_t accempty_lead = tc::mapa_shared(bar_accempty, 0);
        const uint32_t t_lane = (uint32_t)(32 * q) << 16;
        const uint32_t buf = base + STAGES * STAGE_BYTES + (warp - EP_WARP0) * OUT_BYTES<PR>;
        const int M = PR == Product::DX ? p.K : p.N;
        uint16_t* const out = static_cast<uint16_t*>(p.out);
        int ic = 0;
        for (int i = pair; i < work.items; i += npairs) {
            const Item t = work.item(p, i);
            const int m = t.m0 + (int)rank * BM + 32 * q + lane;  // this thread's A row
            const int b = ic & 1;
            if (t.nl > 0) {
                const bool ok = tc::mbar_wait(bar_accfull + 8 * b, (uint32_t)(ic >> 1) & 1u, abort_flag, p.err);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::tc_fence_after();
            }
            if (SPLIT) {
                // fp32: DW 32 columns of this thread's row, Y and DX this thread's
                // column of 32 rows
                const int blocks = ceil_div(t.ncols, 32);
                for (int cb = eh; cb < blocks; cb += 2) {
                    uint32_t v[32];
                    if (t.nl > 0) {
                        tc::tmem_ld_32x32b_x32(tmem_base + 256u * b + 32u * cb + t_lane, v);
                        tc::tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0;
                    }
                    const int n = m < M ? min(32, t.ncols - 32 * cb) : 0;
                    if (PR == Product::DW) {
                        float* o = p.part + (((size_t)t.split * p.E + t.e) * M + m) * p.K + t.c0 + 32 * cb;
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (j < n) *reinterpret_cast<uint4*>(o + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    } else {
                        float* o = p.part + ((size_t)t.split * p.R + t.c0 + 32 * cb) * M + m;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < n) o[(size_t)j * M] = __uint_as_float(v[j]);
                    }
                }
            } else if (PR == Product::DW) {
                // 64 columns at a time: rows of 128 B, 128-byte swizzle, stored by TMA
                const int row0 = t.m0 + (int)rank * BM + 32 * q, blocks = ceil_div(t.ncols, 64);
                const uint32_t dst = buf + 128 * lane;
                for (int cb = eh; cb < blocks; cb += 2) {
                    uint32_t o[32];
                    if (t.nl > 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[32];
                            tc::tmem_ld_32x32b_x32(tmem_base + 256u * b + 64u * cb + 32u * h + t_lane, v);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float lo = __uint_as_float(v[2 * j]), hi = __uint_as_float(v[2 * j + 1]);
                                o[16 * h + j] = p.type ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0;
                    }
                    tc::bulk_wait_read();  // the lane that stores: the buffer has been read
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                                     :: "r"(dst + 16 * (j ^ (lane & 7))), "r"(o[4 * j]), "r"(o[4 * j + 1]), "r"(o[4 * j + 2]),
                                        "r"(o[4 * j + 3]) : "memory");
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (row0 < M && tc::elect_one()) {
                        tc::tma_store_3d(&maps.b[1], buf, t.c0 + 64 * cb, row0, t.e);
                        tc::bulk_commit();
                    }
                    __syncwarp();
                }
            } else {
                const int blocks = ceil_div(t.ncols, 32);
                for (int cb = eh; cb < blocks; cb += 2) {
                    uint32_t v[32];
                    tc::tmem_ld_32x32b_x32(tmem_base + 256u * b + 32u * cb + t_lane, v);
                    tc::tmem_ld_wait();
                    // D holds the output transposed: this thread's column m of 32
                    // rows.  Through shared memory into 64 bytes of a row by 4 lanes.
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float f = __uint_as_float(v[j]);
                        asm volatile("st.shared.b16 [%0], %1;"
                                     :: "r"(buf + 80 * j + 2 * lane), "h"(p.type ? float_to_bf16_bits(f) : float_to_f16_bits(f)) : "memory");
                    }
                    __syncwarp();
                    const int mc = m - lane + 8 * (lane & 3);  // this lane's 8 columns
                    uint16_t* o = out + (size_t)(t.c0 + 32 * cb) * M + mc;
                    const int n = mc < M ? min(32, t.ncols - 32 * cb) : 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = 8 * j + (lane >> 2);
                        if (row < n) {
                            uint4 w;
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(buf + 80 * row + 16 * (lane & 3)) : "memory");
                            *reinterpret_cast<uint4*>(o + (size_t)row * M) = w;
                        }
                    }
                    __syncwarp();
                }
            }
            if (t.nl > 0) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(accempty_lead + 8 * b);
                ++ic;
            }
        }
        if (PR == Product::DW && !SPLIT) tc::bulk_wait();
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

// The shares' sums, in order, rounded to the output: `row` values for each of
// `rows` rows, of which Y and DX write those that a segment holds.  Nothing where a
// segment is out of place.
__global__ void __launch_bounds__(256) grouped_sum_kernel(const GroupedParams p, int rows, int row) {
    grid_dependency_launch();
    grid_dependency_wait();
    const uint32_t none = p.err[WS_NO_SHARES_WORD];
    const int r0 = p.offsets ? __ldg(p.offsets) : 0, r1 = p.offsets ? __ldg(p.offsets + p.E) : rows;
    const size_t n = (size_t)rows * row / 8, step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        // the shares' loads do not wait for the words above
        V8 s = load8<F32>(p.part, i);
        for (int k = 1; k < p.splits; ++k) s = fma(load8<F32>(p.part, k * n + i), 1.f, s);
        const int r = (int)(i * 8 / row);
        if (none || r < r0 || r >= r1) continue;
        if (p.type) store8<Bf16>(p.out, i, s);
        else store8<F16>(p.out, i, s);
    }
}

bool map_2d(CUtensorMap* m, bool bf16, const void* ptr, int cols, int rows, int box_cols, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)cols * 2};
    const uint32_t box[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
    return make_tensor_map_16(m, bf16, ptr, 2, dims, strides, box);
}
bool map_w(CUtensorMap* m, bool bf16, const void* ptr, const GroupedShape& g, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E};
    const uint64_t strides[2] = {(uint64_t)g.K * 2, (uint64_t)g.N * g.K * 2};
    const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
    return make_tensor_map_16(m, bf16, ptr, 3, dims, strides, box);
}

int sm_pairs() { return std::max(1, num_sms() / 2); }

// Tiles of `cols` columns; Y, DX: when all experts have the same rows, or the
// most that there can be.
template <Product PR>
int tile_count(const GroupedShape& g, int cols, bool even) {
    if (PR == Product::DW) return g.E * ceil_div(g.N, 2 * BM) * ceil_div(g.K, cols);
    const int used = std::min(g.R, g.E);  // experts with rows
    const long long tiles = even ? (long long)used * ceil_div(ceil_div(g.R, used), cols) : g.R / cols + used;
    return (int)std::min<long long>(INT32_MAX, tiles * ceil_div(PR == Product::Y ? g.N : g.K, 2 * BM));
}

// Columns of a tile: 256, 128 or 64.  What an SM can receive bounds a pair (50
// bytes a clock), so the least of rounds of tiles x (256 rows of A + columns)
// is the best.  dw of 6624 rows of 2 experts, N 104, K 3616: 21.4, 20.7 and 36.2 us
// (58 tiles of 128, 114 of 64); of 512 rows, N and K 2048: 7.4, 8.0, 10.5; y of
// 3002 rows, N 648, K 896: 9.2, 7.6, 9.4; of 2208 of 3 experts, N 232, K 5608:
// 36.1, 27.4, 23.0.
template <Product PR>
int tile_columns(const GroupedShape& g, int pairs) {
    int best = BN;
    long long least = INT64_MAX;
    for (int cols = BN; cols >= 64; cols >>= 1) {
        const int all = PR == Product::DW ? g.K : ceil_div(g.R, std::min(g.R, g.E));
        const int width = ceil_div(all, ceil_div(all, cols));
        const long long cost = (long long)ceil_div(tile_count<PR>(g, cols, true), pairs) * (2 * BM + width);
        if (cost < least) {
            least = cost;
            best = cols;
        }
    }
    return best;
}

// Shares of the summed index for each tile.  A stage takes a pair 0.23 us; the
// sum's launch takes as long as about 16 of them.  One expert, 512 rows, N 256,
// K 7168: y 20.4 -> 9.9 us; 3851 rows, N 3064, K 96: dw 19.5 -> 12.7; two experts,
// 300 rows, N 5608, K 232: dx 27.2 -> 10.3; 70 rows, N 88, K 2072: y 9.4 -> 7.6.
int split_count(int pairs, int tiles, int stages) {
    const int most = std::min({pairs / tiles, stages / 8, 8});
    return most > 1 && stages - ceil_div(stages, most) >= 16 ? most : 1;
}
template <Product PR>
int tile_splits(const GroupedShape& g, int cols, int pairs) {
    const int stages = ceil_div(PR == Product::Y ? g.K : PR == Product::DX ? g.N : ceil_div(g.R, g.E), BL);
    return split_count(pairs, tile_count<PR>(g, cols, true), stages);
}
// fp32 values of the shares' outputs.
template <Product PR>
size_t split_floats(const GroupedShape& g, int pairs) {
    const int splits = tile_splits<PR>(g, tile_columns<PR>(g, pairs), pairs);
    return splits == 1 ? 0 : (size_t)splits * (PR == Product::DW ? (size_t)g.E * g.N : g.R) * (PR == Product::Y ? g.N : g.K);
}

// No fewer than the shares of a product with R x M outputs, summed over L, take for
// these rows or any smaller number of them (dW's never become fewer with the rows).
// r rows fill at least min(r, E) rows of tiles, mb tiles each, and the shares with
// all tiles are at most the pairs: up to E rows they take pairs / mb x M values,
// beyond that what the tiles can hold.
size_t rows_floats_bound(const GroupedShape& g, int M, int L, int pairs) {
    const int mb = ceil_div(M, 2 * BM), stages = ceil_div(L, BL), used = std::min(g.R, g.E);
    const size_t most = split_count(pairs, 1, stages);
    if (most == 1) return 0;
    const size_t few = std::min(most * used, (size_t)pairs / mb) * M;
    const size_t splits = std::min<size_t>(most, pairs / std::max(1, std::min(pairs, g.E * mb)));
    if (g.R <= g.E || splits < 2) return few;
    return std::max(few, std::min(splits * g.R * M, (size_t)pairs * 2 * BM * BN));
}

template <Product PR, bool SPLIT>
cudaError_t launch(const GroupedShape& g, const void* a, const void* b, void* out, int cols, int splits, cudaStream_t s) {
    const bool bf = g.dtype == MOE_DT_BF16;
    Maps maps;
    bool ok;
    const int items = tile_count<PR>(g, cols, false);
    if (PR == Product::DW) {
        ok = map_2d(&maps.a, bf, a, g.N, g.R, 64, 64) && map_2d(&maps.b[0], bf, b, g.K, g.R, 64, 64) &&
             map_w(&maps.b[1], bf, out, g, 32);
        for (int i = 2; i < BOXES; ++i) maps.b[i] = maps.b[0];
    } else {
        const int L = PR == Product::Y ? g.K : g.N;
        ok = map_w(&maps.a, bf, a, g, PR == Product::Y ? BM : 64);
        for (int i = 0; i < cols / 32 && ok; ++i) ok = map_2d(&maps.b[i], bf, b, L, g.R, 64, (i + 1) * 16);
    }
    if (!ok) return cudaErrorInvalidValue;
    static DeviceValue pairs;  // CTA pairs that the GPU holds at once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int max_pairs = pairs.get(dev, [] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() & ~1));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = smem_bytes<PR>(1024);
        int nc = 0;
        if (allow_smem<grouped_tc_kernel<PR, SPLIT>>() != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&nc, grouped_tc_kernel<PR, SPLIT>, &cfg) != cudaSuccess || nc < 1) {
            (void)cudaGetLastError();
            nc = sm_pairs();
        }
        return nc;
    });
    const GroupedParams p{g.R, g.E, g.N, g.K, g.offsets, out, bf ? 1u : 0u, cols, splits, g.part, g.err};
    const int grid = 2 * (int)std::max<long long>(1, std::min<long long>(max_pairs, (long long)items * splits));
    e = launch_overlapped<grouped_tc_kernel<PR, SPLIT>>(dim3(grid), dim3(THREADS), smem_bytes<PR>(g.E), s, maps, p);
    if (SPLIT && e == cudaSuccess) {
        GroupedParams q = p;
        if (PR == Product::DW) q.offsets = nullptr;
        const int rows = PR == Product::DW ? g.E * g.N : g.R, row = PR == Product::Y ? g.N : g.K;
        const long long blocks = ((long long)rows * row / 8 + 255) / 256;
        e = launch_overlapped(grouped_sum_kernel, (int)std::min<long long>(num_sms() * 8, blocks), 256, 0, s, q, rows, row);
    }
    return e;
}
template <Product PR>
cudaError_t launch(const GroupedShape& g, const void* a, const void* b, void* out, cudaStream_t s) {
    const int pairs = sm_pairs(), cols = tile_columns<PR>(g, pairs), splits = tile_splits<PR>(g, cols, pairs);
    return splits > 1 ? launch<PR, true>(g, a, b, out, cols, splits, s) : launch<PR, false>(g, a, b, out, cols, 1, s);
}

}  // namespace

// E 128, N 1536, K 2048: 8 rows 12.5 us there and 12.7 here, 32 rows 34.7 and
// 35.7, 128 rows 116 and 125; E 256, N 4096, K 7168: 64 rows 531 and 555.  With
// several rows an expert its blocks read the weights again: E 8, N 1024, K 256:
// 16 rows 2.9 and 4.4, 64 rows 5.2 and 4.4; E 1, N and K 2048: 64 rows 13.2 and 9.6
static bool takes_few(const GroupedShape& g) { return g.R <= 32 || (g.R <= 128 && g.R <= g.E); }

size_t grouped_floats(const GroupedShape& g) {
    return g.R == 0 || takes_few(g) ? 0 : split_floats<Product::Y>(g, sm_pairs());
}
size_t grouped_dx_floats(const GroupedShape& g) { return g.R == 0 ? 0 : split_floats<Product::DX>(g, sm_pairs()); }
size_t grouped_dw_floats(const GroupedShape& g) { return g.R == 0 ? 0 : split_floats<Product::DW>(g, sm_pairs()); }

size_t grouped_floats_bound(const GroupedShape& g) {
    if (g.R == 0) return 0;
    const int pairs = sm_pairs();
    return std::max({rows_floats_bound(g, g.N, g.K, pairs), rows_floats_bound(g, g.K, g.N, pairs),
                     split_floats<Product::DW>(g, pairs)});
}
cudaError_t launch_grouped_mm(const GroupedShape& g, const void* x, const void* w, void* y, cudaStream_t s) {
    if (takes_few(g)) return launch_grouped_few(g, x, w, y, s);
    return launch<Product::Y>(g, w, x, y, s);
}
cudaError_t launch_grouped_mm_dx(const GroupedShape& g, const void* dy, const void* w, void* dx, cudaStream_t s) {
    return launch<Product::DX>(g, w, dy, dx, s);
}
cudaError_t launch_grouped_mm_dw(const GroupedShape& g, const void* dy, const void* x, void* dw, cudaStream_t s) {
    if (g.R == 0) return cudaMemsetAsync(dw, 0, (size_t)g.E * g.N * g.K * 2, s);
    return launch<Product::DW>(g, dy, x, dw, s);
}

}  // namespace moe
