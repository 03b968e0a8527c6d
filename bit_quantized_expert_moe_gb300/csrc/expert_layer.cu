// The whole layer of 16-bit experts for a few tokens in one kernel: routing,
// gate_up, SiLU(gate) up, down and the weighted sum.
//
//   e_1 .. e_k = the largest logits of token t,  p = softmax over them
//   h_j = SiLU(Wg[e_j] x) * (Wu[e_j] x),   out = sum_j p_j Wd[e_j] h_j
//
// What counts is reading the weights of the experts that have a token, once:
// 6 d f bytes an expert.  One CTA an SM (cooperative); one producer thread streams
// the CTA's share of both matrices through a ring of 22 KB slots (TMA), sixteen
// warps take them from there.  The share of the down projection does not depend on h, so
// the ring fills with it while the CTAs meet between the two products: the stream
// does not stop there.
//   Phase 0  every CTA routes all tokens; the touched experts' list by one scan.
//   Phase 1  the touched experts' features, one list of n_uniq f, are split evenly
//            over the CTAs to a single feature (its gate and its up row): tiles of 8,
//            4, 2 or 1 features, chunks of at most 704 inputs.  p h goes to memory.
//   Phase 2  output features, split evenly over the CTAs; a CTA goes through all
//            touched experts for its own, so the sum over experts is its own as well:
//            no partial sums between CTAs, a fixed order, one rounding.
// mma.sync m16n8k16 with the weight rows as M (phase 1: 8 features' gate rows and their
// up rows, so that a thread has both) and an expert's tokens as N, 8 at a time: at a
// few tokens an expert the tensor rate is no bound.  Both operands keep K in the order
// in which a thread's 16-byte loads bring it, as in grouped_few.cu.
// h has the weight p already and is kept as two 16-bit numbers, the second one the
// rounding error of the first (in fp16 times 2^11, so that it does not get lost among the
// subnormals where h is small): off by 2^-17 |p h| in bf16, by 2^-23 |p h| or 2^-36
// in fp16, far below the output's rounding unless its sum cancels.  In phase
// 2, up to 8 tokens, a column is a token (zeros where the expert is not the token's), so
// a thread's sums stay its own over all experts.  For more tokens, where most columns would be
// empty, the columns are an expert's tokens and a warp adds them to its
// sums in shared memory.  Up to four tokens, or rows, h and its error are columns of one
// MMA.
//
// What bounds the consumers is latency, a chunk's 0.5 us at the full rate of the stream:
//   - two groups of eight warps take every second chunk of phase 1, its 32-input units
//     dealt out to the warps, and pairs of warps every eighth one of phase 2 (up to 8
//     tokens);
//   - in phase 1 a warp has the tokens' values of its next chunk on their way in
//     registers (they stay in L1 from tile to tile); in phase 2, where every chunk brings
//     another expert's, a warp of its own has an expert's rows of h copied to a ring of
//     rows in shared memory, a bulk copy for all of them (one for each row, issued one
//     after the other, took 0.3 us a row); it takes back what has been read of all batches
//     under way at once (one by one: 28 tokens, 151 experts of 768 x 256, 88 us for 79);
//   - two warps in turn add the sixteen warps' sums of phase 1 up and write h, so that none
//     of them waits for the others (one, and divisions to find each tile: 12 tokens, 128
//     experts of 512 x 1024, 119 us for 89);
//   - small chunks of phase 2 share a slot, so that more of them are under way.
// 2048 x 768, 8 of 128 experts a token: 1 token 18.3 us (4.1 TB/s, 61 % of the copy's
// rate: routing 2.2 us, the meeting 1.0, from there to the end 2.9), 8 tokens 80 us (6.0
// TB/s), 32 tokens 164 us (6.4); 7168 x 2048, 8 of 256: 8 tokens 748 to
// 767 us (6.6 to 6.8).
// One group of eight warps that all wait for each other at a tile's end: 23.6, 109, 530
// and 1084 us; x in the ring of rows as well: 8 tokens at 7168 804, 32 at 2048 432.
#include <type_traits>

#include "decode_ops.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int MAX_T = 32, MAX_R = 256;
constexpr int GROUPS = 2, GW = 8, CW = GROUPS * GW;  // consumer warps
constexpr int CONSUMERS = 32 * CW, FINISHERS = 2, THREADS = CONSUMERS + 64 + 32 * FINISHERS;
constexpr int PRODUCER = CW, ROWS_OF_H = CW + 1, FINISHER = CW + 2;  // warps, the first of FINISHERS
// By NT, the most groups of 8 tokens of an expert.  The ring's slots are a multiple of
// the groups, so that each is always one group's: a wait names a round of its barrier by
// the round's parity, and a group that took every second round of a slot would take the
// end of the round before for that of its own.
template <int NT>
struct Plan {
    // A slot: 8 features' 16 rows of BLOCKS1 64-input blocks, or up to 16 rows of the down
    // projection.  One token at 2048 x 768: eight slots hold the CTA's share of that.
    static constexpr int BLOCKS1 = 11, BLOCKS2 = 12;
    static constexpr int SLOT = 16 * BLOCKS1 * 128, NSLOT = NT == 1 ? 8 : 6;
    static constexpr int UNITS1 = (2 * BLOCKS1 + GW - 1) / GW, UNITS2 = 2 * BLOCKS2;  // of 32 inputs: a warp's most; a chunk's
    // A row of h of a chunk, 256 bytes for 64 inputs; 64 more, so that neighbours use
    // other banks.  A batch's rows are one bulk copy; more than 16 of an expert are two
    // batches, of the tokens below 16 and of the others.
    static constexpr int PITCH = BLOCKS2 * 256 + 64, NROW = NT == 1 ? 8 : 16, NBATCH = 16;
    static constexpr int HALVES = NT <= 2 ? 1 : 2;
    // Phase 2's groups: up to 8 tokens pairs of warps, one for each slot, so that the
    // latency of a chunk counts an eighth.  More tokens take two groups of eight (pairs,
    // with eight slots of 16 KB: 32 tokens at 2048 x 768 243 us for 190).  Barriers of a
    // group's batches.
    static constexpr int GW2 = NT == 1 ? 2 : GW, GROUPS2 = CW / GW2, TURNS = NT == 1 ? NBATCH / GROUPS2 : NBATCH;

    static constexpr int NBUF = 2, SUM_FLOATS = CW * 128;        // sums of 8 tokens: [CW][32][4]
    // phase 2: [CW][8 NT][17]
    static constexpr int SUMS = 4 * (NBUF * SUM_FLOATS > CW * 8 * NT * 17 ? NBUF * SUM_FLOATS : CW * 8 * NT * 17);
    // Phase 2 cuts a slot in up to MOST_PARTS parts, where its chunks are that small.
    static constexpr int MOST_PARTS = 4;
    static constexpr int BARS = 16 * ((1 + MOST_PARTS) * NSLOT + GROUPS2 * TURNS + NBUF) + 16;
    static constexpr int OFF_BARS = NSLOT * SLOT, OFF_ROWS = OFF_BARS + 1280, OFF_SUMS = OFF_ROWS + NROW * PITCH;
    static constexpr int OFF_TAB = OFF_SUMS + SUMS;
    static_assert(NROW >= (NT < 2 ? 8 : 16) && BARS <= 1280, "a batch's rows, the barriers");
    static_assert(NSLOT % GROUPS == 0 && NSLOT % GROUPS2 == 0 && SLOT % 1024 == 0 && PITCH % 128 == 64, "layout");
};

struct Tab {
    int ids[MAX_R];
    float w[MAX_R];
    int tok[MAX_R];      // by sorted position: token
    float pw[MAX_R];     // and weight
    int uexp[MAX_R], uoff[MAX_R], ucnt[MAX_R];  // touched experts, ascending: id, first position, how many tokens
    uint32_t utok[MAX_R];                       // and which, one bit a token
    uint32_t warp_sums[CW];
    int batches[2 * 16];                        // under way: rows, barrier, parity
    int n_uniq, abort;
};

struct Params {
    const uint16_t* x;
    const float* logits;
    uint16_t* out;
    int32_t* ids_out;
    // p h: [chunks of an expert][R by sorted position][pitch bytes]: of 64 features their
    // values, then the rounding errors of these in their unit; as a batch's rows lie in shared
    // memory
    uint8_t* h;
    int pitch, nrow;     // and the rows of the ring of rows, a power of 2
    uint32_t* err;
    unsigned long long* bar_count;
    int T, k, E, d, f;
    int cb1, cb2;        // 64-input blocks of a chunk of either phase
    int cut;             // phase 2 cuts a slot in 1 << cut parts
    int rows2[4];        // rows of the maps of the down projection
};
struct Maps {
    CUtensorMap w13[4], w2[4];  // boxes of 8, 4, 2, 1 features; of rows2[i] rows
};

template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], uint4 a, uint4 b, uint4 v) {
    if constexpr (BF16) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(b.x), "r"(a.y), "r"(b.y), "r"(v.x), "r"(v.y));
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.z), "r"(b.z), "r"(a.w), "r"(b.w), "r"(v.z), "r"(v.w));
    } else {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(b.x), "r"(a.y), "r"(b.y), "r"(v.x), "r"(v.y));
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.z), "r"(b.z), "r"(a.w), "r"(b.w), "r"(v.z), "r"(v.w));
    }
}
template <bool BF16>
__device__ __forceinline__ uint16_t bits16(float v) { return BF16 ? float_to_bf16_bits(v) : float_to_f16_bits(v); }
template <bool BF16>
__device__ __forceinline__ float value16(uint16_t b) {
    return BF16 ? __uint_as_float((uint32_t)b << 16) : half_bits_to_float(b);
}

// The rounding error of an fp16 number is at most 16 below its end, 65520, and an fp16 number
// itself times 2^11.
template <bool BF16>
constexpr float ERROR_UNIT = BF16 ? 1.f : 0x1p-11f;

// Between ordinary accesses to global memory and bulk copies of it.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Part c of `parts` of n things: [share(c), share(c + 1)); n parts is below 2^32.
__device__ __forceinline__ int share(int n, int c, int parts) { return (int)((uint32_t)n * (uint32_t)c / (uint32_t)parts); }

// Phase 1: the tile at feature x of the list, of those before `end`: expert u,
// features i0 .. i0 + n - 1, box of map m (n = 8 >> m).
struct Tile1 {
    int u, i0, n, m;
    __device__ Tile1() : u(0), i0(0), n(0), m(0) {}
    __device__ Tile1(int x, int end, int f) {
        u = x / f;
        i0 = x - u * f;
        size(x, end, f);
    }
    // the tile behind, at x
    __device__ void next(int x, int end, int f) {
        if ((i0 += n) == f) {
            i0 = 0;
            ++u;
        }
        size(x, end, f);
    }
    __device__ void size(int x, int end, int f) {
        const int most = min(min(8, f - i0), end - x);
        m = 3 - (31 - __clz(most));
        n = 8 >> m;
    }
};
// Phase 2: rows of a CTA's `rows` that tile i of `tiles` has, and the first.
struct Tile2 {
    int n, r0;
    __device__ Tile2(int rows, int tiles, int i) {
        const int each = rows / tiles, more = rows - each * tiles;
        n = each + (i < more);
        r0 = i * each + min(i, more);
    }
};

// Where a unit's 16 bytes of line `line` (128 bytes of 64 inputs) are in a slot: 32
// inputs `half`, lane t; the 128-byte swizzle of the box.
__device__ __forceinline__ uint32_t weights_at(uint32_t slot, int line, int half, int t) {
    return slot + 128u * line + ((uint32_t)((4 * half + t) ^ (line & 7)) << 4);
}

// Where a group is in phase 1's list of chunks.
struct Place1 {
    int x, b, q;         // tile's first feature, chunk's first block; chunks before
    int cnt, off;        // of the tile
    Tile1 t;
    __device__ Place1(const Tab& tab, int x_, int end, int f) : x(x_), b(0), q(0), cnt(0), off(0) {
        if (x < end) {
            t = Tile1(x, end, f);
            rows(tab);
        }
    }
    __device__ void rows(const Tab& tab) {
        cnt = tab.ucnt[t.u];
        off = tab.uoff[t.u];
    }
    __device__ void step(const Tab& tab, int end, int f, int nb, int cb) {
        if (x >= end) return;
        ++q;
        if ((b += cb) < nb) return;
        b = 0;
        x += t.n;
        if (x >= end) return;
        t.next(x, end, f);
        rows(tab);
    }
};

// PAIR: up to 4 tokens, whose h and rounding errors are columns of one MMA.
template <bool BF16, int NT, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1) expert_layer_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Plan<NT>;
    constexpr int NSLOT = L::NSLOT, NBATCH = L::NBATCH, NBUF = L::NBUF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t ring = smem_u32(sm), rows_at = ring + L::OFF_ROWS;
    const uint32_t full = ring + L::OFF_BARS, empty = full + 8 * NSLOT;                  // slots
    const uint32_t full2 = empty + 8 * NSLOT, empty2 = full2 + 8 * NSLOT * L::MOST_PARTS;     // their parts, phase 2
    const uint32_t row_full = empty2 + 8 * NSLOT * L::MOST_PARTS, row_empty = row_full + 8 * L::GROUPS2 * L::TURNS;      // rows of a batch
    const uint32_t sum_full = row_empty + 8 * L::GROUPS2 * L::TURNS, sum_empty = sum_full + 8 * NBUF, h_ready = sum_empty + 8 * NBUF;
    float* sums = reinterpret_cast<float*>(sm + L::OFF_SUMS);
    Tab& tab = *reinterpret_cast<Tab*>(sm + L::OFF_TAB);
    volatile int* abort_flag = &tab.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = p.T * p.k, d = p.d, f = p.f, G = gridDim.x, cta = blockIdx.x;
    const int nb1 = d / 64, nb2 = f / 64, cb1 = p.cb1, cb2 = p.cb2;

    // ------------------------------------------------ phase 0: init, routing
    if (threadIdx.x == 0) tab.abort = 0;
    if (warp == PRODUCER && lane == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, GW);
        }
        for (int i = 0; i < NSLOT * L::MOST_PARTS; ++i) {
            tc::mbar_init(full2 + 8 * i, 1);
            tc::mbar_init(empty2 + 8 * i, GW);
        }
        for (int i = 0; i < L::GROUPS2 * L::TURNS; ++i) {
            tc::mbar_init(row_full + 8 * i, 1);
            tc::mbar_init(row_empty + 8 * i, GW);
        }
        for (int i = 0; i < NBUF; ++i) {
            tc::mbar_init(sum_full + 8 * i, CW);
            tc::mbar_init(sum_empty + 8 * i, 1);
        }
        tc::mbar_init(h_ready, 1);
        tc::fence_mbar_init();
        for (int i = 0; i < 4; ++i) {
            tc::tma_prefetch_desc(&maps.w13[i]);
            tc::tma_prefetch_desc(&maps.w2[i]);
        }
    }
    // in the ring's space, which is idle: by expert, its tokens (one bit each) and their
    // first position
    uint32_t* tokens = reinterpret_cast<uint32_t*>(sm);
    int* first = reinterpret_cast<int*>(sm) + p.E;
    static_assert(8 * 1024 <= NSLOT * L::SLOT, "1024 experts");
    for (int i = threadIdx.x; i < p.E; i += THREADS) tokens[i] = 0;
    if (warp == FINISHER) {  // a hint, which returns no value: before the kernel ahead is complete
        const int lines = (p.T * p.E * 4 + 127) / 128;
        for (int i = lane; i < lines; i += 32)
            asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const char*>(p.logits) + 128 * (size_t)i));
    }
    // global memory is read and written from here on
    grid_dependency_wait();
    __syncthreads();
    if (warp < CW)
        for (int t = warp; t < p.T; t += CW) {
            dec::route_token(p.logits + (size_t)t * p.E, p.E, p.k, &tab.ids[t * p.k], &tab.w[t * p.k]);
            if (lane < p.k) {
                const int e = tab.ids[t * p.k + lane];
                // logits that are no numbers may choose no expert
                if ((unsigned)e < (unsigned)p.E) atomicOr(&tokens[e], 1u << t);
                else set_error(p.err, ERRBIT_RANGE);
                if (cta == 0 && p.ids_out) p.ids_out[t * p.k + lane] = e;
            }
        }
    __syncthreads();
    // The touched experts in ascending order: places and positions before each, packed
    // in one sum; two experts a thread.
    uint32_t mask[2] = {0, 0}, mine = 0, before = 0;
    if (warp < CW) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * threadIdx.x + i;
            if (e < p.E) mask[i] = tokens[e];
            mine += mask[i] ? 1u + ((uint32_t)__popc(mask[i]) << 16) : 0u;
        }
        before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) tab.warp_sums[warp] = before;
    }
    __syncthreads();
    if (warp < CW) {
        const uint32_t v = lane < CW ? tab.warp_sums[lane] : 0;
        before += __reduce_add_sync(0xffffffffu, lane < warp ? v : 0) - mine;
        if (warp == 0) {
            const uint32_t all = __reduce_add_sync(0xffffffffu, v);
            if (lane == 0) tab.n_uniq = all & 0xffff;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (mask[i]) {
                const int u = before & 0xffff, e = 2 * threadIdx.x + i, cnt = __popc(mask[i]);
                tab.uexp[u] = e;
                tab.uoff[u] = first[e] = before >> 16;
                tab.ucnt[u] = cnt;
                tab.utok[u] = mask[i];
                before += 1u + ((uint32_t)cnt << 16);
            }
        dec::bar_sync(1, CONSUMERS);
        for (int a = threadIdx.x; a < R; a += CONSUMERS) {
            const int e = tab.ids[a], t = a / p.k;
            if ((unsigned)e < (unsigned)p.E) {
                const int at = first[e] + __popc(tokens[e] & ((1u << t) - 1u));
                tab.tok[at] = t;
                tab.pw[at] = tab.w[a];
            }
        }
        tc::fence_proxy_async_smem();  // before the copies into the ring
    }
    __syncthreads();

    const int n_uniq = tab.n_uniq;
    const int x_lo = share(n_uniq * f, cta, G), x_hi = share(n_uniq * f, cta + 1, G);
    const int r_lo = share(d, cta, G), rows = share(d, cta + 1, G) - r_lo, tiles2 = ceil_div(rows, 16);
    // Part i of the slots in phase 2, which begins at slot s0: the slots become free in
    // that order.
    auto part_at = [&](int i, int s0) {
        const int slot = s0 + (i >> p.cut);
        return ring + (slot < NSLOT ? slot : slot - NSLOT) * L::SLOT + (i & ((1 << p.cut) - 1)) * ((L::SLOT >> p.cut) & ~1023);
    };
    const int slots2 = NSLOT << p.cut;
    // A wait that gave up goes on with what is there: no arrival and no barrier is left
    // out, and every address stays where it was.

    if (warp == PRODUCER) {
        // -------------------------------------------------- weights, by TMA
        if (tc::elect_one()) {
            int s = 0;
            uint32_t phase = 1;
            bool ok = true;
            auto next = [&](uint32_t bytes) {
                ok = ok && tc::mbar_wait(empty + 8 * s, phase, abort_flag, p.err);
                if (ok) tc::mbar_arrive_expect_tx(full + 8 * s, bytes);
                return ok;
            };
            auto advance = [&] {
                if (++s == NSLOT) {
                    s = 0;
                    phase ^= 1u;
                }
            };
            Tile1 t(x_lo, x_hi, f);
            for (int x = x_lo; ok && x < x_hi;) {
                const int e = tab.uexp[t.u];
                for (int b = 0; b < nb1 && next(cb1 * 2 * t.n * 128); b += cb1, advance())
                    asm volatile(
                        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];"
                        :: "r"(ring + s * L::SLOT), "l"(&maps.w13[t.m]), "r"(full + 8 * s), "r"(0), "r"(t.i0), "r"(b), "r"(e) : "memory");
                x += t.n;
                if (x < x_hi) t.next(x, x_hi, f);
            }
            // the first round of the parts waits for the slots of phase 1
            const int s0 = s;
            int at = 0;
            uint32_t round = 0;
            auto next2 = [&](uint32_t bytes) {
                if (round) {
                    ok = ok && tc::mbar_wait(empty2 + 8 * at, (round - 1) & 1u, abort_flag, p.err);
                } else if ((at & ((1 << p.cut) - 1)) == 0) {
                    ok = ok && tc::mbar_wait(empty + 8 * s, phase, abort_flag, p.err);
                    advance();
                }
                if (ok) tc::mbar_arrive_expect_tx(full2 + 8 * at, bytes);
                return ok;
            };
            for (int i = 0; ok && i < tiles2; ++i) {
                const Tile2 t(rows, tiles2, i);
                const int m = t.n == p.rows2[0] ? 0 : t.n == p.rows2[1] ? 1 : t.n == p.rows2[2] ? 2 : 3;
                for (int u = 0; ok && u < n_uniq; ++u) {
                    const int e = tab.uexp[u];
                    for (int b = 0; b < nb2 && next2(cb2 * t.n * 128); b += cb2) {
                        tc::tma_load_4d(part_at(at, s0), &maps.w2[m], full2 + 8 * at, 0, r_lo + t.r0, b, e);
                        if (++at == slots2) {
                            at = 0;
                            ++round;
                        }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == ROWS_OF_H) {
        // ------------------- the tokens' rows of h of the chunks, a lane a bulk copy
        // A window of batches, a lane each: where their rows lie and go, which barrier of
        // its group's TURNS ones a batch has.  Lanes copy as soon as there is room, in order:
        // at most NBATCH batches and the ring's rows are under way.
        constexpr int PER = 32 / L::HALVES;  // chunks of a window
        const int parts = ceil_div(nb2, cb2), chunks = n_uniq * parts, all = tiles2 * chunks;
        const int half = L::HALVES == 1 ? 0 : lane & 1;
        const uint32_t below = (1u << lane) - 1u;
        int head = 0, tail = 0, at = 0, given = 0, turns[2] = {0, 0};  // batches, given back; rows, given back
        bool ok = true;
        for (int base = 0; ok && base < all; base += PER) {
            const int c = base + lane / L::HALVES;
            int cnt = 0, from = 0;  // rows of the batch, the first
            if (c < all) {
                const int j = c % chunks, u = j / parts;
                const uint32_t toks = tab.utok[u];
                from = (j - u * parts) * R + tab.uoff[u];
                cnt = __popc(toks);
                if (L::HALVES > 1) {
                    const int low = __popc(toks & 0xffffu);
                    if (cnt > 16) {
                        cnt = half ? cnt - low : low;
                        from += half ? low : 0;
                    } else if (half) {
                        cnt = 0;
                    }
                }
            }
            const uint32_t any = __ballot_sync(0xffffffffu, cnt > 0), odd = __ballot_sync(0xffffffffu, c & 1);
            const int index = head + __popc(any & below);
            int place = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, place, o);
                if (lane >= o) place += v;
            }
            const int total = __shfl_sync(0xffffffffu, place, 31);
            place += at - cnt;
            const uint32_t ours = c & 1 ? odd : ~odd;
            const int turn = L::HALVES == 1 ? index / L::GROUPS2 : turns[c & 1] + __popc(any & ours & below);
            const int slot = c % L::GROUPS2 * L::TURNS + turn % L::TURNS;
            if (base == 0) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(h_ready, 0, abort_flag, p.err));
                fence_proxy_async_global();  // h was written by ordinary stores
            }
            bool todo = cnt > 0;
            while (ok && __any_sync(0xffffffffu, todo)) {
                const bool go = todo && index - tail < NBATCH && place + cnt - given <= p.nrow;
                if (go) {
                    tab.batches[index % (2 * NBATCH)] = cnt | slot << 8 | (turn / L::TURNS & 1) << 16;
                    const uint32_t bar = row_full + 8 * slot;
                    const int to = place & (p.nrow - 1), front = min(cnt, p.nrow - to);
                    const uint8_t* src = p.h + (size_t)from * p.pitch;
                    tc::mbar_arrive_expect_tx(bar, cnt * p.pitch);
                    tc::bulk_load(rows_at + to * p.pitch, src, front * p.pitch, bar);
                    if (front < cnt) tc::bulk_load(rows_at, src + (size_t)front * p.pitch, (cnt - front) * p.pitch, bar);
                    todo = false;
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, go)) continue;
                // the oldest batch's wait, and how many behind it have been given back too
                const int copied = head + __popc(any & ~__ballot_sync(0xffffffffu, todo));
                const int o = tab.batches[(tail + lane) % (2 * NBATCH)];
                const uint32_t bar = row_empty + 8 * (o >> 8 & 255);
                if (lane == 0) ok = tc::mbar_wait(bar, (uint32_t)o >> 16, abort_flag, p.err);
                const bool back = lane == 0 || (tail + lane < copied && tc::mbar_test_cluster(bar, (uint32_t)o >> 16));
                ok = __all_sync(0xffffffffu, ok);  // (nothing is copied after a wait that gave up)
                const int n = __ffs(~__ballot_sync(0xffffffffu, back)) - 1;
                given += __reduce_add_sync(0xffffffffu, lane < n ? o & 255 : 0);
                tail += n;
            }
            head += __popc(any);
            at += total;
            turns[0] += __popc(any & ~odd);
            turns[1] += __popc(any & odd);
        }
    } else if (warp >= FINISHER) {
        // --------------------- phase 1's sums: h = SiLU(gate) up, two columns a lane
        const int g = lane >> 2, t = lane & 3;
        const int which = warp - FINISHER;
        const uint32_t by_cb2 = (1u << 20) / (uint32_t)cb2 + 1;  // for blocks below 2^9, chunks of at most 12
        int k = 0;
        Tile1 tl(x_lo, x_hi, f);
        for (int x = x_lo; x < x_hi;) {
            const int cnt = tab.ucnt[tl.u], off = tab.uoff[tl.u];
            for (int n = 0; 8 * n < cnt; ++n, ++k) {
                const int buf = k % NBUF;
                if (k % FINISHERS != which) continue;
                tc::mbar_wait(sum_full + 8 * buf, (uint32_t)(k / NBUF) & 1u, abort_flag, p.err);
                __syncwarp();
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < CW; ++w) {
                    const float4 o = *reinterpret_cast<const float4*>(sums + buf * L::SUM_FLOATS + (w * 32 + lane) * 4);
                    v.x += o.x;
                    v.y += o.y;
                    v.z += o.z;
                    v.w += o.w;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(sum_empty + 8 * buf);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 8 * n + 2 * t + i;
                    if (g < tl.n && col < cnt) {
                        const float a = i ? v.y : v.x, u = i ? v.w : v.z;
                        const float h = tab.pw[off + col] * (a / (1.f + expf(-a)) * u);
                        const uint16_t hi = bits16<BF16>(h);
                        const float rest = h - value16<BF16>(hi);
                        if (!BF16 && isfinite(h) && !isfinite(rest)) set_error(p.err, ERRBIT_F16_RANGE);
                        const int i = tl.i0 + g, part = (uint32_t)(i >> 6) * by_cb2 >> 20;
                        auto* to = reinterpret_cast<uint16_t*>(p.h + ((size_t)part * R + off + col) * p.pitch) +
                                   ((i >> 6) - part * cb2) * 128 + (i & 63);
                        to[0] = hi;
                        to[64] = bits16<BF16>(isfinite(rest) ? rest * (1.f / ERROR_UNIT<BF16>) : 0.f);
                    }
                }
            }
            x += tl.n;
            if (x < x_hi) tl.next(x, x_hi, f);
        }
        // Every CTA's h is written before anyone reads it.  The arrival count only
        // grows, G a launch, so a CTA's own arrival tells it the count at which this
        // launch's barrier opens.
        fence_proxy_async_global();  // it is read by bulk copies
        dec::bar_sync(2, 32 * FINISHERS);
        if (which == 0 && lane == 0) {
            const uint64_t old = dec::atom_add_release_gpu(p.bar_count, 1ull);
            const uint64_t target = (old / (uint64_t)G + 1) * (uint64_t)G;
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t it = 1; dec::ld_acquire_gpu64(p.bar_count) < target; ++it)
                if ((it & 63u) == 0) {
                    if (*abort_flag) break;
                    if (globaltimer_ns() - t0 > tc::WAIT_LIMIT_NS) {
                        set_error(p.err, ERRBIT_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                }
            tc::mbar_arrive(h_ready);
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------- consumers
        const int g = lane >> 2, t = lane & 3, group = warp / GW, gw = warp % GW;
        float acc[NT][4];
        auto clear = [&] {
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        };
        auto wait = [&](int q) { tc::mbar_wait(full + 8 * (q % NSLOT), (uint32_t)(q / NSLOT) & 1u, abort_flag, p.err); };
        auto release = [&](int q) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty + 8 * (q % NSLOT));
        };
        // ---- phase 1.  Units gw, gw + GW, ... of a chunk are this warp's.  As soon as the
        // MMAs have a unit's values, those of the warp's next chunk (or next 8 tokens)
        // take their place.
        uint4 v[L::UNITS1];
        struct From {
            const uint16_t* x;
            int units;
        };
        auto from = [&](const Place1& c, int n) {
            return From{p.x + (size_t)tab.tok[c.off + min(8 * n + g, c.cnt - 1)] * d + 64 * c.b + 8 * t, 2 * min(cb1, nb1 - c.b)};
        };
        auto load = [&](int i, const From& o) {
            if (gw + GW * i < o.units) v[i] = __ldg(reinterpret_cast<const uint4*>(o.x + 32 * (gw + GW * i)));
        };
        // every warp has a part of every sum, though it may be zero
        int k = 0;
        auto add_up = [&](int cnt) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (8 * n < cnt) {
                    const int buf = k % NBUF;
                    tc::mbar_wait(sum_empty + 8 * buf, ((uint32_t)(k / NBUF) & 1u) ^ 1u, abort_flag, p.err);
                    *reinterpret_cast<float4*>(sums + buf * L::SUM_FLOATS + (warp * 32 + lane) * 4) =
                        make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(sum_full + 8 * buf);
                    ++k;
                }
            clear();
        };
        Place1 c(tab, x_lo, x_hi, f);
        clear();
        const int first = c.x, first_cnt = c.cnt;
        if (group) c.step(tab, x_hi, f, nb1, cb1);
        if (c.x != first) add_up(first_cnt);  // the first tile was the other group's
        if (c.x < x_hi) {
            const From o = from(c, 0);
#pragma unroll
            for (int i = 0; i < L::UNITS1; ++i) load(i, o);
        }
        while (c.x < x_hi) {
            Place1 mid = c;
            mid.step(tab, x_hi, f, nb1, cb1);
            Place1 to = mid;
            to.step(tab, x_hi, f, nb1, cb1);
            const int units = 2 * min(cb1, nb1 - c.b);
            // The lines of unit gw's gate and up rows (beyond the tile's rows: its last again);
            // those of unit gw + GW are 8 n further, at the same place of the swizzle.
            const uint32_t slot = ring + (c.q % NSLOT) * L::SLOT, further = 1024u * c.t.n;
            const int line = (gw >> 1) * 2 * c.t.n + min(g, c.t.n - 1);
            const uint32_t gate = weights_at(slot, line, gw & 1, t), up = weights_at(slot, line + c.t.n, gw & 1, t);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (8 * n < c.cnt) {
                    From o{nullptr, 0};
                    if (8 * (n + 1) < c.cnt) o = from(c, n + 1);
                    else if (to.x < x_hi) o = from(to, 0);
                    if (n == 0) wait(c.q);
#pragma unroll
                    for (int i = 0; i < L::UNITS1; ++i) {
                        if (gw + GW * i < units) mma<BF16>(acc[n], dec::lds128(gate + i * further), dec::lds128(up + i * further), v[i]);
                        load(i, o);
                    }
                }
            release(c.q);
            if (mid.x != c.x) add_up(c.cnt);
            if (to.x != mid.x) add_up(mid.cnt);  // this one's, or a tile that was the other group's
            c = to;
        }
        const int s0 = c.q % NSLOT;  // behind the last chunk of phase 1

        // ---- phase 2
        tc::mbar_wait(h_ready, 0, abort_flag, p.err);
        grid_dependency_launch();  // the last phase: the next kernel may be scheduled
        constexpr int SETS = 2;  // of accumulators: of h's values and of its errors, or (both in one) of every second unit
        float out[SETS][NT == 1 ? 1 : 2][4];
        auto clear_out = [&] {
#pragma unroll
            for (int s = 0; s < SETS; ++s)
#pragma unroll
                for (int n = 0; n < (NT == 1 ? 1 : 2); ++n) out[s][n][0] = out[s][n][1] = out[s][n][2] = out[s][n][3] = 0.f;
        };
        // a warp's sums: NT = 1: at the end of a tile; else all along
        float* mine = sums + warp * (8 * NT * 17);
        if (NT > 1)
            for (int i = lane; i < 8 * NT * 17; i += 32) mine[i] = 0.f;
        __syncwarp();
        const int group2 = warp / L::GW2, gw2 = warp % L::GW2, parts = ceil_div(nb2, cb2), chunks = n_uniq * parts;
        float total[4];  // NT = 1: over the experts
        const int rows_of_all = n_uniq ? tab.uoff[n_uniq - 1] + tab.ucnt[n_uniq - 1] : 0;
        const int u_step = L::GROUPS2 / parts, part_step = L::GROUPS2 - u_step * parts;
        int turn = 0;  // this group's batches before
        int at_part = group2;  // of the slots, of this group's next chunk
        uint32_t parity = 0;
        for (int i = 0; i < tiles2; ++i) {
            const int q = i * chunks;  // chunks before
            const Tile2 tl(rows, tiles2, i);
            // lines of unit gw2 of rows g and g + 8 (beyond the tile's: its last again), and from
            // there to unit gw2 + GW2
            const int la = (gw2 >> 1) * tl.n + min(g, tl.n - 1), lb = (gw2 >> 1) * tl.n + min(g + 8, tl.n - 1);
            const int step = L::GW2 / 2 * tl.n;
            clear_out();
            total[0] = total[1] = total[2] = total[3] = 0.f;
            int j = (group2 - q) & (L::GROUPS2 - 1), u = j / parts, part = j - u * parts;
            for (; j < chunks; j += L::GROUPS2) {
                const int off = tab.uoff[u];
                const uint32_t toks = tab.utok[u];
                const int units = 2 * min(cb2, nb2 - part * cb2);
                const uint32_t slot = part_at(at_part, s0);
                // the rows before: those of earlier tiles, experts and parts
                int at = parts * (i * rows_of_all + off) + part * __popc(toks);
                tc::mbar_wait(full2 + 8 * at_part, parity, abort_flag, p.err);
                const bool two = L::HALVES > 1 && __popc(toks) > 16;
                for (int half = 0; half <= (int)two; ++half) {
                    const uint32_t few = !two ? toks : half ? toks & 0xffff0000u : toks & 0xffffu;
                    const int cnt = __popc(few);
                    const bool pair = PAIR || (NT > 1 && cnt <= 4);
                    // this lane's column of every 8: its row, if it has one
                    constexpr int NB = NT == 1 ? 1 : 2;
                    uint32_t has[NB], row[NB];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int col = pair ? g & 3 : 8 * n + g;
                        has[n] = NT == 1 ? few >> col & 1u : col < cnt;
                        const int r = at + (NT > 1 ? col : has[n] ? __popc(few & ((1u << col) - 1u)) : 0);
                        row[n] = rows_at + (r & (p.nrow - 1)) * p.pitch + 16 * t + 64 * (gw2 & 1) + 256 * (gw2 >> 1) + (pair ? 128 * (g >> 2) : 0);
                    }
                    const uint32_t batch = 8 * (group2 * L::TURNS + turn % L::TURNS);
                    tc::mbar_wait(row_full + batch, (uint32_t)(turn / L::TURNS) & 1u, abort_flag, p.err);
                    auto units_of = [&](auto both, auto wide) {
                        constexpr bool BOTH = decltype(both)::value, WIDE = decltype(wide)::value;
#pragma unroll(BOTH ? 4 : 3)
                        for (int i = 0; i < L::UNITS2 / L::GW2; ++i) {
                            if (gw2 + L::GW2 * i < units) {
                                const int line = i * step;
                                const uint4 wa = dec::lds128(weights_at(slot, la + line, gw2 & 1, t));
                                const uint4 wb = dec::lds128(weights_at(slot, lb + line, gw2 & 1, t));
                                const uint32_t from = i * (128 * L::GW2);
                                if (BOTH) {
                                    mma<BF16>(out[i & 1][0], wa, wb, dec::lds128_if(row[0] + from, has[0]));
                                } else {
#pragma unroll
                                    for (int n = 0; n < (WIDE ? NB : 1); ++n) {
                                        const uint4 hi = dec::lds128_if(row[n] + from, has[n]);
                                        const uint4 lo = dec::lds128_if(row[n] + from + 128, has[n]);
                                        mma<BF16>(out[0][n], wa, wb, hi);
                                        mma<BF16>(out[1][n], wa, wb, lo);
                                    }
                                }
                            }
                        }
                    };
                    if constexpr (NT == 1) {
                        units_of(std::integral_constant<bool, PAIR>{}, std::false_type{});
                        // a token without this expert has zeros for h, but weights that are no
                        // numbers do not give zeros
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int col = PAIR ? (2 * t + (c & 1)) & 3 : 2 * t + (c & 1);
                            // (both sets have values, in columns up to 3, or the second one has errors)
                            total[c] += few >> col & 1u ? fmaf(out[1][0][c], PAIR ? 1.f : ERROR_UNIT<BF16>, out[0][0][c]) : 0.f;
                        }
                        clear_out();
                    } else {
                        if (pair) units_of(std::true_type{}, std::false_type{});
                        else if (cnt <= 8) units_of(std::false_type{}, std::false_type{});
                        else units_of(std::false_type{}, std::true_type{});
                        // columns 2 t and 2 t + 1, rows g and g + 8, into the tokens' sums
                        const int first = off + (half ? __popc(toks & 0xffffu) : 0);
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            float v[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                v[c] = fmaf(out[1][n][c], pair ? 1.f : ERROR_UNIT<BF16>, out[0][n][c]);
                                const float error = __shfl_xor_sync(0xffffffffu, v[c], 2);  // four columns further
                                if (pair) v[c] = fmaf(error, ERROR_UNIT<BF16>, v[c]);
                            }
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int col = 8 * n + 2 * t + c;
                                if (col < cnt) {
                                    float* o = mine + tab.tok[first + col] * 17 + g;
                                    o[0] += v[c];
                                    o[8] += v[2 + c];
                                }
                            }
                        }
                        clear_out();
                    }
                    __syncwarp();
                    if (lane < GW / L::GW2) tc::mbar_arrive(row_empty + batch);
                    ++turn;
                    at += cnt;
                }
                if (lane < GW / L::GW2) tc::mbar_arrive(empty2 + 8 * at_part);
                if ((at_part += L::GROUPS2) >= slots2) {
                    at_part -= slots2;
                    parity ^= 1u;
                }
                u += u_step;
                if ((part += part_step) >= parts) {
                    part -= parts;
                    ++u;
                }
            }
            if (NT == 1)  // columns 2 t and 2 t + 1, rows g and g + 8
#pragma unroll
                for (int c = 0; c < 4; ++c) mine[(2 * t + (c & 1)) * 17 + g + 4 * (c & 2)] = total[c];
            dec::bar_sync(1, CONSUMERS);
            for (int j = threadIdx.x; j < p.T * 16; j += CONSUMERS) {
                const int tok = j >> 4, r = j & 15;
                float v = 0.f;
#pragma unroll 4  // (run once or a few times: what counts is that little code is fetched)
                for (int w = 0; w < CW; ++w) {
                    float* o = sums + (w * 8 * NT + tok) * 17 + r;
                    v += *o;
                    if (PAIR) v = fmaf(o[4 * 17], ERROR_UNIT<BF16>, v);
                    if (NT > 1) *o = 0.f;
                }
                if (r < tl.n) p.out[(size_t)tok * d + r_lo + tl.r0 + r] = bits16<BF16>(v);
            }
            dec::bar_sync(1, CONSUMERS);
        }
    }
    // A wait that gave up: copies that were issued land well inside this time.
    __syncwarp();
    if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {}
    }
}

template <bool BF16, int NT, bool PAIR = false>
cudaError_t launch(const Maps& maps, Params& p, cudaStream_t s) {
    // narrow rows: more of them
    p.nrow = Plan<NT>::NROW;
    while (2 * p.nrow * p.pitch <= Plan<NT>::NROW * Plan<NT>::PITCH) p.nrow *= 2;
    constexpr size_t smem = 1024 + Plan<NT>::OFF_TAB + sizeof(Tab);
    static_assert(smem <= SMEM_MOST, "shared memory");
    cudaError_t e = allow_smem<expert_layer_kernel<BF16, NT, PAIR>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms());
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    // cooperative: the CTAs meet, so all have to be resident; and a programmatic
    // dependent of the kernel before it
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, expert_layer_kernel<BF16, NT, PAIR>, maps, p);
    if (e == cudaSuccess) note_launch();
    return e;
}

// What the sizes alone settle: a CTA's output features, q or q + 1, come in tiles of at
// most two sizes each; chunks of as many 64-input blocks each, as fit a slot.
struct Cut {
    int rows2[4], cb1, cb2, pitch, cut;
    Cut(int d, int f) {
        const int q = d / num_sms();
        int most = 1;
        for (int i = 0; i < 4; ++i) {
            const int rows = std::max(1, q + (i & 1)), tiles = ceil_div(rows, 16);
            rows2[i] = i < 2 ? rows / tiles : ceil_div(rows, tiles);
            most = std::max(most, rows2[i]);
        }
        using L = Plan<1>;  // (the others' are the same)
        cb1 = ceil_div(d / 64, ceil_div(d / 64, L::BLOCKS1));
        cb2 = ceil_div(f / 64, ceil_div(f / 64, std::min(L::BLOCKS2, 16 * L::BLOCKS1 / most)));
        pitch = 256 * cb2 + 64;
        cut = 0;
        while (1 << cut < L::MOST_PARTS && most * cb2 * 128 <= (L::SLOT >> (cut + 1) & ~1023)) ++cut;
    }
};

}  // namespace

bool expert_layer_supported(int T, int k) { return T <= MAX_T && T * k <= MAX_R && k <= 32; }
size_t expert_layer_bytes(int T, int k, int d, int f) {
    const Cut c(d, f);
    return (size_t)T * k * ceil_div(f / 64, c.cb2) * c.pitch;
}

cudaError_t launch_expert_layer(const ExpertLayer& l, cudaStream_t s) {
    const bool bf = l.dtype == MOE_DT_BF16;
    const uint64_t d = l.d, f = l.f, E = l.E;
    Params p{};
    p.x = static_cast<const uint16_t*>(l.x);
    p.logits = l.logits;
    p.out = static_cast<uint16_t*>(l.out);
    p.ids_out = l.ids_out;
    p.h = l.h;
    p.err = l.header;
    p.bar_count = reinterpret_cast<unsigned long long*>(l.header + WS_BAR_COUNT_WORD);
    p.T = l.T;
    p.k = l.k;
    p.E = l.E;
    p.d = l.d;
    p.f = l.f;
    const Cut c(l.d, l.f);
    std::copy(c.rows2, c.rows2 + 4, p.rows2);
    p.cb1 = c.cb1;
    p.cb2 = c.cb2;
    p.pitch = c.pitch;
    p.cut = c.cut;
    Maps maps;
    bool ok = true;
    // gate_up as [expert][64-input block][gate, up][feature][64 inputs]
    const uint64_t d13[5] = {64, f, 2, d / 64, E}, s13[4] = {2 * d, 2 * f * d, 128, 4 * f * d};
    for (int i = 0; i < 4 && ok; ++i) {
        const uint32_t box[5] = {64, 8u >> i, 2, (uint32_t)p.cb1, 1};
        ok = make_tensor_map_16(&maps.w13[i], bf, l.w13, 5, d13, s13, box);
    }
    // down as [expert][64-input block][output feature][64 inputs]
    const uint64_t d2[4] = {64, d, f / 64, E}, s2[3] = {2 * f, 128, 2 * d * f};
    for (int i = 0; i < 4 && ok; ++i) {
        const uint32_t box[4] = {64, (uint32_t)p.rows2[i], (uint32_t)p.cb2, 1};
        ok = make_tensor_map_16(&maps.w2[i], bf, l.w2, 4, d2, s2, box);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (l.T <= 4) return bf ? launch<true, 1, true>(maps, p, s) : launch<false, 1, true>(maps, p, s);
    if (l.T <= 8) return bf ? launch<true, 1>(maps, p, s) : launch<false, 1>(maps, p, s);
    if (l.T <= 16) return bf ? launch<true, 2>(maps, p, s) : launch<false, 2>(maps, p, s);
    return bf ? launch<true, 4>(maps, p, s) : launch<false, 4>(maps, p, s);
}

}  // namespace moe
