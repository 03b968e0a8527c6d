// The whole layer of 16-bit experts for a few tokens in one kernel: routing,
// gate_up, SiLU(gate) up, down and the weighted sum.
//
//   e_1 .. e_k = the largest logits of token t,  p = softmax over them
//   h_j = SiLU(Wg[e_j] x) * (Wu[e_j] x),   out = sum_j p_j Wd[e_j] h_j
//
// What counts is reading the weights of the experts that have a token, once:
// 6 d f bytes an expert.  One CTA an SM (cooperative); one producer thread streams
// the CTA's share of both matrices through a ring of 32 KB slots (TMA), eight warps
// take them from there.  The share of the down projection does not depend on h, so
// the ring fills with it while the CTAs meet between the two products: the stream
// does not stop there.
//   Phase 0  every CTA routes all tokens and sorts the assignments by expert.
//   Phase 1  the touched experts' features, one list of n_uniq f, are split evenly
//            over the CTAs to a single feature (its gate and its up row): tiles of 8,
//            4, 2 or 1 features, chunks of at most 1024 inputs.  h goes to memory.
//   Phase 2  output features, split evenly over the CTAs; a CTA goes through all
//            touched experts for its own, so the weighted sum over experts is its own
//            as well: no partial sums between CTAs, a fixed order, one rounding.
// mma.sync m16n8k16 with the weight rows as M (phase 1: 8 features' gate rows and their
// up rows, so that a thread has both) and an expert's tokens as N, 8 at a time: at a
// few tokens an expert the tensor rate is no bound.  Both operands keep K in the order
// in which a thread's 16-byte loads bring it, as in grouped_few.cu.
// What bounds the consumers is latency, a chunk's 0.7 us at the full rate of the stream:
// two groups of eight warps take every second chunk, its 32-input units dealt out to
// the warps; the tokens' values of a warp's next chunk are on their way while it has
// one; and a warp of its own adds the warps' sums up and writes h, so that none of
// them waits for the others at the end of a tile.
// h is kept as two 16-bit numbers, the second one the rounding error of the first, so
// the output is rounded once as if h were fp32; twice the (few) MMAs of phase 2.
#include "decode_ops.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int MAX_T = 32, MAX_R = 256;
constexpr int GROUPS = 2, GW = 8, CW = GROUPS * GW;  // consumer warps
constexpr int CONSUMERS = 32 * CW, THREADS = CONSUMERS + 64;
constexpr int PRODUCER = CW, FINISHER = CW + 1;      // warps
constexpr int SLOT = 32768;
constexpr int BLOCKS = 16;                   // most 64-input blocks of a chunk
constexpr int UNITS = 2 * BLOCKS / GW;       // most 32-input units of a chunk for a warp
constexpr int SORTERS = 256;
static_assert(MAX_R <= SORTERS, "one thread an assignment");
// Slots of the ring and buffers for the warps' sums (of 8 tokens each), by NT.  Both
// are multiples of the groups, so that a slot is always one group's: a wait names a
// round of its barrier by the round's parity, and a group that took every second round
// of a slot would take the end of the round before for that of its own.
constexpr int slots(int nt) { return nt <= 2 ? 6 : 4; }
constexpr int buffers(int nt) { return nt <= 2 ? 2 : 4; }
constexpr int SUM_FLOATS = CW * 128;         // of a buffer: [CW][32][4]
constexpr size_t sums_bytes(int nt) {        // phase 1: the buffers; phase 2: [CW][T][17]
    return std::max<size_t>((size_t)buffers(nt) * SUM_FLOATS, (size_t)CW * 8 * nt * 17) * sizeof(float);
}
constexpr int BAR_BYTES = 256;

struct Tab {
    int ids[MAX_R];
    float w[MAX_R];
    int first[MAX_R];
    int tok[MAX_R];      // by sorted position: token
    float pw[MAX_R];     // and weight
    int uexp[MAX_R], uoff[MAX_R], ucnt[MAX_R];  // touched experts, ascending: id, first position, tokens
    int n_uniq, abort;
};

struct Params {
    const uint16_t* x;
    const float* logits;
    uint16_t* out;
    int32_t* ids_out;
    uint16_t *hi, *lo;   // h by sorted position, [R][f] each
    uint32_t* err;
    unsigned long long* bar_count;
    int T, k, E, d, f;
    int cb1, cb2;        // 64-input blocks of a chunk of either phase
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

// Part c of `parts` of n things: [share(c), share(c + 1)).
__device__ __forceinline__ int share(int n, int c, int parts) { return (int)((long long)n * c / parts); }

// Phase 1: the tile at feature x of the list, of those before `end`: expert u,
// features i0 .. i0 + n - 1, box of map m (n = 8 >> m).
struct Tile1 {
    int u, i0, n, m;
    __device__ Tile1(int x, int end, int f) {
        u = x / f;
        i0 = x - u * f;
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

// A unit's 16 bytes of line `line` (128 bytes of 64 inputs) in a slot: 32 inputs
// `half`, lane t; the 128-byte swizzle of the box.
__device__ __forceinline__ uint4 weights_at(uint32_t slot, int line, int half, int t) {
    return dec::lds128(slot + 128u * line + ((uint32_t)((4 * half + t) ^ (line & 7)) << 4));
}

// Where a group is in phase 1's list of chunks.
struct Place1 {
    int x, b, q;                // tile's first feature, chunk's first block; chunks before
    int r0, r1;                 // sums before; of tiles of one chunk: of either group
    int i0, n, m, cnt, off;     // of the tile
    __device__ void tile(const Tab& tab, int end, int f) {
        const Tile1 t(x, end, f);
        i0 = t.i0;
        n = t.n;
        m = t.m;
        cnt = tab.ucnt[t.u];
        off = tab.uoff[t.u];
    }
    __device__ void step(const Tab& tab, int end, int f, int nb, int cb) {
        if (x >= end) return;
        ++q;
        if ((b += cb) < nb) return;
        b = 0;
        if (cb < nb || (q & 1)) r0 += ceil_div(cnt, 8);  // (the chunk was q - 1)
        else r1 += ceil_div(cnt, 8);
        x += n;
        if (x < end) tile(tab, end, f);
    }
};

// The buffer of sum n of a group's tile and the parity of its round: any buffer in
// turn where all warps have a part of every tile, else one of the group's.
template <int NBUF>
struct SumAt {
    int buf;
    uint32_t parity;
    __device__ SumAt(const Place1& c, int n, int group, bool one_chunk) {
        constexpr int EACH = NBUF / GROUPS;
        const int k = n + (one_chunk && group ? c.r1 : c.r0);
        buf = one_chunk ? group * EACH + k % EACH : k % NBUF;
        parity = (uint32_t)(one_chunk ? k / EACH : k / NBUF) & 1u;
    }
};

// NT: most groups of 8 tokens of an expert.
template <bool BF16, int NT>
__global__ void __launch_bounds__(THREADS, 1) expert_layer_kernel(const __grid_constant__ Maps maps, const Params p) {
    constexpr int NSLOT = slots(NT), NBUF = buffers(NT);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t ring = smem_u32(sm), full = ring + NSLOT * SLOT, empty = full + 8 * NSLOT;
    const uint32_t sum_full = empty + 8 * NSLOT, sum_empty = sum_full + 8 * NBUF, h_ready = sum_empty + 8 * NBUF;
    static_assert(16 * NSLOT + 16 * NBUF + 8 <= BAR_BYTES, "barrier area too small");
    static_assert(NSLOT % GROUPS == 0 && NBUF % GROUPS == 0, "a slot and a buffer are one group's");
    float* sums = reinterpret_cast<float*>(sm + NSLOT * SLOT + BAR_BYTES);
    Tab& tab = *reinterpret_cast<Tab*>(sm + NSLOT * SLOT + BAR_BYTES + sums_bytes(NT));
    volatile int* abort_flag = &tab.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = p.T * p.k, d = p.d, f = p.f, G = gridDim.x, cta = blockIdx.x;
    const int nb1 = d / 64, nb2 = f / 64, cb1 = p.cb1, cb2 = p.cb2;
    const bool one_chunk = cb1 >= nb1;  // a tile of phase 1 is one group's

    // ------------------------------------------------ phase 0: init, routing
    if (threadIdx.x == 0) tab.abort = 0;
    if (warp == PRODUCER && lane == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, GW);
        }
        for (int i = 0; i < NBUF; ++i) {
            tc::mbar_init(sum_full + 8 * i, one_chunk ? GW : CW);
            tc::mbar_init(sum_empty + 8 * i, 1);
        }
        tc::mbar_init(h_ready, 1);
        tc::fence_mbar_init();
        for (int i = 0; i < 4; ++i) {
            tc::tma_prefetch_desc(&maps.w13[i]);
            tc::tma_prefetch_desc(&maps.w2[i]);
        }
    }
    if (warp == FINISHER) {  // a hint, which returns no value: before the kernel ahead is complete
        const int lines = (p.T * p.E * 4 + 127) / 128;
        for (int i = lane; i < lines; i += 32)
            asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const char*>(p.logits) + 128 * (size_t)i));
    }
    // global memory is read and written from here on
    grid_dependency_wait();
    if (warp < CW) {
        for (int t = warp; t < p.T; t += CW)
            dec::route_token(p.logits + (size_t)t * p.E, p.E, p.k, &tab.ids[t * p.k], &tab.w[t * p.k]);
        dec::bar_sync(1, CONSUMERS);
    }
    if (threadIdx.x < SORTERS) {
        // Stable counting sort by expert, one thread an assignment.  An id out of
        // range (logits that are no numbers) has no expert.
        const int a = threadIdx.x;
        const int ea = a < R ? tab.ids[a] : INT_MAX;
        const bool va = (unsigned)ea < (unsigned)p.E;
        int lt = 0, before = 0, all = 0;
        for (int b = 0; b < R; ++b) {
            const int eb = tab.ids[b];
            const bool vb = (unsigned)eb < (unsigned)p.E;
            lt += vb && eb < ea;
            all += eb == ea;
            before += eb == ea && b < a;
        }
        const bool first = va && before == 0;
        tab.first[a] = first;
        if (a < R && !va) set_error(p.err, ERRBIT_RANGE);
        dec::bar_sync(2, SORTERS);
        int ui = 0, nu = 0;
        for (int b = 0; b < R; ++b) {
            const int fb = tab.first[b];
            nu += fb;
            ui += fb && tab.ids[b] < ea;
        }
        if (va) {
            tab.tok[lt + before] = a / p.k;
            tab.pw[lt + before] = tab.w[a];
        }
        if (first) {
            tab.uexp[ui] = ea;
            tab.uoff[ui] = lt;
            tab.ucnt[ui] = all;
        }
        if (a == 0) tab.n_uniq = nu;
        if (cta == 0 && p.ids_out && a < R) p.ids_out[a] = tab.ids[a];
    }
    __syncthreads();

    const int n_uniq = tab.n_uniq;
    const int x_lo = share(n_uniq * f, cta, G), x_hi = share(n_uniq * f, cta + 1, G);
    const int r_lo = share(d, cta, G), rows = share(d, cta + 1, G) - r_lo, tiles2 = ceil_div(rows, 16);

    if (warp == PRODUCER) {
        // ---------------------------------------------------------- producer
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
            for (int x = x_lo; ok && x < x_hi;) {
                const Tile1 t(x, x_hi, f);
                const int e = tab.uexp[t.u];
                for (int b = 0; b < nb1 && next(cb1 * 2 * t.n * 128); b += cb1, advance())
                    asm volatile(
                        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];"
                        :: "r"(ring + s * SLOT), "l"(&maps.w13[t.m]), "r"(full + 8 * s), "r"(0), "r"(t.i0), "r"(b), "r"(e) : "memory");
                x += t.n;
            }
            for (int i = 0; ok && i < tiles2; ++i) {
                const Tile2 t(rows, tiles2, i);
                const int m = t.n == p.rows2[0] ? 0 : t.n == p.rows2[1] ? 1 : t.n == p.rows2[2] ? 2 : 3;
                for (int u = 0; ok && u < n_uniq; ++u) {
                    const int e = tab.uexp[u];
                    for (int b = 0; b < nb2 && next(cb2 * t.n * 128); b += cb2, advance())
                        tc::tma_load_4d(ring + s * SLOT, &maps.w2[m], full + 8 * s, 0, r_lo + t.r0, b, e);
                }
            }
        }
        __syncwarp();
    } else if (warp == FINISHER) {
        // --------------------- phase 1's sums: h = SiLU(gate) up, two columns a lane
        const int g = lane >> 2, t = lane & 3;
        Place1 c{x_lo};
        if (c.x < x_hi) c.tile(tab, x_hi, f);
        while (c.x < x_hi) {
            const int group = c.q & 1, w0 = one_chunk ? group * GW : 0, w1 = one_chunk ? w0 + GW : CW;
            for (int n = 0; 8 * n < c.cnt; ++n) {
                const SumAt<NBUF> at(c, n, group, one_chunk);
                const int buf = at.buf;
                tc::mbar_wait(sum_full + 8 * buf, at.parity, abort_flag, p.err);
                __syncwarp();
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int w = w0; w < w1; ++w) {
                    const float4 o = *reinterpret_cast<const float4*>(sums + buf * SUM_FLOATS + (w * 32 + lane) * 4);
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
                    if (g < c.n && col < c.cnt) {
                        const float a = i ? v.y : v.x, u = i ? v.w : v.z;
                        const float h = a / (1.f + expf(-a)) * u;
                        const uint16_t hi = bits16<BF16>(h);
                        const float rest = h - value16<BF16>(hi);
                        const size_t to = (size_t)(c.off + col) * f + c.i0 + g;
                        p.hi[to] = hi;
                        p.lo[to] = bits16<BF16>(isfinite(rest) ? rest : 0.f);
                    }
                }
            }
            for (int b = 0; b < nb1; b += cb1) c.step(tab, x_hi, f, nb1, cb1);
        }
        // Every CTA's h is written before anyone reads it.  The arrival count only
        // grows, G a launch, so a CTA's own arrival tells it the count at which this
        // launch's barrier opens.
        __syncwarp();
        if (lane == 0) {
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
        grid_dependency_launch();
    } else {
        // --------------------------------------------------------- consumers
        const int g = lane >> 2, t = lane & 3, group = warp / GW, gw = warp % GW;
        float acc[NT][4];
        auto clear = [&] {
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        };
        auto release = [&](int q) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty + 8 * (q % NSLOT));
        };
        auto wait = [&](int q) { tc::mbar_wait(full + 8 * (q % NSLOT), (uint32_t)(q / NSLOT) & 1u, abort_flag, p.err); };
        // A wait that gave up goes on with what is in the slot: no barrier is left out,
        // and every address stays where it was.

        // ---- phase 1
        Place1 c{x_lo};
        if (c.x < x_hi) c.tile(tab, x_hi, f);
        if (group) c.step(tab, x_hi, f, nb1, cb1);
        // Units gw, gw + GW, ... of a chunk are this warp's.  As soon as the MMAs have a
        // unit's values, those of the warp's next chunk (or next 8 tokens) take their place.
        uint4 v[UNITS];
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
        clear();
        if (c.x < x_hi) {
            const From o = from(c, 0);
#pragma unroll
            for (int i = 0; i < UNITS; ++i) load(i, o);
        }
        while (c.x < x_hi) {
            Place1 to = c;
            to.step(tab, x_hi, f, nb1, cb1);
            to.step(tab, x_hi, f, nb1, cb1);
            const int units = 2 * min(cb1, nb1 - c.b), gf = min(g, c.n - 1);  // rows beyond the tile's: its last again
            const uint32_t slot = ring + (c.q % NSLOT) * SLOT;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (8 * n < c.cnt) {
                    From o{nullptr, 0};
                    if (8 * (n + 1) < c.cnt) o = from(c, n + 1);
                    else if (to.x < x_hi) o = from(to, 0);
                    if (n == 0) wait(c.q);
#pragma unroll
                    for (int i = 0; i < UNITS; ++i) {
                        const int unit = gw + GW * i, line = (unit >> 1) * 2 * c.n + gf;
                        if (unit < units)
                            mma<BF16>(acc[n], weights_at(slot, line, unit & 1, t), weights_at(slot, line + c.n, unit & 1, t), v[i]);
                        load(i, o);
                    }
                }
            release(c.q);
            if (to.x != c.x) {  // this group's last chunk of the tile
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (8 * n < c.cnt) {
                        const SumAt<NBUF> at(c, n, group, one_chunk);
                        const int buf = at.buf;
                        tc::mbar_wait(sum_empty + 8 * buf, at.parity ^ 1u, abort_flag, p.err);
                        *reinterpret_cast<float4*>(sums + buf * SUM_FLOATS + (warp * 32 + lane) * 4) =
                            make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(sum_full + 8 * buf);
                    }
                clear();
            }
            c = to;
        }

        // ---- phase 2
        tc::mbar_wait(h_ready, 0, abort_flag, p.err);
        grid_dependency_launch();  // the last phase: the next kernel may be scheduled
        float* mine = sums + warp * p.T * 17;
        for (int i = lane; i < p.T * 17; i += 32) mine[i] = 0.f;
        __syncwarp();
        int q = c.q;  // all of phase 1
        const int parts = ceil_div(nb2, cb2), chunks = n_uniq * parts;
        uint4 lo[UNITS];
        for (int i = 0; i < tiles2; ++i, q += chunks) {
            const Tile2 tl(rows, tiles2, i);
            const int ga = min(g, tl.n - 1), gb = min(g + 8, tl.n - 1);
            struct FromH {
                size_t at;
                int units;
            };
            auto from_h = [&](int j, int n) {
                const int u = j / parts, b = (j - u * parts) * cb2;
                return FromH{(size_t)(tab.uoff[u] + min(8 * n + g, tab.ucnt[u] - 1)) * f + 64 * b + 8 * t, 2 * min(cb2, nb2 - b)};
            };
            auto load_h = [&](int i, const FromH& o) {
                if (gw + GW * i < o.units) {
                    v[i] = dec::ldg_cg16(p.hi + o.at + 32 * (gw + GW * i));
                    lo[i] = dec::ldg_cg16(p.lo + o.at + 32 * (gw + GW * i));
                }
            };
            int j = (group + q) & 1;  // chunks that are even in the whole list are group 0's
            if (j < chunks) {
                const FromH o = from_h(j, 0);
#pragma unroll
                for (int i = 0; i < UNITS; ++i) load_h(i, o);
            }
            for (; j < chunks; j += GROUPS) {
                const int u = j / parts, b = (j - u * parts) * cb2, cnt = tab.ucnt[u], off = tab.uoff[u];
                const int units = 2 * min(cb2, nb2 - b);
                const uint32_t slot = ring + ((q + j) % NSLOT) * SLOT;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (8 * n < cnt) {
                        FromH o{0, 0};
                        if (8 * (n + 1) < cnt) o = from_h(j, n + 1);
                        else if (j + GROUPS < chunks) o = from_h(j + GROUPS, 0);
                        if (n == 0) wait(q + j);
#pragma unroll
                        for (int i = 0; i < UNITS; ++i) {
                            const int unit = gw + GW * i, line = (unit >> 1) * tl.n;
                            if (unit < units) {
                                const uint4 wa = weights_at(slot, line + ga, unit & 1, t), wb = weights_at(slot, line + gb, unit & 1, t);
                                mma<BF16>(acc[n], wa, wb, v[i]);
                                mma<BF16>(acc[n], wa, wb, lo[i]);
                            }
                            load_h(i, o);
                        }
                    }
                release(q + j);
                if ((j + GROUPS) / parts != u) {  // the group's last chunk of the expert
                    // columns 2 t and 2 t + 1, rows g and g + 8, into the tokens' sums
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int col = 8 * n + 2 * t + c;
                            if (col < cnt) {
                                const float w = tab.pw[off + col];
                                float* o = mine + tab.tok[off + col] * 17 + g;
                                o[0] += w * acc[n][c];
                                o[8] += w * acc[n][2 + c];
                            }
                        }
                    clear();
                    __syncwarp();
                }
            }
            dec::bar_sync(1, CONSUMERS);
            for (int j = threadIdx.x; j < p.T * 16; j += CONSUMERS) {
                const int tok = j >> 4, row = j & 15;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < CW; ++w) {
                    float* o = sums + (w * p.T + tok) * 17 + row;
                    s += *o;
                    *o = 0.f;
                }
                if (row < tl.n) p.out[(size_t)tok * d + r_lo + tl.r0 + row] = bits16<BF16>(s);
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

template <bool BF16, int NT>
cudaError_t launch(const Maps& maps, const Params& p, cudaStream_t s) {
    constexpr size_t smem = 1024 + (size_t)slots(NT) * SLOT + BAR_BYTES + sums_bytes(NT) + sizeof(Tab);
    static_assert(smem <= SMEM_MOST, "shared memory");
    cudaError_t e = allow_smem<expert_layer_kernel<BF16, NT>>();
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
    e = cudaLaunchKernelEx(&cfg, expert_layer_kernel<BF16, NT>, maps, p);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace

bool expert_layer_supported(int T, int k) { return T <= MAX_T && T * k <= MAX_R && k <= 32; }
size_t expert_layer_halves(int T, int k, int f) { return (size_t)2 * T * k * f; }

cudaError_t launch_expert_layer(const ExpertLayer& l, cudaStream_t s) {
    const bool bf = l.dtype == MOE_DT_BF16;
    const uint64_t d = l.d, f = l.f, E = l.E;
    Params p{};
    p.x = static_cast<const uint16_t*>(l.x);
    p.logits = l.logits;
    p.out = static_cast<uint16_t*>(l.out);
    p.ids_out = l.ids_out;
    p.hi = l.h;
    p.lo = l.h + (size_t)l.T * l.k * l.f;
    p.err = l.header;
    p.bar_count = reinterpret_cast<unsigned long long*>(l.header + WS_BAR_COUNT_WORD);
    p.T = l.T;
    p.k = l.k;
    p.E = l.E;
    p.d = l.d;
    p.f = l.f;
    // chunks of as many 64-input blocks each, at most BLOCKS
    p.cb1 = ceil_div(l.d / 64, ceil_div(l.d / 64, BLOCKS));
    p.cb2 = ceil_div(l.f / 64, ceil_div(l.f / 64, BLOCKS));
    Maps maps;
    bool ok = true;
    // gate_up as [expert][64-input block][gate, up][feature][64 inputs]
    const uint64_t d13[5] = {64, f, 2, d / 64, E}, s13[4] = {2 * d, 2 * f * d, 128, 4 * f * d};
    for (int i = 0; i < 4 && ok; ++i) {
        const uint32_t box[5] = {64, 8u >> i, 2, (uint32_t)p.cb1, 1};
        ok = make_tensor_map_16(&maps.w13[i], bf, l.w13, 5, d13, s13, box);
    }
    // down as [expert][64-input block][output feature][64 inputs]; a CTA has q or q + 1 of
    // them, in tiles of at most two sizes
    const uint64_t d2[4] = {64, d, f / 64, E}, s2[3] = {2 * f, 128, 2 * d * f};
    const int q = l.d / num_sms();
    for (int i = 0; i < 4 && ok; ++i) {
        const int rows = std::max(1, q + (i & 1)), tiles = ceil_div(rows, 16);
        p.rows2[i] = i < 2 ? rows / tiles : ceil_div(rows, tiles);
        const uint32_t box[4] = {64, (uint32_t)p.rows2[i], (uint32_t)p.cb2, 1};
        ok = make_tensor_map_16(&maps.w2[i], bf, l.w2, 4, d2, s2, box);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (l.T <= 8) return bf ? launch<true, 1>(maps, p, s) : launch<false, 1>(maps, p, s);
    if (l.T <= 16) return bf ? launch<true, 2>(maps, p, s) : launch<false, 2>(maps, p, s);
    return bf ? launch<true, 4>(maps, p, s) : launch<false, 4>(maps, p, s);
}

}  // namespace moe
