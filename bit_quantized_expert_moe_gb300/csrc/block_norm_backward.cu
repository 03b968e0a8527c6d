// Gradients of the block norms (block_norm.cu), given dx' and dh, with the
// statistics taken again from y and x':
//   D  = dx' + r2 v - x' r2^3 mean(v x'),   v = dh gamma_pre;   dx = D
//   q  = alpha gate gamma_post D;  dy = r1 q - y r1^3 mean(q y)
//   dgamma_pre = sum dh x' r2,  dgate = sum alpha D n,  dgamma_post = sum alpha gate D y r1
// x' is the stored one, the value that every later reader sees.  Each tensor is
// read and written once: bound by memory.
#include "block_norm.cuh"

namespace moe {
namespace norm {
namespace {

constexpr int BLOCK_THREADS = 512;  // most threads of a block: 128 registers each

// Rows of about 2^40 (1e12) and more, whose sums or coefficients (gradients over
// squares) would leave fp32's range, are taken a second time, in units that make them
// of ordinary size: a sum at a time, since the six at once spill registers of the
// ordinary rows (4096 x 5120 with 64 gates 81.6 -> 87.2 us; so 81.8).
constexpr float LARGE_SUM = 0x1p80f;
__device__ __forceinline__ float unit(float sum) { return !(sum < INFINITY) ? 0x1p-80f : sum < 0x1p40f ? 1.f : 0x1p-40f; }

// A row group takes p.rows consecutive rows, the loads of the next SLOTS - 1
// under way while it computes one (SLOTS = 1: none).  One reduction a row:
// sum(q y) is taken apart into sums that do not wait for D, with
// w = alpha gate gamma_post y:
//   sum(q y) = sum(w dx') + r2 sum(w v) - r2^3 mean(v x') sum(w x').
// The parameters' gradients add up in registers.  While the gate row stays the
// same, gate and gamma_post are factors of one sum z = sum D y r1:
// dgate = alpha gamma_post z, dgamma_post = sum over gate rows of alpha gate z.
// A gate row that lies wholly inside the group's rows is written at once; one
// that is shared with the neighbours, the group's first or last, goes to gate_part.
// A chunk's tensors stay in registers for the second half of a row (VPT = 1) or are
// taken a second time from where they lie (4096 x 5120 fp32 171 -> 120 us, where
// they did not all fit; bf16 with 64 gates 161 -> 81).
// ALL: y, gamma_post, gamma_pre, dx' and dh are there and the rows share one gate.
template <class T, int VPT, int SLOTS, bool ALL>
__global__ void __launch_bounds__(BLOCK_THREADS, 1) block_norm_backward_kernel(const Args p) {
    extern __shared__ __align__(16) float smem[];
    // the kernel that adds the blocks' sums up may take its place already
    grid_dependency_launch();
    grid_dependency_wait();
    const int grp = threadIdx.x / p.threads;
    RowGroup rg(p.threads, grp, smem + grp * RowGroup::SUM_FLOATS);
    const int chunks = p.D / 8, n = VPT * p.threads;
    const bool one_gate = p.S == p.T, row_gate = !ALL && p.gate && !one_gate;
    const ParamTable table(smem + p.groups * RowGroup::SUM_FLOATS, n);
    float* const space = smem + p.groups * RowGroup::SUM_FLOATS + 16 * n;
    // places in a slot: x', dh, dx', y
    ThreadRing<T, 4 * VPT, SLOTS> ring(space);
    const float inv_d = 1.f / (float)p.D;
    const int vb = blockIdx.x * p.groups + grp;
    const int r_begin = min(p.T, vb * p.rows), r_end = min(p.T, r_begin + p.rows);
    const int g_first = r_begin / p.S;
    constexpr size_t CH = 8 * T::BYTES;
    const bool has_y = ALL || p.y, has_post = ALL || p.gamma_post, has_dh = ALL || p.dh, has_dx = ALL || p.dx_out;
    const size_t row_bytes = (size_t)chunks * CH, next = CH * p.threads;
    size_t off = row_bytes * r_begin + CH * rg.tid, foff = off;
    int fr = r_begin;  // the next row to fetch, at foff
    bool in[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) in[i] = i * p.threads + rg.tid < chunks;
    auto fetch = [&]() {
        if (fr < r_end) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) {
                    if (has_dh) {
                        ring.fetch(i, at(p.x, foff + i * next));
                        ring.fetch(VPT + i, at(p.dh, foff + i * next));
                    }
                    if (has_dx) ring.fetch(2 * VPT + i, at(p.dx_out, foff + i * next));
                    if (has_y) ring.fetch(3 * VPT + i, at(p.y, foff + i * next));
                }
        }
        ++fr;
        foff += row_bytes;
        ring.commit();
    };
    if (SLOTS > 1)
#pragma unroll
        for (int k = 0; k < SLOTS - 1; ++k) fetch();
    table.fill(p);
    for (int i = threadIdx.x; i < p.groups * RowGroup::SUM_FLOATS; i += blockDim.x) smem[i] = 0.f;
    __syncthreads();
    V8 a_post[VPT], a_pre[VPT], z[VPT];
    V8 ka = v8(0.f), kb = v8(0.f);  // the parameters of a chunk: kept for VPT = 1
#pragma unroll
    for (int i = 0; i < VPT; ++i) a_post[i] = a_pre[i] = z[i] = v8(0.f);
    // A and B into ka, kb.  VPT = 1: when a gate begins, its row at chunk grow.
    // Else: before each use; a block is one row group then (of more than 256
    // threads), and its table's A is filled again when a gate begins, by the thread
    // that reads it.
    auto params = [&](int c, size_t grow) {
        ka = table.get(0, c);
        if (VPT == 1 && row_gate) ka = mul(ka, load8(p.ptype, p.gate, grow + c));
        if (has_dh) kb = table.get(1, c);
    };
    bool fresh = true;  // the row is the first of its gate here
    for (int r = r_begin; r < r_end; ++r, off += row_bytes) {
        const int g = ALL ? 0 : r / p.S;
        const size_t grow = (size_t)g * chunks;
        if (SLOTS > 1) {
            fetch();
            ring.wait();
        }
        // a chunk of the row's tensors: kept (VPT = 1) or taken a second time
        struct Chunk {
            typename T::Raw x, dh, dx, y;
        } kept;
        auto load = [&](int i) {
            Chunk k{};
            if (has_dh) {
                k.x = SLOTS > 1 ? ring.get(i) : raw_at<T>(p.x, off + i * next);
                k.dh = SLOTS > 1 ? ring.get(VPT + i) : raw_at<T>(p.dh, off + i * next);
            }
            if (has_dx) k.dx = SLOTS > 1 ? ring.get(2 * VPT + i) : raw_at<T>(p.dx_out, off + i * next);
            if (has_y) k.y = SLOTS > 1 ? ring.get(3 * VPT + i) : raw_at<T>(p.y, off + i * next);
            return k;
        };
        float2 s[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) s[k] = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * p.threads + rg.tid;
            if (in[i]) {
                const Chunk k = load(i);
                if (VPT == 1) kept = k;
                if (VPT > 1 && row_gate && fresh) table.fill_a(p, c, grow + c, true);
                if (VPT > 1 || fresh) params(c, grow);
                const V8 x = unpack8<T>(k.x), v = mul(unpack8<T>(k.dh), kb), y = unpack8<T>(k.y);
                dot(s[0], x, x);
                dot(s[1], v, x);
                if (has_post) {
                    const V8 w = mul(ka, y);
                    dot(s[2], y, y);
                    dot(s[3], w, unpack8<T>(k.dx));
                    dot(s[4], w, v);
                    dot(s[5], w, x);
                }
            }
        }
        fresh = false;
        float t[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) t[k] = s[k].x + s[k].y;
        rg.sum6(t);
        float r2 = has_dh ? rsqrtf(t[0] * inv_d + p.eps) : 0.f;
        // r^3 by itself may leave fp32's range (a row of zeros and an eps of 1e-26),
        // which 0 does not bring back: one factor r after the other
        float c2 = r2 * (r2 * (r2 * (t[1] * inv_d)));
        float r1 = has_post ? rsqrtf(t[2] * inv_d + p.eps) : 1.f;
        float c1 = has_post ? r1 * (r1 * (r1 * ((t[3] + r2 * t[4] - c2 * t[5]) * inv_d))) : 0.f;
        // The row's outputs.  LARGE: x' in units of 1 / ux, y of 1 / uy.
        auto finish = [&](auto large, float ux, float uy) {
            constexpr bool LARGE = decltype(large)::value;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * p.threads + rg.tid;
                if (in[i]) {
                    const Chunk k = VPT == 1 ? kept : load(i);
                    if (VPT > 1) params(c, grow);
                    V8 x = unpack8<T>(k.x), d;
                    const V8 dh = mul(unpack8<T>(k.dh), r2);
                    if (LARGE) x = mul(x, ux);
                    a_pre[i] = fma(dh, x, a_pre[i]);
                    if (LARGE) d = fma(fma(x, -c2, mul(dh, kb)), ux, unpack8<T>(k.dx));
                    else d = fma(x, -c2, fma(dh, kb, unpack8<T>(k.dx)));
                    store_at<T>(p.dx, off + i * next, d);
                    if (has_y) {
                        V8 y = unpack8<T>(k.y);
                        const V8 dr = mul(d, r1);
                        if (LARGE) y = mul(y, uy);
                        z[i] = fma(dr, y, z[i]);
                        V8 e = fma(y, -c1, mul(dr, ka));
                        if (LARGE) e = mul(e, uy);
                        store_at<T>(p.dy, off + i * next, e);
                    }
                }
            }
        };
        // the same for the group's threads, and true for a NaN
        if (__builtin_expect(!(t[0] + t[2] < LARGE_SUM), 0)) {
            const float ux = unit(t[0]), uy = has_post ? unit(t[2]) : 1.f;
            auto sum = [&](auto term) {
                float2 q = f2(0.f);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (in[i]) {
                        const Chunk k = VPT == 1 ? kept : load(i);
                        if (VPT > 1) params(i * p.threads + rg.tid, grow);
                        term(q, k);
                    }
                return q.x + q.y;
            };
            auto xs = [&](const Chunk& k) { return mul(unpack8<T>(k.x), ux); };
            auto ys = [&](const Chunk& k) { return mul(unpack8<T>(k.y), uy); };
            auto vs = [&](const Chunk& k) { return mul(unpack8<T>(k.dh), kb); };
            t[0] = sum([&](float2& q, const Chunk& k) { dot(q, xs(k), xs(k)); });
            t[1] = sum([&](float2& q, const Chunk& k) { dot(q, vs(k), xs(k)); });
            if (has_post) {
                t[2] = sum([&](float2& q, const Chunk& k) { dot(q, ys(k), ys(k)); });
                t[3] = sum([&](float2& q, const Chunk& k) { dot(q, mul(ka, ys(k)), unpack8<T>(k.dx)); });
                t[4] = sum([&](float2& q, const Chunk& k) { dot(q, mul(ka, ys(k)), vs(k)); });
                t[5] = sum([&](float2& q, const Chunk& k) { dot(q, mul(ka, ys(k)), xs(k)); });
            }
            rg.sum6(t);
            r2 = has_dh ? rsqrtf(t[0] * inv_d + p.eps * ux * ux) : 0.f;
            c2 = r2 * (r2 * (r2 * (t[1] * inv_d)));
            r1 = has_post ? rsqrtf(t[2] * inv_d + p.eps * uy * uy) : 1.f;
            c1 = has_post ? r1 * (r1 * (r1 * ((t[3] + ux * (r2 * t[4] - c2 * t[5])) * inv_d))) : 0.f;
            finish(std::true_type{}, ux, uy);
        } else {
            finish(std::false_type{}, 1.f, 1.f);
        }
        ring.next();
        // the gate row ends here
        if (has_y && (r + 1 == r_end || (!ALL && r + 1 == (g + 1) * p.S))) {
            fresh = true;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * p.threads + rg.tid;
                if (c < chunks) {
                    const V8 az = mul(z[i], p.alpha), post = p.gate ? mul(load8(p.ptype, p.gate, grow + c), az) : az;
                    a_post[i] = ALL ? post : fma(post, 1.f, a_post[i]);
                    const V8 w = p.gamma_post ? mul(load8(p.ptype, p.gamma_post, c), az) : az;
                    z[i] = one_gate ? w : v8(0.f);
                    if (p.dgate && !one_gate) {
                        float* gp = p.gate_part + (size_t)vb * 2 * p.D;
                        if (g * p.S >= r_begin && r_end - g * p.S >= p.S) store8(p.ptype, p.dgate, grow + c, w);
                        else store8<F32>(gp + (g == g_first ? 0 : p.D), c, w);
                    }
                }
            }
        }
    }

    // the block's groups add theirs up in order and write one partial sum; the
    // ring's space is free
    cp_async_wait<0>();
    for (int k = 1; k < p.groups; ++k) {
        __syncthreads();
        if (grp == k)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * p.threads + rg.tid;
                store8<F32>(space, c, a_post[i]);
                store8<F32>(space, n + c, a_pre[i]);
                store8<F32>(space, 2 * n + c, z[i]);
            }
        __syncthreads();
        if (grp == 0)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * p.threads + rg.tid;
                a_post[i] = fma(load8<F32>(space, c), 1.f, a_post[i]);
                a_pre[i] = fma(load8<F32>(space, n + c), 1.f, a_pre[i]);
                z[i] = fma(load8<F32>(space, 2 * n + c), 1.f, z[i]);
            }
    }
    if (grp == 0) {
        float* const part = p.part + (size_t)blockIdx.x * 3 * p.D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * p.threads + rg.tid;
            if (c < chunks) {
                if (p.dgamma_post) store8<F32>(part, c, a_post[i]);
                if (p.dgamma_pre) store8<F32>(part + p.D, c, a_pre[i]);
                if (p.dgate && one_gate) store8<F32>(part + 2 * p.D, c, z[i]);
            }
        }
    }
}

// Sums partial sums in their order, 32 columns a block.  gamma_post and
// gamma_pre (and the one gate row that all rows share): 32 threads a column,
// so that a thread's few loads are all under way at once.  A gate row of
// several that row groups share: the groups are few, 8 threads a column and four
// gate rows a block; there are at most `shared` such rows.  Launched as a
// programmatic dependent: it starts beside the gradients' kernel and waits for
// its results here.
__global__ void __launch_bounds__(1024) block_norm_reduce_kernel(const Args p, int sums, int shared) {
    __shared__ float red[32][33];
    grid_dependency_launch();
    grid_dependency_wait();
    const int tx = threadIdx.x, ty = threadIdx.y, col = blockIdx.x * 32 + tx;
    if ((int)blockIdx.y < sums) {
        const int what = blockIdx.y;
        void* out = what == 0 ? p.dgamma_post : what == 1 ? p.dgamma_pre : p.dgate;
        if (!out) return;
        float s = 0.f;
        if (col < p.D) {
            const float* src = p.part + (size_t)what * p.D + col;
#pragma unroll 8
            for (int b = ty; b < p.blocks; b += 32) s += src[(size_t)b * 3 * p.D];
        }
        red[ty][tx] = s;
        __syncthreads();
        float t[1] = {red[tx][ty]};  // warp ty: column ty
        warp_sum(t);
        if (tx == 0 && blockIdx.x * 32 + ty < p.D) store1(p.ptype, out, blockIdx.x * 32 + ty, t[0]);
        return;
    }
    for (int j0 = 4 * ((int)blockIdx.y - sums); j0 < shared; j0 += 4 * ((int)gridDim.y - sums)) {
        const int j = j0 + (ty >> 3);
        // gate row j, or the one that the row groups j and j + 1 share
        const bool by_gate = p.S >= p.rows;
        const int g = by_gate ? j : (int)((long long)(j + 1) * p.rows / p.S);
        const int first = g * p.S, end = first + p.S;  // the gate row's rows
        const int b0 = first / p.rows, b1 = (end - 1) / p.rows;
        const bool todo = j < shared && col < p.D && b0 != b1 && (by_gate || b0 == j);
        float s = 0.f;
        if (todo)
#pragma unroll 4
            for (int b = b0 + (ty & 7); b <= b1; b += 8)
                // the row group starts in this gate row, or in an earlier one
                s += p.gate_part[((size_t)b * 2 + (b * p.rows < first)) * p.D + col];
        red[ty][tx] = s;
        __syncthreads();
        if (todo && (ty & 7) == 0) {
            for (int i = 1; i < 8; ++i) s += red[ty + i][tx];
            store1(p.ptype, p.dgate, (size_t)g * p.D + col, s);
        }
        __syncthreads();
    }
}

// How the backward pass splits the rows: one block an SM with as many row
// groups as its threads hold (15 named barriers), fewer where the rows are few.
// 4096 x 2048: 25 us with two groups of 256 threads; 40 with three at 80
// registers, which spill; two chunks a thread and four groups of 128 take the
// same there and 22 instead of 14 us at 1155 x 1288, whose row groups would have
// half the threads.
struct BackwardPlan {
    int vpt, threads, groups, rows, blocks;
};
BackwardPlan backward_plan(int T, int D) {
    BackwardPlan b;
    b.vpt = chunks_per_thread(D);
    b.threads = group_threads(D, b.vpt);
    b.groups = std::max(1, std::min({BLOCK_THREADS / b.threads, 15, ceil_div(T, num_sms())}));
    b.rows = std::max(1, ceil_div(T, num_sms() * b.groups));
    b.blocks = ceil_div(ceil_div(T, b.rows), b.groups);
    return b;
}

template <class T>
cudaError_t run_backward(const Args& p, const BackwardPlan& b, bool all, cudaStream_t s) {
    const int threads = b.groups * b.threads;
    const size_t slot = (size_t)4 * b.vpt * 8 * T::BYTES * threads;
    const size_t other = b.groups * RowGroup::SUM_FLOATS * sizeof(float) + ParamTable::bytes(b.vpt * b.threads);
    const int slots = b.rows > 1 && b.vpt < 4 ? ring_slots(slot, other) : 1;
    const size_t merge = b.groups > 1 ? (size_t)3 * b.vpt * b.threads * 8 * sizeof(float) : 0;
    const size_t smem = other + std::max(slots > 1 ? slots * slot : 0, merge);
    return with_shape(b.vpt, slots, [&](auto v, auto n) {
        constexpr int V = decltype(v)::value, N = decltype(n)::value;
        return all ? launch_overlapped<block_norm_backward_kernel<T, V, N, true>>(b.blocks, threads, smem, s, p)
                   : launch_overlapped<block_norm_backward_kernel<T, V, N, false>>(b.blocks, threads, smem, s, p);
    });
}

cudaError_t run_reduce(const Args& p, cudaStream_t s) {
    const bool one_gate = p.S == p.T;
    const int sums = p.dgate && one_gate ? 3 : 2;
    // gate rows of at least a group's rows: each may be shared; smaller ones: one
    // for two neighbouring groups, and none where every group starts with a gate
    // row (2048 x 4096 with a gate for every row: 287 -> 47 us, when every gate row
    // had its blocks here)
    const int shared = !p.dgate || one_gate ? 0 : p.S >= p.rows ? p.T / p.S : p.rows % p.S ? ceil_div(p.T, p.rows) - 1 : 0;
    return launch_overlapped(block_norm_reduce_kernel, dim3(ceil_div(p.D, 32), sums + std::min(ceil_div(shared, 4), 1024)),
                            dim3(32, 32), 0, s, p, sums, shared);
}

}  // namespace
}  // namespace norm

// No plan has more blocks than SMs or rows, and its row groups never become fewer
// with the rows: so what does for many rows does for fewer, whose blocks may be more.
size_t block_norm_partial_floats(int T, int D, int G) {
    const norm::BackwardPlan b = norm::backward_plan(T, D);
    return (size_t)std::min(T, num_sms()) * D * (3 + (G > 1 ? 2 * b.groups : 0));
}

cudaError_t launch_block_norm_backward(const NormShape& n, const NormGrads& g, float* part, cudaStream_t s) {
    const bool all = g.y && n.gamma_post && g.dh && g.dx_out && n.G == 1;
    const norm::BackwardPlan b = norm::backward_plan(n.T, n.D);
    norm::Args a = norm::common_args(n);
    a.x = g.x_out;
    a.y = g.y;
    a.dx_out = g.dx_out;
    a.dh = g.dh;
    a.dx = g.dx;
    a.dy = g.dy;
    a.dgamma_post = g.dgamma_post;
    a.dgate = g.dgate;
    a.dgamma_pre = g.dgamma_pre;
    a.threads = b.threads;
    a.groups = b.groups;
    a.rows = b.rows;
    a.blocks = b.blocks;
    a.part = part;
    a.gate_part = part + (size_t)b.blocks * 3 * n.D;
    const cudaError_t e = n.dtype == MOE_DT_BF16  ? norm::run_backward<Bf16>(a, b, all, s)
                    : n.dtype == MOE_DT_F16 ? norm::run_backward<F16>(a, b, all, s)
                                            : norm::run_backward<F32>(a, b, all, s);
    if (e != cudaSuccess || (!g.dgamma_post && !g.dgate && !g.dgamma_pre)) return e;
    return norm::run_reduce(a, s);
}

}  // namespace moe
