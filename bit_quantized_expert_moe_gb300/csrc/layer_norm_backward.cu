// Gradients of the layer norm (layer_norm.cu), given dh and dx', with the
// statistics taken again from x':
//   n  = (x' - m) r,  v = dh gamma
//   dx = dx' + r (v - mean v - n mean(v n));  dgamma = sum dh n,  dbeta = sum dh
// x' is the stored one, the value that every later reader sees.  Each tensor is
// read and written once.  Few rows are bound by the latency of two launches, one behind the
// other (100 rows 7.2 us); many by that and by the row groups' barriers rather than by memory:
// 4096 x 2048 17.1 to 18.1 us (3.7 to 3.9 TB/s), 4096 x 7168 48.9 (4.8), fp32 102.  4096 x 2048
// with two reductions a row 20.0, with one chunk a thread (two row groups for four) 22.9.
#include "layer_norm.cuh"

namespace moe {
namespace lnorm {
namespace {

constexpr int BLOCK_THREADS = 512;  // most threads of a block: 128 registers each

// A row group takes p.rows consecutive rows, the loads of the next SLOTS - 1
// under way while it computes one (SLOTS = 1: none).  One reduction a row, of x', x'^2,
// v and v x', and a second one around the mean where layer_norm.cu takes one.  The
// parameters' gradients add up in registers, then over the block's groups, then over the
// blocks, in a fixed order.
template <class T, int VPT, int SLOTS>
__global__ void __launch_bounds__(BLOCK_THREADS, 1) layer_norm_backward_kernel(const Args p) {
    extern __shared__ __align__(16) float smem[];
    // the kernel that adds the blocks' sums up may take its place already
    grid_dependency_launch();
    grid_dependency_wait();
    constexpr size_t CH = 8 * T::BYTES;
    const int grp = threadIdx.x / p.threads;
    RowGroup rg(p.threads, grp, smem + grp * RowGroup::SUM_FLOATS);
    const int chunks = p.D / 8, n = VPT * p.threads;
    const norm::ParamTable table(smem + p.groups * RowGroup::SUM_FLOATS, n);
    float* const space = smem + p.groups * RowGroup::SUM_FLOATS + 16 * n;
    // places in a slot: x', dh, dx'
    ThreadRing<T, 3 * VPT, SLOTS> ring(space);
    const float inv_d = 1.f / (float)p.D;
    const int vb = blockIdx.x * p.groups + grp;
    const int r_begin = min(p.T, vb * p.rows), r_end = min(p.T, r_begin + p.rows);
    const size_t row_bytes = (size_t)chunks * CH, next = CH * p.threads;
    const bool has_dx = p.dx_out;
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
                    ring.fetch(i, at(p.x, foff + i * next));
                    ring.fetch(VPT + i, at(p.dh, foff + i * next));
                    if (has_dx) ring.fetch(2 * VPT + i, at(p.dx_out, foff + i * next));
                }
        }
        ++fr;
        foff += row_bytes;
        ring.commit();
    };
    if (SLOTS > 1)
#pragma unroll
        for (int k = 0; k < SLOTS - 1; ++k) fetch();
    fill(table, p, false);
    for (int i = threadIdx.x; i < p.groups * RowGroup::SUM_FLOATS; i += blockDim.x) smem[i] = 0.f;
    __syncthreads();
    V8 a_gamma[VPT], a_beta[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) a_gamma[i] = a_beta[i] = v8(0.f);
    for (int r = r_begin; r < r_end; ++r, off += row_bytes) {
        if (SLOTS > 1) {
            fetch();
            ring.wait();
        }
        V8 x[VPT];
        typename T::Raw dhs[VPT];
        float2 q[4];
        // the sums of x, x^2, v and v x
        auto sums = [&](float (&t)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) q[k] = f2(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) {
                    const V8 v = mul(unpack8<T>(dhs[i]), table.get(0, i * p.threads + rg.tid));
                    add(q[0], x[i]);
                    dot(q[1], x[i], x[i]);
                    add(q[2], v);
                    dot(q[3], v, x[i]);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = q[k].x + q[k].y;
            rg.sum4(t);
        };
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in[i]) {
                x[i] = unpack8<T>(SLOTS > 1 ? ring.get(i) : raw_at<T>(p.x, off + i * next));
                dhs[i] = SLOTS > 1 ? ring.get(VPT + i) : raw_at<T>(p.dh, off + i * next);
            }
        float t[4], eps = p.eps, unit = 1.f;
        sums(t);
        float shift = t[0] * inv_d, var = t[1] * inv_d - shift * shift;
        if (__builtin_expect(!(shift * shift <= var && t[1] < INFINITY), 0)) {  // as in layer_norm.cu
            auto centre = [&](float sum) {
                const float2 m = f2(-sum * inv_d);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (in[i]) x[i] = fma(x[i], 1.f, V8{{m, m, m, m}});
                sums(t);
            };
            const bool ordinary = fabsf(t[0]) < 0x1p63f;
            if (ordinary) centre(t[0]);
            if (!(ordinary && t[1] < INFINITY)) {
                unit = UNIT;
                eps = fmaxf(eps * UNIT * UNIT, 0x1p-126f);
                float2 s = f2(0.f);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (in[i]) {
                        x[i] = mul(x[i], UNIT);
                        add(s, x[i]);
                    }
                centre(rg.sum(s.x + s.y));
            }
            shift = t[0] * inv_d;
            var = variance(t[1] * inv_d, shift);
        }
        const float rs = rsqrtf(var + eps);
        const float vm = t[2] * inv_d, vn = rs * (t[3] * inv_d - shift * vm), r1 = rs * unit;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in[i]) {
                const V8 nn = fma(x[i], rs, v8(-shift * rs)), dh = unpack8<T>(dhs[i]);
                a_gamma[i] = fma(dh, nn, a_gamma[i]);
                a_beta[i] = fma(dh, 1.f, a_beta[i]);
                const V8 v = fma(dh, table.get(0, i * p.threads + rg.tid), fma(nn, -vn, v8(-vm)));
                const V8 o = has_dx ? unpack8<T>(SLOTS > 1 ? ring.get(2 * VPT + i) : raw_at<T>(p.dx_out, off + i * next)) : v8(0.f);
                store_at<T>(p.dx, off + i * next, fma(v, r1, o));
            }
        ring.next();
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
                store8<F32>(space, c, a_gamma[i]);
                store8<F32>(space, n + c, a_beta[i]);
            }
        __syncthreads();
        if (grp == 0)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * p.threads + rg.tid;
                a_gamma[i] = fma(load8<F32>(space, c), 1.f, a_gamma[i]);
                a_beta[i] = fma(load8<F32>(space, n + c), 1.f, a_beta[i]);
            }
    }
    if (grp == 0) {
        float* const part = p.part + (size_t)blockIdx.x * 2 * p.D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * p.threads + rg.tid;
            if (c < chunks) {
                if (p.dgamma) store8<F32>(part, c, a_gamma[i]);
                if (p.dbeta) store8<F32>(part + p.D, c, a_beta[i]);
            }
        }
    }
}

// Adds the blocks' sums up in their order: 32 columns a block, 32 threads a column,
// so that a thread's few loads are all under way at once.  Launched as a programmatic
// dependent: it starts beside the gradients' kernel and waits for its results here.
__global__ void __launch_bounds__(1024) layer_norm_reduce_kernel(const Args p) {
    __shared__ float red[32][33];
    grid_dependency_launch();
    grid_dependency_wait();
    const int tx = threadIdx.x, ty = threadIdx.y, col = blockIdx.x * 32 + tx;
    void* const out = blockIdx.y ? p.dbeta : p.dgamma;
    if (!out) return;
    float s = 0.f;
    if (col < p.D) {
        const float* src = p.part + (size_t)blockIdx.y * p.D + col;
#pragma unroll 8
        for (int b = ty; b < p.blocks; b += 32) s += src[(size_t)b * 2 * p.D];
    }
    red[ty][tx] = s;
    __syncthreads();
    float t[1] = {red[tx][ty]};  // warp ty: column ty
    warp_sum(t);
    if (tx == 0 && blockIdx.x * 32 + ty < p.D) store1(p.ptype, out, blockIdx.x * 32 + ty, t[0]);
}

// One block an SM with as many row groups as its threads hold (15 named barriers),
// fewer where the rows are few.  640 threads: the same times; 768, which spill: 22.7 us
// at 4096 x 2048 for 18.1.
struct Plan {
    int vpt, threads, groups, rows, blocks;
};
Plan plan(int T, int D) {
    Plan b;
    b.vpt = D <= 1024 ? 1 : D <= 8192 ? 2 : 4;
    b.threads = norm::group_threads(D, b.vpt);
    b.groups = std::max(1, std::min({BLOCK_THREADS / b.threads, 15, ceil_div(T, num_sms())}));
    b.rows = std::max(1, ceil_div(T, num_sms() * b.groups));
    b.blocks = ceil_div(ceil_div(T, b.rows), b.groups);
    return b;
}

template <class T>
cudaError_t run_backward(const Args& p, const Plan& b, cudaStream_t s) {
    const int threads = b.groups * b.threads;
    const size_t slot = (size_t)3 * b.vpt * 8 * T::BYTES * threads;
    const size_t other = b.groups * RowGroup::SUM_FLOATS * sizeof(float) + norm::ParamTable::bytes(b.vpt * b.threads);
    const int slots = b.rows > 1 && b.vpt < 4 ? norm::ring_slots(slot, other) : 1;
    const size_t merge = b.groups > 1 ? (size_t)2 * b.vpt * b.threads * 8 * sizeof(float) : 0;
    const size_t smem = other + std::max(slots > 1 ? slots * slot : 0, merge);
    return norm::with_shape(b.vpt, slots, [&](auto v, auto n) {
        return launch_overlapped<layer_norm_backward_kernel<T, decltype(v)::value, decltype(n)::value>>(b.blocks, threads, smem, s, p);
    });
}

}  // namespace
}  // namespace lnorm

// No plan has more blocks than SMs or rows.
size_t layer_norm_partial_floats(int T, int D) { return (size_t)std::min(T, num_sms()) * 2 * D; }

cudaError_t launch_layer_norm_backward(const LayerNormShape& n, const LayerNormGrads& g, float* part, cudaStream_t s) {
    const lnorm::Plan b = lnorm::plan(n.T, n.D);
    lnorm::Args a{};
    a.T = n.T;
    a.D = n.D;
    a.eps = n.eps;
    a.ptype = n.param_dtype;
    a.gamma = n.gamma;
    a.x = g.x_out;
    a.dh = g.dh;
    a.dx_out = g.dx_out;
    a.dx = g.dx;
    a.dgamma = g.dgamma;
    a.dbeta = g.dbeta;
    a.threads = b.threads;
    a.groups = b.groups;
    a.rows = b.rows;
    a.blocks = b.blocks;
    a.part = part;
    const cudaError_t e = n.dtype == MOE_DT_BF16  ? lnorm::run_backward<Bf16>(a, b, s)
                          : n.dtype == MOE_DT_F16 ? lnorm::run_backward<F16>(a, b, s)
                                                  : lnorm::run_backward<F32>(a, b, s);
    if (e != cudaSuccess || (!g.dgamma && !g.dbeta)) return e;
    return launch_overlapped(lnorm::layer_norm_reduce_kernel, dim3(ceil_div(n.D, 32), 2), dim3(32, 32), 0, s, a);
}

}  // namespace moe
