// Layer norm before a block, with the residual sum in front of it.
//
//   x' = x + y                       (without y: x' = x, and x' is not written)
//   h  = (x' - m) r gamma + beta     m = mean x',  r = (mean (x' - m)^2 + eps)^-1/2
//
// h is taken from x' before its rounding, so both outputs are rounded once.
// Every tensor is read and written once: bound by memory.  The threads of a
// RowGroup share a row and hold it in registers, VPT chunks of 8 elements each.
//
// One reduction a row, of sum x' and sum x'^2, where the mean is no larger than the
// deviation: the difference of the mean square and the squared mean then loses a bit at
// most.  Rows farther from zero, which would lose |m|^2 / variance of their digits, and
// those whose squares leave fp32, take a second reduction, of c = x' - m0 and c^2 around
// m0, the mean as fp32 has it (off by some 2^-24 |m|):
//   m = m0 + mean c,  variance = mean c^2 - (mean c)^2
// without loss, since mean c is a rounding's size.
// 4096 x 7168 with the residual 41 us (5.7 TB/s, 84 % of the copy's rate), 4096 x 2048
// 13.0 (5.2 TB/s); with two reductions for every row 15.0.
#include "layer_norm.cuh"

namespace moe {
namespace lnorm {
namespace {

// A block's row groups take every gridDim-th set of rows, SLOTS - 1 of a group's
// rows under way while it computes one (SLOTS = 1: a call with few rows, one for
// a group, which takes the parameters as it needs them).
template <class T, int VPT, int SLOTS, bool RESIDUAL>
__global__ void __launch_bounds__(SLOTS == 1 || VPT == 4 ? 512 : 1024, 1) layer_norm_kernel(const Args p) {
    extern __shared__ __align__(16) float smem[];
    grid_dependency_launch();
    grid_dependency_wait();
    constexpr size_t CH = 8 * T::BYTES;
    constexpr int PLACES = RESIDUAL ? 2 * VPT : VPT;
    const int groups = blockDim.x / p.threads, grp = threadIdx.x / p.threads;
    RowGroup rg(p.threads, grp, smem + grp * RowGroup::SUM_FLOATS);
    ThreadRing<T, PLACES, SLOTS> ring(smem + groups * RowGroup::SUM_FLOATS);
    const norm::ParamTable table(smem + groups * RowGroup::SUM_FLOATS +
                                 (SLOTS > 1 ? ring.BYTES_PER_THREAD / 4 * (int)blockDim.x : 0), VPT * p.threads);
    const int chunks = p.D / 8, step = gridDim.x * groups;
    const float inv_d = 1.f / (float)p.D;
    const size_t row_bytes = (size_t)chunks * CH, step_bytes = row_bytes * step, next = CH * p.threads;
    bool in[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) in[i] = i * p.threads + rg.tid < chunks;

    int r = blockIdx.x * groups + grp, fr = r;
    size_t off = row_bytes * r + CH * rg.tid, foff = off;  // of this thread's first chunk in row r; in the next to fetch
    auto fetch = [&]() {
        if (fr < p.T) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) {
                    ring.fetch(i, at(p.x, foff + i * next));
                    if (RESIDUAL) ring.fetch(VPT + i, at(p.y, foff + i * next));
                }
        }
        fr += step;
        foff += step_bytes;
        ring.commit();
    };
    if (SLOTS > 1) {
#pragma unroll
        for (int k = 0; k < SLOTS - 1; ++k) fetch();
        fill(table, p, true);
    }
    for (int i = threadIdx.x; i < groups * RowGroup::SUM_FLOATS; i += blockDim.x) smem[i] = 0.f;
    __syncthreads();
    for (; r < p.T; r += step, off += step_bytes) {
        if (SLOTS > 1) {
            fetch();
            ring.wait();
        }
        V8 x[VPT];
        float2 s = f2(0.f), sq = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            x[i] = v8(0.f);
            if (in[i]) {
                x[i] = unpack8<T>(SLOTS > 1 ? ring.get(i) : raw_at<T>(p.x, off + i * next));
                if (RESIDUAL)
                    x[i] = fma(unpack8<T>(SLOTS > 1 ? ring.get(VPT + i) : raw_at<T>(p.y, off + i * next)), 1.f, x[i]);
                add(s, x[i]);
                dot(sq, x[i], x[i]);
            }
        }
        float t[2] = {s.x + s.y, sq.x + sq.y};
        rg.sum2(t);
        float shift = t[0] * inv_d, var = t[1] * inv_d - shift * shift, eps = p.eps;
        if (RESIDUAL)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) store_at<T>(p.x_out, off + i * next, x[i]);
        // the same for the group's threads, and true for a NaN
        if (__builtin_expect(!(shift * shift <= var && t[1] < INFINITY), 0)) {
            // around the mean: x is centred
            auto centre = [&](float sum) {
                const float2 m = f2(-sum * inv_d);
                s = sq = f2(0.f);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (in[i]) {
                        x[i] = fma(x[i], 1.f, V8{{m, m, m, m}});
                        add(s, x[i]);
                        dot(sq, x[i], x[i]);
                    }
                t[0] = s.x + s.y;
                t[1] = sq.x + sq.y;
                rg.sum2(t);
            };
            const bool ordinary = fabsf(t[0]) < 0x1p63f;
            if (ordinary) centre(t[0]);
            // squares beyond fp32: in other units (x' or x' - m0, whose normalised row is the same)
            if (!(ordinary && t[1] < INFINITY)) {
                eps = fmaxf(eps * UNIT * UNIT, 0x1p-126f);
                s = f2(0.f);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    x[i] = mul(x[i], UNIT);
                    if (in[i]) add(s, x[i]);
                }
                centre(rg.sum(s.x + s.y));
            }
            shift = t[0] * inv_d;
            var = variance(t[1] * inv_d, shift);
        }
        const float rs = rsqrtf(var + eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in[i]) {
                const int c = i * p.threads + rg.tid;
                const V8 g = SLOTS > 1 ? table.get(0, c) : gamma_of(p, c), b = SLOTS > 1 ? table.get(1, c) : beta_of(p, c);
                store_at<T>(p.h, off + i * next, fma(fma(x[i], rs, v8(-shift * rs)), g, b));
            }
        ring.next();
    }
    cp_async_wait<0>();
}

template <class T>
cudaError_t run(Args p, cudaStream_t s) {
    const int vpt = norm::chunks_per_thread(p.D);
    p.threads = norm::group_threads(p.D, vpt);
    const size_t sums = RowGroup::SUM_FLOATS * sizeof(float), table = norm::ParamTable::bytes(vpt * p.threads);
    // one block an SM, with as many row groups as 1024 threads hold and the rows fill
    int groups = std::max(1, std::min({(vpt == 4 ? 512 : 1024) / p.threads, 15, p.T / num_sms()}));
    const size_t slot = (size_t)(p.y ? 2 : 1) * vpt * 8 * T::BYTES * p.threads;  // of one group
    int slots = 1;
    if (p.T > num_sms() && vpt < 4)
        for (; slots == 1 && groups > 0; --groups)
            if ((slots = norm::ring_slots(slot * groups, sums * groups + table)) > 1) break;
    if (slots == 1) groups = 1;
    const int threads = groups * p.threads;
    const int blocks = slots > 1 ? std::min(ceil_div(p.T, groups), num_sms()) : p.T;
    const size_t smem = groups * sums + (slots > 1 ? slots * slot * groups + table : 0);
    return norm::with_shape(vpt, slots, [&](auto v, auto n) {
        constexpr int V = decltype(v)::value, N = decltype(n)::value;
        return p.y ? launch_overlapped<layer_norm_kernel<T, V, N, true>>(blocks, threads, smem, s, p)
                   : launch_overlapped<layer_norm_kernel<T, V, N, false>>(blocks, threads, smem, s, p);
    });
}

}  // namespace
}  // namespace lnorm

cudaError_t launch_layer_norm(const LayerNormShape& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s) {
    lnorm::Args a{};
    a.T = n.T;
    a.D = n.D;
    a.eps = n.eps;
    a.ptype = n.param_dtype;
    a.gamma = n.gamma;
    a.beta = n.beta;
    a.x = x;
    a.y = y;
    a.x_out = x_out;
    a.h = h;
    return n.dtype == MOE_DT_BF16  ? lnorm::run<Bf16>(a, s)
           : n.dtype == MOE_DT_F16 ? lnorm::run<F16>(a, s)
                                   : lnorm::run<F32>(a, s);
}

}  // namespace moe
