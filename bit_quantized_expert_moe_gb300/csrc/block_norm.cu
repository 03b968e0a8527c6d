// Norms before and after a block, fused with its gate and residual scale.
//
//   n  = y r1 gamma_post   (r1 = (mean y^2 + eps)^-1/2; without gamma_post n = y)
//   x' = x + alpha gate n  (gate per channel, one row for each T / G tokens)
//   h  = x' r2 gamma_pre   (r2 = (mean x'^2 + eps)^-1/2)
//
// h is taken from x' before its rounding, so both outputs are rounded once.
// Every tensor is read and written once: bound by memory.  The threads of a
// RowGroup share a row and hold it in registers, VPT chunks of 8 elements each.
#include "block_norm.cuh"

namespace moe {
namespace norm {
namespace {

constexpr float UNIT = 0x1p-80f;

// A block's row groups take every gridDim-th set of rows, SLOTS - 1 of a
// group's rows under way while it computes one (SLOTS = 1: a call with few
// rows, one for a group, which takes the parameters as it needs them).
// One reduction a row: with w = alpha gate gamma_post y (A y in the code)
//   sum x'^2 = sum x^2 + 2 r1 sum x w + r1^2 sum w^2,
// four sums that do not wait for r1.  Where x' is small beside x and r1 w the
// terms cancel: below a quarter of sum x^2 + r1^2 sum w^2, where an error of the
// sums could grow more than fourfold, sum x'^2 is taken from x' itself; so it is
// where a sum leaves fp32's range (|x|, |y| or |w| of 2^57 and more).  There y enters
// r1, and x' enters r2, in units of 2^80 if their own squares overflow: a row at its
// type's lowest value has a norm like any other.  (4096 x 2048 12.6 -> 12.9 us; as a
// function outside the loop, whose call spills, 17.3.)
// ALL: y, gamma_post and gamma_pre are there and the rows share one gate.
template <class T, int VPT, int SLOTS, bool ALL>
__global__ void __launch_bounds__(SLOTS == 1 || VPT == 4 ? 512 : 1024, 1) block_norm_kernel(const Args p) {
    extern __shared__ __align__(16) float smem[];
    grid_dependency_launch();
    grid_dependency_wait();
    constexpr size_t CH = 8 * T::BYTES;
    const int groups = blockDim.x / p.threads, grp = threadIdx.x / p.threads;
    RowGroup rg(p.threads, grp, smem + grp * RowGroup::SUM_FLOATS);
    ThreadRing<T, 2 * VPT, SLOTS> ring(smem + groups * RowGroup::SUM_FLOATS);
    const ParamTable table(smem + groups * RowGroup::SUM_FLOATS +
                           (SLOTS > 1 ? ring.BYTES_PER_THREAD / 4 * (int)blockDim.x : 0), VPT * p.threads);
    const int chunks = p.D / 8, step = gridDim.x * groups;
    const float inv_d = 1.f / (float)p.D;
    const bool has_y = ALL || p.y, has_post = ALL || p.gamma_post, has_h = ALL || p.h;
    const bool row_gate = !ALL && p.gate && (SLOTS == 1 || p.S != p.T);
    const size_t row_bytes = (size_t)chunks * CH, step_bytes = row_bytes * step, col = CH * rg.tid, next = CH * p.threads;
    bool in[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) in[i] = i * p.threads + rg.tid < chunks;

    int r = blockIdx.x * groups + grp;
    size_t off = row_bytes * r + col;  // of this thread's first chunk in row r
    int fr = r;                        // the next row to fetch
    size_t foff = off;
    auto fetch = [&]() {
        if (fr < p.T) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) {
                    ring.fetch(i, at(p.x, foff + i * next));
                    if (has_y) ring.fetch(VPT + i, at(p.y, foff + i * next));
                }
        }
        fr += step;
        foff += step_bytes;
        ring.commit();
    };
    if (SLOTS > 1) {
#pragma unroll
        for (int k = 0; k < SLOTS - 1; ++k) fetch();
        table.fill(p);
    }
    if (rg.tid < 128) rg.red[rg.tid] = rg.red[128 + rg.tid] = 0.f;
    if (p.threads < 128)
        for (int i = rg.tid + p.threads; i < 128; i += p.threads) rg.red[i] = rg.red[128 + i] = 0.f;
    __syncthreads();
    for (; r < p.T; r += step, off += step_bytes) {
        if (SLOTS > 1) {
            fetch();
            ring.wait();
        }
        const size_t gchunk = row_gate ? (size_t)(r / p.S) * chunks + rg.tid : 0;
        auto load_x = [&](int i) { return unpack8<T>(SLOTS > 1 ? ring.get(i) : raw_at<T>(p.x, off + i * next)); };
        auto load_y = [&](int i) { return unpack8<T>(SLOTS > 1 ? ring.get(VPT + i) : raw_at<T>(p.y, off + i * next)); };
        auto weighted = [&](int i, const V8& y) {
            const int c = i * p.threads + rg.tid;
            V8 a;
            if (SLOTS > 1) a = table.get(0, c);
            else a = has_post ? mul(load8(p.ptype, p.gamma_post, c), p.alpha) : v8(p.alpha);
            if (row_gate) a = mul(a, load8(p.ptype, p.gate, gchunk + i * p.threads));
            if (SLOTS == 1 && ALL && p.gate) a = mul(a, load8(p.ptype, p.gate, c));
            return mul(a, y);
        };
        V8 x[VPT], w[VPT];
        float2 s[4];  // y^2, x^2, x w, w^2
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            x[i] = w[i] = v8(0.f);
            if (in[i]) {
                x[i] = load_x(i);
                if (has_y) {
                    const V8 y = load_y(i);
                    w[i] = weighted(i, y);
                    dot(s[0], y, y);
                    dot(s[2], x[i], w[i]);
                    dot(s[3], w[i], w[i]);
                }
                dot(s[1], x[i], x[i]);
            }
        }
        float r1 = 1.f, r2 = 0.f;
        if (has_post || has_h) {
            float t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = s[k].x + s[k].y;
            rg.sum4(t);
            if (has_post) r1 = rsqrtf(t[0] * inv_d + p.eps);
            const float plain = t[1] + r1 * r1 * t[3];
            float sum = plain + 2.f * r1 * t[2];
#pragma unroll
            for (int i = 0; i < VPT; ++i) x[i] = fma(w[i], r1, x[i]);
            r2 = rsqrtf(sum * inv_d + p.eps);
            // the same for the group's threads, and true for a NaN
            if (__builtin_expect(!(t[0] + plain < INFINITY && sum >= 0.25f * plain), 0)) {
                auto squares = [&](auto value, float u) {
                    float2 q = f2(0.f);
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (in[i]) {
                            const V8 v = mul(value(i), u);
                            dot(q, v, v);
                        }
                    return rg.sum(q.x + q.y);
                };
                if (has_post && !(t[0] < INFINITY)) {
                    r1 = rsqrtf(squares(load_y, UNIT) * inv_d + p.eps * UNIT * UNIT);
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (in[i]) x[i] = fma(weighted(i, mul(load_y(i), UNIT)), r1, load_x(i));
                }
                if (has_h) {
                    auto stream = [&](int i) { return x[i]; };
                    sum = squares(stream, 1.f);
                    r2 = rsqrtf(sum * inv_d + p.eps);
                    if (!(sum < INFINITY)) r2 = rsqrtf(squares(stream, UNIT) * inv_d + p.eps * UNIT * UNIT) * UNIT;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) x[i] = fma(w[i], r1, x[i]);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in[i]) {
                const int c = i * p.threads + rg.tid;
                if (has_y) store_at<T>(p.x_out, off + i * next, x[i]);
                if (has_h)
                    store_at<T>(p.h, off + i * next,
                                mul(mul(x[i], r2), SLOTS > 1 ? table.get(1, c) : load8(p.ptype, p.gamma_pre, c)));
            }
        ring.next();
    }
    cp_async_wait<0>();
}

template <class T>
cudaError_t run(Args p, cudaStream_t s) {
    const int vpt = chunks_per_thread(p.D);
    p.threads = group_threads(p.D, vpt);
    const size_t sums = RowGroup::SUM_FLOATS * sizeof(float), table = ParamTable::bytes(vpt * p.threads);
    // one block an SM, with as many row groups as 1024 threads hold and the rows fill
    int groups = std::max(1, std::min({(vpt == 4 ? 512 : 1024) / p.threads, 15, p.T / num_sms()}));
    const size_t slot = (size_t)2 * vpt * 8 * T::BYTES * p.threads;  // of one group
    int slots = 1;
    if (p.T > num_sms() && vpt < 4)
        for (; slots == 1 && groups > 0; --groups)
            if ((slots = ring_slots(slot * groups, sums * groups + table)) > 1) break;
    if (slots == 1) groups = 1;
    const int threads = groups * p.threads;
    const int blocks = slots > 1 ? std::min(ceil_div(p.T, groups), num_sms()) : p.T;
    const size_t smem = groups * sums + (slots > 1 ? slots * slot * groups + table : 0);
    const bool all = p.y && p.gamma_post && p.h && (!p.gate || p.S == p.T);
    return with_shape(vpt, slots, [&](auto v, auto n) {
        constexpr int V = decltype(v)::value, N = decltype(n)::value;
        return all ? launch_overlapped<block_norm_kernel<T, V, N, true>>(blocks, threads, smem, s, p)
                   : launch_overlapped<block_norm_kernel<T, V, N, false>>(blocks, threads, smem, s, p);
    });
}

}  // namespace
}  // namespace norm

cudaError_t launch_block_norm(const NormShape& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s) {
    norm::Args a = norm::common_args(n);
    a.x = x;
    a.y = y;
    a.x_out = x_out;
    a.h = h;
    return n.dtype == MOE_DT_BF16  ? norm::run<Bf16>(a, s)
           : n.dtype == MOE_DT_F16 ? norm::run<F16>(a, s)
                                   : norm::run<F32>(a, s);
}

}  // namespace moe
