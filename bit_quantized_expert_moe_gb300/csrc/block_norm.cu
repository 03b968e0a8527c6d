// Norms before and after a block, fused with its gate and residual scale.
//
//   n  = y r1 gamma_post   (r1 = (mean y^2 + eps)^-1/2; without gamma_post n = y)
//   x' = x + alpha gate n  (gate per channel, one row for each T / G tokens)
//   h  = x' r2 gamma_pre   (r2 = (mean x'^2 + eps)^-1/2)
// and, given dx' and dh, with the statistics taken again from y and x':
//   D  = dx' + r2 v - x' r2^3 mean(v x'),   v = dh gamma_pre;   dx = D
//   q  = alpha gate gamma_post D;  dy = r1 q - y r1^3 mean(q y)
//   dgamma_pre = sum dh x' r2,  dgate = sum alpha D n,  dgamma_post = sum alpha gate D y r1
// h is taken from x' before its rounding, so both outputs are rounded once;
// the backward pass sees the stored x', the value that every later reader sees.
// Every tensor is read and written once: bound by memory.  NT threads share a
// row and hold it in registers, VPT chunks of 8 elements a thread.
#include "internal.h"
#include "vec8.cuh"

namespace moe {
namespace {

struct NormArgs {
    int T, D, S;  // S = T / G rows share a gate row
    float alpha, eps;
    const void *gamma_post, *gate, *gamma_pre;
    const void *x, *y;           // backward: x is the stream after the block
    void *x_out, *h;             // forward
    const void *dx_out, *dh;     // backward
    void *dx, *dy;
    void *dgamma_post, *dgate, *dgamma_pre;
    float* part;                 // backward: [blocks][4][D] (gamma_post, gamma_pre, first gate row, last gate row)
    int rows_per_block;
    int blocks;
};

template <class T, class P, int NT, int VPT>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) block_norm_kernel(const NormArgs p) {
    __shared__ float red[2 * (NT / 32)];
    const int rpb = blockDim.x / NT, tid = threadIdx.x % NT;
    const int r = blockIdx.x * rpb + threadIdx.x / NT;
    if (r >= p.T) return;  // whole warps, and whole blocks when NT > 32
    const int chunks = p.D / 8;
    const size_t row = (size_t)r * chunks;
    const float inv_d = 1.f / (float)p.D;
    int buf = 0;
    float x[VPT][8], y[VPT][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = i * NT + tid;
        if (c < chunks) {
            load8<T>(p.x, row + c, x[i]);
            if (p.y) {
                load8<T>(p.y, row + c, y[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] += y[i][j] * y[i][j];
            }
        }
    }
    if (p.y) {
        float r1 = 1.f;
        if (p.gamma_post) {
            row_sum<NT, 1>(sum, red, buf);
            r1 = rsqrtf(sum[0] * inv_d + p.eps);
        }
        const size_t grow = p.gate ? (size_t)(r / p.S) * chunks : 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * NT + tid;
            if (c < chunks) {
                float g[8];
                if (p.gamma_post) {
                    load8<P>(p.gamma_post, c, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * r1 * g[j];
                }
                if (p.gate) {
                    load8<P>(p.gate, grow + c, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[i][j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] += p.alpha * y[i][j];
                store8<T>(p.x_out, row + c, x[i]);
            }
        }
    }
    if (p.h) {
        sum[0] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i * NT + tid < chunks)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] += x[i][j] * x[i][j];
        row_sum<NT, 1>(sum, red, buf);
        const float r2 = rsqrtf(sum[0] * inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * NT + tid;
            if (c < chunks) {
                float g[8];
                load8<P>(p.gamma_pre, c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = x[i][j] * r2 * g[j];
                store8<T>(p.h, row + c, g);
            }
        }
    }
}

// A block takes rows_per_block consecutive rows and adds up its rows'
// parameter gradients in registers.  A gate row that lies wholly inside the
// block's rows is written at once; the block's first and last one may be
// shared with its neighbours and go to its partial sums.
template <class T, class P, int NT, int VPT>
__global__ void __launch_bounds__(NT) block_norm_backward_kernel(const NormArgs p) {
    __shared__ float red[2 * 3 * (NT / 32)];
    const int tid = threadIdx.x;
    const int chunks = p.D / 8;
    const float inv_d = 1.f / (float)p.D;
    const int r_begin = blockIdx.x * p.rows_per_block;
    const int r_end = min(p.T, r_begin + p.rows_per_block);
    int buf = 0;
    float a_post[VPT][8], a_pre[VPT][8], a_gate[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) a_post[i][j] = a_pre[i][j] = a_gate[i][j] = 0.f;
    float* const part = p.part + (size_t)blockIdx.x * 4 * p.D;
    const int g_first = r_begin / p.S, g_last = (r_end - 1) / p.S;

    for (int r = r_begin; r < r_end; ++r) {
        const size_t row = (size_t)r * chunks;
        const int g = r / p.S;
        float x[VPT][8], dh[VPT][8], y[VPT][8], dx[VPT][8];
        float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * NT + tid;
            if (c < chunks) {
                if (p.dx_out) {
                    load8<T>(p.dx_out, row + c, dx[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dx[i][j] = 0.f;
                }
                if (p.dh) {
                    float gp[8];
                    load8<T>(p.x, row + c, x[i]);
                    load8<T>(p.dh, row + c, dh[i]);
                    load8<P>(p.gamma_pre, c, gp);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sum[0] += x[i][j] * x[i][j];
                        sum[1] += dh[i][j] * gp[j] * x[i][j];
                    }
                }
                if (p.y) {
                    load8<T>(p.y, row + c, y[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[2] += y[i][j] * y[i][j];
                }
            }
        }
        row_sum<NT, 3>(sum, red, buf);
        if (p.dh) {
            const float r2 = rsqrtf(sum[0] * inv_d + p.eps);
            const float c2 = r2 * r2 * r2 * sum[1] * inv_d;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * NT + tid;
                if (c < chunks) {
                    float gp[8];
                    load8<P>(p.gamma_pre, c, gp);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        a_pre[i][j] += dh[i][j] * (x[i][j] * r2);
                        dx[i][j] += r2 * (dh[i][j] * gp[j]) - x[i][j] * c2;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i * NT + tid;
            if (c < chunks) store8<T>(p.dx, row + c, dx[i]);
        }
        if (p.y) {
            const float r1 = p.gamma_post ? rsqrtf(sum[2] * inv_d + p.eps) : 1.f;
            float s2[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * NT + tid;
                if (c < chunks) {
                    float ga[8], po[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) ga[j] = po[j] = 1.f;
                    if (p.gate) load8<P>(p.gate, (size_t)g * chunks + c, ga);
                    if (p.gamma_post) load8<P>(p.gamma_post, c, po);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float ad = p.alpha * dx[i][j];
                        const float yn = y[i][j] * r1;
                        a_gate[i][j] += ad * (yn * po[j]);
                        const float dn = ad * ga[j];
                        a_post[i][j] += dn * yn;
                        dx[i][j] = dn * po[j];
                        s2[0] += dx[i][j] * y[i][j];
                    }
                }
            }
            float c1 = 0.f;
            if (p.gamma_post) {
                row_sum<NT, 3>(s2, red, buf);
                c1 = r1 * r1 * r1 * s2[0] * inv_d;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * NT + tid;
                if (c < chunks) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dx[i][j] = r1 * dx[i][j] - y[i][j] * c1;
                    store8<T>(p.dy, row + c, dx[i]);
                }
            }
            // the gate row ends here
            if (p.dgate && (r + 1 == r_end || (r + 1) % p.S == 0)) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int c = i * NT + tid;
                    if (c < chunks) {
                        if (g == g_first) store8<F32>(part + 2 * p.D, c, a_gate[i]);
                        else if (g == g_last) store8<F32>(part + 3 * p.D, c, a_gate[i]);
                        else store8<P>(p.dgate, (size_t)g * chunks + c, a_gate[i]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) a_gate[i][j] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = i * NT + tid;
        if (c < chunks) {
            if (p.dgamma_post) store8<F32>(part, c, a_post[i]);
            if (p.dgamma_pre) store8<F32>(part + p.D, c, a_pre[i]);
        }
    }
}

// Sums the blocks' partial sums in block order.  `what`: 0 gamma_post, 1
// gamma_pre, 2 + g gate row g.  32 columns a block, 8 threads a column.
template <class P>
__device__ __forceinline__ void reduce_one(const NormArgs& p, int what, float (&red)[8][33]) {
    const int col = blockIdx.x * 32 + threadIdx.x;
    int b0 = 0, b1 = p.blocks - 1;
    void* out = what == 0 ? p.dgamma_post : p.dgamma_pre;
    size_t at = col;
    if (what >= 2) {
        const int g = what - 2;
        b0 = (int)((long long)g * p.S / p.rows_per_block);
        b1 = (int)(((long long)(g + 1) * p.S - 1) / p.rows_per_block);
        const int r_end = min(p.T, (b0 + 1) * p.rows_per_block);
        // wholly inside one block, and neither its first nor its last gate row
        if (b0 == b1 && b0 * p.rows_per_block / p.S != g && (r_end - 1) / p.S != g) return;
        out = p.dgate;
        at += (size_t)g * p.D;
    }
    if (!out) return;
    float s = 0.f;
    if (col < p.D)
        for (int b = b0 + threadIdx.y; b <= b1; b += 8) {
            const int slot = what < 2 ? what : (b * p.rows_per_block / p.S == what - 2 ? 2 : 3);
            s += p.part[((size_t)b * 4 + slot) * p.D + col];
        }
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < p.D) {
        for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
        store1<P>(out, at, s);
    }
    __syncthreads();
}

template <class P>
__global__ void __launch_bounds__(256) block_norm_reduce_kernel(const NormArgs p, int gates) {
    __shared__ float red[8][33];
    for (int what = blockIdx.y; what < 2 + gates; what += gridDim.y) reduce_one<P>(p, what, red);
}

int norm_blocks(int T) { return std::min(T, num_sms() * 2); }

template <class T, class P>
void run_forward(const NormArgs& p, cudaStream_t s) {
    const int D = p.D;
    if (D <= 1024) block_norm_kernel<T, P, 32, 4><<<ceil_div(p.T, 4), 128, 0, s>>>(p);
    else if (D <= 2048) block_norm_kernel<T, P, 256, 1><<<p.T, 256, 0, s>>>(p);
    else if (D <= 4096) block_norm_kernel<T, P, 512, 1><<<p.T, 512, 0, s>>>(p);
    else if (D <= 8192) block_norm_kernel<T, P, 512, 2><<<p.T, 512, 0, s>>>(p);
    else block_norm_kernel<T, P, 512, 4><<<p.T, 512, 0, s>>>(p);
}

template <class T, class P>
void run_backward(const NormArgs& p, cudaStream_t s) {
    const int D = p.D;
    if (D <= 1024) block_norm_backward_kernel<T, P, 128, 1><<<p.blocks, 128, 0, s>>>(p);
    else if (D <= 2048) block_norm_backward_kernel<T, P, 256, 1><<<p.blocks, 256, 0, s>>>(p);
    else if (D <= 4096) block_norm_backward_kernel<T, P, 512, 1><<<p.blocks, 512, 0, s>>>(p);
    else if (D <= 8192) block_norm_backward_kernel<T, P, 512, 2><<<p.blocks, 512, 0, s>>>(p);
    else block_norm_backward_kernel<T, P, 512, 4><<<p.blocks, 512, 0, s>>>(p);
}

template <class P>
void run_reduce(const NormArgs& p, int gates, cudaStream_t s) {
    block_norm_reduce_kernel<P><<<dim3(ceil_div(p.D, 32), std::min(2 + gates, 1024)), dim3(32, 8), 0, s>>>(p, gates);
}

NormArgs common_args(const NormShape& n) {
    NormArgs a{};
    a.T = n.T;
    a.D = n.D;
    a.S = n.T / n.G;
    a.alpha = n.alpha;
    a.eps = n.eps;
    a.gamma_post = n.gamma_post;
    a.gate = n.gate;
    a.gamma_pre = n.gamma_pre;
    return a;
}

// Calls f with the activation and the parameter type as tags.
template <class F>
void with_types(moe_dtype_t dt, moe_dtype_t pt, F f) {
    if (dt == MOE_DT_F32) f(F32{}, F32{});
    else if (dt == MOE_DT_BF16 && pt == MOE_DT_BF16) f(Bf16{}, Bf16{});
    else if (dt == MOE_DT_BF16) f(Bf16{}, F32{});
    else if (pt == MOE_DT_F16) f(F16{}, F16{});
    else f(F16{}, F32{});
}

}  // namespace

size_t block_norm_partial_floats(int T, int D) { return (size_t)norm_blocks(T) * 4 * D; }

cudaError_t launch_block_norm(const NormShape& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s) {
    NormArgs a = common_args(n);
    a.x = x;
    a.y = y;
    a.x_out = x_out;
    a.h = h;
    with_types(n.dtype, n.param_dtype, [&](auto t, auto p) { run_forward<decltype(t), decltype(p)>(a, s); });
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_block_norm_backward(const NormShape& n, const NormGrads& g, float* part, cudaStream_t s) {
    NormArgs a = common_args(n);
    a.x = g.x_out;
    a.y = g.y;
    a.dx_out = g.dx_out;
    a.dh = g.dh;
    a.dx = g.dx;
    a.dy = g.dy;
    a.dgamma_post = g.dgamma_post;
    a.dgate = g.dgate;
    a.dgamma_pre = g.dgamma_pre;
    a.part = part;
    a.rows_per_block = ceil_div(n.T, norm_blocks(n.T));
    a.blocks = ceil_div(n.T, a.rows_per_block);
    with_types(n.dtype, n.param_dtype, [&](auto t, auto p) { run_backward<decltype(t), decltype(p)>(a, s); });
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    note_launch();
    if (!g.dgamma_post && !g.dgate && !g.dgamma_pre) return e;
    const int gates = g.dgate ? n.G : 0;
    with_types(n.dtype, n.param_dtype, [&](auto, auto p) { run_reduce<decltype(p)>(a, gates, s); });
    note_launch();
    return cudaGetLastError();
}

}  // namespace moe
