// What the two passes of the layer norm share.
#pragma once

#include "block_norm.cuh"

namespace moe {
namespace lnorm {

using norm::at;
using norm::raw_at;
using norm::store_at;

struct Args {
    int T, D;
    float eps;
    moe_dtype_t ptype;        // of gamma, beta and their gradients
    const void *gamma, *beta;
    const void *x, *y;        // backward: x is the stream that was normalised
    void *x_out, *h;          // forward
    const void *dh, *dx_out;  // backward
    void *dx, *dgamma, *dbeta;
    int threads;              // of a row group
    int groups, rows;         // backward: row groups of a block, consecutive rows of a row group
    float* part;              // backward: [blocks][2][D]: gamma, beta
    int blocks;
};

// Rows whose sums leave fp32's range are taken again in units of 2^80.
constexpr float UNIT = 0x1p-80f;

// From mean c^2 and d = mean c.  d is a rounding of the mean; where all of c is that
// and no more (a row of one value) the difference is a rounding's as well, of either
// sign: a floor below which fp32 rows have no variance (a deviation of 2^-35 |mean|)
// keeps (c - d) r small there.
__device__ __forceinline__ float variance(float c2, float d) { return fmaxf(c2 - d * d, 0x1p-22f * d * d); }

// The sum of a chunk added to s.
__device__ __forceinline__ void add(float2& s, const V8& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) s = ffma2(x.p[k], f2(1.f), s);
}

// gamma and beta of a thread's columns in fp32, side by side for neighbouring threads.
__device__ __forceinline__ V8 gamma_of(const Args& p, int c) { return p.gamma ? load8(p.ptype, p.gamma, c) : v8(1.f); }
__device__ __forceinline__ V8 beta_of(const Args& p, int c) { return p.beta ? load8(p.ptype, p.beta, c) : v8(0.f); }
__device__ __forceinline__ void fill(const norm::ParamTable& t, const Args& p, bool with_beta) {
    for (int c = threadIdx.x; c < p.D / 8; c += blockDim.x) {
        const V8 g = gamma_of(p, c), b = with_beta ? beta_of(p, c) : v8(0.f);
        t.put(0, c, g);
        if (with_beta) t.put(1, c, b);
    }
}

}  // namespace lnorm
}  // namespace moe
