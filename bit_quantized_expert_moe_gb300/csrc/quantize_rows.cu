// Rows to 8-bit codes with a scale for each row, gathered on the way:
//   a = max |x[i]|,  scale = a / 127,  code = 127 x / a rounded to nearest even
// for x = row (row_map[r] / k), so that the rows of a permutation go to their places
// without a 16-bit copy in between.
//
// Bound by memory: a thread holds its part of the row in registers, 16 elements at a
// time, between the maximum and the codes.  The codes are those of the formula
// exactly: where fp32 leaves a value too close to the border between two codes, the
// border is compared in 64 bits.
#include "internal.h"
#include "vec8.cuh"

namespace moe {
namespace {

struct QuantArgs {
    const void* x;
    const int32_t* row_map;  // or null: row r of x
    int k, T, R, D;
    int8_t* codes;
    float* scales;
};

// The code of v; t: v 127 / top in fp32, off by less than 3e-5.
__device__ __forceinline__ int code_of(float v, float t, float top) {
    const float q = rintf(t);
    if (__builtin_expect(fabsf(fabsf(t - q) - 0.5f) < 4e-5f, 0)) {
        // between m and m + 1: 254 |v| against (2 m + 1) top, exact in 64 bits
        const int m = (int)fabsf(t);
        const double a = 254.0 * fabs((double)v), b = (2.0 * m + 1.0) * (double)top;
        const int c = a > b || (a == b && (m & 1)) ? m + 1 : m;
        return t < 0.f ? -c : c;
    }
    return (int)q;
}

// THREADS threads share a row, VPT times 16 elements each; 256 / THREADS rows a block.
template <class T, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS > 256 ? THREADS : 256) quantize_rows_kernel(const QuantArgs p) {
    constexpr int ROWS = THREADS >= 256 ? 1 : 256 / THREADS;
    __shared__ uint32_t most[ROWS][THREADS / 32];
    grid_dependency_launch();
    grid_dependency_wait();
    const int grp = threadIdx.x / THREADS, tid = threadIdx.x % THREADS;
    const int r = blockIdx.x * ROWS + grp, units = p.D / 16;
    int src = r;
    if (r < p.R && p.row_map) {
        const int a = __ldg(p.row_map + r);
        src = a < 0 ? -1 : a / p.k;
    }
    const bool there = r < p.R && src >= 0 && src < p.T;
    V8 v[VPT][2];
    uint32_t top = 0;  // |x| as bits: ordered, and a NaN is above infinity
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int u = i * THREADS + tid;
        v[i][0] = v[i][1] = v8(0.f);
        if (there && u < units) {
            const size_t c = (size_t)src * units * 2 + 2 * u;
            v[i][0] = load8<T>(p.x, c);
            v[i][1] = load8<T>(p.x, c + 1);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = max(top, max(__float_as_uint(v[i][h].p[j].x) & 0x7FFFFFFFu, __float_as_uint(v[i][h].p[j].y) & 0x7FFFFFFFu));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (THREADS > 32) {
        if ((tid & 31) == 0) most[grp][tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) top = max(top, most[grp][w]);
    }
    if (r >= p.R) return;
    const bool finite = top < 0x7F800000u, any = finite && top > 0;
    const float a = __uint_as_float(top);
    // units in which 127 / a is an ordinary number
    const float unit = a < 0x1p-60f ? 0x1p80f : 1.f, inv = any ? 127.f / (a * unit) : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int u = i * THREADS + tid;
        if (u >= units) continue;
        uint32_t o[4] = {0, 0, 0, 0};
        if (any)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = v[i][h].p[j];
                    const int lo = code_of(f.x, f.x * unit * inv, a), hi = code_of(f.y, f.y * unit * inv, a);
                    o[2 * h + (j >> 1)] |= ((uint32_t)(lo & 255) | (uint32_t)(hi & 255) << 8) << (16 * (j & 1));
                }
        reinterpret_cast<uint4*>(p.codes)[(size_t)r * units + u] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    // a row with an infinity or a NaN has no codes: its scale, and all that is made with it, is NaN
    if (tid == 0) p.scales[r] = finite ? a / 127.f : __uint_as_float(0x7FC00000u);
}

template <class T, int VPT, int THREADS>
cudaError_t run(const QuantArgs& p, cudaStream_t s) {
    constexpr int rows = THREADS >= 256 ? 1 : 256 / THREADS;
    return launch_overlapped(quantize_rows_kernel<T, VPT, THREADS>, ceil_div(p.R, rows), rows * THREADS, 0, s, p);
}
template <class T>
cudaError_t run(const QuantArgs& p, cudaStream_t s) {
    // threads of a row: 16 elements each, 32 and 64 where 1024 threads do not reach
    const int units = p.D / 16;
    if (units <= 32) return run<T, 1, 32>(p, s);
    if (units <= 64) return run<T, 1, 64>(p, s);
    if (units <= 128) return run<T, 1, 128>(p, s);
    if (units <= 256) return run<T, 1, 256>(p, s);
    if (units <= 512) return run<T, 2, 256>(p, s);
    if (units <= 1024) return run<T, 2, 512>(p, s);
    return run<T, 4, 512>(p, s);
}

}  // namespace

cudaError_t launch_quantize_rows(moe_dtype_t dt, const void* x, const int32_t* row_map, int k, int T, int R, int D,
                                 int8_t* codes, float* scales, cudaStream_t s) {
    const QuantArgs p{x, row_map, k, T, R, D, codes, scales};
    return dt == MOE_DT_BF16 ? run<Bf16>(p, s) : dt == MOE_DT_F16 ? run<F16>(p, s) : run<F32>(p, s);
}

}  // namespace moe
