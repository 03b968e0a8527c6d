// Products of 16-bit expert weights with ragged row segments.
//
// Segment e is rows offsets[e] .. offsets[e+1]-1.
//   y[r][n]     = sum_k x[r][k] W[e][n][k]
//   dx[r][k]    = sum_n dy[r][n] W[e][n][k]
//   dW[e][n][k] = sum_{r in e} dy[r][n] x[r][k]
// One block computes 64 x 64 outputs of one segment, 16 of the summed index
// at a time from shared memory, in fp32.
#include "internal.h"
#include "vec8.cuh"

namespace moe {
namespace {

enum class Product { Y, DX, DW };

template <class T, Product PR>
__global__ void __launch_bounds__(256) grouped_kernel(const void* __restrict__ a, const void* __restrict__ b,
                                                      void* __restrict__ out, GroupedShape g) {
    __shared__ float sa[16][65], sb[16][65];
    const int e = blockIdx.z;
    const int i = g.offsets[e], j = g.offsets[e + 1];
    const bool bad = i < 0 || j < i || j > g.R;
    if (bad && threadIdx.x == 0) set_error(g.err, ERRBIT_RANGE);
    const int r0 = bad ? 0 : i, cnt = bad ? 0 : j - i;
    const int M = PR == Product::DW ? g.N : cnt;                               // output rows
    const int C = PR == Product::Y ? g.N : g.K;                                // output columns
    const int L = PR == Product::Y ? g.K : PR == Product::DX ? g.N : cnt;      // summed index
    const size_t we = (size_t)e * g.N * g.K;
    const int c0 = blockIdx.x * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int m0 = blockIdx.y * 64; m0 < M; m0 += gridDim.y * 64) {
        float acc[4][4] = {};
        for (int l0 = 0; l0 < L; l0 += 16) {
            for (int t = threadIdx.x; t < 64 * 16; t += 256) {
                const int l = PR == Product::DW ? t / 64 : t % 16, m = PR == Product::DW ? t % 64 : t / 16;
                float v = 0.f;
                if (m0 + m < M && l0 + l < L)
                    v = PR == Product::DW ? load1<T>(a, (size_t)(r0 + l0 + l) * g.N + m0 + m)
                                          : load1<T>(a, (size_t)(r0 + m0 + m) * L + l0 + l);
                sa[l][m] = v;
            }
            for (int t = threadIdx.x; t < 64 * 16; t += 256) {
                const int l = PR == Product::Y ? t % 16 : t / 64, c = PR == Product::Y ? t / 16 : t % 64;
                float v = 0.f;
                if (c0 + c < C && l0 + l < L)
                    v = PR == Product::Y    ? load1<T>(b, we + (size_t)(c0 + c) * g.K + l0 + l)
                        : PR == Product::DX ? load1<T>(b, we + (size_t)(l0 + l) * g.K + c0 + c)
                                            : load1<T>(b, (size_t)(r0 + l0 + l) * g.K + c0 + c);
                sb[l][c] = v;
            }
            __syncthreads();
#pragma unroll
            for (int l = 0; l < 16; ++l)
#pragma unroll
                for (int p = 0; p < 4; ++p)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(sa[l][ty + 16 * p], sb[l][tx + 16 * q], acc[p][q]);
            __syncthreads();
        }
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int m = m0 + ty + 16 * p, c = c0 + tx + 16 * q;
                if (m < M && c < C)
                    store1<T>(out, PR == Product::DW ? we + (size_t)m * g.K + c : (size_t)(r0 + m) * C + c, acc[p][q]);
            }
    }
}

template <Product PR>
cudaError_t launch(const GroupedShape& g, const void* a, const void* b, void* out, cudaStream_t s) {
    const int M = PR == Product::DW ? g.N : g.R, C = PR == Product::Y ? g.N : g.K;
    const dim3 grid(ceil_div(C, 64), std::min(ceil_div(M, 64), PR == Product::DW ? 65535 : 16), g.E);
    if (g.dtype == MOE_DT_BF16) grouped_kernel<Bf16, PR><<<grid, 256, 0, s>>>(a, b, out, g);
    else grouped_kernel<F16, PR><<<grid, 256, 0, s>>>(a, b, out, g);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_mm(const GroupedShape& g, const void* x, const void* w, void* y, cudaStream_t s) {
    return launch<Product::Y>(g, x, w, y, s);
}
cudaError_t launch_grouped_mm_dx(const GroupedShape& g, const void* dy, const void* w, void* dx, cudaStream_t s) {
    return launch<Product::DX>(g, dy, w, dx, s);
}
cudaError_t launch_grouped_mm_dw(const GroupedShape& g, const void* dy, const void* x, void* dw, cudaStream_t s) {
    return launch<Product::DW>(g, dy, x, dw, s);
}

}  // namespace moe
