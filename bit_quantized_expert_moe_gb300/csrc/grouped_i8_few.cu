// y = (x W_e^T) by the rows' and the output channels' scales, of 8-bit codes, for a
// handful of rows in all or for about one an expert: decoding.
//
// As for 16-bit weights (grouped_few.cu) the weights' bytes are all that counts: a
// block takes 16 weight rows of one expert and up to 8 of its rows, its warps share K
// and add up in shared memory.  mma.sync m16n8k32 on the codes as they are, 32-bit
// integer sums, so the sum is exact in any order; one rounding at the end.  (int8
// runs at 1/11 of the 16-bit rate here, which 8 rows do not reach.)  Both operands
// keep K in the order in which a thread's 16-byte loads bring it: lane 4 g + t holds
// elements 16 t .. 16 t + 15 of every 64 for weight rows g and g + 8 and row g of x.
#include "internal.h"

namespace moe {
namespace {

constexpr int ROWS = 16, COLS = 8, AHEAD = 4;

__device__ __forceinline__ uint4 load_codes(const int8_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ void mma16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) grouped_i8_few_kernel(const GroupedI8Shape g, const GroupedI8Data d) {
    __shared__ int cnt[WARPS];
    __shared__ int part[WARPS][COLS][ROWS + 1];
    grid_dependency_launch();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y, n0 = blockIdx.x * ROWS;
    // the row's expert: how many segments end at or before it
    int c = 0;
    bool bad = false;
    for (int i = threadIdx.x; i < g.E; i += 32 * WARPS) {
        const int lo = __ldg(g.offsets + i), hi = __ldg(g.offsets + i + 1);
        c += hi <= r;
        bad |= lo < 0 || hi < lo || hi > g.R;
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) cnt[warp] = c;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && r == 0) set_error(g.err, ERRBIT_RANGE);
        return;
    }
    int e = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) e += cnt[i];
    if (e >= g.E) return;  // behind the last segment
    const int r0 = __ldg(g.offsets + e), r1 = __ldg(g.offsets + e + 1);
    if (r < r0 || (r - r0) % COLS) return;  // in front of the first; another block's
    const int rows = min(COLS, r1 - r);

    const int gi = lane >> 2, t = lane & 3;
    const int kq = ceil_div(g.K, 64 * WARPS) * 64, k0 = warp * kq, k1 = min(g.K, k0 + kq);
    const size_t ld = (size_t)g.K;
    const int8_t* wa = d.w + ((size_t)e * g.N + min(n0 + gi, g.N - 1)) * ld + 16 * t;
    const int8_t* wb = d.w + ((size_t)e * g.N + min(n0 + gi + 8, g.N - 1)) * ld + 16 * t;
    const int8_t* xr = d.x + (size_t)(r + min(gi, rows - 1)) * ld + 16 * t;
    const bool has = gi < rows;
    int acc[4] = {0, 0, 0, 0};
    for (int k = k0; k < k1; k += 64 * AHEAD) {
        uint4 a[AHEAD], b[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = k + 64 * i + 16 * t < k1;
            a[i] = in ? load_codes(wa + k + 64 * i) : make_uint4(0, 0, 0, 0);
            b[i] = in ? load_codes(wb + k + 64 * i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = has && k + 64 * i + 16 * t < k1;
            const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(xr + k + 64 * i)) : make_uint4(0, 0, 0, 0);
            mma16832(acc, a[i].x, b[i].x, a[i].y, b[i].y, v.x, v.y);
            mma16832(acc, a[i].z, b[i].z, a[i].w, b[i].w, v.z, v.w);
        }
    }
    part[warp][2 * t][gi] = acc[0];
    part[warp][2 * t + 1][gi] = acc[1];
    part[warp][2 * t][gi + 8] = acc[2];
    part[warp][2 * t + 1][gi + 8] = acc[3];
    __syncthreads();
    const int col = threadIdx.x / ROWS, n = threadIdx.x % ROWS;
    if (col < rows && n0 + n < g.N) {  // (the first 128 threads)
        int s = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += part[i][col][n];
        const float v = (float)s * __ldg(d.w_scale + (size_t)e * g.N + n0 + n) * __ldg(d.x_scale + r + col);
        static_cast<uint16_t*>(d.y)[(size_t)(r + col) * g.N + n0 + n] =
            g.out == MOE_DT_BF16 ? float_to_bf16_bits(v) : float_to_f16_bits(v);
    }
}

}  // namespace

// Warps that share K: four, more where the blocks leave SMs without loads under way.
cudaError_t launch_grouped_i8_few(const GroupedI8Shape& g, const GroupedI8Data& d, cudaStream_t s) {
    const dim3 grid(ceil_div(g.N, ROWS), g.R);
    // blocks with work, at most
    const long long blocks = (long long)grid.x * std::min(g.R, g.E + g.R / COLS);
    const int warps = blocks > 4 * num_sms() ? 4 : blocks > 2 * num_sms() || g.K < 2048 ? 8 : 16;
    auto* kernel = warps == 4 ? grouped_i8_few_kernel<4> : warps == 8 ? grouped_i8_few_kernel<8> : grouped_i8_few_kernel<16>;
    return launch_overlapped(kernel, grid, dim3(32 * warps), 0, s, g, d);
}

}  // namespace moe
