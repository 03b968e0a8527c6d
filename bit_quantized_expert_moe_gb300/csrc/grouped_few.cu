// y = x W_e^T for a handful of rows in all, or for about one an expert: decoding.
//
// The weights' bytes are all that counts, and a few tiles of 256 weight rows
// would not occupy every SM.  A block takes 16 weight rows of one expert and up
// to 8 of its rows; its warps (4 to 16) share K and add up in shared memory.  A
// weight goes from memory to a register once and from there into the tensor
// cores (mma.sync m16n8k16: 16 weight rows, 8 rows of x): with so few rows the
// tcgen05 path's staging would only add latency.  Both operands keep K in the
// order in which a thread's 16-byte loads bring it (the same for both, so the
// dot product is unchanged): lane 4 g + t holds elements 8 t .. 8 t + 7 of every
// 32 for weight rows g and g + 8 and for row g of x.
#include "internal.h"

namespace moe {
namespace {

// A weight load, read once: it leaves L1 alone and asks L2 for the 256 bytes
// around it, of which the warp's other loads take the rest (16 rows of 8 of 256
// experts, N 4096, K 7168: 154 -> 139 us; one token at N 1536, K 2048 12.3 -> 12.1).
__device__ __forceinline__ uint4 load_weights(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// AHEAD: pairs of weight loads under way, 32 registers of the 54 that the four-warp
// kernel takes.  With 8 the compiler puts loads behind the first products (46
// registers in all).  us with 2, 4, 8: 8 rows of 8 experts, N 1536, K 2048 12.6, 12.4,
// 12.8; N 4096, K 7168 76.1, 73.5, 75.9; 32 rows of 32 36.9, 34.2, 36.6; 16 rows of 8,
// N 1024, K 256 3.0, 2.9, 3.4.
constexpr int ROWS = 16, COLS = 8, AHEAD = 4;

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool BF16, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) grouped_few_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w,
                                                                 uint16_t* __restrict__ y, GroupedShape g) {
    __shared__ int cnt[WARPS];
    __shared__ float part[WARPS][COLS][ROWS + 1];
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
    const int kq = (ceil_div(g.K, 32 * WARPS)) * 32, k0 = warp * kq, k1 = min(g.K, k0 + kq);
    const size_t ld = (size_t)g.K;
    const uint16_t* wa = w + ((size_t)e * g.N + min(n0 + gi, g.N - 1)) * ld + 8 * t;
    const uint16_t* wb = w + ((size_t)e * g.N + min(n0 + gi + 8, g.N - 1)) * ld + 8 * t;
    const uint16_t* xr = x + (size_t)(r + min(gi, rows - 1)) * ld + 8 * t;
    const bool has = gi < rows;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = k0; k < k1; k += 32 * AHEAD) {
        uint4 a[AHEAD], b[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = k + 32 * i + 8 * t < k1;
            a[i] = in ? load_weights(wa + k + 32 * i) : make_uint4(0, 0, 0, 0);
            b[i] = in ? load_weights(wb + k + 32 * i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = has && k + 32 * i + 8 * t < k1;
            const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(xr + k + 32 * i)) : make_uint4(0, 0, 0, 0);
            mma16816<BF16>(acc, a[i].x, b[i].x, a[i].y, b[i].y, v.x, v.y);
            mma16816<BF16>(acc, a[i].z, b[i].z, a[i].w, b[i].w, v.z, v.w);
        }
    }
    part[warp][2 * t][gi] = acc[0];
    part[warp][2 * t + 1][gi] = acc[1];
    part[warp][2 * t][gi + 8] = acc[2];
    part[warp][2 * t + 1][gi + 8] = acc[3];
    __syncthreads();
    const int col = threadIdx.x / ROWS, n = threadIdx.x % ROWS;
    if (col < rows && n0 + n < g.N) {  // (the first 128 threads)
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += part[i][col][n];
        y[(size_t)(r + col) * g.N + n0 + n] = BF16 ? float_to_bf16_bits(s) : float_to_f16_bits(s);
    }
}

}  // namespace

// Warps that share K: four, more where the blocks leave SMs without loads under
// way.  us with 4, 8, 16 warps: 66 blocks, K 6592 28.1, 14.4, 8.7; 256, K 4096 15.6, 10.5,
// 8.7; 64, K 512 2.5, 2.3, 2.5; 512, K 1024 6.6, 6.0, 6.9; 768, K 2048 12.5, 13.6, 13.5.
cudaError_t launch_grouped_few(const GroupedShape& g, const void* x, const void* w, void* y, cudaStream_t s) {
    const dim3 grid(ceil_div(g.N, ROWS), g.R);
    const auto *xp = static_cast<const uint16_t*>(x), *wp = static_cast<const uint16_t*>(w);
    auto* yp = static_cast<uint16_t*>(y);
    const bool bf = g.dtype == MOE_DT_BF16;
    // blocks with work, at most
    const long long blocks = (long long)grid.x * std::min(g.R, g.E + g.R / COLS);
    const int warps = blocks > 4 * num_sms() ? 4 : blocks > 2 * num_sms() || g.K < 1024 ? 8 : 16;
    auto* kernel = bf ? grouped_few_kernel<true, 4> : grouped_few_kernel<false, 4>;
    if (warps == 8) kernel = bf ? grouped_few_kernel<true, 8> : grouped_few_kernel<false, 8>;
    if (warps == 16) kernel = bf ? grouped_few_kernel<true, 16> : grouped_few_kernel<false, 16>;
    return launch_overlapped(kernel, grid, dim3(32 * warps), 0, s, xp, wp, yp, g);
}

}  // namespace moe
