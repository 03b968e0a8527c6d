// y = (x W_e^T) by the rows' and the output channels' scales, of 8-bit codes, for a
// handful of rows in all or for about one an expert: decoding.
//
// As for 16-bit weights (grouped_few.cu) the weights' bytes are all that counts: KW
// warps take 16 weight rows of one expert and up to 8 of its rows; they share K and add
// up in shared memory.  Integer sums, exact in any order; one rounding at the
// end.  Lane 4 g + t holds elements 16 t .. 16 t + 15 of every 64 for weight rows g and
// g + 8.  Up to four rows by dp4a, a row at a time; more by mma.sync m16n8k32, which
// runs at 1/11 of the 16-bit rate here and, at one row, costs more than the weights:
// 8 rows of 8 experts, N 1536, K 2048 9.4 us, by dp4a 7.1; N 4096, K 7168 42.2 and 38.0.
#include <type_traits>

#include "internal.h"

namespace moe {
namespace {

constexpr int ROWS = 16, COLS = 8;

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

// This warp's part of K [k0, k1) of the products of weight rows wa and wb with RW rows.
template <int RW, int AHEAD>
__device__ __forceinline__ void dots(const int8_t* wa, const int8_t* wb, const int8_t* x, size_t ld, int k0, int k1, int t,
                                     int (&acc)[RW][2]) {
    for (int k = k0; k < k1; k += 64 * AHEAD) {
        uint4 a[AHEAD], b[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = k + 64 * i + 16 * t < k1;
            a[i] = in ? load_codes(wa + k + 64 * i) : make_uint4(0, 0, 0, 0);
            b[i] = in ? load_codes(wb + k + 64 * i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int j = 0; j < RW; ++j) {
                const bool in = k + 64 * i + 16 * t < k1;
                const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(x + j * ld + k + 64 * i)) : make_uint4(0, 0, 0, 0);
                const uint32_t c[4] = {v.x, v.y, v.z, v.w};
                const uint32_t p[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, q[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    acc[j][0] = __dp4a((int)p[m], (int)c[m], acc[j][0]);
                    acc[j][1] = __dp4a((int)q[m], (int)c[m], acc[j][1]);
                }
            }
    }
}

// AHEAD: pairs of weight loads under way.
template <int WARPS, int AHEAD, int KW = WARPS>
__global__ void __launch_bounds__(32 * WARPS) grouped_i8_few_kernel(const GroupedI8Shape g, const GroupedI8Data d) {
    __shared__ int seg[3];
    __shared__ int part[WARPS][COLS][ROWS + 1];
    if (threadIdx.x == 0) seg[0] = -1;
    grid_dependency_launch();
    __syncthreads();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int NW = WARPS / KW;  // times 16 weight rows
    const int r = blockIdx.y, n0 = (blockIdx.x * NW + warp / KW) * ROWS;
    // the row's expert and its segment
    bool bad = false;
    for (int i = threadIdx.x; i < g.E; i += 32 * WARPS) {
        const int lo = __ldg(g.offsets + i), hi = __ldg(g.offsets + i + 1);
        bad |= lo < 0 || hi < lo || hi > g.R;
        if (lo <= r && r < hi) {
            seg[0] = i;
            seg[1] = lo;
            seg[2] = hi;
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && r == 0) set_error(g.err, ERRBIT_RANGE);
        return;
    }
    const int e = seg[0], r0 = seg[1], r1 = seg[2];
    if (e < 0 || (r - r0) % COLS) return;  // in no segment; another block's
    const int rows = min(COLS, r1 - r);

    const int gi = lane >> 2, t = lane & 3;
    const int kq = ceil_div(g.K, 64 * KW) * 64, k0 = warp % KW * kq, k1 = min(g.K, k0 + kq);
    const size_t ld = (size_t)g.K;
    const int8_t* wa = d.w + ((size_t)e * g.N + min(n0 + gi, g.N - 1)) * ld + 16 * t;
    const int8_t* wb = d.w + ((size_t)e * g.N + min(n0 + gi + 8, g.N - 1)) * ld + 16 * t;
    const int8_t* x0 = d.x + (size_t)r * ld + 16 * t;
    // the lanes' sums of RW rows, added up over t
    auto few = [&](auto n) {
        constexpr int RW = decltype(n)::value;
        int acc[RW][2] = {};
        dots<RW, AHEAD>(wa, wb, x0, ld, k0, k1, t, acc);
#pragma unroll
        for (int j = 0; j < RW; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int v = acc[j][h];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (t == 0) part[warp][j][gi + 8 * h] = v;
            }
    };
    if (rows == 1) few(std::integral_constant<int, 1>{});
    else if (rows == 2) few(std::integral_constant<int, 2>{});
    else if (rows == 3) few(std::integral_constant<int, 3>{});
    else if (rows == 4) few(std::integral_constant<int, 4>{});
    else {
        const int8_t* xr = x0 + (size_t)min(gi, rows - 1) * ld;
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
    }
    __syncthreads();
    for (int i = threadIdx.x; i < NW * COLS * ROWS; i += 32 * WARPS) {
        const int nw = i / (COLS * ROWS), col = i / ROWS % COLS, n = (blockIdx.x * NW + nw) * ROWS + i % ROWS;
        if (col >= rows || n >= g.N) continue;
        int s = 0;
#pragma unroll
        for (int w = 0; w < KW; ++w) s += part[nw * KW + w][col][i % ROWS];
        const float v = (float)s * __ldg(d.w_scale + (size_t)e * g.N + n) * __ldg(d.x_scale + r + col);
        static_cast<uint16_t*>(d.y)[(size_t)(r + col) * g.N + n] =
            g.out == MOE_DT_BF16 ? float_to_bf16_bits(v) : float_to_f16_bits(v);
    }
}

}  // namespace

// Warps that share K: four, more where the blocks leave SMs without loads under way (two:
// 8 rows of 1536 x 2048 7.9 us for 6.4, 32 of 2048 x 768 9.8 for 9.4; eight 7.8 and 14.7).
// Of the four, each asks for its part of K at once, or in as few and as even rounds as
// 8 pairs of loads allow: with 4, 8 and 3 pairs 8 rows of 1536 x 2048 6.8, 6.4 us; 32 rows of
// 2048 x 768 10.8, 11.7 and 9.4.  Where K is short, two of them or each one has weight rows
// of its own: a block's set-up takes longer than its part of K
// (105 rows, 176 experts of 2704 x 176 21.8 -> 10.3 us, 75 rows, 249 of 3272 x 128 8.1 -> 5.0,
// 16 rows, 128 of 2048 x 512 7.8 -> 7.0).
cudaError_t launch_grouped_i8_few(const GroupedI8Shape& g, const GroupedI8Data& d, cudaStream_t s) {
    // blocks with work, at most, if all warps share K
    const long long blocks = (long long)ceil_div(g.N, ROWS) * std::min(g.R, g.E + g.R / COLS);
    const int warps = blocks > 4 * num_sms() ? 4 : blocks > 2 * num_sms() || g.K < 2048 ? 8 : 16;
    const int share = warps > 4 || g.K > 512 ? warps : g.K > 256 ? 2 : 1;
    const int units = ceil_div(g.K, 64 * share), ahead = ceil_div(units, ceil_div(units, 8));
    auto* kernel = warps == 16  ? grouped_i8_few_kernel<16, 4>
                   : warps == 8 ? grouped_i8_few_kernel<8, 4>
                   : share == 1 ? grouped_i8_few_kernel<4, 4, 1>
                   : share == 2 ? grouped_i8_few_kernel<4, 4, 2>
                   : ahead > 6  ? grouped_i8_few_kernel<4, 8>
                   : ahead > 4  ? grouped_i8_few_kernel<4, 6>
                   : ahead > 3  ? grouped_i8_few_kernel<4, 4>
                                : grouped_i8_few_kernel<4, 3>;
    const dim3 grid(ceil_div(g.N, ROWS * (warps / share)), g.R);
    return launch_overlapped(kernel, grid, dim3(32 * warps), 0, s, g, d);
}

}  // namespace moe
