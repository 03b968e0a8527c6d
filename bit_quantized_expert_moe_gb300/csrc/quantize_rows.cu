// Rows to 8-bit codes with a scale for each row, gathered on the way:
//   a = max |x[i]|,  scale = a / 127,  code = 127 x / a rounded to nearest even
// for x = row (row_map[r] / k), so that the rows of a permutation go to their places
// without a 16-bit copy in between.
//
// What bounds it is not the memory but the instructions of an element, and packed ones
// keep them at about five: the maximum of pairs of 16-bit patterns, products and sums of
// pairs in fp32, and rounding by adding 1.5 2^23, whose low byte is the code.  A thread
// holds its part of the row in registers between the maximum and the codes.  Where the
// gather makes several rows of one, as top-k routing does, the rows of x are quantised
// once into the workspace and their codes copied.
// 4096 rows of 2048 bf16 gathered to 32768: 17 us, 67 MB written; each of the 32768
// quantised by itself 32 us, with each code's border looked at alone 59 us, and 77 us
// where bf16's frequent ties took a branch.
//
// The codes are those of the formula exactly.  With y = 1 / a, t0 = (127 x) y and the
// residual 127 x - t0 a, which an fma has exactly, t = t0 + residual y is the quotient
// rounded to fp32, and the quotient itself where it lies on the border n + 1/2 between
// two codes.  Any other quotient of 16-bit numbers is at least 2^-19 t away from a border
// (254 x and (2 n + 1) a are multiples of x's last place), 32 roundings.  fp32 rows can
// be closer: where t is a border there, it is compared in 64 bits.
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

// The largest |x| of eight elements as its pattern in T's width: ordered, and a NaN is
// above infinity.  16 bits: of either half, to be joined at the end.
template <class T>
__device__ __forceinline__ uint32_t largest(uint32_t m, const typename T::Raw& r) {
    if constexpr (T::BYTES == 2) {
        m = __vmaxu2(__vmaxu2(m, r.x & 0x7FFF7FFFu), r.y & 0x7FFF7FFFu);
        return __vmaxu2(__vmaxu2(m, r.z & 0x7FFF7FFFu), r.w & 0x7FFF7FFFu);
    } else {
        const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
        return m;
    }
}
// That pattern as fp32.
template <class T>
__device__ __forceinline__ float value(uint32_t m) {
    if constexpr (T::BYTES == 4) return __uint_as_float(m);
    const uint32_t h = max(m & 0xFFFFu, m >> 16);
    if constexpr (__is_same(T, Bf16)) return __uint_as_float(h << 16);
    else return half_bits_to_float((uint16_t)h);
}

// The code of v where v 127 / top is next to t = m + 1/2 in fp32.
__device__ __noinline__ int border_code(float v, float t, float top) {
    const int m = (int)fabsf(t);
    const double a = 254.0 * fabs((double)v), b = (2.0 * m + 1.0) * (double)top;
    const int c = a > b || (a == b && (m & 1)) ? m + 1 : m;
    return t < 0.f ? -c : c;
}

// Eight codes; y = 1 / top (0 for a row of zeros).
template <class T>
__device__ __forceinline__ uint2 codes8(const V8& v, float y, float top) {
    constexpr float M = 12582912.f;
    float2 t[4], s[4];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = f2_mul(v.p[i], f2(127.f));
        t[i] = f2_mul(x, f2(y));
        float2 r = ffma2(t[i], f2(-top), x);
        if (T::BYTES == 4)  // 127 x is rounded itself
            r = ffma2(ffma2(v.p[i], f2(127.f), make_float2(-x.x, -x.y)), f2(1.f), r);
        t[i] = ffma2(r, f2(y), t[i]);
        s[i] = ffma2(t[i], f2(1.f), f2(M));
        if (T::BYTES == 4) {
            const float2 d = ffma2(ffma2(s[i], f2(1.f), f2(-M)), f2(-1.f), t[i]);
            off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
        }
    }
    if (T::BYTES == 4 && __builtin_expect(off == 0.5f, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (fabsf(t[i].x - rintf(t[i].x)) == 0.5f) s[i].x = __int_as_float(border_code(v.p[i].x, t[i].x, top));
            if (fabsf(t[i].y - rintf(t[i].y)) == 0.5f) s[i].y = __int_as_float(border_code(v.p[i].y, t[i].y, top));
        }
    }
    auto bytes = [](float2 a, float2 b) {
        return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                           __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
    };
    return make_uint2(bytes(s[0], s[1]), bytes(s[2], s[3]));
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
    typename T::Raw v[VPT][2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int u = i * THREADS + tid;
        v[i][0] = v[i][1] = typename T::Raw{};
        if (there && u < units) {
            const size_t c = (size_t)src * units * 2 + 2 * u;
            v[i][0] = load_raw<T>(p.x, c);
            v[i][1] = load_raw<T>(p.x, c + 1);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) top = largest<T>(largest<T>(top, v[i][0]), v[i][1]);
    if (T::BYTES == 2) top = max(top & 0xFFFFu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if (THREADS > 32) {
        if ((tid & 31) == 0) most[grp][tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) top = max(top, most[grp][w]);
    }
    if (r >= p.R) return;
    const float a = value<T>(top);
    const bool finite = a < INFINITY;  // (false for a NaN)
    // rows whose 127 a or 1 / a is no ordinary number: in other units
    const float unit = a < 0x1p-60f ? 0x1p80f : a > 0x1p100f ? 0x1p-20f : 1.f;
    const float y = finite && a > 0.f ? 1.f / (a * unit) : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int u = i * THREADS + tid;
        if (u >= units) continue;
        uint2 o[2] = {make_uint2(0, 0), make_uint2(0, 0)};
        if (finite)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                V8 x = unpack8<T>(v[i][h]);
                if (unit != 1.f) x = mul(x, unit);
                o[h] = codes8<T>(x, y, a * unit);
            }
        reinterpret_cast<uint4*>(p.codes)[(size_t)r * units + u] = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y);
    }
    // a row with an infinity or a NaN has no codes: its scale, and all that is made with it, is NaN
    if (tid == 0) p.scales[r] = finite ? a / 127.f : __uint_as_float(0x7FC00000u);
}

// codes[r] = made[row_map[r] / k], and the scales: G lanes a row, four loads under way.
struct CopyArgs {
    const int32_t* row_map;
    int k, T, R, units;
    const uint4* made;
    const float* made_scales;
    uint4* codes;
    float* scales;
};
template <int G>
__global__ void __launch_bounds__(256) gather_codes_kernel(const CopyArgs p) {
    constexpr int ROWS = 256 / G, AHEAD = 4;
    grid_dependency_launch();
    grid_dependency_wait();
    const int r = blockIdx.x * ROWS + threadIdx.x / G, t = threadIdx.x % G;
    if (r >= p.R) return;
    const int a = __ldg(p.row_map + r), src = a < 0 ? -1 : a / p.k;
    const bool there = src >= 0 && src < p.T;
    const uint4* from = p.made + (size_t)(there ? src : 0) * p.units;
    uint4* to = p.codes + (size_t)r * p.units;
    for (int u = t; u < p.units; u += AHEAD * G) {
        uint4 v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (there && u + i * G < p.units) v[i] = __ldg(from + u + i * G);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (u + i * G < p.units) to[u + i * G] = v[i];
    }
    if (t == 0) p.scales[r] = there ? __ldg(p.made_scales + src) : 0.f;
}

template <class T, int VPT, int THREADS>
cudaError_t run(const QuantArgs& p, cudaStream_t s) {
    constexpr int rows = THREADS >= 256 ? 1 : 256 / THREADS;
    return launch_overlapped(quantize_rows_kernel<T, VPT, THREADS>, ceil_div(p.R, rows), rows * THREADS, 0, s, p);
}
template <class T>
cudaError_t run(const QuantArgs& p, cudaStream_t s) {
    // a thread's elements of a row: 32, fewer where the rows do not fill the GPU
    const int units = p.D / 16;
    if ((long long)p.R * units < 32ll * 1024 * num_sms()) {
        if (units <= 32) return run<T, 1, 32>(p, s);
        if (units <= 64) return run<T, 1, 64>(p, s);
        if (units <= 128) return run<T, 1, 128>(p, s);
        if (units <= 256) return run<T, 1, 256>(p, s);
    }
    if (units <= 64) return run<T, 2, 32>(p, s);
    if (units <= 128) return run<T, 2, 64>(p, s);
    if (units <= 256) return run<T, 2, 128>(p, s);
    if (units <= 512) return run<T, 2, 256>(p, s);
    if (units <= 1024) return run<T, 2, 512>(p, s);
    return run<T, 4, 512>(p, s);
}

constexpr long long MADE_ONCE = 16 << 20;
size_t made_scales_bytes(int T) { return ((size_t)T * 4 + 255) / 256 * 256; }

}  // namespace

// A second launch pays where rows of x are taken at least twice on average and there is
// more to save than its latency.  By themselves and once: 4096 rows of 2048 bf16 taken
// 8 times 31.6, 17.5 us, 512 of 7168 12.2, 9.8; 4096 of 2048 taken twice 8.8, 8.9; 512 of
// 2048 taken 8 times 5.1, 5.9.
size_t quantize_rows_bytes(int T, int R, int D) {
    if (R / 2 < T || (long long)R * D < MADE_ONCE) return 0;
    return made_scales_bytes(T) + (size_t)T * D;
}
cudaError_t launch_quantize_rows(moe_dtype_t dt, const void* x, const int32_t* row_map, int k, int T, int R, int D,
                                 int8_t* codes, float* scales, void* ws, cudaStream_t s) {
    auto rows = [&](const QuantArgs& p) {
        return dt == MOE_DT_BF16 ? run<Bf16>(p, s) : dt == MOE_DT_F16 ? run<F16>(p, s) : run<F32>(p, s);
    };
    if (!ws || !row_map || T == 0 || quantize_rows_bytes(T, R, D) == 0)
        return rows(QuantArgs{x, row_map, k, T, R, D, codes, scales});
    auto* made_scales = static_cast<float*>(ws);
    auto* made = static_cast<int8_t*>(ws) + made_scales_bytes(T);
    const cudaError_t err = rows(QuantArgs{x, nullptr, 1, T, T, D, made, made_scales});
    if (err != cudaSuccess) return err;
    const int units = D / 16, lanes = units < 32 ? 8 : 32;
    const CopyArgs p{row_map, k, T, R, units, reinterpret_cast<const uint4*>(made), made_scales,
                     reinterpret_cast<uint4*>(codes), scales};
    return launch_overlapped(lanes == 8 ? gather_codes_kernel<8> : gather_codes_kernel<32>, ceil_div(R, 256 / lanes), 256,
                             0, s, p);
}

}  // namespace moe
