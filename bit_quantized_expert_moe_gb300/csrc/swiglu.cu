// Gated activation between the two expert products, with the routing weight.
//
//   h[r] = w_r * a s u,          s = 1 / (1 + e^-a), a = gu[r][0..F), u = gu[r][F..2F)
//   da = w_r dh u s (1 + a (1 - s)),  du = w_r dh a s,  dw_r = sum_f dh a s u
// with w_r = row_w[row_map[r]].  Each element is read and written once: bound
// by memory.  NT threads share a row (its sum is dw_r).
#include <type_traits>

#include "internal.h"
#include "vec8.cuh"

namespace moe {
namespace {

// SiLU and its slope for two gates a, s(a) = 1 / (1 + e^-a) from t = e^-|a|, so
// that nothing overflows: 1 / (1 + t) for a >= 0, t / (1 + t) below.  Each is
// a factor by itself and the others come in one by one: where s is 0, a (its type's
// lowest value even) times s is 0 and stays 0, whatever the others' product.
// 16-bit rows: the hardware's reciprocal (2 ulp; a division takes the backward
// kernel from 45 to 50 us at 32768 x 768).  Where nothing but 16-bit outputs is made
// (EXACT = false) the hardware's exponential too, whose documented bound of 2 + 1.173
// |a| ulp is 2^-18 at |a| = 24, below which fp16 results are subnormal or zero for
// |up| < 2^11, and 2^-16.2 at |a| = 87, where s leaves the normal numbers: a 64th of
// the half ulp of fp16, a 90th of bf16's.  The routing weight's gradient is fp32 and
// gets the library's (2 ulp).  us with the library's and the hardware's: forward
// 32768 x 768 30.0 and 23.7, backward 43.5 and 43.4, 40000 x 264 30.0 and 27.8.
template <class T, bool EXACT>
struct Silu {
    float2 as, ss;  // a s, s (1 + a (1 - s))
    __device__ __forceinline__ static void sigmoid(float a, float& s, float& other) {
        const float t = EXACT ? expf(-fabsf(a)) : __expf(-fabsf(a));
        const float inv = __fdividef(1.f, 1.f + t);
        s = a < 0.f ? t * inv : inv;
        other = 1.f - s;
    }
    __device__ __forceinline__ explicit Silu(float2 a) {
        float2 s, other;
        sigmoid(a.x, s.x, other.x);
        sigmoid(a.y, s.y, other.y);
        as = f2_mul(a, s);
        ss = f2_mul(s, ffma2(a, other, f2(1.f)));
    }
    __device__ __forceinline__ float2 rest(float2 v) const { return v; }
};
// fp32 outputs: s = q^2 / (1 + t^2) with t = e^(-|a| / 2) and q = 1 or t.  as and ss
// hold one factor q and rest(v), which comes last, the second: nothing before
// it underflows unless the result does, and 1 - s does not cancel.  The hardware's
// reciprocal (2 ulp); with a division the forward pass takes 57 us for 50 at 32768 x 768.
template <bool EXACT>
struct Silu<F32, EXACT> {
    float2 as, ss, q;
    __device__ __forceinline__ static void sigmoid(float a, float& s, float& q, float& other) {
        const float t = expf(-0.5f * fabsf(a)), inv = __fdividef(1.f, 1.f + t * t);
        const float qo = a < 0.f ? 1.f : t;
        q = a < 0.f ? t : 1.f;
        s = inv * q;
        other = inv * qo * qo;
    }
    __device__ __forceinline__ explicit Silu(float2 a) {
        float2 s, other;
        sigmoid(a.x, s.x, q.x, other.x);
        sigmoid(a.y, s.y, q.y, other.y);
        as = f2_mul(a, s);
        ss = f2_mul(s, ffma2(a, other, f2(1.f)));
    }
    __device__ __forceinline__ float2 rest(float2 v) const { return f2_mul(v, q); }
};

// Weight index of row r, -1 when the map's entry is out of range.
__device__ __forceinline__ int weight_index(const int32_t* row_map, int r, int R) {
    const int i = row_map ? row_map[r] : r;
    return (unsigned)i < (unsigned)R ? i : -1;
}

template <class T>
__global__ void __launch_bounds__(256) swiglu_kernel(const void* __restrict__ gu, const float* __restrict__ row_w,
                                                     const int32_t* __restrict__ row_map, int R, int F,
                                                     void* __restrict__ h) {
    grid_dependency_launch();
    grid_dependency_wait();
    const int chunks = F / 8;
    const long long total = (long long)R * chunks;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
        const int r = (int)(i / chunks), c = (int)(i - (long long)r * chunks);
        float w = 1.f;
        if (row_w) {
            const int wi = weight_index(row_map, r, R);
            w = wi >= 0 ? row_w[wi] : 0.f;
        }
        const V8 a = load8<T>(gu, (size_t)r * 2 * chunks + c);
        const V8 u = load8<T>(gu, (size_t)r * 2 * chunks + chunks + c);
        V8 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Silu<T, false> f(a.p[j]);
            v.p[j] = f2_mul(f2_mul(f.as, f2(w)), f.rest(u.p[j]));
        }
        store8<T>(h, (size_t)i, v);
    }
}

// A row by RowGroups of `threads` threads.  The chunks of a group's rows follow
// each other, the loads of the next SLOTS - 1 under way while one is computed.  fp32
// with two slots: four blocks an SM instead of three, 32768 x 768 78 -> 105 us.
constexpr int SLOTS = 3;
template <class T>
using BackwardRing = ThreadRing<T, 3, SLOTS>;

template <class T, bool EXACT>
__global__ void __launch_bounds__(256)
    swiglu_backward_kernel(const void* __restrict__ dh, const void* gu, const float* __restrict__ row_w,
                           const int32_t* __restrict__ row_map, int R, int F, void* dgu /* may be gu */,
                           float* __restrict__ drow_w, int threads) {
    extern __shared__ __align__(16) float smem[];
    grid_dependency_launch();
    grid_dependency_wait();
    const int groups = blockDim.x / threads, grp = threadIdx.x / threads;
    RowGroup rg(threads, grp, smem + grp * RowGroup::SUM_FLOATS);
    BackwardRing<T> ring(smem + groups * RowGroup::SUM_FLOATS);
    if (rg.tid < 16) rg.red[rg.tid] = rg.red[128 + rg.tid] = 0.f;
    rg.sync();
    const int chunks = F / 8, step = gridDim.x * groups;
    int fr = blockIdx.x * groups + grp, fc = rg.tid;  // the next chunk to fetch
    auto fetch = [&]() {
        if (fr < R) {
            if (fc < chunks) {
                constexpr size_t CH = 8 * T::BYTES;
                const unsigned char* a = static_cast<const unsigned char*>(gu) + ((size_t)fr * 2 * chunks + fc) * CH;
                ring.fetch(0, a);
                ring.fetch(1, a + chunks * CH);
                ring.fetch(2, static_cast<const unsigned char*>(dh) + ((size_t)fr * chunks + fc) * CH);
            }
            fc += threads;
            if (fc - rg.tid >= chunks) {
                fc = rg.tid;
                fr += step;
            }
        }
        ring.commit();
    };
#pragma unroll
    for (int k = 0; k < SLOTS - 1; ++k) fetch();
    for (int r = blockIdx.x * groups + grp; r < R; r += step) {
        const int wi = row_w ? weight_index(row_map, r, R) : -1;
        const float w = row_w ? (wi >= 0 ? row_w[wi] : 0.f) : 1.f;
        float sum = 0.f;
        for (int c0 = 0; c0 < chunks; c0 += threads) {
            fetch();
            ring.wait();
            const int c = c0 + rg.tid;
            if (c < chunks) {
                const V8 a = unpack8<T>(ring.get(0)), u = unpack8<T>(ring.get(1)), d = unpack8<T>(ring.get(2));
                V8 ga, gu_;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Silu<T, EXACT> f(a.p[j]);
                    const float2 das = f2_mul(f.as, d.p[j]), ur = f.rest(u.p[j]), h = f2_mul(das, ur);
                    sum += h.x + h.y;
                    gu_.p[j] = f2_mul(das, f.rest(f2(w)));
                    ga.p[j] = f2_mul(f2_mul(f2_mul(f.ss, d.p[j]), f2(w)), ur);
                }
                store8<T>(dgu, (size_t)r * 2 * chunks + c, ga);
                store8<T>(dgu, (size_t)r * 2 * chunks + chunks + c, gu_);
            }
            ring.next();
        }
        if (drow_w) {
            sum = rg.sum(sum);
            if (rg.tid == 0 && wi >= 0) drow_w[wi] = sum;
        }
    }
    cp_async_wait<0>();
}

}  // namespace

cudaError_t launch_swiglu(moe_dtype_t dt, const void* gu, const float* row_w, const int32_t* row_map, int R, int F,
                          void* h, cudaStream_t s) {
    const long long work = (long long)R * (F / 8);
    const int blocks = (int)std::min<long long>((long long)num_sms() * 8, (work + 255) / 256);
    auto* kernel = dt == MOE_DT_BF16 ? swiglu_kernel<Bf16> : dt == MOE_DT_F16 ? swiglu_kernel<F16> : swiglu_kernel<F32>;
    return launch_overlapped(kernel, blocks, 256, 0, s, gu, row_w, row_map, R, F, h);
}

namespace {
template <class T>
cudaError_t run_backward(const void* dh, const void* gu, const float* row_w, const int32_t* row_map, int R, int F, void* dgu,
                  float* drow_w, cudaStream_t s) {
    // rows enough for every warp of the GPU: a warp to a row, no barriers;
    // else more warps to a row
    const int want = num_sms() * 32;
    const int warps = std::max(1, std::min({8, ceil_div(F / 8, 32), want / R}));
    const int threads = 32 * warps, groups = 8 / warps;
    const int blocks = std::min(num_sms() * 5, ceil_div(R, groups));
    const size_t smem = groups * RowGroup::SUM_FLOATS * sizeof(float) + (size_t)threads * groups * BackwardRing<T>::BYTES_PER_THREAD;
    const auto launch = [&](auto exact) {
        return launch_overlapped<swiglu_backward_kernel<T, decltype(exact)::value>>(
            blocks, threads * groups, smem, s, dh, gu, row_w, row_map, R, F, dgu, drow_w, threads);
    };
    if constexpr (T::BYTES == 2)
        if (!drow_w) return launch(std::false_type{});
    return launch(std::true_type{});
}
}  // namespace

cudaError_t launch_swiglu_backward(moe_dtype_t dt, const void* dh, const void* gu, const float* row_w,
                                   const int32_t* row_map, int R, int F, void* dgu, float* drow_w, cudaStream_t s) {
    return dt == MOE_DT_BF16  ? run_backward<Bf16>(dh, gu, row_w, row_map, R, F, dgu, drow_w, s)
           : dt == MOE_DT_F16 ? run_backward<F16>(dh, gu, row_w, row_map, R, F, dgu, drow_w, s)
                              : run_backward<F32>(dh, gu, row_w, row_map, R, F, dgu, drow_w, s);
}

}  // namespace moe
