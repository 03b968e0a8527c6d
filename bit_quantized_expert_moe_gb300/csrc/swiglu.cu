// Gated activation between the two expert products, with the routing weight.
//
//   h[r] = w_r * a s u,          s = 1 / (1 + e^-a), a = gu[r][0..F), u = gu[r][F..2F)
//   da = w_r dh u s (1 + a (1 - s)),  du = w_r dh a s,  dw_r = sum_f dh a s u
// with w_r = row_w[row_map[r]].  Each element is read and written once: bound
// by memory.  NT threads share a row (its sum is dw_r).
#include "internal.h"
#include "vec8.cuh"

namespace moe {
namespace {

// s(a) = 1 / (1 + e^-a) as inv * q * q with t = e^(-|a| / 2), inv = 1 / (1 + t^2)
// and q = 1 for a >= 0, t for a < 0: nothing overflows, and a product that
// takes the two factors q last underflows no earlier than its value does.
struct Sigmoid {
    float inv, q, other;  // other = 1 - s
    __device__ __forceinline__ explicit Sigmoid(float a) {
        const float t = expf(-0.5f * fabsf(a));
        inv = 1.f / (1.f + t * t);
        q = a < 0.f ? t : 1.f;
        const float qo = a < 0.f ? 1.f : t;
        other = inv * qo * qo;
    }
    __device__ __forceinline__ float times(float v) const { return v * inv * q * q; }
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
    const int chunks = F / 8;
    const long long total = (long long)R * chunks;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
        const int r = (int)(i / chunks), c = (int)(i - (long long)r * chunks);
        float w = 1.f;
        if (row_w) {
            const int wi = weight_index(row_map, r, R);
            w = wi >= 0 ? row_w[wi] : 0.f;
        }
        float a[8], u[8];
        load8<T>(gu, (size_t)r * 2 * chunks + c, a);
        load8<T>(gu, (size_t)r * 2 * chunks + chunks + c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = Sigmoid(a[j]).times(w * a[j] * u[j]);
        store8<T>(h, (size_t)i, a);
    }
}

template <class T, int NT>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT)
    swiglu_backward_kernel(const void* __restrict__ dh, const void* gu, const float* __restrict__ row_w,
                           const int32_t* __restrict__ row_map, int R, int F, void* dgu /* may be gu */,
                           float* __restrict__ drow_w) {
    __shared__ float red[2 * (NT / 32)];
    const int rpb = blockDim.x / NT, tid = threadIdx.x % NT;
    const int chunks = F / 8;
    int buf = 0;
    for (int r = blockIdx.x * rpb + threadIdx.x / NT; r < R; r += gridDim.x * rpb) {
        const int wi = row_w ? weight_index(row_map, r, R) : -1;
        const float w = row_w ? (wi >= 0 ? row_w[wi] : 0.f) : 1.f;
        float sum[1] = {0.f};
        for (int c = tid; c < chunks; c += NT) {
            float a[8], u[8], d[8];
            load8<T>(gu, (size_t)r * 2 * chunks + c, a);
            load8<T>(gu, (size_t)r * 2 * chunks + chunks + c, u);
            load8<T>(dh, (size_t)r * chunks + c, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Sigmoid s(a[j]);
                const float du = d[j] * u[j], wd = w * d[j];
                sum[0] += s.times(du * a[j]);
                u[j] = s.times(wd * a[j]);
                a[j] = s.times(w * du * (1.f + a[j] * s.other));
            }
            store8<T>(dgu, (size_t)r * 2 * chunks + c, a);
            store8<T>(dgu, (size_t)r * 2 * chunks + chunks + c, u);
        }
        if (drow_w) {  // the same for every thread of the block
            row_sum<NT, 1>(sum, red, buf);
            if (tid == 0 && wi >= 0) drow_w[wi] = sum[0];
        }
    }
}

}  // namespace

cudaError_t launch_swiglu(moe_dtype_t dt, const void* gu, const float* row_w, const int32_t* row_map, int R, int F,
                          void* h, cudaStream_t s) {
    const long long work = (long long)R * (F / 8);
    const int blocks = (int)std::min<long long>((long long)num_sms() * 8, (work + 255) / 256);
    if (dt == MOE_DT_BF16) swiglu_kernel<Bf16><<<blocks, 256, 0, s>>>(gu, row_w, row_map, R, F, h);
    else if (dt == MOE_DT_F16) swiglu_kernel<F16><<<blocks, 256, 0, s>>>(gu, row_w, row_map, R, F, h);
    else swiglu_kernel<F32><<<blocks, 256, 0, s>>>(gu, row_w, row_map, R, F, h);
    note_launch();
    return cudaGetLastError();
}

namespace {
template <class T>
void run_backward(const void* dh, const void* gu, const float* row_w, const int32_t* row_map, int R, int F, void* dgu,
                  float* drow_w, cudaStream_t s) {
    if (F <= 1024) {
        const int blocks = std::min(num_sms() * 16, ceil_div(R, 4));
        swiglu_backward_kernel<T, 32><<<blocks, 128, 0, s>>>(dh, gu, row_w, row_map, R, F, dgu, drow_w);
    } else {
        const int blocks = std::min(num_sms() * 8, R);
        swiglu_backward_kernel<T, 256><<<blocks, 256, 0, s>>>(dh, gu, row_w, row_map, R, F, dgu, drow_w);
    }
}
}  // namespace

cudaError_t launch_swiglu_backward(moe_dtype_t dt, const void* dh, const void* gu, const float* row_w,
                                   const int32_t* row_map, int R, int F, void* dgu, float* drow_w, cudaStream_t s) {
    if (dt == MOE_DT_BF16) run_backward<Bf16>(dh, gu, row_w, row_map, R, F, dgu, drow_w, s);
    else if (dt == MOE_DT_F16) run_backward<F16>(dh, gu, row_w, row_map, R, F, dgu, drow_w, s);
    else run_backward<F32>(dh, gu, row_w, row_map, R, F, dgu, drow_w, s);
    note_launch();
    return cudaGetLastError();
}

}  // namespace moe
