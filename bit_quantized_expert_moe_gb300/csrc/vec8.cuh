// Eight consecutive elements of a row as fp32: the unit in which the 16-bit
// expert operators read and write rows (16 bytes of bf16 or fp16, 32 of fp32).
#pragma once

#include "common.cuh"

namespace moe {

struct Bf16 { using Raw = uint4; static constexpr int BYTES = 2; };
struct F16 { using Raw = uint4; static constexpr int BYTES = 2; };
struct Raw32 { uint4 a, b; };
struct F32 { using Raw = Raw32; static constexpr int BYTES = 4; };

// Chunk c (elements 8 c .. 8 c + 7) behind `base`, as stored.
template <class T>
__device__ __forceinline__ typename T::Raw load_raw(const void* base, size_t chunk) {
    if constexpr (T::BYTES == 2) {
        return static_cast<const uint4*>(base)[chunk];
    } else {
        Raw32 r;
        r.a = static_cast<const uint4*>(base)[2 * chunk];
        r.b = static_cast<const uint4*>(base)[2 * chunk + 1];
        return r;
    }
}

template <class T>
__device__ __forceinline__ void unpack8(const typename T::Raw& r, float (&v)[8]) {
    if constexpr (T::BYTES == 4) {
        const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    } else {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (__is_same(T, Bf16)) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

template <class T>
__device__ __forceinline__ void load8(const void* base, size_t chunk, float (&v)[8]) {
    unpack8<T>(load_raw<T>(base, chunk), v);
}

// Rounds once (nearest even) to the stored type.
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (__is_same(T, Bf16)) return pack_bf16x2(lo, hi);
    else return pack_f16x2(lo, hi);
}

template <class T>
__device__ __forceinline__ void store8(void* base, size_t chunk, const float (&v)[8]) {
    if constexpr (T::BYTES == 4) {
        static_cast<float4*>(base)[2 * chunk] = make_float4(v[0], v[1], v[2], v[3]);
        static_cast<float4*>(base)[2 * chunk + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        static_cast<uint4*>(base)[chunk] =
            make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
}

// One element.
template <class T>
__device__ __forceinline__ float load1(const void* base, size_t i) {
    if constexpr (__is_same(T, Bf16)) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[i] << 16);
    else if constexpr (__is_same(T, F16)) return half_bits_to_float(static_cast<const uint16_t*>(base)[i]);
    else return static_cast<const float*>(base)[i];
}
template <class T>
__device__ __forceinline__ void store1(void* base, size_t i, float v) {
    if constexpr (__is_same(T, Bf16)) static_cast<uint16_t*>(base)[i] = float_to_bf16_bits(v);
    else if constexpr (__is_same(T, F16)) static_cast<uint16_t*>(base)[i] = float_to_f16_bits(v);
    else static_cast<float*>(base)[i] = v;
}

// Sum of one value a thread over the NT threads that share a row; every thread
// gets it.  NT = 32: by shuffles.  NT = the whole block: shuffles, then one
// block barrier; `buf` alternates between two halves of `red` ([2][MAXV][NT / 32]),
// so that a value is not overwritten before the slowest warp has read it.
template <int NT, int MAXV, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* red, int& buf) {
    static_assert(NV <= MAXV, "sums exceed the buffer");
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (NT > 32) {
        constexpr int W = NT / 32;
        float* r = red + buf * MAXV * W;
        buf ^= 1;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) r[i * W + warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += r[i * W + w];
            v[i] = s;
        }
    }
}

}  // namespace moe
