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

// Eight values as four pairs, the operands of Blackwell's two-wide fp32
// instructions (half as many as one value at a time; each is rounded alone).
struct V8 {
    float2 p[4];
};
__device__ __forceinline__ unsigned long long f2_bits(float2 v) { return *reinterpret_cast<unsigned long long*>(&v); }
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ V8 v8(float v) { return V8{{f2(v), f2(v), f2(v), f2(v)}}; }
// a b, a b + c, the sum of a b added to s
__device__ __forceinline__ V8 mul(const V8& a, const V8& b) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = f2_mul(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ V8 mul(const V8& a, float b) { return mul(a, v8(b)); }
__device__ __forceinline__ V8 fma(const V8& a, const V8& b, const V8& c) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = ffma2(a.p[i], b.p[i], c.p[i]);
    return r;
}
__device__ __forceinline__ V8 fma(const V8& a, float b, const V8& c) { return fma(a, v8(b), c); }
__device__ __forceinline__ void dot(float2& s, const V8& a, const V8& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = ffma2(a.p[i], b.p[i], s);
}

template <class T>
__device__ __forceinline__ V8 unpack8(const typename T::Raw& r) {
    V8 v;
    if constexpr (T::BYTES == 4) {
        const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
    } else {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (__is_same(T, Bf16))
                v.p[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
            else
                v.p[i] = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        }
    }
    return v;
}

template <class T>
__device__ __forceinline__ V8 load8(const void* base, size_t chunk) {
    return unpack8<T>(load_raw<T>(base, chunk));
}

// Rounds once (nearest even) to the stored type.
template <class T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
    if constexpr (__is_same(T, Bf16)) return pack_bf16x2(v.x, v.y);
    else return pack_f16x2(v.x, v.y);
}

template <class T>
__device__ __forceinline__ void store8(void* base, size_t chunk, const V8& v) {
    if constexpr (T::BYTES == 4) {
        static_cast<float4*>(base)[2 * chunk] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
        static_cast<float4*>(base)[2 * chunk + 1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
    } else {
        static_cast<uint4*>(base)[chunk] = make_uint4(pack2<T>(v.p[0]), pack2<T>(v.p[1]), pack2<T>(v.p[2]), pack2<T>(v.p[3]));
    }
}

// A chunk of a parameter whose type is known at run time only.
__device__ __forceinline__ V8 load8(moe_dtype_t t, const void* base, size_t chunk) {
    return t == MOE_DT_F32 ? load8<F32>(base, chunk) : t == MOE_DT_BF16 ? load8<Bf16>(base, chunk) : load8<F16>(base, chunk);
}
__device__ __forceinline__ void store8(moe_dtype_t t, void* base, size_t chunk, const V8& v) {
    if (t == MOE_DT_F32) store8<F32>(base, chunk, v);
    else if (t == MOE_DT_BF16) store8<Bf16>(base, chunk, v);
    else store8<F16>(base, chunk, v);
}
// One element.
__device__ __forceinline__ void store1(moe_dtype_t t, void* base, size_t i, float v) {
    if (t == MOE_DT_F32) static_cast<float*>(base)[i] = v;
    else static_cast<uint16_t*>(base)[i] = t == MOE_DT_BF16 ? float_to_bf16_bits(v) : float_to_f16_bits(v);
}

// Sums of NV values a thread over one warp; every lane gets them.
template <int NV>
__device__ __forceinline__ void warp_sum(float (&v)[NV]) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// The W warps (at most 16) that share a row and meet at a named barrier of
// their own, so that several rows can be on their way in one block.
struct RowGroup {
    static constexpr int SUM_FLOATS = 2 * 8 * 16;  // shared memory of a group: [2][8][16]
    int tid, threads, warps, warp, lane, bar;
    float* red;
    int buf;

    // Group `g` of `threads` threads; `red` is the group's SUM_FLOATS, cleared.
    __device__ __forceinline__ RowGroup(int threads_, int g, float* red_)
        : threads(threads_), warps(threads_ >> 5), bar(1 + g), red(red_), buf(0) {
        tid = (int)threadIdx.x - g * threads_;
        warp = tid >> 5;
        lane = tid & 31;
    }
    __device__ __forceinline__ void sync() const {
        if (warps > 1) asm volatile("bar.sync %0, %1;" :: "r"(bar), "r"(threads) : "memory");
    }
    // One value a thread.  `buf` alternates between two halves of `red`: a value
    // is overwritten two sums later, when every warp has passed the barrier in
    // between and so has read it.
    __device__ __forceinline__ float sum(float v) {
        float a[1] = {v};
        warp_sum(a);
        if (warps == 1) return a[0];
        float* r = red + buf * 128;
        buf ^= 1;
        if (lane == 0) r[warp] = a[0];
        sync();
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = reinterpret_cast<const float4*>(r)[i];
            s += (f.x + f.y) + (f.z + f.w);
        }
        return s;
    }
    // Two values a thread, likewise: one step of exchange, then lane l holds value l / 16.
    __device__ __forceinline__ void sum2(float (&v)[2]) {
        const bool h4 = lane & 16;
        float c = (h4 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, h4 ? v[0] : v[1], 16);
        c += __shfl_xor_sync(0xffffffffu, c, 8);
        c += __shfl_xor_sync(0xffffffffu, c, 4);
        c += __shfl_xor_sync(0xffffffffu, c, 2);
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        if (warps == 1) {
            v[0] = __shfl_sync(0xffffffffu, c, 0);
            v[1] = __shfl_sync(0xffffffffu, c, 16);
            return;
        }
        float* r = red + buf * 128;
        buf ^= 1;
        if ((lane & 15) == 0) r[(lane >> 4) * 16 + warp] = c;
        sync();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = reinterpret_cast<const float4*>(r + 16 * k)[i];
                v[k] += (f.x + f.y) + (f.z + f.w);
            }
        }
    }
    // Four values a thread.  Halving exchange: each step sends half of the
    // values a lane still holds to the lane across, so four values take 6
    // shuffles instead of 20; lane l ends up with value l / 8.
    __device__ __forceinline__ void sum4(float (&v)[4]) {
        float a[2], c;
        const bool h4 = lane & 16, h3 = lane & 8;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            a[i] = (h4 ? v[2 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, h4 ? v[i] : v[2 + i], 16);
        c = (h3 ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, h3 ? a[0] : a[1], 8);
        c += __shfl_xor_sync(0xffffffffu, c, 4);
        c += __shfl_xor_sync(0xffffffffu, c, 2);
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        if (warps > 1) {
            float* r = red + buf * 128;
            buf ^= 1;
            if ((lane & 7) == 0) r[(lane >> 3) * 16 + warp] = c;
            sync();
            const float2 f = reinterpret_cast<const float2*>(r)[lane];  // value lane / 8, two warps' sums
            c = f.x + f.y;
            c += __shfl_xor_sync(0xffffffffu, c, 4);
            c += __shfl_xor_sync(0xffffffffu, c, 2);
            c += __shfl_xor_sync(0xffffffffu, c, 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, c, 8 * i);
    }
    // Six values a thread, likewise: 8 values, two of them zero, take 9
    // shuffles; lane l ends up with value l / 4.
    __device__ __forceinline__ void sum6(float (&v)[6]) {
        float a[4], b[2], c;
        const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = v[i], hi = i < 2 ? v[4 + i] : 0.f;
            a[i] = (h4 ? hi : lo) + __shfl_xor_sync(0xffffffffu, h4 ? lo : hi, 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            b[i] = (h3 ? a[2 + i] : a[i]) + __shfl_xor_sync(0xffffffffu, h3 ? a[i] : a[2 + i], 8);
        c = (h2 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, h2 ? b[0] : b[1], 4);
        c += __shfl_xor_sync(0xffffffffu, c, 2);
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        if (warps > 1) {
            float* r = red + buf * 128;
            buf ^= 1;
            if ((lane & 3) == 0) r[(lane >> 2) * 16 + warp] = c;
            sync();
            const float4 f = reinterpret_cast<const float4*>(r)[lane];  // value lane / 4, four warps' sums
            c = (f.x + f.y) + (f.z + f.w);
            c += __shfl_xor_sync(0xffffffffu, c, 2);
            c += __shfl_xor_sync(0xffffffffu, c, 1);
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, c, 4 * i);
    }
};

// A thread's own ring in shared memory for chunks that cp.async brings: SLOTS
// slots of N chunks, so SLOTS - 1 rounds of loads are under way while one is
// used, without registers to hold them and without a barrier (a thread reads
// only what it copied).  `base`: BYTES_PER_THREAD times the block's threads, laid
// out so that neighbouring threads' 16-byte pieces lie side by side.
template <class T, int N, int SLOTS>
struct ThreadRing {
    static constexpr int PIECES = T::BYTES == 2 ? 1 : 2;  // of 16 bytes in a chunk
    static constexpr int BYTES_PER_THREAD = SLOTS * N * PIECES * 16;
    uint32_t first, end, stride, fill, use;  // shared addresses
    __device__ __forceinline__ explicit ThreadRing(const void* base) {
        stride = 16u * blockDim.x;
        first = fill = use = smem_u32(base) + 16u * threadIdx.x;
        end = first + (uint32_t)(SLOTS * N * PIECES) * stride;
    }
    // The chunk at `src` into place i of the slot being filled.
    __device__ __forceinline__ void fetch(int i, const void* src) const {
        // An fp32 chunk is two pieces, and a warp's copies of either reach half of
        // every 32-byte sector: through L1, so that the other half finds the
        // sector there (norms of 4096 x 2048 fp32 37 -> 28 us, gradients 60 -> 39).
        if constexpr (PIECES == 1) {
            cp_async16(fill + (uint32_t)i * stride, src);
        } else {
#pragma unroll
            for (int k = 0; k < PIECES; ++k)
                cp_async16_l1(fill + (uint32_t)(i * PIECES + k) * stride, static_cast<const unsigned char*>(src) + 16 * k);
        }
    }
    // Closes the slot, whether anything was fetched into it or not.
    __device__ __forceinline__ void commit() {
        cp_async_commit();
        fill += (uint32_t)(N * PIECES) * stride;
        if (fill == end) fill = first;
    }
    // With SLOTS - 1 newer slots closed: waits until the oldest has landed;
    // place i of it; gives it back.
    __device__ __forceinline__ void wait() const { cp_async_wait<SLOTS - 1>(); }
    __device__ __forceinline__ uint4 piece(int i) const {
        uint4 r;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(use + (uint32_t)i * stride) : "memory");
        return r;
    }
    __device__ __forceinline__ typename T::Raw get(int i) const {
        if constexpr (PIECES == 1) return piece(i);
        else return typename T::Raw{piece(2 * i), piece(2 * i + 1)};
    }
    __device__ __forceinline__ void next() {
        use += (uint32_t)(N * PIECES) * stride;
        if (use == end) use = first;
    }
};

}  // namespace moe
