// What the two passes of the block norms share.
#pragma once

#include <type_traits>

#include "internal.h"
#include "vec8.cuh"

namespace moe {
namespace norm {

struct Args {
    int T, D, S;  // S = T / G rows share a gate row
    float alpha, eps;
    moe_dtype_t ptype;           // of the parameters and their gradients
    const void *gamma_post, *gate, *gamma_pre;
    const void *x, *y;           // backward: x is the stream after the block
    void *x_out, *h;             // forward
    const void *dx_out, *dh;     // backward
    void *dx, *dy;
    void *dgamma_post, *dgate, *dgamma_pre;
    int threads;                 // of a row group
    // backward
    int groups, rows;            // row groups of a block, consecutive rows of a row group
    int blocks;
    float* part;                 // [blocks][3][D]: gamma_post, gamma_pre, gate (G = 1)
    float* gate_part;            // [blocks * groups][2][D]: a group's first and last gate row (G > 1)
};

// The parameters' chunks of a thread's columns in fp32, side by side for
// neighbouring threads in shared memory: they would not stay in L1 beside the
// rings.  A: alpha gamma_post, and gate where all rows share it; B: gamma_pre.
struct ParamTable {
    uint32_t base, n16;  // shared address; 16 bytes times the chunks of a row group's threads
    __device__ __forceinline__ ParamTable(const float* b, int chunks) : base(smem_u32(b)), n16(16u * chunks) {}
    __device__ __forceinline__ static void st(uint32_t a, float2 u, float2 v) {
        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" :: "r"(a), "f"(u.x), "f"(u.y), "f"(v.x), "f"(v.y) : "memory");
    }
    __device__ __forceinline__ static void ld(uint32_t a, float2& u, float2& v) {
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(u.x), "=f"(u.y), "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    }
    __device__ __forceinline__ void put(int which, int c, const V8& v) const {
        const uint32_t a = base + 2 * which * n16 + 16u * c;
        st(a, v.p[0], v.p[1]);
        st(a + n16, v.p[2], v.p[3]);
    }
    __device__ __forceinline__ V8 get(int which, int c) const {
        const uint32_t a = base + 2 * which * n16 + 16u * c;
        V8 v;
        ld(a, v.p[0], v.p[1]);
        ld(a + n16, v.p[2], v.p[3]);
        return v;
    }
    // By every thread of the block, which then has to meet.
    __device__ __forceinline__ void fill(const Args& p) const {
        for (int c = threadIdx.x; c < p.D / 8; c += blockDim.x) {
            // all loads first: one latency, not three
            V8 b = v8(1.f);
            if (p.gamma_pre) b = load8(p.ptype, p.gamma_pre, c);
            fill_a(p, c, c, p.gate && p.S == p.T);
            put(1, c, b);
        }
    }
    // A of chunk c, with the gate's chunk g if there is one to be included.
    __device__ __forceinline__ void fill_a(const Args& p, int c, size_t g, bool gated) const {
        V8 a = v8(p.alpha), k = v8(1.f);
        if (p.gamma_post) a = load8(p.ptype, p.gamma_post, c);
        if (gated) k = load8(p.ptype, p.gate, g);
        if (p.gamma_post) a = mul(a, p.alpha);
        put(0, c, mul(a, k));
    }
    static constexpr size_t bytes(int chunks) { return (size_t)chunks * 64; }
};

__device__ __forceinline__ const unsigned char* at(const void* base, size_t off) {
    return static_cast<const unsigned char*>(base) + off;
}
// Chunk at byte offset `off`, as stored; and a chunk stored there.
template <class T>
__device__ __forceinline__ typename T::Raw raw_at(const void* base, size_t off) { return load_raw<T>(at(base, off), 0); }
template <class T>
__device__ __forceinline__ void store_at(void* base, size_t off, const V8& v) {
    store8<T>(static_cast<unsigned char*>(base) + off, 0, v);
}

// ------------------------------------------------------------------- host
// Chunks of 8 a thread: a row group has at most 512 threads.
inline int chunks_per_thread(int D) { return D <= 4096 ? 1 : D <= 8192 ? 2 : 4; }
inline int group_threads(int D, int vpt) { return ceil_div(ceil_div(D / 8, vpt), 32) * 32; }

constexpr size_t SMEM_BLOCK = 220 * 1024;  // shared memory that a block with rings may take

// Ring slots of `slot` bytes beside `other` bytes: what fits of 4, else 2, else none (1).
inline int ring_slots(size_t slot, size_t other) {
    const size_t n = other < SMEM_BLOCK ? (SMEM_BLOCK - other) / slot : 0;
    return n >= 4 ? 4 : n >= 2 ? 2 : 1;
}

// Calls f with the chunks a thread and the number of slots as constants.
template <int V, class F>
cudaError_t with_slots(int slots, F f) {
    using std::integral_constant;
    if (slots == 4) return f(integral_constant<int, V>{}, integral_constant<int, 4>{});
    if (slots == 2) return f(integral_constant<int, V>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, V>{}, integral_constant<int, 1>{});
}
template <class F>
cudaError_t with_shape(int vpt, int slots, F f) {
    if (vpt == 1) return with_slots<1>(slots, f);
    if (vpt == 2) return with_slots<2>(slots, f);
    return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
}

inline Args common_args(const NormShape& n) {
    Args a{};
    a.T = n.T;
    a.D = n.D;
    a.S = n.T / n.G;
    a.alpha = n.alpha;
    a.eps = n.eps;
    a.ptype = n.param_dtype;
    a.gamma_post = n.gamma_post;
    a.gate = n.gate;
    a.gamma_pre = n.gamma_pre;
    return a;
}

}  // namespace norm
}  // namespace moe
