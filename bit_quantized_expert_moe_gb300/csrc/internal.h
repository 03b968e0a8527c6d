// Internal declarations shared by the library's translation units.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace moe {

// ---------------------------------------------------------------- routing
cudaError_t launch_route_topk(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                              cudaStream_t s);

// ------------------------------------------------------------ permutation
// Token tiles of the grouped tensor-core GEMM: one entry per (expert, <=256 rows).
constexpr int TILE_ROWS = 256;
struct Tile {
    int32_t expert;
    int32_t row0;    // first permuted row
    int32_t nrows;   // 1..TILE_ROWS
    int32_t pad;
};

struct AlignOut {
    int32_t* counts;    // [E]
    int32_t* offsets;   // [E+1]
    int32_t* sorted;    // [R]
    int32_t* inv;       // [R]
    int32_t* uniq;      // [E]  experts with rows, ascending
    Tile* tiles;        // [R/TILE_ROWS + E]
    DevPlan* plan;      // n_uniq, n_tiles
    uint16_t* x_perm;   // [R][d] or null
    int x_perm_f16;     // 1: write x_perm as fp16 in the tensor-core operand order (K interleaved
                        //    in groups of 8, k8_interleave); values outside fp16 set the error word
    int32_t* blockcnt;  // [nblocks][E] scratch for the multi-block path
    uint32_t* err;
};
constexpr int ALIGN_SMALL_MAX_R = 2048;   // single-CTA permutation up to this many rows
constexpr int ALIGN_BLOCK_ROWS = 1024;    // most assignments per CTA on the multi-block path
// Assignments per CTA on the multi-block path: the smallest of 32, 64 and 256
// (more CTAs for the stable placement and the row copy) whose per-block count
// table stays within 64 KB, else 1024.
int align_block_rows(int R, int E);
size_t align_blockcnt_bytes(int R, int E);
cudaError_t launch_align(const int32_t* ids, int T, int k, int E, const uint16_t* x, int d,
                         const AlignOut& o, cudaStream_t s);
// uniq list + tile list from an offsets array already on the device.
// bf16 -> fp16 copy of n elements (n % 8 == 0); out-of-range values set the error word.
// bf16 rows -> fp16 in the tensor-core operand order (K interleaved in groups of 8)
cudaError_t launch_bf16_to_f16(const uint16_t* in, uint16_t* out, size_t n, uint32_t* err, cudaStream_t s);
cudaError_t launch_plan_from_offsets(const int32_t* offsets, int E, int32_t* uniq, Tile* tiles,
                                     DevPlan* plan, cudaStream_t s);

// ---------------------------------------------------------------- combine
// y_perm is bf16 (y_f16 = false) or fp16 (y_f16 = true).
cudaError_t launch_combine(const uint16_t* y_perm, bool y_f16, const int32_t* inv, const float* w, int T, int k,
                           int d, uint16_t* out, cudaStream_t s);

// ------------------------------------------------- decode regime (GEMV)
struct GemvShape {
    int E, d, f;
    int R;          // rows (assignments) in the permuted order
    int max_uniq;   // upper bound on experts with rows: min(R, E)
};
struct GemvIn {
    const uint32_t *w13_q, *w2_q;
    const uint16_t *w13_s, *w13_z, *w2_s, *w2_z;
    const int32_t* offsets;
    const int32_t* uniq;
    const DevPlan* plan;
    const int32_t* sorted;   // gate_up input row i = x[sorted[i] / k] when non-null, else x[i]
    int k;
    const uint16_t* x;       // bf16 [*][d]
    float* h;                // fp32 [R][f] (written by gate_up, read by down)
    // down outputs: exactly one of (y_perm) or (out with topk_w, inv, T)
    uint16_t* y_perm;        // bf16 [R][d]
    const float* row_w;      // optional row scale for y_perm
    uint16_t* out;           // bf16 [T][d]: fused combine
    const float* topk_w;
    const int32_t* inv;
    int T;
    uint32_t* err;
};
bool gemv_supported(const GemvShape& sh, int T_tokens);
cudaError_t launch_gemv_gateup(const GemvShape& sh, const GemvIn& in, cudaStream_t s);
cudaError_t launch_gemv_down(const GemvShape& sh, const GemvIn& in, cudaStream_t s);

// ------------------------- decode regime: the whole layer in one kernel
// Routing, gate_up, down and combine of T <= 8 tokens in one cooperative
// persistent launch (decode_fused.cu).
struct FusedIn {
    const moe_w4_layer* L;
    const uint16_t* x;       // bf16 [T][d]
    const float* logits;     // fp32 [T][E]
    int T, k;
    uint16_t* out;           // bf16 [T][d]
    int32_t* ids_out;        // [T][k] or null
    uint16_t* hb;            // fp16 scratch, [T*k][f]
    void* ws;                // workspace (header: error word and the kernels' counters)
};
bool decode_fused_supported(int T, int k, int E, int d, int f);
cudaError_t launch_decode_fused(const FusedIn& in, cudaStream_t s);

// ---------------------------------------------- prefill regime (tcgen05)
struct TcIn {
    const uint32_t *w13_q, *w2_q;
    const uint16_t *w13_s, *w13_z, *w2_s, *w2_z;
    const Tile* tiles;
    const DevPlan* plan;
    const uint16_t* x16;     // fp16 [R][d]: permuted activations
    uint16_t* h16;           // fp16 [R][f]
    uint16_t* y_out;         // [R][d], fp16 if y_f16 else bf16
    int y_f16;
    const float* row_w;      // optional
    uint32_t* err;
};
bool tc_supported(int E, int d, int f);
int tc_max_tiles(int R, int E);
cudaError_t launch_tc_gateup(int E, int d, int f, int R, const TcIn& in, cudaStream_t s);
cudaError_t launch_tc_down(int E, int d, int f, int R, const TcIn& in, cudaStream_t s);

// ------------------------------------------- 16-bit expert operators
struct GroupedShape {
    moe_dtype_t dtype;       // bf16 or fp16
    int R, E, N, K;
    const int32_t* offsets;  // [E+1]
    uint32_t* err;
    float* part;             // values of the functions below
};
// What y, dx or dw puts down before its output, for the sizes alone; and what no
// product exceeds for these sizes or any smaller number of rows.
size_t grouped_floats(const GroupedShape& g);
size_t grouped_dx_floats(const GroupedShape& g);
size_t grouped_dw_floats(const GroupedShape& g);
size_t grouped_floats_bound(const GroupedShape& g);
// y = x W_e^T, dx = dy W_e, dW_e = dy_e^T x_e over the segments of `offsets`.
cudaError_t launch_grouped_mm(const GroupedShape& g, const void* x, const void* w, void* y, cudaStream_t s);
cudaError_t launch_grouped_mm_dx(const GroupedShape& g, const void* dy, const void* w, void* dx, cudaStream_t s);
cudaError_t launch_grouped_mm_dw(const GroupedShape& g, const void* dy, const void* x, void* dw, cudaStream_t s);

// The same as launch_grouped_mm by another kernel, for few rows in all.
cudaError_t launch_grouped_few(const GroupedShape& g, const void* x, const void* w, void* y, cudaStream_t s);

cudaError_t launch_swiglu(moe_dtype_t dt, const void* gu, const float* row_w, const int32_t* row_map, int R, int F,
                          void* h, cudaStream_t s);
cudaError_t launch_swiglu_backward(moe_dtype_t dt, const void* dh, const void* gu, const float* row_w,
                                   const int32_t* row_map, int R, int F, void* dgu, float* drow_w, cudaStream_t s);

struct NormShape {
    moe_dtype_t dtype, param_dtype;
    int T, D, G;
    float alpha, eps;
    const void *gamma_post, *gate, *gamma_pre;  // any may be null
};
struct NormGrads {
    const void *x_out, *y, *dx_out, *dh;
    void *dx, *dy, *dgamma_post, *dgate, *dgamma_pre;
};
size_t block_norm_partial_floats(int T, int D, int G);  // scratch of the backward pass
cudaError_t launch_block_norm(const NormShape& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s);
cudaError_t launch_block_norm_backward(const NormShape& n, const NormGrads& g, float* part, cudaStream_t s);

// ------------------------------------ expert blocks in 8 and 16 bits
struct LayerNormShape {
    moe_dtype_t dtype, param_dtype;
    int T, D;
    float eps;
    const void *gamma, *beta;  // either may be null
};
struct LayerNormGrads {
    const void *x_out, *dh, *dx_out;
    void *dx, *dgamma, *dbeta;
};
size_t layer_norm_partial_floats(int T, int D);  // scratch of the backward pass
cudaError_t launch_layer_norm(const LayerNormShape& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const LayerNormShape& n, const LayerNormGrads& g, float* part, cudaStream_t s);

// Rows x[row_map[r] / k] (x[r] without a map) as 8-bit codes and scales.  `ws`: as many bytes
// as quantize_rows_bytes(), behind the workspace's header, or null.
size_t quantize_rows_bytes(int T, int R, int D);
cudaError_t launch_quantize_rows(moe_dtype_t dt, const void* x, const int32_t* row_map, int k, int T, int R, int D,
                                 int8_t* codes, float* scales, void* ws, cudaStream_t s);

struct GroupedI8Shape {
    moe_dtype_t out;         // bf16 or fp16
    int R, E, N, K;
    const int32_t* offsets;  // [E+1]
    uint32_t* err;
    uint16_t* x16;           // the codes of x as fp16, where the tensor-core kernel runs
};
struct GroupedI8Data {
    const int8_t *x, *w;
    const float *x_scale, *w_scale;
    void* y;
};
size_t grouped_i8_halves(int R, int E, int N, int K);  // of x16, for R rows or fewer
cudaError_t launch_grouped_i8(const GroupedI8Shape& g, const GroupedI8Data& d, cudaStream_t s);
// The same by another kernel, for few rows in all.
cudaError_t launch_grouped_i8_few(const GroupedI8Shape& g, const GroupedI8Data& d, cudaStream_t s);

// The whole layer of 16-bit experts for a few tokens.
struct ExpertLayer {
    moe_dtype_t dtype;       // bf16 or fp16
    const void* x;           // [T][d]
    const float* logits;     // [T][E]
    const void *w13, *w2;    // [E][2f][d], [E][d][f]
    int T, k, E, d, f;
    void* out;               // [T][d]
    int32_t* ids_out;        // [T][k] or null
    uint32_t* header;        // of the workspace
    uint8_t* h;              // expert_layer_bytes() behind it
};
bool expert_layer_supported(int T, int k);
size_t expert_layer_bytes(int T, int k, int d, int f);
cudaError_t launch_expert_layer(const ExpertLayer& l, cudaStream_t s);

// 3D tensor map over 32-bit words: dims {d0, d1, d2} (d0 contiguous), byte
// strides s1 (dim 1) and s2 (dim 2), box {b0, b1, b2}, 128-byte swizzle.
bool make_tensor_map_3d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                        uint64_t s2, uint32_t b0, uint32_t b1, uint32_t b2);
// Tensor map of rank 1..5 over 32-bit words: dims[0] contiguous, strides[i]
// the byte stride of dimension i + 1, box per dimension, 128-byte swizzle.
bool make_tensor_map_u32(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                         const uint32_t* box);
// The same over 16-bit elements, without swizzle.
bool make_tensor_map_u16(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                         const uint32_t* box);
// The same over bf16 or fp16 elements, 128-byte swizzle, zeros out of bounds.
bool make_tensor_map_16(CUtensorMap* m, bool bf16, const void* ptr, int rank, const uint64_t* dims,
                        const uint64_t* strides, const uint32_t* box);

// The same over bytes.
bool make_tensor_map_8(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                       const uint32_t* box);

// ----------------------------------------------------------- device info
int num_sms();  // of the current device
// Counts one kernel launch of this library (reported by moe_kernel_launches).
void note_launch(int n = 1);
// Lets a kernel without static shared memory take all of an SM's as dynamic
// shared memory, once for each device.
constexpr int SMEM_MOST = 232448;
template <auto Kernel>
cudaError_t allow_smem() {
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && allowed[dev].load(std::memory_order_relaxed))) return e;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST);
    if (e == cudaSuccess && dev < 64) allowed[dev].store(true, std::memory_order_relaxed);
    return e;
}
// Launches a kernel that waits for the one before it in the stream with
// grid_dependency_wait(), and may start before that one has ended.
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) note_launch();
    return e;
}
// The same for a kernel that may need more than the default 48 KB.
template <auto Kernel, class... A>
cudaError_t launch_overlapped(dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
    const cudaError_t e = smem > 48 * 1024 ? allow_smem<Kernel>() : cudaSuccess;
    return e == cudaSuccess ? launch_overlapped(Kernel, grid, block, smem, s, args...) : e;
}

}  // namespace moe
