// C ABI of the 16-bit expert operators (grouped products, gated activation,
// block norms) declared in include/moe_w4.h: argument checks and workspaces.
#include <climits>
#include <cmath>

#include "internal.h"
#include "moe_w4.h"

using namespace moe;

namespace {

constexpr int MAX_WIDTH = 32768;  // N, K, F of the expert operators
constexpr int MAX_NORM_WIDTH = 16384;
// Rows: the kernels step through them in 32 bits, by at most a few tens of thousands
// beyond the last (a block norm's row groups by T / 152).
constexpr int MAX_ROWS = INT32_MAX - (1 << 24);

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <size_t N>
bool all_aligned(const void* const (&ps)[N]) {
    for (const void* p : ps)
        if (!aligned16(p)) return false;
    return true;
}
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool grouped_sizes_ok(int32_t R, int32_t E, int32_t N, int32_t K) {
    return R >= 0 && E >= 1 && E <= 1024 && N >= 1 && K >= 1;
}
bool width_supported(int32_t w, int32_t most) { return w % 8 == 0 && w <= most; }

size_t with_header(size_t floats) { return WS_HEADER + floats * sizeof(float); }

// The checks that the three products share; MOE_OK, or the status to return.
// Without rows the operands may be null, and y and dx too.  `floats`: what the
// product itself needs, which may be less than the size that callers are told.
moe_status_t check_grouped(size_t (*floats)(const GroupedShape&), moe_dtype_t dtype, const void* a, const void* b, const int32_t* offsets, int32_t R, int32_t E,
                           int32_t N, int32_t K, bool needs_out, const void* out, const void* ws, size_t ws_bytes) {
    if (!grouped_sizes_ok(R, E, N, K)) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
    if (R > MAX_ROWS || !width_supported(N, MAX_WIDTH) || !width_supported(K, MAX_WIDTH)) return MOE_ERR_UNSUPPORTED;
    if (!offsets || !ws || (R > 0 && (!a || !b)) || (needs_out && !out)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({a, b, offsets, out, ws})) return MOE_ERR_MISALIGNED;
    return ws_bytes < with_header(floats(GroupedShape{dtype, R, E, N, K})) ? MOE_ERR_WORKSPACE : MOE_OK;
}

GroupedShape shape(moe_dtype_t dtype, const int32_t* offsets, int32_t R, int32_t E, int32_t N, int32_t K, void* ws) {
    return GroupedShape{dtype, R, E, N, K, offsets, &static_cast<WsHeader*>(ws)->err,
                        reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + WS_HEADER)};
}

moe_status_t check_swiglu(moe_dtype_t dtype, int32_t R, int32_t F) {
    if (R < 0 || F < 1) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16 && dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    return R <= MAX_ROWS && width_supported(F, MAX_WIDTH) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status_t check_norm(const NormShape& n, const void* y) {
    if (n.T < 0 || n.D < 1 || n.G < 1) return MOE_ERR_INVALID_ARG;
    if (n.T % n.G) return MOE_ERR_INVALID_ARG;
    if (!(n.eps > 0.f) || !std::isfinite(n.eps) || !std::isfinite(n.alpha)) return MOE_ERR_INVALID_ARG;
    if (n.dtype != MOE_DT_BF16 && n.dtype != MOE_DT_F16 && n.dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if (n.param_dtype != n.dtype && n.param_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if (n.T > MAX_ROWS || !width_supported(n.D, MAX_NORM_WIDTH)) return MOE_ERR_UNSUPPORTED;
    if (n.T > 0 && !y && (n.gamma_post || n.gate)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_grouped_mm_workspace_size(int32_t R, int32_t E, int32_t N, int32_t K) {
    if (!grouped_sizes_ok(R, E, N, K)) return 0;
    return with_header(grouped_floats_bound(GroupedShape{MOE_DT_BF16, R, E, N, K}));
}

moe_status_t moe_grouped_mm(moe_dtype_t dtype, const void* x, const void* w, const int32_t* offsets, int32_t R, int32_t E,
                            int32_t N, int32_t K, void* y, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    const moe_status_t st = check_grouped(grouped_floats, dtype, x, w, offsets, R, E, N, K, R > 0, y, workspace, workspace_bytes);
    if (st != MOE_OK || R == 0) return st;
    return cuda_status(launch_grouped_mm(shape(dtype, offsets, R, E, N, K, workspace), x, w, y, stream));
}

moe_status_t moe_grouped_mm_dx(moe_dtype_t dtype, const void* dy, const void* w, const int32_t* offsets, int32_t R,
                               int32_t E, int32_t N, int32_t K, void* dx, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
    const moe_status_t st = check_grouped(grouped_dx_floats, dtype, dy, w, offsets, R, E, N, K, R > 0, dx, workspace, workspace_bytes);
    if (st != MOE_OK || R == 0) return st;
    return cuda_status(launch_grouped_mm_dx(shape(dtype, offsets, R, E, N, K, workspace), dy, w, dx, stream));
}

moe_status_t moe_grouped_mm_dw(moe_dtype_t dtype, const void* dy, const void* x, const int32_t* offsets, int32_t R,
                               int32_t E, int32_t N, int32_t K, void* dw, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
    const moe_status_t st = check_grouped(grouped_dw_floats, dtype, dy, x, offsets, R, E, N, K, true, dw, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    return cuda_status(launch_grouped_mm_dw(shape(dtype, offsets, R, E, N, K, workspace), dy, x, dw, stream));
}

moe_status_t moe_swiglu(moe_dtype_t dtype, const void* gu, const float* row_w, const int32_t* row_map, int32_t R,
                        int32_t F, void* h, cudaStream_t stream) {
    const moe_status_t st = check_swiglu(dtype, R, F);
    if (st != MOE_OK || R == 0) return st;
    if (!gu || !h || (row_map && !row_w)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({gu, row_w, row_map, h})) return MOE_ERR_MISALIGNED;
    return cuda_status(launch_swiglu(dtype, gu, row_w, row_map, R, F, h, stream));
}

moe_status_t moe_swiglu_backward(moe_dtype_t dtype, const void* dh, const void* gu, const float* row_w,
                                 const int32_t* row_map, int32_t R, int32_t F, void* dgu, float* drow_w,
                                 cudaStream_t stream) {
    const moe_status_t st = check_swiglu(dtype, R, F);
    if (st != MOE_OK || R == 0) return st;
    if (!dh || !gu || !dgu || (row_map && !row_w) || (drow_w && !row_w)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({dh, gu, row_w, row_map, dgu, drow_w})) return MOE_ERR_MISALIGNED;
    return cuda_status(launch_swiglu_backward(dtype, dh, gu, row_w, row_map, R, F, dgu, drow_w, stream));
}

moe_status_t moe_block_norm(moe_dtype_t dtype, moe_dtype_t param_dtype, int32_t T, int32_t D, int32_t G, float alpha,
                            float eps, const void* gamma_post, const void* gate, const void* gamma_pre, const void* x,
                            const void* y, void* x_out, void* h, cudaStream_t stream) {
    const NormShape n{dtype, param_dtype, T, D, G, alpha, eps, gamma_post, gate, gamma_pre};
    const moe_status_t st = check_norm(n, y);
    if (st != MOE_OK || T == 0) return st;
    // the stream after the block comes with y, h with gamma_pre, and there is something to write
    if (!x || !y != !x_out || !gamma_pre != !h || (!y && !h)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({gamma_post, gate, gamma_pre, x, y, x_out, h})) return MOE_ERR_MISALIGNED;
    return cuda_status(launch_block_norm(n, x, y, x_out, h, stream));
}

size_t moe_block_norm_backward_workspace_size(int32_t T, int32_t D, int32_t G) {
    if (T < 0 || D < 1 || G < 1 || T % G) return 0;
    return with_header(block_norm_partial_floats(T, D, G));
}

moe_status_t moe_block_norm_backward(moe_dtype_t dtype, moe_dtype_t param_dtype, int32_t T, int32_t D, int32_t G,
                                     float alpha, float eps, const void* gamma_post, const void* gate,
                                     const void* gamma_pre, const void* x_out, const void* y, const void* dx_out,
                                     const void* dh, void* dx, void* dy, void* dgamma_post, void* dgate,
                                     void* dgamma_pre, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    const NormShape n{dtype, param_dtype, T, D, G, alpha, eps, gamma_post, gate, gamma_pre};
    const moe_status_t st = check_norm(n, y);
    if (st != MOE_OK) return st;
    // a gradient has its parameter
    if ((dgamma_post && !gamma_post) || (dgate && !gate) || (dgamma_pre && !gamma_pre)) return MOE_ERR_INVALID_ARG;
    if (T == 0) {  // sums over no rows
        const size_t row = (size_t)D * (param_dtype == MOE_DT_F32 ? 4 : 2);
        cudaError_t e = cudaSuccess;
        if (dgamma_post) e = cudaMemsetAsync(dgamma_post, 0, row, stream);
        if (dgate && e == cudaSuccess) e = cudaMemsetAsync(dgate, 0, row * G, stream);
        if (dgamma_pre && e == cudaSuccess) e = cudaMemsetAsync(dgamma_pre, 0, row, stream);
        return cuda_status(e);
    }
    if (!dx || (!dx_out && !dh) || !y != !dy || !gamma_pre != !dh) return MOE_ERR_INVALID_ARG;
    if ((dh && !x_out) || !workspace) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({gamma_post, gate, gamma_pre, x_out, y, dx_out, dh, dx, dy, dgamma_post, dgate, dgamma_pre, workspace}))
        return MOE_ERR_MISALIGNED;
    if (workspace_bytes < moe_block_norm_backward_workspace_size(T, D, G)) return MOE_ERR_WORKSPACE;
    float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + WS_HEADER);
    const NormGrads g{x_out, y, dx_out, dh, dx, dy, dgamma_post, dgate, dgamma_pre};
    return cuda_status(launch_block_norm_backward(n, g, part, stream));
}

}  // extern "C"
