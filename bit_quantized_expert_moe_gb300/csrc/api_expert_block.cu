// C ABI of the operators of expert blocks in 8 and 16 bits (layer norm, quantisation of
// rows, 8-bit grouped products, the 16-bit layer for a few tokens) declared in include/moe_w4.h: argument checks and
// workspaces.
#include <climits>
#include <cmath>

#include "internal.h"
#include "moe_w4.h"

using namespace moe;

namespace {

constexpr int MAX_WIDTH = 32768;
constexpr int MAX_NORM_WIDTH = 16384;
constexpr int MAX_ROWS = INT32_MAX - (1 << 24);  // as the 16-bit expert operators'

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <size_t N>
bool all_aligned(const void* const (&ps)[N]) {
    for (const void* p : ps)
        if (!aligned16(p)) return false;
    return true;
}
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool width_supported(int32_t w, int32_t unit, int32_t most) { return w % unit == 0 && w <= most; }
bool row_type(moe_dtype_t t) { return t == MOE_DT_BF16 || t == MOE_DT_F16 || t == MOE_DT_F32; }

moe_status_t check_norm(const LayerNormShape& n) {
    if (n.T < 0 || n.D < 1 || !(n.eps > 0.f) || !std::isfinite(n.eps)) return MOE_ERR_INVALID_ARG;
    if (!row_type(n.dtype) || (n.param_dtype != n.dtype && n.param_dtype != MOE_DT_F32)) return MOE_ERR_UNSUPPORTED;
    return n.T <= MAX_ROWS && width_supported(n.D, 8, MAX_NORM_WIDTH) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

bool grouped_sizes_ok(int32_t R, int32_t E, int32_t N, int32_t K) {
    return R >= 0 && E >= 1 && E <= 1024 && N >= 1 && K >= 1;
}

bool layer_sizes_ok(int32_t T, int32_t k, int32_t E, int32_t d, int32_t f) {
    return T >= 0 && k >= 1 && E >= 1 && E <= 1024 && k <= E && d >= 1 && f >= 1;
}
bool layer_supported(int32_t T, int32_t k, int32_t d, int32_t f) {
    return expert_layer_supported(T, k) && width_supported(d, 64, MAX_WIDTH) && width_supported(f, 64, MAX_WIDTH);
}

}  // namespace

extern "C" {

moe_status_t moe_layer_norm(moe_dtype_t dtype, moe_dtype_t param_dtype, int32_t T, int32_t D, float eps, const void* gamma,
                            const void* beta, const void* x, const void* y, void* x_out, void* h, cudaStream_t stream) {
    const LayerNormShape n{dtype, param_dtype, T, D, eps, gamma, beta};
    const moe_status_t st = check_norm(n);
    if (st != MOE_OK || T == 0) return st;
    if (!x || !h || !y != !x_out) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({gamma, beta, x, y, x_out, h})) return MOE_ERR_MISALIGNED;
    return cuda_status(launch_layer_norm(n, x, y, x_out, h, stream));
}

size_t moe_layer_norm_backward_workspace_size(int32_t T, int32_t D) {
    if (T < 0 || D < 1) return 0;
    return WS_HEADER + layer_norm_partial_floats(T, D) * sizeof(float);
}

moe_status_t moe_layer_norm_backward(moe_dtype_t dtype, moe_dtype_t param_dtype, int32_t T, int32_t D, float eps,
                                     const void* gamma, const void* x_out, const void* dh, const void* dx_out, void* dx,
                                     void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
    const LayerNormShape n{dtype, param_dtype, T, D, eps, gamma, nullptr};
    const moe_status_t st = check_norm(n);
    if (st != MOE_OK) return st;
    if (dgamma && !gamma) return MOE_ERR_INVALID_ARG;
    if (T == 0) {  // sums over no rows
        const size_t row = (size_t)D * (param_dtype == MOE_DT_F32 ? 4 : 2);
        cudaError_t e = cudaSuccess;
        if (dgamma) e = cudaMemsetAsync(dgamma, 0, row, stream);
        if (dbeta && e == cudaSuccess) e = cudaMemsetAsync(dbeta, 0, row, stream);
        return cuda_status(e);
    }
    if (!x_out || !dh || !dx || !workspace) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({gamma, x_out, dh, dx_out, dx, dgamma, dbeta, workspace})) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < moe_layer_norm_backward_workspace_size(T, D)) return MOE_ERR_WORKSPACE;
    float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + WS_HEADER);
    return cuda_status(launch_layer_norm_backward(n, LayerNormGrads{x_out, dh, dx_out, dx, dgamma, dbeta}, part, stream));
}

size_t moe_quantize_rows_workspace_size(int32_t T, int32_t R, int32_t D) {
    if (T < 1 || R < 0 || T > MAX_ROWS || R > MAX_ROWS || !width_supported(D, 16, MAX_WIDTH)) return 0;
    const size_t bytes = quantize_rows_bytes(T, R, D);
    return bytes ? WS_HEADER + bytes : 0;
}

moe_status_t moe_quantize_rows(moe_dtype_t dtype, const void* x, const int32_t* row_map, int32_t k, int32_t T, int32_t R,
                               int32_t D, int8_t* codes, float* scales, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
    if (T < 0 || R < 0 || D < 1 || k < 1 || (!row_map && R != T && R > 0)) return MOE_ERR_INVALID_ARG;
    if (!row_type(dtype) || T > MAX_ROWS || R > MAX_ROWS || !width_supported(D, 16, MAX_WIDTH)) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if ((T > 0 && !x) || !codes || !scales) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({x, row_map, codes, scales, workspace})) return MOE_ERR_MISALIGNED;
    if (workspace && workspace_bytes < moe_quantize_rows_workspace_size(T, R, D)) return MOE_ERR_WORKSPACE;
    // the header stays as it is: a workspace that other calls use has its error word and counters there
    void* const space = workspace ? static_cast<unsigned char*>(workspace) + WS_HEADER : nullptr;
    return cuda_status(launch_quantize_rows(dtype, x, row_map, k, T, R, D, codes, scales, space, stream));
}

size_t moe_grouped_mm_i8_workspace_size(int32_t R, int32_t E, int32_t N, int32_t K) {
    if (!grouped_sizes_ok(R, E, N, K)) return 0;
    return WS_HEADER + 2 * grouped_i8_halves(R, E, N, K);
}

moe_status_t moe_grouped_mm_i8(moe_dtype_t out_dtype, const int8_t* x, const float* x_scale, const int8_t* w,
                               const float* w_scale, const int32_t* offsets, int32_t R, int32_t E, int32_t N, int32_t K,
                               void* y, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!grouped_sizes_ok(R, E, N, K)) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
    if (R > MAX_ROWS || !width_supported(N, 8, MAX_WIDTH) || !width_supported(K, 16, MAX_WIDTH)) return MOE_ERR_UNSUPPORTED;
    if (!offsets || !workspace || (R > 0 && (!x || !x_scale || !w || !w_scale || !y))) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({x, x_scale, w, w_scale, offsets, y, workspace})) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < moe_grouped_mm_i8_workspace_size(R, E, N, K)) return MOE_ERR_WORKSPACE;
    if (R == 0) return MOE_OK;
    auto* ws = static_cast<unsigned char*>(workspace);
    const GroupedI8Shape g{out_dtype, R, E, N, K, offsets, &static_cast<WsHeader*>(workspace)->err,
                           reinterpret_cast<uint16_t*>(ws + WS_HEADER)};
    return cuda_status(launch_grouped_i8(g, GroupedI8Data{x, w, x_scale, w_scale, y}, stream));
}

size_t moe_expert_layer_workspace_size(int32_t T, int32_t k, int32_t E, int32_t d_model, int32_t d_ff) {
    if (!layer_sizes_ok(T, k, E, d_model, d_ff) || !layer_supported(T, k, d_model, d_ff)) return 0;
    return WS_HEADER + expert_layer_bytes(T, k, d_model, d_ff);
}

moe_status_t moe_expert_layer(moe_dtype_t dtype, const void* x, const float* logits, const void* w13, const void* w2,
                              int32_t T, int32_t k, int32_t E, int32_t d_model, int32_t d_ff, void* out,
                              int32_t* topk_ids_out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!layer_sizes_ok(T, k, E, d_model, d_ff)) return MOE_ERR_INVALID_ARG;
    if ((dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) || !layer_supported(T, k, d_model, d_ff)) return MOE_ERR_UNSUPPORTED;
    if (!workspace || (T > 0 && (!x || !logits || !w13 || !w2 || !out))) return MOE_ERR_INVALID_ARG;
    if (!all_aligned({x, logits, w13, w2, out, topk_ids_out, workspace})) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < moe_expert_layer_workspace_size(T, k, E, d_model, d_ff)) return MOE_ERR_WORKSPACE;
    if (T == 0) return MOE_OK;
    auto* ws = static_cast<unsigned char*>(workspace);
    return cuda_status(launch_expert_layer(ExpertLayer{dtype, x, logits, w13, w2, T, k, E, d_model, d_ff, out, topk_ids_out,
                                                       reinterpret_cast<uint32_t*>(ws), ws + WS_HEADER},
                                           stream));
}

}  // extern "C"
