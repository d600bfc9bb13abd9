// The C ABI of what surrounds the layer in a transformer block (include/moe.h): the RMS norm and its
// backward pass, and the gradient norm.  Argument checks, then the launches on the caller's stream.
#include <cmath>

#include "abi_checks.h"
#include "common.cuh"
#include "launch.h"

#define MOE_EXPORT __attribute__((visibility("default")))

using namespace moe;

namespace {

#define MOE_TRY(expr)                  \
    do {                               \
        moe_status_t _s = (expr);      \
        if (_s != MOE_OK) return _s;   \
    } while (0)
#define MOE_CUDA(expr)                                  \
    do {                                                \
        if ((expr) != cudaSuccess) return MOE_ERR_CUDA; \
    } while (0)

moe_status_t check_rows(int32_t dtype, int64_t rows, int32_t d) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || d < 1) return MOE_ERR_INVALID_ARG;
    if (rows >= (1LL << 31) || d > NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
    if (dtype == MOE_BF16 && d % 8) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(int32_t dtype, std::initializer_list<const void*> ptrs) {
    uintptr_t a = 0;
    for (const void* p : ptrs) a |= (uintptr_t)p;
    return a & (dtype == MOE_BF16 ? 15u : 3u);
}

}  // namespace

extern "C" {

MOE_EXPORT moe_status_t moe_rmsnorm(int32_t dtype, int64_t rows, int32_t d, const void* x, const void* residual,
                                    const void* weight, float eps, void* sum, void* y, int32_t fmt, uint8_t* codes,
                                    void* scales, float* rstd, moe_stream_t stream) {
    MOE_TRY(check_rows(dtype, rows, d));
    if (fmt != MOE_FMT_NATIVE && fmt != MOE_FMT_E4M3 && fmt != MOE_FMT_MXFP8) return MOE_ERR_INVALID_ARG;
    if (fmt != MOE_FMT_NATIVE && dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (!weight || (rows > 0 && (!x || !y))) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (residual != nullptr) != (sum != nullptr)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (fmt != MOE_FMT_NATIVE ? !codes || !scales : codes || scales)) return MOE_ERR_INVALID_ARG;
    if (misaligned(dtype, {x, residual, weight, sum, y}) || ((uintptr_t)codes & 15u) || ((uintptr_t)rstd & 3u) ||
        (fmt == MOE_FMT_E4M3 && ((uintptr_t)scales & 3u)))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    MOE_TRY(check_device());
    cudaGetLastError();
    MOE_CUDA(launch_rmsnorm(dtype == MOE_BF16, fmt, x, residual, weight, eps, rows, d, sum, y, codes, scales, rstd,
                            (cudaStream_t)stream));
    return MOE_OK;
}

MOE_EXPORT size_t moe_rmsnorm_backward_workspace_bytes(int32_t dtype, int64_t rows, int32_t d) {
    if (check_rows(dtype, rows, d) != MOE_OK) return 0;
    const size_t n = (size_t)norm_bwd_partials(rows) * d * sizeof(float);
    return n < 256 ? 256 : n;
}

MOE_EXPORT moe_status_t moe_rmsnorm_backward(int32_t dtype, int64_t rows, int32_t d, const void* dy, const void* s,
                                             const void* weight, const float* rstd, const void* dsum, void* dx,
                                             float* dweight, void* ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_TRY(check_rows(dtype, rows, d));
    if (!weight || !dweight || (rows > 0 && (!dy || !s || !rstd || !dx))) return MOE_ERR_INVALID_ARG;
    if (misaligned(dtype, {dy, s, weight, dsum, dx}) || (((uintptr_t)dweight | (uintptr_t)rstd) & 3u))
        return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < moe_rmsnorm_backward_workspace_bytes(dtype, rows, d) || ((uintptr_t)ws & 15u))
        return MOE_ERR_WORKSPACE;
    MOE_TRY(check_device());
    cudaGetLastError();
    if (rows == 0) {
        MOE_CUDA(cudaMemsetAsync(dweight, 0, (size_t)d * sizeof(float), (cudaStream_t)stream));
        return MOE_OK;
    }
    MOE_CUDA(launch_rmsnorm_bwd(dtype == MOE_BF16, dy, s, weight, rstd, dsum, rows, d, dx, dweight,
                                static_cast<float*>(ws), (cudaStream_t)stream));
    return MOE_OK;
}

MOE_EXPORT size_t moe_grad_workspace_bytes(void) { return grad_workspace_bytes(); }

static moe_status_t check_tensors(const moe_tensor_t* t, int32_t n) {
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].dtype != MOE_F32 && t[i].dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
        if (t[i].numel < 0 || (t[i].numel > 0 && !t[i].data)) return MOE_ERR_INVALID_ARG;
        if ((uintptr_t)t[i].data & (t[i].dtype == MOE_BF16 ? 1u : 3u)) return MOE_ERR_INVALID_ARG;
        if (t[i].numel >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

static moe_status_t grads_impl(const moe_tensor_t* grads, const moe_tensor_t* out, int32_t n, float max_norm, float* norm,
                               void* ws, size_t ws_bytes, cudaStream_t st) {
    if (n < 0 || (n > 0 && !grads) || !norm || ((uintptr_t)norm & 3u)) return MOE_ERR_INVALID_ARG;
    if (n > GRAD_MAX_TENSORS) return MOE_ERR_UNSUPPORTED;
    MOE_TRY(check_tensors(grads, n));
    if (out) {
        MOE_TRY(check_tensors(out, n));
        for (int32_t i = 0; i < n; ++i)
            if (out[i].numel != grads[i].numel || out[i].dtype != grads[i].dtype) return MOE_ERR_INVALID_ARG;
    }
    if (!ws || ws_bytes < grad_workspace_bytes() || ((uintptr_t)ws & 15u)) return MOE_ERR_WORKSPACE;
    MOE_TRY(check_device());
    cudaGetLastError();
    MOE_CUDA(launch_grad_norm(grads, out, n, max_norm, norm, ws, st));
    return MOE_OK;
}

MOE_EXPORT moe_status_t moe_grad_norm(const moe_tensor_t* grads, int32_t n, float* norm, void* ws, size_t ws_bytes,
                                      moe_stream_t stream) {
    return grads_impl(grads, nullptr, n, -1.f, norm, ws, ws_bytes, (cudaStream_t)stream);
}

MOE_EXPORT moe_status_t moe_clip_grads(const moe_tensor_t* grads, const moe_tensor_t* out, int32_t n, float max_norm,
                                       float* norm, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!(max_norm >= 0.f)) return MOE_ERR_INVALID_ARG;
    return grads_impl(grads, out, n, max_norm, norm, ws, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
