// ffn_abi.cu -- the C ABI of the feed-forward operators (include/fp8q_ffn.h):
// argument checks, then the launches.  Nothing here allocates, synchronizes or
// keeps state.

#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "abi_checks.h"
#include "fp8q_ffn.h"
#include "fp8q_launch.h"
#include "gemm_gated.h"
#include "rmsnorm.h"

using namespace fp8q_abi;

extern "C" {

int fp8q_rmsnorm_quantize(const void* x, int dtype, const void* residual, const void* weight, int w_dtype, int64_t rows,
                          int64_t cols, float eps, int fmt, uint8_t* q, float* scales, void* h, void* y, float* rstd,
                          void* stream) {
    if (!fmt_ok(fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(dtype) || !dtype_ok(w_dtype)) return FP8_ERR_DTYPE;
    if (!size_ok(rows, cols)) return FP8_ERR_SHAPE;
    if (!(eps > 0.0f) || std::isinf(eps)) return FP8_ERR_ARG;
    if (rows == 0 || cols == 0) return FP8_OK;
    if (x == nullptr || weight == nullptr || q == nullptr || scales == nullptr) return FP8_ERR_NULL;
    if (residual != nullptr && h == nullptr) return FP8_ERR_NULL;
    if (residual == nullptr) h = nullptr;  // not written
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(q, 16) || !aligned(h, 16) ||
        !aligned(y, 16) || !aligned(scales, 4) || !aligned(rstd, 4))
        return FP8_ERR_ALIGN;
    const int64_t n = rows * cols, bytes = n * esize(dtype);
    const Range rx{x, bytes}, rr{residual, bytes}, rw{weight, cols * esize(w_dtype)}, rh{h, bytes};
    if ((h != x && overlap(rh, rx)) || (h != residual && overlap(rh, rr)) || overlap(rh, rw)) return FP8_ERR_ARG;
    if (any_overlap({{q, n}, {scales, rows * ((cols + 127) / 128) * 4}, {y, bytes}, {rstd, rows * 4}}, {rx, rr, rw, rh}))
        return FP8_ERR_ARG;
    const fp8q::RmsNormArgs a{x, residual, weight, w_dtype == FP8_BF16, rows, cols, eps, q, scales, h, y, rstd};
    return status_of(fp8q::launch_rmsnorm_quantize(a, dtype, fmt, static_cast<cudaStream_t>(stream)));
}

int64_t fp8q_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
    if (!size_ok(rows, cols)) return FP8_ERR_SHAPE;
    return fp8q::rmsnorm_backward_one_launch(rows, cols) ? 0 : fp8q::rmsnorm_backward_partials(rows) * cols * 4;
}

int fp8q_rmsnorm_backward(const void* dy, const void* h, int dtype, const float* rstd, const void* weight, int w_dtype,
                          const void* dh, int64_t rows, int64_t cols, void* dx, float* dweight, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype) || !dtype_ok(w_dtype)) return FP8_ERR_DTYPE;
    if (!size_ok(rows, cols)) return FP8_ERR_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cols == 0) return FP8_OK;
    if (!aligned(dweight, 4)) return FP8_ERR_ALIGN;
    if (rows == 0)
        return dweight == nullptr ? FP8_OK : status_of(cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols) * 4, st));
    if (dy == nullptr || h == nullptr || rstd == nullptr || weight == nullptr || dx == nullptr) return FP8_ERR_NULL;
    const int64_t need = fp8q_rmsnorm_backward_workspace(rows, cols);
    if (dweight != nullptr && need > 0 && workspace == nullptr) return FP8_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(dh, 16) || !aligned(dx, 16) ||
        !aligned(rstd, 4) || !aligned(workspace, 16))
        return FP8_ERR_ALIGN;
    if (dweight != nullptr && workspace_bytes < need) return FP8_ERR_ARG;
    const int64_t bytes = rows * cols * esize(dtype);
    const Range ry{dy, bytes}, rg{dh, bytes}, rx{dx, bytes}, rh{h, bytes}, rr{rstd, rows * 4},
        rw{weight, cols * esize(w_dtype)};
    if ((dx != dy && overlap(rx, ry)) || (dx != dh && overlap(rx, rg)) || any_overlap({rx}, {rh, rr, rw}))
        return FP8_ERR_ARG;
    if (dweight != nullptr &&
        any_overlap({{dweight, cols * 4}, {workspace, need}}, {ry, rg, rx, rh, rr, rw}))
        return FP8_ERR_ARG;
    const fp8q::RmsNormBackwardArgs a{dy, h, rstd, weight, w_dtype == FP8_BF16, dh, rows, cols, dx,
                                      dweight, dweight != nullptr ? static_cast<float*>(workspace) : nullptr};
    return status_of(fp8q::launch_rmsnorm_backward(a, dtype, st));
}

int fp8q_gemm_gated(const uint8_t* a, const float* sa, int a_fmt, const uint8_t* b, const float* sb, int b_fmt,
                    int64_t M, int64_t F, int64_t K, int act, int fmt, uint8_t* q, float* scales, void* gu,
                    int gu_dtype, void* stream) {
    if (!fmt_ok(a_fmt) || !fmt_ok(b_fmt) || !fmt_ok(fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(gu_dtype)) return FP8_ERR_DTYPE;
    if (!act_ok(act)) return FP8_ERR_ARG;
    if (M < 0 || F < 0 || K < 0 || F % 128 != 0 || K % 128 != 0) return FP8_ERR_SHAPE;
    if (M >= kMaxDim || F >= kMaxDim || K >= kMaxDim) return FP8_ERR_SHAPE;
    if (!size_ok(M, 2 * F) || !size_ok(M, K) || !size_ok(2 * F, K)) return FP8_ERR_SHAPE;
    if (M == 0 || F == 0) return FP8_OK;
    if ((q == nullptr) != (scales == nullptr) || (q == nullptr && gu == nullptr)) return FP8_ERR_NULL;
    if (K > 0 && (a == nullptr || sa == nullptr || b == nullptr || sb == nullptr)) return FP8_ERR_NULL;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(q, 16) || !aligned(gu, 16) || !aligned(sa, 4) ||
        !aligned(sb, 4) || !aligned(scales, 4))
        return FP8_ERR_ALIGN;
    const int64_t kb = K / 128;
    if (any_overlap({{q, M * F}, {scales, M * (F / 128) * 4}, {gu, M * 2 * F * esize(gu_dtype)}},
                    {{a, M * K}, {sa, M * kb * 4}, {b, 2 * F * K}, {sb, 2 * F / 128 * kb * 4}}))
        return FP8_ERR_ARG;
    const fp8q::GatedArgs p{a, sa, a_fmt, b, sb, b_fmt, M, F, K, act, fmt, q, scales, gu, gu_dtype};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return status_of(fp8q::launch_gemm_gated_empty(p, st));
    if (!fp8q::gemm_blockwise_supported()) return FP8_ERR_CUDA;
    return status_of(fp8q::launch_gemm_gated(p, st));
}

int fp8q_gated_backward(const void* gu, const void* dh, int dtype, int64_t M, int64_t F, int act, int fmt, uint8_t* q,
                        float* scales, uint8_t* qt, float* scales_t, uint8_t* ht, float* ht_scales, void* stream) {
    if (!fmt_ok(fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(dtype)) return FP8_ERR_DTYPE;
    if (!act_ok(act)) return FP8_ERR_ARG;
    if (M < 0 || F < 0 || F % 128 != 0 || M >= kMaxDim || F >= kMaxDim || !size_ok(M + 127, 2 * F))
        return FP8_ERR_SHAPE;
    if ((qt == nullptr) != (scales_t == nullptr) || (ht == nullptr) != (ht_scales == nullptr)) return FP8_ERR_NULL;
    if (M == 0 || F == 0) return FP8_OK;
    if (gu == nullptr || dh == nullptr || q == nullptr || scales == nullptr) return FP8_ERR_NULL;
    if (!aligned(gu, 16) || !aligned(dh, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(ht, 16) ||
        !aligned(scales, 4) || !aligned(scales_t, 4) || !aligned(ht_scales, 4))
        return FP8_ERR_ALIGN;
    const int64_t mt = (M + 127) / 128 * 128, e = esize(dtype);
    if (any_overlap({{q, M * 2 * F},
                     {scales, M * (2 * F / 128) * 4},
                     {qt, 2 * F * mt},
                     {scales_t, 2 * F * (mt / 128) * 4},
                     {ht, F * mt},
                     {ht_scales, F * (mt / 128) * 4}},
                    {{gu, M * 2 * F * e}, {dh, M * F * e}}))
        return FP8_ERR_ARG;
    const fp8q::GatedBackwardArgs p{gu, dh, M, F, act, q, scales, qt, scales_t, ht, ht_scales};
    return status_of(fp8q::launch_gated_backward(p, dtype, fmt, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
