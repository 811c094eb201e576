// moe_abi.cu -- the C ABI of the routed feed-forward block's operators
// (include/fp8q_ffn.h): argument checks, then the launches.  Nothing here
// allocates, synchronizes or keeps state.

#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "abi_checks.h"
#include "fp8q_ffn.h"
#include "fp8q_launch.h"
#include "moe.h"

using namespace fp8q_abi;

namespace {

bool experts_ok(int num_experts) { return num_experts >= 1 && num_experts <= fp8q::kMaxExperts; }
bool align_ok(int align) { return align >= 1 && align <= 128 && (align & (align - 1)) == 0; }
// tokens * top_k pairs that 32-bit indices hold
bool pairs_ok(int64_t tokens, int64_t top_k) {
    return tokens >= 0 && top_k >= 1 && top_k <= kMaxDim && tokens <= kMaxDim / top_k;
}
constexpr int64_t kMaxRows = kMaxDim + int64_t(fp8q::kMaxExperts) * 128;

// The rows that hold any routing of the pairs: min(E, pairs) experts, each with up to align - 1 rows more.
int64_t rows_needed(int64_t pairs, int num_experts, int align) {
    return (pairs + std::min<int64_t>(num_experts, pairs) * (align - 1)) / align * align;
}

struct RouteRanges {
    Range offsets, pos, src;
};
RouteRanges ranges(const fp8q::MoeRoute& r) {
    return {{r.offsets, (int64_t(r.num_experts) + 1) * 4}, {r.pos, r.tokens * r.top_k * 4}, {r.src, r.rows * 4}};
}
bool route_ok(const fp8q::MoeRoute& r) {
    return experts_ok(r.num_experts) && pairs_ok(r.tokens, r.top_k) && r.rows >= 0 && r.rows <= kMaxRows;
}
bool route_null(const fp8q::MoeRoute& r) {
    return r.offsets == nullptr || (r.pos == nullptr && r.tokens > 0) || (r.src == nullptr && r.rows > 0);
}
bool route_aligned(const fp8q::MoeRoute& r) { return aligned(r.offsets, 4) && aligned(r.pos, 4) && aligned(r.src, 4); }

}  // namespace

extern "C" {

int64_t fp8q_moe_rows(int64_t tokens, int64_t top_k, int num_experts, int align) {
    if (!pairs_ok(tokens, top_k) || !experts_ok(num_experts)) return FP8_ERR_SHAPE;
    if (!align_ok(align)) return FP8_ERR_ARG;
    return rows_needed(tokens * top_k, num_experts, align);
}

int64_t fp8q_moe_sort_workspace(int64_t tokens, int64_t top_k, int num_experts) {
    if (!pairs_ok(tokens, top_k) || !experts_ok(num_experts)) return FP8_ERR_SHAPE;
    return fp8q::moe_sort_workspace_bytes(tokens * top_k, num_experts);
}

int fp8q_moe_sort(const int32_t* experts, int64_t tokens, int64_t top_k, int num_experts, int align, int64_t rows,
                  int32_t* offsets, int32_t* pos, int32_t* src, int32_t* counts, void* workspace,
                  int64_t workspace_bytes, void* stream) {
    if (!pairs_ok(tokens, top_k) || !experts_ok(num_experts) || rows < 0 || rows > kMaxRows) return FP8_ERR_SHAPE;
    if (!align_ok(align)) return FP8_ERR_ARG;
    const int64_t pairs = tokens * top_k;
    if (rows < rows_needed(pairs, num_experts, align)) return FP8_ERR_SHAPE;
    if (offsets == nullptr || (pairs > 0 && (experts == nullptr || pos == nullptr)) || (rows > 0 && src == nullptr))
        return FP8_ERR_NULL;
    const int64_t need = fp8q::moe_sort_workspace_bytes(pairs, num_experts);
    if (need > 0 && workspace == nullptr) return FP8_ERR_NULL;
    if (!aligned(experts, 4) || !aligned(offsets, 4) || !aligned(pos, 4) || !aligned(src, 4) || !aligned(counts, 4) ||
        (need > 0 && !aligned(workspace, 16)))
        return FP8_ERR_ALIGN;
    if (workspace_bytes < need) return FP8_ERR_ARG;
    if (any_overlap({{offsets, (int64_t(num_experts) + 1) * 4},
                     {pos, pairs * 4},
                     {src, rows * 4},
                     {counts, int64_t(num_experts) * 4},
                     {workspace, need}},
                    {{experts, pairs * 4}}))
        return FP8_ERR_ARG;
    const fp8q::MoeSortArgs p{experts, pairs, num_experts, align, rows, offsets, pos, src, counts, static_cast<int32_t*>(workspace)};
    return status_of(fp8q::launch_moe_sort(p, static_cast<cudaStream_t>(stream)));
}

int fp8q_moe_dispatch(const void* x, int dtype, int64_t cols, const int32_t* offsets, int num_experts, const int32_t* pos,
                      const int32_t* src, int64_t tokens, int64_t top_k, int64_t rows, int fmt, uint8_t* q,
                      float* scales, uint8_t* qt, float* scales_t, void* stream) {
    if (!fmt_ok(fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(dtype)) return FP8_ERR_DTYPE;
    const fp8q::MoeRoute r{offsets, num_experts, pos, src, tokens, top_k, rows};
    if (!route_ok(r) || cols < 0 || cols % 128 != 0 || cols >= kMaxDim || !size_ok(tokens, cols) || !size_ok(rows, cols))
        return FP8_ERR_SHAPE;
    if ((qt == nullptr) != (scales_t == nullptr)) return FP8_ERR_NULL;
    if (qt != nullptr && rows % 128 != 0) return FP8_ERR_SHAPE;
    if (tokens == 0 || rows == 0 || cols == 0) return FP8_OK;
    if (x == nullptr || route_null(r) || q == nullptr || scales == nullptr) return FP8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(scales, 4) || !aligned(scales_t, 4) ||
        !route_aligned(r))
        return FP8_ERR_ALIGN;
    const RouteRanges rr = ranges(r);
    if (any_overlap({{q, rows * cols}, {scales, rows * (cols / 128) * 4}, {qt, rows * cols}, {scales_t, cols * (rows / 128) * 4}},
                    {{x, tokens * cols * esize(dtype)}, rr.offsets, rr.pos, rr.src}))
        return FP8_ERR_ARG;
    const fp8q::MoeDispatchArgs p{r, x, nullptr, nullptr, cols, q, scales, qt, scales_t};
    return status_of(fp8q::launch_moe_dispatch(p, dtype, fmt, static_cast<cudaStream_t>(stream)));
}

int fp8q_moe_dispatch_codes(const uint8_t* xq, const float* xs, int fmt, int64_t cols, const int32_t* offsets,
                            int num_experts, const int32_t* pos, const int32_t* src, int64_t tokens, int64_t top_k,
                            int64_t rows, uint8_t* q, float* scales, void* stream) {
    if (!fmt_ok(fmt)) return FP8_ERR_FORMAT;
    const fp8q::MoeRoute r{offsets, num_experts, pos, src, tokens, top_k, rows};
    if (!route_ok(r) || cols < 0 || cols % 128 != 0 || cols >= kMaxDim || !size_ok(tokens, cols) || !size_ok(rows, cols))
        return FP8_ERR_SHAPE;
    if (tokens == 0 || rows == 0 || cols == 0) return FP8_OK;
    if (xq == nullptr || xs == nullptr || route_null(r) || q == nullptr || scales == nullptr) return FP8_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(q, 16) || !aligned(xs, 4) || !aligned(scales, 4) || !route_aligned(r)) return FP8_ERR_ALIGN;
    const RouteRanges rr = ranges(r);
    if (any_overlap({{q, rows * cols}, {scales, rows * (cols / 128) * 4}},
                    {{xq, tokens * cols}, {xs, tokens * (cols / 128) * 4}, rr.offsets, rr.pos, rr.src}))
        return FP8_ERR_ARG;
    const fp8q::MoeDispatchArgs p{r, xq, xs, nullptr, cols, q, scales, nullptr, nullptr};
    return status_of(fp8q::launch_moe_dispatch_codes(p, fmt, static_cast<cudaStream_t>(stream)));
}

int fp8q_moe_combine(const void* x, int dtype, int64_t rows, int64_t cols, const int32_t* pos, const float* weights,
                     const void* residual, int64_t tokens, int64_t top_k, void* y, void* stream) {
    if (!dtype_ok(dtype)) return FP8_ERR_DTYPE;
    if (!pairs_ok(tokens, top_k) || rows < 0 || rows > kMaxRows || cols < 0 || cols % 128 != 0 || cols >= kMaxDim ||
        !size_ok(tokens, cols) || !size_ok(rows, cols))
        return FP8_ERR_SHAPE;
    if (tokens == 0 || cols == 0) return FP8_OK;
    if ((x == nullptr && rows > 0) || pos == nullptr || y == nullptr) return FP8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(pos, 4) || !aligned(weights, 4))
        return FP8_ERR_ALIGN;
    const int64_t e = esize(dtype), n = tokens * cols * e;
    if (any_overlap({{y, n}}, {{x, rows * cols * e}, {residual, n}, {pos, tokens * top_k * 4}, {weights, tokens * top_k * 4}}))
        return FP8_ERR_ARG;
    const fp8q::MoeCombineArgs p{x, residual, weights, pos, tokens, top_k, rows, cols, y};
    return status_of(fp8q::launch_moe_combine(p, dtype, static_cast<cudaStream_t>(stream)));
}

int fp8q_moe_combine_backward(const void* dy, const void* x, int dtype, int64_t cols, const int32_t* offsets,
                              int num_experts, const int32_t* pos, const int32_t* src, int64_t tokens, int64_t top_k,
                              int64_t rows, const float* weights, int fmt, uint8_t* q, float* scales, uint8_t* qt,
                              float* scales_t, float* dweights, void* stream) {
    if (!fmt_ok(fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(dtype)) return FP8_ERR_DTYPE;
    const fp8q::MoeRoute r{offsets, num_experts, pos, src, tokens, top_k, rows};
    if (!route_ok(r) || cols < 0 || cols % 128 != 0 || cols >= kMaxDim || !size_ok(tokens, cols) || !size_ok(rows, cols))
        return FP8_ERR_SHAPE;
    if ((q == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr) || (qt != nullptr && q == nullptr))
        return FP8_ERR_NULL;
    if (qt != nullptr && rows % 128 != 0) return FP8_ERR_SHAPE;
    if (tokens == 0) return FP8_OK;
    if (q == nullptr && dweights == nullptr && rows > 0 && cols > 0) return FP8_ERR_NULL;
    if (route_null(r) || (cols > 0 && dy == nullptr)) return FP8_ERR_NULL;
    if (dweights != nullptr && rows > 0 && cols > 0 && x == nullptr) return FP8_ERR_NULL;
    if (q != nullptr && weights == nullptr) return FP8_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(scales, 4) ||
        !aligned(scales_t, 4) || !aligned(weights, 4) || !aligned(dweights, 4) || !route_aligned(r))
        return FP8_ERR_ALIGN;
    const int64_t e = esize(dtype), pairs = tokens * top_k;
    const RouteRanges rr = ranges(r);
    if (any_overlap({{q, rows * cols},
                     {scales, rows * (cols / 128) * 4},
                     {qt, rows * cols},
                     {scales_t, cols * (rows / 128) * 4},
                     {dweights, pairs * 4}},
                    {{dy, tokens * cols * e}, {x, rows * cols * e}, {weights, pairs * 4}, rr.offsets, rr.pos, rr.src}))
        return FP8_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dweights != nullptr) {
        const int s = status_of(fp8q::launch_moe_weight_grad(dy, x, dtype, pos, tokens, top_k, rows, cols, dweights, st));
        if (s != FP8_OK) return s;
    }
    if (q == nullptr || rows == 0 || cols == 0) return FP8_OK;
    const fp8q::MoeDispatchArgs p{r, dy, nullptr, weights, cols, q, scales, qt, scales_t};
    return status_of(fp8q::launch_moe_dispatch(p, dtype, fmt, st));
}

static int gemm_grouped(const uint8_t* a, const float* sa, int a_fmt, const uint8_t* b, const float* sb, int b_fmt,
                        const int32_t* offsets, int num_experts, int64_t R, int64_t N, int64_t K, bool gated, int act,
                        int fmt, uint8_t* q, float* scales, void* c, int c_dtype, void* stream) {
    // N is a multiple of 128 (gated: of 256)
    if (R < 0 || K < 0 || K % 128 != 0 || R > kMaxRows || N >= kMaxDim || K >= kMaxDim || !experts_ok(num_experts) ||
        N > INT32_MAX / num_experts || !size_ok(R, N) || !size_ok(R, K) || !size_ok(N * num_experts, K))
        return FP8_ERR_SHAPE;
    if (R == 0 || N == 0) return FP8_OK;
    if (offsets == nullptr || (q == nullptr && c == nullptr) || (q == nullptr) != (scales == nullptr)) return FP8_ERR_NULL;
    if (K > 0 && (a == nullptr || sa == nullptr || b == nullptr || sb == nullptr)) return FP8_ERR_NULL;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(q, 16) || !aligned(c, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
        !aligned(scales, 4) || !aligned(offsets, 4))
        return FP8_ERR_ALIGN;
    const int64_t kb = K / 128, F = N / 2, E = num_experts;
    if (any_overlap({{q, R * F}, {scales, R * (F / 128) * 4}, {c, R * N * esize(c_dtype)}},
                    {{a, R * K}, {sa, R * kb * 4}, {b, E * N * K}, {sb, E * (N / 128) * kb * 4}, {offsets, (E + 1) * 4}}))
        return FP8_ERR_ARG;
    const fp8q::GroupedArgs p{a, sa, a_fmt, b, sb, b_fmt, offsets, num_experts, R, N, K, act, fmt, q, scales, c, c_dtype};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return status_of(fp8q::launch_gemm_grouped_empty(p, gated, st));
    if (!fp8q::gemm_blockwise_supported()) return FP8_ERR_CUDA;
    return status_of(fp8q::gemm_grouped_few_fits(p) ? fp8q::launch_gemm_grouped_few(p, gated, st)
                                                    : fp8q::launch_gemm_grouped(p, gated, st));
}

int fp8q_gemm_grouped(const uint8_t* a, const float* sa, int a_fmt, const uint8_t* b, const float* sb, int b_fmt,
                      const int32_t* offsets, int num_experts, int64_t rows, int64_t N, int64_t K, void* c,
                      int c_dtype, void* stream) {
    if (!fmt_ok(a_fmt) || !fmt_ok(b_fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(c_dtype)) return FP8_ERR_DTYPE;
    if (N < 0 || N % 128 != 0) return FP8_ERR_SHAPE;
    return gemm_grouped(a, sa, a_fmt, b, sb, b_fmt, offsets, num_experts, rows, N, K, false, FP8Q_ACT_SILU, FP8_E4M3,
                        nullptr, nullptr, c, c_dtype, stream);
}

int fp8q_gemm_gated_grouped(const uint8_t* a, const float* sa, int a_fmt, const uint8_t* b, const float* sb, int b_fmt,
                            const int32_t* offsets, int num_experts, int64_t rows, int64_t F, int64_t K, int act,
                            int fmt, uint8_t* q, float* scales, void* gu, int gu_dtype, void* stream) {
    if (!fmt_ok(a_fmt) || !fmt_ok(b_fmt) || !fmt_ok(fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(gu_dtype)) return FP8_ERR_DTYPE;
    if (!act_ok(act)) return FP8_ERR_ARG;
    if (F < 0 || F % 128 != 0 || F >= kMaxDim / 2) return FP8_ERR_SHAPE;
    return gemm_grouped(a, sa, a_fmt, b, sb, b_fmt, offsets, num_experts, rows, 2 * F, K, true, act, fmt, q, scales, gu,
                        gu_dtype, stream);
}

int fp8q_gemm_grouped_wgrad(const uint8_t* at, const float* sat, int a_fmt, const uint8_t* bt, const float* sbt, int b_fmt,
                            const int32_t* offsets, int num_experts, int64_t rows, int64_t N, int64_t K, void* dw,
                            int dw_dtype, void* stream) {
    if (!fmt_ok(a_fmt) || !fmt_ok(b_fmt)) return FP8_ERR_FORMAT;
    if (!dtype_ok(dw_dtype)) return FP8_ERR_DTYPE;
    if (rows < 0 || rows % 128 != 0 || rows > kMaxRows || N < 0 || N % 128 != 0 || K < 0 || K % 128 != 0 || N >= kMaxDim ||
        K >= kMaxDim || !experts_ok(num_experts) || N > INT32_MAX / num_experts || !size_ok(rows, N) || !size_ok(rows, K) ||
        !size_ok(N * num_experts, K))
        return FP8_ERR_SHAPE;
    if (N == 0 || K == 0) return FP8_OK;
    if (offsets == nullptr || dw == nullptr) return FP8_ERR_NULL;
    if (rows > 0 && (at == nullptr || sat == nullptr || bt == nullptr || sbt == nullptr)) return FP8_ERR_NULL;
    if (!aligned(at, 16) || !aligned(bt, 16) || !aligned(dw, 16) || !aligned(sat, 4) || !aligned(sbt, 4) || !aligned(offsets, 4))
        return FP8_ERR_ALIGN;
    const int64_t rb = rows / 128, E = num_experts;
    if (any_overlap({{dw, E * N * K * esize(dw_dtype)}},
                    {{at, N * rows}, {sat, N * rb * 4}, {bt, K * rows}, {sbt, K * rb * 4}, {offsets, (E + 1) * 4}}))
        return FP8_ERR_ARG;
    if (!fp8q::gemm_blockwise_supported()) return FP8_ERR_CUDA;
    const fp8q::GroupedWgradArgs p{at, sat, a_fmt, bt, sbt, b_fmt, offsets, num_experts, rows, N, K, dw, dw_dtype};
    return status_of(fp8q::launch_gemm_grouped_wgrad(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
