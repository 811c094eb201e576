// moe.h -- launchers of the routed feed-forward block: the sort by expert
// (moe_sort.cu), the rows' movement (moe_rows.cu) and the experts' products
// (gemm_grouped.cu, gemm_grouped_few.cu, gemm_grouped_wgrad.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fp8q {

constexpr int kMaxExperts = 1024;

// Rows of the experts, one after another: expert e has rows offsets[e] .. offsets[e + 1] - 1.
struct MoeSortArgs {
    const int32_t* experts;  // [pairs]
    int64_t pairs;
    int num_experts, align;
    int64_t rows;      // of src; holds any sort of the pairs
    int32_t* offsets;  // [num_experts + 1]
    int32_t* pos;      // [pairs]
    int32_t* src;      // [rows]
    int32_t* counts;   // [num_experts] or null
    int32_t* workspace;
};
int64_t moe_sort_workspace_bytes(int64_t pairs, int num_experts);
cudaError_t launch_moe_sort(const MoeSortArgs& p, cudaStream_t stream);

struct MoeRoute {
    const int32_t* offsets;
    int num_experts;
    const int32_t* pos;  // [tokens, top_k]
    const int32_t* src;  // [rows]
    int64_t tokens, top_k, rows;
};
struct MoeDispatchArgs {
    MoeRoute r;
    const void* x;         // [tokens, cols]
    const float* xs;       // the scales of codes x, else null
    const float* weights;  // [tokens, top_k]: a row is its token's times its weight; or null
    int64_t cols;
    uint8_t* q;            // [rows, cols], scales [rows, cols / 128]
    float* scales;
    uint8_t* qt;           // [cols, rows], scales_t [cols, rows / 128], or null
    float* scales_t;
};
cudaError_t launch_moe_dispatch(const MoeDispatchArgs& p, int dtype, int fmt, cudaStream_t stream);
cudaError_t launch_moe_dispatch_codes(const MoeDispatchArgs& p, int fmt, cudaStream_t stream);

struct MoeCombineArgs {
    const void* x;         // [rows, cols]
    const void* residual;  // [tokens, cols] or null
    const float* weights;  // [tokens, top_k] or null
    const int32_t* pos;    // [tokens, top_k]
    int64_t tokens, top_k, rows, cols;
    void* y;               // [tokens, cols]
};
cudaError_t launch_moe_combine(const MoeCombineArgs& p, int dtype, cudaStream_t stream);
// dweights[t, k] = <dy[t], x[pos[t, k]]>, 0 where a pair has no row
cudaError_t launch_moe_weight_grad(const void* dy, const void* x, int dtype, const int32_t* pos, int64_t tokens,
                                   int64_t top_k, int64_t rows, int64_t cols, float* dweights, cudaStream_t stream);

struct GroupedArgs {
    const uint8_t* a;        // [R, K] codes, 1x128 scales sa [R, K / 128]
    const float* sa;
    int a_fmt;
    const uint8_t* b;        // [E, N, K] codes, 128x128 scales sb [E, N / 128, K / 128]; gated: N = 2 F, gate rows first
    const float* sb;
    int b_fmt;
    const int32_t* offsets;  // [E + 1]
    int E;
    int64_t R, N, K;
    int act, fmt;
    uint8_t* q;              // gated: [R, F] codes and [R, F / 128] scales of act(G) * U, or both null
    float* scales;
    void* c;                 // [R, N] the products, or null
    int c_dtype;
};
// K > 0; N (gated: F) and K multiples of 128.
cudaError_t launch_gemm_grouped(const GroupedArgs& p, bool gated, cudaStream_t stream);
// K == 0: every product is an empty sum.
cudaError_t launch_gemm_grouped_empty(const GroupedArgs& p, bool gated, cudaStream_t stream);
// The form for few rows an expert, and whether it is the faster one.
bool gemm_grouped_few_fits(const GroupedArgs& p);
cudaError_t launch_gemm_grouped_few(const GroupedArgs& p, bool gated, cudaStream_t stream);

struct GroupedWgradArgs {
    const uint8_t* at;       // [N, R] codes, 1x128 scales sat [N, R / 128]
    const float* sat;
    int a_fmt;
    const uint8_t* bt;       // [K, R] codes, 1x128 scales sbt [K, R / 128]
    const float* sbt;
    int b_fmt;
    const int32_t* offsets;  // [E + 1], multiples of 128
    int E;
    int64_t R, N, K;
    void* dw;                // [E, N, K]
    int dw_dtype;
};
// N, K and R multiples of 128.
cudaError_t launch_gemm_grouped_wgrad(const GroupedWgradArgs& p, cudaStream_t stream);

}  // namespace fp8q
