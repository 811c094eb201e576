// gemm_gated.h -- launchers of the gated projections (gemm_gated.cu,
// gemm_gated_few.cu) and of their backward pass (gated_backward.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fp8q {

struct GatedArgs {
    const uint8_t* a;   // [M, K] codes, 1x128 scales sa [M, K/128]
    const float* sa;
    int a_fmt;
    const uint8_t* b;   // [2F, K] codes, gate rows first; 128x128 scales sb [2F/128, K/128]
    const float* sb;
    int b_fmt;
    int64_t M, F, K;
    int act, fmt;
    uint8_t* q;         // [M, F] codes and [M, F/128] scales of act(G) * U, or both null
    float* scales;
    void* gu;           // [M, 2F] the projections, or null
    int gu_dtype;
};

// Any M and K > 0; F and K multiples of 128.
cudaError_t launch_gemm_gated(const GatedArgs& p, cudaStream_t stream);
// K == 0: every projection is an empty sum.
cudaError_t launch_gemm_gated_empty(const GatedArgs& p, cudaStream_t stream);

// The form for few tokens (the weights' rows take the tensor core's M side), and whether it is the faster one.
bool gemm_gated_few_fits(const GatedArgs& p);
cudaError_t launch_gemm_gated_few(const GatedArgs& p, cudaStream_t stream);

struct GatedBackwardArgs {
    const void* gu;  // [M, 2F]
    const void* dh;  // [M, F]
    int64_t M, F;
    int act;
    uint8_t* q;      // [M, 2F] codes of [dG | dU], scales [M, 2F/128]
    float* scales;
    uint8_t* qt;     // [2F, Mt] codes of [dG | dU]^T, scales [2F, Mt/128], or both null
    float* scales_t;
    uint8_t* ht;     // [F, Mt] codes of H^T, scales [F, Mt/128], or both null
    float* ht_scales;
};
cudaError_t launch_gated_backward(const GatedBackwardArgs& p, int dtype, int fmt, cudaStream_t stream);

// [rows, K] bytes, K-major, boxes of box_rows x 128 bytes with the 128-byte
// swizzle; rows past the end read as zeros.
bool make_code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, uint32_t box_rows);

}  // namespace fp8q
