// rmsnorm.h -- launchers of the root-mean-square norm (rmsnorm.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fp8q {

struct RmsNormArgs {
    const void* x;
    const void* residual;  // or null
    const void* weight;
    int w_bf16;
    int64_t rows, cols;
    float eps;
    uint8_t* q;
    float* scales;
    void* h;      // written when residual is given
    void* y;      // or null
    float* rstd;  // or null
};
cudaError_t launch_rmsnorm_quantize(const RmsNormArgs& p, int dtype, int fmt, cudaStream_t stream);

struct RmsNormBackwardArgs {
    const void* dy;
    const void* h;
    const float* rstd;
    const void* weight;
    int w_bf16;
    const void* dh;  // or null
    int64_t rows, cols;
    void* dx;
    float* dweight;  // or null
    float* partial;  // [rmsnorm_backward_partials(rows), cols] workspace for dweight
};
// Rows of the workspace that the weight gradient's partial sums take.
int64_t rmsnorm_backward_partials(int64_t rows);
// Whether rows are so few that, whatever their type, one launch writes dweight itself and needs no workspace.
bool rmsnorm_backward_one_launch(int64_t rows, int64_t cols);
cudaError_t launch_rmsnorm_backward(const RmsNormBackwardArgs& p, int dtype, cudaStream_t stream);

}  // namespace fp8q
