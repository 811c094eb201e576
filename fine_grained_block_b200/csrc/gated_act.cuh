// gated_act.cuh -- the activations of the gated feed-forward product, both as
// act(g) = g * sigmoid(p(g)):
//   SiLU       p = g
//   tanh GELU  p = 2 sqrt(2/pi) (g + 0.044715 g^3)   (0.5 (1 + tanh z) = sigmoid(2z))
// With sg = sigmoid(p):  act' = sg + g * sg * (1 - sg) * p'.
// (Written with tanh the GELU would lose its small values to cancellation.)
//
// Two elements at a time in packed fp32 arithmetic.  sg = 1 / (1 + 2^t) with
// t = -p log2(e), whose roundings put 2^t off by |p| 2^-24 relative times
//   SiLU  1.3  (the constant 0.23, the product 1)
//   GELU  4    (the cubic term's constant 0.9 and g^2 1, the sum 1, the product 1)
// and the hardware's 2^t and 1/x by a few 2^-24 more: far inside the half step
// 2^-4 of the codes made from them and of what 32-bit scales show.  2^t overflows
// to infinity for very negative p, where 1 / infinity = 0 is the right limit.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fp8q_device.cuh"

namespace fp8q {

constexpr int kActSilu = 0;
constexpr int kActGeluTanh = 1;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// max(|a|, |b|, |c|); a NaN counts for nothing
__device__ __forceinline__ float absmax3(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t both(float v) { return f32x2(v, v); }

// sigmoid(p(g)); g2sq = g^2 is used by the GELU only
template <int ACT>
__device__ __forceinline__ uint64_t gate_sigmoid2(uint64_t g2, uint64_t g2sq) {
    const uint64_t t2 = ACT == kActSilu
                            ? mul_f32x2(g2, both(-kLog2e))
                            : mul_f32x2(g2, fma_f32x2(g2sq, both(-kLog2e * kGeluC * kGeluA), both(-kLog2e * kGeluC)));
    const float2 t = f32x2_split(t2);
    const float2 d = f32x2_split(add_f32x2(f32x2(ex2_approx(t.x), ex2_approx(t.y)), both(1.0f)));
    return f32x2(rcp_approx(d.x), rcp_approx(d.y));
}

template <int ACT>
__device__ __forceinline__ uint64_t gate_act2(uint64_t g2) {
    return mul_f32x2(g2, gate_sigmoid2<ACT>(g2, ACT == kActSilu ? 0 : mul_f32x2(g2, g2)));
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void gate_act_grad2(uint64_t g2, uint64_t& a2, uint64_t& da2) {
    uint64_t g2sq = 0;
    if (ACT != kActSilu) {  // held finite: 1 - sg is 0 long before, and 0 * infinity is no slope
        const float2 q = f32x2_split(mul_f32x2(g2, g2));
        g2sq = f32x2(fminf(q.x, 1e30f), fminf(q.y, 1e30f));
    }
    const uint64_t sg2 = gate_sigmoid2<ACT>(g2, g2sq);
    a2 = mul_f32x2(g2, sg2);
    uint64_t rest = fma_f32x2(sg2, both(-1.0f), both(1.0f));  // 1 - sg
    if (ACT != kActSilu) rest = mul_f32x2(rest, fma_f32x2(g2sq, both(3.0f * kGeluA * kGeluC), both(kGeluC)));
    da2 = fma_f32x2(a2, rest, sg2);
}

}  // namespace fp8q
