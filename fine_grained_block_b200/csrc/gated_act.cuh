// gated_act.cuh -- the activations of the gated feed-forward product, both as
// act(g) = g * sigmoid(p(g)):
//   SiLU       p = g
//   tanh GELU  p = 2 sqrt(2/pi) (g + 0.044715 g^3)   (0.5 (1 + tanh z) = sigmoid(2z))
// With sg = sigmoid(p):  act' = sg + g * sg * (1 - sg) * p'.
// exp(-p) overflows to infinity for very negative p, where 1 / (1 + inf) = 0
// is the right limit; written with tanh the GELU would lose its small values
// to cancellation.
#pragma once

#include <cuda_runtime.h>

namespace fp8q {

constexpr int kActSilu = 0;
constexpr int kActGeluTanh = 1;
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float gate_sigmoid(float g, int act) {
    const float p = act == kActSilu ? g : kGeluC * g * fmaf(kGeluA * g, g, 1.0f);
    return __fdividef(1.0f, 1.0f + expf(-p));
}

// 1 / (1 + x) for x in [0, inf]: __fdividef gives 0 from 2^126 on, as the limit asks.
__device__ __forceinline__ float gate_act(float g, int act) { return g * gate_sigmoid(g, act); }

// act(g) and act'(g)
__device__ __forceinline__ float2 gate_act_grad(float g, int act) {
    const float sg = gate_sigmoid(g, act);
    const float slope = act == kActSilu ? 1.0f : kGeluC * fmaf(3.0f * kGeluA * g, g, 1.0f);
    const float a = g * sg;
    return make_float2(a, fmaf(a * (1.0f - sg), slope, sg));
}

}  // namespace fp8q
