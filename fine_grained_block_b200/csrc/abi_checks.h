// abi_checks.h -- argument checks that the C ABI's files share.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "fp8q_ffn.h"

namespace fp8q_abi {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool fmt_ok(int fmt) { return fmt == FP8_E4M3 || fmt == FP8_E5M2; }
inline bool dtype_ok(int dt) { return dt == FP8_F32 || dt == FP8_BF16; }
inline bool act_ok(int act) { return act == FP8Q_ACT_SILU || act == FP8Q_ACT_GELU_TANH; }
inline int64_t esize(int dt) { return dt == FP8_F32 ? 4 : 2; }
inline int status_of(cudaError_t e) { return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA; }

// Sizes whose products with element sizes and 128-padded copies stay far from overflow.
inline bool size_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 0 && (rows == 0 || cols <= (INT64_MAX >> 6) / rows);
}

struct Range {
    const void* p;
    int64_t bytes;
};
inline bool overlap(const Range& a, const Range& b) {
    if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}
// Whether an output overlaps an input or an earlier output.
inline bool any_overlap(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
    for (const Range* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Range& i : inputs)
            if (overlap(*o, i)) return true;
        for (const Range* e = outputs.begin(); e != o; ++e)
            if (overlap(*o, *e)) return true;
    }
    return false;
}

constexpr int64_t kMaxDim = int64_t(1) << 30;

}  // namespace fp8q_abi
