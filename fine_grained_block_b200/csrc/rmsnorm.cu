// rmsnorm.cu -- root-mean-square norm with the residual's addition and an FP8
// output in 1x128 blocks, and its backward pass.
//
// Forward, per row of [rows, cols]:
//   h    = RN_dtype(x + residual)          (h = x without a residual)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y    = (h * rstd) * w                  fp32, two roundings
//   s    = MAX / max(amax(y block), eps'), q = fp8(RN_f32(y * s))
// The norm is that of the stored (rounded) h, so the backward pass, which
// reads h, differentiates what was computed.  The codes come from the fp32 y,
// not from a rounded copy.
//
// Backward, with n = h * rstd, a = dy * w, c = sum(a * n) / cols:
//   dx = rstd * (a - n * c) + dh,   dw = sum over rows of dy * n.
//
// Both stream their tensors once and are bound by HBM.  A CTA walks rows
// first, first + grid, ... (persistent: the weight, and the backward's dw sums,
// stay in registers), a thread owns the same columns of every row, and the next
// row's loads are issued before the current row's reduction, so that data is in
// flight across the row's one barrier.  All sums are fp32.  The order of every
// sum is fixed by the shape and the device, so results repeat bit for bit.

#include <algorithm>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "lane_vec.cuh"
#include "launch_util.h"
#include "rmsnorm.h"

namespace fp8q {
namespace {

template <typename T>
__device__ __forceinline__ float load_f(const T* p);
template <>
__device__ __forceinline__ float load_f(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const volatile uint16_t*>(p)) << 16);
}
template <>
__device__ __forceinline__ float load_f(const float* p) {
    return *reinterpret_cast<const volatile float*>(p);
}
__device__ __forceinline__ float load_w(const void* w, int w_bf16, int64_t i) {
    return w_bf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(w) + i)) << 16)
                  : __ldg(static_cast<const float*>(w) + i);
}
// RN_dtype(v), as fp32
template <typename T>
__device__ __forceinline__ float round_to(float v) {
    if constexpr (sizeof(T) == 2) return bf16_lo(pack_bf16x2(v, 0.0f));
    else return v;
}
template <typename T>
__device__ __forceinline__ void store_f(T* p, float v) {
    if constexpr (sizeof(T) == 2) *p = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    else *p = v;
}

// One lane vector of BYTES bytes as fp32 values, and back.
template <typename T, int BYTES>
struct Vec {
    using W = Words<BYTES / 4>;
    static constexpr int kElems = BYTES / static_cast<int>(sizeof(T));
    static __device__ __forceinline__ W zero() {
        W v;
#pragma unroll
        for (int k = 0; k < BYTES / 4; ++k) v.w[k] = 0u;
        return v;
    }
    static __device__ __forceinline__ float get(const W& v, int e) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(v.w[e]);
        else return (e & 1) ? bf16_hi(v.w[e >> 1]) : bf16_lo(v.w[e >> 1]);
    }
    static __device__ __forceinline__ W pack(const float (&f)[kElems]) {
        W v;
#pragma unroll
        for (int k = 0; k < BYTES / 4; ++k) {
            if constexpr (sizeof(T) == 4) v.w[k] = __float_as_uint(f[k]);
            else v.w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
        }
        return v;
    }
    static __device__ __forceinline__ void store(void* base, int64_t vec, const W& v) {
        if constexpr (BYTES == 32) {
            V32 o;
#pragma unroll
            for (int k = 0; k < 8; ++k) o.w[k] = v.w[k];
            st32_stream(static_cast<char*>(base) + vec * 32, o);
        } else {
            st_stream(static_cast<uint4*>(base) + vec, make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
        }
    }
};

template <int WIDTH>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = WIDTH / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Sum over the CTA (or, WARP_ROW, over the warp).  `red` holds 32 words; the caller alternates two of
// them, so that one barrier per sum is enough: a warp writes red[i] again only after the barrier of the
// sum in between, which every reader of red[i] has passed.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum<32>(v);
    if (WARP_ROW) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum<32>(lane < warps ? red[lane] : 0.0f);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// One row in registers: nvec lane vectors, VPT per thread.  WARP_ROW: a warp per row (narrow rows, no
// barrier); else a CTA per row.
template <typename T, int FMT, int BYTES, int VPT, int MAXT, bool WARP_ROW>
__global__ void __launch_bounds__(MAXT)
k_rmsnorm_quantize(RmsNormArgs p) {
    pdl_enter();
    using V = Vec<T, BYTES>;
    using W = typename V::W;
    using Out = typename LaneVec<T, BYTES>::Out;
    constexpr int E = V::kElems;
    constexpr int kLanes = 128 / E;  // lanes of one 1x128 block
    __shared__ float red[2][32];
    const int lane = threadIdx.x & 31;
    const int tid = WARP_ROW ? lane : static_cast<int>(threadIdx.x);
    const int stride = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
    const int64_t first = WARP_ROW ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP_ROW ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
    const int nvec = static_cast<int>(p.cols / E);
    const int64_t nblk = (p.cols + 127) >> 7;
    const W* x = static_cast<const W*>(p.x);
    const W* res = static_cast<const W*>(p.residual);

    float w[VPT][E];
    W xv[VPT], rv[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int vec = tid + v * stride;
        xv[v] = rv[v] = V::zero();
        if (vec < nvec && first < p.rows) {
            xv[v] = ld_words_stream(x + first * nvec + vec);
            if (res != nullptr) rv[v] = ld_words_stream(res + first * nvec + vec);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) w[v][e] = vec < nvec ? load_w(p.weight, p.w_bf16, static_cast<int64_t>(vec) * E + e) : 0.0f;
    }
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    int parity = 0;
    for (int64_t row = first; row < p.rows; row += step, parity ^= 1) {
        float f[VPT][E];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int vec = tid + v * stride;
            if (res != nullptr) {
                float t[E];
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] = __fadd_rn(V::get(xv[v], e), V::get(rv[v], e));
                const W hv = V::pack(t);
                if (vec < nvec) V::store(p.h, row * nvec + vec, hv);
#pragma unroll
                for (int e = 0; e < E; ++e) f[v][e] = V::get(hv, e);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) f[v][e] = V::get(xv[v], e);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) ss = __fmaf_rn(f[v][e], f[v][e], ss);
            const int64_t next = row + step;
            if (vec < nvec && next < p.rows) {
                xv[v] = ld_words_stream(x + next * nvec + vec);
                if (res != nullptr) rv[v] = ld_words_stream(res + next * nvec + vec);
            }
        }
        ss = row_sum<WARP_ROW>(ss, red[parity]);
        const float rstd = rsqrtf(__fmaf_rn(ss, inv_cols, p.eps));
        if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int vec = tid + v * stride;
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                f[v][e] = __fmul_rn(__fmul_rn(f[v][e], rstd), w[v][e]);
                amax = fmaxf(amax, fabsf(f[v][e]));
            }
            const float s = scale_from_amax<FMT>(warp_max<kLanes>(amax));
            const uint64_t s2 = f32x2(s, s);
            if (vec < nvec) {
                uint32_t c[E / 4];
#pragma unroll
                for (int k = 0; k < E / 4; ++k) {
                    const float2 a = f32x2_split(mul_f32x2(f32x2(f[v][4 * k], f[v][4 * k + 1]), s2));
                    const float2 b = f32x2_split(mul_f32x2(f32x2(f[v][4 * k + 2], f[v][4 * k + 3]), s2));
                    c[k] = cvt_fp8x2<FMT>(a.x, a.y) | (cvt_fp8x2<FMT>(b.x, b.y) << 16);
                }
                st_stream(reinterpret_cast<Out*>(p.q) + row * nvec + vec, CodeWords<E / 4>::make(c));
                if (vec % kLanes == 0) p.scales[row * nblk + vec / kLanes] = s;
                if (p.y != nullptr) V::store(p.y, row * nvec + vec, V::pack(f[v]));
            }
        }
    }
}

// Any width and any 16-byte-aligned pointers, element by element: the row is read twice (the second time
// from L2 or L1), a warp per 1x128 block in the second pass.
template <typename T, int FMT>
__global__ void __launch_bounds__(512)
k_rmsnorm_quantize_general(RmsNormArgs p) {
    pdl_enter();
    __shared__ float red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t nblk = (p.cols + 127) >> 7;
    const T* x = static_cast<const T*>(p.x);
    const T* res = static_cast<const T*>(p.residual);
    T* h = static_cast<T*>(p.h);
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
        const int64_t r0 = row * p.cols;
        float ss = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float f = load_f(x + r0 + c);
            if (res != nullptr) {
                f = round_to<T>(__fadd_rn(f, load_f(res + r0 + c)));
                store_f(h + r0 + c, f);
            }
            ss = __fmaf_rn(f, f, ss);
        }
        ss = row_sum<false>(ss, red[parity]);  // its barrier also orders the h stores before the reads below
        const float rstd = rsqrtf(__fmaf_rn(ss, inv_cols, p.eps));
        if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
        const T* src = res != nullptr ? h : x;
        for (int64_t blk = warp; blk < nblk; blk += warps) {
            float f[4];
            float amax = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = blk * 128 + 32 * k + lane;
                f[k] = c < p.cols ? __fmul_rn(__fmul_rn(load_f(src + r0 + c), rstd), load_w(p.weight, p.w_bf16, c)) : 0.0f;
                amax = fmaxf(amax, fabsf(f[k]));
            }
            const float s = scale_from_amax<FMT>(warp_max<32>(amax));
            if (lane == 0) p.scales[row * nblk + blk] = s;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = blk * 128 + 32 * k + lane;
                if (c < p.cols) {
                    p.q[r0 + c] = static_cast<uint8_t>(cvt_fp8x2<FMT>(__fmul_rn(f[k], s), 0.0f) & 0xFFu);
                    if (p.y != nullptr) store_f(static_cast<T*>(p.y) + r0 + c, f[k]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// A CTA per row, persistent; each thread keeps the dw sums of its columns in registers and writes them to
// the CTA's row of the workspace at the end.
template <typename T, int BYTES, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT)
k_rmsnorm_backward(RmsNormBackwardArgs p) {
    pdl_enter();
    using V = Vec<T, BYTES>;
    using W = typename V::W;
    constexpr int E = V::kElems;
    __shared__ float red[2][32];
    const int tid = threadIdx.x, stride = blockDim.x;
    const int64_t first = blockIdx.x, step = gridDim.x;
    const int nvec = static_cast<int>(p.cols / E);
    const W* dy = static_cast<const W*>(p.dy);
    const W* h = static_cast<const W*>(p.h);
    const W* dh = static_cast<const W*>(p.dh);

    float w[VPT][E], dw[VPT][E];
    W yv[VPT], hv[VPT], gv[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int vec = tid + v * stride;
        yv[v] = hv[v] = gv[v] = V::zero();
        if (vec < nvec) {
            yv[v] = ld_words_stream(dy + first * nvec + vec);
            hv[v] = ld_words_stream(h + first * nvec + vec);
            if (dh != nullptr) gv[v] = ld_words_stream(dh + first * nvec + vec);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w[v][e] = vec < nvec ? load_w(p.weight, p.w_bf16, static_cast<int64_t>(vec) * E + e) : 0.0f;
            dw[v][e] = 0.0f;
        }
    }
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    int parity = 0;
    for (int64_t row = first; row < p.rows; row += step, parity ^= 1) {
        const float rstd = __ldg(p.rstd + row);
        W cy[VPT], ch[VPT], cg[VPT];
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int vec = tid + v * stride;
            cy[v] = yv[v];
            ch[v] = hv[v];
            cg[v] = gv[v];
            const int64_t next = row + step;
            if (vec < nvec && next < p.rows) {
                yv[v] = ld_words_stream(dy + next * nvec + vec);
                hv[v] = ld_words_stream(h + next * nvec + vec);
                if (dh != nullptr) gv[v] = ld_words_stream(dh + next * nvec + vec);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = __fmul_rn(V::get(ch[v], e), rstd);
                const float d = V::get(cy[v], e);
                dot = __fmaf_rn(__fmul_rn(d, w[v][e]), n, dot);
                dw[v][e] = __fmaf_rn(d, n, dw[v][e]);
            }
        }
        const float c = __fmul_rn(row_sum<false>(dot, red[parity]), inv_cols);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int vec = tid + v * stride;
            float t[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = __fmul_rn(V::get(ch[v], e), rstd);
                const float a = __fmul_rn(V::get(cy[v], e), w[v][e]);
                t[e] = __fmaf_rn(rstd, __fmaf_rn(-n, c, a), dh != nullptr ? V::get(cg[v], e) : 0.0f);
            }
            if (vec < nvec) V::store(p.dx, row * nvec + vec, V::pack(t));
        }
    }
    if (p.partial == nullptr) return;
    float* out = p.partial + first * p.cols;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int vec = tid + v * stride;
        if (vec < nvec) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k)
                reinterpret_cast<float4*>(out + static_cast<int64_t>(vec) * E)[k] =
                    make_float4(dw[v][4 * k], dw[v][4 * k + 1], dw[v][4 * k + 2], dw[v][4 * k + 3]);
        }
    }
}

// Any width: element by element, dw summed in the CTA's workspace row (each element by one thread).
template <typename T>
__global__ void __launch_bounds__(512)
k_rmsnorm_backward_general(RmsNormBackwardArgs p) {
    pdl_enter();
    __shared__ float red[2][32];
    const T* dy = static_cast<const T*>(p.dy);
    const T* h = static_cast<const T*>(p.h);
    const T* dh = static_cast<const T*>(p.dh);
    T* dx = static_cast<T*>(p.dx);
    float* out = p.partial != nullptr ? p.partial + blockIdx.x * p.cols : nullptr;
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
        const int64_t r0 = row * p.cols;
        const float rstd = __ldg(p.rstd + row);
        float dot = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const float n = __fmul_rn(load_f(h + r0 + c), rstd);
            const float d = load_f(dy + r0 + c);
            dot = __fmaf_rn(__fmul_rn(d, load_w(p.weight, p.w_bf16, c)), n, dot);
            if (out != nullptr) out[c] = __fmaf_rn(d, n, row == blockIdx.x ? 0.0f : out[c]);
        }
        const float cc = __fmul_rn(row_sum<false>(dot, red[parity]), inv_cols);
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const float n = __fmul_rn(load_f(h + r0 + c), rstd);
            const float a = __fmul_rn(load_f(dy + r0 + c), load_w(p.weight, p.w_bf16, c));
            store_f(dx + r0 + c, __fmaf_rn(rstd, __fmaf_rn(-n, cc, a), dh != nullptr ? load_f(dh + r0 + c) : 0.0f));
        }
    }
}

// dweight[c] = sum of the `parts` partial rows.  A CTA takes 32 columns; its 32 warps take the rows
// w, w + 32, ... and their sums meet in shared memory.
__global__ void __launch_bounds__(1024)
k_rmsnorm_dweight(const float* __restrict__ partial, int parts, int64_t cols, float* __restrict__ dweight) {
    pdl_enter();
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float v = 0.0f;
    if (c < cols)
        for (int r = warp; r < parts; r += 32) v += partial[r * cols + c];
    sum[warp][lane] = v;
    __syncthreads();
    v = warp_sum<32>(sum[lane][warp]);  // this warp: column blockIdx.x * 32 + warp
    const int64_t cw = static_cast<int64_t>(blockIdx.x) * 32 + warp;
    if (lane == 0 && cw < cols) dweight[cw] = v;
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

int round_up32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

template <typename T, int FMT, int BYTES, int VPT, int MAXT>
cudaError_t launch_forward_vec(const RmsNormArgs& p, int threads, cudaStream_t st) {
    const int64_t grid = std::min<int64_t>(p.rows, device_sm_count() * std::max(1, 1024 / threads));
    return launch_kernel(k_rmsnorm_quantize<T, FMT, BYTES, VPT, MAXT, false>, dim3(static_cast<unsigned>(grid)),
                         dim3(threads), 0, st, p);
}

template <typename T, int FMT>
cudaError_t launch_forward(const RmsNormArgs& p, cudaStream_t st) {
    constexpr int E32 = 32 / static_cast<int>(sizeof(T)), E16 = E32 / 2;
    const bool wide = p.cols % E32 == 0 && aligned32(p.x) && aligned32(p.residual) && aligned32(p.h) && aligned32(p.y);
    if (wide && p.cols / E32 <= 1024) {
        const int64_t nvec = p.cols / E32;
        if (nvec <= 32) {
            constexpr int kWarps = 8;
            const int64_t grid = std::min<int64_t>((p.rows + kWarps - 1) / kWarps, device_sm_count() * 8);
            return launch_kernel(k_rmsnorm_quantize<T, FMT, 32, 1, 256, true>, dim3(static_cast<unsigned>(grid)),
                                 dim3(kWarps * 32), 0, st, p);
        }
        return nvec <= 512 ? launch_forward_vec<T, FMT, 32, 1, 512>(p, round_up32(nvec), st)
                           : launch_forward_vec<T, FMT, 32, 2, 512>(p, round_up32((nvec + 1) / 2), st);
    }
    if (p.cols % E16 == 0 && p.cols / E16 <= 1024)
        return launch_forward_vec<T, FMT, 16, 1, 1024>(p, round_up32(p.cols / E16), st);
    const int64_t grid = std::min<int64_t>(p.rows, device_sm_count() * 4);
    return launch_kernel(k_rmsnorm_quantize_general<T, FMT>, dim3(static_cast<unsigned>(grid)), dim3(512), 0, st, p);
}

template <typename T, int BYTES, int VPT, int MAXT>
cudaError_t launch_backward_vec(const RmsNormBackwardArgs& p, int threads, int64_t most, int64_t* parts,
                                cudaStream_t st) {
    *parts = std::min<int64_t>(most, device_sm_count() * std::max(1, std::min(4, 1024 / threads)));
    return launch_kernel(k_rmsnorm_backward<T, BYTES, VPT, MAXT>, dim3(static_cast<unsigned>(*parts)), dim3(threads), 0,
                         st, p);
}

template <typename T>
cudaError_t launch_backward(const RmsNormBackwardArgs& p, int64_t* parts, cudaStream_t st) {
    constexpr int E16 = 16 / static_cast<int>(sizeof(T));
    const int64_t nvec = p.cols / E16;
    const int64_t most = rmsnorm_backward_partials(p.rows);
    if (p.cols % E16 == 0 && nvec <= 1024)
        return launch_backward_vec<T, 16, 1, 1024>(p, round_up32(nvec), most, parts, st);
    if constexpr (sizeof(T) == 4) {
        if (p.cols % E16 == 0 && nvec <= 2048)
            return launch_backward_vec<T, 16, 2, 1024>(p, round_up32((nvec + 1) / 2), most, parts, st);
    }
    *parts = most;
    return launch_kernel(k_rmsnorm_backward_general<T>, dim3(static_cast<unsigned>(most)), dim3(512), 0, st, p);
}

}  // namespace

int64_t rmsnorm_backward_partials(int64_t rows) { return std::min<int64_t>(rows, device_sm_count() * 4); }

cudaError_t launch_rmsnorm_quantize(const RmsNormArgs& p, int dtype, int fmt, cudaStream_t st) {
    if (dtype == 1)
        return fmt == kE4M3 ? launch_forward<uint16_t, kE4M3>(p, st) : launch_forward<uint16_t, kE5M2>(p, st);
    return fmt == kE4M3 ? launch_forward<float, kE4M3>(p, st) : launch_forward<float, kE5M2>(p, st);
}

cudaError_t launch_rmsnorm_backward(const RmsNormBackwardArgs& p, int dtype, float* dweight, cudaStream_t st) {
    int64_t parts = 0;
    const cudaError_t e = dtype == 1 ? launch_backward<uint16_t>(p, &parts, st) : launch_backward<float>(p, &parts, st);
    if (e != cudaSuccess || dweight == nullptr) return e;
    return launch_kernel(k_rmsnorm_dweight, dim3(static_cast<unsigned>((p.cols + 31) / 32)), dim3(1024), 0, st,
                         static_cast<const float*>(p.partial), static_cast<int>(parts), p.cols, dweight);
}

}  // namespace fp8q
