// moe_rows.cu -- tokens to the rows of their experts and back.
//
//   dispatch   row r of token t = src[r] / top_k:  v = w * x[t] (w = 1 without weights), in 1x128 blocks as codes:
//              s = MAX / max(amax(v), eps), q = fp8(RN_f32(v * s)); rows without a pair (src -1) are zeros
//   combine    y[t] = RN(residual[t] + sum over k of w[t, k] * x[pos[t, k]]), fp32, k ascending
//   weights    dw[t, k] = <dy[t], x[pos[t, k]]>, fp32
//
// The dispatch without a transposed copy goes by tokens: a token is read and quantized once and its codes are written
// to its top_k rows.  (Row by row it would be read from DRAM top_k times: an expert's rows sweep all tokens.)  With a
// weight the block's amax is RN(|w| amax(x)), the same as the maximum of the rounded products because rounding is
// monotonic.  With the transposed copy it goes by tiles of 128 rows x 128 columns, as the blockwise quantizer of x and
// x^T does, with gathered rows; the tiles walk a slab of columns down all rows before the next slab, so that the
// tokens' slab (16384 x 512 bf16: 16 MiB) stays in L2 while its experts read it again.
//
// All of these are bound by memory.

#include <algorithm>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "lane_vec.cuh"
#include "launch_util.h"
#include "moe.h"
#include "tile_transpose.cuh"

namespace fp8q {
namespace {

#ifndef FP8Q_SLAB
#define FP8Q_SLAB 2
#endif
constexpr int kThreads = 256;

// 16 consecutive elements of a row, in fp32.
template <typename T>
struct Run16;
template <>
struct Run16<uint16_t> {
    static __device__ __forceinline__ void load(const uint16_t* p, float (&v)[16]) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        const uint4 a = ld_stream(q), b = ld_stream(q + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
    }
    static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[16]) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        st_stream(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        st_stream(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
};
template <>
struct Run16<float> {
    static __device__ __forceinline__ void load(const float* p, float (&v)[16]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 a = ld_stream(reinterpret_cast<const uint4*>(p) + k);
            v[4 * k] = __uint_as_float(a.x);
            v[4 * k + 1] = __uint_as_float(a.y);
            v[4 * k + 2] = __uint_as_float(a.z);
            v[4 * k + 3] = __uint_as_float(a.w);
        }
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[16]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            st_stream(reinterpret_cast<uint4*>(p) + k,
                      make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                                 __float_as_uint(v[4 * k + 3])));
    }
};

__device__ __forceinline__ float absmax16(const float (&v)[16]) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; j += 2) a = absmax3(a, v[j], v[j + 1]);
    return a;
}

template <int FMT>
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float s) {
    const uint64_t s2 = f32x2(s, s);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 lo = f32x2_split(mul_f32x2(f32x2(v[4 * k], v[4 * k + 1]), s2));
        const float2 hi = f32x2_split(mul_f32x2(f32x2(v[4 * k + 2], v[4 * k + 3]), s2));
        w[k] = cvt_fp8x2<FMT>(lo.x, lo.y) | (cvt_fp8x2<FMT>(hi.x, hi.y) << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of the route that are in use.
__device__ __forceinline__ int64_t rows_used(const MoeRoute& r) {
    return min(max(static_cast<int64_t>(r.offsets[r.num_experts]), int64_t(0)), r.rows);
}

// Zeros on the rows without a pair, a warp for 32 of them.
template <int FMT>
__device__ __forceinline__ void zero_rows(const MoeDispatchArgs& p, int64_t used) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int64_t pairs = p.r.tokens * p.r.top_k, blocks = p.cols / 128;
    for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * 32; r0 < used; r0 += warps * 32) {
        const int64_t r = r0 + lane;
        const int64_t pair = r < used ? p.r.src[r] : 0;
        unsigned empty = __ballot_sync(0xFFFFFFFFu, pair < 0 || pair >= pairs);
        while (empty != 0) {
            const int64_t row = r0 + __ffs(empty) - 1;
            empty &= empty - 1;
            for (int64_t j = lane; j < p.cols / 16; j += 32)
                st_stream(reinterpret_cast<uint4*>(p.q + row * p.cols) + j, make_uint4(0, 0, 0, 0));
            for (int64_t j = lane; j < blocks; j += 32) p.scales[row * blocks + j] = scale_from_amax<FMT>(0.0f);
        }
    }
}

// By tokens: 8 lanes a block of 128, 16 elements a lane.  T uint8_t: codes, which are moved with their scales.
template <typename T, int FMT, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch(MoeDispatchArgs p) {
    pdl_enter();
    const int sub = threadIdx.x & 7;
    const int64_t blocks = p.cols / 128, total = p.r.tokens * blocks;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 8);
    // whole warps stay in the loop: a group past the end repeats the last block and writes nothing
    for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * (kThreads / 8) + (threadIdx.x / 32) * 4; g0 < total; g0 += step) {
        const int64_t g = g0 + ((threadIdx.x & 31) >> 3);
        const bool live = g < total;
        const int64_t t = (live ? g : total - 1) / blocks, blk = (live ? g : total - 1) - t * blocks;
        const int64_t at = blk * 128 + sub * 16;
        float v[16], amax = 0.0f, s = 0.0f;
        uint4 c = make_uint4(0, 0, 0, 0);
        if constexpr (sizeof(T) == 1) {
            c = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + t * p.cols + at));
            s = __ldg(p.xs + t * blocks + blk);
        } else {
            Run16<T>::load(static_cast<const T*>(p.x) + t * p.cols + at, v);
            amax = warp_max<8>(absmax16(v));
            if (!WEIGHTED) {
                s = scale_from_amax<FMT>(amax);
                c = codes16<FMT>(v, s);
            }
        }
        for (int64_t k = 0; k < p.r.top_k; ++k) {
            const int64_t row = __ldg(p.r.pos + t * p.r.top_k + k);
            if (row < 0 || row >= p.r.rows || !live) continue;
            if constexpr (WEIGHTED) {
                const float w = __ldg(p.weights + t * p.r.top_k + k);
                s = scale_from_amax<FMT>(fmaxf(__fmul_rn(fabsf(w), amax), 0.0f));
                float u[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) u[j] = __fmul_rn(w, v[j]);
                c = codes16<FMT>(u, s);
            }
            st_stream(reinterpret_cast<uint4*>(p.q + row * p.cols + at), c);
            if (sub == 0) p.scales[row * blocks + blk] = s;
        }
    }
    zero_rows<FMT>(p, rows_used(p.r));
}

// The transposed copy, by tiles of 128 rows x 128 columns.  A lane holds 8 columns of 8 consecutive rows, so that the
// codes of two rows of a column leave the conversion side by side: no bytes are permuted.  16 lanes a row (a 256-byte
// run of bf16), 16 rows a warp.  Codes pass through shared memory as [column][row]; the 8-byte piece of rows
// 8 k .. 8 k + 7 of a column is at place k ^ (column / 8), where both the lanes that write (16 column groups) and those
// that read (whole columns) meet every bank once.
template <typename T>
struct Cols8;  // 8 consecutive elements of a row
template <>
struct Cols8<uint16_t> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t* p) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ float at(int j) const { return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]); }
};
template <>
struct Cols8<float> {
    float f[8];
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    }
    __device__ __forceinline__ float at(int j) const { return f[j]; }
};

template <typename T, int FMT, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) k_moe_transpose(MoeDispatchArgs p, int slab) {
    __shared__ __align__(16) uint8_t tile[kTT * kTT];
    __shared__ __align__(16) float part[kThreads / 32][kTT];  // column maxima of a warp's rows
    __shared__ __align__(16) float col_scale[kTT];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane & 15, half = lane >> 4;
    // slab after slab of `slab` column tiles; down the rows within one
    const int64_t tiles_c = p.cols / kTT, tiles_r = p.r.rows / kTT, in_slab = slab * tiles_r;
    const int64_t sl = blockIdx.x / in_slab, rest = blockIdx.x - sl * in_slab;
    const int64_t width = min(static_cast<int64_t>(slab), tiles_c - sl * slab);
    const int64_t tr = rest / width, tc = sl * slab + (rest - tr * width);
    const int64_t r0 = tr * kTT, c0 = tc * kTT;
    const int64_t used = rows_used(p.r);
    if (r0 >= used) return;
    // lane l < 16 finds the token of the warp's row l
    const int64_t row = r0 + warp * 16 + group;
    const int64_t pair = row < used ? __ldg(p.r.src + row) : -1;
    int token = -1;
    float weight = 0.0f;
    if (pair >= 0 && pair < p.r.tokens * p.r.top_k) {
        token = static_cast<int>(static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.r.top_k));
        if (WEIGHTED) weight = __ldg(p.weights + pair);
    }
    Cols8<T> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = __shfl_sync(0xFFFFFFFFu, token, half * 8 + i);
        if (t >= 0) x[i].load(static_cast<const T*>(p.x) + t * p.cols + c0 + group * 8);
        else x[i].zero();
    }
    uint64_t w2[4];  // the weights of two rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w2[i] = 0;
        if (WEIGHTED)
            w2[i] = f32x2(__shfl_sync(0xFFFFFFFFu, weight, half * 8 + 2 * i), __shfl_sync(0xFFFFFFFFu, weight, half * 8 + 2 * i + 1));
    }
    auto rows2 = [&](int i, int j) {  // rows 2 i, 2 i + 1 of column j
        const uint64_t v = f32x2(x[2 * i].at(j), x[2 * i + 1].at(j));
        return WEIGHTED ? mul_f32x2(v, w2[i]) : v;
    };
    float m[8];
    if constexpr (sizeof(T) == 2 && !WEIGHTED) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t a = x[0].w[k];
#pragma unroll
            for (int i = 1; i < 8; ++i) a = xabsmax_bf16x2(a, x[i].w[k]);
            a = xabsmax_bf16x2(a, __shfl_xor_sync(0xFFFFFFFFu, a, 16)) & 0x7FFF7FFFu;
            m[2 * k] = bf16_lo(a);
            m[2 * k + 1] = bf16_hi(a);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = f32x2_split(rows2(i, j));
                m[j] = absmax3(m[j], v.x, v.y);
            }
            m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
        }
    }
    if (half == 0) {
        *reinterpret_cast<float4*>(&part[warp][group * 8]) = make_float4(m[0], m[1], m[2], m[3]);
        *reinterpret_cast<float4*>(&part[warp][group * 8 + 4]) = make_float4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    if (threadIdx.x < kTT) {
        float a = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) a = fmaxf(a, part[w][threadIdx.x]);
        const float s = scale_from_amax<FMT>(a);
        col_scale[threadIdx.x] = s;
        p.scales_t[(c0 + threadIdx.x) * tiles_r + tr] = s;
    }
    __syncthreads();
    uint8_t* piece = tile + group * 8 * kTT + (((warp * 2 + half) ^ group) * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float s = col_scale[group * 8 + j];
        const uint64_t s2 = f32x2(s, s);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = f32x2_split(mul_f32x2(rows2(i, j), s2));
            c[i] = cvt_fp8x2<FMT>(v.x, v.y);
        }
        *reinterpret_cast<uint2*>(piece + j * kTT) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTT * kTT / 16 / kThreads; ++i) {  // 8 lanes a column: whole lines
        const int u = i * kThreads + static_cast<int>(threadIdx.x), col = u >> 3, b = u & 7, g = col >> 3;
        uint4 v = *reinterpret_cast<const uint4*>(tile + col * kTT + ((b ^ (g >> 1)) * 16));
        if (g & 1) v = make_uint4(v.z, v.w, v.x, v.y);
        st_stream(reinterpret_cast<uint4*>(p.qt + (c0 + col) * p.r.rows + r0 + b * 16), v);
    }
}

// y[t] over 16 columns a thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_moe_combine(MoeCombineArgs p) {
    pdl_enter();
    const int64_t runs = p.cols / 16, total = p.tokens * runs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = i / runs, at = (i - t * runs) * 16;
        float acc[16];
        if (p.residual != nullptr) {
            Run16<T>::load(static_cast<const T*>(p.residual) + t * p.cols + at, acc);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
        }
        for (int64_t k = 0; k < p.top_k; ++k) {
            const int64_t row = __ldg(p.pos + t * p.top_k + k);
            if (row < 0 || row >= p.rows) continue;
            const float w = p.weights != nullptr ? __ldg(p.weights + t * p.top_k + k) : 1.0f;
            float v[16];
            Run16<T>::load(static_cast<const T*>(p.x) + row * p.cols + at, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] = __fmaf_rn(w, v[j], acc[j]);
        }
        Run16<T>::store(static_cast<T*>(p.y) + t * p.cols + at, acc);
    }
}

// A CTA a token: every thread a share of the columns, the sums joined in a fixed order.
constexpr int kDotThreads = 128;
constexpr int kDots = 8;  // weights at a time

template <typename T>
__global__ void __launch_bounds__(kDotThreads) k_moe_weight_grad(const T* __restrict__ dy, const T* __restrict__ x,
                                                                 const int32_t* __restrict__ pos, int64_t top_k,
                                                                 int64_t rows, int64_t cols, float* __restrict__ dweights) {
    __shared__ float part[kDotThreads / 32][kDots];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    for (int64_t k0 = 0; k0 < top_k; k0 += kDots) {
        const int n = static_cast<int>(min(static_cast<int64_t>(kDots), top_k - k0));
        int64_t row[kDots];
        float acc[kDots];
#pragma unroll
        for (int k = 0; k < kDots; ++k) {
            row[k] = k < n ? __ldg(pos + t * top_k + k0 + k) : -1;
            if (row[k] >= rows) row[k] = -1;
            acc[k] = 0.0f;
        }
        for (int64_t at = threadIdx.x * 16; at < cols; at += kDotThreads * 16) {
            float d[16];
            Run16<T>::load(dy + t * cols + at, d);
#pragma unroll
            for (int k = 0; k < kDots; ++k) {
                if (row[k] < 0) continue;
                float v[16];
                Run16<T>::load(x + row[k] * cols + at, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[k] = __fmaf_rn(d[j], v[j], acc[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kDots; ++k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[k] += __shfl_xor_sync(0xFFFFFFFFu, acc[k], o);
            if (lane == 0) part[warp][k] = acc[k];
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n)
            dweights[t * top_k + k0 + threadIdx.x] =
                (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
        __syncthreads();
    }
}

constexpr int kSlab = FP8Q_SLAB;  // column tiles that are walked together

unsigned grid_of(int64_t work, int64_t per_cta) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((work + per_cta - 1) / per_cta, 1 << 20)));
}

template <typename T, int FMT, bool WEIGHTED>
cudaError_t dispatch_typed(const MoeDispatchArgs& p, cudaStream_t st) {
    const int64_t groups = std::max(p.r.tokens * (p.cols / 128), (p.r.rows + 3) / 4);
    const cudaError_t e =
        launch_kernel(k_moe_dispatch<T, FMT, WEIGHTED>, dim3(grid_of(groups, kThreads / 8)), dim3(kThreads), 0, st, p);
    if constexpr (sizeof(T) > 1) {
        if (p.qt != nullptr && e == cudaSuccess) {
            const int64_t tiles = p.cols / kTT * (p.r.rows / kTT);
            if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
            return launch_kernel(k_moe_transpose<T, FMT, WEIGHTED>, dim3(static_cast<unsigned>(tiles)), dim3(kThreads), 0, st,
                                 p, kSlab);
        }
    }
    return e;
}

template <typename T>
cudaError_t dispatch_fmt(const MoeDispatchArgs& p, int fmt, cudaStream_t st) {
    if (p.weights != nullptr)
        return fmt == kE4M3 ? dispatch_typed<T, kE4M3, true>(p, st) : dispatch_typed<T, kE5M2, true>(p, st);
    return fmt == kE4M3 ? dispatch_typed<T, kE4M3, false>(p, st) : dispatch_typed<T, kE5M2, false>(p, st);
}

}  // namespace

cudaError_t launch_moe_dispatch(const MoeDispatchArgs& p, int dtype, int fmt, cudaStream_t st) {
    return dtype == 0 ? dispatch_fmt<float>(p, fmt, st) : dispatch_fmt<uint16_t>(p, fmt, st);
}

cudaError_t launch_moe_dispatch_codes(const MoeDispatchArgs& p, int fmt, cudaStream_t st) {
    return fmt == kE4M3 ? dispatch_typed<uint8_t, kE4M3, false>(p, st) : dispatch_typed<uint8_t, kE5M2, false>(p, st);
}

cudaError_t launch_moe_combine(const MoeCombineArgs& p, int dtype, cudaStream_t st) {
    const dim3 grid(grid_of(p.tokens * (p.cols / 16), kThreads));
    return dtype == 0 ? launch_kernel(k_moe_combine<float>, grid, dim3(kThreads), 0, st, p)
                      : launch_kernel(k_moe_combine<uint16_t>, grid, dim3(kThreads), 0, st, p);
}

cudaError_t launch_moe_weight_grad(const void* dy, const void* x, int dtype, const int32_t* pos, int64_t tokens,
                                   int64_t top_k, int64_t rows, int64_t cols, float* dweights, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(tokens));
    if (dtype == 0)
        return launch_kernel(k_moe_weight_grad<float>, grid, dim3(kDotThreads), 0, st, static_cast<const float*>(dy),
                             static_cast<const float*>(x), pos, top_k, rows, cols, dweights);
    return launch_kernel(k_moe_weight_grad<uint16_t>, grid, dim3(kDotThreads), 0, st, static_cast<const uint16_t*>(dy),
                         static_cast<const uint16_t*>(x), pos, top_k, rows, cols, dweights);
}

}  // namespace fp8q
