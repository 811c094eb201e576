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

// By tiles of 128 rows x 128 columns, with the transposed copy.  8 lanes a row, 16 elements a lane, 4 rows a warp and
// load, 16 rows a warp.
template <typename T, int FMT, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, 2) k_moe_dispatch_transpose(MoeDispatchArgs p, int slab) {
    __shared__ __align__(16) uint8_t tile[kTT * kTT];
    __shared__ __align__(16) float part[kThreads / 32][kTT];
    __shared__ __align__(16) float col_scale[kTT];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7;
    // slab after slab of `slab` column tiles; down the rows within one
    const int64_t tiles_c = p.cols / kTT, tiles_r = p.r.rows / kTT, in_slab = slab * tiles_r;
    const int64_t sl = blockIdx.x / in_slab, rest = blockIdx.x - sl * in_slab;
    const int64_t width = min(static_cast<int64_t>(slab), tiles_c - sl * slab);
    const int64_t tr = rest / width, tc = sl * slab + (rest - tr * width);
    const int64_t r0 = tr * kTT, c0 = tc * kTT;
    const int64_t used = rows_used(p.r);
    if (r0 >= used) return;
    const int64_t pairs = p.r.tokens * p.r.top_k;
    constexpr int kLoads = 4;
    float v[kLoads][16];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t r = r0 + warp * 16 + i * 4 + (lane >> 3);
        const int64_t pair = r < used ? __ldg(p.r.src + r) : -1;
        if (pair >= 0 && pair < pairs) {
            Run16<T>::load(static_cast<const T*>(p.x) + pair / p.r.top_k * p.cols + c0 + sub * 16, v[i]);
            if (WEIGHTED) {
                const float w = __ldg(p.weights + pair);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[i][j] = __fmul_rn(w, v[i][j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = 0.0f;
        }
    }
    float m[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) m[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t r = r0 + warp * 16 + i * 4 + (lane >> 3);
        const float s = scale_from_amax<FMT>(warp_max<8>(absmax16(v[i])));
        if (r < used) {
            st_stream(reinterpret_cast<uint4*>(p.q + r * p.cols + c0 + sub * 16), codes16<FMT>(v[i], s));
            if (sub == 0) p.scales[r * tiles_c + tc] = s;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) m[j] = fmaxf(m[j], fabsf(v[i][j]));
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 8));
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
    }
    if (lane < 8) {
#pragma unroll
        for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(&part[warp][sub * 16 + j]) = make_float4(m[j], m[j + 1], m[j + 2], m[j + 3]);
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
    uint64_t cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 s = *reinterpret_cast<const float2*>(&col_scale[sub * 16 + 2 * j]);
        cs[j] = f32x2(s.x, s.y);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 lo = f32x2_split(mul_f32x2(f32x2(v[i][4 * k], v[i][4 * k + 1]), cs[2 * k]));
            const float2 hi = f32x2_split(mul_f32x2(f32x2(v[i][4 * k + 2], v[i][4 * k + 3]), cs[2 * k + 1]));
            w[k] = cvt_fp8x2<FMT>(lo.x, lo.y) | (cvt_fp8x2<FMT>(hi.x, hi.y) << 16);
        }
        *reinterpret_cast<uint4*>(tile + tile_off(warp * 16 + i * 4 + (lane >> 3), sub * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    tile_transpose_out(tile, p.qt, p.r.rows, r0, c0, lane, warp);
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

unsigned grid_of(int64_t work, int64_t per_cta) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((work + per_cta - 1) / per_cta, 1 << 20)));
}

template <typename T, int FMT, bool WEIGHTED>
cudaError_t dispatch_typed(const MoeDispatchArgs& p, cudaStream_t st) {
    if constexpr (sizeof(T) > 1) {
        if (p.qt != nullptr) {
            const int64_t tiles = p.cols / kTT * (p.r.rows / kTT);
            if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
            if (tiles == 0) return cudaSuccess;
            constexpr int kSlab = 4;
            return launch_kernel(k_moe_dispatch_transpose<T, FMT, WEIGHTED>, dim3(static_cast<unsigned>(tiles)),
                                 dim3(kThreads), 0, st, p, kSlab);
        }
    }
    const int64_t groups = std::max(p.r.tokens * (p.cols / 128), (p.r.rows + 3) / 4);
    return launch_kernel(k_moe_dispatch<T, FMT, WEIGHTED>, dim3(grid_of(groups, kThreads / 8)), dim3(kThreads), 0, st, p);
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
