// gated_backward.cu -- the backward pass of H = act(G) * U, quantized for the
// GEMMs that consume it.
//
//   dG = dH * U * act'(G),  dU = dH * act(G),  H = act(G) * U (recomputed)
// Outputs, each in the layout that fp8_gemm_blockwise reads:
//   q   [M, 2F]   [dG | dU] in 1x128 blocks: A of the data gradient
//                 dX = [dG | dU] [Wg; Wu]
//   qt  [2F, Mt]  [dG | dU]^T in 1x128 blocks along the tokens: A of the
//                 weight gradient d[Wg; Wu] = [dG | dU]^T X
//   ht  [F, Mt]   H^T in 1x128 blocks along the tokens: B of dWd = dY^T H
// Mt is M rounded up to 128; the tokens from M on get zero codes and do not
// count toward an amax.  Everything is quantized from fp32; nothing is rounded
// to bf16 between.
//
// One CTA per 128x128 tile.  A lane takes 16 columns of a row, 8 lanes the
// block of a row, a warp 16 rows in 4 steps.  First pass: the values, the row
// scales (shuffles), the row codes, and the column maxima of the three
// tensors.  Second pass, after the column scales are known: the inputs again
// (from L2) and the values again, cast with the column scales into three
// shared code tiles that go out transposed.  Keeping the first pass's values
// instead would take 192 fp32 registers a thread.

#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "gemm_gated.h"
#include "lane_vec.cuh"
#include "launch_util.h"
#include "tile_transpose.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kE = 16;  // elements of a lane's slice

// 16 consecutive elements as they lie in memory.
template <typename T>
struct Slice {
    static constexpr int kWords = kE * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        else return (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    }
    __device__ __forceinline__ void set(int k, uint4 v) {
        w[4 * k] = v.x;
        w[4 * k + 1] = v.y;
        w[4 * k + 2] = v.z;
        w[4 * k + 3] = v.w;
    }
};
template <typename T>
__device__ __forceinline__ Slice<T> load_slice(const T* p, bool live) {
    Slice<T> s;
#pragma unroll
    for (int k = 0; k < Slice<T>::kWords / 4; ++k)
        s.set(k, live ? ld_stream(reinterpret_cast<const uint4*>(p) + k) : make_uint4(0, 0, 0, 0));
    return s;
}

// A warp's ring of two steps of input: per step 4 rows x 128 columns of G, U and dH, copied asynchronously
// (cp.async) so that a step's loads are in flight while the step before it is computed, without holding
// registers.  A copy instruction covers whole 512-byte runs; the 16-byte chunks of a row are swizzled so
// that the lanes' slices read back without bank conflicts.
template <typename T>
struct Ring {
    static constexpr int kChunks = kTT * static_cast<int>(sizeof(T)) / 16;  // 16-byte chunks of a row
    static constexpr int kPer = 4 * kChunks / 32;                          // copies of a lane per tensor and step
    static constexpr int kTensorBytes = 4 * kChunks * 16;
    static constexpr int kStepBytes = 3 * kTensorBytes;
    static constexpr int kRowsPerCopy = 32 / kChunks;
    static __device__ __forceinline__ int swizzle(int c) { return c ^ ((c >> 3) & 3); }

    static __device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
    }
    // rows row0 .. row0 + 3 of the block column at c0 into `stage`; rows from M on read as zeros
    static __device__ __forceinline__ void issue(const GatedBackwardArgs& p, int64_t row0, int64_t c0, uint32_t stage,
                                                 int lane) {
        const int c = lane % kChunks, r = lane / kChunks;
        const T* g = static_cast<const T*>(p.gu) + c0;
        const T* d = static_cast<const T*>(p.dh) + c0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int rr = r + j * kRowsPerCopy;
            const int64_t row = row0 + rr;
            const bool live = row < p.M;
            const int64_t at = (live ? row : 0) * p.F;
            const uint32_t dst = stage + static_cast<uint32_t>((rr * kChunks + swizzle(c)) * 16);
            copy16(dst, reinterpret_cast<const char*>(g + 2 * at) + c * 16, live);
            copy16(dst + kTensorBytes, reinterpret_cast<const char*>(g + 2 * at + p.F) + c * 16, live);
            copy16(dst + 2 * kTensorBytes, reinterpret_cast<const char*>(d + at) + c * 16, live);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    static __device__ __forceinline__ Slice<T> read(const uint8_t* stage, int tensor, int lane) {
        constexpr int kN = Slice<T>::kWords / 4;
        const uint8_t* row = stage + tensor * kTensorBytes + (lane / 8) * kChunks * 16;
        Slice<T> s;
#pragma unroll
        for (int k = 0; k < kN; ++k)
            s.set(k, *reinterpret_cast<const uint4*>(row + swizzle((lane % 8) * kN + k) * 16));
        return s;
    }
};
static_assert(Ring<uint16_t>::kRowsPerCopy == 2 && Ring<float>::kRowsPerCopy == 1, "a copy covers whole rows");

// dG, dU and H of a lane's 16 elements.
template <int ACT, typename T>
__device__ __forceinline__ void gated_grads(const Slice<T>& g, const Slice<T>& u, const Slice<T>& d, float (&dg)[kE],
                                            float (&du)[kE], float (&h)[kE]) {
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
        const uint64_t u2 = f32x2(u.get(e), u.get(e + 1)), d2 = f32x2(d.get(e), d.get(e + 1));
        uint64_t a2, da2;
        gate_act_grad2<ACT>(f32x2(g.get(e), g.get(e + 1)), a2, da2);
        const float2 x = f32x2_split(mul_f32x2(mul_f32x2(d2, u2), da2));
        const float2 y = f32x2_split(mul_f32x2(d2, a2));
        const float2 z = f32x2_split(mul_f32x2(a2, u2));
        dg[e] = x.x;
        dg[e + 1] = x.y;
        du[e] = y.x;
        du[e + 1] = y.y;
        h[e] = z.x;
        h[e + 1] = z.y;
    }
}

// 16 fp32 values times a scale each -> 16 codes.
template <int FMT>
__device__ __forceinline__ uint4 cast16(const float (&v)[kE], const float (&s)[kE]) {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 a = f32x2_split(mul_f32x2(f32x2(v[4 * k], v[4 * k + 1]), f32x2(s[4 * k], s[4 * k + 1])));
        const float2 b = f32x2_split(mul_f32x2(f32x2(v[4 * k + 2], v[4 * k + 3]), f32x2(s[4 * k + 2], s[4 * k + 3])));
        c[k] = cvt_fp8x2<FMT>(a.x, a.y) | (cvt_fp8x2<FMT>(b.x, b.y) << 16);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}
template <int FMT>
__device__ __forceinline__ uint4 cast16(const float (&v)[kE], float s) {
    float t[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) t[e] = s;
    return cast16<FMT>(v, t);
}

// The row codes and scales of one lane slice of dG and dU.
template <int FMT>
__device__ __forceinline__ void row_codes(const GatedBackwardArgs& p, const float (&dg)[kE], const float (&du)[kE],
                                          int64_t row, int64_t c0, int slice, bool live) {
    float ag = 0.0f, au = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        ag = fmaxf(ag, fabsf(dg[e]));
        au = fmaxf(au, fabsf(du[e]));
    }
    ag = warp_max<8>(ag);
    au = warp_max<8>(au);
    // one division a lane: even lanes form dG's scale, odd ones dU's
    const float mine = scale_from_amax<FMT>((slice & 1) ? au : ag);
    const float other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
    const float sg = (slice & 1) ? other : mine, su = (slice & 1) ? mine : other;
    if (!live) return;
    uint8_t* q = p.q + row * 2 * p.F + c0;
    st_stream(reinterpret_cast<uint4*>(q) + slice, cast16<FMT>(dg, sg));
    st_stream(reinterpret_cast<uint4*>(q + p.F) + slice, cast16<FMT>(du, su));
    if (slice == 0) {
        float* s = p.scales + row * (2 * p.F / 128) + c0 / 128;
        s[0] = sg;
        s[p.F / 128] = su;
    }
}

constexpr int kTileBytes = kTT * kTT;
template <typename T>
struct Smem {  // code tiles (the warps' column maxima before them), column scales, the warps' input rings
    static constexpr int kScales = 3 * kTileBytes;
    static constexpr int kRing = kScales + 3 * kTT * 4;
    static constexpr int kBytes = kRing + kWarps * 2 * Ring<T>::kStepBytes;
};
static_assert(kWarps * 3 * kTT * 4 <= 3 * kTileBytes, "the warps' column maxima fit where the code tiles will be");

template <typename T, int FMT, int ACT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
k_gated_backward_tile(GatedBackwardArgs p) {
    pdl_enter();
    extern __shared__ __align__(16) uint8_t smem[];
    using R = Ring<T>;
    float* part = reinterpret_cast<float*>(smem);  // [warp][tensor][column]
    float* col_scale = reinterpret_cast<float*>(smem + Smem<T>::kScales);  // [tensor][column]
    const int64_t tiles_c = p.F / kTT;
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const int64_t r0 = tr * kTT, c0 = tc * kTT;
    const int64_t mt = (p.M + kTT - 1) / kTT * kTT, tiles_r = mt / kTT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lr0 = warp * 16 + lane / 8, slice = lane % 8;
    const uint8_t* ring = smem + Smem<T>::kRing + warp * 2 * R::kStepBytes;
    const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

    // Steps 0-3 are the first pass over the warp's 16 rows, steps 4-7 the second.
    auto issue = [&](int step) {
        R::issue(p, r0 + warp * 16 + 4 * (step & 3), c0, ring_u + static_cast<uint32_t>((step & 1) * R::kStepBytes), lane);
    };
    Slice<T> g, u, d;
    auto fetch = [&](int step) {
        if (step < 7) {
            issue(step + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        const uint8_t* stage = ring + (step & 1) * R::kStepBytes;
        g = R::read(stage, 0, lane);
        u = R::read(stage, 1, lane);
        d = R::read(stage, 2, lane);
        __syncwarp();  // before the next copies into this stage
    };
    issue(0);

    float cm[3][kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) cm[0][e] = cm[1][e] = cm[2][e] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int64_t row = r0 + lr0 + 4 * i;
        fetch(i);
        float dg[kE], du[kE], hh[kE];
        gated_grads<ACT, T>(g, u, d, dg, du, hh);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            cm[0][e] = fmaxf(cm[0][e], fabsf(dg[e]));
            cm[1][e] = fmaxf(cm[1][e], fabsf(du[e]));
            cm[2][e] = fmaxf(cm[2][e], fabsf(hh[e]));
        }
        row_codes<FMT>(p, dg, du, row, c0, slice, row < p.M);
    }
    // The maxima over the warp's 4 row groups: lanes exchange halves, so that each ends with 4 columns.
    {
        const bool b3 = lane & 8, b4 = lane & 16;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            float m8[8], m4[4];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float send = b3 ? cm[k][e] : cm[k][e + 8];
                m8[e] = fmaxf(b3 ? cm[k][e + 8] : cm[k][e], __shfl_xor_sync(0xFFFFFFFFu, send, 8));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float send = b4 ? m8[e] : m8[e + 4];
                m4[e] = fmaxf(b4 ? m8[e + 4] : m8[e], __shfl_xor_sync(0xFFFFFFFFu, send, 16));
            }
            *reinterpret_cast<float4*>(part + (warp * 3 + k) * kTT + slice * kE + (b3 ? 8 : 0) + (b4 ? 4 : 0)) =
                make_float4(m4[0], m4[1], m4[2], m4[3]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = threadIdx.x + j * kThreads;
        if (i < 3 * kTT) {
            float m = part[i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, part[w * 3 * kTT + i]);
            const float s = scale_from_amax<FMT>(m);
            col_scale[i] = s;
            const int k = i / kTT, c = i % kTT;
            if (k < 2 && p.scales_t != nullptr) p.scales_t[(k * p.F + c0 + c) * tiles_r + tr] = s;
            if (k == 2 && p.ht_scales != nullptr) p.ht_scales[(c0 + c) * tiles_r + tr] = s;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int lr = lr0 + 4 * i;
        fetch(4 + i);
        float v[3][kE];
        gated_grads<ACT, T>(g, u, d, v[0], v[1], v[2]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            float s[kE];
#pragma unroll
            for (int e = 0; e < kE; e += 4) {
                const float4 f = *reinterpret_cast<const float4*>(col_scale + k * kTT + slice * kE + e);
                s[e] = f.x;
                s[e + 1] = f.y;
                s[e + 2] = f.z;
                s[e + 3] = f.w;
            }
            *reinterpret_cast<uint4*>(smem + k * kTileBytes + tile_off(lr, slice * kE)) = cast16<FMT>(v[k], s);
        }
    }
    __syncthreads();
    if (p.qt != nullptr) {
        tile_transpose_out(smem, p.qt, mt, r0, c0, lane, warp);
        tile_transpose_out(smem + kTileBytes, p.qt + p.F * mt, mt, r0, c0, lane, warp);
    }
    if (p.ht != nullptr) tile_transpose_out(smem + 2 * kTileBytes, p.ht, mt, r0, c0, lane, warp);
}

// Row codes only (frozen weights): a warp per 4 rows of a block column, nothing shared.
template <typename T, int FMT, int ACT>
__global__ void __launch_bounds__(kThreads)
k_gated_backward_rows(GatedBackwardArgs p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t blocks = p.F / 128;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t r4 = unit / blocks, c0 = (unit - r4 * blocks) * 128;
    const int64_t row = r4 * 4 + lane / 8;
    const int slice = lane % 8;
    const bool live = row < p.M;
    const T* gu = static_cast<const T*>(p.gu) + row * 2 * p.F + c0 + slice * kE;
    const Slice<T> g = load_slice<T>(gu, live);
    const Slice<T> u = load_slice<T>(gu + p.F, live);
    const Slice<T> d = load_slice<T>(static_cast<const T*>(p.dh) + row * p.F + c0 + slice * kE, live);
    float dg[kE], du[kE], hh[kE];
    gated_grads<ACT, T>(g, u, d, dg, du, hh);
    row_codes<FMT>(p, dg, du, row, c0, slice, live);
}

template <typename T, int FMT, int ACT>
cudaError_t launch_typed(const GatedBackwardArgs& p, cudaStream_t st) {
    if (p.qt == nullptr && p.ht == nullptr) {
        const int64_t units = (p.M + 3) / 4 * (p.F / 128);
        const int64_t grid = (units + kWarps - 1) / kWarps;
        if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
        return launch_kernel(k_gated_backward_rows<T, FMT, ACT>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                             st, p);
    }
    auto kern = k_gated_backward_tile<T, FMT, ACT>;
    static std::atomic<bool> opted[128];  // the shared-memory opt-in, once per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<T>::kBytes);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (p.M + kTT - 1) / kTT * (p.F / kTT);
    if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_kernel(kern, dim3(static_cast<unsigned>(tiles)), dim3(kThreads), Smem<T>::kBytes, st, p);
}

template <typename T, int FMT>
cudaError_t launch_act(const GatedBackwardArgs& p, cudaStream_t st) {
    return p.act == kActSilu ? launch_typed<T, FMT, kActSilu>(p, st) : launch_typed<T, FMT, kActGeluTanh>(p, st);
}

}  // namespace

cudaError_t launch_gated_backward(const GatedBackwardArgs& p, int dtype, int fmt, cudaStream_t st) {
    if (dtype == 1) return fmt == kE4M3 ? launch_act<uint16_t, kE4M3>(p, st) : launch_act<uint16_t, kE5M2>(p, st);
    return fmt == kE4M3 ? launch_act<float, kE4M3>(p, st) : launch_act<float, kE5M2>(p, st);
}

}  // namespace fp8q
