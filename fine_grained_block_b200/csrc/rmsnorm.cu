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
// Rows of whole vectors (forward: up to 16384 bf16 or 8192 fp32 elements; backward: up
// to 8192 of either) are streamed once, bound by HBM.  A CTA walks rows
// first, first + grid, ... (persistent: the weight, and the backward's dw sums,
// stay in registers), a thread owns the same columns of every row, and the next
// row's loads are issued before the current row's reduction, so that data is in
// flight across the row's one barrier.  16384 x 7168 bf16 with a residual: 172 us
// forward, 154 us backward, 93-94 % of the device's copy rate; one row of 4096 takes
// 3 us, the launch and one round trip to memory.  Odd widths up to 8192 are read once,
// element by element (4096 x 7001 bf16: 86 and 131 us).  Wider rows are read twice; the
// backward pass keeps their dw sums in memory and runs at 20-36 % of the copy rate
// (4096 x 12288 bf16: 77 us forward in registers, 286 us backward).
// All sums are fp32.  The order of a row's sums is fixed by its width and type, that of the
// weight gradient by the shape and the device, so results repeat bit for bit.

#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "lane_vec.cuh"
#include "launch_util.h"
#include "rmsnorm.h"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kRanks = 8;  // CTAs of a cluster

template <typename T>
__device__ __forceinline__ float load_f(const T* p);
template <>
__device__ __forceinline__ float load_f(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
template <>
__device__ __forceinline__ float load_f(const float* p) {
    return *p;
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

// One lane vector of BYTES bytes as fp32 values, and back.  ACCESS: bytes of a memory access, 16 for 32-byte vectors at
// addresses that are only 16-byte aligned.
template <typename T, int BYTES, int ACCESS = BYTES>
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
    // Of a tensor that the kernel may also write (h over x or residual, dx over dy or dh).  The non-coherent loads of
    // ld_words_stream are for memory that nobody writes while the kernel runs.
    static __device__ __forceinline__ W load(const W* p) {
        W v;
        if constexpr (ACCESS == 32) {
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]),
                           "=r"(v.w[6]), "=r"(v.w[7])
                         : "l"(p)
                         : "memory");
        } else if constexpr (BYTES == 32) {  // the two halves are in one sector: the second comes from L1
#pragma unroll
            for (int k = 0; k < 8; k += 4)
                asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.w[k]), "=r"(v.w[k + 1]), "=r"(v.w[k + 2]), "=r"(v.w[k + 3])
                             : "l"(p->w + k)
                             : "memory");
        } else {
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
                         : "l"(p)
                         : "memory");
        }
        return v;
    }
    static __device__ __forceinline__ void store(void* base, int64_t vec, const W& v) {
        if constexpr (ACCESS == 32) {
            V32 o;
#pragma unroll
            for (int k = 0; k < 8; ++k) o.w[k] = v.w[k];
            st32_stream(static_cast<char*>(base) + vec * 32, o);
        } else {
#pragma unroll
            for (int k = 0; k < BYTES / 4; k += 4)
                st_stream(reinterpret_cast<uint4*>(static_cast<char*>(base) + vec * BYTES + 4 * k),
                          make_uint4(v.w[k], v.w[k + 1], v.w[k + 2], v.w[k + 3]));
        }
    }
};

template <int WIDTH>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = WIDTH / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// A row belongs to a group of GROUP threads (a multiple of 32); narrow rows have several groups in a CTA.
// The sum over the group: `red` holds a word per warp; the caller alternates two such arrays, so that one
// barrier per sum is enough: a warp writes red[i] again only after the barrier of the sum in between, which
// every reader of red[i] has passed.
template <int GROUP>  // 0: the group is the whole CTA
__device__ __forceinline__ float group_sum(float v, float* red) {
    v = warp_sum<32>(v);
    if (GROUP == 0) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        return warp_sum<32>(lane < warps ? red[lane] : 0.0f);
    }
    if (GROUP == 32) return v;
    constexpr int kWarps = GROUP / 32 > 0 ? GROUP / 32 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = warp / kWarps;
    if (lane == 0) red[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(GROUP) : "memory");
    return warp_sum<32>(lane < kWarps ? red[g * kWarps + lane] : 0.0f);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Rows in registers: a row is nvec lane vectors, VPT per thread of its group.  AHEAD: rows whose loads are in
// flight behind the current one (their registers are named by an unrolled loop: a copy from one row's to the next
// would wait for the load).  RES: with a residual; without one two CTAs fit an SM.
template <typename T, int FMT, int BYTES, int VPT, int MAXT, int GROUP, int AHEAD = 1, bool RES = true, int ACCESS = BYTES>
__global__ void __launch_bounds__(MAXT, RES ? 0 : 2)
k_rmsnorm_quantize(RmsNormArgs p) {
    pdl_enter();
    using V = Vec<T, BYTES, ACCESS>;
    using W = typename V::W;
    using Out = typename LaneVec<T, BYTES>::Out;
    constexpr int E = V::kElems;
    constexpr int kLanes = 128 / E;  // lanes of one 1x128 block
    __shared__ float red[2][32];
    constexpr int kGroups = GROUP == 0 ? 1 : MAXT / GROUP, G = GROUP == 0 ? 1 : GROUP;
    const int tid = GROUP == 0 ? threadIdx.x : threadIdx.x % G, stride = GROUP == 0 ? blockDim.x : G;
    const int64_t first = GROUP == 0 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const int nvec = static_cast<int>(p.cols / E);
    const int64_t nblk = (p.cols + 127) >> 7;
    const W* x = static_cast<const W*>(p.x);
    const W* res = RES ? static_cast<const W*>(p.residual) : nullptr;

    float w[VPT][E];
    static_assert(AHEAD == 1 || GROUP == 0, "rows of a CTA end together");
    W xv[AHEAD][VPT], rv[AHEAD][VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int vec = tid + v * stride;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            xv[a][v] = rv[a][v] = V::zero();
            if (vec < nvec && first + a * step < p.rows) {
                xv[a][v] = V::load(x + (first + a * step) * nvec + vec);
                if (res != nullptr) rv[a][v] = V::load(res + (first + a * step) * nvec + vec);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) w[v][e] = vec < nvec ? load_w(p.weight, p.w_bf16, static_cast<int64_t>(vec) * E + e) : 0.0f;
    }
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    int parity = 0;
    for (int64_t row0 = first; row0 < p.rows; row0 += AHEAD * step)
#pragma unroll
    for (int a = 0; a < AHEAD; ++a, parity ^= 1) {
        const int64_t row = row0 + a * step;
        if (AHEAD > 1 && row >= p.rows) break;
        float f[VPT][E];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int vec = tid + v * stride;
            if (res != nullptr) {
                float t[E];
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] = __fadd_rn(V::get(xv[a][v], e), V::get(rv[a][v], e));
                const W hv = V::pack(t);
                if (vec < nvec) V::store(p.h, row * nvec + vec, hv);
#pragma unroll
                for (int e = 0; e < E; ++e) f[v][e] = V::get(hv, e);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) f[v][e] = V::get(xv[a][v], e);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) ss = __fmaf_rn(f[v][e], f[v][e], ss);
            const int64_t next = row + AHEAD * step;
            if (vec < nvec && next < p.rows) {
                xv[a][v] = V::load(x + next * nvec + vec);
                if (res != nullptr) rv[a][v] = V::load(res + next * nvec + vec);
            }
        }
        ss = group_sum<GROUP>(ss, red[parity]);
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

// Widths that are not whole vectors, element by element, a warp per 1x128 block (lane l has elements l,
// l + 32, ..).  Up to kHeld blocks a warp stay in registers with their weights (cols <= kHeldCols); a group
// of the fewest warps that hold a row takes it.
constexpr int kOddThreads = 512;
constexpr int kHeld = 4;
constexpr int64_t kHeldCols = kHeld * 128 * (kOddThreads / 32);

// One block's codes, scale and y from its values.
template <typename T, int FMT>
__device__ __forceinline__ void store_block(const RmsNormArgs& p, const float (&f)[4], float s, int64_t row, int64_t blk,
                                            int64_t nblk, int lane) {
    if (lane == 0) p.scales[row * nblk + blk] = s;
    const int64_t at = row * p.cols + blk * 128 + lane;
    const int64_t left = p.cols - blk * 128 - lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (32 * k < left) {
            p.q[at + 32 * k] = static_cast<uint8_t>(cvt_fp8x2<FMT>(__fmul_rn(f[k], s), 0.0f) & 0xFFu);
            if (p.y != nullptr) store_f(static_cast<T*>(p.y) + at + 32 * k, f[k]);
        }
    }
}

template <typename T, int FMT, int GROUP>  // the group's threads
__global__ void __launch_bounds__(GROUP < 256 ? 256 : GROUP, GROUP < 512 ? 2 : 1)
k_rmsnorm_quantize_odd(RmsNormArgs p) {
    pdl_enter();
    __shared__ float red[2][32];
    constexpr int warps = GROUP / 32, kGroups = GROUP < 256 ? 256 / GROUP : 1;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % warps;
    const int cols = static_cast<int>(p.cols), nblk = (cols + 127) >> 7;
    const int c0 = warp * 128 + lane, left = cols - c0;
    const T* x = static_cast<const T*>(p.x);
    const T* res = static_cast<const T*>(p.residual);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / GROUP;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    float w[kHeld][4];
    T xv[kHeld][4], rv[kHeld][4];  // the next row
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = j * warps * 128 + 32 * k;  // from this lane's first element
                const bool in = at < left && row < p.rows;
                // (plain loads: h may be written over either)
                xv[j][k] = in ? x[row * cols + c0 + at] : T(0);
                rv[j][k] = in && res != nullptr ? res[row * cols + c0 + at] : T(0);
            }
    };
    load(first);
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = j * warps * 128 + 32 * k;
            w[j][k] = at < left ? load_w(p.weight, p.w_bf16, c0 + at) : 0.0f;
        }
    int parity = 0;
    for (int64_t row = first; row < p.rows; row += step, parity ^= 1) {
        float f[kHeld][4];
        float ss = 0.0f;
        T* h = static_cast<T*>(p.h) + row * cols + c0;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[j][k] = load_f(&xv[j][k]);
                if (res != nullptr) {
                    const int at = j * warps * 128 + 32 * k;
                    f[j][k] = round_to<T>(__fadd_rn(f[j][k], load_f(&rv[j][k])));
                    if (at < left) store_f(h + at, f[j][k]);
                }
                ss = __fmaf_rn(f[j][k], f[j][k], ss);
            }
        load(row + step);
        ss = group_sum<GROUP>(ss, red[parity]);
        const float rstd = rsqrtf(__fmaf_rn(ss, inv_cols, p.eps));
        if (p.rstd != nullptr && warp == 0 && lane == 0) p.rstd[row] = rstd;
        float s[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            s[j] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[j][k] = __fmul_rn(__fmul_rn(f[j][k], rstd), w[j][k]);
                s[j] = fmaxf(s[j], fabsf(f[j][k]));
            }
        }
#pragma unroll
        for (int j = 0; j < kHeld; ++j) s[j] = scale_from_amax<FMT>(warp_max<32>(s[j]));
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (warp + j * warps < nblk) store_block<T, FMT>(p, f[j], s[j], row, warp + j * warps, nblk, lane);
    }
}

// Wider rows than the kernels above hold: a CTA per row, read twice (the second time from L2, each element
// by the lane that read and wrote it the first time).
template <typename T, int FMT>
__global__ void __launch_bounds__(kOddThreads)
k_rmsnorm_quantize_wide(RmsNormArgs p) {
    pdl_enter();
    __shared__ float red[2][32];
    constexpr int kWarps = kOddThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t nblk = (p.cols + 127) >> 7;
    const T* x = static_cast<const T*>(p.x);
    const T* res = static_cast<const T*>(p.residual);
    T* h = static_cast<T*>(p.h);
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
        const int64_t r0 = row * p.cols;
        float ss = 0.0f;
        for (int64_t b0 = warp; b0 < nblk; b0 += kWarps * kHeld) {
            float v[kHeld][4], r[kHeld][4];
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t c = (b0 + j * kWarps) * 128 + 32 * k + lane;
                    v[j][k] = c < p.cols ? load_f(x + r0 + c) : 0.0f;
                    r[j][k] = res != nullptr && c < p.cols ? load_f(res + r0 + c) : 0.0f;
                }
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t c = (b0 + j * kWarps) * 128 + 32 * k + lane;
                    if (res != nullptr) {
                        v[j][k] = round_to<T>(__fadd_rn(v[j][k], r[j][k]));
                        if (c < p.cols) store_f(h + r0 + c, v[j][k]);
                    }
                    ss = __fmaf_rn(v[j][k], v[j][k], ss);
                }
        }
        ss = group_sum<0>(ss, red[parity]);
        const float rstd = rsqrtf(__fmaf_rn(ss, inv_cols, p.eps));
        if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
        const T* src = res != nullptr ? h : x;
        for (int64_t blk = warp; blk < nblk; blk += kWarps) {
            float f[4];
            float amax = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = blk * 128 + 32 * k + lane;
                f[k] = c < p.cols ? __fmul_rn(__fmul_rn(load_f(src + r0 + c), rstd), load_w(p.weight, p.w_bf16, c)) : 0.0f;
                amax = fmaxf(amax, fabsf(f[k]));
            }
            store_block<T, FMT>(p, f, scale_from_amax<FMT>(warp_max<32>(amax)), row, blk, nblk, lane);
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// The weight gradient of a launch of one cluster: every CTA has its sums in shared memory; rank by rank they
// are added, each CTA a share of the columns.
__device__ __forceinline__ void cluster_dweight(const float* sums, int64_t cols, float* dweight) {
    __syncthreads();  // the groups meet
    umma::cluster_sync();
    const uint32_t base = umma::smem_u32(sums);
    const int step = kRanks * static_cast<int>(blockDim.x);
    for (int c = static_cast<int>(umma::cluster_ctarank() * blockDim.x + threadIdx.x); c < cols; c += step) {
        float v[kRanks];
#pragma unroll
        for (int r = 0; r < kRanks; ++r) {
            const uint32_t at = umma::mapa(base, static_cast<uint32_t>(r)) + static_cast<uint32_t>(4 * c);
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(at) : "memory");
        }
#pragma unroll
        for (int r = 1; r < kRanks; ++r) v[0] += v[r];
        dweight[c] = v[0];
    }
    __syncwarp();
    umma::cluster_sync();  // no CTA leaves while another may read its shared memory
}

// Each thread keeps the dw sums of its columns in registers; at the end the groups of a CTA add theirs, one
// after the other, into the CTA's row of the workspace.
template <typename T, int BYTES, int VPT, int MAXT, int GROUP, bool CLUSTER>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1024 / MAXT)
k_rmsnorm_backward(RmsNormBackwardArgs p) {
    pdl_enter();
    extern __shared__ __align__(16) float sums[];  // [cols] in a cluster
    using V = Vec<T, BYTES>;
    using W = typename V::W;
    constexpr int E = V::kElems;
    __shared__ float red[2][32];
    constexpr int kGroups = GROUP == 0 ? 1 : MAXT / GROUP, G = GROUP == 0 ? 1 : GROUP;
    const int tid = GROUP == 0 ? threadIdx.x : threadIdx.x % G, stride = GROUP == 0 ? blockDim.x : G;
    const int mine = GROUP == 0 ? 0 : threadIdx.x / G;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups + mine;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const int nvec = static_cast<int>(p.cols / E);
    const W* dy = static_cast<const W*>(p.dy);
    const W* h = static_cast<const W*>(p.h);
    const W* dh = static_cast<const W*>(p.dh);

    float w[VPT][E], dw[VPT][E];
    // dh is used behind the row's barrier, so its load may go out with the row itself, which takes fewer
    // registers.  Ahead with the others it is better only for wide bf16 rows (16384 x 7168: 154 us against 155;
    // 16384 x 1024 bf16: 33 against 29; 8192 x 7168 fp32, where it spills: 193 against 139).
    constexpr bool kAheadDh = sizeof(T) == 2 && GROUP == 0;
    W yv[VPT], hv[VPT], gv[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int vec = tid + v * stride;
        yv[v] = hv[v] = gv[v] = V::zero();
        if (vec < nvec && first < p.rows) {
            yv[v] = V::load(dy + first * nvec + vec);
            hv[v] = ld_words_stream(h + first * nvec + vec);
            if (kAheadDh && dh != nullptr) gv[v] = V::load(dh + first * nvec + vec);
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
            if (!kAheadDh && dh != nullptr && vec < nvec) cg[v] = V::load(dh + row * nvec + vec);
            const int64_t next = row + step;
            if (vec < nvec && next < p.rows) {
                yv[v] = V::load(dy + next * nvec + vec);
                hv[v] = ld_words_stream(h + next * nvec + vec);
                if (kAheadDh && dh != nullptr) gv[v] = V::load(dh + next * nvec + vec);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = __fmul_rn(V::get(ch[v], e), rstd);
                const float d = V::get(cy[v], e);
                dot = __fmaf_rn(__fmul_rn(d, w[v][e]), n, dot);
                dw[v][e] = __fmaf_rn(d, n, dw[v][e]);
            }
        }
        const float c = __fmul_rn(group_sum<GROUP>(dot, red[parity]), inv_cols);
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
    float* out = CLUSTER ? sums : p.partial + static_cast<int64_t>(blockIdx.x) * p.cols;
    for (int g = 0; g < kGroups; ++g) {
        if (g > 0) __syncthreads();  // the row so far is visible to this group
        if (g != mine) continue;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int vec = tid + v * stride;
            if (vec < nvec) {
#pragma unroll
                for (int k = 0; k < E / 4; ++k) {
                    float* o = out + static_cast<int64_t>(vec) * E + 4 * k;
                    if ((reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
                        float4 t = make_float4(dw[v][4 * k], dw[v][4 * k + 1], dw[v][4 * k + 2], dw[v][4 * k + 3]);
                        float4* o4 = reinterpret_cast<float4*>(o);
                        if (g > 0) t = make_float4(o4->x + t.x, o4->y + t.y, o4->z + t.z, o4->w + t.w);
                        *o4 = t;
                    } else {  // the caller's weight gradient, on a 4-byte boundary
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = g > 0 ? o[i] + dw[v][4 * k + i] : dw[v][4 * k + i];
                    }
                }
            }
        }
    }
    if constexpr (CLUSTER) cluster_dweight(sums, p.cols, p.dweight);
}

// Widths that are not whole vectors, element by element: a group of `group` threads takes the elements
// thread, thread + group, ... of a row, up to kOddElems each, with their weights and dw sums in registers.
// (16 elements a thread with the next row's loads ahead spill: 263 us against 132 at 4096 x 7001 bf16.)
constexpr int kOddElems = 8;
static_assert(kOddElems * 1024 == kHeldCols, "the odd widths that fit");
template <typename T, int GROUP, bool CLUSTER>
__global__ void __launch_bounds__(GROUP < 256 ? 256 : GROUP, GROUP < 256 ? 4 : 1024 / GROUP)
k_rmsnorm_backward_odd(RmsNormBackwardArgs p) {
    pdl_enter();
    extern __shared__ __align__(16) float sums[];  // [cols] in a cluster
    __shared__ float red[2][32];
    constexpr int kN = kOddElems;
    constexpr int kGroups = GROUP < 256 ? 256 / GROUP : 1;
    const int tid = threadIdx.x % GROUP, mine = threadIdx.x / GROUP;
    const int cols = static_cast<int>(p.cols);
    const int left = cols - tid;
    const T* dy = static_cast<const T*>(p.dy);
    const T* h = static_cast<const T*>(p.h);
    const T* dh = static_cast<const T*>(p.dh);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups + mine;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const float inv_cols = __frcp_rn(static_cast<float>(p.cols));
    float w[kN], dw[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        w[k] = k * GROUP < left ? load_w(p.weight, p.w_bf16, tid + k * GROUP) : 0.0f;
        dw[k] = 0.0f;
    }
    int parity = 0;
    for (int64_t row = first; row < p.rows; row += step, parity ^= 1) {
        const float rstd = __ldg(p.rstd + row);
        float n[kN], a[kN];
        float g[kN];
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const bool in = k * GROUP < left;
            const int64_t at = row * cols + tid;
            n[k] = in ? load_f(h + at + k * GROUP) : 0.0f;
            a[k] = in ? load_f(dy + at + k * GROUP) : 0.0f;
            g[k] = in && dh != nullptr ? load_f(dh + at + k * GROUP) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            n[k] = __fmul_rn(n[k], rstd);
            dw[k] = __fmaf_rn(a[k], n[k], dw[k]);
            a[k] = __fmul_rn(a[k], w[k]);
            dot = __fmaf_rn(a[k], n[k], dot);
        }
        const float cc = __fmul_rn(group_sum<GROUP>(dot, red[parity]), inv_cols);
        T* dx = static_cast<T*>(p.dx) + row * cols + tid;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (k * GROUP < left) store_f(dx + k * GROUP, __fmaf_rn(rstd, __fmaf_rn(-n[k], cc, a[k]), g[k]));
        }
    }
    if (p.partial == nullptr) return;
    float* out = CLUSTER ? sums : p.partial + static_cast<int64_t>(blockIdx.x) * p.cols;
    for (int g = 0; g < kGroups; ++g) {
        if (g > 0) __syncthreads();  // the row so far is visible to this group
        if (g != mine) continue;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const int c = tid + k * GROUP;
            if (c < cols) out[c] = g > 0 ? out[c] + dw[k] : dw[k];
        }
    }
    if constexpr (CLUSTER) cluster_dweight(sums, p.cols, p.dweight);
}

// Wider rows: a CTA per row, read twice; dw is summed in the CTA's workspace row (each element by one thread), in L2.
// One element a load, so far from HBM's rate: 4096 x 12288 bf16 286 us (22 %), fp32 339 (36 %); 16384 x 16384 bf16 1644.
template <typename T>
__global__ void __launch_bounds__(kOddThreads)
k_rmsnorm_backward_wide(RmsNormBackwardArgs p) {
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
        for (int64_t c = threadIdx.x; c < p.cols; c += kOddThreads) {
            const float n = __fmul_rn(load_f(h + r0 + c), rstd);
            const float d = load_f(dy + r0 + c);
            dot = __fmaf_rn(__fmul_rn(d, load_w(p.weight, p.w_bf16, c)), n, dot);
            if (out != nullptr) out[c] = __fmaf_rn(d, n, row == blockIdx.x ? 0.0f : out[c]);
        }
        const float cc = __fmul_rn(group_sum<0>(dot, red[parity]), inv_cols);
        for (int64_t c = threadIdx.x; c < p.cols; c += kOddThreads) {
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

// CTAs of `threads` threads that the current device holds at once.  The last answer is kept per kernel and
// device: programs repeat a width.
template <auto KERN>
int64_t resident(int threads) {
    static std::atomic<int> last[128];  // threads << 8 | CTAs per SM
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return device_sm_count();
    int v = last[dev].load(std::memory_order_relaxed);
    if ((v >> 8) != threads) {
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERN, threads, 0) != cudaSuccess || per_sm < 1) {
            (void)cudaGetLastError();
            per_sm = 1;
        }
        v = threads << 8 | std::min(per_sm, 255);
        last[dev].store(v, std::memory_order_relaxed);
    }
    return static_cast<int64_t>(v & 255) * device_sm_count();
}

// Persistent CTAs of `threads`, `groups` rows at a time: as many as the device holds, at most one per row group.
template <auto KERN>
cudaError_t launch_rows(const RmsNormArgs& p, int threads, int groups, cudaStream_t st) {
    const int64_t grid = std::min((p.rows + groups - 1) / groups, resident<KERN>(threads));
    return launch_kernel(KERN, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)), 0, st, p);
}
// The weight gradient of few rows comes from the launch itself, without a workspace: of one CTA for up to 2
// turns, else of one cluster of 8 whose sums meet in distributed shared memory.  Against one CTA and against a
// workspace and a second launch, bf16 with 4096 columns: 8 rows take 4.1 us (7.4 in one CTA), 16 rows 5.0 (4.6 in
// two launches) and 8.3 a call (12.5).  More rows are slower in the cluster (32: 6.6 us against 4.8), and the wide
// kernel's turns are long.
constexpr int kOneCtaTurns = 2, kOneLaunchTurns = kOneCtaTurns * kRanks;
template <auto KERN, auto CLUSTER_KERN>
cudaError_t launch_rows(const RmsNormBackwardArgs& p, int threads, int groups, int64_t* parts, cudaStream_t st) {
    constexpr bool kCluster = CLUSTER_KERN != KERN;
    const int64_t turns = (p.rows + groups - 1) / groups;
    RmsNormBackwardArgs args = p;
    *parts = 0;  // partial rows left to sum
    if (kCluster && p.dweight != nullptr && turns > kOneCtaTurns && turns <= kOneLaunchTurns) {
        args.partial = p.dweight;  // only told from null
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kRanks);
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = static_cast<size_t>(p.cols) * 4;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kRanks;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
#if FP8Q_PDL
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
#endif
        const cudaError_t e = cudaLaunchKernelEx(&cfg, CLUSTER_KERN, args);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    int64_t grid = 1;
    if (p.dweight != nullptr && turns <= (kCluster ? kOneCtaTurns : 1)) {
        args.partial = p.dweight;  // the one partial row
    } else {
        grid = std::min({rmsnorm_backward_partials(p.rows), turns, resident<KERN>(threads)});
        if (p.dweight != nullptr) *parts = grid;
    }
    return launch_kernel(KERN, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)), 0, st, args);
}

int round_up32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

// Rows of up to 128 vectors share CTAs of 256 threads, in groups of a power of two.
template <typename T, int FMT, int BYTES, int ACCESS = BYTES>
cudaError_t launch_forward_narrow(const RmsNormArgs& p, int64_t nvec, cudaStream_t st) {
    if (nvec <= 32) return launch_rows<k_rmsnorm_quantize<T, FMT, BYTES, 1, 256, 32, 1, true, ACCESS>>(p, 256, 8, st);
    if (nvec <= 64) return launch_rows<k_rmsnorm_quantize<T, FMT, BYTES, 1, 256, 64, 1, true, ACCESS>>(p, 256, 4, st);
    return launch_rows<k_rmsnorm_quantize<T, FMT, BYTES, 1, 256, 128, 1, true, ACCESS>>(p, 256, 2, st);
}

template <typename T, int FMT>
cudaError_t launch_forward(const RmsNormArgs& p, cudaStream_t st) {
    constexpr int E32 = 32 / static_cast<int>(sizeof(T)), E16 = E32 / 2;
    const bool aligned = aligned32(p.x) && aligned32(p.residual) && aligned32(p.h) && aligned32(p.y);
    if (p.cols % E32 == 0 && !aligned) {
        // The same vectors in two accesses each, so that a row's sums, and with them every output, do not depend on its
        // address.  Against vectors of 16 bytes, summed in another order: 16384 x 7168 bf16 184 us and 184, 16384 x 2048
        // 54 and 50, 8192 x 4096 fp32 without a residual 52 and 63, one row of 4096 3.0 and 2.4.
        const int64_t nvec = p.cols / E32;
        if (nvec <= 128) return launch_forward_narrow<T, FMT, 32, 16>(p, nvec, st);
        if (nvec <= 512)
            return launch_rows<k_rmsnorm_quantize<T, FMT, 32, 1, 512, 0, 1, true, 16>>(p, round_up32(nvec), 1, st);
        if (nvec <= 1024)
            return launch_rows<k_rmsnorm_quantize<T, FMT, 32, 2, 512, 0, 1, true, 16>>(p, round_up32((nvec + 1) / 2), 1, st);
    } else if (p.cols % E32 == 0) {
        const int64_t nvec = p.cols / E32;
        if (nvec <= 128) return launch_forward_narrow<T, FMT, 32>(p, nvec, st);
        if (nvec <= 512) {
            // Two rows ahead where that costs no CTA of an SM, or where two inputs make up for it: 16384 x 7168 bf16
            // 175 -> 172 us, 8192 x 4096 fp32 with a residual 96 -> 90; but 16384 x 2560 bf16 47 -> 48, 8192 x 4096
            // fp32 without 48 -> 60, and one row 2.8 -> 3.0.
            const bool two = p.rows > 4 * device_sm_count() && p.residual != nullptr && (sizeof(T) == 4 || nvec > 384);
            if (two) return launch_rows<k_rmsnorm_quantize<T, FMT, 32, 1, 512, 0, 2>>(p, round_up32(nvec), 1, st);
            // Without a residual 64 registers do, so that a row's serial chain (reduction, scale, codes) runs beside
            // another CTA's: 16384 x 7168 bf16 91 -> 67 us, 16384 x 4096 with y 65 -> 56.  (With one they spill: 175
            // -> 187.  fp32 takes fewer registers either way.)
            if (sizeof(T) == 2 && p.residual == nullptr)
                return launch_rows<k_rmsnorm_quantize<T, FMT, 32, 1, 512, 0, 1, false>>(p, round_up32(nvec), 1, st);
            return launch_rows<k_rmsnorm_quantize<T, FMT, 32, 1, 512, 0>>(p, round_up32(nvec), 1, st);
        }
        if (nvec <= 1024)
            return launch_rows<k_rmsnorm_quantize<T, FMT, 32, 2, 512, 0>>(p, round_up32((nvec + 1) / 2), 1, st);
    }
    if (p.cols % E16 == 0) {
        const int64_t nvec = p.cols / E16;
        if (nvec <= 128) return launch_forward_narrow<T, FMT, 16>(p, nvec, st);
        if (nvec <= 1024) return launch_rows<k_rmsnorm_quantize<T, FMT, 16, 1, 1024, 0>>(p, round_up32(nvec), 1, st);
        if (nvec <= 2048)
            return launch_rows<k_rmsnorm_quantize<T, FMT, 16, 2, 1024, 0>>(p, round_up32((nvec + 1) / 2), 1, st);
    }
    const int64_t warps = (p.cols + 128 * kHeld - 1) / (128 * kHeld);
    if (warps <= 1) return launch_rows<k_rmsnorm_quantize_odd<T, FMT, 32>>(p, 256, 8, st);
    if (warps <= 2) return launch_rows<k_rmsnorm_quantize_odd<T, FMT, 64>>(p, 256, 4, st);
    if (warps <= 4) return launch_rows<k_rmsnorm_quantize_odd<T, FMT, 128>>(p, 256, 2, st);
    if (warps <= 8) return launch_rows<k_rmsnorm_quantize_odd<T, FMT, 256>>(p, 256, 1, st);
    if (warps <= 16) return launch_rows<k_rmsnorm_quantize_odd<T, FMT, 512>>(p, 512, 1, st);
    return launch_rows<k_rmsnorm_quantize_wide<T, FMT>>(p, kOddThreads, 1, st);
}

template <typename T, int VPT, int MAXT, int GROUP>
cudaError_t launch_vectors(const RmsNormBackwardArgs& p, int threads, int groups, int64_t* parts, cudaStream_t st) {
    return launch_rows<k_rmsnorm_backward<T, 16, VPT, MAXT, GROUP, false>, k_rmsnorm_backward<T, 16, VPT, MAXT, GROUP, true>>(
        p, threads, groups, parts, st);
}
template <typename T, int GROUP>
cudaError_t launch_odd(const RmsNormBackwardArgs& p, int threads, int groups, int64_t* parts, cudaStream_t st) {
    return launch_rows<k_rmsnorm_backward_odd<T, GROUP, false>, k_rmsnorm_backward_odd<T, GROUP, true>>(p, threads, groups,
                                                                                                        parts, st);
}

template <typename T>
cudaError_t launch_backward(const RmsNormBackwardArgs& p, int64_t* parts, cudaStream_t st) {
    constexpr int E16 = 16 / static_cast<int>(sizeof(T));
    if (p.cols % E16 == 0) {
        const int64_t nvec = p.cols / E16;
        if (nvec <= 32) return launch_vectors<T, 1, 256, 32>(p, 256, 8, parts, st);
        if (nvec <= 64) return launch_vectors<T, 1, 256, 64>(p, 256, 4, parts, st);
        if (nvec <= 128) return launch_vectors<T, 1, 256, 128>(p, 256, 2, parts, st);
        if (nvec <= 512) return launch_vectors<T, 1, 512, 0>(p, round_up32(nvec), 1, parts, st);
        if (nvec <= 1024) return launch_vectors<T, 1, 1024, 0>(p, round_up32(nvec), 1, parts, st);
        if constexpr (sizeof(T) == 4) {  // bf16 vectors hold twice the elements: two a thread would spill
            const int threads = round_up32((nvec + 1) / 2);
            // 640 threads may have 96 registers each, 1024 only 64: 8192 x 4112 with dh takes 90.0 us against 91.0, 64 x
            // 4112 4.80 against 4.85; 8192 x 5120 104.1 either way.
            if (nvec <= 1280) return launch_vectors<T, 2, 640, 0>(p, threads, 1, parts, st);
            if (nvec <= 2048) return launch_vectors<T, 2, 1024, 0>(p, threads, 1, parts, st);
        }
    }
    const int64_t threads = (p.cols + kOddElems - 1) / kOddElems;
    if (threads <= 64) return launch_odd<T, 64>(p, 256, 4, parts, st);
    if (threads <= 128) return launch_odd<T, 128>(p, 256, 2, parts, st);
    if (threads <= 256) return launch_odd<T, 256>(p, 256, 1, parts, st);
    if (threads <= 512) return launch_odd<T, 512>(p, 512, 1, parts, st);
    if (threads <= 1024) return launch_odd<T, 1024>(p, 1024, 1, parts, st);
    return launch_rows<k_rmsnorm_backward_wide<T>, k_rmsnorm_backward_wide<T>>(p, kOddThreads, 1, parts, st);
}

}  // namespace

int64_t rmsnorm_backward_partials(int64_t rows) { return std::min<int64_t>(rows, device_sm_count() * 4); }

bool rmsnorm_backward_one_launch(int64_t rows, int64_t cols) {
    return rows <= (cols <= kHeldCols ? kOneLaunchTurns : 1);
}

cudaError_t launch_rmsnorm_quantize(const RmsNormArgs& p, int dtype, int fmt, cudaStream_t st) {
    if (dtype == 1)
        return fmt == kE4M3 ? launch_forward<uint16_t, kE4M3>(p, st) : launch_forward<uint16_t, kE5M2>(p, st);
    return fmt == kE4M3 ? launch_forward<float, kE4M3>(p, st) : launch_forward<float, kE5M2>(p, st);
}

cudaError_t launch_rmsnorm_backward(const RmsNormBackwardArgs& p, int dtype, cudaStream_t st) {
    int64_t parts = 0;
    const cudaError_t e = dtype == 1 ? launch_backward<uint16_t>(p, &parts, st) : launch_backward<float>(p, &parts, st);
    if (e != cudaSuccess || parts == 0) return e;
    return launch_kernel(k_rmsnorm_dweight, dim3(static_cast<unsigned>((p.cols + 31) / 32)), dim3(1024), 0, st,
                         static_cast<const float*>(p.partial), static_cast<int>(parts), p.cols, p.dweight);
}

}  // namespace fp8q
