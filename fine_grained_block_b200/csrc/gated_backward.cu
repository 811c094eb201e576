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
// A CTA takes a 128x128 tile, since a token-wise block is 128 tokens of a column
// and a row-wise one 128 columns of a row.  A lane has 4 columns of a row: a row's
// amax is one warp reduction (redux on |x|), and a column's maximum stays in its
// lane.  Bound by instructions (two exponentials' worth of arithmetic, three
// scaled casts and five maxima an element) as much as by HBM.  Two kernels:
// tiles, and row codes alone.

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "gemm_gated.h"
#include "lane_vec.cuh"
#include "launch_util.h"
#include "tensor_map.h"
#include "tile_transpose.cuh"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// 4 consecutive elements as they lie in memory.
template <typename T>
struct Quad {
    static constexpr int kWords = static_cast<int>(sizeof(T));
    alignas(4 * kWords) uint32_t w[kWords];
    __device__ __forceinline__ uint64_t pair(int k) const {  // elements 2k, 2k + 1
        if constexpr (sizeof(T) == 4) return f32x2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        else return f32x2(bf16_lo(w[k]), bf16_hi(w[k]));
    }
};
__device__ __forceinline__ Quad<uint16_t> load_quad(const uint16_t* p) {
    Quad<uint16_t> q;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(q.w[0]), "=r"(q.w[1]) : "l"(p));
    return q;
}
__device__ __forceinline__ Quad<float> load_quad(const float* p) {
    const uint4 v = ld_stream(reinterpret_cast<const uint4*>(p));
    return Quad<float>{{v.x, v.y, v.z, v.w}};
}
// A row's inputs at this lane's columns.
template <typename T>
struct Inputs {
    Quad<T> g, u, d;
    __device__ __forceinline__ void load(const T* gu, const T* dh, int64_t F, int64_t row, bool live) {
        if (live) {
            g = load_quad(gu + row * 2 * F);
            u = load_quad(gu + row * 2 * F + F);
            d = load_quad(dh + row * F);
        } else {
#pragma unroll
            for (int k = 0; k < Quad<T>::kWords; ++k) g.w[k] = u.w[k] = d.w[k] = 0u;
        }
    }
    // from a part of a slab, `stride` bytes from one input to the next
    __device__ __forceinline__ void shared(const uint8_t* src, int stride) {
        using W = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
        *reinterpret_cast<W*>(g.w) = *reinterpret_cast<const W*>(src);
        *reinterpret_cast<W*>(u.w) = *reinterpret_cast<const W*>(src + stride);
        *reinterpret_cast<W*>(d.w) = *reinterpret_cast<const W*>(src + 2 * stride);
    }
};

// dG, dU and H of a lane's 4 elements, as pairs.
template <int ACT, typename T>
__device__ __forceinline__ void gated_grads(const Inputs<T>& in, uint64_t (&dg)[2], uint64_t (&du)[2], uint64_t (&h)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint64_t u2 = in.u.pair(k), d2 = in.d.pair(k);
        uint64_t a2, da2;
        gate_act_grad2<ACT>(in.g.pair(k), a2, da2);
        dg[k] = mul_f32x2(mul_f32x2(d2, u2), da2);
        du[k] = mul_f32x2(d2, a2);
        h[k] = mul_f32x2(a2, u2);
    }
}

// 4 values times their scales -> 4 codes.
template <int FMT>
__device__ __forceinline__ uint32_t cast4(const uint64_t (&v)[2], uint64_t s01, uint64_t s23) {
    const float2 a = f32x2_split(mul_f32x2(v[0], s01)), b = f32x2_split(mul_f32x2(v[1], s23));
    return cvt_fp8x2<FMT>(a.x, a.y) | (cvt_fp8x2<FMT>(b.x, b.y) << 16);
}

__device__ __forceinline__ float row_absmax(const uint64_t (&v)[2]) {
    const float2 a = f32x2_split(v[0]), b = f32x2_split(v[1]);
    const float m = fmaxf(absmax3(a.x, a.y, b.x), fabsf(b.y));
    float r;
    asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}
// m = the larger of m and two rows' magnitudes, column by column
__device__ __forceinline__ void col_absmax(float (&m)[4], const uint64_t (&v)[2], const uint64_t (&w)[2]) {
    const float2 a = f32x2_split(v[0]), b = f32x2_split(v[1]), c = f32x2_split(w[0]), d = f32x2_split(w[1]);
    m[0] = absmax3(m[0], a.x, c.x);
    m[1] = absmax3(m[1], a.y, c.y);
    m[2] = absmax3(m[2], b.x, d.x);
    m[3] = absmax3(m[3], b.y, d.y);
}

// Row codes and scales of N rows (row0 ..; N a power of two up to 16) at this lane's 4 columns (col: from the row's
// first element).  FULL: all N rows exist.
template <int FMT, int N, bool FULL>
__device__ __forceinline__ void row_codes(const GatedBackwardArgs& p, const uint64_t (&dg)[N][2],
                                          const uint64_t (&du)[N][2], int64_t row0, int64_t col, int lane) {
    // lane l forms the scale of row l % N, of dG (l & N clear) or dU
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float ag = row_absmax(dg[i]), au = row_absmax(du[i]);
        if ((lane & (2 * N - 1)) == i) mine = ag;
        if ((lane & (2 * N - 1)) == i + N) mine = au;
    }
    const float s_mine = scale_from_amax<FMT>(mine);
    const int rows = FULL ? N : static_cast<int>(min(p.M - row0, static_cast<int64_t>(N)));
    const int64_t blocks = p.F / 128;
    if (lane < 2 * N && (FULL || (lane & (N - 1)) < rows))
        p.scales[(row0 + (lane & (N - 1))) * 2 * blocks + (lane & N ? blocks : 0) + col / 128] = s_mine;
    uint8_t* q = p.q + row0 * 2 * p.F + col;
#pragma unroll
    for (int i = 0; i < N; ++i, q += 2 * p.F) {
        const float sg = __shfl_sync(0xFFFFFFFFu, s_mine, i), su = __shfl_sync(0xFFFFFFFFu, s_mine, i + N);
        if (FULL || i < rows) {
            st_stream(reinterpret_cast<uint32_t*>(q), cast4<FMT>(dg[i], both(sg), both(sg)));
            st_stream(reinterpret_cast<uint32_t*>(q + p.F), cast4<FMT>(du[i], both(su), both(su)));
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles: one persistent CTA of 16 warps an SM, every element evaluated once
// ---------------------------------------------------------------------------
// A warp has 8 rows of the tile.  Its inputs come by TMA into its own slab of shared memory, in parts of 3 x 1 KiB
// (4 rows of bf16, 2 of fp32) for which the slab has two slots with an mbarrier each: a slot's next part is requested
// as soon as it is consumed, so that loads are in flight through the barriers and the write-out.  dG and dU of its 8 rows stay in
// registers (64), H as fp32 in shared memory, until the column scales are known: the evaluation, which is most
// of the instructions, is done once, and the inputs are read once.  The token-wise codes are converted two
// tokens of a column at a time and stored transposed, so that nothing is permuted on the way out.
// Measured at 16384 x 4096 bf16: 140-144 us on a card that rested between the calls, 151-157 held for a second
// (slabs in one part took 12 us more, in four 15).  By leaving parts out: the evaluation takes 82, the row codes 33, the
// column codes 23, the write-out 15; the four hardly overlap.  fp32 takes 181 us there, 97 % of the copy rate, and
// 7.9-8.7 at 1000 x 2048.
namespace tma {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = kTT / kWarps;                       // rows of a warp
constexpr int kSlots = 2;                                 // parts that a warp's slab holds
constexpr int kTensorBytes = 1024;                        // of one input in a part
constexpr int kPartBytes = 3 * kTensorBytes;
constexpr int kSlabBytes = kSlots * kPartBytes;
template <typename T>
constexpr int kPartRows = kTensorBytes / (kTT * static_cast<int>(sizeof(T)));
constexpr int kTileBytes = kTT * kTT;
struct Smem {
    static constexpr int kCode = 0;                                  // 3 code tiles
    static constexpr int kH = kCode + 3 * kTileBytes;                // H, fp32
    static constexpr int kSlab = kH + kTT * kTT * 4;
    static constexpr int kScales = kSlab + kWarps * kSlabBytes;      // column scales [tensor][column]
    static constexpr int kMax = kScales + 3 * kTT * 4;               // column maxima [tile parity][tensor][column]
    static constexpr int kBars = kMax + 2 * 3 * kTT * 4;
    static constexpr int kBytes = kBars + kWarps * kSlots * 8 + 128; // alignment slack
};
static_assert(Smem::kBytes <= 227 * 1024, "one CTA an SM");

// The code tiles are stored transposed: 128 tokens of a column in a row of 128 bytes.  A warp's 8 tokens of a
// column are one 8-byte piece; its place in the row is XORed so that the 16 lanes of a store, 4 columns apart,
// hit all banks: bits 2-4 of the column move 16-byte pieces, bit 5 swaps the halves of one.
__device__ __forceinline__ int piece_off(int c, int piece) {
    return c * kTT + ((piece * 8) ^ (((c >> 2) & 7) * 16) ^ (((c >> 5) & 1) * 8));
}

template <typename T, int FMT, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
k_gated_backward_tma(const __grid_constant__ CUtensorMap map_gu, const __grid_constant__ CUtensorMap map_dh,
                     const __grid_constant__ GatedBackwardArgs p, unsigned int* status) {
    constexpr int kRowsIn = kPartRows<T>, kParts = kRows / kRowsIn;  // parts of a tile
    constexpr int kUses = kParts / kSlots;                           // of a slot in a tile
    static_assert(kRowsIn % 2 == 0 && kParts % kSlots == 0, "rows go in pairs, slots in turn");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    unsigned int* col_max = reinterpret_cast<unsigned int*>(sm + Smem::kMax);
    float* col_scale = reinterpret_cast<float*>(sm + Smem::kScales);
    uint8_t* slab = sm + Smem::kSlab + warp * kSlabBytes;
    float* hrow = reinterpret_cast<float*>(sm + Smem::kH) + warp * kRows * kTT + 4 * lane;
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Smem::kBars) + warp * kSlots;
    // this lane's columns 4 lane + e: the XOR is the same for all four
    uint8_t* code = sm + Smem::kCode + piece_off(4 * lane, warp);

    const int tiles_c = static_cast<int>(p.F / kTT), tiles_r = static_cast<int>((p.M + kTT - 1) / kTT);
    const int64_t mt = static_cast<int64_t>(tiles_r) * kTT;
    const int tiles = tiles_r * tiles_c;  // the launcher sees that it fits
    if (lane == 0) {
        for (int q = 0; q < kSlots; ++q) umma::mbar_init(&bar[q], 1);
        umma::fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 2 * 3 * kTT; i += kThreads) col_max[i] = 0u;
    __syncthreads();
    pdl_enter();  // the inputs may come from the previous kernel

    auto request = [&](int tr, int c0, int q) {  // lane 0: part q of the warp's rows (rows from M on arrive as zeros)
        const int row = tr * kTT + warp * kRows + q * kRowsIn;
        uint64_t* b = &bar[q % kSlots];
        uint8_t* dst = slab + q % kSlots * kPartBytes;
        umma::mbar_arrive_expect_tx(b, kPartBytes);
        umma::tma_load_2d(dst, &map_gu, b, c0, row);
        umma::tma_load_2d(dst + kTensorBytes, &map_gu, b, static_cast<int>(p.F) + c0, row);
        umma::tma_load_2d(dst + 2 * kTensorBytes, &map_dh, b, c0, row);
    };
    const int grid = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
    int tr = first / tiles_c, c0 = (first - tr * tiles_c) * kTT;
    if (lane == 0)
        for (int q = 0; q < kSlots; ++q) request(tr, c0, q);

    uint32_t phase = 0;
    bool timed_out = false;
    for (int tile = first; tile < tiles; tile += grid, phase ^= 1u) {
        const int next = tile < tiles - grid ? tile + grid : -1;
        const int next_tr = next / tiles_c, next_c0 = (next - next_tr * tiles_c) * kTT;
        const int64_t row0 = static_cast<int64_t>(tr) * kTT + warp * kRows;
        bool ok = true;
        uint64_t dg[kRows][2], du[kRows][2];
        float cm[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cm[0][e] = cm[1][e] = cm[2][e] = 0.0f;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
            const uint32_t use = (phase * kUses + q / kSlots) & 1u;  // parity of the slot's uses
            ok = ok && umma::mbar_wait(&bar[q % kSlots], use, kWaitLimitNs);
            if (!ok) break;
#pragma unroll
            for (int i = q * kRowsIn; i < (q + 1) * kRowsIn; i += 2) {
                uint64_t h[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    Inputs<T> in;
                    in.shared(slab + q % kSlots * kPartBytes + ((i + j - q * kRowsIn) * kTT + 4 * lane) * sizeof(T),
                              kTensorBytes);
                    gated_grads<ACT, T>(in, dg[i + j], du[i + j], h[j]);
                    const float2 a = f32x2_split(h[j][0]), b = f32x2_split(h[j][1]);
                    *reinterpret_cast<float4*>(hrow + (i + j) * kTT) = make_float4(a.x, a.y, b.x, b.y);
                }
                col_absmax(cm[0], dg[i], dg[i + 1]);
                col_absmax(cm[1], du[i], du[i + 1]);
                col_absmax(cm[2], h[0], h[1]);
            }
            __syncwarp();
            if (lane == 0) {  // this part is consumed: its slot's next one
                if (q + kSlots < kParts) request(tr, c0, q + kSlots);
                else if (next >= 0) request(next_tr, next_c0, q + kSlots - kParts);
            }
        }
        if (ok) {
            // magnitudes order as their bits do, and the maximum does not depend on the order of the warps
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    atomicMax(col_max + phase * 3 * kTT + k * kTT + 32 * e + lane, __float_as_uint(cm[k][e]));
            if (row0 + kRows <= p.M) row_codes<FMT, kRows, true>(p, dg, du, row0, c0 + 4 * lane, lane);
            else row_codes<FMT, kRows, false>(p, dg, du, row0, c0 + 4 * lane, lane);
        }
        if (__syncthreads_or(!ok)) {
            timed_out = true;
            break;
        }
        if (threadIdx.x < 3 * kTT) {
            const int i = threadIdx.x, k = i / kTT, c = (i % 32) * 4 + (i % kTT) / 32;  // col_max: element-major
            const float m = __uint_as_float(col_max[phase * 3 * kTT + i]);
            col_max[phase * 3 * kTT + i] = 0u;  // for the tile after the next
            const float s = scale_from_amax<FMT>(m);
            col_scale[k * kTT + c] = s;
            if (k < 2 && p.scales_t != nullptr) p.scales_t[(k * p.F + c0 + c) * tiles_r + tr] = s;
            if (k == 2 && p.ht_scales != nullptr) p.ht_scales[static_cast<int64_t>(c0 + c) * tiles_r + tr] = s;
        }
        __syncthreads();
        // The codes with the column scales, two tokens of a column per conversion.
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float4 s = *reinterpret_cast<const float4*>(col_scale + k * kTT + 4 * lane);
            const uint64_t s01 = f32x2(s.x, s.y), s23 = f32x2(s.z, s.w);
            uint32_t c[4][2];  // [column][4 tokens]
#pragma unroll
            for (int i = 0; i < kRows; i += 2) {
                float2 v[2][2];  // [token][column pair]
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (k == 2) {
                        const float4 h = *reinterpret_cast<const float4*>(hrow + (i + j) * kTT);
                        v[j][0] = f32x2_split(mul_f32x2(f32x2(h.x, h.y), s01));
                        v[j][1] = f32x2_split(mul_f32x2(f32x2(h.z, h.w), s23));
                    } else {
                        v[j][0] = f32x2_split(mul_f32x2(k == 0 ? dg[i + j][0] : du[i + j][0], s01));
                        v[j][1] = f32x2_split(mul_f32x2(k == 0 ? dg[i + j][1] : du[i + j][1], s23));
                    }
                }
                const uint32_t t[4] = {cvt_fp8x2<FMT>(v[0][0].x, v[1][0].x), cvt_fp8x2<FMT>(v[0][0].y, v[1][0].y),
                                       cvt_fp8x2<FMT>(v[0][1].x, v[1][1].x), cvt_fp8x2<FMT>(v[0][1].y, v[1][1].y)};
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e][i / 4] = i % 4 == 0 ? t[e] : c[e][i / 4] | (t[e] << 16);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint2*>(code + k * kTileBytes + e * kTT) = make_uint2(c[e][0], c[e][1]);
        }
        __syncthreads();
        // Out: 8 lanes a column, whole lines.
        const int oc = warp * 4 + (lane >> 3);  // and 64 on
        const uint8_t* src = sm + Smem::kCode + oc * kTT + ((lane & 7) ^ ((oc >> 2) & 7)) * 16;
        const int64_t at = (static_cast<int64_t>(c0 + oc) * tiles_r + tr) * kTT + (lane & 7) * 16;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint8_t* dst = k < 2 ? p.qt : p.ht;
            if (dst == nullptr) continue;
            dst += k == 1 ? at + p.F * mt : at;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint4 v = *reinterpret_cast<const uint4*>(src + k * kTileBytes + half * 64 * kTT);
                if ((oc >> 5) & 1) v = make_uint4(v.z, v.w, v.x, v.y);
                st_stream(reinterpret_cast<uint4*>(half ? dst + 64 * mt : dst), v);
            }
        }
        tr = next_tr;
        c0 = next_c0;
    }
    if (timed_out) {
        if (threadIdx.x == 0) {
            atomicOr(status, kStatusWaitTimeout);
            // loads may still be landing in this CTA's shared memory: let them finish (bounded)
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
        __syncthreads();
    }
}

template <typename T, int FMT, int ACT>
cudaError_t launch(const GatedBackwardArgs& p, cudaStream_t st) {
    CUtensorMap map_gu, map_dh;
    constexpr auto make_map = sizeof(T) == 4 ? make_f32_tile_map : make_bf16_tile_map;
    if (!make_map(&map_gu, p.gu, p.M, 2 * p.F, kPartRows<T>, kTT) ||
        !make_map(&map_dh, p.dh, p.M, p.F, kPartRows<T>, kTT))
        return cudaErrorInvalidValue;
    unsigned int* status = device_status_word();
    if (status == nullptr) return cudaErrorInvalidValue;
    auto kern = k_gated_backward_tma<T, FMT, ACT>;
    static std::atomic<bool> opted[128];  // the shared-memory opt-in, once per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kBytes);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (p.M + kTT - 1) / kTT * (p.F / kTT);
    if (tiles > 0x7FFFFFFF - 1024) return cudaErrorInvalidValue;  // 3e13 elements
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tiles, device_sm_count())));
    return launch_kernel(kern, grid, dim3(kThreads), Smem::kBytes, st, map_gu, map_dh, p, status);
}

}  // namespace tma

// Row codes only (frozen weights): a warp per 4 rows of a block column, nothing shared.  Bound by HBM: 16384 x 4096 takes
// 88 us in bf16 (93 % of the copy rate) and 142 in fp32 (the copy rate), 200 x 4096 2.8, a launch.
template <typename T, int FMT, int ACT>
__global__ void __launch_bounds__(kThreads)
k_gated_backward_rows(GatedBackwardArgs p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const uint32_t blocks = static_cast<uint32_t>(p.F / 128);
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint32_t r4 = unit / blocks;
    const int64_t row0 = static_cast<int64_t>(r4) * 4, col = static_cast<int64_t>(unit - r4 * blocks) * 128 + 4 * lane;
    const T* gu = static_cast<const T*>(p.gu) + col;
    const T* dh = static_cast<const T*>(p.dh) + col;
    Inputs<T> in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i].load(gu, dh, p.F, row0 + i, row0 + i < p.M);
    uint64_t dg[4][2], du[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t h[2];
        gated_grads<ACT, T>(in[i], dg[i], du[i], h);
    }
    row_codes<FMT, 4, false>(p, dg, du, row0, col, lane);
}

template <typename T, int FMT, int ACT>
cudaError_t launch_typed(const GatedBackwardArgs& p, cudaStream_t st) {
    if (p.qt == nullptr && p.ht == nullptr) {
        const int64_t units = (p.M + 3) / 4 * (p.F / 128);
        const int64_t grid = (units + kWarps - 1) / kWarps;
        if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;
        return launch_kernel(k_gated_backward_rows<T, FMT, ACT>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                             st, p);
    }
    return tma::launch<T, FMT, ACT>(p, st);
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
