// gemm_grouped_wgrad.cu -- the gradients of the experts' weights: products over each expert's tokens.
//
//   dW[e][n][k] = sum over the expert's 128-token chunks c (offsets[e] / 128 .. offsets[e + 1] / 128 - 1) of
//                 P_c[n][k] / (sat[n][c] * sbt[k][c]),
//   P_c[n][k] = sum over tokens r in c of decode(At[n][r]) * decode(Bt[k][r])
// with At [N, R] and Bt [K, R] codes in 1x128 blocks along the rows.  An expert without rows gets zeros.
//
// The pipeline is that of gemm_blockwise.cu with 1x128 scales on both sides: a CTA takes 128 x 256 outputs, with a TMA
// producer, an MMA issuer, warps 2-3 with the reciprocal scales of the tile's columns in a ring, and 8 promotion warps.
// A tile's chunks are its expert's, so tiles differ in length; consecutive tiles are one expert's, whose rows of both
// operands stay in L2.  Results leave in boxes by TMA: a thread that writes its row's 16 bytes touches 32 lines a store,
// 6 us a tile.  ptxas spills 56 bytes of the promotion.
//
// Bound by the promotion beside shared memory: a chunk is two packed instructions for two results (512 cycles an SM) and
// 128 KB of column scales read from shared memory, next to the operands' 48 KB in and out; without the scales' product
// 2956 us, with it 3692 (8 experts with 65536 rows, 4096 x 1024, in pairs of CTAs).  8192 tokens, 8 of 32 experts,
// 4096 x 4096: 2830 us in pairs, 2323 with the boxes, 2084 with a CTA a tile.  Slower: a second box a warp (2218), 16
// promotion warps (3456), tiles of 192 columns that a thread reads whole (2578), both sides' scales by warps 2-3 (2558),
// two rows and 64 columns a thread, which halves the scales' reads (256 x 128 outputs a CTA: 2266),
// matrix fragments from tensor memory, which need a quarter of the scales' reads (4795: such loads run at a tenth of the
// rate).

#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gemm_gated.h"
#include "launch_util.h"
#include "moe.h"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kBM = 128;                  // rows of dW per CTA (TMEM lanes)
constexpr int kBN = 256;                  // columns of dW per tile (MMA N)
constexpr int kBK = 128;                  // tokens a chunk = one promotion = one stage
constexpr int kMmaK = 32;
constexpr int kThreads = 384;             // 3 warpgroups: control, promotion x2
constexpr int kABytes = kBM * kBK;
constexpr int kStageBytes = kABytes + kBN * kBK;  // rows of At and of Bt
constexpr int kStages = 3;
constexpr uint32_t kTmemCols = 2 * kBN;   // two accumulators
// The register split of the CTA's launch total (setmaxnreg): 3 x 168 = 56 + 2 x 224.
constexpr int kLaunchRegs = 168;
constexpr int kControlRegs = 56;
constexpr int kPromoteRegs = 224;
static_assert(kControlRegs + 2 * kPromoteRegs == 3 * kLaunchRegs, "register split must equal the launch total");
static_assert(kLaunchRegs * kThreads <= 65536, "launch registers exceed the register file");
constexpr int kRbSlots = 8;               // chunks whose reciprocal column scales are held
constexpr int kRbGroup = 4;               // chunks whose scales one fill round loads together
constexpr int kAhead = 2;                 // chunks ahead that a row's scales are loaded

struct Tail {  // behind the operand stages
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint64_t rb_full[kRbSlots];
    uint64_t rb_empty[kRbSlots];
    uint32_t tmem_base;
    alignas(16) float rb[kRbSlots][kBN];  // 1 / sbt of the tile's columns, by chunk
};
constexpr int kPromoteWarps = 8;
constexpr int kOutBox = 32 * 128;         // results on their way out, per promotion warp: 32 rows x 128 bytes
constexpr int kOutBytes = kPromoteWarps * kOutBox;
constexpr int kSmemBytes = kStages * kStageBytes + kOutBytes + 1024 /* alignment */ + static_cast<int>(sizeof(Tail));
static_assert(kSmemBytes <= 227 * 1024, "stages and barriers must fit in shared memory");

// Tile t: its expert, chunks and place.
struct Tile {
    int e, col, row, c0, c1;
    __device__ __forceinline__ Tile(const GroupedWgradArgs& p, uint32_t t, uint32_t tiles_r, uint32_t tiles_c) {
        const uint32_t per = tiles_r * tiles_c, r = t % per;
        e = static_cast<int>(t / per);
        row = static_cast<int>(r % tiles_r);
        col = static_cast<int>(r / tiles_r);
        const int R = static_cast<int>(p.R);
        c0 = min(max(__ldg(p.offsets + e), 0), R) / kBK;
        c1 = max(min(max(__ldg(p.offsets + e + 1), 0), R) / kBK, c0);
    }
};

template <int OUT>
__global__ void __launch_bounds__(kThreads, 1)
k_gemm_grouped_wgrad(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap map_dw, const __grid_constant__ GroupedWgradArgs p, uint32_t idesc,
                     unsigned int* status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* out = stages + kStages * kStageBytes;
    Tail* tail = reinterpret_cast<Tail*>(out + kOutBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t tiles_r = static_cast<uint32_t>(p.N / kBM);
    const uint32_t tiles_c = static_cast<uint32_t>((p.K + kBN - 1) / kBN);
    const uint32_t tiles = static_cast<uint32_t>(p.E) * tiles_r * tiles_c;
    const uint32_t first = blockIdx.x, step = gridDim.x;
    const int64_t kc_stride = p.R / kBK;  // scales per row of sat / sbt

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            umma::mbar_init(&tail->full[s], 1);
            umma::mbar_init(&tail->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            umma::mbar_init(&tail->acc_full[b], 1);
            umma::mbar_init(&tail->acc_empty[b], kPromoteWarps);
        }
        umma::mbar_init(&tail->mma_done, 1);
        for (int r = 0; r < kRbSlots; ++r) {
            umma::mbar_init(&tail->rb_full[r], 2);   // warps 2 and 3
            umma::mbar_init(&tail->rb_empty[r], kPromoteWarps);
        }
        umma::fence_mbar_init();
    }
    if (warp == 1) umma::tmem_alloc(&tail->tmem_base, kTmemCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tail->tmem_base;
    pdl_enter();  // the codes, scales and offsets may come from the previous kernel

    bool timed_out = false;
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0) {
        // ---- TMA producer ----------------------------------------------------
        if (lane == 0) {
            uint32_t g = 0;
            for (uint32_t t = first; t < tiles && !timed_out; t += step) {
                const Tile c(p, t, tiles_r, tiles_c);
                const int m0 = c.row * kBM;
                const int n0 = c.col * kBN;
                for (int kc = c.c0; kc < c.c1; ++kc, ++g) {
                    const uint32_t s = g % kStages;
                    if (!umma::mbar_wait(&tail->empty[s], ((g / kStages) & 1u) ^ 1u, kWaitLimitNs)) {
                        timed_out = true;
                        break;
                    }
                    uint8_t* stage = stages + s * kStageBytes;
                    umma::mbar_arrive_expect_tx(&tail->full[s], kStageBytes);
                    umma::tma_load_2d(stage, &map_a, &tail->full[s], kc * kBK, m0);
                    umma::tma_load_2d(stage + kABytes, &map_b, &tail->full[s], kc * kBK, n0);
                }
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer ----------------------------------------------------------
        if (lane == 0) {
            uint32_t g = 0;
            for (uint32_t t = first; t < tiles && !timed_out; t += step) {
                const Tile c(p, t, tiles_r, tiles_c);
                for (int kc = c.c0; kc < c.c1; ++kc, ++g) {
                    const uint32_t s = g % kStages;
                    const uint32_t buf = g & 1u;
                    if (!umma::mbar_wait(&tail->acc_empty[buf], ((g >> 1) & 1u) ^ 1u, kWaitLimitNs) ||
                        !umma::mbar_wait(&tail->full[s], (g / kStages) & 1u, kWaitLimitNs)) {
                        timed_out = true;
                        break;
                    }
                    umma::fence_after_sync();
                    const uint32_t a_addr = umma::smem_u32(stages + s * kStageBytes);
                    const uint64_t a_desc = umma::smem_desc_kmajor_sw128(a_addr);
                    const uint64_t b_desc = umma::smem_desc_kmajor_sw128(a_addr + kABytes);
                    const uint32_t d = tmem + buf * static_cast<uint32_t>(kBN);
#pragma unroll
                    for (int k = 0; k < kBK / kMmaK; ++k) umma::mma_f8f6f4(d, a_desc + 2 * k, b_desc + 2 * k, idesc, k > 0);
                    umma::commit(&tail->empty[s]);
                    umma::commit(&tail->acc_full[buf]);
                }
            }
            umma::commit(&tail->mma_done);
            if (!umma::mbar_wait(&tail->mma_done, 0, kWaitLimitNs)) timed_out = true;
        }
    } else if (warp < 4) {
        // ---- reciprocal column scales, warps 2-3 --------------------------------
        // A round loads the scales of up to kRbGroup chunks, groups at multiples of kRbGroup, with one 16-byte load
        // per column where every group starts on a 16-byte boundary; then waits for their ring slots.
        const int ft = (warp - 2) * 32 + lane;  // 0..63; columns ft + 64 i of the tile
        const bool vec4 = (kc_stride % kRbGroup) == 0 && (reinterpret_cast<uintptr_t>(p.sbt) & 15u) == 0;
        uint32_t g = 0;
        for (uint32_t t = first; t < tiles && !timed_out; t += step) {
            const Tile c(p, t, tiles_r, tiles_c);
            const float* sb[kBN / 64];
#pragma unroll
            for (int i = 0; i < kBN / 64; ++i)  // columns past K: any scale will do
                sb[i] = p.sbt + min(static_cast<int64_t>(c.col) * kBN + ft + 64 * i, p.K - 1) * kc_stride;
            for (int kc0 = c.c0; kc0 < c.c1 && !timed_out;) {
                const int cnt = min(kRbGroup - kc0 % kRbGroup, c.c1 - kc0);
                float v[kRbGroup][kBN / 64];
                if (vec4 && cnt == kRbGroup) {
#pragma unroll
                    for (int i = 0; i < kBN / 64; ++i) {
                        const float4 w = __ldg(reinterpret_cast<const float4*>(sb[i] + kc0));
                        v[0][i] = w.x;
                        v[1][i] = w.y;
                        v[2][i] = w.z;
                        v[3][i] = w.w;
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < kRbGroup; ++u)
#pragma unroll
                        for (int i = 0; i < kBN / 64; ++i) v[u][i] = (u < cnt) ? __ldg(sb[i] + kc0 + u) : 1.0f;
                }
#pragma unroll
                for (int u = 0; u < kRbGroup; ++u) {
                    if (u >= cnt) break;
                    const uint32_t slot = (g + u) % kRbSlots;
                    if (!umma::mbar_wait(&tail->rb_empty[slot], (((g + u) / kRbSlots) & 1u) ^ 1u, kWaitLimitNs)) {
                        timed_out = true;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < kBN / 64; ++i) tail->rb[slot][ft + 64 * i] = __frcp_rn(v[u][i]);
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(&tail->rb_full[slot]);
                }
                g += static_cast<uint32_t>(cnt);
                kc0 += cnt;
            }
        }
    } else {
        // ---- promotion warps -------------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPromoteRegs));
        const int quarter = warp & 3;            // TMEM lanes this warp may access
        const int half = (warp - 4) >> 2;        // column half of the tile
        const int row = quarter * 32 + lane;     // row within this CTA's 128 = TMEM lane
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * 128);
        uint8_t* box = out + (warp - 4) * kOutBox;
        uint32_t g = 0;
        for (uint32_t t = first; t < tiles && !timed_out; t += step) {
            const Tile c(p, t, tiles_r, tiles_c);
            const int64_t m = static_cast<int64_t>(c.row) * kBM + row;
            const int64_t col0 = static_cast<int64_t>(c.col) * kBN + half * 128;
            const bool live = col0 < p.K;  // the last tile may have one half
            // N is a multiple of 128, so the clamp changes no index; without it ptxas shares the registers out differently
            // (8192 tokens, 8 of 32 experts, 4096 x 4096: 2145 us against 2050)
            const float* sa_row = p.sat + min(m, p.N - 1) * kc_stride;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
            float sa_q[kAhead];
#pragma unroll
            for (int d = 0; d < kAhead; ++d) sa_q[d] = c.c0 + d < c.c1 ? __ldg(sa_row + c.c0 + d) : 1.0f;
            for (int kc = c.c0; kc < c.c1; ++kc, ++g) {
                const uint32_t buf = g & 1u;
                const float f = __frcp_rn(sa_q[0]);
#pragma unroll
                for (int d = 0; d + 1 < kAhead; ++d) sa_q[d] = sa_q[d + 1];
                if (kc + kAhead < c.c1) sa_q[kAhead - 1] = __ldg(sa_row + kc + kAhead);
                const uint32_t slot = g % kRbSlots;
                if (!umma::mbar_wait(&tail->acc_full[buf], (g >> 1) & 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                umma::fence_after_sync();
                const uint32_t tm = t_lane + buf * static_cast<uint32_t>(kBN);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[64];
                    umma::tmem_ld32(tm + h * 64, v);
                    umma::tmem_ld32(tm + h * 64 + 32, v + 32);
                    umma::wait_ld(v);
                    umma::hold_after_wait(v + 32);
                    if (h == 1) {  // every partial sum of this buffer is in registers: hand it back
                        umma::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(&tail->acc_empty[buf]);
                    }
                    if (h == 0 && !umma::mbar_wait(&tail->rb_full[slot], (g / kRbSlots) & 1u, kWaitLimitNs)) {
                        timed_out = true;
                        break;
                    }
                    // RN(p * 1/sat), then fma(that, 1/sbt, acc), two elements an instruction
                    const float4* rb = reinterpret_cast<const float4*>(&tail->rb[slot][half * 128 + h * 64]);
                    const uint64_t f2 = f32x2(f, f);
#pragma unroll
                    for (int j4 = 0; j4 < 16; ++j4) {
                        const float4 r = rb[j4];
                        float* a = acc + h * 64 + 4 * j4;
                        const float2 lo = f32x2_split(
                            fma_f32x2(mul_f32x2(f32x2(v[4 * j4], v[4 * j4 + 1]), f2), f32x2(r.x, r.y), f32x2(a[0], a[1])));
                        const float2 hi = f32x2_split(
                            fma_f32x2(mul_f32x2(f32x2(v[4 * j4 + 2], v[4 * j4 + 3]), f2), f32x2(r.z, r.w), f32x2(a[2], a[3])));
                        a[0] = lo.x;
                        a[1] = lo.y;
                        a[2] = hi.x;
                        a[3] = hi.y;
                    }
                    if (h == 1) {
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(&tail->rb_empty[slot]);
                    }
                }
                if (timed_out) break;
            }
            // Results leave in boxes of the warp's 32 rows x 128 bytes, in the swizzle that the tensor map names; all or
            // none of a box lies inside, because N and K are multiples of 128.
            if (timed_out || !live) continue;
            const int out_y = static_cast<int>(c.e * p.N + m) - lane;
            constexpr int kBoxCols = OUT == 0 ? 32 : 64;
#pragma unroll
            for (int b = 0; b < 128 / kBoxCols; ++b) {
                if (lane == 0) umma::tma_store_wait_read();  // the box before
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float* a = acc + b * kBoxCols + j * (kBoxCols / 8);
                    uint4 w;
                    if (OUT == 0)
                        w = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
                    else
                        w = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                                       pack_bf16x2(a[6], a[7]));
                    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) * 16)) = w;
                }
                umma::fence_to_async();
                __syncwarp();
                if (lane == 0) umma::tma_store_2d(&map_dw, box, static_cast<int>(col0) + b * kBoxCols, out_y);
            }
        }
        // the boxes are written before the CTA's shared memory goes away and the grid ends
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (timed_out) atomicOr(status, kStatusWaitTimeout);
    umma::fence_before_sync();
    if (__syncthreads_or(timed_out)) {
        // A wait ran out: give copies that may still be landing in this CTA's shared memory time to
        // finish (bounded) before it goes away.
        if (threadIdx.x == 0) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
        __syncthreads();
    }
    if (warp == 1) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, kTmemCols);
    }
}

// R == 0: every sum is empty.
__global__ void k_zero16(uint4* p, int64_t n) {
    pdl_enter();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        p[i] = make_uint4(0, 0, 0, 0);
}

template <int OUT>
cudaError_t launch_typed(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_dw,
                         const GroupedWgradArgs& p, uint32_t idesc, unsigned int* status, cudaStream_t st) {
    auto kern = k_gemm_grouped_wgrad<OUT>;
    static std::atomic<bool> opted[128];  // the shared-memory opt-in, once per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (p.N / kBM) * ((p.K + kBN - 1) / kBN) * p.E;
    if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(tiles, device_sm_count()));
    return launch_kernel(kern, dim3(ctas), dim3(kThreads), kSmemBytes, st, map_a, map_b, map_dw, p, idesc, status);
}

}  // namespace

cudaError_t launch_gemm_grouped_wgrad(const GroupedWgradArgs& p, cudaStream_t st) {
    if (p.R == 0) {
        const int64_t n = p.E * p.N * p.K * (p.dw_dtype == 0 ? 4 : 2) / 16;
        return launch_kernel(k_zero16, dim3(static_cast<unsigned>(device_sm_count() * 4)), dim3(256), 0, st,
                             static_cast<uint4*>(p.dw), n);
    }
    CUtensorMap map_a, map_b, map_dw;
    const bool f32 = p.dw_dtype == 0;
    if (!make_out_map(&map_dw, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f32 ? 4 : 2,
                      CU_TENSOR_MAP_SWIZZLE_128B, p.dw, p.E * p.N, p.K, f32 ? 32 : 64))
        return cudaErrorInvalidValue;
    if (!make_code_map(&map_a, p.at, p.N, p.R, kBM) || !make_code_map(&map_b, p.bt, p.K, p.R, kBN))
        return cudaErrorInvalidValue;
    unsigned int* status = device_status_word();
    if (status == nullptr) return cudaErrorInvalidValue;
    const uint32_t idesc = umma::instr_desc_f8f6f4(p.a_fmt, p.b_fmt, kBM, kBN);
    return f32 ? launch_typed<0>(map_a, map_b, map_dw, p, idesc, status, st)
               : launch_typed<1>(map_a, map_b, map_dw, p, idesc, status, st);
}

}  // namespace fp8q
