// gemm_gated.cu -- the gated feed-forward projections in one kernel: two FP8
// GEMMs over the same activations, the activation, the product, and the FP8
// quantization of the result.
//
//   G = A Wg^T, U = A Wu^T   (block scales applied in fp32 every 128 products,
//                             as in gemm_blockwise.cu)
//   H[m][f] = act(G[m][f]) * U[m][f]
//   s[m][j] = MAX / max(amax of H[m] over block j, eps), q = fp8(RN_f32(H * s))
// with B = [Wg; Wu] as one [2F, K] operand.  H never leaves the chip in high
// precision: what goes to memory is its codes (1 byte an element instead of
// the 2 written, 4 read and 1 written of a bf16 G|U, an activation kernel and
// a quantizer), and the projections themselves only where the backward pass
// asks for them.
//
// The tile is 256 rows x 128 columns of H by a CTA pair.  A pair's MMA has
// N 256, of which each CTA holds 128 rows of B: the even CTA brings the gate
// rows f0.., the odd one the up rows F + f0.., so that accumulator columns
// 0-127 are G and 128-255 are U of the same 128 columns of H -- one 1x128
// block a row.  Roles and pipeline are those of gemm_blockwise.cu (TMA producer,
// MMA issuer, 8 promotion warps, two accumulators, register split), and warps
// 2-3 form the dequant factors; here a promotion thread owns one row and 64
// columns of both G and U, so the activation and the product stay in its
// registers.  The block's amax is the
// larger of two threads' (the two column halves of a row), exchanged through
// shared memory by a two-warp mbarrier; the exchange slots alternate by tile
// parity: a warp writes a slot again only after the barrier of the tile in
// between, which its partner passes after reading the slot.  Results leave
// through shared memory by TMA, in boxes of the warp's own 32 rows x 64 columns
// (no barrier), so that the stores run beside the next tile's promotion.
//
// Few tiles leave pairs idle: then two pairs share a tile, each with half of K (SPLIT).
//
// Bound by the accumulators' way out of tensor memory, as gemm_blockwise.cu:
// 0.60 us a chunk, of which the MMAs are 0.28.  Beside its chunks a tile takes 3.0 us
// (16384 tokens, F 4096, the intercept over K from 256 to 2048), 1.5 with the
// projections alone and 2.1 with the codes alone: the epilogue, as far as the MMAs,
// two chunks ahead, do not cover it.  Of the codes' part the activation's two
// special-function operations an element are 1.04 us (16 a clock and SM); what the rest
// waits for is not shown.
// Measured at 16384 x 7168 x 4096: 1029-1041 us with the projections kept in bf16
// (1850-1870 TFLOP/s) on a card that rested between the calls, 1183-1213 when calls
// are held for a second (power cap), 992 without the projections and 1192 with them in
// fp32; in turn with it, fp8_gemm_blockwise takes 1046 us for the projections alone.

#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "gemm_gated.h"
#include "launch_util.h"
#include "tensor_map.h"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kBM = 128;                  // rows of H per CTA (TMEM lanes)
constexpr int kTileM = 2 * kBM;           // per pair
constexpr int kTileF = 128;               // columns of H per tile
constexpr int kBN = 2 * kTileF;           // MMA N: gate columns, then up columns
constexpr int kBK = 128;                  // K chunk = one promotion = one stage
constexpr int kMmaK = 32;
constexpr int kThreads = 384;             // 3 warpgroups: control, promotion x2
constexpr int kABytes = kBM * kBK;
constexpr int kStageBytes = 2 * kABytes;  // A rows and this CTA's 128 rows of B
constexpr int kStages = 4;
constexpr uint32_t kTmemCols = 2 * kBN;   // two accumulators
// The register split of the CTA's launch total (setmaxnreg): 3 x 168 = 56 + 2 x 224.
constexpr int kLaunchRegs = 168;
constexpr int kControlRegs = 56;
constexpr int kPromoteRegs = 224;
static_assert(kControlRegs + 2 * kPromoteRegs == 3 * kLaunchRegs, "register split must equal the launch total");
static_assert(kLaunchRegs * kThreads <= 65536, "launch registers exceed the register file");
// Rows of tiles that are walked together: a wave of 74 tiles then takes 16 x 5, whose operands stay in L2 beside the next
// ones.  16384 x 7168 x 4096: 1029 us and, held for seconds at the power cap, 1183 a call; 1042 and 1215 with 4, 1033 and
// 1196 with 8, 1038 and 1209 with 24, 1162 and 1341 with all 64; 1047 and 1262 row by row (0.84 GB read from DRAM).
constexpr uint32_t kGroup = 16;
constexpr int kFacSlots = 4;              // chunks whose dequant factors are held

struct Tail {  // behind the operand stages
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint64_t amax_bar[4];     // one per quarter: its two promotion warps
    uint32_t tmem_base;
    float amax[2][2][kBM];    // [tile parity][column half][row]
    alignas(16) float2 fac[kFacSlots][kBM];  // 1 / (sa * sg), 1 / (sa * su) of a row and chunk
};
// Results on their way out, per promotion warp: 32 rows x 64 columns of G and of U in bf16 and of codes.
constexpr int kOutGu = 32 * 64 * 2;
constexpr int kOutQ = 32 * 64;
constexpr int kPromoteWarps = 8;
constexpr int kOutBytes = kPromoteWarps * (2 * kOutGu + kOutQ);
constexpr int kSmemBytes = kStages * kStageBytes + kOutBytes + 1024 /* alignment */ + static_cast<int>(sizeof(Tail));
static_assert(kSmemBytes <= 227 * 1024, "stages and barriers must fit in shared memory");

// A box of this warp's staged results to the tensor at (x, y); rows past its end are not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(umma::smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's earlier stores have read their shared memory.
__device__ __forceinline__ void tma_store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
// Shared-memory writes of this thread become visible to the copy engine.
__device__ __forceinline__ void fence_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// SPLIT: a cluster of two CTA pairs takes one tile, each pair half of K.
template <int FMT, int ACT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
k_gemm_gated(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
             const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_gu,
             const __grid_constant__ GatedArgs p, uint32_t idesc, unsigned int* status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* out = stages + kStages * kStageBytes;
    Tail* tail = reinterpret_cast<Tail*>(out + kOutBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t cta = umma::cluster_ctarank();
    const uint32_t rank = SPLIT ? cta & 1u : cta;   // 0: this CTA issues the pair's MMAs
    const uint32_t even = SPLIT ? cta & ~1u : 0u;   // the pair's even CTA
    const int64_t tiles_f = p.F / kTileF;
    const uint32_t tf = static_cast<uint32_t>(tiles_f), tiles_m = static_cast<uint32_t>((p.M + kTileM - 1) / kTileM);
    const uint32_t tiles = tiles_m * tf;  // the launcher sees that it fits
    // Tiles go by groups of kGroup rows of tiles, column by column within a group.
    auto tile_at = [&](uint32_t t, int64_t& row, int64_t& col) {
        const uint32_t in_group = kGroup * tf, g0 = t / in_group, r = t - g0 * in_group;
        const uint32_t height = min(kGroup, tiles_m - g0 * kGroup);
        col = r / height;
        row = g0 * kGroup + (r - static_cast<uint32_t>(col) * height);
    };
    const uint32_t first = blockIdx.x / (SPLIT ? 4 : 2);
    const uint32_t step = SPLIT ? tiles : gridDim.x / 2;
    const int all_chunks = static_cast<int>(p.K / kBK);
    const int c0 = SPLIT && cta >= 2 ? all_chunks / 2 : 0;  // this pair's chunks
    const int nchunks = SPLIT ? (cta >= 2 ? all_chunks - c0 : all_chunks / 2) : all_chunks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            umma::mbar_init(&tail->full[s], 1);
            umma::mbar_init(&tail->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            umma::mbar_init(&tail->acc_full[b], 3);  // the MMAs and the two factor warps
            umma::mbar_init(&tail->acc_empty[b], 16);  // both CTAs' promotion warps
        }
        umma::mbar_init(&tail->mma_done, 1);
        for (int q = 0; q < 4; ++q) umma::mbar_init(&tail->amax_bar[q], 2);
        umma::fence_mbar_init();
    }
    if (warp == 1) umma::tmem_alloc_pair(&tail->tmem_base, kTmemCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::cluster_sync();  // the peer's barriers are initialised before any remote arrival
    umma::fence_after_sync();
    const uint32_t tmem = tail->tmem_base;
    pdl_enter();  // the codes and scales may come from the previous kernel

    bool timed_out = false;
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0) {
        // ---- TMA producer ----------------------------------------------------
        if (lane == 0) {
            uint32_t g = 0;
            for (uint32_t t = first; t < tiles && !timed_out; t += step) {
                int64_t tr, tc;
                tile_at(t, tr, tc);
                const int m0 = static_cast<int>(tr * kTileM + rank * kBM);
                const int n0 = static_cast<int>(tc * kTileF + rank * p.F);  // gate rows, or up rows
                for (int kc = 0; kc < nchunks; ++kc, ++g) {
                    const uint32_t s = g % kStages;
                    if (!umma::mbar_wait(&tail->empty[s], ((g / kStages) & 1u) ^ 1u, kWaitLimitNs)) {
                        timed_out = true;
                        break;
                    }
                    uint8_t* stage = stages + s * kStageBytes;
                    // both CTAs' copies complete on the even CTA's barrier
                    const uint32_t full0 = umma::mapa(umma::smem_u32(&tail->full[s]), even);
                    if (rank == 0) umma::mbar_arrive_expect_tx(&tail->full[s], 2 * kStageBytes);
                    umma::tma_load_2d_pair(stage, &map_a, full0, (c0 + kc) * kBK, m0);
                    umma::tma_load_2d_pair(stage + kABytes, &map_b, full0, (c0 + kc) * kBK, n0);
                }
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer (the even CTA) -----------------------------------------
        if (lane == 0 && rank == 0) {
            const uint32_t peer_empty0 = umma::mapa(umma::smem_u32(&tail->empty[0]), even + 1);
            const uint32_t peer_accf0 = umma::mapa(umma::smem_u32(&tail->acc_full[0]), even + 1);
            uint32_t g = 0;
            for (uint32_t t = first; t < tiles && !timed_out; t += step) {
                for (int kc = 0; kc < nchunks; ++kc, ++g) {
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
                    for (int k = 0; k < kBK / kMmaK; ++k)
                        umma::mma_f8f6f4_pair(d, a_desc + 2 * k, b_desc + 2 * k, idesc, k > 0);
                    umma::commit_pair(umma::smem_u32(&tail->empty[s]));
                    umma::commit_pair(peer_empty0 + s * static_cast<uint32_t>(sizeof(uint64_t)));
                    umma::commit_pair(umma::smem_u32(&tail->acc_full[buf]));
                    umma::commit_pair(peer_accf0 + buf * static_cast<uint32_t>(sizeof(uint64_t)));
                }
            }
            umma::commit_pair(umma::smem_u32(&tail->mma_done));
            if (!umma::mbar_wait(&tail->mma_done, 0, kWaitLimitNs)) timed_out = true;
        }
    } else if (warp < 4) {
        // ---- dequant factors, warps 2-3 ------------------------------------------
        // Two rows a thread.  The factors of chunk g go to slot g % kFacSlots and complete the accumulator's
        // "full" barrier together with its MMAs: one wait covers both.  They are written once chunk g - 2, of
        // the same accumulator, is full (before that the arrival would count for it), which says that chunk
        // g - 4 has been promoted: its slot is free.
        const int r0 = (warp - 2) * 32 + lane;
        uint32_t g = 0;
        for (uint32_t t = first; t < tiles && !timed_out; t += step) {
            int64_t tr, tc;
            tile_at(t, tr, tc);
            const int64_t m0 = tr * kTileM + rank * kBM + r0;
            const float* sa0 = p.sa + std::min<int64_t>(m0, p.M - 1) * all_chunks + c0;  // rows past M: any factor will do
            const float* sa1 = p.sa + std::min<int64_t>(m0 + 64, p.M - 1) * all_chunks + c0;
            const float* sg = p.sb + tc * all_chunks + c0;
            const float* su = sg + tiles_f * all_chunks;
            float a0 = __ldg(sa0), a1 = __ldg(sa1), bg = __ldg(sg), bu = __ldg(su);
            for (int kc = 0; kc < nchunks; ++kc, ++g) {
                const float2 f0 = make_float2(__frcp_rn(__fmul_rn(a0, bg)), __frcp_rn(__fmul_rn(a0, bu)));
                const float2 f1 = make_float2(__frcp_rn(__fmul_rn(a1, bg)), __frcp_rn(__fmul_rn(a1, bu)));
                if (kc + 1 < nchunks) {
                    a0 = __ldg(sa0 + kc + 1);
                    a1 = __ldg(sa1 + kc + 1);
                    bg = __ldg(sg + kc + 1);
                    bu = __ldg(su + kc + 1);
                }
                if (g >= 2 && !umma::mbar_wait(&tail->acc_full[g & 1u], ((g - 2) >> 1) & 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                tail->fac[g % kFacSlots][r0] = f0;
                tail->fac[g % kFacSlots][r0 + 64] = f1;
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&tail->acc_full[g & 1u]);
            }
        }
    } else {
        // ---- promotion and epilogue ---------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPromoteRegs));
        const int quarter = warp & 3;            // TMEM lanes this warp may access
        const int half = (warp - 4) >> 2;        // columns 64 * half .. of G and of U
        const int row = quarter * 32 + lane;     // row within this CTA's 128 = TMEM lane
        const uint32_t acc_empty0 = umma::mapa(umma::smem_u32(&tail->acc_empty[0]), even);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * 64);
        const int64_t f_blocks = tiles_f;
        uint8_t* out_gu = out + (warp - 4) * 2 * kOutGu;
        uint8_t* out_q = out + kPromoteWarps * 2 * kOutGu + (warp - 4) * kOutQ;
        uint32_t g = 0, parity = 0;
        for (uint32_t t = first, turn = 0; t < tiles && !timed_out; t += step, ++turn) {
            int64_t tr, fb;                      // fb: 1x128 block of H
            tile_at(t, tr, fb);
            const int64_t m = tr * kTileM + rank * kBM + row;
            float acc[2][64];                    // G, U
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[0][j] = acc[1][j] = 0.0f;
            for (int kc = 0; kc < nchunks; ++kc, ++g) {
                const uint32_t buf = g & 1u;
                if (!umma::mbar_wait(&tail->acc_full[buf], (g >> 1) & 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                umma::fence_after_sync();
                const float2 f = tail->fac[g % kFacSlots][row];
                const float fac[2] = {f.x, f.y};
                const uint32_t tm = t_lane + buf * static_cast<uint32_t>(kBN);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[64];
                    umma::tmem_ld32(tm + h * kTileF, v);
                    umma::tmem_ld32(tm + h * kTileF + 32, v + 32);
                    umma::wait_ld(v);
                    umma::hold_after_wait(v + 32);
                    if (h == 1) {  // every partial sum of this buffer is in registers: hand it back
                        umma::fence_before_sync();
                        __syncwarp();
                        if (lane == 0)
                            umma::mbar_arrive_cluster(acc_empty0 + buf * static_cast<uint32_t>(sizeof(uint64_t)));
                    }
#pragma unroll
                    for (int j = 0; j < 64; ++j) acc[h][j] = __fmaf_rn(v[j], fac[h], acc[h][j]);
                }
            }
            if constexpr (SPLIT) {
                // The two pairs' sums meet in distributed shared memory: pair 0 finishes rows 0-63 of each CTA, pair
                // 1 the others, so a warp either gives its sums away or adds the other pair's to its own.  (Every
                // MMA of this pair has completed: the operand stages are free.)
                const bool keeps = quarter / 2 == static_cast<int>(cta / 2);
                float4* part = reinterpret_cast<float4*>(stages) + half * 16 * kBM + row;  // [4 columns][row]
                if (!keeps && !timed_out) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            part[(h * 32 + j) * kBM] =
                                make_float4(acc[h][4 * j], acc[h][4 * j + 1], acc[h][4 * j + 2], acc[h][4 * j + 3]);
                }
                __syncwarp();
                umma::cluster_sync();
                if (!keeps || timed_out) break;
                const uint32_t at = umma::mapa(umma::smem_u32(part), cta ^ 2u);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = umma::ld_cluster_f32x4(at + (h * 32 + j) * kBM * 16);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        acc[h][4 * j] += v[j].x;
                        acc[h][4 * j + 1] += v[j].y;
                        acc[h][4 * j + 2] += v[j].z;
                        acc[h][4 * j + 3] += v[j].w;
                    }
                }
            }
            if (timed_out) break;
            const bool live = m < p.M;
            const int out_x = static_cast<int>(fb * kTileF) + half * 64;
            const int out_y = static_cast<int>(m) - lane;  // the warp's first row
            if (lane == 0) tma_store_wait_read();          // the previous tile's boxes
            __syncwarp();
            if (p.gu != nullptr && p.gu_dtype != 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 8; ++j)  // 16-byte chunks, in the 128-byte swizzle that the tensor map names
                        *reinterpret_cast<uint4*>(out_gu + h * kOutGu + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                            make_uint4(pack_bf16x2(acc[h][8 * j], acc[h][8 * j + 1]),
                                       pack_bf16x2(acc[h][8 * j + 2], acc[h][8 * j + 3]),
                                       pack_bf16x2(acc[h][8 * j + 4], acc[h][8 * j + 5]),
                                       pack_bf16x2(acc[h][8 * j + 6], acc[h][8 * j + 7]));
                fence_to_async();
                __syncwarp();
                if (lane == 0 && out_y < p.M) {
                    tma_store_2d(&map_gu, out_gu, out_x, out_y);
                    tma_store_2d(&map_gu, out_gu + kOutGu, static_cast<int>(p.F) + out_x, out_y);
                }
            } else if (p.gu != nullptr && live) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.gu) + m * 2 * p.F + h * p.F + out_x);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        dst[j] = make_float4(acc[h][4 * j], acc[h][4 * j + 1], acc[h][4 * j + 2], acc[h][4 * j + 3]);
                }
            }
            if (p.q != nullptr) {
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    const uint64_t h2 = mul_f32x2(gate_act2<ACT>(f32x2(acc[0][j], acc[0][j + 1])),
                                                  f32x2(acc[1][j], acc[1][j + 1]));
                    const float2 h = f32x2_split(h2);
                    acc[0][j] = h.x;
                    acc[0][j + 1] = h.y;
                    amax = absmax3(amax, h.x, h.y);
                }
                const uint32_t slot = turn & 1u;
                tail->amax[slot][half][row] = amax;
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&tail->amax_bar[quarter]);
                if (!umma::mbar_wait(&tail->amax_bar[quarter], parity, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                parity ^= 1u;
                const float s = scale_from_amax<FMT>(fmaxf(amax, tail->amax[slot][half ^ 1][row]));
                const uint64_t s2 = f32x2(s, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // 16-byte chunks, in the 64-byte swizzle
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float* a = acc[0] + 16 * j + 4 * k;
                        const float2 lo = f32x2_split(mul_f32x2(f32x2(a[0], a[1]), s2));
                        const float2 hi = f32x2_split(mul_f32x2(f32x2(a[2], a[3]), s2));
                        w[k] = cvt_fp8x2<FMT>(lo.x, lo.y) | (cvt_fp8x2<FMT>(hi.x, hi.y) << 16);
                    }
                    *reinterpret_cast<uint4*>(out_q + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_to_async();
                __syncwarp();
                if (lane == 0 && out_y < p.M) tma_store_2d(&map_q, out_q, out_x, out_y);
                if (half == 0 && live) p.scales[m * f_blocks + fb] = s;
            }
        }
        // the boxes are written before the CTA's shared memory goes away and the grid ends
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if constexpr (SPLIT) {
        if (warp < 4) {  // the promotion warps' barrier on the sums
            __syncwarp();
            umma::cluster_sync();
        }
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
    // The even CTA's MMAs read the odd CTA's shared memory and write its tensor memory (and with SPLIT other
    // pairs read this CTA's sums): no CTA frees or leaves before all are done.
    umma::cluster_sync();
    if (warp == 1) {
        umma::fence_after_sync();
        umma::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// K == 0: zeros everywhere, and the scale of a zero block.
template <int FMT>
__global__ void k_gemm_gated_empty(GatedArgs p) {
    pdl_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    if (p.q != nullptr) {
        for (int64_t i = i0; i < p.M * p.F / 16; i += step) reinterpret_cast<uint4*>(p.q)[i] = make_uint4(0, 0, 0, 0);
        for (int64_t i = i0; i < p.M * (p.F / 128); i += step) p.scales[i] = scale_from_amax<FMT>(0.0f);
    }
    if (p.gu != nullptr) {
        const int64_t n = p.M * 2 * p.F * (p.gu_dtype == 0 ? 4 : 2) / 16;
        for (int64_t i = i0; i < n; i += step) static_cast<uint4*>(p.gu)[i] = make_uint4(0, 0, 0, 0);
    }
}

// [rows, cols] results in boxes of 32 rows x 64 columns.
bool make_out_map(CUtensorMap* map, CUtensorMapDataType type, int esize, CUtensorMapSwizzle swizzle, void* base,
                  int64_t rows, int64_t cols) {
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * esize)};
    const cuuint32_t box[2] = {64, 32};
    const cuuint32_t elem_strides[2] = {1, 1};
    return encode(map, type, 2, base, dims, strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The shared-memory opt-in and the clusters that the device holds at once, asked once per device and kernel; cfg has
// the rest of the launch.
template <int FMT, int ACT, bool SPLIT>
cudaError_t prepare(cudaLaunchConfig_t& cfg, int* clusters) {
    auto kern = k_gemm_gated<FMT, ACT, SPLIT>;
    static std::atomic<int> active[128];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    *clusters = active[dev].load(std::memory_order_acquire);
    if (*clusters > 0) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    const int size = static_cast<int>(cfg.attrs[0].val.clusterDim.x);
    *clusters = device_sm_count() / size;
    int n = 0;
    cfg.gridDim = dim3(static_cast<unsigned>(size * *clusters));
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) (void)cudaGetLastError();  // keep the estimate
    else if (n > 0) *clusters = std::min(*clusters, n);
    *clusters = std::max(*clusters, 1);
    active[dev].store(*clusters, std::memory_order_release);
    return cudaSuccess;
}

template <int FMT, int ACT>
cudaError_t launch_typed(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_q,
                         const CUtensorMap& map_gu, const GatedArgs& p, uint32_t idesc, unsigned int* status,
                         cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int na = 0;
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 2;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
#if FP8Q_PDL
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
#endif
    cfg.attrs = attr;
    cfg.numAttrs = na;
    const int64_t tiles = ((p.M + kTileM - 1) / kTileM) * (p.F / kTileF);
    if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    // Half of K a pair where all tiles still run at once.  The exchange and the larger cluster cost 3.5 us, 6 chunks:
    // 256 tokens, 4096 columns take 28.0 us against 40.0 with K 7168, 14.3 against 15.4 with 2048, and the same 12.8
    // with 1536.  (Four pairs a tile were never the fastest: only 16 clusters of 8 run at once.)
    constexpr int kSplitChunks = 12;
    int clusters = 0;
    if (p.K / kBK > kSplitChunks && tiles * 4 <= device_sm_count()) {
        attr[0].val.clusterDim.x = 4;
        const cudaError_t e = prepare<FMT, ACT, true>(cfg, &clusters);
        if (e != cudaSuccess) return e;
        if (tiles <= clusters) {
            cfg.gridDim = dim3(static_cast<unsigned>(4 * tiles));
            const cudaError_t l = cudaLaunchKernelEx(&cfg, k_gemm_gated<FMT, ACT, true>, map_a, map_b, map_q, map_gu, p,
                                                     idesc, status);
            return l != cudaSuccess ? l : cudaGetLastError();
        }
        attr[0].val.clusterDim.x = 2;
    }
    cudaError_t e = prepare<FMT, ACT, false>(cfg, &clusters);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, clusters)));
    e = cudaLaunchKernelEx(&cfg, k_gemm_gated<FMT, ACT, false>, map_a, map_b, map_q, map_gu, p, idesc, status);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool make_code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, uint32_t box_rows) {
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t elem_strides[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem_strides,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_gemm_gated(const GatedArgs& p, cudaStream_t st) {
    if (gemm_gated_few_fits(p)) return launch_gemm_gated_few(p, st);
    CUtensorMap map_a, map_b, map_q = {}, map_gu = {};
    if (!make_code_map(&map_a, p.a, p.M, p.K, kBM) || !make_code_map(&map_b, p.b, 2 * p.F, p.K, kTileF))
        return cudaErrorInvalidValue;
    if (p.q != nullptr && !make_out_map(&map_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, CU_TENSOR_MAP_SWIZZLE_64B, p.q, p.M, p.F))
        return cudaErrorInvalidValue;
    if (p.gu != nullptr && p.gu_dtype != 0 &&
        !make_out_map(&map_gu, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, CU_TENSOR_MAP_SWIZZLE_128B, p.gu, p.M, 2 * p.F))
        return cudaErrorInvalidValue;
    unsigned int* status = device_status_word();
    if (status == nullptr) return cudaErrorInvalidValue;
    const uint32_t idesc = umma::instr_desc_f8f6f4(p.a_fmt, p.b_fmt, kTileM, kBN);
    if (p.fmt == kE4M3)
        return p.act == kActSilu ? launch_typed<kE4M3, kActSilu>(map_a, map_b, map_q, map_gu, p, idesc, status, st)
                                 : launch_typed<kE4M3, kActGeluTanh>(map_a, map_b, map_q, map_gu, p, idesc, status, st);
    return p.act == kActSilu ? launch_typed<kE5M2, kActSilu>(map_a, map_b, map_q, map_gu, p, idesc, status, st)
                             : launch_typed<kE5M2, kActGeluTanh>(map_a, map_b, map_q, map_gu, p, idesc, status, st);
}

cudaError_t launch_gemm_gated_empty(const GatedArgs& p, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(device_sm_count() * 4));
    return p.fmt == kE4M3 ? launch_kernel(k_gemm_gated_empty<kE4M3>, grid, dim3(256), 0, st, p)
                          : launch_kernel(k_gemm_gated_empty<kE5M2>, grid, dim3(256), 0, st, p);
}

}  // namespace fp8q
