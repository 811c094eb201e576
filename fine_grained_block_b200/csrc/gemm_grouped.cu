// gemm_grouped.cu -- the products of experts: rows of A, one expert's after another's, each times its own weights.
//
//   expert e, its rows m = offsets[e] .. offsets[e + 1] - 1:
//     C[m][n] = sum over 128-wide K chunks c of P_c[m][n] / (sa[m][c] * sb[e][n/128][c]),
//     P_c[m][n] = sum over k in c of decode(A[m][k]) * decode(B[e][n][k])
//   plain   C in bf16 or fp32
//   gated   B[e] = [Wg; Wu], C = G | U:  H = act(G) * U as 1x128 codes, and C itself where it is asked for
// with the roundings of gemm_blockwise.cu and gemm_gated.cu.
//
// A CTA computes 128 rows x 256 columns of C with the roles and the epilogue of gemm_gated.cu: TMA producer, MMA issuer,
// two warps for the dequant factors, 8 promotion warps.  It holds 128 rows of A and two boxes of 128 rows of B: gate and
// up rows of the same columns, or the two halves of 256 columns.  Pairs of CTAs (256 rows, each with one box of B), as
// the products of one expert have them, were no faster with 4096 rows an expert (gated 7168 x 4096, 8 experts: 2176 us
// against 2191; plain 4096 x 7168: 1081 and 1066) and slower with fewer, whose last tile they leave emptier (64 experts,
// 2048 x 7168: 1258 and 1205 us with 1024 rows an expert, 516 and 447 with 312, 341 and 261 with 125).
//
// Only the device knows the experts' rows.  Every CTA reads the offsets, adds up the experts' row tiles in shared memory,
// and walks the tiles first, first + step, ...: expert by expert, within one in groups of 16 row tiles, column by column,
// so that a wave shares few experts' weights in L2.  A row tile may reach into the next expert's rows: they are
// multiplied, and not stored (a box of 32 rows that ends inside is stored row by row).  Rows behind the last expert's are
// left as they were.
//
// Bound by the promotion: the accumulators' trip out of tensor memory (ptxas spills 40 bytes of it).  Full tiles in
// bf16 run at 1.73 PFLOP/s (65536 rows, 32 experts of 4096 x 2048: 634 us); tiles that an expert fills to 62 % do 1.4 of
// whole tiles.  fp32 results leave row by row, 32 lines a store, and not in boxes: 984 us for the same product, 1566
// against 1272 for gated projections kept in fp32 (8192 tokens, 8 of 32 experts, 4096 x 2048).

#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "gemm_gated.h"
#include "launch_util.h"
#include "moe.h"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kBM = 128;                  // rows per CTA (TMEM lanes)
constexpr int kBlock = 128;               // rows of B in a box; a tile has two
constexpr int kBN = 2 * kBlock;           // MMA N
constexpr int kBK = 128;                  // K chunk = one promotion = one stage
constexpr int kMmaK = 32;
constexpr int kThreads = 384;             // 3 warpgroups: control, promotion x2
constexpr int kABytes = kBM * kBK;
constexpr uint32_t kTmemCols = 2 * kBN;   // two accumulators
// The register split of the CTA's launch total (setmaxnreg): 3 x 168 = 56 + 2 x 224.
constexpr int kLaunchRegs = 168;
constexpr int kControlRegs = 56;
constexpr int kPromoteRegs = 224;
static_assert(kControlRegs + 2 * kPromoteRegs == 3 * kLaunchRegs, "register split must equal the launch total");
static_assert(kLaunchRegs * kThreads <= 65536, "launch registers exceed the register file");
constexpr uint32_t kGroup = 16;           // row tiles that are walked together
constexpr int kFacSlots = 4;              // chunks whose dequant factors are held

constexpr int kStages = 3;
constexpr int kStageBytes = 3 * kABytes;  // A rows and the two boxes of B
constexpr int kPromoteWarps = 8;
// Results on their way out, per promotion warp: a box of 32 rows x 64 columns in bf16 for each block, the first of which
// the codes take after it.
constexpr int kOutC = 32 * 64 * 2;
constexpr int kOutBytes = kPromoteWarps * 2 * kOutC;
struct Tail {  // behind the operand stages and the results
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint64_t amax_bar[4];     // one per quarter: its two promotion warps
    uint32_t tmem_base;
    uint32_t warp_sum[kThreads / 32];
    float amax[2][2][kBM];    // [tile parity][column half][row]
    alignas(16) float2 fac[kFacSlots][kBM];  // the factors of both 128-column blocks, by row and chunk
    int32_t rows[kMaxExperts + 1];           // an expert's first row
    uint32_t tiles[kMaxExperts + 1];         // row tiles before an expert
};
constexpr int kSmemBytes = kStages * kStageBytes + kOutBytes + 1024 /* alignment */ + static_cast<int>(sizeof(Tail));
static_assert(kSmemBytes <= 227 * 1024, "stages and barriers must fit in shared memory");

// The tile that a role works on: experts only go up.
struct Cursor {
    int e = 0;
    int64_t row = 0, end = 0;  // first row of the tile, and the one behind the expert's last
    int col = 0;               // column tile
    __device__ __forceinline__ void seek(const Tail* tail, uint32_t t, uint32_t tiles_n) {
        while (t >= tail->tiles[e + 1] * tiles_n) ++e;
        const uint32_t height_all = tail->tiles[e + 1] - tail->tiles[e];
        const uint32_t r = t - tail->tiles[e] * tiles_n;
        const uint32_t in_group = kGroup * tiles_n, g = r / in_group, s = r - g * in_group;
        const uint32_t height = min(kGroup, height_all - g * kGroup);
        col = static_cast<int>(s / height);
        row = tail->rows[e] + static_cast<int64_t>(g * kGroup + (s - static_cast<uint32_t>(col) * height)) * kBM;
        end = tail->rows[e + 1];
    }
};

template <bool GATED, int FMT, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
k_gemm_grouped(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c,
               const __grid_constant__ GroupedArgs p, uint32_t idesc, unsigned int* status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* out = stages + kStages * kStageBytes;
    Tail* tail = reinterpret_cast<Tail*>(out + kOutBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int nchunks = static_cast<int>(p.K / kBK);
    const int blocks = static_cast<int>(p.N / kBlock);              // of B's rows, per expert
    // tiles of 256 columns; the two blocks of a tile are `apart` blocks from one another
    const uint32_t tiles_n = static_cast<uint32_t>((blocks + 1) / 2);
    const int apart = GATED ? blocks / 2 : 1;
    const int per_tile = GATED ? 1 : 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            umma::mbar_init(&tail->full[s], 1);
            umma::mbar_init(&tail->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            umma::mbar_init(&tail->acc_full[b], 3);  // the MMAs and the two factor warps
            umma::mbar_init(&tail->acc_empty[b], kPromoteWarps);
        }
        umma::mbar_init(&tail->mma_done, 1);
        for (int q = 0; q < 4; ++q) umma::mbar_init(&tail->amax_bar[q], 2);
        umma::fence_mbar_init();
    }
    if (warp == 1) umma::tmem_alloc(&tail->tmem_base, kTmemCols);
    umma::fence_before_sync();
    __syncthreads();  // allocated before the next kernel may start
    umma::fence_after_sync();
    const uint32_t tmem = tail->tmem_base;
    pdl_enter();  // the codes, scales and offsets may come from the previous kernel
    {   // row tiles before each expert: a scan, up to 3 experts a thread
        constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
        const int per = (p.E + kThreads - 1) / kThreads;
        uint32_t n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = static_cast<int>(threadIdx.x) * per + i;
            n[i] = 0;
            if (i < per && e < p.E) {
                const int R = static_cast<int>(p.R);
                const int r0 = min(max(p.offsets[e], 0), R), r1 = min(max(p.offsets[e + 1], 0), R);
                tail->rows[e] = r0;
                if (e == p.E - 1) tail->rows[p.E] = r1;
                n[i] = r1 > r0 ? static_cast<uint32_t>(r1 - r0 + kBM - 1) / kBM : 0u;
            }
            sum += n[i];
        }
        uint32_t upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) tail->warp_sum[warp] = upto;
        __syncthreads();
        uint64_t before = upto - sum;
        for (int w = 0; w < warp; ++w) before += tail->warp_sum[w];
        // offsets that ascend never reach the limit; others must not lead past the last expert
        const uint64_t most = static_cast<uint64_t>(p.R / kBM + p.E);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = static_cast<int>(threadIdx.x) * per + i;
            if (i < per && e < p.E) {
                tail->tiles[e] = static_cast<uint32_t>(min(before, most));
                before += n[i];
                if (e == p.E - 1) tail->tiles[p.E] = static_cast<uint32_t>(min(before, most));
            }
        }
    }
    __syncthreads();
    const uint32_t tiles = tail->tiles[p.E] * tiles_n;
    const uint32_t first = blockIdx.x, step = gridDim.x;

    bool timed_out = false;
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0) {
        // ---- TMA producer ----------------------------------------------------
        if (lane == 0) {
            uint32_t g = 0;
            Cursor c;
            for (uint32_t t = first; t < tiles && !timed_out; t += step) {
                c.seek(tail, t, tiles_n);
                const int m0 = static_cast<int>(c.row);
                const int n0 = static_cast<int>(c.e * p.N + c.col * per_tile * kBlock);
                for (int kc = 0; kc < nchunks; ++kc, ++g) {
                    const uint32_t s = g % kStages;
                    if (!umma::mbar_wait(&tail->empty[s], ((g / kStages) & 1u) ^ 1u, kWaitLimitNs)) {
                        timed_out = true;
                        break;
                    }
                    uint8_t* stage = stages + s * kStageBytes;
                    umma::mbar_arrive_expect_tx(&tail->full[s], kStageBytes);
                    umma::tma_load_2d(stage, &map_a, &tail->full[s], kc * kBK, m0);
                    umma::tma_load_2d(stage + kABytes, &map_b, &tail->full[s], kc * kBK, n0);
                    umma::tma_load_2d(stage + 2 * kABytes, &map_b, &tail->full[s], kc * kBK, n0 + apart * kBlock);
                }
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer ----------------------------------------------------------
        if (lane == 0) {
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
                    for (int k = 0; k < kBK / kMmaK; ++k) umma::mma_f8f6f4(d, a_desc + 2 * k, b_desc + 2 * k, idesc, k > 0);
                    umma::commit(&tail->empty[s]);
                    umma::commit(&tail->acc_full[buf]);
                }
            }
            umma::commit(&tail->mma_done);
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
        Cursor c;
        for (uint32_t t = first; t < tiles && !timed_out; t += step) {
            c.seek(tail, t, tiles_n);
            const int64_t m0 = c.row + r0;
            const float* sa0 = p.sa + std::min<int64_t>(m0, p.R - 1) * nchunks;  // rows past R: any factor will do
            const float* sa1 = p.sa + std::min<int64_t>(m0 + 64, p.R - 1) * nchunks;
            const int b0 = c.col * per_tile, b1 = min(b0 + apart, blocks - 1);   // the last tile may have one block
            const float* sg = p.sb + (static_cast<int64_t>(c.e) * blocks + b0) * nchunks;
            const float* su = p.sb + (static_cast<int64_t>(c.e) * blocks + b1) * nchunks;
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
        const int half = (warp - 4) >> 2;        // columns 64 * half .. of both blocks
        const int row = quarter * 32 + lane;     // row within this CTA's 128 = TMEM lane
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * 64);
        uint8_t* out_c = out + (warp - 4) * 2 * kOutC;
        uint32_t g = 0, parity = 0;
        Cursor c;
        for (uint32_t t = first, turn = 0; t < tiles && !timed_out; t += step, ++turn) {
            float acc[2][64];                    // both blocks
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
                    umma::tmem_ld32(tm + h * kBlock, v);
                    umma::tmem_ld32(tm + h * kBlock + 32, v + 32);
                    umma::wait_ld(v);
                    umma::hold_after_wait(v + 32);
                    if (h == 1) {  // every partial sum of this buffer is in registers: hand it back
                        umma::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(&tail->acc_empty[buf]);
                    }
#pragma unroll
                    for (int j = 0; j < 64; ++j) acc[h][j] = __fmaf_rn(v[j], fac[h], acc[h][j]);
                }
            }
            if (timed_out) break;
            c.seek(tail, t, tiles_n);
            const int64_t m = c.row + row;
            const bool live = m < c.end;
            const int out_y = static_cast<int>(m) - lane;        // the warp's first row
            const bool boxes = out_y + 32 <= c.end;              // all 32 rows are the expert's
            const int out_x = c.col * per_tile * kBlock + half * 64;
            const bool second = GATED || c.col * 2 + 1 < blocks;  // the last tile may have one block
            if (lane == 0) umma::tma_store_wait_read();          // the previous tile's boxes
            __syncwarp();
            if (p.c != nullptr && p.c_dtype != 0) {
                if (boxes) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1 && !second) break;
                        uint8_t* box = out_c + h * kOutC;
#pragma unroll
                        for (int j = 0; j < 8; ++j)  // 16-byte chunks, in the 128-byte swizzle that the tensor map names
                            *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                                make_uint4(pack_bf16x2(acc[h][8 * j], acc[h][8 * j + 1]),
                                           pack_bf16x2(acc[h][8 * j + 2], acc[h][8 * j + 3]),
                                           pack_bf16x2(acc[h][8 * j + 4], acc[h][8 * j + 5]),
                                           pack_bf16x2(acc[h][8 * j + 6], acc[h][8 * j + 7]));
                        umma::fence_to_async();
                        __syncwarp();
                        if (lane == 0) umma::tma_store_2d(&map_c, box, out_x + h * apart * kBlock, out_y);
                    }
                } else if (live) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1 && !second) break;
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c) + m * p.N + out_x + h * apart * kBlock);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j] = make_uint4(pack_bf16x2(acc[h][8 * j], acc[h][8 * j + 1]),
                                                pack_bf16x2(acc[h][8 * j + 2], acc[h][8 * j + 3]),
                                                pack_bf16x2(acc[h][8 * j + 4], acc[h][8 * j + 5]),
                                                pack_bf16x2(acc[h][8 * j + 6], acc[h][8 * j + 7]));
                    }
                }
            } else if (p.c != nullptr && live) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && !second) break;
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.c) + m * p.N + out_x + h * apart * kBlock);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        dst[j] = make_float4(acc[h][4 * j], acc[h][4 * j + 1], acc[h][4 * j + 2], acc[h][4 * j + 3]);
                }
            }
            if constexpr (GATED) {
                if (p.q != nullptr) {
                    const int64_t F = p.N / 2;
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
                    uint4 w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t u[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float* a = acc[0] + 16 * j + 4 * k;
                            const float2 lo = f32x2_split(mul_f32x2(f32x2(a[0], a[1]), s2));
                            const float2 hi = f32x2_split(mul_f32x2(f32x2(a[2], a[3]), s2));
                            u[k] = cvt_fp8x2<FMT>(lo.x, lo.y) | (cvt_fp8x2<FMT>(hi.x, hi.y) << 16);
                        }
                        w[j] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    if (boxes) {
                        // the first block's box is read; the second's may still be
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // 16-byte chunks, in the 64-byte swizzle
                            *reinterpret_cast<uint4*>(out_c + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) = w[j];
                        umma::fence_to_async();
                        __syncwarp();
                        if (lane == 0) umma::tma_store_2d(&map_q, out_c, out_x, out_y);
                    } else if (live) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) reinterpret_cast<uint4*>(p.q + m * F + out_x)[j] = w[j];
                    }
                    if (half == 0 && live) p.scales[m * (F / kBlock) + c.col] = s;
                }
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

// K == 0: zeros on every expert's rows, and the scale of a zero block.  Expert by expert, because their rows need not start
// at the tensors' first row, and offsets that no sort makes need not ascend.
template <int FMT>
__global__ void k_gemm_grouped_empty(GroupedArgs p, bool gated) {
    pdl_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t R = p.R, F = p.N / 2, c_row = p.N * (p.c_dtype == 0 ? 4 : 2) / 16;
    for (int e = 0; e < p.E; ++e) {
        const int64_t lo = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), R);
        const int64_t rows = min(max(static_cast<int64_t>(p.offsets[e + 1]), int64_t(0)), R) - lo;
        if (gated && p.q != nullptr) {
            uint4* q = reinterpret_cast<uint4*>(p.q + lo * F);
            for (int64_t i = i0; i < rows * F / 16; i += step) q[i] = make_uint4(0, 0, 0, 0);
            float* scales = p.scales + lo * (F / 128);
            for (int64_t i = i0; i < rows * (F / 128); i += step) scales[i] = scale_from_amax<FMT>(0.0f);
        }
        if (p.c != nullptr) {
            uint4* c = static_cast<uint4*>(p.c) + lo * c_row;
            for (int64_t i = i0; i < rows * c_row; i += step) c[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

template <bool GATED, int FMT, int ACT>
cudaError_t launch_typed(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_q,
                         const CUtensorMap& map_c, const GroupedArgs& p, unsigned int* status, cudaStream_t st) {
    auto kern = k_gemm_grouped<GATED, FMT, ACT>;
    static std::atomic<bool> opted[128];  // the shared-memory opt-in, once per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_release);
    }
    // no more tiles than these, however the rows are shared out
    const int64_t tiles_n = (p.N / kBlock + 1) / 2;
    const int64_t most = (p.R / kBM + std::min<int64_t>(p.E, p.R)) * tiles_n;
    if ((p.R / kBM + p.E) * tiles_n > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(most, device_sm_count()));
    const uint32_t idesc = umma::instr_desc_f8f6f4(p.a_fmt, p.b_fmt, kBM, kBN);
    return launch_kernel(kern, dim3(ctas), dim3(kThreads), kSmemBytes, st, map_a, map_b, map_q, map_c, p, idesc, status);
}

}  // namespace

cudaError_t launch_gemm_grouped(const GroupedArgs& p, bool gated, cudaStream_t st) {
    CUtensorMap map_a, map_b, map_q = {}, map_c = {};
    if (!make_code_map(&map_a, p.a, p.R, p.K, kBM) || !make_code_map(&map_b, p.b, p.E * p.N, p.K, kBlock))
        return cudaErrorInvalidValue;
    if (p.q != nullptr && !make_out_map(&map_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, CU_TENSOR_MAP_SWIZZLE_64B, p.q, p.R, p.N / 2))
        return cudaErrorInvalidValue;
    if (p.c != nullptr && p.c_dtype != 0 &&
        !make_out_map(&map_c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, CU_TENSOR_MAP_SWIZZLE_128B, p.c, p.R, p.N))
        return cudaErrorInvalidValue;
    unsigned int* status = device_status_word();
    if (status == nullptr) return cudaErrorInvalidValue;
    if (!gated) return launch_typed<false, kE4M3, kActSilu>(map_a, map_b, map_q, map_c, p, status, st);
    if (p.fmt == kE4M3)
        return p.act == kActSilu ? launch_typed<true, kE4M3, kActSilu>(map_a, map_b, map_q, map_c, p, status, st)
                                 : launch_typed<true, kE4M3, kActGeluTanh>(map_a, map_b, map_q, map_c, p, status, st);
    return p.act == kActSilu ? launch_typed<true, kE5M2, kActSilu>(map_a, map_b, map_q, map_c, p, status, st)
                             : launch_typed<true, kE5M2, kActGeluTanh>(map_a, map_b, map_q, map_c, p, status, st);
}

cudaError_t launch_gemm_grouped_empty(const GroupedArgs& p, bool gated, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(device_sm_count() * 4));
    return p.fmt == kE4M3 ? launch_kernel(k_gemm_grouped_empty<kE4M3>, grid, dim3(256), 0, st, p, gated)
                          : launch_kernel(k_gemm_grouped_empty<kE5M2>, grid, dim3(256), 0, st, p, gated);
}

}  // namespace fp8q
