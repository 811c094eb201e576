// gemm_gated_few.cu -- the gated projections for few tokens: the form for
// single tokens, decode batches and short prompts.
//
// The products and factors of gemm_gated.cu, whose sums over K it repeats bit for
// bit where K is not split (K < 512); split, they are added in another order.
//
// With few tokens the work is reading the 2 F K bytes of weights once, so the
// tensor core's M side (128 lanes) takes weight rows and its N side the tokens,
// NT of them (16, 32 or 64; more tokens take several token blocks, whose weights
// come from L2):
//   G^T tile [128 gate rows x NT] and U^T tile [128 up rows x NT], in two
//   accumulators of the same lanes, so a thread meets G and U of one f.
// A tile is 128 columns of H, one 1x128 block of every token.  There are only
// F / 128 tiles, so K is split over a cluster of S CTAs (S = 1, 2, 4 or 8):
// each walks its chunks of 128 with its own pipeline; at the end the partial
// sums meet through distributed shared memory, added in rank order (the result
// does not depend on timing), and each CTA finishes the tokens m % S == rank, a
// warp a token.
//
// Warp 0 is the TMA producer (both weight boxes and the tokens' box of a chunk),
// warp 1 the MMA issuer, the others (8, or 16 for 64 tokens) the promotion: warp w
// reads TMEM lanes 32 (w & 3).. of 8 or 16 tokens, and adds partial * 1/(sa*sb) in
// fp32.  The factor of a token, RN(1 / RN(sa*sb)) as in gemm_gated.cu, is formed by
// one lane and passed to the warp through shared memory.  A chunk needs 2 NT TMEM
// columns, so up to 8 chunks are in flight between the MMAs and the promotion and
// the trip out of tensor memory, which bounds the large kernel, is hidden here.
//
// Bound by HBM (the weights) beside a fixed part: one token, 7168 x 4096, takes
// 12.9 us (58.7 MB: 9.0 at the copy rate), and 8.3 more with twice the K.  The
// fixed 4 us are the launch, the first chunk's trip, the cluster's reduction and
// the drain; with 64-token tiles, one CTA an SM, they are 8 (48 tokens, 4096 x
// 8192: 17.8 us for 67 MB).  Tried without gain: two tokens a warp at the end,
// two CTAs an SM for 64 tokens (spills), both accumulators read at once.

#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "gemm_gated.h"
#include "launch_util.h"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kTileF = 128;
constexpr int kBK = 128;
constexpr int kMmaK = 32;
constexpr int kWBytes = kTileF * kBK;  // one weight box
constexpr int kAhead = 2;              // chunks ahead that the scales are loaded
constexpr int kMaxSplit = 8;
constexpr int kPrefetch = 3;           // chunks of weights brought to L2 before the previous kernel has ended

template <int NT>
struct Few {
    static constexpr int kPer = NT / 2 < 16 ? NT / 2 : 16;  // tokens of a promotion warp
    static constexpr int kPromoteWarps = 4 * NT / kPer;
    static constexpr int kThreads = 32 * (2 + kPromoteWarps);
    static_assert(NT <= 64, "wider tiles spill: 128 tokens measured 1.7 us a chunk against 0.58");
    static constexpr int kCtas = NT <= 32 ? 2 : 1;        // CTAs per SM
    static constexpr int kStages = NT <= 32 ? 3 : 5;
    static constexpr uint32_t kTmemCols = NT <= 32 ? 256 : 512;
    static constexpr int kBufs = static_cast<int>(kTmemCols) / (2 * NT);
    static constexpr int kStageBytes = 2 * kWBytes + NT * kBK;
    struct Tail {
        uint64_t full[kStages];
        uint64_t empty[kStages];
        uint64_t acc_full[kBufs];
        uint64_t acc_empty[kBufs];
        uint32_t tmem_base;
        alignas(16) float fac[kPromoteWarps][2][2][kPer];  // [warp][chunk parity][gate, up][token]
    };
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024 /* alignment */ + static_cast<int>(sizeof(Tail));
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "the CTAs of an SM share its shared memory");
    static_assert(2 * NT * kTileF * 4 <= kStages * kStageBytes, "the partial sums fit where the stages were");
};

// N consecutive fp32 columns of this thread's TMEM lane, complete on return.
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t addr, float (&v)[N]);
template <>
__device__ __forceinline__ void tmem_read<8>(uint32_t addr, float (&v)[8]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void tmem_read<16>(uint32_t addr, float (&v)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

// A warp finishes a token: its 128 columns, 4 a lane.  The sums over the ranks in rank order, all loads
// before the first use (one trip through the cluster's network), H, the block's amax by shuffles, and the
// codes.
template <int NT, int FMT, int SPLIT>
__device__ __forceinline__ void finish(const GatedArgs& p, uint32_t part0, int rank, int pw, int lane, int64_t tile,
                                       int64_t m0, int M) {
    const int64_t f = tile * kTileF + 4 * lane;
    for (int m = rank + SPLIT * pw; m < M; m += SPLIT * Few<NT>::kPromoteWarps) {
        float4 g[SPLIT], u[SPLIT];
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
            const uint32_t at = umma::mapa(part0, static_cast<uint32_t>(r)) + static_cast<uint32_t>((m * kTileF + 4 * lane) * 4);
            g[r] = umma::ld_cluster_f32x4(at);
            u[r] = umma::ld_cluster_f32x4(at + NT * kTileF * 4);
        }
#pragma unroll
        for (int r = 1; r < SPLIT; ++r) {
            g[0] = make_float4(g[0].x + g[r].x, g[0].y + g[r].y, g[0].z + g[r].z, g[0].w + g[r].w);
            u[0] = make_float4(u[0].x + u[r].x, u[0].y + u[r].y, u[0].z + u[r].z, u[0].w + u[r].w);
        }
        if (p.gu != nullptr) {
            const int64_t at = (m0 + m) * 2 * p.F + f;
            if (p.gu_dtype == 0) {
                *reinterpret_cast<float4*>(static_cast<float*>(p.gu) + at) = g[0];
                *reinterpret_cast<float4*>(static_cast<float*>(p.gu) + at + p.F) = u[0];
            } else {
                uint16_t* gu = static_cast<uint16_t*>(p.gu) + at;
                *reinterpret_cast<uint2*>(gu) = make_uint2(pack_bf16x2(g[0].x, g[0].y), pack_bf16x2(g[0].z, g[0].w));
                *reinterpret_cast<uint2*>(gu + p.F) = make_uint2(pack_bf16x2(u[0].x, u[0].y), pack_bf16x2(u[0].z, u[0].w));
            }
        }
        if (p.q == nullptr) continue;
        const uint64_t g01 = f32x2(g[0].x, g[0].y), g23 = f32x2(g[0].z, g[0].w);
        uint64_t a01, a23;
        if (p.act == kActSilu) {
            a01 = gate_act2<kActSilu>(g01);
            a23 = gate_act2<kActSilu>(g23);
        } else {
            a01 = gate_act2<kActGeluTanh>(g01);
            a23 = gate_act2<kActGeluTanh>(g23);
        }
        const uint64_t h01 = mul_f32x2(a01, f32x2(u[0].x, u[0].y)), h23 = mul_f32x2(a23, f32x2(u[0].z, u[0].w));
        const float2 x = f32x2_split(h01), y = f32x2_split(h23);
        const float s = scale_from_amax<FMT>(
            warp_max<32>(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)))));
        const float2 c = f32x2_split(mul_f32x2(h01, both(s))), d = f32x2_split(mul_f32x2(h23, both(s)));
        *reinterpret_cast<uint32_t*>(p.q + (m0 + m) * p.F + f) =
            cvt_fp8x2<FMT>(c.x, c.y) | (cvt_fp8x2<FMT>(d.x, d.y) << 16);
        if (lane == 0) p.scales[(m0 + m) * (p.F / kTileF) + tile] = s;
    }
}

__device__ __forceinline__ void prefetch_l2(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

template <int NT, int FMT>
__global__ void __launch_bounds__(Few<NT>::kThreads, Few<NT>::kCtas)
k_gemm_gated_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
                 const __grid_constant__ GatedArgs p, uint32_t idesc, unsigned int* status, int split) {
    using C = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto* tail = reinterpret_cast<typename C::Tail*>(stages + C::kStages * C::kStageBytes);
    float* part = reinterpret_cast<float*>(stages);  // after the last chunk: [G, U][token][f]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(umma::cluster_ctarank());
    const int64_t tile = blockIdx.x / static_cast<unsigned>(split);
    const int64_t f0 = tile * kTileF;
    const int64_t tiles = p.F / kTileF;
    const int all_chunks = static_cast<int>(p.K / kBK);
    const int c0 = all_chunks * rank / split, c1 = all_chunks * (rank + 1) / split;
    const int m0 = static_cast<int>(blockIdx.y) * NT;                        // this CTA's tokens
    const int M = static_cast<int>(min(p.M - m0, static_cast<int64_t>(NT)));  // how many

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            umma::mbar_init(&tail->full[s], 1);
            umma::mbar_init(&tail->empty[s], 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            umma::mbar_init(&tail->acc_full[b], 1);
            umma::mbar_init(&tail->acc_empty[b], C::kPromoteWarps);
        }
        umma::fence_mbar_init();
    }
    if (warp == 1) umma::tmem_alloc(&tail->tmem_base, C::kTmemCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tail->tmem_base;
    if (warp == 0 && lane == 0) {
        // The weights' first chunks into L2 while the previous kernel still runs.  Only a hint: should that
        // kernel write them, its writes go through the same L2.  Behind the norm that makes the codes (one
        // token, 4096 x 7168): 14.8 us for both kernels, 16.1 without, 15.7 with 8 chunks.
        for (int c = c0; c < min(c1, c0 + kPrefetch); ++c) {
            prefetch_l2(&map_w, c * kBK, static_cast<int>(f0));
            prefetch_l2(&map_w, c * kBK, static_cast<int>(p.F + f0));
        }
    }
    pdl_enter();  // the codes and scales may come from the previous kernel

    bool timed_out = false;
    if (warp == 0) {
        if (lane == 0) {
            for (int c = c0; c < c1; ++c) {
                const uint32_t g = static_cast<uint32_t>(c - c0), s = g % C::kStages;
                if (!umma::mbar_wait(&tail->empty[s], ((g / C::kStages) & 1u) ^ 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                uint8_t* stage = stages + s * C::kStageBytes;
                umma::mbar_arrive_expect_tx(&tail->full[s], C::kStageBytes);
                umma::tma_load_2d(stage, &map_w, &tail->full[s], c * kBK, static_cast<int>(f0));
                umma::tma_load_2d(stage + kWBytes, &map_w, &tail->full[s], c * kBK, static_cast<int>(p.F + f0));
                umma::tma_load_2d(stage + 2 * kWBytes, &map_t, &tail->full[s], c * kBK, m0);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int c = c0; c < c1; ++c) {
                const uint32_t g = static_cast<uint32_t>(c - c0), s = g % C::kStages, buf = g % C::kBufs;
                if (!umma::mbar_wait(&tail->acc_empty[buf], ((g / C::kBufs) & 1u) ^ 1u, kWaitLimitNs) ||
                    !umma::mbar_wait(&tail->full[s], (g / C::kStages) & 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                umma::fence_after_sync();
                const uint32_t w_addr = umma::smem_u32(stages + s * C::kStageBytes);
                const uint64_t t_desc = umma::smem_desc_kmajor_sw128(w_addr + 2 * kWBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // gate rows, up rows
                    const uint64_t w_desc = umma::smem_desc_kmajor_sw128(w_addr + h * kWBytes);
                    const uint32_t d = tmem + buf * static_cast<uint32_t>(2 * NT) + static_cast<uint32_t>(h * NT);
#pragma unroll
                    for (int k = 0; k < kBK / kMmaK; ++k)
                        umma::mma_f8f6f4(d, w_desc + 2 * k, t_desc + 2 * k, idesc, k > 0);
                }
                umma::commit(&tail->empty[s]);
                umma::commit(&tail->acc_full[buf]);
            }
        }
    } else {
        const int quarter = warp & 3;
        const int group = (warp - 2) >> 2;
        constexpr int H = C::kPer;
        float acc[2][H];
#pragma unroll
        for (int j = 0; j < H; ++j) acc[0][j] = acc[1][j] = 0.0f;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(group * H);
        const float* sg_row = p.sb + tile * all_chunks;
        const float* su_row = p.sb + (tiles + tile) * all_chunks;
        // lane j < H forms the factors of the warp's token j
        const int my_token = group * H + lane;
        const bool mine = lane < H && my_token < M;
        const float* sa_row = p.sa + static_cast<int64_t>(m0 + (mine ? my_token : 0)) * all_chunks;
        float sa_q[kAhead], sg_q[kAhead], su_q[kAhead];
        auto load_scales = [&](int d, int c) {
            sa_q[d] = mine && c < c1 ? __ldg(sa_row + c) : 1.0f;
            sg_q[d] = c < c1 ? __ldg(sg_row + c) : 1.0f;
            su_q[d] = c < c1 ? __ldg(su_row + c) : 1.0f;
        };
#pragma unroll
        for (int d = 0; d < kAhead; ++d) load_scales(d, c0 + d);
        for (int c = c0; c < c1; ++c) {
            const uint32_t g = static_cast<uint32_t>(c - c0), buf = g % C::kBufs;
            float (*fac)[H] = tail->fac[warp - 2][g & 1u];  // written again two chunks on, behind a __syncwarp
            if (lane < H) {
                fac[0][lane] = __frcp_rn(__fmul_rn(sa_q[0], sg_q[0]));
                fac[1][lane] = __frcp_rn(__fmul_rn(sa_q[0], su_q[0]));
            }
#pragma unroll
            for (int d = 0; d + 1 < kAhead; ++d) {
                sa_q[d] = sa_q[d + 1];
                sg_q[d] = sg_q[d + 1];
                su_q[d] = su_q[d + 1];
            }
            load_scales(kAhead - 1, c + kAhead);
            __syncwarp();
            if (!umma::mbar_wait(&tail->acc_full[buf], (g / C::kBufs) & 1u, kWaitLimitNs)) {
                timed_out = true;
                break;
            }
            umma::fence_after_sync();
            const uint32_t tm = t_lane + buf * static_cast<uint32_t>(2 * NT);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // (both at once: 64 tokens spill)
                float v[H];
                tmem_read<H>(tm + h * NT, v);
                if (h == 1) {  // the buffer is read: hand it back
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(&tail->acc_empty[buf]);
                }
#pragma unroll
                for (int j = 0; j < H; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&fac[h][j]);
                    acc[h][j] = __fmaf_rn(v[j], f.x, acc[h][j]);
                    acc[h][j + 1] = __fmaf_rn(v[j + 1], f.y, acc[h][j + 1]);
                    acc[h][j + 2] = __fmaf_rn(v[j + 2], f.z, acc[h][j + 2]);
                    acc[h][j + 3] = __fmaf_rn(v[j + 3], f.w, acc[h][j + 3]);
                }
            }
        }
        if (!timed_out) {
            // Every MMA of this CTA has completed (the last commit covered them all), so the stages are free.
            const int f = quarter * 32 + lane;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < H; ++j) part[(h * NT + group * H + j) * kTileF + f] = acc[h][j];
        }
    }
    __syncwarp();
    umma::fence_before_sync();
    if (timed_out) atomicOr(status, kStatusWaitTimeout);
    const bool bad = __syncthreads_or(timed_out);
    if (bad && threadIdx.x == 0) {
        // A wait ran out: give copies and MMAs still in flight time to finish (bounded).
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
    __syncwarp();
    umma::cluster_sync();  // every CTA's partial sums are in its shared memory
    if (warp >= 2 && !bad) {  // the tokens m % split == rank
        const uint32_t part0 = umma::smem_u32(part);
        switch (split) {
            case 1: finish<NT, FMT, 1>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
            case 2: finish<NT, FMT, 2>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
            case 4: finish<NT, FMT, 4>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
            default: finish<NT, FMT, kMaxSplit>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
        }
    }
    __syncwarp();
    umma::cluster_sync();  // no CTA leaves while another may read its shared memory
    if (warp == 1) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int NT, int FMT>
cudaError_t launch_typed(const GatedArgs& p, cudaStream_t st) {
    using C = Few<NT>;
    CUtensorMap map_w, map_t;
    if (!make_code_map(&map_w, p.b, 2 * p.F, p.K, kTileF) || !make_code_map(&map_t, p.a, p.M, p.K, NT))
        return cudaErrorInvalidValue;
    unsigned int* status = device_status_word();
    if (status == nullptr) return cudaErrorInvalidValue;
    auto kern = k_gemm_gated_few<NT, FMT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    const int64_t tiles = p.F / kTileF, blocks = (p.M + NT - 1) / NT, chunks = p.K / kBK;
    if (blocks > 65535 || tiles * kMaxSplit > 0x7FFFFFFF || chunks * kMaxSplit > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int na = 0;
    attr[na].id = cudaLaunchAttributeClusterDimension;
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
    // Clusters of 2, 4 and 8 that the device holds at once (its SMs come in groups that a cluster cannot
    // leave), and the shared-memory opt-in, once per device.
    static std::atomic<int> active[128][3];
    if (active[dev][2].load(std::memory_order_acquire) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        for (int i = 0; i < 3; ++i) {
            int n = 0;
            attr[0].val.clusterDim.x = 2u << i;
            cfg.gridDim = dim3((2u << i) * 512u);
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
                (void)cudaGetLastError();
                n = 1;
            }
            active[dev][i].store(n, std::memory_order_release);
        }
    }
    // The widest split of K whose clusters all run at once.  With two CTAs an
    // SM counting CTAs is better than counting clusters, though a cluster or two may have to wait: one starts as
    // soon as another's CTAs drain (one token, 7168 x 4096: 12.9 us in 32 clusters of 8, 14.7 in 32 of 4).
    // A rank takes two chunks at least, four of eight (4096 columns, K 1024: 4.9 us in 4, 6.1 in 8; K 2048: 6.5
    // and 7.0; K 4096: 10.8 and 9.9).
    int split = 1;
    for (int i = 0; i < 3 && (2 << i) * (i < 2 ? 2 : 4) <= chunks; ++i) {
        const int64_t room = C::kCtas > 1 ? static_cast<int64_t>(device_sm_count()) * C::kCtas / (2 << i)
                                          : active[dev][i].load(std::memory_order_relaxed);
        if (tiles * blocks > room) break;
        split = 2 << i;
    }
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), static_cast<unsigned>(blocks));
    const uint32_t idesc = umma::instr_desc_f8f6f4(p.b_fmt, p.a_fmt, kTileF, NT);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, map_w, map_t, p, idesc, status, split);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT>
cudaError_t launch_fmt(const GatedArgs& p, cudaStream_t st) {
    return p.fmt == kE4M3 ? launch_typed<NT, kE4M3>(p, st) : launch_typed<NT, kE5M2>(p, st);
}

}  // namespace

bool gemm_gated_few_fits(const GatedArgs& p) {
    // Up to one token block always.  More while K can still be split in two, that is while its CTAs fill at
    // most half the SMs: a chunk then costs 0.58 us here and 0.59 in gemm_gated.cu's pairs, but each CTA has half
    // of them.  4096 x 1024 by 256 tokens: 12.4 us here, 17.7 there (two pairs a tile); 7168 x 4096 by 256: 41.1 and 28.0.
    return p.M <= 64 || (p.M + 63) / 64 * (p.F / kTileF) * 2 <= device_sm_count();
}

cudaError_t launch_gemm_gated_few(const GatedArgs& p, cudaStream_t st) {
    // The smallest token tile that holds them: a narrower one keeps more chunks in flight.  Blocks of 32, two CTAs
    // an SM, also where there would be room for all of them with K split in eight, whatever the split is (K < 4096
    // gives fewer ranks).  K x F, blocks of 32 against 64: 64 tokens 512 x 1024 5.0 us and 6.2, 1024 x 1024 5.1 and 6.8,
    // 4096 x 1024 8.7 and 9.5; 128 tokens 256 x 256 5.7 and 6.8, 7168 x 1024 13.3 and 14.7.  At the rule's end they
    // meet (64 tokens, F 2048: K 2048 7.3 and 8.3, K 4096 11.7 and 11.2, K 7168 13.8 and 14.8); with more CTAs the
    // weights' second trip through L2 costs more (48 tokens, 4096 x 8192: 20.5 against 17.8).
    if (p.M <= 16) return launch_fmt<16>(p, st);
    if (p.M <= 32 || (p.M + 31) / 32 * (p.F / kTileF) * kMaxSplit <= 2 * device_sm_count()) return launch_fmt<32>(p, st);
    return launch_fmt<64>(p, st);
}

}  // namespace fp8q
