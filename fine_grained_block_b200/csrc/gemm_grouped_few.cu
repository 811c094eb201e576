// gemm_grouped_few.cu -- the experts' products for few rows an expert: single tokens, decode batches, short prompts.
//
// The products and factors of gemm_grouped.cu, whose sums over K it repeats bit for bit where K is not split; split,
// they are added in another order.
//
// The work is reading the weights of the experts that have rows.  As in gemm_gated_few.cu the tensor core's M side takes
// 256 weight rows in two accumulators (gate and up rows of 128 columns, or 256 columns of a plain product), its N side
// NT rows of A (16 or 32; an expert with more takes several blocks, whose weights come from L2), and K is split over a
// cluster of S CTAs whose partial sums meet in distributed shared memory in rank order.  The grid's y is a list of
// (expert, block of NT rows): the device alone knows it, so every CTA counts the experts' blocks up (one load and a
// scan), takes its own, and leaves where there is none.
//
// Bound by HBM (the weights): one token and 8 of 64 experts of 7168 x 2048 gated, 235 MB, takes 40 us (36 at the copy
// rate); 48 tokens and 4 of 32 experts of 2048 x 7168, 473 MB, 78 us (72).

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

constexpr int kBlock = 128;              // weight rows of an accumulator
constexpr int kBK = 128;
constexpr int kMmaK = 32;
constexpr int kWBytes = kBlock * kBK;    // one weight box
constexpr int kAhead = 2;                // chunks ahead that the scales are loaded
constexpr int kMaxSplit = 8;

constexpr int kPromoteWarps = 8;
constexpr int kWarps = 2 + kPromoteWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtas = 2;                 // CTAs per SM
constexpr int kStages = 3;
constexpr uint32_t kTmemCols = 256;

template <int NT>
struct Few {
    static constexpr int kPer = NT / 2;  // rows of a promotion warp
    static constexpr int kBufs = static_cast<int>(kTmemCols) / (2 * NT);
    static constexpr int kStageBytes = 2 * kWBytes + NT * kBK;
    struct Tail {
        uint64_t full[kStages];
        uint64_t empty[kStages];
        uint64_t acc_full[kBufs];
        uint64_t acc_empty[kBufs];
        uint32_t tmem_base;
        int32_t item[3];          // this CTA's expert (-1: none), first row, rows
        uint32_t warp_sum[kWarps];
        alignas(16) float fac[kPromoteWarps][2][2][kPer];  // [warp][chunk parity][block][row]
    };
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024 /* alignment */ + static_cast<int>(sizeof(Tail));
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "the CTAs of an SM share its shared memory");
    static_assert(2 * NT * kBlock * 4 <= kStages * kStageBytes, "the partial sums fit where the stages were");
};

// A warp finishes a row of A: its 128 columns of both blocks, 4 a lane.  The sums over the ranks in rank order, all
// loads before the first use (one trip through the cluster's network).
template <int NT, bool GATED, int FMT, int SPLIT>
__device__ __forceinline__ void finish(const GroupedArgs& p, uint32_t part0, int rank, int pw, int lane, int tile,
                                       int64_t m0, int M) {
    const int64_t F = p.N / 2;
    const int64_t x = static_cast<int64_t>(tile) * (GATED ? kBlock : 2 * kBlock) + 4 * lane, apart = GATED ? F : kBlock;
    const bool second = GATED || (static_cast<int64_t>(tile) * 2 + 1) * kBlock < p.N;  // the last tile may have one block
    for (int m = rank + SPLIT * pw; m < M; m += SPLIT * kPromoteWarps) {
        float4 g[SPLIT], u[SPLIT];
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
            const uint32_t at = umma::mapa(part0, static_cast<uint32_t>(r)) + static_cast<uint32_t>((m * kBlock + 4 * lane) * 4);
            g[r] = umma::ld_cluster_f32x4(at);
            u[r] = umma::ld_cluster_f32x4(at + NT * kBlock * 4);
        }
#pragma unroll
        for (int r = 1; r < SPLIT; ++r) {
            g[0] = make_float4(g[0].x + g[r].x, g[0].y + g[r].y, g[0].z + g[r].z, g[0].w + g[r].w);
            u[0] = make_float4(u[0].x + u[r].x, u[0].y + u[r].y, u[0].z + u[r].z, u[0].w + u[r].w);
        }
        if (p.c != nullptr) {
            const int64_t at = (m0 + m) * p.N + x;
            if (p.c_dtype == 0) {
                *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) = g[0];
                if (second) *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at + apart) = u[0];
            } else {
                uint16_t* c = static_cast<uint16_t*>(p.c) + at;
                *reinterpret_cast<uint2*>(c) = make_uint2(pack_bf16x2(g[0].x, g[0].y), pack_bf16x2(g[0].z, g[0].w));
                if (second)
                    *reinterpret_cast<uint2*>(c + apart) = make_uint2(pack_bf16x2(u[0].x, u[0].y), pack_bf16x2(u[0].z, u[0].w));
            }
        }
        if constexpr (GATED) {
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
            const float2 v = f32x2_split(h01), w = f32x2_split(h23);
            const float s = scale_from_amax<FMT>(
                warp_max<32>(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(w.x), fabsf(w.y)))));
            const float2 c = f32x2_split(mul_f32x2(h01, both(s))), d = f32x2_split(mul_f32x2(h23, both(s)));
            *reinterpret_cast<uint32_t*>(p.q + (m0 + m) * F + x) =
                cvt_fp8x2<FMT>(c.x, c.y) | (cvt_fp8x2<FMT>(d.x, d.y) << 16);
            if (lane == 0) p.scales[(m0 + m) * (F / kBlock) + tile] = s;
        }
    }
}

template <int NT, bool GATED, int FMT>
__global__ void __launch_bounds__(kThreads, kCtas)
k_gemm_grouped_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
                   const __grid_constant__ GroupedArgs p, uint32_t idesc, unsigned int* status, int split) {
    using C = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto* tail = reinterpret_cast<typename C::Tail*>(stages + kStages * C::kStageBytes);
    float* part = reinterpret_cast<float*>(stages);  // after the last chunk: [block][row][column]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(umma::cluster_ctarank());
    const int tile = static_cast<int>(blockIdx.x / static_cast<unsigned>(split));
    const int blocks = static_cast<int>(p.N / kBlock);  // of an expert's weight rows
    const int b0 = GATED ? tile : 2 * tile;             // this tile's two blocks
    const int b1 = GATED ? tile + blocks / 2 : 2 * tile + 1;
    const int all_chunks = static_cast<int>(p.K / kBK);
    const int c0 = static_cast<int>(static_cast<int64_t>(all_chunks) * rank / split);
    const int c1 = static_cast<int>(static_cast<int64_t>(all_chunks) * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            umma::mbar_init(&tail->full[s], 1);
            umma::mbar_init(&tail->empty[s], 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            umma::mbar_init(&tail->acc_full[b], 1);
            umma::mbar_init(&tail->acc_empty[b], kPromoteWarps);
        }
        umma::fence_mbar_init();
        tail->item[0] = -1;
    }
    if (warp == 1) umma::tmem_alloc(&tail->tmem_base, kTmemCols);
    umma::fence_before_sync();
    __syncthreads();  // allocated before the next kernel may start
    umma::fence_after_sync();
    const uint32_t tmem = tail->tmem_base;
    pdl_enter();  // the codes, scales and offsets may come from the previous kernel
    {   // this CTA's expert and rows: the blocks of the experts before, by a scan of up to 4 experts a thread
        constexpr int kPerThread = (kMaxExperts + kThreads - 1) / kThreads;
        const int per = (p.E + kThreads - 1) / kThreads, R = static_cast<int>(p.R);
        int lo[kPerThread + 1];
        uint32_t n[kPerThread], sum = 0;
        const int e0 = static_cast<int>(threadIdx.x) * per;
#pragma unroll
        for (int i = 0; i <= kPerThread; ++i) lo[i] = i <= per ? min(max(p.offsets[min(e0 + i, p.E)], 0), R) : 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            n[i] = i < per && e0 + i < p.E && lo[i + 1] > lo[i] ? static_cast<uint32_t>(lo[i + 1] - lo[i] + NT - 1) / NT : 0u;
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
        uint32_t before = upto - sum;
        for (int w = 0; w < warp; ++w) before += tail->warp_sum[w];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (blockIdx.y >= before && blockIdx.y < before + n[i]) {
                const int m = lo[i] + static_cast<int>(blockIdx.y - before) * NT;
                tail->item[0] = e0 + i;
                tail->item[1] = m;
                tail->item[2] = min(lo[i + 1] - m, NT);
            }
            before += n[i];
        }
    }
    __syncthreads();
    const int e = tail->item[0], m0 = tail->item[1], M = tail->item[2];
    if (e < 0) {  // no rows left: the whole cluster leaves
        if (warp == 1) umma::tmem_dealloc(tmem, kTmemCols);
        return;
    }
    const int w0 = static_cast<int>(e * p.N) + b0 * kBlock, w1 = static_cast<int>(e * p.N) + b1 * kBlock;

    bool timed_out = false;
    if (warp == 0) {
        if (lane == 0) {
            for (int c = c0; c < c1; ++c) {
                const uint32_t g = static_cast<uint32_t>(c - c0), s = g % kStages;
                if (!umma::mbar_wait(&tail->empty[s], ((g / kStages) & 1u) ^ 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                uint8_t* stage = stages + s * C::kStageBytes;
                umma::mbar_arrive_expect_tx(&tail->full[s], C::kStageBytes);
                umma::tma_load_2d(stage, &map_w, &tail->full[s], c * kBK, w0);
                umma::tma_load_2d(stage + kWBytes, &map_w, &tail->full[s], c * kBK, w1);
                umma::tma_load_2d(stage + 2 * kWBytes, &map_t, &tail->full[s], c * kBK, m0);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int c = c0; c < c1; ++c) {
                const uint32_t g = static_cast<uint32_t>(c - c0), s = g % kStages, buf = g % C::kBufs;
                if (!umma::mbar_wait(&tail->acc_empty[buf], ((g / C::kBufs) & 1u) ^ 1u, kWaitLimitNs) ||
                    !umma::mbar_wait(&tail->full[s], (g / kStages) & 1u, kWaitLimitNs)) {
                    timed_out = true;
                    break;
                }
                umma::fence_after_sync();
                const uint32_t w_addr = umma::smem_u32(stages + s * C::kStageBytes);
                const uint64_t t_desc = umma::smem_desc_kmajor_sw128(w_addr + 2 * kWBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
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
        const float* sg_row = p.sb + (static_cast<int64_t>(e) * blocks + b0) * all_chunks;
        const float* su_row = p.sb + (static_cast<int64_t>(e) * blocks + min(b1, blocks - 1)) * all_chunks;
        // lane j < H forms the factors of the warp's row j
        const int my_row = group * H + lane;
        const bool mine = lane < H && my_row < M;
        const float* sa_row = p.sa + static_cast<int64_t>(m0 + (mine ? my_row : 0)) * all_chunks;
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
            for (int h = 0; h < 2; ++h) {
                float v[H];
                umma::tmem_read<H>(tm + h * NT, v);
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
                for (int j = 0; j < H; ++j) part[(h * NT + group * H + j) * kBlock + f] = acc[h][j];
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
    if (warp >= 2 && !bad) {  // the rows m % split == rank
        const uint32_t part0 = umma::smem_u32(part);
        switch (split) {
            case 1: finish<NT, GATED, FMT, 1>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
            case 2: finish<NT, GATED, FMT, 2>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
            case 4: finish<NT, GATED, FMT, 4>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
            default: finish<NT, GATED, FMT, kMaxSplit>(p, part0, rank, warp - 2, lane, tile, m0, M); break;
        }
    }
    __syncwarp();
    umma::cluster_sync();  // no CTA leaves while another may read its shared memory
    if (warp == 1) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, kTmemCols);
    }
}

// Blocks of NT rows: with a last one half full for each expert that can have rows, or one for each.
int64_t likely_blocks(const GroupedArgs& p, int nt) {
    const int64_t experts = std::min<int64_t>(p.E, p.R);
    return std::max(p.R / nt + experts / 2, experts);
}

template <int NT, bool GATED, int FMT>
cudaError_t launch_typed(const GroupedArgs& p, cudaStream_t st) {
    using C = Few<NT>;
    CUtensorMap map_w, map_t;
    if (!make_code_map(&map_w, p.b, p.E * p.N, p.K, kBlock) || !make_code_map(&map_t, p.a, p.R, p.K, NT))
        return cudaErrorInvalidValue;
    unsigned int* status = device_status_word();
    if (status == nullptr) return cudaErrorInvalidValue;
    auto kern = k_gemm_grouped_few<NT, GATED, FMT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    const int64_t tiles = (p.N / kBlock + 1) / 2, chunks = p.K / kBK;
    const int64_t items = p.R / NT + std::min<int64_t>(p.E, p.R);  // no more than these, however the rows are shared out
    if (items > 65535 || tiles * kMaxSplit > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
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
    static std::atomic<bool> opted[128];  // the shared-memory opt-in, once per device
    if (!opted[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_release);
    }
    // The widest split of K whose CTAs fill the device no more than once; a rank takes two chunks at least, four of eight.
    int split = 1;
    const int64_t work = tiles * likely_blocks(p, NT);
    for (int i = 0; i < 3 && (2 << i) * (i < 2 ? 2 : 4) <= chunks; ++i) {
        if (work * (2 << i) > static_cast<int64_t>(device_sm_count()) * kCtas) break;
        split = 2 << i;
    }
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), static_cast<unsigned>(items));
    const uint32_t idesc = umma::instr_desc_f8f6f4(p.b_fmt, p.a_fmt, kBlock, NT);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, map_w, map_t, p, idesc, status, split);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT>
cudaError_t launch_kind(const GroupedArgs& p, bool gated, cudaStream_t st) {
    if (!gated) return launch_typed<NT, false, kE4M3>(p, st);
    return p.fmt == kE4M3 ? launch_typed<NT, true, kE4M3>(p, st) : launch_typed<NT, true, kE5M2>(p, st);
}

}  // namespace

bool gemm_grouped_few_fits(const GroupedArgs& p) {
    // Up to 24 rows an expert on average (64 experts of 7168 x 2048 gated: 308 us here and 336 in gemm_grouped.cu with 24,
    // 336 and 338 with 32; 32 experts of 2048 x 7168: 91 and 97 with 20, 99 and 99 with 24, 101 and 92 with 32), and more
    // while K can still be split in two with all CTAs resident (4 experts of 4096 x 1024 gated: 20.6 and 24.5 us with 100
    // rows, 34.2 and 24.8 with 150; of 4096 x 2048: 21.5 and 25.9 with 50, 34.7 and 26.8 with 75).
    const int64_t experts = std::min<int64_t>(p.E, p.R);
    if (p.R / 16 + experts > 65535) return false;
    return p.R <= 24 * experts || (p.N / kBlock + 1) / 2 * likely_blocks(p, 32) <= device_sm_count() * kCtas / 2;
}

cudaError_t launch_gemm_grouped_few(const GroupedArgs& p, bool gated, cudaStream_t st) {
    // Up to 8 rows an expert on average 16 a block, else 32 (64 experts of 7168 x 2048 gated: 267 and 282 us with 8, 296
    // and 276 with 10; one row 40 and 42).  Blocks of 64, one CTA an SM, were never the fastest.
    return p.R <= 8 * std::min<int64_t>(p.E, p.R) ? launch_kind<16>(p, gated, st) : launch_kind<32>(p, gated, st);
}

}  // namespace fp8q
