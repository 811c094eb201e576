// moe_rows.cu -- tokens to the rows of their experts and back.
//
//   dispatch   row r of token t = src[r] / top_k:  v = w * x[t] (w = 1 without weights), in 1x128 blocks as codes:
//              s = MAX / max(amax(v), eps), q = fp8(RN_f32(v * s)); rows without a pair (src -1, or pos gives the
//              pair another row or none) are zeros
//   combine    y[t] = RN(residual[t] + sum over k of w[t, k] * x[pos[t, k]]), fp32, k ascending
//   weights    dw[t, k] = <dy[t], x[pos[t, k]]>, fp32
//
// The dispatch goes by tokens: a token is read and quantized once and its codes are written to its top_k rows.  (Row by
// row it would be read from DRAM top_k times: an expert's rows sweep all tokens.)  With a weight the block's amax is
// RN(|w| amax(x)), the same as the maximum of the rounded products because rounding is monotonic.  The transposed copy
// needs the maxima of 128 rows, so it is a kernel of its own over blocks of rows, which reads a token top_k times; its
// tiles walk down all rows before the next 256 bytes of columns, so that these of all tokens (16384 x 128 bf16: 4 MiB)
// stay in L2 meanwhile.
//
// 16384 tokens of 7168 bf16 to 8 of 64 experts: the codes 198 us (1.2 GB, 93 % of the copy rate), bound by memory; the
// transposed copy 368 us.  Its reads alone, 1.9 GB from L2 in copies of 256 bytes, took 300 (of 355, before it compared
// src with pos), whether by bytes or by copies is not known: L2 and DRAM are each below a third of their rates.  Forms that
// moved the tile through registers and shared memory with three barriers, or through registers alone, took 400 to 440.
// Rows without a pair hold small calls (a warp zeroes 32 of them, a thread its row of a transposed tile): 300 tokens to 8 of
// 16 experts, each rounded up to 128 rows, 24 us for the codes (5.7 with packed rows) and 54 with the transposed copy.

#include <algorithm>

#include "fp8q_device.cuh"
#include "fp8q_launch.h"
#include "gated_act.cuh"
#include "launch_util.h"
#include "moe.h"
#include "umma.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kTT = 128;  // rows of a block of the transposed copy

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

// The pair that src gives row `row`, or none (negative); and the row that pos gives a pair.  A row has a pair where both
// agree, because a program may drop pairs of a route by their pos.  Each is looked up one step before it is needed: in one
// step the two loads cost 64 tokens 0.15 us (of 2.47), 16384 x 7168 with the transposed copy 32 (of 551); so, nothing and 12.
__device__ __forceinline__ int src_pair(const MoeRoute& r, int64_t row, int64_t rows) {
    const int pair = row < rows ? __ldg(r.src + row) : -1;
    return pair < r.tokens * r.top_k ? pair : -1;
}
__device__ __forceinline__ int pos_row(const MoeRoute& r, int pair) { return pair >= 0 ? __ldg(r.pos + pair) : -1; }

// Zeros on the rows without a pair, a warp for 32 of them; `pair` is src_pair of the lane's first row.
__device__ __forceinline__ int64_t first_row() {
    return (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * 32 + (threadIdx.x & 31);
}
template <int FMT>
__device__ __forceinline__ void zero_rows(const MoeDispatchArgs& p, int64_t used, int pair) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads, blocks = p.cols / 128;
    for (int64_t r = first_row(); r - lane < used; r += step) {
        const int at = pos_row(p.r, pair);
        pair = src_pair(p.r, r + step, used);
        unsigned empty = __ballot_sync(0xFFFFFFFFu, r < used && at != r);
        while (empty != 0) {
            const int64_t row = r - lane + __ffs(empty) - 1;
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
    const int64_t blocks = p.cols / 128, total = p.r.tokens * blocks, used = rows_used(p.r);
    const int first_pair = src_pair(p.r, first_row(), p.r.rows);  // for zero_rows, on its way meanwhile
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
        // 8 pairs at a time: lane k of the block finds row, weight and scale of pair k, and writes the scale
        for (int64_t k0 = 0; k0 < p.r.top_k; k0 += 8) {
            const int n = static_cast<int>(min(int64_t(8), p.r.top_k - k0));
            int mine = -1;
            float w = 0.0f;
            if (live && sub < n) {
                mine = __ldg(p.r.pos + t * p.r.top_k + k0 + sub);
                if (mine >= used) mine = -1;  // behind the last expert named
                if (WEIGHTED) {
                    w = __ldg(p.weights + t * p.r.top_k + k0 + sub);
                    s = scale_from_amax<FMT>(fmaxf(__fmul_rn(fabsf(w), amax), 0.0f));
                }
                if (mine >= 0) p.scales[mine * blocks + blk] = s;
            }
            for (int k = 0; k < n; ++k) {
                const int row = __shfl_sync(0xFFFFFFFFu, mine, k, 8);
                if constexpr (WEIGHTED) {
                    const float wk = __shfl_sync(0xFFFFFFFFu, w, k, 8), sk = __shfl_sync(0xFFFFFFFFu, s, k, 8);
                    const uint64_t w2 = f32x2(wk, wk);
                    float u[16];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 x = f32x2_split(mul_f32x2(f32x2(v[j], v[j + 1]), w2));
                        u[j] = x.x;
                        u[j + 1] = x.y;
                    }
                    c = codes16<FMT>(u, sk);
                }
                if (row >= 0) st_stream(reinterpret_cast<uint4*>(p.q + static_cast<int64_t>(row) * p.cols + at), c);
            }
        }
    }
    zero_rows<FMT>(p, used, first_pair);
}

// The transposed copy, in tiles of 128 rows (one block of every column) x 256 bytes of a row.  A warp takes 64 bytes of
// all 128 rows and needs no other warp: lane (r8, c4), r8 = lane / 4 and c4 = lane % 4, holds rows 16 r8 .. 16 r8 + 15 of
// 16 bytes of columns.  A column's maximum is one in the lane and three shuffles; the codes of two rows of a column leave
// the conversion side by side, so that a lane has 16 consecutive bytes of each of its columns and the 8 lanes of a column
// write its 128-byte line.  The CTAs are persistent: the next tile's rows are on their way to shared memory, a bulk copy
// a row, while this one is computed from registers, and the tokens of the one after it are looked up.
template <typename T>
struct Vec16;  // 16 bytes of a row: kCols columns
template <>
struct Vec16<uint16_t> {
    static constexpr int kCols = 8;
    uint32_t w[4];
    __device__ __forceinline__ float at(int j) const { return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]); }
    static __device__ __forceinline__ Vec16 load(const uint16_t* p) {
        const uint4 v = ld_stream(reinterpret_cast<const uint4*>(p));
        return Vec16{{v.x, v.y, v.z, v.w}};
    }
    static __device__ __forceinline__ void store(uint16_t* p, const float* a) {
        st_stream(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                          pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])));
    }
};
template <>
struct Vec16<float> {
    static constexpr int kCols = 4;
    uint32_t w[4];
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(w[j]); }
    static __device__ __forceinline__ Vec16 load(const float* p) {
        const uint4 v = ld_stream(reinterpret_cast<const uint4*>(p));
        return Vec16{{v.x, v.y, v.z, v.w}};
    }
    static __device__ __forceinline__ void store(float* p, const float* a) {
        st_stream(reinterpret_cast<uint4*>(p),
                  make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3])));
    }
};

constexpr int kTransposeThreads = 128;  // a row of the tile each
// CTAs an SM: as many as registers allow without spills that cost more.  16384 x 7168 bf16 to 8 of 64 experts without
// weights 563 us a call with 5, 592 with 4; 16384 x 4096 bf16 with weights 530 us a call with 3, 571 with 4.
template <typename T, bool WEIGHTED>
constexpr int kTransposeCtas = sizeof(T) == 4 ? 4 : WEIGHTED ? 3 : 5;
constexpr int kRowBytes = 256;
static_assert(kTransposeThreads == kTT, "a thread a row");

// Where row r of a tile starts: rows 16 apart, which a load takes together, lie 64 bytes apart in the banks.
__device__ __forceinline__ int row_place(int r) { return r * kRowBytes + (r >> 4) * 64; }
constexpr int kTileBytes = kTT * kRowBytes + 8 * 64;

// 256 bytes of a row to shared memory, counted on `bar`.
__device__ __forceinline__ void copy_row(void* dst, const void* src, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     umma::smem_u32(dst)),
                 "l"(src), "r"(kRowBytes), "r"(umma::smem_u32(bar))
                 : "memory");
}

template <typename T, int FMT, bool WEIGHTED>
__global__ void __launch_bounds__(kTransposeThreads, (kTransposeCtas<T, WEIGHTED>))
k_moe_transpose(MoeDispatchArgs p, uint32_t magic, int shift, unsigned int* status) {
    using V = Vec16<T>;
    constexpr int kCols = V::kCols;
    __shared__ __align__(128) uint8_t buf[kTileBytes];
    __shared__ __align__(16) float weights[kTT];
    __shared__ uint64_t full;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r8 = lane >> 2, c4 = lane & 3;
    if (tid == 0) {
        umma::mbar_init(&full, kTT);
        umma::fence_mbar_init();
    }
    pdl_enter();
    const int64_t used = rows_used(p.r);
    // Tiles (block of rows, tile of columns), down the rows in use, a column tile after another.
    const unsigned tiles_r = static_cast<unsigned>((used + kTT - 1) / kTT), tiles_c = static_cast<unsigned>(p.cols / (16 * kCols));
    if (tiles_r == 0) return;
    struct Place {
        unsigned r, c;
    };
    const unsigned step_c = gridDim.x / tiles_r, step_r = gridDim.x - step_c * tiles_r;
    auto after = [&](Place t) {
        t.r += step_r;
        t.c += step_c;
        if (t.r >= tiles_r) {
            t.r -= tiles_r;
            ++t.c;
        }
        return t;
    };
    // This thread's row of the tile to be fetched: its pair, and the row and weight that the pair has.  The pair of the
    // tile after that is looked up one tile earlier than they are.
    int pair = -1, at = -1, pair_after = -1;
    float weight = 0.0f;
    auto row_of = [&](Place t) { return static_cast<int64_t>(t.r) * kTT + tid; };
    auto look_up_pair = [&](Place t) { pair_after = src_pair(p.r, row_of(t), t.c < tiles_c ? used : 0); };
    auto look_up = [&] {
        pair = pair_after;
        at = pos_row(p.r, pair);
        if (WEIGHTED) weight = pair >= 0 ? __ldg(p.weights + pair) : 0.0f;
    };
    auto fetch = [&](Place t) {
        uint8_t* dst = buf + row_place(tid);
        const bool real = pair >= 0 && at == row_of(t);
        if (WEIGHTED) weights[tid] = real ? weight : 0.0f;
        if (real) {
            const int64_t token = (static_cast<uint64_t>(static_cast<uint32_t>(pair)) * magic) >> shift;
            umma::fence_to_async();  // this row may hold zeros written by this thread
            umma::mbar_arrive_expect_tx(&full, kRowBytes);
            copy_row(dst, static_cast<const T*>(p.x) + token * p.cols + static_cast<int64_t>(t.c) * (16 * kCols), &full);
        } else {
#pragma unroll 4
            for (int i = 0; i < kRowBytes / 16; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
            umma::mbar_arrive(&full);
        }
    };
    Place t = {blockIdx.x % tiles_r, blockIdx.x / tiles_r};
    __syncthreads();
    Place next = after(t);
    if (t.c < tiles_c) {
        look_up_pair(t);
        look_up();
        look_up_pair(next);
        fetch(t);
        look_up();
        look_up_pair(after(next));
    }
    for (uint32_t phase = 0; t.c < tiles_c; phase ^= 1) {
        const bool ok = umma::mbar_wait(&full, phase, kWaitLimitNs);
        V x[16];
        const uint8_t* from = buf + row_place(r8 * 16) + (warp * 4 + c4) * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(from + i * kRowBytes);
            x[i].w[0] = v.x, x[i].w[1] = v.y, x[i].w[2] = v.z, x[i].w[3] = v.w;
        }
        uint64_t w2[8];  // the weights of two rows
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w2[i] = 0;
            if (WEIGHTED) {
                const float2 w = *reinterpret_cast<const float2*>(&weights[r8 * 16 + 2 * i]);
                w2[i] = f32x2(w.x, w.y);
            }
        }
        if (__syncthreads_or(!ok)) {  // every thread has read the tile; or a copy did not come: nothing more is fetched
            if (tid == 0) {
                atomicOr(status, kStatusWaitTimeout);
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000ull) {
                }
            }
            __syncthreads();
            return;
        }
        const int64_t r0 = static_cast<int64_t>(t.r) * kTT;
        const int64_t c0 = static_cast<int64_t>(t.c) * (16 * kCols) + (warp * 4 + c4) * kCols;  // the lane's first column
        if (next.c < tiles_c) fetch(next);
        t = next;
        next = after(next);
        look_up();
        look_up_pair(after(next));
        auto rows2 = [&](int i, int j) {  // rows 2 i, 2 i + 1 of column j
            const uint64_t v = f32x2(x[2 * i].at(j), x[2 * i + 1].at(j));
            return WEIGHTED ? mul_f32x2(v, w2[i]) : v;
        };
        float m[kCols];
        if constexpr (sizeof(T) == 2 && !WEIGHTED) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t a = x[0].w[k];
#pragma unroll
                for (int i = 1; i < 16; ++i) a = xabsmax_bf16x2(a, x[i].w[k]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) a = xabsmax_bf16x2(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
                a &= 0x7FFF7FFFu;
                m[2 * k] = bf16_lo(a);
                m[2 * k + 1] = bf16_hi(a);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                m[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 v = f32x2_split(rows2(i, j));
                    m[j] = absmax3(m[j], v.x, v.y);
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], d));
            }
        }
        // one scale a lane: column r8 of its kCols (fp32: every scale twice)
        float mine = m[0];
#pragma unroll
        for (int j = 1; j < kCols; ++j) mine = r8 % kCols == j ? m[j] : mine;
        const float s_mine = scale_from_amax<FMT>(mine);
        if (r8 < kCols) p.scales_t[(c0 + r8) * (p.r.rows / kTT) + r0 / kTT] = s_mine;
        uint8_t* dst = p.qt + c0 * p.r.rows + r0 + r8 * 16;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float s = __shfl_sync(0xFFFFFFFFu, s_mine, j * 4 + c4);
            const uint64_t s2 = f32x2(s, s);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = f32x2_split(mul_f32x2(rows2(2 * i, j), s2)), b = f32x2_split(mul_f32x2(rows2(2 * i + 1, j), s2));
                w[i] = cvt_fp8x2<FMT>(a.x, a.y) | (cvt_fp8x2<FMT>(b.x, b.y) << 16);
            }
            st_stream(reinterpret_cast<uint4*>(dst + j * p.r.rows), make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

// y[t] over 32 bytes of columns a thread, two pairs' rows in flight.  16384 x 7168 bf16, 8 rows a token and a residual:
// 350 us, the same with four rows in flight (385 with eight), 361 with one; 1001 x 4096 fp32, 6 rows: 19.8, 20.5 and 22.5.
constexpr int kAtOnce = 2;
constexpr int kVecs = 2;

template <typename T>
__global__ void __launch_bounds__(kThreads) k_moe_combine(MoeCombineArgs p) {
    using V = Vec16<T>;
    constexpr int kRun = kVecs * V::kCols;
    pdl_enter();
    const int64_t runs = p.cols / kRun, total = p.tokens * runs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = i / runs, at = (i - t * runs) * kRun;
        const T* x = static_cast<const T*>(p.x) + at;
        const int32_t* pos = p.pos + t * p.top_k;
        float acc[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) acc[j] = 0.0f;
        if (p.residual != nullptr) {
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const V v = V::load(static_cast<const T*>(p.residual) + t * p.cols + at + u * V::kCols);
#pragma unroll
                for (int j = 0; j < V::kCols; ++j) acc[u * V::kCols + j] = v.at(j);
            }
        }
        for (int64_t k0 = 0; k0 < p.top_k; k0 += kAtOnce) {
            V v[kAtOnce][kVecs];
            float w[kAtOnce];
            bool real[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int64_t row = k0 + k < p.top_k ? __ldg(pos + k0 + k) : -1;
                real[k] = row >= 0 && row < p.rows;
                if (real[k]) {
#pragma unroll
                    for (int u = 0; u < kVecs; ++u) v[k][u] = V::load(x + row * p.cols + u * V::kCols);
                    w[k] = p.weights != nullptr ? __ldg(p.weights + t * p.top_k + k0 + k) : 1.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (!real[k]) continue;
#pragma unroll
                for (int j = 0; j < kRun; ++j) acc[j] = __fmaf_rn(w[k], v[k][j / V::kCols].at(j % V::kCols), acc[j]);
            }
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) V::store(static_cast<T*>(p.y) + t * p.cols + at + u * V::kCols, acc + u * V::kCols);
    }
}

// A CTA a token: every thread a share of the columns, two rows in flight, the sums joined in a fixed order.  16384 x 4096
// bf16, 8 rows a token, 1.2 GB: 172 us, 187 with one row in flight, 200 with 256 threads.
constexpr int kDotThreads = 128;
constexpr int kDots = 8;  // weights at a time

template <typename T>
__global__ void __launch_bounds__(kDotThreads) k_moe_weight_grad(const T* __restrict__ dy, const T* __restrict__ x,
                                                                 const int32_t* __restrict__ pos, int64_t top_k,
                                                                 int64_t rows, int64_t cols, float* __restrict__ dweights) {
    using V = Vec16<T>;
    constexpr int kRun = kVecs * V::kCols;
    __shared__ float part[kDotThreads / 32][kDots];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    for (int64_t k0 = 0; k0 < top_k; k0 += kDots) {
        const int n = static_cast<int>(min(static_cast<int64_t>(kDots), top_k - k0));
        int row[kDots];
        float acc[kDots];
#pragma unroll
        for (int k = 0; k < kDots; ++k) {
            row[k] = k < n ? __ldg(pos + t * top_k + k0 + k) : -1;
            if (row[k] >= rows) row[k] = -1;
            acc[k] = 0.0f;
        }
        for (int64_t at = threadIdx.x * kRun; at < cols; at += kDotThreads * kRun) {
            V d[kVecs];
#pragma unroll
            for (int u = 0; u < kVecs; ++u) d[u] = V::load(dy + t * cols + at + u * V::kCols);
#pragma unroll
            for (int k1 = 0; k1 < kDots; k1 += kAtOnce) {
                if (k1 >= n) break;
                V v[kAtOnce][kVecs];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                    for (int u = 0; u < kVecs; ++u)
                        if (row[k1 + k] >= 0) v[k][u] = V::load(x + static_cast<int64_t>(row[k1 + k]) * cols + at + u * V::kCols);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    if (row[k1 + k] < 0) continue;
#pragma unroll
                    for (int j = 0; j < kRun; ++j)
                        acc[k1 + k] = __fmaf_rn(d[j / V::kCols].at(j % V::kCols), v[k][j / V::kCols].at(j % V::kCols), acc[k1 + k]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kDots; ++k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[k] += __shfl_xor_sync(0xFFFFFFFFu, acc[k], o);
            if (lane == 0) part[warp][k] = acc[k];
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n) {
            float sum = part[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kDotThreads / 32; ++w) sum += part[w][threadIdx.x];
            dweights[t * top_k + k0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

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
            const int64_t tiles = p.cols / (16 * Vec16<T>::kCols) * (p.r.rows / kTT);
            if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;
            unsigned int* status = device_status_word();
            if (status == nullptr) return cudaErrorInvalidValue;
            // n / top_k = (n * magic) >> shift for 0 <= n < 2^31: with 2^(k-1) < top_k <= 2^k and magic the next whole number
            // above 2^(31+k) / top_k, magic * top_k - 2^(31+k) <= 2^k
            int k = 0;
            while ((int64_t(1) << k) < p.r.top_k) ++k;
            const uint32_t magic = static_cast<uint32_t>((uint64_t(1) << (31 + k)) / static_cast<uint64_t>(p.r.top_k) + 1);
            const int64_t ctas = std::min<int64_t>(tiles, static_cast<int64_t>(device_sm_count()) * kTransposeCtas<T, WEIGHTED>);
            return launch_kernel(k_moe_transpose<T, FMT, WEIGHTED>, dim3(static_cast<unsigned>(ctas)), dim3(kTransposeThreads), 0,
                                 st, p, magic, 31 + k, status);
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
    const int64_t run = kVecs * (dtype == 0 ? Vec16<float>::kCols : Vec16<uint16_t>::kCols);
    const dim3 grid(grid_of(p.tokens * (p.cols / run), kThreads));
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
