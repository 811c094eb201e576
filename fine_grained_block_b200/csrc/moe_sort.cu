// moe_sort.cu -- (token, expert) pairs sorted by expert.
//
// A counting sort of the pairs p = t * top_k + k by e = experts[p]:
//   counts[e]  = #{p : experts[p] = e}
//   offsets[e] = sum over f < e of counts[f] rounded up to `align`
//   pos[p]     = offsets[e] + #{p' < p : experts[p'] = e}, -1 for an id outside 0 .. E - 1
//   src        = the inverse of pos; -1 on the rows between the experts and behind the last
// Stable, and whole numbers only: the result does not depend on timing.
//
// The pairs are cut into chunks, one a CTA.  The first kernel counts each chunk; in the second every CTA adds the
// counts up itself (chunks before its own, and all), forms the offsets by a scan over the experts, and ranks its
// pairs, 1024 at a time: a pair's rank is that among its warp's equals (match_any), plus the equals of the warps
// before (a 32-entry row per expert in shared memory, scanned by one thread), plus those of the batches before.
// Few pairs are one chunk and one kernel; up to 1024, one batch, need no counting pass: the ranks' rows give the counts.
//
// Bound by latency: 131072 pairs are 0.5 MB read and 1.2 MB written.

#include <algorithm>

#include "launch_util.h"
#include "moe.h"

namespace fp8q {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 128;
constexpr int64_t kMinChunk = 2 * kThreads;
constexpr int64_t kOneChunk = 4096;  // pairs that one CTA sorts alone

__device__ __forceinline__ int expert_of(const int32_t* experts, int64_t p, int num_experts) {
    const int e = experts[p];
    return static_cast<unsigned>(e) < static_cast<unsigned>(num_experts) ? e : -1;
}

__global__ void __launch_bounds__(kThreads) k_moe_count(MoeSortArgs p, int64_t chunk) {
    __shared__ int count[kMaxExperts];
    pdl_enter();
    const int tid = threadIdx.x;
    if (tid < p.num_experts) count[tid] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * chunk, hi = min(lo + chunk, p.pairs);
    for (int64_t i = lo + tid; i < hi; i += kThreads) {
        const int e = expert_of(p.experts, i, p.num_experts);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (tid < p.num_experts) p.workspace[static_cast<int64_t>(blockIdx.x) * p.num_experts + tid] = count[tid];
}

// Exclusive sum of v over the CTA's threads, and in `all` of all of them.
__device__ __forceinline__ int scan(int v, int* warp_sum, int* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += u;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    // every warp adds the warps' sums up itself
    int s = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += u;
    }
    *all = __shfl_sync(0xFFFFFFFFu, s, 31);
    const int before = __shfl_sync(0xFFFFFFFFu, s, max(warp - 1, 0));
    return sum - v + (warp > 0 ? before : 0);
}

// An expert's row of a batch: its pairs by warp become those of the warps before; returns their number.
__device__ __forceinline__ int scan_row(uint16_t* hist_row) {
    uint4* row = reinterpret_cast<uint4*>(hist_row);
    uint32_t run = 0;
#pragma unroll
    for (int j = 0; j < kWarps / 8; ++j) {
        const uint4 v = row[j];
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t a = w[k] & 0xFFFFu, c = w[k] >> 16;
            w[k] = run | ((run + a) << 16);
            run += a + c;
        }
        row[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return static_cast<int>(run);
}

__device__ __forceinline__ void clear_row(uint16_t* hist_row) {
#pragma unroll
    for (int j = 0; j < kWarps / 8; ++j) reinterpret_cast<uint4*>(hist_row)[j] = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ int padded(int n, int align) { return (n + align - 1) & -align; }

// One batch: a pair a thread.
__global__ void __launch_bounds__(kThreads) k_moe_sort_few(MoeSortArgs p) {
    extern __shared__ __align__(16) uint16_t hist[];
    __shared__ int first[kMaxExperts + 1], last[kMaxExperts];  // offsets, and the rows behind the experts' pairs
    __shared__ int warp_sum[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = p.num_experts;
    if (tid < E) clear_row(hist + tid * kWarps);
    pdl_enter();
    const int e = tid < p.pairs ? expert_of(p.experts, tid, E) : -1;
    __syncthreads();
    const unsigned equal = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(equal & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) hist[e * kWarps + warp] = static_cast<uint16_t>(__popc(equal));
    __syncthreads();
    const int n = tid < E ? scan_row(hist + tid * kWarps) : 0;
    int all;
    const int at = scan(tid < E ? padded(n, p.align) : 0, warp_sum, &all);
    if (tid < E) {
        first[tid] = at;
        last[tid] = at + n;
        p.offsets[tid] = at;
        if (p.counts != nullptr) p.counts[tid] = n;
        if (tid == E - 1) first[E] = p.offsets[E] = all;
    }
    __syncthreads();
    if (tid < p.pairs) {
        const int r = e >= 0 ? first[e] + hist[e * kWarps + warp] + rank : -1;
        p.pos[tid] = r;
        if (e >= 0) p.src[r] = tid;
    }
    for (int i = warp; i < E; i += kWarps)
        for (int r = last[i] + lane; r < first[i + 1]; r += 32) p.src[r] = -1;
    for (int64_t r = all + tid; r < p.rows; r += kThreads) p.src[r] = -1;
}

// ONE: the only chunk, which it counts itself.
template <bool ONE>
__global__ void __launch_bounds__(kThreads) k_moe_sort(MoeSortArgs p, int64_t chunk) {
    extern __shared__ __align__(16) uint16_t hist[];  // [E][kWarps]: a batch's pairs of an expert by warp, then those before
    __shared__ int total[kMaxExperts];                // pairs of an expert
    __shared__ int next[kMaxExperts];                 // rows of an expert before this batch
    __shared__ int first[kMaxExperts + 1];            // offsets
    __shared__ int warp_sum[kWarps];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = p.num_experts;
    const int64_t lo = blockIdx.x * chunk, hi = min(lo + chunk, p.pairs);
    if (tid < E) total[tid] = next[tid] = 0;
    int e_next = lo + tid < hi ? expert_of(p.experts, lo + tid, E) : -1;  // of the first batch
    __syncthreads();
    if (ONE) {
        for (int64_t i = lo + tid; i < hi; i += kThreads) {
            const int e = expert_of(p.experts, i, E);
            if (e >= 0) atomicAdd(&total[e], 1);
        }
    } else {
        const int parts = kThreads / E, part = tid / E, e = tid - part * E;
        if (part < parts) {
            int all = 0, before = 0;
            const int chunks = static_cast<int>(gridDim.x);
            for (int c0 = part; c0 < chunks; c0 += 16 * parts) {  // 16 loads at a time
                int n[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) n[k] = c0 + k * parts < chunks ? p.workspace[(c0 + k * parts) * E + e] : 0;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    all += n[k];
                    if (c0 + k * parts < static_cast<int>(blockIdx.x)) before += n[k];
                }
            }
            atomicAdd(&total[e], all);
            atomicAdd(&next[e], before);
        }
    }
    __syncthreads();
    // offsets: a scan over the experts, one a thread
    const int mine = tid < E ? padded(total[tid], p.align) : 0;
    int all;
    const int offset = scan(mine, warp_sum, &all);
    int at = 0;  // this thread's expert: its rows before this batch
    if (tid < E) {
        first[tid] = offset;
        if (tid == E - 1) first[E] = all;
        at = offset + next[tid];
        if (blockIdx.x == 0) {
            p.offsets[tid] = offset;
            if (tid == E - 1) p.offsets[E] = all;
            if (p.counts != nullptr) p.counts[tid] = total[tid];
        }
    }
    for (int64_t b = lo; b < hi; b += kThreads) {
        __syncthreads();
        if (tid < E) clear_row(hist + tid * kWarps);
        __syncthreads();
        const int64_t i = b + tid;
        const int e = e_next;
        e_next = i + kThreads < hi ? expert_of(p.experts, i + kThreads, E) : -1;
        const unsigned equal = __match_any_sync(0xFFFFFFFFu, e);
        const int rank = __popc(equal & ((1u << lane) - 1u));
        if (e >= 0 && rank == 0) hist[e * kWarps + warp] = static_cast<uint16_t>(__popc(equal));
        __syncthreads();
        if (tid < E) {
            next[tid] = at;
            at += scan_row(hist + tid * kWarps);
        }
        __syncthreads();
        if (i < hi) {
            const int r = e >= 0 ? next[e] + hist[e * kWarps + warp] + rank : -1;
            p.pos[i] = r;
            if (e >= 0) p.src[r] = static_cast<int32_t>(i);
        }
    }
    __syncthreads();
    // rows without a pair: behind an expert's last (a warp an expert), and behind the last expert
    for (int e = static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) * warp; e < E; e += static_cast<int>(gridDim.x) * kWarps)
        for (int r = first[e] + total[e] + lane; r < first[e + 1]; r += 32) p.src[r] = -1;
    for (int64_t r = first[E] + static_cast<int64_t>(blockIdx.x) * kThreads + tid; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * kThreads)
        p.src[r] = -1;
}

// Pairs a chunk: whole batches, two at least, so many that there are at most kMaxChunks chunks.  131072 pairs, 256 experts:
// 10.8 us in 64 chunks, 14.5 in 128 (whose counts every CTA adds up), 15.8 in 32.
int64_t chunk_pairs(int64_t pairs) {
    if (pairs <= kOneChunk) return std::max<int64_t>(pairs, 1);
    return std::max(kMinChunk, ((pairs + kThreads - 1) / kThreads + kMaxChunks - 1) / kMaxChunks * kThreads);
}
int64_t chunk_count(int64_t pairs) {
    const int64_t c = chunk_pairs(pairs);
    return std::max<int64_t>((pairs + c - 1) / c, 1);
}

}  // namespace

int64_t moe_sort_workspace_bytes(int64_t pairs, int num_experts) {
    const int64_t n = chunk_count(pairs);
    return n > 1 ? n * num_experts * 4 : 0;
}

cudaError_t launch_moe_sort(const MoeSortArgs& p, cudaStream_t st) {
    const int64_t chunk = chunk_pairs(p.pairs);
    const unsigned chunks = static_cast<unsigned>(chunk_count(p.pairs));
    const size_t smem = static_cast<size_t>(p.num_experts) * kWarps * sizeof(uint16_t);
    auto kern = chunks > 1 ? k_moe_sort<false> : k_moe_sort<true>;
    const bool few = p.pairs <= kThreads;
    if (smem > 32 * 1024) {  // beside up to 12 KiB of static shared memory
        constexpr int kMost = kMaxExperts * kWarps * static_cast<int>(sizeof(uint16_t));
        const cudaError_t e = few ? cudaFuncSetAttribute(k_moe_sort_few, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)
                                  : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
    }
    if (few) return launch_kernel(k_moe_sort_few, dim3(1), dim3(kThreads), smem, st, p);
    if (chunks > 1) {
        const cudaError_t e = launch_kernel(k_moe_count, dim3(chunks), dim3(kThreads), 0, st, p, chunk);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(kern, dim3(chunks), dim3(kThreads), smem, st, p, chunk);
}

}  // namespace fp8q
