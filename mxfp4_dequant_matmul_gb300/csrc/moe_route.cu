// moe_route.cu -- routing of tokens to experts and back (include/mx4.h
// mxfp4_moe_sort, _dispatch, _combine and their gradients).
//
// The sort is a stable counting sort of P = tokens * top_k pairs by expert id.
// One cluster of CTAs does it in one launch: every warp owns a contiguous run of
// pairs and a histogram of its own in shared memory (equal ids of a 32-pair step
// found by match, the lowest lane adds their count), the CTAs add up their
// totals through distributed shared memory, and each warp walks its run again
// with its histogram turned into running positions.  Latency-bound: two passes
// over 4 P bytes that stay in L1.
//
// The other kernels move rows and are bound by HBM.
#include <cooperative_groups.h>

#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mx4_kernels.h"

namespace mxk {
namespace {

namespace cg = cooperative_groups;

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;

__global__ void __launch_bounds__(kSortThreads)
    k_moe_sort(const int32_t* __restrict__ ids, int n_pairs, int top_k, int n_experts, int run,
               int32_t* __restrict__ token_at, int32_t* __restrict__ pos_of,
               int32_t* __restrict__ offsets) {
    extern __shared__ int32_t sort_smem[];
    int32_t* hist = sort_smem;                              // [kSortWarps][n_experts]
    int32_t* total = sort_smem + kSortWarps * n_experts;    // [n_experts], read by the cluster
    __shared__ int32_t warp_sum[kSortWarps];
    __shared__ int32_t n_kept;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int n_cta = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* mine = hist + warp * n_experts;

    for (int i = tid; i < kSortWarps * n_experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    const long long p0 = (static_cast<long long>(rank) * kSortWarps + warp) * run;
    const int lo = static_cast<int>(min(p0, static_cast<long long>(n_pairs)));
    const int hi = static_cast<int>(min(p0 + run, static_cast<long long>(n_pairs)));
    for (int p = lo; p < hi; p += 32) {
        const int id = p + lane < hi ? __ldg(ids + p + lane) : -1;
        const bool ok = id >= 0 && id < n_experts;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, ok ? id : -1);
        if (ok && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // per expert: exclusive sums over the warps, and the CTA's total
    for (int e = tid; e < n_experts; e += kSortThreads) {
        int32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = hist[w * n_experts + e];
            hist[w * n_experts + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    cluster.sync();
    // all CTAs' totals (n_experts <= kSortThreads: one expert per thread) and the
    // exclusive sum over the experts
    int32_t all = 0, before = 0;
    if (tid < n_experts) {
        for (int c = 0; c < n_cta; ++c) {
            const int32_t t = cluster.map_shared_rank(total, c)[tid];
            if (c < rank) before += t;
            all += t;
        }
    }
    int32_t scan = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, scan, d);
        if (lane >= d) scan += o;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int32_t s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= d) s += o;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    const int32_t start = scan - all + (warp > 0 ? warp_sum[warp - 1] : 0);
    if (tid < n_experts) {
        for (int w = 0; w < kSortWarps; ++w) hist[w * n_experts + tid] += start + before;
        if (rank == 0) offsets[tid] = start;
    }
    if (tid == n_experts - 1) {
        n_kept = start + all;
        if (rank == 0) offsets[n_experts] = start + all;
    }
    cluster.sync();   // the totals are read; positions and n_kept are written
    for (int p = lo; p < hi; p += 32) {
        const int id = p + lane < hi ? __ldg(ids + p + lane) : -1;
        const bool ok = id >= 0 && id < n_experts;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, ok ? id : -1);
        int32_t pos = -1;
        if (ok) pos = mine[id] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (ok && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
        if (p + lane < hi) {
            pos_of[p + lane] = pos;
            if (ok) token_at[pos] = (p + lane) / top_k;
        }
    }
    for (int i = n_kept + rank * kSortThreads + tid; i < n_pairs; i += n_cta * kSortThreads)
        token_at[i] = -1;
}

constexpr int kRThreads = 256;

// xs[i] = x[token_at[i]], one row a block, P its access unit.
template <typename P>
__global__ void __launch_bounds__(kRThreads)
    k_moe_dispatch(const P* __restrict__ x, int n_tokens, int per_row,
                   const int32_t* __restrict__ token_at, P* __restrict__ xs) {
    const size_t row = blockIdx.x;
    const int t = __ldg(token_at + row);
    const bool in = t >= 0 && t < n_tokens;
    for (int c = threadIdx.x; c < per_row; c += kRThreads)
        xs[row * per_row + c] = in ? x[static_cast<size_t>(t) * per_row + c] : P{};
}

// y[t] = sum_j w[t][j] o[pos_of[t][j]] (w == nullptr: 1), one token a block.
template <typename T, int N>
__global__ void __launch_bounds__(kRThreads)
    k_moe_gather_sum(const Pack<T, N>* __restrict__ o, int n_rows, int top_k, int per_row,
                     const int32_t* __restrict__ pos_of, const float* __restrict__ w,
                     Pack<T, N>* __restrict__ y) {
    const size_t t = blockIdx.x;
    for (int c = threadIdx.x; c < per_row; c += kRThreads) {
        float acc[N] = {};
        for (int j = 0; j < top_k; ++j) {
            const int pos = __ldg(pos_of + t * top_k + j);
            if (pos < 0 || pos >= n_rows) continue;
            const float wt = w != nullptr ? __ldg(w + t * top_k + j) : 1.0f;
            const Pack<T, N> a = o[static_cast<size_t>(pos) * per_row + c];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(wt, to_f32(a.v[i]), acc[i]);
        }
        Pack<T, N> r;
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(acc[i]);
        y[t * per_row + c] = r;
    }
}

// d_o[pos] = w dy[t], d_w = <dy[t], o[pos]>: one pair a block.
template <typename T, int N>
__global__ void __launch_bounds__(kRThreads)
    k_moe_combine_grad(const Pack<T, N>* __restrict__ dy, const Pack<T, N>* __restrict__ o,
                       int n_rows, int top_k, int per_row, const int32_t* __restrict__ pos_of,
                       const float* __restrict__ w, Pack<T, N>* __restrict__ d_o,
                       float* __restrict__ d_w) {
    __shared__ float part[kRThreads / 32];
    const size_t p = blockIdx.x, t = p / top_k;
    const int pos = __ldg(pos_of + p);
    if (pos < 0 || pos >= n_rows) {
        if (threadIdx.x == 0) d_w[p] = 0.0f;
        return;
    }
    const float wt = __ldg(w + p);
    float acc = 0.0f;
    for (int c = threadIdx.x; c < per_row; c += kRThreads) {
        const Pack<T, N> a = dy[t * per_row + c];
        const Pack<T, N> b = o[static_cast<size_t>(pos) * per_row + c];
        Pack<T, N> r;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float g = to_f32(a.v[i]);
            acc = fmaf(g, to_f32(b.v[i]), acc);
            r.v[i] = from_f32<T>(wt * g);
        }
        d_o[static_cast<size_t>(pos) * per_row + c] = r;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kRThreads / 32; ++i) acc += part[i];
        d_w[p] = acc;
    }
}

// Calls f(T{}, vector width): 16-byte accesses when the rows keep the base
// pointers' alignment, else one element at a time.
template <class F>
cudaError_t by_type(int type, int width, F&& f) {
    const bool vec = static_cast<long long>(width) * type_bytes(type) % 16 == 0;
    if (type == kTypeF32)
        return vec ? f(Pack<float, 4>{}) : f(Pack<float, 1>{});
    if (type == kTypeBF16)
        return vec ? f(Pack<__nv_bfloat16, 8>{}) : f(Pack<__nv_bfloat16, 1>{});
    return vec ? f(Pack<__half, 8>{}) : f(Pack<__half, 1>{});
}

}  // namespace

cudaError_t launch_moe_sort(const int32_t* ids, int n_pairs, int top_k, int n_experts,
                            int32_t* token_at, int32_t* pos_of, int32_t* offsets,
                            cudaStream_t s) {
    const size_t smem = static_cast<size_t>(kSortWarps + 1) * n_experts * sizeof(int32_t);
    static PerDevice memo;
    const cudaError_t attr_err = static_cast<cudaError_t>(memo.get([] {
        return static_cast<int>(cudaFuncSetAttribute(
            k_moe_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
            static_cast<int>((kSortWarps + 1) * kSortThreads * sizeof(int32_t))));
    }));
    if (attr_err != cudaSuccess) return attr_err;
    const int n_cta = n_pairs <= kSortThreads ? 1 : kSortCluster;
    const int run = (n_pairs + n_cta * kSortThreads - 1) / (n_cta * kSortThreads) * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_cta));
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(n_cta);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_moe_sort, ids, n_pairs, top_k, n_experts, run,
                                             token_at, pos_of, offsets);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_moe_dispatch(const void* x, int type, int n_tokens, int n_rows, int width,
                                const int32_t* token_at, void* xs, cudaStream_t s) {
    const long long bytes = static_cast<long long>(width) * type_bytes(type);
    auto go = [&](auto unit) {
        using P = decltype(unit);
        k_moe_dispatch<P><<<static_cast<unsigned>(n_rows), kRThreads, 0, s>>>(
            static_cast<const P*>(x), n_tokens, static_cast<int>(bytes / sizeof(P)), token_at,
            static_cast<P*>(xs));
        return cudaGetLastError();
    };
    if (bytes % 16 == 0) return go(uint4{});
    if (bytes % 4 == 0) return go(uint32_t{});
    return go(uint16_t{});
}

cudaError_t launch_moe_gather_sum(const void* o, int type, int n_tokens, int top_k, int width,
                                  const int32_t* pos_of, const float* route_w, void* y,
                                  cudaStream_t s) {
    return by_type(type, width, [&](auto unit) {
        using P = decltype(unit);
        constexpr int kN = sizeof(unit.v) / sizeof(unit.v[0]);
        using T = std::remove_reference_t<decltype(unit.v[0])>;
        k_moe_gather_sum<T, kN><<<static_cast<unsigned>(n_tokens), kRThreads, 0, s>>>(
            static_cast<const P*>(o), n_tokens * top_k, top_k, width / kN, pos_of, route_w,
            static_cast<P*>(y));
        return cudaGetLastError();
    });
}

cudaError_t launch_moe_combine_grad(const void* dy, const void* o, int type, int n_tokens,
                                    int top_k, int width, const int32_t* pos_of,
                                    const float* route_w, void* d_o, float* d_route_w,
                                    cudaStream_t s) {
    return by_type(type, width, [&](auto unit) {
        using P = decltype(unit);
        constexpr int kN = sizeof(unit.v) / sizeof(unit.v[0]);
        using T = std::remove_reference_t<decltype(unit.v[0])>;
        k_moe_combine_grad<T, kN><<<static_cast<unsigned>(n_tokens * top_k), kRThreads, 0, s>>>(
            static_cast<const P*>(dy), static_cast<const P*>(o), n_tokens * top_k, top_k,
            width / kN, pos_of, route_w, static_cast<P*>(d_o), d_route_w);
        return cudaGetLastError();
    });
}

}  // namespace mxk
