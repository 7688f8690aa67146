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
// The other kernels move rows.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mx4_kernels.h"
#include "pdl.cuh"

namespace mxk {
namespace {

namespace cg = cooperative_groups;

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;   // at most
constexpr int kMaxExperts = 1024;
constexpr int kSortCluster = 8;

__global__ void __launch_bounds__(kSortThreads)
    k_moe_sort(const int32_t* ids, int n_pairs, int top_k, int n_experts, int run,
               int32_t* __restrict__ token_at, int32_t* __restrict__ pos_of,
               int32_t* __restrict__ offsets) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ int32_t sort_smem[];
    const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
    int32_t* total = sort_smem;              // [n_experts], read by the cluster
    int32_t* base = total + n_experts;       // [n_experts]
    int32_t* hist = base + n_experts;        // [warps][n_experts]
    __shared__ int32_t warp_sum[kSortWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int n_cta = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* mine = hist + warp * n_experts;

    const long long p0 = (static_cast<long long>(rank) * warps + warp) * run;
    const int lo = static_cast<int>(min(p0, static_cast<long long>(n_pairs)));
    const int hi = static_cast<int>(min(p0 + run, static_cast<long long>(n_pairs)));
    // the ids of the run's first 32 pairs (all of it, often) stay in a register
    const int id0 = lo + lane < hi ? ld_dep(ids + lo + lane) : -1;
    auto id_of = [&](int p) {
        const int id = p == lo ? id0 : p + lane < hi ? ld_dep(ids + p + lane) : -1;
        return id >= 0 && id < n_experts ? id : -1;
    };
    for (int e = lane; e < n_experts; e += 32) mine[e] = 0;
    __syncwarp();
    for (int p = lo; p < hi; p += 32) {
        const int id = id_of(p);
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // per expert: exclusive sums over the warps, and the CTA's total
    for (int e = tid; e < n_experts; e += threads) {
        int32_t c[kSortWarps], sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = w < warps ? hist[w * n_experts + e] : 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warps) hist[w * n_experts + e] = sum;
            sum += c[w];
        }
        total[e] = sum;
    }
    if (n_cta > 1) cluster.sync();
    else __syncthreads();
    // all CTAs' totals and the exclusive sum over the experts, a block of experts at a time
    int32_t kept = 0;
    for (int e0 = 0; e0 < n_experts; e0 += threads) {
        const int e = e0 + tid;
        int32_t all = 0, before = 0;
        if (e < n_experts) {
            if (n_cta == 1) {
                all = total[e];
            } else {
                int32_t t[kSortCluster];
#pragma unroll
                for (int c = 0; c < kSortCluster; ++c) t[c] = cluster.map_shared_rank(total, c)[e];
#pragma unroll
                for (int c = 0; c < kSortCluster; ++c) {
                    if (c < rank) before += t[c];
                    all += t[c];
                }
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
        int32_t s = lane < warps ? warp_sum[lane] : 0;   // (every warp for itself)
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= d) s += o;
        }
        const int32_t ahead = __shfl_sync(0xFFFFFFFFu, s, max(warp - 1, 0));
        const int32_t start = kept + scan - all + (warp > 0 ? ahead : 0);
        if (e < n_experts) {
            base[e] = start + before;
            if (rank == 0) offsets[e] = start;
        }
        kept += __shfl_sync(0xFFFFFFFFu, s, 31);
        __syncthreads();
    }
    if (rank == 0 && tid == 0) offsets[n_experts] = kept;
    for (int p = lo; p < hi; p += 32) {
        const int id = id_of(p);
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        int32_t pos = -1;
        if (id >= 0) pos = base[id] + mine[id] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
        if (p + lane < hi) {
            pos_of[p + lane] = pos;
            if (id >= 0) token_at[pos] = (p + lane) / top_k;
        }
    }
    for (int i = kept + rank * threads + tid; i < n_pairs; i += n_cta * threads) token_at[i] = -1;
    if (n_cta > 1) cluster.sync();   // no CTA leaves while its totals may be read
}

// --- moving rows ------------------------------------------------------------------------
//
// Bound by HBM, and for few rows by latency.  A row is cut into the widest units that keep
// every row aligned (32 bytes down to one element); a thread takes one unit of the flat
// [rows][units] space, or in dispatch four of fewer than 32 bytes, loaded ahead (one of 16 bytes
// a thread takes 28 us instead of 20 for 4096 tokens, top-4, 2888 wide, one of 4 bytes 13.6
// instead of 4.5 for 1111 tokens, top-3, 1001 floats; four of 32 bytes 6.9 instead of 5.5 for
// 1024 tokens, top-4, 2880 wide, and 2 % less for 4096).
// 4096 tokens of 2880 in bfloat16: dispatch 20.6 us, 5.7 TB/s; combine and the gradient of
// dispatch 20.4 us each, 5.8 TB/s (16-byte units: 23.9); the gradient of combine 34.3 us, 6.2
// TB/s.

constexpr int kRThreads = 256;

template <typename P>
constexpr int kUnits = sizeof(P) < 32 ? 4 : 1;

// xs[i] = x[token_at[i]].
template <typename P>
__global__ void __launch_bounds__(kRThreads)
    k_moe_dispatch(const P* x, int n_tokens, uint32_t row0, uint32_t units,
                   FastDiv per_row, const int32_t* token_at, P* __restrict__ xs) {
    pdl_trigger();
    pdl_wait();
    constexpr int kU = kUnits<P>;
    P v[kU];
    const uint32_t i0 = blockIdx.x * (kRThreads * kU) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint32_t i = i0 + u * kRThreads;
        const uint32_t row = per_row.of(i);
        const int t = i < units ? ld_dep(token_at + row0 + row) : -1;
        v[u].raw = {};
        if (t >= 0 && t < n_tokens)
            v[u] = load_pack(x + static_cast<size_t>(t) * per_row.d + (i - row * per_row.d));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint32_t i = i0 + u * kRThreads;
        if (i < units) store_pack(xs + static_cast<size_t>(row0) * per_row.d + i, v[u]);
    }
}

// y[t] = sum_j w[t][j] o[pos_of[t][j]] (w == nullptr: 1): one unit a thread, four pairs'
// rows in flight.
template <typename T, int N>
__global__ void __launch_bounds__(kRThreads)
    k_moe_gather_sum(const Pack<T, N>* o, int n_rows, int top_k, uint32_t row0,
                     uint32_t units, FastDiv per_row, const int32_t* pos_of,
                     const float* w, Pack<T, N>* __restrict__ y) {
    pdl_trigger();
    pdl_wait();
    const uint32_t i = blockIdx.x * kRThreads + threadIdx.x;
    if (i >= units) return;
    const uint32_t row = per_row.of(i), c = i - row * per_row.d;
    const size_t p0 = (static_cast<size_t>(row0) + row) * top_k;
    float acc[N] = {};
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        int pos[4];
        float wt[4];
        Pack<T, N> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = j0 + j < top_k;
            pos[j] = in ? ld_dep(pos_of + p0 + j0 + j) : -1;
            wt[j] = in && w != nullptr ? ld_dep(w + p0 + j0 + j) : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = pos[j] >= 0 && pos[j] < n_rows;
            if (!in) wt[j] = 0.0f;
            v[j].raw = {};
            if (in) v[j] = load_pack(o + static_cast<size_t>(pos[j]) * per_row.d + c);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[N];
            v[j].get(f);
#pragma unroll
            for (int q = 0; q < N; ++q) acc[q] = fmaf(wt[j], f[q], acc[q]);
        }
    }
    Pack<T, N> r;
    r.set(acc);
    store_pack(y + static_cast<size_t>(row0) * per_row.d + i, r);
}

// d_o[pos] = w dy[t], d_w = <dy[t], o[pos]>: one token a block, four pairs at a time, each
// unit of dy read once for the four.
template <typename T, int N>
__global__ void
    k_moe_combine_grad(const Pack<T, N>* dy, const Pack<T, N>* o,
                       int n_rows, int top_k, int per_row, const int32_t* pos_of,
                       const float* w, Pack<T, N>* __restrict__ d_o,
                       float* __restrict__ d_w) {
    pdl_trigger();
    pdl_wait();
    __shared__ float part[4][32];
    const size_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_warps = static_cast<int>(blockDim.x) >> 5;
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        const size_t p = t * top_k + j0;
        int pos[4];
        float wt[4], acc[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            pos[j] = j0 + j < top_k ? ld_dep(pos_of + p + j) : -1;
            if (pos[j] >= n_rows) pos[j] = -1;
            wt[j] = pos[j] >= 0 ? ld_dep(w + p + j) : 0.0f;
        }
        for (int c = threadIdx.x; c < per_row; c += blockDim.x) {
            const Pack<T, N> a = load_pack(dy + t * per_row + c);
            Pack<T, N> b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                b[j].raw = {};
                if (pos[j] >= 0) b[j] = load_pack(o + static_cast<size_t>(pos[j]) * per_row + c);
            }
            float g[N];
            a.get(g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[N];
                b[j].get(f);
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    acc[j] = pos[j] >= 0 ? fmaf(g[q], f[q], acc[j]) : 0.0f;
                    f[q] = wt[j] * g[q];
                }
                Pack<T, N> r;
                r.set(f);
                if (pos[j] >= 0) store_pack(d_o + static_cast<size_t>(pos[j]) * per_row + c, r);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], m);
            if (lane == 0) part[j][warp] = acc[j];
        }
        __syncthreads();
        if (warp < 4) {   // warp j adds pair j's sums (at least four warps a block)
            float s = lane < n_warps ? part[warp][lane] : 0.0f;
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
            if (lane == 0 && j0 + warp < top_k) d_w[p + warp] = s;
        }
        __syncthreads();
    }
}

// Calls f(Pack<T, N>{}) with the widest unit that keeps every row of `width` elements
// aligned: 32 (where `base`, the buffers' addresses together, allows it), 16, 8 or 4 bytes,
// or one element; no more than kMost elements of 16-bit types.
template <int kMost, class F>
cudaError_t by_type(int type, int width, uintptr_t base, F&& f) {
    const bool wide =
        (base | static_cast<uintptr_t>(width) * static_cast<uintptr_t>(type_bytes(type))) % 32 == 0;
    if (type == kTypeF32) {
        if (wide) return f(Pack<float, 8>{});
        if (width % 4 == 0) return f(Pack<float, 4>{});
        if (width % 2 == 0) return f(Pack<float, 2>{});
        return f(Pack<float, 1>{});
    }
    auto half_width = [&](auto zero) {
        using T = decltype(zero);
        if constexpr (kMost >= 16) {
            if (wide) return f(Pack<T, 16>{});
        }
        if (width % 8 == 0) return f(Pack<T, 8>{});
        if (width % 4 == 0) return f(Pack<T, 4>{});
        if (width % 2 == 0) return f(Pack<T, 2>{});
        return f(Pack<T, 1>{});
    };
    return type == kTypeBF16 ? half_width(__nv_bfloat16{}) : half_width(__half{});
}

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

unsigned blocks_of(uint32_t units, int per_thread) {
    const uint32_t per_block = static_cast<uint32_t>(kRThreads * per_thread);
    return (units + per_block - 1) / per_block;
}

}  // namespace

cudaError_t launch_moe_sort(const int32_t* ids, int n_pairs, int top_k, int n_experts,
                            int32_t* token_at, int32_t* pos_of, int32_t* offsets,
                            cudaStream_t s) {
    static PerDevice memo;
    const cudaError_t attr_err = static_cast<cudaError_t>(memo.get([] {
        return static_cast<int>(cudaFuncSetAttribute(
            k_moe_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
            static_cast<int>((kSortWarps + 2) * kMaxExperts * sizeof(int32_t))));
    }));
    if (attr_err != cudaSuccess) return attr_err;
    // one CTA for as many pairs as its warps take in two steps of 32, else a cluster of 8
    const int n_cta = n_pairs <= 2 * kSortThreads ? 1 : kSortCluster;
    const int warps = std::min(kSortWarps, std::max(4, (n_pairs + 32 * n_cta - 1) / (32 * n_cta)));
    const int run = (n_pairs + n_cta * warps * 32 - 1) / (n_cta * warps * 32) * 32;
    const size_t smem = static_cast<size_t>(warps + 2) * n_experts * sizeof(int32_t);
    return launch_after(k_moe_sort, dim3(static_cast<unsigned>(n_cta)),
                        static_cast<unsigned>(warps * 32), smem, s,
                        static_cast<unsigned>(n_cta), ids, n_pairs, top_k, n_experts, run,
                        token_at, pos_of, offsets);
}

cudaError_t launch_moe_dispatch(const void* x, int type, int n_tokens, int n_rows, int width,
                                const int32_t* token_at, void* xs, cudaStream_t s) {
    return by_type<16>(type, width, bits(x) | bits(xs), [&](auto unit) {
        using P = decltype(unit);
        const int per_row = width / P::kN;
        const FastDiv div(static_cast<uint32_t>(per_row));
        return over_rows(n_rows, per_row, [&](uint32_t row0, uint32_t units) {
            return launch_after(k_moe_dispatch<P>, dim3(blocks_of(units, kUnits<P>)), kRThreads, 0,
                                s, 1, static_cast<const P*>(x), n_tokens, row0, units, div,
                                token_at, static_cast<P*>(xs));
        });
    });
}

cudaError_t launch_moe_gather_sum(const void* o, int type, int n_tokens, int top_k, int width,
                                  const int32_t* pos_of, const float* route_w, void* y,
                                  cudaStream_t s) {
    return by_type<16>(type, width, bits(o) | bits(y), [&](auto unit) {
        using P = decltype(unit);
        using T = typename P::Elem;
        const FastDiv div(static_cast<uint32_t>(width / P::kN));
        return over_rows(n_tokens, width / P::kN, [&](uint32_t row0, uint32_t units) {
            return launch_after(k_moe_gather_sum<T, P::kN>, dim3(blocks_of(units, 1)), kRThreads,
                                0, s, 1, static_cast<const P*>(o), n_tokens * top_k, top_k, row0,
                                units, div, pos_of, route_w, static_cast<P*>(y));
        });
    });
}

cudaError_t launch_moe_combine_grad(const void* dy, const void* o, int type, int n_tokens,
                                    int top_k, int width, const int32_t* pos_of,
                                    const float* route_w, void* d_o, float* d_route_w,
                                    cudaStream_t s) {
    // (eight elements a unit at most: a thread holds six units, and 32 bytes of 16-bit elements
    // leave too few threads an SM)
    return by_type<8>(type, width, bits(dy) | bits(o) | bits(d_o), [&](auto unit) {
        using P = decltype(unit);
        constexpr int kN = P::kN;
        using T = typename P::Elem;
        const int per_row = width / kN;
        // Many tokens: small blocks, so that some load while others store and reduce ([4096 x 4,
        // 2880] bfloat16 34.3 us against 38.6; of small units twice as many threads, [1111 x 3,
        // 1001] floats 7.2 against 8.3); few: a whole row in flight at once (256 tokens 3.5 us
        // against 4.0).
        const int most = n_tokens < 152 * 4 ? 512 : sizeof(P) < 16 ? 256 : 128;
        const int threads = std::min(most, std::max(128, (per_row + 31) / 32 * 32));
        return launch_after(k_moe_combine_grad<T, kN>, dim3(static_cast<unsigned>(n_tokens)),
                            static_cast<unsigned>(threads), 0, s, 1, static_cast<const P*>(dy),
                            static_cast<const P*>(o), n_tokens * top_k, top_k, per_row, pos_of,
                            route_w, static_cast<P*>(d_o), d_route_w);
    });
}

}  // namespace mxk
