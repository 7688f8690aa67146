// f8_mm.cu -- products of E4M3 codes with a scale for each block of 128, and their gradient by the
// rows (include/f8.h mxfp4_f8_mm, mxfp4_f8_moe_mm, mxfp4_f8_mm_grad, mxfp4_f8_moe_mm_grad;
// tcgen05 kind::f8f6f4, sm_103a).
//
// Y[i][o] = sum_b sx[b][i] sw[o/128][b] sum_{k in b} W[o][k] X[i][k], b the blocks of 128 of the
// sum.  The tensor core adds a block's 128 products in FP32; tensor memory then hands the block
// over, and other warps add it, times the product of the two scales, to sums that they hold
// in registers.  The gradient is the same sum with W read along its other side: its
// scale blocks are square, so the codes serve both, and only the operand's descriptor (which
// side is contiguous) and the strides of the scales change.
//
// The matrix's outputs are the MMA's 128 rows and the tokens its columns: one scale of W for
// a whole tile and block, one of X for a column.
//
// Warps have roles: copies (TMA, 128-byte swizzled rows: a ring stage is one block of 128 of
// both operands), MMAs, scales (by asynchronous copies of 4 bytes, 16 blocks ahead), and the sums
// (eight warps: each quarter of the lanes twice, each half of the columns).  Persistent: CTA c
// takes tiles c, c + grid, ...  With few tiles a cluster of CTAs shares one, each a slice
// of the blocks, and adds the partial sums through distributed shared memory in rank order.
//
// Every wait is bounded; a CTA that gives up sets the fault word, lets its copies land, frees its
// tensor memory and returns.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "f8_kernels.h"
#include "kernels.h"
#include "pdl.cuh"
#include "tc5.cuh"

namespace mxk {
namespace {

namespace cg = cooperative_groups;

constexpr int kM = 128;                      // outputs per tile
constexpr uint32_t kABytes = kM * kF8Block;  // W's part of a stage
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;                 // CTAs of a cluster sharing a tile
constexpr int kTileTable = 64;               // this CTA's first tiles, worked out at the start
constexpr int kFac = 16;                     // blocks whose scales are held ahead
constexpr int kThreads = 384, kEpiWarp = 4, kEpiWarps = 8;
constexpr long long kWait = 1ll << 32, kDrain = 1ll << 24;   // SM cycles: about 2 s and 8 ms

__device__ int g_fault_f8;

struct F8Args {
    const float* w_scales;
    const float* x_scales;
    const int32_t* offsets;     // nullptr: one matrix
    int n_experts, n_out, n_rows;
    int n_k;                    // blocks of the sum
    long long sw_expert;        // strides of W's scales: matrix, block of outputs, block of the sum
    int sw_out, sw_k;
    int tn, box, n_stages;      // most tokens of a tile (a multiple of 16), rows of a copy
    uint32_t stage_bytes;
    int n_rt, n_tt;             // output tiles; token tiles (one matrix)
};

struct alignas(16) Tile {
    int e, r0, t0, t1;
};

// Instruction descriptor: D = F32, A = B = E4M3; W (A) by its contiguous side.
template <bool kGrad>
__device__ __forceinline__ uint32_t idesc_f8(int n) {
    return (1u << 4) | (kGrad ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kM >> 4) << 24);
}

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 4 bytes, global to shared, completing on a later async_arrive.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival once its copies so far have landed.
__device__ __forceinline__ void async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// NC: most tokens of a tile.  kAcc accumulators of NC columns.
template <int NC, bool kSplit>
struct Shape {
    static constexpr int kAcc = NC == 16 ? 8 : kSplit && NC == 128 ? 2 : 4;
    static constexpr uint32_t kTmem = kAcc * NC;
    static constexpr int kHalf = NC / 2;      // columns a warp
    static constexpr int kFacRow = NC + 4;    // floats of a block's scales: X's, then W's
};

template <typename T, int NC, bool kSplit, bool kGrad>
__global__ void __launch_bounds__(kThreads, 1)
    k_f8_mm(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
            const F8Args a, T* __restrict__ Y) {
    using S = Shape<NC, kSplit>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[S::kAcc], acc_empty[S::kAcc];
    __shared__ uint64_t fac_full[kFac], fac_empty[kFac], drain;
    __shared__ __align__(16) float fac[kFac][S::kFacRow];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word, n_tiles_sh;
    __shared__ Tile table[kTileTable];
    volatile int* abort_flag = &abort_word;
    // after the ring: the experts' row offsets and first tiles.  The partial sums of a split
    // tile lie over the ring, which is read out by then.
    uint8_t* after = smem + static_cast<size_t>(a.n_stages) * a.stage_bytes;
    int32_t* off = reinterpret_cast<int32_t*>(after);
    int32_t* first = off + a.n_experts + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kSplit ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int n_rank = kSplit ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;

    if (warp == 1) tmem_take(&tmem_base, S::kTmem);
    if (tid == 0) {
        for (int i = 0; i < a.n_stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < S::kAcc; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kEpiWarps);
        }
        for (int i = 0; i < kFac; ++i) {
            mbar_init(&fac_full[i], 32);
            mbar_init(&fac_empty[i], kEpiWarps);
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        n_tiles_sh = a.n_rt * a.n_tt;
        fence_mbar_init();
    }
    if (tid == 32 * 2) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&wmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the next launch may be placed now that this CTA has its tensor memory
    pdl_trigger();
    if (a.offsets != nullptr) {
        pdl_wait();
        for (int e = tid; e <= a.n_experts; e += kThreads)
            off[e] = min(max(ld_dep(a.offsets + e), 0), a.n_rows);
        __syncthreads();
        if (warp == 0) {   // first[e]: tiles of the experts before e
            int base = 0;
            for (int e0 = 0; e0 < a.n_experts; e0 += 32) {
                const int e = e0 + lane;
                int n = 0;
                if (e < a.n_experts)
                    n = a.n_rt * ((max(off[e + 1] - off[e], 0) + a.tn - 1) / a.tn);
                int sum = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                    if (lane >= d) sum += o;
                }
                if (e < a.n_experts) first[e] = base + sum - n;
                base += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            if (lane == 0) {
                first[a.n_experts] = base;
                n_tiles_sh = base;
            }
        }
    }
    __syncthreads();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    const int n_tiles = __shfl_sync(0xFFFFFFFFu, n_tiles_sh, 0);
    const int s_lo = kSplit ? static_cast<int>(static_cast<long long>(a.n_k) * rank / n_rank) : 0;
    const int s_hi =
        kSplit ? static_cast<int>(static_cast<long long>(a.n_k) * (rank + 1) / n_rank) : a.n_k;
    // a cluster's tiles (split: one)
    const int tile0 = static_cast<int>(blockIdx.x) / n_rank;
    const int tile_step = kSplit ? n_tiles : static_cast<int>(gridDim.x);

    // An output tile's token tiles come one after the other, so that its part of the matrix is
    // read again from L2; an expert's rows are cut into equal tiles of a multiple of 16.
    auto locate = [&](int tile) {
        Tile t;
        if (a.offsets == nullptr) {
            t.e = 0;
            const int rt = tile / a.n_tt;
            t.r0 = rt * kM;
            t.t0 = (tile - rt * a.n_tt) * a.tn;
            t.t1 = min(t.t0 + a.tn, a.n_rows);
        } else {
            int lo = 0, hi = a.n_experts;   // first[lo] <= tile < first[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= tile) lo = mid;
                else hi = mid;
            }
            t.e = lo;
            const int n = off[lo + 1] - off[lo];
            const int n_tt = (n + a.tn - 1) / a.tn;
            const int per = ((n + n_tt - 1) / n_tt + 15) & ~15;
            const int local = tile - first[lo], rt = local / n_tt;
            t.r0 = rt * kM;
            t.t0 = off[lo] + (local - rt * n_tt) * per;
            t.t1 = min(t.t0 + per, off[lo + 1]);
        }
        return t;
    };
    if (tid < kTileTable && tile0 + tid * tile_step < n_tiles)
        table[tid] = locate(tile0 + tid * tile_step);
    __syncthreads();
    if (a.offsets == nullptr) pdl_wait();   // nothing in memory was needed so far
    auto tile_at = [&](int tile, int j) { return j < kTileTable ? table[j] : locate(tile); };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_fault_f8, 1);
    };

    if (warp == 0) {
        // --- copies (the whole warp walks, one elected lane issues)
        const bool leader = elect_one();
        const uint64_t keep = l2_evict_last();
        const uint64_t w_policy = a.offsets != nullptr && a.tn <= 32 ? l2_evict_first()
                                                                      : l2_evict_normal();
        const uint32_t ring = smem_u32(smem);
        const uint32_t box_bytes = static_cast<uint32_t>(a.box) * kF8Block;
        uint32_t st = 0, phase = 1;   // the first round of the ring passes at once
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int n_box = (t.t1 - t.t0 + a.box - 1) / a.box;
            const uint32_t bytes = kABytes + static_cast<uint32_t>(n_box) * box_bytes;
            for (int s = s_lo; s < s_hi; ++s) {
                ok = mbar_wait_for(&empty[st], phase, kWait);
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&full[st], bytes);
                    const uint32_t dst = ring + st * a.stage_bytes;
                    if constexpr (kGrad)
                        tma3d(dst, &wmap, t.r0, s * kF8Block, t.e, &full[st], w_policy);
                    else
                        tma3d(dst, &wmap, s * kF8Block, t.r0, t.e, &full[st], w_policy);
                    for (int b = 0; b < n_box; ++b)
                        tma2d(dst + kABytes + static_cast<uint32_t>(b) * box_bytes, &xmap,
                              s * kF8Block, t.t0 + b * a.box, &full[st], keep);
                }
                __syncwarp();
                if (++st == static_cast<uint32_t>(a.n_stages)) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
        __syncwarp();
    } else if (warp == 1) {
        // --- MMAs: a block's four of K = 32 into the next accumulator
        const bool leader = elect_one();
        const uint32_t ring = smem_u32(smem);
        const uint64_t a0 = kGrad ? operand_desc_mn(ring, kABytes) : operand_desc(ring);
        const uint64_t b0 = operand_desc(ring + kABytes);
        // K = 32: 32 bytes of a row, or 32 rows of 128 bytes
        constexpr uint32_t kAStep = kGrad ? 32 * kF8Block / 16 : 2;
        uint32_t st = 0, phase = 0, ab = 0, acc_phase = 1;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const uint32_t id =
                idesc_f8<kGrad>(__shfl_sync(0xFFFFFFFFu, (t.t1 - t.t0 + 15) & ~15, 0));
            for (int s = s_lo; s < s_hi; ++s) {
                ok = mbar_wait_for(&acc_empty[ab], acc_phase, kWait) &&
                     mbar_wait_for(&full[st], phase, kWait);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t at = st * (a.stage_bytes >> 4);
                    const uint32_t d = tmem + ab * NC;
#pragma unroll
                    for (uint32_t q = 0; q < 4; ++q)
                        umma_f8(d, a0 + at + q * kAStep, b0 + at + q * 2, id, q);
                    umma_commit(&empty[st]);
                    umma_commit(&acc_full[ab]);
                }
                __syncwarp();
                if (++st == static_cast<uint32_t>(a.n_stages)) {
                    st = 0;
                    phase ^= 1u;
                }
                if (++ab == S::kAcc) {
                    ab = 0;
                    acc_phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) {
            fail();
            if (leader) umma_commit(&drain);
            mbar_wait_for(&drain, 0u, kWait);
        }
        __syncwarp();
    } else if (warp == 2) {
        // --- scales
        const uint32_t slots = smem_u32(&fac[0][0]);
        uint32_t f = 0, phase = 1;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const float* w = a.w_scales + t.e * a.sw_expert +
                             static_cast<long long>(t.r0 / kM) * a.sw_out;
            const int n = t.t1 - t.t0;
            for (int s = s_lo; s < s_hi; ++s) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_for(&fac_empty[f], phase, kWait));
                if (!ok) break;
                const uint32_t dst = slots + f * (S::kFacRow * 4);
                const float* x = a.x_scales + static_cast<size_t>(s) * a.n_rows + t.t0;
                for (int i = lane; i < n; i += 32) copy4(dst + i * 4, x + i);
                if (lane == 0)
                    copy4(dst + NC * 4, w + static_cast<long long>(s) * a.sw_k);
                async_arrive(&fac_full[f]);
                if (++f == kFac) {
                    f = 0;
                    phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp >= kEpiWarp) {
        // --- sums: lane = output, columns half * kHalf on = tokens
        const int quarter = warp & 3, half = (warp - kEpiWarp) >> 2;
        constexpr int kChunk = S::kHalf < 32 ? S::kHalf : 32;
        uint32_t ab = 0, acc_phase = 0, f = 0, fac_phase = 0;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int n = t.t1 - t.t0 - half * S::kHalf;   // of this half (may be none)
            float2 sum[S::kHalf / 2];
#pragma unroll
            for (int i = 0; i < S::kHalf / 2; ++i) sum[i] = make_float2(0.0f, 0.0f);
            for (int s = s_lo; s < s_hi; ++s) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_for(&fac_full[f], fac_phase, kWait) &&
                                                 mbar_wait_for(&acc_full[ab], acc_phase, kWait));
                if (!ok) break;
                tc_fence_after();
                const float w = fac[f][NC];
#pragma unroll
                for (int c = 0; c < S::kHalf; c += kChunk) {
                    if (c >= n) break;
                    uint32_t v[kChunk];
                    tmem_ld<kChunk>(tmem + ab * NC + half * S::kHalf + c +
                                        (static_cast<uint32_t>(quarter * 32) << 16),
                                    v);
                    tmem_ld_wait();
                    const float4* x = reinterpret_cast<const float4*>(&fac[f][half * S::kHalf + c]);
#pragma unroll
                    for (int i = 0; i < kChunk / 4; ++i) {
                        const float4 p = x[i];
                        float2& s0 = sum[c / 2 + 2 * i];
                        float2& s1 = sum[c / 2 + 2 * i + 1];
                        s0 = __ffma2_rn(make_float2(__uint_as_float(v[4 * i]),
                                                    __uint_as_float(v[4 * i + 1])),
                                        __fmul2_rn(make_float2(p.x, p.y), make_float2(w, w)), s0);
                        s1 = __ffma2_rn(make_float2(__uint_as_float(v[4 * i + 2]),
                                                    __uint_as_float(v[4 * i + 3])),
                                        __fmul2_rn(make_float2(p.z, p.w), make_float2(w, w)), s1);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_m(&acc_empty[ab]);
                    mbar_arrive_m(&fac_empty[f]);
                }
                if (++ab == S::kAcc) {
                    ab = 0;
                    acc_phase ^= 1u;
                }
                if (++f == kFac) {
                    f = 0;
                    fac_phase ^= 1u;
                }
            }
            if (!ok) {
                fail();
                break;
            }
            const int r = t.r0 + quarter * 32 + lane;
            if constexpr (kSplit) {
                // [token][128 outputs] partial sums of this rank, over the ring: every copy and
                // MMA of this CTA is done once its last block was handed over
                float* part = reinterpret_cast<float*>(smem) + half * S::kHalf * kM +
                              quarter * 32 + lane;
#pragma unroll
                for (int i = 0; i < S::kHalf; ++i)
                    if (i < n) part[i * kM] = i % 2 ? sum[i / 2].y : sum[i / 2].x;
            } else if (r < a.n_out) {
                T* dst = Y + static_cast<size_t>(t.t0 + half * S::kHalf) * a.n_out + r;
#pragma unroll
                for (int i = 0; i < S::kHalf; ++i)
                    if (i < n)
                        dst[static_cast<size_t>(i) * a.n_out] =
                            from_f32<T>(i % 2 ? sum[i / 2].y : sum[i / 2].x);
            }
            ok = ok && !*abort_flag;
        }
    }

    __syncthreads();
    if constexpr (kSplit) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();   // every rank's partial sums are written
        const Tile t = tile_at(tile0, 0);
        float* part = reinterpret_cast<float*>(smem);
        const int n_out = (t.t1 - t.t0) * kM;
        for (int i = rank * kThreads + tid; i < n_out && !*abort_flag; i += n_rank * kThreads) {
            const int r = t.r0 + (i & (kM - 1)), tok = t.t0 + i / kM;
            float v[kMaxSplit], sum = 0.0f;   // all loads on their way before the first sum
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                v[q] = cluster.map_shared_rank(part, q < n_rank ? q : rank)[i];
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                if (q < n_rank) sum += v[q];
            if (r < a.n_out) Y[static_cast<size_t>(tok) * a.n_out + r] = from_f32<T>(sum);
        }
        cluster.sync();   // no rank leaves while its sums are being read
    }
    __syncthreads();
    if (*abort_flag && tid == 0) {
        // a CTA that gave up: its copies in flight land long before this
        for (const long long t0 = clock64(); clock64() - t0 < kDrain;) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_give(tmem, S::kTmem);
    }
}

// --- host side --------------------------------------------------------------------------

// `n` matrices of codes [rows][cols], copies of 128 columns x box_rows.
bool code_map(CUtensorMap* map, const void* base, int cols, int rows, int n, int box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols),
                                   static_cast<cuuint64_t>(cols) * rows};
    const cuuint32_t box[3] = {kF8Block, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, n > 0 ? 3 : 2, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmemMax = 227 * 1024, kSmemSlack = 12 * 1024;   // (the static arrays)

template <typename T, int NC, bool kSplit, bool kGrad>
cudaError_t launch_k(const F8Product& p, F8Args a, int split, int per_sm, unsigned grid,
                     cudaStream_t s) {
    a.stage_bytes = kABytes + static_cast<uint32_t>(a.tn) * kF8Block;
    const size_t extra =
        p.offsets != nullptr ? static_cast<size_t>(p.n_experts + 1) * 8 : 0;
    const size_t budget = kSmemMax / per_sm - kSmemSlack - 1024 - extra;
    a.n_stages = std::min(kMaxStages, static_cast<int>(budget / a.stage_bytes));
    if (kSplit) {
        // no more stages than a slice has, but room for the partial sums
        const int most = (a.n_k + split - 1) / split;
        const int sums = (a.tn * kM * 4 + static_cast<int>(a.stage_bytes) - 1) /
                         static_cast<int>(a.stage_bytes);
        a.n_stages = std::min(a.n_stages, std::max(std::max(most, sums), 2));
    }
    const size_t ring = static_cast<size_t>(a.n_stages) * a.stage_bytes + extra + 1024;
    // CTAs that share an SM never ask for more than its 512 columns of tensor memory together (2.25
    // a KB): one that waits for columns must not hold up its cluster
    const size_t smem = kSplit ? std::max(ring, static_cast<size_t>(Shape<NC, kSplit>::kTmem) *
                                                    1024 * 4 / 9)
                               : kSmemMax - kSmemSlack;
    auto kernel = k_f8_mm<T, NC, kSplit, kGrad>;
    static PerDevice memo;
    const cudaError_t attr_err = static_cast<cudaError_t>(memo.get([&] {
        return static_cast<int>(cudaFuncSetAttribute(kernel,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(kSmemMax - kSmemSlack)));
    }));
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap wmap, xmap;
    const int k = p.grad ? p.rows : p.cols;
    if (!code_map(&wmap, p.bank, p.cols, p.rows, p.n_experts, kM) ||
        !code_map(&xmap, p.x, k, p.n_rows, 0, a.box))
        return cudaErrorNotSupported;
    return launch_after(kernel, dim3(grid), kThreads, smem, s, static_cast<unsigned>(split), wmap,
                        xmap, a, static_cast<T*>(p.y));
}

}  // namespace

cudaError_t launch_f8_mm(const F8Product& p, cudaStream_t s) {
    const int sms = sm_count();
    const int row_blocks = f8_blocks(p.rows), col_blocks = f8_blocks(p.cols);
    F8Args a{};
    a.w_scales = p.bank_scales;
    a.x_scales = p.x_scales;
    a.offsets = p.offsets;
    a.n_experts = p.n_experts;
    a.n_rows = p.n_rows;
    a.n_out = p.grad ? p.cols : p.rows;
    a.n_k = p.grad ? row_blocks : col_blocks;
    a.sw_expert = static_cast<long long>(row_blocks) * col_blocks;
    a.sw_out = p.grad ? 1 : col_blocks;
    a.sw_k = p.grad ? col_blocks : 1;
    a.n_rt = f8_blocks(a.n_out);
    int split = 1, per_sm = 1;
    if (p.offsets != nullptr) {
        const int mean = (p.n_rows + p.n_experts - 1) / p.n_experts;
        a.tn = mean <= 8 ? 16 : mean <= 24 ? 32 : mean <= 48 ? 64 : 128;
        a.box = 16;
        a.n_tt = 0;
    } else {
        a.tn = p.n_rows <= 16 ? 16 : p.n_rows <= 32 ? 32 : p.n_rows <= 64 ? 64 : 128;
        a.box = std::min(a.tn, (p.n_rows + 15) / 16 * 16);
        a.n_tt = (p.n_rows + a.tn - 1) / a.tn;
        const int fit = a.tn <= 32 ? 2 : 1;   // CTAs whose registers an SM holds
        while (a.n_tt == 1 && split < kMaxSplit && 3 * a.n_rt < 2 * sms &&
               a.n_rt * split * 2 <= fit * sms && split * 2 <= a.n_k)
            split *= 2;
        if (split > 1) per_sm = (a.n_rt * split + sms - 1) / sms;
    }
    const long tiles = static_cast<long>(a.n_rt) * a.n_tt;
    const unsigned grid = split > 1                 ? static_cast<unsigned>(a.n_rt * split)
                          : p.offsets != nullptr || tiles > sms ? static_cast<unsigned>(sms)
                                                                : static_cast<unsigned>(tiles);
    auto by_grad = [&](auto one, auto nc, auto sp) {
        using T = decltype(one);
        return p.grad ? launch_k<T, nc(), sp(), true>(p, a, split, per_sm, grid, s)
                      : launch_k<T, nc(), sp(), false>(p, a, split, per_sm, grid, s);
    };
    auto by_split = [&](auto one, auto nc) {
        return split > 1 ? by_grad(one, nc, std::true_type{}) : by_grad(one, nc, std::false_type{});
    };
    auto by_width = [&](auto one) {
        switch (a.tn) {
            case 16: return by_split(one, std::integral_constant<int, 16>{});
            case 32: return by_split(one, std::integral_constant<int, 32>{});
            case 64: return by_split(one, std::integral_constant<int, 64>{});
            default: return by_split(one, std::integral_constant<int, 128>{});
        }
    };
    return p.y_type == kTypeF32 ? by_width(float{}) : by_width(__nv_bfloat16{});
}

cudaError_t read_fault_f8(int* value, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_f8, sizeof(int));
    if (e != cudaSuccess || !reset) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_fault_f8, &zero, sizeof(int));
}

}  // namespace mxk
