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
// Two kernels, by the number of tokens; in both, warps have roles: copies (TMA, 128-byte swizzled
// rows), MMAs, scales (asynchronous copies of 4 bytes, several blocks ahead: fetched when they
// are needed, their latency bounded a block), and eight warps for the sums.
//
// What bounds them: few tokens, HBM (64 experts 2880x2880, 32 tokens, top-4: 65 to 71 us, 6.6 TB/s;
// one token 14336x4096 12.8 us, of which the stream of the weights is 8.8); many tokens, about 900 to
// 1000 cycles a block of 128 x 256 sums, of which the MMAs are 512: by single CTAs copies and MMAs
// take 935, as 48 KB of operands go through shared memory, by pairs the accumulators' way
// round (2048 tokens 4096x14336 109 to 114 us, 2.1 to 2.2 PFLOP/s; 4096 tokens 4096x4096 by the rows
// 65 to 68 us, 2.1; 2048 tokens, top-4 of 64 experts 2880x2880, 123 to 135 us).
//
// Every wait is bounded; a CTA that gives up sets the fault word, lets its copies land, frees its
// tensor memory and returns.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "f8_kernels.h"
#include "kernels.h"
#include "pdl.cuh"
#include "tc5.cuh"

namespace mxk {
namespace {

namespace cg = cooperative_groups;

// --- few tokens -------------------------------------------------------------------------
//
// The matrix's outputs are the MMA's 128 rows and the tokens its columns: one scale of W for a
// whole tile and block, one of X for a column.  A warp has a quarter of the rows and half of the
// columns.  Persistent: CTA c takes tiles c, c + grid, ...  With few tiles a cluster of CTAs
// shares one, each a slice of the blocks, and adds the partial sums through distributed
// shared memory in rank order.

constexpr int kM = 128;                      // outputs per tile
constexpr uint32_t kABytes = kM * kF8Block;  // W's part of a stage
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;                 // CTAs of a cluster sharing a tile
constexpr int kTileTable = 64;               // this CTA's first tiles, worked out at the start
constexpr int kFac = 8;                      // units whose scales are held ahead
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

// The experts' row offsets, and the tiles of the experts before each, in shared memory (all
// threads; *n_tiles is there after the next barrier).
template <int kN>
__device__ __forceinline__ void read_experts(const F8Args& a, int32_t* off, int32_t* first,
                                             int* n_tiles) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e <= a.n_experts; e += kN)
        off[e] = min(max(ld_dep(a.offsets + e), 0), a.n_rows);
    __syncthreads();
    if (tid < 32) {
        int base = 0;
        for (int e0 = 0; e0 < a.n_experts; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < a.n_experts) n = a.n_rt * ((max(off[e + 1] - off[e], 0) + a.tn - 1) / a.tn);
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
            *n_tiles = base;
        }
    }
}

// Tile `tile` of `width` outputs.  An output tile's token tiles come one after the other, so that
// its part of the matrix is read again from L2; an expert's rows are cut into equal tiles of a
// multiple of 16.
__device__ __forceinline__ Tile locate(const F8Args& a, const int32_t* off, const int32_t* first,
                                       int tile, int width) {
    Tile t;
    if (a.offsets == nullptr) {
        t.e = 0;
        const int rt = tile / a.n_tt;
        t.r0 = rt * width;
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
        t.r0 = rt * width;
        t.t0 = off[lo] + (local - rt * n_tt) * per;
        t.t1 = min(t.t0 + per, off[lo + 1]);
    }
    return t;
}

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

// NC: most tokens of a tile.  A ring stage is a unit of kU blocks (one barrier each way for
// both), and so is an accumulator: kAcc of them, kU * NC columns each.
template <int NC, bool kSplit>
struct Shape {
    static constexpr int kU = NC <= 64 ? 2 : 1;
    static constexpr int kAcc = NC == 16 || (NC == 32 && !kSplit) ? 4 : 2;
    static constexpr uint32_t kUnit = kU * NC, kTmem = kAcc * kUnit;   // columns
    static constexpr int kHalf = NC / 2;      // columns a warp
    static constexpr int kFacRow = NC + 4;    // floats of a block's scales: X's, then W's
};

// Two CTAs an SM: for the split form, whose clusters share SMs.  (The unsplit one asks for all of the
// shared memory and is alone on its SM; under the same bound it spills 36 bytes a thread at 32 tokens.)
template <typename T, int NC, bool kSplit, bool kGrad>
__global__ void __launch_bounds__(kThreads, NC <= 32 ? 2 : 1)
    k_f8_mm(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
            const F8Args a, T* __restrict__ Y) {
    using S = Shape<NC, kSplit>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[S::kAcc], acc_empty[S::kAcc];
    __shared__ uint64_t fac_full[kFac], fac_empty[kFac], drain;
    __shared__ __align__(16) float fac[kFac][S::kU][S::kFacRow];
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
            mbar_init(&fac_full[i], 64);
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
        read_experts<kThreads>(a, off, first, &n_tiles_sh);
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

    if (tid < kTileTable && tile0 + tid * tile_step < n_tiles)
        table[tid] = locate(a, off, first, tile0 + tid * tile_step, kM);
    __syncthreads();
    if (a.offsets == nullptr) pdl_wait();   // nothing in memory was needed so far
    auto tile_at = [&](int tile, int j) {
        return j < kTileTable ? table[j] : locate(a, off, first, tile, kM);
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_fault_f8, 1);
    };
    const uint32_t block_bytes = kABytes + static_cast<uint32_t>(a.tn) * kF8Block;

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
            for (int s0 = s_lo; s0 < s_hi; s0 += S::kU) {
                ok = mbar_wait_for(&empty[st], phase, kWait);
                if (!ok) break;
                if (leader) {
                    const int n_s = min(S::kU, s_hi - s0);
                    mbar_arrive_expect_tx(&full[st], n_s * bytes);
#pragma unroll
                    for (int u = 0; u < S::kU; ++u) {
                        if (u == n_s) break;
                        const uint32_t dst = ring + st * a.stage_bytes + u * block_bytes;
                        const int k = (s0 + u) * kF8Block;
                        if constexpr (kGrad) tma3d(dst, &wmap, t.r0, k, t.e, &full[st], w_policy);
                        else tma3d(dst, &wmap, k, t.r0, t.e, &full[st], w_policy);
                        for (int b = 0; b < n_box; ++b)
                            tma2d(dst + kABytes + static_cast<uint32_t>(b) * box_bytes, &xmap, k,
                                  t.t0 + b * a.box, &full[st], keep);
                    }
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
        // --- MMAs: a block's four of K = 32 each into its accumulator
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
            for (int s0 = s_lo; s0 < s_hi; s0 += S::kU) {
                ok = warp_wait_both(&full[st], phase, &acc_empty[ab], acc_phase, kWait);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t at = st * (a.stage_bytes >> 4);
#pragma unroll
                    for (int u = 0; u < S::kU; ++u) {
                        if (u > 0 && s0 + u >= s_hi) break;
                        const uint32_t d = tmem + ab * S::kUnit + u * NC;
                        const uint32_t at_u = at + u * (block_bytes >> 4);
#pragma unroll
                        for (uint32_t q = 0; q < 4; ++q)
                            umma_f8(d, a0 + at_u + q * kAStep, b0 + at_u + q * 2, id, q);
                    }
                    umma_commit(&acc_full[ab]);
                    umma_commit(&empty[st]);
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
    } else if (warp < kEpiWarp) {
        // --- scales (two warps)
        const uint32_t slots = smem_u32(&fac[0][0][0]);
        uint32_t f = 0, phase = 1;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const float* w = a.w_scales + t.e * a.sw_expert +
                             static_cast<long long>(t.r0 / kM) * a.sw_out;
            const int n = t.t1 - t.t0;
            for (int s0 = s_lo; s0 < s_hi; s0 += S::kU) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_for(&fac_empty[f], phase, kWait));
                if (!ok) break;
                const int n_s = min(S::kU, s_hi - s0);
#pragma unroll
                for (int i0 = 0; i0 < S::kU * NC; i0 += 64) {
                    const int u = (i0 + tid - 64) / NC, c = (i0 + tid - 64) % NC;
                    if (c < n && u < n_s)
                        copy4(slots + ((f * S::kU + u) * S::kFacRow + c) * 4,
                              a.x_scales + static_cast<size_t>(s0 + u) * a.n_rows + t.t0 + c);
                }
                if (warp == 3 && lane < n_s)
                    copy4(slots + ((f * S::kU + lane) * S::kFacRow + NC) * 4,
                          w + static_cast<long long>(s0 + lane) * a.sw_k);
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
        constexpr int kLd = S::kHalf < 32 ? S::kHalf : 32;
        uint32_t ab = 0, acc_phase = 0, f = 0, fac_phase = 0;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int n = t.t1 - t.t0 - half * S::kHalf;   // of this half (may be none)
            float2 sum[S::kHalf / 2];
#pragma unroll
            for (int i = 0; i < S::kHalf / 2; ++i) sum[i] = make_float2(0.0f, 0.0f);
            for (int s0 = s_lo; s0 < s_hi; s0 += S::kU) {
                ok = warp_wait_both(&acc_full[ab], acc_phase, &fac_full[f], fac_phase, kWait);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[S::kU][S::kHalf];
#pragma unroll
                for (int u = 0; u < S::kU; ++u)
#pragma unroll
                    for (int c = 0; c < S::kHalf; c += kLd)
                        if (c < n && (u == 0 || s0 + u < s_hi))
                            tmem_ld<kLd>(tmem + ab * S::kUnit + u * NC + half * S::kHalf + c +
                                             (static_cast<uint32_t>(quarter * 32) << 16),
                                         &v[u][c]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_m(&acc_empty[ab]);
#pragma unroll
                for (int u = 0; u < S::kU; ++u) {
                    if (n <= 0 || (u > 0 && s0 + u >= s_hi)) break;
                    const float w = fac[f][u][NC];
                    const float4* x = reinterpret_cast<const float4*>(&fac[f][u][half * S::kHalf]);
#pragma unroll
                    for (int i = 0; i < S::kHalf / 4; ++i) {
                        const float4 p = x[i];
                        float2& s_0 = sum[2 * i];
                        float2& s_1 = sum[2 * i + 1];
                        s_0 = __ffma2_rn(make_float2(__uint_as_float(v[u][4 * i]),
                                                     __uint_as_float(v[u][4 * i + 1])),
                                         __fmul2_rn(make_float2(p.x, p.y), make_float2(w, w)), s_0);
                        s_1 = __ffma2_rn(make_float2(__uint_as_float(v[u][4 * i + 2]),
                                                     __uint_as_float(v[u][4 * i + 3])),
                                         __fmul2_rn(make_float2(p.z, p.w), make_float2(w, w)), s_1);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_m(&fac_empty[f]);
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
        // four outputs a thread (one each took 3 us more for 333 tokens, 2303x2880: a remote load
        // answers after several hundred cycles)
        const int n_quads = (t.t1 - t.t0) * (kM / 4);
        const bool whole = a.n_out % 4 == 0 && t.r0 + kM <= a.n_out;
        for (int i = rank * kThreads + tid; i < n_quads && !*abort_flag; i += n_rank * kThreads) {
            float4 v[kMaxSplit];   // all loads on their way before the first sum
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                if (q < n_rank)
                    v[q] = reinterpret_cast<const float4*>(cluster.map_shared_rank(part, q))[i];
            float sum[4] = {};
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                if (q < n_rank) {
                    sum[0] += v[q].x;
                    sum[1] += v[q].y;
                    sum[2] += v[q].z;
                    sum[3] += v[q].w;
                }
            const int r = t.r0 + i % (kM / 4) * 4;
            T* dst = Y + static_cast<size_t>(t.t0 + i / (kM / 4)) * a.n_out + r;
            if (whole) {
                Pack<T, 4> p;
                p.set(sum);
                store_pack(reinterpret_cast<Pack<T, 4>*>(dst), p);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (r + q < a.n_out) dst[q] = from_f32<T>(sum[q]);
            }
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

// --- many tokens ------------------------------------------------------------------------
//
// The other way round: 128 tokens are the MMA's rows and 256 outputs its columns, so that in
// the sums one thread has one token, and a block's two scales are one factor for all its
// columns.  Eight warps hold the 128 x 256 sums (128 columns a thread); tensor memory holds two
// blocks of the tile, in halves of 128 outputs, each with a warp that multiplies it and four that
// add it: multiplying, handing over and reading overlap.
//
// kPair: two CTAs share each MMA (256 tokens; either brings its 128 and half of the outputs'
// rows), so that an operand byte is fetched for twice the products.  Then the hand-over crosses the
// pair, and tiles are coarser: better for one matrix with many tokens, not for experts (us, one after
// the other on one GPU: 2048 tokens 4096x14336 108, single CTAs 123; a prompt's experts 147 and 131).
// Results leave by copies from shared memory where rows are 16-byte aligned (4096 tokens 8192x2048
// into f32 72 us, by stores 79); an expert's last tile must not write past its rows, so there by
// stores.
constexpr int kWN = 256;
constexpr uint32_t kWHalf = kM * kF8Block;   // 128 rows of a stage
constexpr int kWThreads = 384, kWEpiWarp = 4, kWEpiWarps = 8, kWCols = 128;
constexpr int kWFac = 8;           // blocks whose scales are held
template <bool kPair>
struct Wide {
    static constexpr uint32_t kWRows = kPair ? kM : kWN;   // outputs that a CTA brings
    static constexpr uint32_t kStage = kWHalf + kWRows * kF8Block;
    static constexpr int kStages = kPair ? 5 : 4;
    static constexpr int kPatch = kPair ? 4096 : 2048;     // bytes a warp stores at a time
    static constexpr int kBox = kPair ? 64 : 128;          // outputs of a copy: a CTA's of a half
    static constexpr size_t kSmem = kStages * kStage + kWEpiWarps * kPatch + 1024;
};

// 16 of a lane's sums (n of them exist) for rows of any alignment: as store_turned, element by
// element, two rows' 16 outputs a store.
template <typename T>
__device__ __forceinline__ void store_any(T* y, size_t pitch, int rows, const float2* sum, int n,
                                          float* patch, int lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        patch[lane * 16 + ((2 * i) ^ (lane >> 1 & 15))] = sum[i].x;
        patch[lane * 16 + ((2 * i + 1) ^ (lane >> 1 & 15))] = sum[i].y;
    }
    __syncwarp();
    const int c = lane & 15;
    if (c < n)
        for (int r = lane >> 4; r < rows; r += 2)
            y[static_cast<size_t>(r) * pitch + c] =
                from_f32<T>(patch[r * 16 + (c ^ (r >> 1 & 15))]);
    __syncwarp();
}

template <bool kPair>
__device__ __forceinline__ void wide_umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else umma_f8(d, a, b, idesc, accumulate);
}
template <bool kPair>
__device__ __forceinline__ void wide_commit(uint64_t* bar) {
    if constexpr (kPair) pair_commit(bar);
    else umma_commit(bar);
}

template <typename T, bool kGrad, bool kPair>
__global__ void __launch_bounds__(kWThreads, 1)
    k_f8_wide(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
              const __grid_constant__ CUtensorMap ymap, const F8Args a, T* __restrict__ Y) {
    using S = Wide<kPair>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[4], acc_empty[4];
    __shared__ uint64_t fac_full[kWFac], fac_empty[kWFac], drain[2];
    __shared__ float fac[kWFac][kM + 4];   // a block's scales: X's, then W's two
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word, n_tiles_sh;
    __shared__ Tile table[kTileTable];
    volatile int* abort_flag = &abort_word;
    uint8_t* patches = smem + S::kStages * S::kStage;
    int32_t* off = reinterpret_cast<int32_t*>(patches + kWEpiWarps * S::kPatch);
    int32_t* first = off + a.n_experts + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kPair ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    auto sync_all = [] {   // of the pair
        if constexpr (kPair) cg::this_cluster().sync();
        else __syncthreads();
    };

    if (warp == 1) {
        if constexpr (kPair) pair_tmem_take(&tmem_base, 2 * kWN);
        else tmem_take(&tmem_base, 2 * kWN);
    }
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);    // (a pair's: rank 0's, for both CTAs' copies)
            mbar_init(&empty[i], 2);   // both halves' MMAs
        }
        for (int i = 0; i < 4; ++i) {   // [two blocks][two halves of the outputs]
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kWEpiWarps / 2 * (kPair ? 2 : 1));   // (a pair's: rank 0's)
        }
        for (int i = 0; i < kWFac; ++i) {
            mbar_init(&fac_full[i], 32);
            mbar_init(&fac_empty[i], kWEpiWarps);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);   // one for each warp that multiplies
        abort_word = 0;
        n_tiles_sh = a.n_rt * a.n_tt;
        fence_mbar_init();
    }
    if (tid == 32 * 2) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&wmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
    }
    tc_fence_before();
    sync_all();   // barriers and tensor memory are there
    tc_fence_after();
    pdl_trigger();
    if (a.offsets != nullptr) {
        pdl_wait();
        read_experts<kWThreads>(a, off, first, &n_tiles_sh);
    }
    __syncthreads();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    const int n_tiles = __shfl_sync(0xFFFFFFFFu, n_tiles_sh, 0);
    constexpr int kCtas = kPair ? 2 : 1;
    const int tile0 = static_cast<int>(blockIdx.x) / kCtas;
    const int tile_step = static_cast<int>(gridDim.x) / kCtas;
    if (tid < kTileTable && tile0 + tid * tile_step < n_tiles)
        table[tid] = locate(a, off, first, tile0 + tid * tile_step, kWN);
    __syncthreads();
    if (a.offsets == nullptr) pdl_wait();   // nothing in memory was needed so far
    auto tile_at = [&](int tile, int j) {
        return j < kTileTable ? table[j] : locate(a, off, first, tile, kWN);
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_fault_f8, 1);
    };

    // 384 threads of 168 registers: the sums' warps take what the others do not need
    if (warp < kWEpiWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
        // --- copies: this CTA's 128 tokens (where it has any) and its outputs of both halves
        const bool leader = elect_one();
        const uint64_t keep = l2_evict_last(), w_policy = l2_evict_normal();
        const uint32_t ring = smem_u32(smem);
        const uint32_t full0 = kPair ? leader_addr(&full[0]) : smem_u32(&full[0]);
        uint32_t st = 0, phase = 1;   // the first round of the ring passes at once
        int j = 0;
        bool ok = true;
        auto next = [&]() {
            if (++st == S::kStages) {
                st = 0;
                phase ^= 1u;
            }
        };
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const bool both = kPair && t.t0 + kM < t.t1;
            const uint32_t bytes = kWN * kF8Block + (both ? 2 : 1) * kWHalf;
            for (int s = 0; s < a.n_k; ++s) {
                ok = mbar_wait_for(&empty[st], phase, kWait);
                if (!ok) break;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
                    const uint32_t bar = full0 + st * 8, dst = ring + st * S::kStage;
                    const int k = s * kF8Block;
                    if constexpr (kPair) {
                        if (rank == 0 || both)
                            pair_tma2d(dst, &xmap, k, t.t0 + rank * kM, bar, keep);
                    } else {
                        tma2d(dst, &xmap, k, t.t0, &full[st], keep);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w = dst + kWHalf + h * S::kBox * kF8Block;
                        const int out = t.r0 + h * kM + rank * S::kBox;
                        const int x = kGrad ? out : k, y = kGrad ? k : out;
                        if constexpr (kPair) pair_tma3d(w, &wmap, x, y, t.e, bar, w_policy);
                        else tma3d(w, &wmap, x, y, t.e, &full[st], w_policy);
                    }
                }
                __syncwarp();
                next();
            }
            ok = ok && !*abort_flag;
        }
        if constexpr (kPair)   // the pair's last arrivals here land before this CTA may leave
            for (int i = 0; i < S::kStages && ok; ++i, next())
                ok = mbar_wait_for(&empty[st], phase, kWait);
        if (!ok) fail();
        __syncwarp();
    } else if (warp == 2) {
        // --- scales: a block's 128 of X and two of W
        uint32_t f = 0, phase = 1;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const float* xs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                xs[i] = a.x_scales + min(t.t0 + rank * kM + 32 * i + lane, a.n_rows - 1);
            const float* ws = a.w_scales + t.e * a.sw_expert +
                              static_cast<long long>(t.r0 / kF8Block) * a.sw_out +
                              (lane == 1 && t.r0 + kF8Block < a.n_out ? a.sw_out : 0);
            for (int s = 0; s < a.n_k; ++s) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_for(&fac_empty[f], phase, kWait));
                if (!ok) break;
                const uint32_t dst = smem_u32(&fac[f][0]) + lane * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    copy4(dst + i * 128, xs[i]);
                    xs[i] += a.n_rows;
                }
                if (lane < 2) copy4(dst + kM * 4, ws);
                ws += a.sw_k;
                async_arrive(&fac_full[f]);
                if (++f == kWFac) {
                    f = 0;
                    phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp < kWEpiWarp && rank == 0) {
        // --- MMAs: warp 1 the first half of the outputs, warp 3 the second
        const uint32_t h = warp == 1 ? 0u : 1u;
        const bool leader = elect_one();
        const uint32_t ring = smem_u32(smem);
        const uint32_t w = ring + kWHalf + h * S::kBox * kF8Block;
        const uint64_t a0 = operand_desc(ring);
        const uint64_t b0 = !kGrad  ? operand_desc(w)
                            : kPair ? operand_desc_mn64(w)
                                    : operand_desc_mn(w, kWHalf);
        // K = 32: 32 bytes of a row, or 32 rows of a copy
        constexpr uint32_t kBStep = kGrad ? 32 * S::kBox / 16 : 2;
        // D = F32, A = B = E4M3, W (B) by its contiguous side
        constexpr uint32_t id = (1u << 4) | (kGrad ? 1u << 16 : 0u) |
                                (static_cast<uint32_t>(kWN / 2 >> 3) << 17) |
                                (static_cast<uint32_t>(kCtas * kM >> 4) << 24);
        uint32_t st = 0, phase = 0, ab = 0, acc_phase = 1;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            for (int s = 0; s < a.n_k; ++s) {
                ok = warp_wait_both(&full[st], phase, &acc_empty[2 * ab + h], acc_phase, kWait);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t at = st * (S::kStage >> 4);
                    const uint32_t d = tmem + ab * kWN + h * (kWN / 2);
#pragma unroll
                    for (uint32_t q = 0; q < 4; ++q)
                        wide_umma<kPair>(d, a0 + at + q * 2, b0 + at + q * kBStep, id, q);
                    wide_commit<kPair>(&acc_full[2 * ab + h]);
                    wide_commit<kPair>(&empty[st]);
                }
                __syncwarp();
                if (++st == S::kStages) {
                    st = 0;
                    phase ^= 1u;
                }
                ab ^= 1u;
                acc_phase ^= ab ^ 1u;
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) {
            fail();
            if (leader) wide_commit<kPair>(&drain[h]);
            mbar_wait_for(&drain[h], 0u, kWait);
        }
        __syncwarp();
    } else if (warp >= kWEpiWarp) {
        // --- sums: lane = token, 128 outputs a warp
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int quarter = warp & 3, group = (warp - kWEpiWarp) >> 2;
        const uint32_t src =
            tmem + group * kWCols + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t done =
            kPair ? leader_addr(&acc_empty[group]) : smem_u32(&acc_empty[group]);
        const uint32_t align = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(Y) |
                                                     static_cast<size_t>(a.n_out) * sizeof(T));
        uint8_t* patch = patches + (warp - kWEpiWarp) * S::kPatch;
        uint32_t ab = 0, acc_phase = 0, slot = 0, fac_phase = 0;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int row0 = t.t0 + rank * kM + quarter * 32, c0 = t.r0 + group * kWCols;
            const int rows = min(t.t1 - row0, 32);   // of this warp's (may be none)
            float2 sum[kWCols / 2];
#pragma unroll
            for (int i = 0; i < kWCols / 2; ++i) sum[i] = make_float2(0.0f, 0.0f);
            for (int s = 0; s < a.n_k; ++s) {
                ok = warp_wait_both(&acc_full[2 * ab + group], acc_phase, &fac_full[slot], fac_phase,
                                    kWait);
                if (!ok) break;
                tc_fence_after();
                const float f = fac[slot][quarter * 32 + lane] * fac[slot][kM + group];
#pragma unroll
                for (int c = 0; c < kWCols; c += 64) {
                    uint32_t u[64];
                    if (rows > 0) {
                        tmem_ld<32>(src + ab * kWN + c, u);
                        tmem_ld<32>(src + ab * kWN + c + 32, u + 32);
                    }
                    tmem_ld_wait();
                    if (c + 64 == kWCols) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (kPair) pair_arrive(done + ab * 16);
                            else mbar_arrive_m(&acc_empty[2 * ab + group]);
                            mbar_arrive_m(&fac_empty[slot]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sum[c / 2 + i] = __ffma2_rn(make_float2(__uint_as_float(u[2 * i]),
                                                                __uint_as_float(u[2 * i + 1])),
                                                    make_float2(f, f), sum[c / 2 + i]);
                }
                ab ^= 1u;
                acc_phase ^= ab ^ 1u;
                if (++slot == kWFac) {
                    slot = 0;
                    fac_phase ^= 1u;
                }
            }
            if (!ok) {
                fail();
                break;
            }
            T* dst = Y + static_cast<size_t>(row0) * a.n_out + c0;
            if (kPair && align % 16 == 0) {
                // 128 bytes of the 32 rows at a time, by copies from shared memory (which cut off
                // at the matrix's edges): the warp goes on while they run
                constexpr int kE = 128 / sizeof(T), kUnit = 16 / sizeof(T);
#pragma unroll
                for (int c = 0; c < kWCols; c += kE) {
                    if (lane == 0) bulk_wait_read<0>();   // the last copy has read the patch
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float f[kUnit];
#pragma unroll
                        for (int i = 0; i < kUnit; ++i) {
                            const float2 v = sum[(c + q * kUnit + i) / 2];
                            f[i] = i % 2 ? v.y : v.x;
                        }
                        Pack<T, kUnit> p;
                        p.set(f);
                        *reinterpret_cast<uint4*>(patch + lane * 128 + (q ^ (lane & 7)) * 16) =
                            p.raw;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (c0 + c < a.n_out && rows > 0)
                            tma2d_store(&ymap, c0 + c, row0, smem_u32(patch));
                        bulk_commit();
                    }
                }
            } else if (align % 16 == 0) {
                constexpr int kE = 64 / sizeof(T);
#pragma unroll
                for (int c = 0; c < kWCols; c += kE)
                    if (c0 + c < a.n_out)
                        store_turned(dst + c, static_cast<size_t>(a.n_out), rows, &sum[c / 2],
                                     a.n_out - c0 - c, patch, lane, align % 32 == 0);
            } else {
#pragma unroll
                for (int c = 0; c < kWCols; c += 16)
                    if (c0 + c < a.n_out)
                        store_any(dst + c, static_cast<size_t>(a.n_out), rows, &sum[c / 2],
                                  a.n_out - c0 - c, reinterpret_cast<float*>(patch), lane);
            }
            ok = !*abort_flag;
        }
        if constexpr (kPair) {
            if (lane == 0) bulk_wait_all();
            __syncwarp();
        }
    }

    __syncthreads();
    if (*abort_flag && tid == 0) {
        // a CTA that gave up: its copies in flight land long before this
        for (const long long t0 = clock64(); clock64() - t0 < kDrain;) __nanosleep(1000);
    }
    tc_fence_before();
    sync_all();   // neither of a pair leaves while the other still multiplies from its memory
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kPair) pair_tmem_give(tmem, 2 * kWN);
        else tmem_give(tmem, 2 * kWN);
    }
}

// --- host side --------------------------------------------------------------------------

// `n` matrices of codes [rows][cols], copies of box_rows x box_cols (128 or 64, as is the swizzle).
bool code_map(CUtensorMap* map, const void* base, int cols, int rows, int n, int box_rows,
              int box_cols = kF8Block) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols),
                                   static_cast<cuuint64_t>(cols) * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows),
                               1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, n > 0 ? 3 : 2, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_cols == kF8Block ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Y [n_rows][n_out], copies of 128 bytes x 32 rows.
template <typename T>
bool out_map(CUtensorMap* map, void* y, int n_out, int n_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n_out), static_cast<cuuint64_t>(n_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(n_out) * sizeof(T)};
    const cuuint32_t box[2] = {128 / sizeof(T), 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map,
              sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmemMax = 227 * 1024, kSmemSlack = 8 * 1024;   // (the static arrays)

template <typename T, int NC, bool kSplit, bool kGrad>
cudaError_t launch_k(const F8Product& p, F8Args a, int split, int per_sm, unsigned grid,
                     cudaStream_t s) {
    using S = Shape<NC, kSplit>;
    a.stage_bytes = S::kU * (kABytes + static_cast<uint32_t>(a.tn) * kF8Block);
    const size_t extra =
        p.offsets != nullptr ? static_cast<size_t>(p.n_experts + 1) * 8 : 0;
    const size_t budget = kSmemMax / per_sm - kSmemSlack - 1024 - extra;
    a.n_stages = std::min(kMaxStages, static_cast<int>(budget / a.stage_bytes));
    if (kSplit) {
        // no more stages than a slice has, but room for the partial sums
        const int most = ((a.n_k + split - 1) / split + S::kU - 1) / S::kU;
        const int sums = (a.tn * kM * 4 + static_cast<int>(a.stage_bytes) - 1) /
                         static_cast<int>(a.stage_bytes);
        a.n_stages = std::min(a.n_stages, std::max(std::max(most, sums), 2));
    }
    const size_t ring = static_cast<size_t>(a.n_stages) * a.stage_bytes + extra + 1024;
    // CTAs that share an SM never ask for more than its 512 columns of tensor memory together (2.25
    // a KB): one that waits for columns must not hold up its cluster
    const size_t smem = kSplit ? std::max(ring, static_cast<size_t>(S::kTmem) * 1024 * 4 / 9)
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

// Clusters of `split` CTAs, per_sm (1 or 2) on an SM, that the device holds at once (its SMs come
// in groups that a cluster does not cross), 0 where it cannot say.
int clusters_at_once(int split, int per_sm) {
    static PerDevice memo[2][3];
    return memo[per_sm - 1][split / 4].get([&] {
        auto kernel = per_sm == 1 ? k_f8_mm<float, 128, true, false> : k_f8_mm<float, 32, true, false>;
        const size_t smem = kSmemMax / per_sm - kSmemSlack;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(split));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(split);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemMax - kSmemSlack)) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        return n;
    });
}

template <typename T, bool kGrad, bool kPair>
cudaError_t launch_wide(const F8Product& p, const F8Args& a, cudaStream_t s) {
    using S = Wide<kPair>;
    const size_t extra = p.offsets != nullptr ? static_cast<size_t>(p.n_experts + 1) * 8 : 0;
    auto kernel = k_f8_wide<T, kGrad, kPair>;
    static PerDevice memo;
    const cudaError_t attr_err = static_cast<cudaError_t>(memo.get([&] {
        return static_cast<int>(
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemMax - kSmemSlack)));
    }));
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap wmap, xmap;
    if (!code_map(&wmap, p.bank, p.cols, p.rows, p.n_experts, kGrad ? kF8Block : S::kBox,
                  kGrad ? S::kBox : kF8Block) ||
        !code_map(&xmap, p.x, kGrad ? p.rows : p.cols, p.n_rows, 0, kM))
        return cudaErrorNotSupported;
    CUtensorMap ymap = xmap;
    if (kPair && (reinterpret_cast<uintptr_t>(p.y) | static_cast<size_t>(a.n_out) * sizeof(T)) % 16 ==
                     0 &&
        !out_map<T>(&ymap, p.y, a.n_out, p.n_rows))
        return cudaErrorNotSupported;
    constexpr unsigned kCtas = kPair ? 2 : 1;
    const long tiles = static_cast<long>(a.n_rt) * a.n_tt, most = sm_count() / kCtas;
    const unsigned grid =
        kCtas * static_cast<unsigned>(p.offsets != nullptr || tiles > most ? most : tiles);
    return launch_after(kernel, dim3(grid), kWThreads, S::kSmem + extra, s, kCtas, wmap, xmap, ymap, a,
                        static_cast<T*>(p.y));
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
    const int mean = (p.n_rows + p.n_experts - 1) / p.n_experts;
    int split = 1, per_sm = 1;
    bool wide;
    if (p.offsets != nullptr) {
        // the narrowest tile that takes the mean expert's rows; past 48 of them the tiles of 128
        // tokens (us, 64 experts 2880x2880: 32 rows each 91 in tiles of 64, 105 in tiles of 128;
        // 48 rows 98 and 105; 64 rows 143 and 106)
        wide = mean > 48;
        a.tn = mean <= 8 ? 16 : mean <= 24 ? 32 : 64;
        a.box = 16;
        a.n_tt = 0;
    } else {
        a.tn = p.n_rows <= 16 ? 16 : p.n_rows <= 32 ? 32 : p.n_rows <= 64 ? 64 : 128;
        a.box = std::min(a.tn, (p.n_rows + 15) / 16 * 16);
        a.n_tt = (p.n_rows + a.tn - 1) / a.tn;
        // tiles for less than two thirds of the SMs: slices of the sum over a cluster, as many as
        // there is room for at once (us: 4096x14336, one token 23.1 unsplit, 15.0 by 2, 13.3 by 4;
        // 4096x4096, 128 tokens 21.1, 18.3 and 11.5; 2048x4096, 128 tokens by 4 10.5, by 8, whose
        // clusters are not all there at once, 17.8; with 112 tiles, 14336x4096, one token, 12.7
        // unsplit, by 2 13.6)
        const int fit = a.tn <= 32 ? 2 : 1;   // CTAs whose registers an SM holds
        const long tiles = static_cast<long>(a.n_rt) * a.n_tt;
        while (split < kMaxSplit && 3 * tiles < 2 * sms && split * 2 <= a.n_k &&
               tiles <= clusters_at_once(split * 2, fit))
            split *= 2;
        if (split > 1) per_sm = tiles <= clusters_at_once(split, 1) ? 1 : 2;
        // Past 64 tokens either kernel takes about as long for a block of its tile (1000 cycles),
        // and the other one's tiles are twice as large: it is slower only where this one is split
        // (us: 4096x4096, 256 tokens 14.9 by 2, 21.8 the other; 512 tokens, not split, 20.4 the
        // other; 2303x2880, 333 tokens 12.8 by 2 and 21.5).  Up to 128 tokens its tiles are not full:
        // a pair's second CTA then brings outputs but has no token (14336x4096: 64 tokens 15.5, 65 to
        // 128 as long as 256, 21; this kernel unsplit was not timed there).
        wide = a.tn == 128 && split == 1;
    }
    if (wide) {
        a.n_rt = (a.n_out + kWN - 1) / kWN;
        auto rounds = [&](int tokens, int at_once) {   // of tiles over the SMs
            return (static_cast<long>(a.n_rt) * ((p.n_rows + tokens - 1) / tokens) + at_once - 1) /
                   at_once;
        };
        const bool pair = p.offsets == nullptr && rounds(2 * kM, sms / 2) <= rounds(kM, sms);
        a.tn = pair ? 2 * kM : kM;
        a.n_tt = p.offsets != nullptr ? 0 : (p.n_rows + a.tn - 1) / a.tn;
        auto by_pair = [&](auto one, auto grad) {
            using T = decltype(one);
            return pair ? launch_wide<T, grad(), true>(p, a, s)
                        : launch_wide<T, grad(), false>(p, a, s);
        };
        auto go = [&](auto one) {
            return p.grad ? by_pair(one, std::true_type{}) : by_pair(one, std::false_type{});
        };
        return p.y_type == kTypeF32 ? go(float{}) : go(__nv_bfloat16{});
    }
    const long tiles = static_cast<long>(a.n_rt) * a.n_tt;
    const unsigned grid = split > 1                 ? static_cast<unsigned>(tiles * split)
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
            default: return by_grad(one, std::integral_constant<int, 128>{}, std::true_type{});
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
