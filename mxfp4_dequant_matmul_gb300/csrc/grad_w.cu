// grad_w.cu -- the gradient of a product by its matrices (include/f8.h mxfp4_mm_grad_w,
// mxfp4_moe_mm_grad_w; tcgen05 kind::f16, sm_103a).
//
// dW_e[r][c] = sum_{i in e} dY[i][r] X[i][c]: both operands lie with the sum's side (the rows i)
// outermost, so each copy brings 64 rows of 64 elements (128 bytes) as they are, and the
// descriptors say that the M and N sides are contiguous: nothing is transposed.
//
// A tile is 256 rows by 256 columns of a dW_e, its sum the rows of expert e, 64 a ring stage.  A
// pair of CTAs shares its MMAs: either brings 128 of the tile's rows and of its columns, and gets
// its 128 rows' sums, so that each operand byte is fetched for twice the products.  The tensor
// core's FP32 sums lose up to a bit with each addition; after 256 rows (four stages) they are added,
// rounded to nearest, to sums that eight warps hold in registers (two accumulators, in turn).
//
// Rows past the expert's end (another expert's, or none) are no part of it: the MMAs stop at the
// last 16 rows that hold one of its own, and what follows in those 16 is overwritten by zeros in
// shared memory (in both operands: zero times whatever lies there may be NaN).  That last stage
// lands on a barrier of its own CTA, a warp of which writes the zeros before it reports the stage.
//
// What bounds it: 4096 tokens top-4 of 16 experts 2880x2880 bf16 into f32, 235 to 255 us, 1.07 to 1.16
// PFLOP/s: 182 without the stores, in which a stage takes about 700 cycles (the MMAs 512), as either
// CTA's 32 KB come from L2 at some 50 bytes a cycle; the stores are as much again as a fifth of those
// copies.  One matrix 2048x2048, 8192 rows: 47 us, 1.45 PFLOP/s; 4096x4096, 4096 rows 94 us, 1.46.
//
// Warps: copies, MMAs (even ranks), those zeros, eight for the sums.  Persistent: pair c takes tiles
// c, c + pairs, ...  With few tiles and long sums (kSplit) a cluster of two or four pairs shares a
// tile, each a slice of the stages, and adds the partial sums through distributed shared memory
// in rank order.
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

constexpr int kM = 128, kN = 256, kK = 64;    // a CTA's rows, a tile's columns, rows of a stage
constexpr int kBox = 64;                      // elements of a copied row (128 bytes)
constexpr uint32_t kBoxBytes = kBox * kK * 2;
constexpr uint32_t kABytes = 2 * kBoxBytes, kStageBytes = 2 * kABytes;   // of dY; and of X
constexpr int kStages = 5, kChunk = 4;        // ring; stages an accumulator takes
constexpr int kMaxSplit = 4;                  // pairs that share a tile
constexpr int kPatch = 32 * 128;               // bytes a warp stores at a time
constexpr int kThreads = 384, kEpiWarp = 4, kEpiWarps = 8, kCols = 128;
constexpr int kMaxExperts = 1024;
constexpr long long kWait = 1ll << 32, kDrain = 1ll << 24;   // SM cycles: about 2 s and 8 ms

__device__ int g_fault_grad_w;

struct WArgs {
    const int32_t* offsets;   // nullptr: one matrix
    int n_experts, rows, cols, n_rows;
    int n_rt, n_ct;           // tiles down and across a matrix
    uint32_t idesc;
};

__device__ __forceinline__ void pair_umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <typename T, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    k_grad_w(const __grid_constant__ CUtensorMap dymap, const __grid_constant__ CUtensorMap xmap,
             const __grid_constant__ CUtensorMap dwmap, const WArgs a, T* __restrict__ dw) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kStages], empty[kStages], last_full[kStages], acc_full[2], acc_empty[2];
    __shared__ uint64_t drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    __shared__ int32_t off[kMaxExperts + 1];
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    cg::cluster_group cluster = cg::this_cluster();
    const int cluster_rank = static_cast<int>(cluster.block_rank());
    const int rank = cluster_rank & 1, lead = kSplit ? cluster_rank & ~1 : 0;   // of the pair
    const int n_split = kSplit ? static_cast<int>(cluster.num_blocks()) / 2 : 1;

    if (warp == 1) pair_tmem_take(&tmem_base, 2 * kN);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 2);        // (the leader's) both CTAs' parts
            mbar_init(&empty[i], 1);
            mbar_init(&last_full[i], 1);   // a stage with rows to be zeroed
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpiWarps);   // (the leader's) both CTAs' warps
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_mbar_init();
    }
    if (tid == 32 * 2) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&dymap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
        if (!kSplit) asm volatile("prefetch.tensormap [%0];" ::"l"(&dwmap) : "memory");
    }
    tc_fence_before();
    cluster.sync();   // both CTAs' barriers and tensor memory are there
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    for (int e = tid; e <= a.n_experts; e += kThreads)
        off[e] = a.offsets == nullptr ? e * a.n_rows
                                      : min(max(ld_dep(a.offsets + e), 0), a.n_rows);
    __syncthreads();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);

    struct Tile {
        int e, r0, c0, i0, m;
        int lo, hi;   // this pair's rows of the m, from a multiple of kK on
    };
    const int per_e = a.n_rt * a.n_ct, n_tiles = per_e * a.n_experts;
    const int tile0 = static_cast<int>(blockIdx.x) / (2 * n_split);
    const int tile_step = static_cast<int>(gridDim.x) / (2 * n_split);   // (split: one tile each)
    auto tile_at = [&](int tile) {
        Tile t;
        t.e = tile / per_e;
        const int local = tile - t.e * per_e, rt = local / a.n_ct;
        t.r0 = rt * 2 * kM;
        t.c0 = (local - rt * a.n_ct) * kN;
        t.i0 = off[t.e];
        t.m = max(off[t.e + 1] - t.i0, 0);
        t.lo = 0;
        t.hi = t.m;
        if constexpr (kSplit) {
            const int stages = (t.m + kK - 1) / kK, q = lead / 2;
            t.lo = static_cast<int>(static_cast<long long>(stages) * q / n_split) * kK;
            t.hi = min(static_cast<int>(static_cast<long long>(stages) * (q + 1) / n_split) * kK,
                       t.m);
        }
        return t;
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_fault_grad_w, 1);
    };

    // 384 threads of 168 registers: the sums' warps take what the others do not need
    if (warp < kEpiWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
        // --- copies
        const bool leader = elect_one();
        const uint64_t policy = l2_evict_normal();
        const uint32_t ring = smem_u32(smem), full0 = leader_addr(&full[0], lead);
        uint32_t st = 0, phase = 1;   // the first round of the ring passes at once
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            const Tile t = tile_at(tile);
            const int r = t.r0 + rank * kM, c = t.c0 + rank * (kN / 2);
            for (int i = t.lo; i < t.hi; i += kK) {
                ok = mbar_wait_for(&empty[st], phase, kWait);
                if (!ok) break;
                if (leader) {
                    const bool zeros = i + kK > t.m && (t.m & 15) != 0;
                    uint32_t bar = full0 + st * 8;
                    if (zeros) bar = smem_u32(&last_full[st]);
                    if (zeros) mbar_arrive_expect_tx(&last_full[st], kStageBytes);
                    else pair_arrive_expect_tx(bar, kStageBytes);
                    const uint32_t dst = ring + st * kStageBytes;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        pair_tma2d(dst + b * kBoxBytes, &dymap, r + b * kBox, t.i0 + i, bar, policy);
                        pair_tma2d(dst + kABytes + b * kBoxBytes, &xmap, c + b * kBox, t.i0 + i,
                                   bar, policy);
                    }
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        // the pair's last arrivals on these barriers land before this CTA may leave
        for (int i = 0; i < kStages && ok; ++i) {
            ok = mbar_wait_for(&empty[st], phase, kWait);
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }
        if (!ok) fail();
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // --- MMAs
        const bool leader = elect_one();
        const uint32_t ring = smem_u32(smem);
        const uint64_t a0 = operand_desc_mn(ring, kBoxBytes);
        const uint64_t b0 = operand_desc_mn(ring + kABytes, kBoxBytes);
        uint32_t st = 0, phase = 0, ab = 0, acc_phase = 1;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            const Tile t = tile_at(tile);
            int in_chunk = 0;
            for (int i = t.lo; i < t.hi; i += kK) {
                ok = in_chunk > 0 || mbar_wait_for(&acc_empty[ab], acc_phase, kWait);
                ok = ok && mbar_wait_for(&full[st], phase, kWait);
                if (!ok) break;
                const int steps = min(kK, t.m - i + 15) >> 4;   // of 16 rows
                const bool done = in_chunk + 1 == kChunk || i + kK >= t.hi;
                tc_fence_after();
                if (leader) {
                    const uint32_t at = st * (kStageBytes >> 4);
#pragma unroll
                    for (int q = 0; q < kK / 16; ++q)   // 16 rows of 128 bytes
                        if (q < steps)
                            pair_umma_f16(tmem + ab * kN, a0 + at + q * 128, b0 + at + q * 128,
                                          a.idesc, in_chunk + q);
                    pair_commit(&empty[st], lead);
                    if (done) pair_commit(&acc_full[ab], lead);
                }
                __syncwarp();
                ++in_chunk;
                if (done) {
                    in_chunk = 0;
                    ab ^= 1u;
                    acc_phase ^= ab ^ 1u;
                }
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) {
            fail();
            if (leader) pair_commit(&drain, lead);
            mbar_wait_for(&drain, 0u, kWait);
        }
        __syncwarp();
    } else if (warp == 2) {
        // --- zeros behind an expert's last row, up to the next multiple of 16
        uint32_t st = 0, phases = 0;   // the last stage of the tiles so far; a bit a barrier
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            const Tile t = tile_at(tile);
            st = (st + static_cast<uint32_t>((t.hi - t.lo + kK - 1) / kK)) % kStages;
            if ((t.m & 15) == 0 || t.hi < t.m || t.hi <= t.lo) continue;
            const uint32_t last = (st + kStages - 1) % kStages;
            ok = __all_sync(0xFFFFFFFFu,
                            mbar_wait_for(&last_full[last], (phases >> last) & 1u, kWait));
            if (!ok) break;
            phases ^= 1u << last;
            const int n = (16 - (t.m & 15)) * 8;   // 16-byte units a box
            uint8_t* from = smem + last * kStageBytes + (t.m & (kK - 1)) * 128;
            for (int u = lane; u < n; u += 32)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    *reinterpret_cast<uint4*>(from + b * kBoxBytes + u * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) pair_arrive_release(leader_addr(&full[last], lead));
            ok = !*abort_flag;
        }
        if (!ok) fail();
        __syncwarp();
    } else if (warp >= kEpiWarp) {
        // --- sums: lane = row, 128 columns a warp
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int quarter = warp & 3, half = (warp - kEpiWarp) >> 2;
        const uint32_t src = tmem + half * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t done = leader_addr(&acc_empty[0], lead);
        uint8_t* patch = smem + kStages * kStageBytes + (warp - kEpiWarp) * kPatch;
        uint32_t ab = 0, acc_phase = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            const Tile t = tile_at(tile);
            float2 sum[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = make_float2(0.0f, 0.0f);
            for (int i = t.lo; i < t.hi; i += kK * kChunk) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_for(&acc_full[ab], acc_phase, kWait));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kCols; c += 64) {
                    uint32_t v[64];
                    tmem_ld<32>(src + ab * kN + c, v);
                    tmem_ld<32>(src + ab * kN + c + 32, v + 32);
                    tmem_ld_wait();
                    if (c + 64 == kCols) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) pair_arrive(done + ab * 8);
                    }
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        sum[c / 2 + q] = __fadd2_rn(sum[c / 2 + q],
                                                    make_float2(__uint_as_float(v[2 * q]),
                                                                __uint_as_float(v[2 * q + 1])));
                }
                ab ^= 1u;
                acc_phase ^= ab ^ 1u;
            }
            if (!ok) {
                fail();
                break;
            }
            if constexpr (kSplit) {
                // [row][column] partial sums of this CTA, over the ring: every copy and MMA of the
                // pair is done once its last accumulator was handed over
                float4* part = reinterpret_cast<float4*>(smem) + (quarter * 32 + lane) * (kN / 4);
#pragma unroll
                for (int c = 0; c < kCols / 4; ++c)
                    part[(half * (kCols / 4) + c) ^ lane] = make_float4(
                        sum[2 * c].x, sum[2 * c].y, sum[2 * c + 1].x, sum[2 * c + 1].y);
                continue;   // (its one tile)
            }
            // 128 bytes of the 32 rows at a time, by copies from shared memory (which cut off at
            // the matrix's edges): the warp goes on while they run (one after the other on one GPU:
            // 16 experts as above 235 us, by stores of whole lines 243, of 32 bytes of 32 rows 274;
            // top-4 of 64 experts, 2048 tokens, into bf16 249, 280 and 314)
            const int r = t.r0 + rank * kM + quarter * 32, c0 = t.c0 + half * kCols;
            constexpr int kE = 128 / sizeof(T), kUnit = 16 / sizeof(T);
#pragma unroll
            for (int c = 0; c < kCols; c += kE) {
                uint8_t* to = patch;
                if (lane == 0) bulk_wait_read<0>();   // the last copy has read it
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
                    *reinterpret_cast<uint4*>(to + lane * 128 + (q ^ (lane & 7)) * 16) = p.raw;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (c0 + c < a.cols && r < a.rows)
                        tma3d_store(&dwmap, c0 + c, r, t.e, smem_u32(to));
                    bulk_commit();
                }
            }
            ok = !*abort_flag;
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    __syncthreads();
    if (*abort_flag && tid == 0) {
        // a CTA that gave up: its copies in flight land long before this
        for (const long long t0 = clock64(); clock64() - t0 < kDrain;) __nanosleep(1000);
    }
    if constexpr (kSplit) {
        cluster.sync();   // every pair's partial sums are written
        const Tile t = tile_at(tile0);
        const int q = lead / 2, row_lo = kM * q / n_split, row_hi = kM * (q + 1) / n_split;
        for (int i = row_lo * (kN / 4) + tid; i < row_hi * (kN / 4) && !*abort_flag; i += kThreads) {
            const int row = i / (kN / 4), c4 = i % (kN / 4);
            const int at = row * (kN / 4) + (c4 ^ (row & 31));
            float4 v[kMaxSplit];   // all loads on their way before the first sum
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s)
                if (s < n_split)
                    v[s] = cluster.map_shared_rank(reinterpret_cast<const float4*>(smem),
                                                   2 * s + rank)[at];
            float f[4] = {};
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s)
                if (s < n_split) {
                    f[0] += v[s].x;
                    f[1] += v[s].y;
                    f[2] += v[s].z;
                    f[3] += v[s].w;
                }
            const int r = t.r0 + rank * kM + row, c = t.c0 + c4 * 4;
            Pack<T, 4> p;
            p.set(f);
            if (r < a.rows && c < a.cols)
                store_pack(reinterpret_cast<Pack<T, 4>*>(
                               dw + (static_cast<size_t>(t.e) * a.rows + r) * a.cols + c),
                           p);
        }
    }
    tc_fence_before();
    cluster.sync();   // neither leaves while the other still multiplies from its memory
    if (warp == 1) {
        tc_fence_after();
        pair_tmem_give(tmem, 2 * kN);
    }
}

// Rows of 16-bit elements, copies of 64 x 64.
bool row_map(CUtensorMap* map, const void* base, int width, int n_rows, int type) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(n_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * 2};
    const cuuint32_t box[2] = {kBox, kK};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map,
              type == kTypeBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dW, copies of 128 bytes x 32 rows.
template <typename T>
bool out_map(CUtensorMap* map, void* dw, const WArgs& a) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(a.cols) * sizeof(T);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.cols), static_cast<cuuint64_t>(a.rows),
                                static_cast<cuuint64_t>(a.n_experts)};
    const cuuint64_t strides[2] = {row, row * a.rows};
    const cuuint32_t box[3] = {128 / sizeof(T), 32, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map,
              sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              dw, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmem = kStages * kStageBytes + kEpiWarps * kPatch + 1024;

template <typename T, bool kSplit>
cudaError_t allow_smem() {
    static PerDevice memo;
    return static_cast<cudaError_t>(memo.get([] {
        return static_cast<int>(cudaFuncSetAttribute(k_grad_w<T, kSplit>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(kSmem)));
    }));
}

// Clusters of 2 * split CTAs that the device holds at once (its SMs come in groups that a cluster
// does not cross), 0 where it cannot say.
template <typename T>
int clusters_at_once(int split) {
    static PerDevice memo[2];
    return memo[split / 4].get([&] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2u * static_cast<unsigned>(split));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2u * static_cast<unsigned>(split);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (allow_smem<T, true>() != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, k_grad_w<T, true>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        return n;
    });
}

template <typename T, bool kSplit>
cudaError_t launch_t(const CUtensorMap& dymap, const CUtensorMap& xmap, const WArgs& a, int split,
                     void* dw, cudaStream_t s) {
    const cudaError_t attr_err = allow_smem<T, kSplit>();
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap dwmap;
    if (!out_map<T>(&dwmap, dw, a)) return cudaErrorNotSupported;
    const int tiles = a.n_rt * a.n_ct * a.n_experts;
    const unsigned ctas = 2u * static_cast<unsigned>(split);
    return launch_after(k_grad_w<T, kSplit>,
                        dim3(ctas * static_cast<unsigned>(std::min(tiles, sm_count() / 2))),
                        kThreads, kSmem, s, ctas, dymap, xmap, dwmap, a, static_cast<T*>(dw));
}

}  // namespace

cudaError_t launch_mm_grad_w(const void* dy, const void* x, int type, int n_experts, int rows,
                             int cols, int n_rows, const int32_t* offsets, void* dw, int dw_type,
                             cudaStream_t s) {
    WArgs a{};
    a.offsets = offsets;
    a.n_experts = n_experts;
    a.rows = rows;
    a.cols = cols;
    a.n_rows = n_rows;
    a.n_rt = (rows + 2 * kM - 1) / (2 * kM);
    a.n_ct = (cols + kN - 1) / kN;
    // D = F32, A and B both of `type` and contiguous along M and N
    const uint32_t t = type == kTypeBF16 ? 1u : 0u;
    a.idesc = (1u << 4) | (t << 7) | (t << 10) | (1u << 15) | (1u << 16) |
              (static_cast<uint32_t>(kN >> 3) << 17) | (static_cast<uint32_t>(2 * kM >> 4) << 24);
    CUtensorMap dymap, xmap;
    if (!row_map(&dymap, dy, rows, n_rows, type) || !row_map(&xmap, x, cols, n_rows, type))
        return cudaErrorNotSupported;
    const long tiles = static_cast<long>(a.n_rt) * a.n_ct * n_experts;
    auto go = [&](auto one) {
        using T = decltype(one);
        // slices of a tile's rows where their clusters are all there at once, and the mean
        // expert has four stages a slice
        int split = 1;
        while (split < kMaxSplit && n_rows / n_experts >= split * 2 * 4 * kK &&
               tiles <= clusters_at_once<T>(split * 2))
            split *= 2;
        return split > 1 ? launch_t<T, true>(dymap, xmap, a, split, dw, s)
                         : launch_t<T, false>(dymap, xmap, a, 1, dw, s);
    };
    return dw_type == kTypeF32 ? go(float{}) : go(__nv_bfloat16{});
}

cudaError_t read_fault_grad_w(int* value, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_grad_w, sizeof(int));
    if (e != cudaSuccess || !reset) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_fault_grad_w, &zero, sizeof(int));
}

}  // namespace mxk
