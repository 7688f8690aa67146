// grad_w.cu -- the gradient of a product by its matrices (include/f8.h mxfp4_mm_grad_w,
// mxfp4_moe_mm_grad_w; tcgen05 kind::f16, sm_103a).
//
// dW_e[r][c] = sum_{i in e} dY[i][r] X[i][c]: both operands lie with the sum's side (the rows i)
// outermost, so each copy brings 64 rows of 64 elements (128 bytes) as they are, and the
// descriptors say that the M and N sides are contiguous: nothing is transposed.
//
// A tile is 128 rows by 256 columns of a dW_e, its sum the rows of expert e, 64 a ring stage.
// Rows past the expert's end (another expert's, or none) are no part of it: the MMAs stop at the
// last 16 rows that hold one of its own, and what follows in those 16 is overwritten by zeros in
// shared memory (in both operands: zero times whatever lies there may be NaN).
//
// Warps: copies, MMAs (and those zeros), eight that store the accumulators (two, in turn).
// Persistent: CTA c takes tiles c, c + grid, ...
//
// Every wait is bounded; a CTA that gives up sets the fault word, lets its copies land, frees its
// tensor memory and returns.
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

constexpr int kM = 128, kN = 256, kK = 64;    // rows and columns of a tile, rows of a stage
constexpr int kBox = 64;                      // elements of a copied row (128 bytes)
constexpr uint32_t kBoxBytes = kBox * kK * 2;
constexpr uint32_t kABytes = kM / kBox * kBoxBytes, kStageBytes = kABytes + kN / kBox * kBoxBytes;
constexpr int kStages = 4;
constexpr int kThreads = 320, kEpiWarp = 2, kEpiWarps = 8;
constexpr int kMaxExperts = 1024;
constexpr long long kWait = 1ll << 32, kDrain = 1ll << 24;   // SM cycles: about 2 s and 8 ms

__device__ int g_fault_grad_w;

struct WArgs {
    const int32_t* offsets;   // nullptr: one matrix
    int n_experts, rows, cols, n_rows;
    int n_rt, n_ct;           // tiles down and across a matrix
    uint32_t idesc;
    int wide;                 // rows of dW are 32-byte aligned
};

__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// n elements (a multiple of 8) of the 32 in v.
template <typename T, int kN>
__device__ __forceinline__ void store_row(T* dst, const uint32_t (&v)[32], int n) {
#pragma unroll
    for (int q = 0; q < 32 / kN; ++q) {
        float f[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] = __uint_as_float(v[q * kN + i]);
        Pack<T, kN> p;
        p.set(f);
        if (q * kN < n) store_pack(reinterpret_cast<Pack<T, kN>*>(dst) + q, p);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    k_grad_w(const __grid_constant__ CUtensorMap dymap, const __grid_constant__ CUtensorMap xmap,
             const WArgs a, T* __restrict__ dw) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    __shared__ int32_t off[kMaxExperts + 1];
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 1) tmem_take(&tmem_base, 2 * kN);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kEpiWarps);
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_mbar_init();
    }
    if (tid == 32 * 2) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&dymap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();   // (this CTA has its tensor memory)
    pdl_wait();
    for (int e = tid; e <= a.n_experts; e += kThreads)
        off[e] = a.offsets == nullptr ? e * a.n_rows
                                      : min(max(ld_dep(a.offsets + e), 0), a.n_rows);
    __syncthreads();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);

    struct Tile {
        int e, r0, c0, i0, m;
    };
    const int per_e = a.n_rt * a.n_ct, n_tiles = per_e * a.n_experts;
    const int tile0 = static_cast<int>(blockIdx.x), tile_step = static_cast<int>(gridDim.x);
    auto tile_at = [&](int tile) {
        Tile t;
        t.e = tile / per_e;
        const int local = tile - t.e * per_e, rt = local / a.n_ct;
        t.r0 = rt * kM;
        t.c0 = (local - rt * a.n_ct) * kN;
        t.i0 = off[t.e];
        t.m = max(off[t.e + 1] - t.i0, 0);
        return t;
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_fault_grad_w, 1);
    };

    if (warp == 0) {
        // --- copies
        const bool leader = elect_one();
        const uint64_t policy = l2_evict_normal();
        const uint32_t ring = smem_u32(smem);
        uint32_t st = 0, phase = 1;   // the first round of the ring passes at once
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            const Tile t = tile_at(tile);
            for (int i = 0; i < t.m; i += kK) {
                ok = mbar_wait_for(&empty[st], phase, kWait);
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&full[st], kStageBytes);
                    const uint32_t dst = ring + st * kStageBytes;
#pragma unroll
                    for (int b = 0; b < kM / kBox; ++b)
                        tma2d(dst + b * kBoxBytes, &dymap, t.r0 + b * kBox, t.i0 + i, &full[st],
                              policy);
#pragma unroll
                    for (int b = 0; b < kN / kBox; ++b)
                        tma2d(dst + kABytes + b * kBoxBytes, &xmap, t.c0 + b * kBox, t.i0 + i,
                              &full[st], policy);
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
        __syncwarp();
    } else if (warp == 1) {
        // --- MMAs
        const bool leader = elect_one();
        const uint32_t ring = smem_u32(smem);
        const uint64_t a0 = operand_desc_mn(ring, kBoxBytes);
        const uint64_t b0 = operand_desc_mn(ring + kABytes, kBoxBytes);
        uint32_t st = 0, phase = 0;
        int j = 0;
        bool ok = true;
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            const Tile t = tile_at(tile);
            if (t.m == 0) continue;
            const int ab = j & 1;
            ok = mbar_wait_for(&acc_empty[ab], (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u, kWait);
            ++j;
            for (int i = 0; i < t.m && ok; i += kK) {
                ok = mbar_wait_for(&full[st], phase, kWait);
                if (!ok) break;
                const int steps = min(kK, t.m - i + 15) >> 4;   // of 16 rows
                if (t.m - i < kK && (t.m & 15) != 0) {
                    // zeros behind the expert's last row, up to the next multiple of 16
                    const int n = (16 - (t.m & 15)) * 8;   // 16-byte units a box
                    uint8_t* from = smem + st * kStageBytes + (t.m & (kK - 1)) * 128;
                    for (int u = lane; u < n; u += 32)
#pragma unroll
                        for (int b = 0; b < (kM + kN) / kBox; ++b)
                            *reinterpret_cast<uint4*>(from + b * kBoxBytes + u * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (leader) {
                    const uint32_t at = st * (kStageBytes >> 4);
#pragma unroll
                    for (int q = 0; q < kK / 16; ++q)   // 16 rows of 128 bytes
                        if (q < steps)
                            umma_f16(tmem + ab * kN, a0 + at + q * 128, b0 + at + q * 128,
                                     a.idesc, i + q);
                    umma_commit(&empty[st]);
                    if (i + kK >= t.m) umma_commit(&acc_full[ab]);
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1u;
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
    } else {
        // --- accumulators to memory: lane = row, 128 columns a warp
        const int quarter = warp & 3, half = (warp - kEpiWarp) >> 2;
        int j = 0;
        for (int tile = tile0; tile < n_tiles && !*abort_flag; tile += tile_step) {
            const Tile t = tile_at(tile);
            const int ab = j & 1;
            if (t.m > 0) {
                if (!__all_sync(0xFFFFFFFFu,
                                mbar_wait_for(&acc_full[ab], static_cast<uint32_t>(j >> 1) & 1u,
                                              kWait))) {
                    fail();
                    break;
                }
                ++j;
                tc_fence_after();
            }
            const int r = t.r0 + quarter * 32 + lane, c0 = t.c0 + half * (kN / 2);
            T* dst = dw + (static_cast<size_t>(t.e) * a.rows + r) * a.cols + c0;
#pragma unroll 1
            for (int c = 0; c < kN / 2 && c0 + c < a.cols; c += 32) {
                uint32_t v[32];
                if (t.m > 0) {
                    tmem_ld<32>(tmem + ab * kN + half * (kN / 2) + c +
                                    (static_cast<uint32_t>(quarter * 32) << 16),
                                v);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                }
                if (r < a.rows) {
                    if (a.wide) store_row<T, 32 / sizeof(T)>(dst + c, v, a.cols - c0 - c);
                    else store_row<T, 16 / sizeof(T)>(dst + c, v, a.cols - c0 - c);
                }
            }
            if (t.m > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_m(&acc_empty[ab]);
            }
        }
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
        tmem_give(tmem, 2 * kN);
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

template <typename T>
cudaError_t launch_t(const CUtensorMap& dymap, const CUtensorMap& xmap, WArgs a, void* dw,
                     cudaStream_t s) {
    constexpr size_t kSmem = kStages * kStageBytes + 1024;
    static PerDevice memo;
    const cudaError_t attr_err = static_cast<cudaError_t>(memo.get([] {
        return static_cast<int>(cudaFuncSetAttribute(
            k_grad_w<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)));
    }));
    if (attr_err != cudaSuccess) return attr_err;
    a.wide = (reinterpret_cast<uintptr_t>(dw) | static_cast<uintptr_t>(a.cols) * sizeof(T)) % 32 == 0;
    const int tiles = a.n_rt * a.n_ct * a.n_experts;
    return launch_after(k_grad_w<T>, dim3(static_cast<unsigned>(std::min(tiles, sm_count()))),
                        kThreads, kSmem, s, 1, dymap, xmap, a, static_cast<T*>(dw));
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
    a.n_rt = (rows + kM - 1) / kM;
    a.n_ct = (cols + kN - 1) / kN;
    // D = F32, A and B both of `type` and contiguous along M and N
    const uint32_t t = type == kTypeBF16 ? 1u : 0u;
    a.idesc = (1u << 4) | (t << 7) | (t << 10) | (1u << 15) | (1u << 16) |
              (static_cast<uint32_t>(kN >> 3) << 17) | (static_cast<uint32_t>(kM >> 4) << 24);
    CUtensorMap dymap, xmap;
    if (!row_map(&dymap, dy, rows, n_rows, type) || !row_map(&xmap, x, cols, n_rows, type))
        return cudaErrorNotSupported;
    return dw_type == kTypeF32 ? launch_t<float>(dymap, xmap, a, dw, s)
                               : launch_t<__nv_bfloat16>(dymap, xmap, a, dw, s);
}

cudaError_t read_fault_grad_w(int* value, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_grad_w, sizeof(int));
    if (e != cudaSuccess || !reset) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_fault_grad_w, &zero, sizeof(int));
}

}  // namespace mxk
