// mx_mm.cu -- products of two MXFP4 matrices on the block-scaled 4-bit tensor cores
// (include/mx4.h mxfp4_mm_mx, mxfp4_moe_mm_mx; tcgen05 kind::mxf4, sm_103a).
//
// Y[i][r] = sum_g 2^(kw-127) 2^(kx-127) sum_{c in g} e2m1(W[r][c]) e2m1(X[i][c]): the
// tensor core multiplies the codes, applies both groups' scale bytes and adds in FP32.
// The weights are the MMA's 128-row operand A and the tokens its N columns, so one
// kernel serves one token (N = 16) and a prompt (N up to 208), and a warp's 32 TMEM
// lanes are 32 consecutive outputs of one token: stores are coalesced without a
// transpose.
//
// Code planes arrive by TMA as they lie in memory (128-byte swizzled rows of 256
// elements: one ring stage, four MMAs of K = 64).  Scale bytes lie row-major with a
// row stride of cols/32 bytes, which no copy engine can turn into the layout the
// tensor core wants (32 lanes x 16 bytes: byte 4j + b of lane l is group b of row l +
// 32j), so warps of their own take them 32 bytes a row (four stages) and store them in
// that layout, and tcgen05.cp moves them to tensor memory ahead of each stage's MMAs.  A
// slot of four stages is handed over at a time: the proxy fence and the barriers cost
// several hundred cycles, more than a stage has when few tokens stream through.
//
// Warps have roles: copies, MMAs, scales, and the reading and storing of finished
// accumulators (two, in turn).  Persistent: CTA c takes tiles c, c + grid, ...  With few
// tokens the tiles are too few to fill the SMs; then a cluster of CTAs shares a tile, each
// a slice of K, and adds the partial sums through distributed shared memory in rank order.
//
// What bounds it: many experts with few rows each, HBM (64 experts 2880x2880, 32 tokens,
// top-4: 38 us, 6.5 TB/s).  Elsewhere the chain of barriers between the roles: without
// copies, MMAs, scales and stores it took 420 cycles a stage of 256 columns (one barrier
// for two stages now, where they fit), and a stage's copies, its MMAs (257 cycles at 128
// tokens) and the last tile's stores are hidden behind it only in part.  One token
// 14336x4096 8.4 us (13 matrices in turn, 407 MB: every weight from HBM; 7.7 where some lie in
// L2); 2048 tokens 4096x4096 21.9 us, 3.1 PFLOP/s; 4096 tokens 37.4 us, 3.7; 2048 tokens, top-4
// of 64 experts 2880x2880, 67.0 us.
//
// Every wait is bounded; a CTA that gives up sets the fault word, lets its copies land,
// frees its tensor memory and returns.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mx4_kernels.h"
#include "pdl.cuh"

namespace mxk {
namespace {

namespace cg = cooperative_groups;

constexpr int kM = 128;                     // weight rows per tile
constexpr int kK = 256;                     // elements per ring stage: 128 code bytes a row
constexpr int kGroupsStage = kK / kGroup;   // 8 scale bytes a row
// Warps.  0, and unsplit 5 and 7: copies; 1: MMAs; 2: W's scales; 3 and 4: X's scales (128
// tokens each; 4 unused when split or with one block); 6 (unsplit): scales to tensor memory;
// then the epilogue.  A role is one warp's chain of waits and issues, 400 to 700 cycles a
// stage whatever it does: a copy holds its registers for some 200 cycles after it is issued,
// a poll answers after 100.  One copy warp for both operands needs 700, so three take the
// stages in turn.  The epilogue has each TMEM lane quarter once, or twice: a warp's stores
// wait for each other (33 MB of FP32 results, 128 bytes a store: 18.5 us by four warps an SM,
// 12.4 us by eight).
template <bool kSplit>
struct Roles {
    static constexpr int kToTmem = 6, kCopiers = kSplit ? 1 : 3;
    static constexpr int kEpi = kSplit ? 4 : 8, kEpiWarps = kSplit ? 4 : 8;
    static constexpr int kThreads = 32 * (kEpi + kEpiWarps);
};
constexpr uint32_t kABytes = kM * kK / 2;
constexpr uint32_t kSfChunk = 512;          // scale bytes of 128 rows x 4 groups
constexpr int kMaxStages = 10;
constexpr int kMaxSplit = 8;                // CTAs of a cluster sharing a tile
constexpr int kTileTable = 64;              // this CTA's first tiles, worked out at the start
constexpr int kMaxTokens = 208;             // two accumulators and the scales in 512 columns
constexpr long long kWaitMx = 1ll << 32, kDrainMx = 1ll << 24;   // SM cycles: about 2 s and 8 ms

__device__ int g_fault_mx;

// One launch's shape.  tn: most tokens of a tile (a multiple of 16); box: token rows of
// one TMA copy (divides tn).
struct MxArgs {
    const uint8_t* w_scales;      // scale plane of expert 0
    size_t bank_stride;
    const uint8_t* x_scales;
    const int32_t* offsets;       // nullptr: one matrix
    int n_experts, rows, gpr, n_rows;
    int n_steps;                  // ring stages per tile
    int tn, box, n_stages;
    uint32_t stage_bytes, tmem_cols;
    int n_sc;                     // 2 tile buffers of scale rows, or 0: loaded from global memory
    uint32_t sc_w, sc_bytes;      // bytes of W's rows in a buffer, of a buffer
    int n_rt, n_tt;               // row tiles; token tiles (one matrix)
};

struct alignas(16) Tile {
    int e, r0, t0, t1;
};

__device__ __forceinline__ void tma3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                      uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                      uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint64_t l2_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Shared-memory matrix descriptors: operands K-major with 128-byte swizzle (8-row groups
// 1024 bytes apart); scale chunks unswizzled 8 x 16-byte core matrices 128 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// Instruction descriptor of kind::mxf4: A = B = E2M1 (1), K-major, UE8M0 scales, M = 128,
// N; sf: which half of a 4-byte scale cell (0 or 2) holds the two groups of this K = 64.
__device__ __forceinline__ uint32_t idesc_mxf4(int n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (1u << 23) | (1u << 27) | (sf << 29);
}

__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
        "[%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

// 512 bytes of scales -> 4 TMEM columns, the 32 lanes repeated in every lane quarter.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
}

// A stage's scales: two chunks of W, then two times NB of X.
template <int NB>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
#pragma unroll
    for (uint32_t i = 0; i < 2u * (1 + NB); ++i)
        cp_scales(taddr + 4u * i, desc + i * (kSfChunk >> 4));
}

__device__ __forceinline__ void umma_commit_mx(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void fence_after_mx() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before_mx() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// One poll that does not suspend.  Its answer takes about a hundred cycles: a role asks
// about its next stage before it issues the current one.
__device__ __forceinline__ bool mbar_ready(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait for the phase with the given parity, for at most `cycles` SM cycles (a poll may
// itself be suspended for a while, so polls are not counted).
__device__ __forceinline__ bool mbar_wait_for(uint64_t* bar, uint32_t parity, long long cycles) {
    if (mbar_wait(bar, parity, 1)) return true;
    const long long t0 = clock64();
    do {
        if (mbar_wait(bar, parity, 1)) return true;
    } while (clock64() - t0 < cycles);
    return false;
}

// 16 accumulator columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void sts128_mx(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// The scale bytes of kAhead stages (8 groups each, from g0) of rows row0 + lane + 32 j, j < 4, of
// a plane with gpr bytes a row; bytes past a row's end are 0 (2^-127: their codes are 0),
// rows at or past row_end arbitrary (their results are not stored).  Rows that are not
// 16-byte aligned: aligned words shifted together, none of them past the row's last byte's
// word.
template <int kAhead>
struct Scales {
    uint32_t w[4][2 * kAhead];
};
// kShared: the rows lie in shared memory (bulk-copied, row 0 at `plane`).
template <bool kShared, typename V>
__device__ __forceinline__ V load_word(const V* p) {
    if constexpr (kShared) return *p;
    else return ld_dep(p);
}
template <bool kShared, int kAhead>
__device__ __forceinline__ void load_scales(Scales<kAhead>& s, const uint8_t* plane, int gpr,
                                            int g0, int row0, int row_end, int lane) {
    constexpr int kWords = 2 * kAhead;
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(plane));
    const bool wide = ((gpr | g0 | base) & 15) == 0;
    const int nv = gpr - g0;   // bytes of the row from g0 on
    const uint8_t* at = plane + static_cast<size_t>(row0 + lane) * gpr + g0;
    const size_t next = static_cast<size_t>(32) * gpr;
    if (wide) {
#pragma unroll
        for (int j = 0; j < 4; ++j, at += next) {
#pragma unroll
            for (int q = 0; q < kWords / 4; ++q) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (row0 + lane + 32 * j < row_end && 16 * q < nv)
                    v = load_word<kShared>(reinterpret_cast<const uint4*>(at) + q);
                s.w[j][4 * q] = v.x;
                s.w[j][4 * q + 1] = v.y;
                s.w[j][4 * q + 2] = v.z;
                s.w[j][4 * q + 3] = v.w;
            }
        }
    } else if (nv >= 4 * kWords + 4) {   // all words count, and the one a shift draws in
#pragma unroll
        for (int j = 0; j < 4; ++j, at += next) {
            if (row0 + 32 * j >= row_end) {   // the same for the whole warp
#pragma unroll
                for (int i = 0; i < kWords; ++i) s.w[j][i] = 0u;
                continue;
            }
            // rows past the end repeat row row0: their results are not stored
            const uint8_t* p8 = row0 + lane + 32 * j < row_end
                                    ? at
                                    : plane + static_cast<size_t>(row0) * gpr + g0;
            const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p8)) & 3u;
            const uint32_t* p = reinterpret_cast<const uint32_t*>(p8 - skew);
            uint32_t raw[kWords + 1];
#pragma unroll
            for (int i = 0; i <= kWords; ++i) raw[i] = load_word<kShared>(p + i);
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                s.w[j][i] = __funnelshift_r(raw[i], raw[i + 1], 8u * skew);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j, at += next) {
            const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 3);
            const uint32_t* p = reinterpret_cast<const uint32_t*>(at - skew);
            const bool in = row0 + lane + 32 * j < row_end;
            uint32_t raw[kWords + 1];
#pragma unroll
            for (int i = 0; i <= kWords; ++i)
                raw[i] = in && 4 * i < nv + skew ? load_word<kShared>(p + i) : 0u;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int left = nv - 4 * i;   // bytes of this word that count
                const uint32_t keep =
                    left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                s.w[j][i] = __funnelshift_r(raw[i], raw[i + 1], 8u * skew) & keep;
            }
        }
    }
}

// Both chunks (groups 0..3 and 4..7) of stage q's 128 rows; chunk 1 is `second` bytes on.
template <int kAhead>
__device__ __forceinline__ void store_scales(const Scales<kAhead>& s, int q, uint32_t saddr,
                                             uint32_t second, int lane) {
    sts128_mx(saddr + lane * 16, s.w[0][2 * q], s.w[1][2 * q], s.w[2][2 * q], s.w[3][2 * q]);
    sts128_mx(saddr + second + lane * 16, s.w[0][2 * q + 1], s.w[1][2 * q + 1],
              s.w[2][2 * q + 1], s.w[3][2 * q + 1]);
}

// 32 outputs (TMEM lanes; `valid` of them exist) of every other 16 of n tokens (columns of
// `src`, from c0) to y, tokens `pitch` elements apart.  Where the pitch is a multiple of four,
// lanes trade so that each holds four consecutive outputs of four tokens, and a store is four
// tokens' 64 (BF16) or 128 bytes: a store costs about the same whatever a lane gives it (FP32,
// 3000 tokens 8192x1024: 26.0 us, with one token's 128 bytes a store 35.9).
template <typename T>
__device__ __forceinline__ void store_tile(T* y, int pitch, int valid, int c0, int n,
                                           uint32_t src, int lane) {
    if (valid <= 0) return;
    const bool quads = (pitch & 3) == 0 && valid == 32;
    for (int c = c0; c < n; c += 32) {
        uint32_t v[16];
        tmem_ld16(src + c, v);
        if (quads && sizeof(T) == 4) {
            // lane pair (l, l ^ 1): both rows of columns 0..7 (even) or 8..15
            float2 a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t give = (lane & 1) ? v[i] : v[i + 8];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
                a[i].x = __uint_as_float((lane & 1) ? got : v[i]);
                a[i].y = __uint_as_float((lane & 1) ? v[i + 8] : got);
            }
            // lane pair (l, l ^ 2): rows 0..3 of the quad for half of the eight columns
            const int col0 = (lane & 1) * 8 + ((lane & 2) ? 4 : 0);
            T* dst = y + static_cast<size_t>(c + col0) * pitch + (lane & ~3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 give = (lane & 2) ? a[i] : a[i + 4];
                float2 got;
                got.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, 2);
                got.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, 2);
                const float2 lo = (lane & 2) ? got : a[i], hi = (lane & 2) ? a[i + 4] : got;
                if (c + col0 + i < n)
                    *reinterpret_cast<float4*>(dst + static_cast<size_t>(i) * pitch) =
                        make_float4(lo.x, lo.y, hi.x, hi.y);
            }
        } else if (quads) {
            // columns as BF16 pairs of this lane's row: u[i] = (column i, column i + 8)
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // lane pair (l, l ^ 1): the even lane ends with both rows of columns 0..7,
                // the odd one with both rows of columns 8..15
                const uint32_t give = (lane & 1) ? v[i] : v[i + 8];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
                const float lo = __uint_as_float((lane & 1) ? got : v[i]);
                const float hi = __uint_as_float((lane & 1) ? v[i + 8] : got);
                const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
                u[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
            // lane pair (l, l ^ 2): rows 0..3 of the quad for half of the eight columns
            const int col0 = (lane & 1) * 8 + ((lane & 2) ? 4 : 0);
            T* dst = y + static_cast<size_t>(c + col0) * pitch + (lane & ~3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t give = (lane & 2) ? u[i] : u[i + 4];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, 2);
                if (c + col0 + i < n)
                    *reinterpret_cast<uint2*>(dst + static_cast<size_t>(i) * pitch) =
                        (lane & 2) ? make_uint2(got, u[i + 4]) : make_uint2(u[i], got);
            }
        } else if (lane < valid) {
            T* dst = y + static_cast<size_t>(c) * pitch + lane;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < n)
                    dst[static_cast<size_t>(i) * pitch] = from_f32<T>(__uint_as_float(v[i]));
        }
    }
}

// NB: 128-token blocks of a stage's scales.  Split tiles (few tokens) leave registers for
// three CTAs on an SM.
template <typename T, bool kSplit, int NB, int kP>
__global__ void __launch_bounds__(Roles<kSplit>::kThreads, kSplit ? 3 : 1)
    k_mx_mm(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
            const MxArgs a, T* __restrict__ Y) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // (one barrier of each for a unit of kP stages)
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint64_t sc_full[2], sc_empty[2], sf_full[2], sf_empty[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word, n_tiles_sh;
    __shared__ Tile table[kTileTable];
    volatile int* abort_flag = &abort_word;
    // after the ring: two slots of scales in the tensor core's layout, each for kAhead
    // stages, the buffers of scale rows, then the experts' row offsets and first
    // tiles (experts) or the partial sums of a split tile
    constexpr int kAhead = kSplit ? 2 : 4;
    constexpr uint32_t kSfStage = 2u * kSfChunk * (1 + NB), kSfSlot = kAhead * kSfStage;
    uint8_t* sf_buf = smem + static_cast<size_t>(a.n_stages) * a.stage_bytes;
    uint8_t* sc_buf = sf_buf + 2u * kSfSlot;
    uint8_t* after = sc_buf + static_cast<size_t>(a.n_sc) * a.sc_bytes;
    int32_t* off = reinterpret_cast<int32_t*>(after);
    int32_t* first = off + a.n_experts + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kSplit ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int n_rank = kSplit ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;

    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base)),
                     "r"(a.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < a.n_stages / kP; ++i) {
            mbar_init(&full[i], kSplit ? 1 : 2);   // the copies, and scales in tensor memory
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], Roles<kSplit>::kEpiWarps);
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], 1 + NB);   // W's and X's scale warps
            mbar_init(&sf_full[i], 1 + NB);
            mbar_init(&sf_empty[i], 1);
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
    fence_before_mx();
    __syncthreads();
    fence_after_mx();
    // the next launch may be placed now that this CTA has its tensor memory (a CTA of the
    // next one that waits for columns then waits for CTAs that need nothing more)
    pdl_trigger();
    if (a.offsets != nullptr) {
        pdl_wait();
        for (int e = tid; e <= a.n_experts; e += Roles<kSplit>::kThreads)
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
    // (split) slices of whole pairs of stages, so that 16-byte scale loads stay aligned
    const int pairs = (a.n_steps + 1) / 2;
    auto slice = [&](int r) {
        return 2 * static_cast<int>(static_cast<long long>(pairs) * r / n_rank);
    };
    const int s_lo = kSplit ? slice(rank) : 0;
    const int s_hi = kSplit ? min(a.n_steps, slice(rank + 1)) : a.n_steps;
    // a cluster's tiles (split: one)
    const int tile0 = static_cast<int>(blockIdx.x) / n_rank;
    const int tile_step = kSplit ? n_tiles : static_cast<int>(gridDim.x) / n_rank;
    const int tile_units = (s_hi - s_lo + kP - 1) / kP;
    const uint32_t n_units = static_cast<uint32_t>(a.n_stages / kP);   // of the ring
    constexpr int kAcc = kSplit ? 1 : 2;   // accumulators, of tn columns each
    const uint32_t sf_cols = tmem + kAcc * a.tn;
    constexpr uint32_t sf_stage = 8u + 8u * NB;   // TMEM columns of a stage's scales

    // A tile's token tiles come first, so that the weights of a row tile are read again
    // from L2; an expert's rows are cut into equal tiles of a multiple of 16.
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
    // Finding a tile takes over a thousand cycles (a search, divisions), and every role needs
    // it: the CTA's first tiles are found once, by all threads together.
    if (tid < kTileTable && tile0 + tid * tile_step < n_tiles)
        table[tid] = locate(tile0 + tid * tile_step);
    __syncthreads();
    if (a.offsets == nullptr) pdl_wait();   // nothing in memory was needed so far
    auto tile_at = [&](int tile, int j) { return j < kTileTable ? table[j] : locate(tile); };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_fault_mx, 1);
    };
    if (warp == 0 || (!kSplit && (warp == 5 || warp == 7))) {
        // --- copies (the whole warp walks, one elected lane issues: as for the MMAs)
        const int turn = warp == 0 ? 0 : warp == 5 ? 1 : 2;
        constexpr int kTurns = Roles<kSplit>::kCopiers;
        const bool leader = elect_one();
        const uint64_t keep = l2_evict_last();
        // Experts' weights pass through once when few tokens are with each; more tokens read a
        // row tile again (2048 tokens, top-4 of 64 experts 2880x2880: 68.7 us, evicted first
        // 73.2).  One matrix may still be there at its next use.
        const uint64_t w_policy = a.offsets != nullptr && a.tn <= 32 ? l2_evict_first()
                                  : kSplit || a.offsets != nullptr   ? l2_evict_normal()
                                                                     : keep;
        const uint32_t ring = smem_u32(smem);
        const uint32_t box_bytes = static_cast<uint32_t>(a.box) * 128u;
        // the ring position of this warp's next unit; phase of the empty barriers: the first
        // round passes at once
        uint32_t un = 0, phase = 1;
        auto advance = [&](uint32_t by) {
            for (un += by; un >= n_units; un -= n_units) phase ^= 1u;
        };
        advance(turn);
        int j = 0, sc_issued = 0, u = turn;
        bool ok = true, ready = false;
        // a tile's scale rows, contiguous in both planes, one tile ahead of its codes
        auto copy_scales = [&](const Tile& t) {
            const int b = sc_issued % 2;
            if (!mbar_wait_for(&sc_empty[b], (static_cast<uint32_t>(sc_issued / 2) & 1u) ^ 1u,
                               kWaitMx))
                return false;
            ++sc_issued;
            uint8_t* dst = sc_buf + static_cast<size_t>(b) * a.sc_bytes;
            const size_t w_at = static_cast<size_t>(t.r0) * a.gpr;   // a multiple of 16
            const size_t x_at = static_cast<size_t>(t.t0) * a.gpr;
            const uint32_t skew = static_cast<uint32_t>(x_at) & 15u;
            const uint32_t wb =
                (static_cast<uint32_t>(min(kM, a.rows - t.r0) * a.gpr) + 15u) & ~15u;
            const uint32_t xb = (skew + static_cast<uint32_t>((t.t1 - t.t0) * a.gpr) + 15u) & ~15u;
            if (leader) {
                mbar_arrive_expect_tx(&sc_full[b], wb + xb);
                bulk_g2s(dst, a.w_scales + static_cast<size_t>(t.e) * a.bank_stride + w_at, wb,
                         &sc_full[b], w_policy);
                bulk_g2s(dst + a.sc_w, a.x_scales + (x_at - skew), xb, &sc_full[b], keep);
            }
            __syncwarp();
            return true;
        };
        const bool scales = a.n_sc > 0 && turn == 0;
        if (scales && tile0 < n_tiles) ok = copy_scales(tile_at(tile0, 0));
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int n_box = (t.t1 - t.t0 + a.box - 1) / a.box;
            const uint32_t bytes = kABytes + static_cast<uint32_t>(n_box) * box_bytes;
            if (scales && tile + tile_step < n_tiles) {
                ok = copy_scales(tile_at(tile + tile_step, j + 1));
                if (!ok) break;
            }
            for (; u < tile_units; u += kTurns) {
                ok = ready || mbar_wait_for(&empty[un], phase, kWaitMx);
                if (!ok) break;
                const uint32_t now = un;
                advance(kTurns);
                ready = mbar_ready(&empty[un], phase);
                if (leader) {
                    const int s0 = s_lo + u * kP, n_s = min(kP, s_hi - s0);
                    mbar_arrive_expect_tx(&full[now], n_s * bytes);
#pragma unroll
                    for (int i = 0; i < kP; ++i) {
                        if (i == n_s) break;
                        const uint32_t dst = ring + (now * kP + i) * a.stage_bytes;
                        const int x = (s0 + i) * (kK / 2);
                        tma3d(dst, &wmap, x, t.r0, t.e, &full[now], w_policy);
                        for (int b = 0; b < n_box; ++b)
                            tma2d(dst + kABytes + static_cast<uint32_t>(b) * box_bytes, &xmap, x,
                                  t.t0 + b * a.box, &full[now], keep);
                    }
                }
                __syncwarp();
            }
            u -= tile_units;   // units of the next tile before this warp's turn
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
        __syncwarp();
    } else if (warp == 1) {
        // --- MMAs: the whole warp walks the stages, so that descriptors and addresses stay
        // in uniform registers (computed by one lane alone they cost several hundred cycles
        // a stage); one elected lane issues
        const bool leader = elect_one();
        const uint32_t ring = smem_u32(smem);
        const uint64_t op0 = operand_desc(ring), sf0 = scale_desc(smem_u32(sf_buf));
        const uint32_t stage16 = a.stage_bytes >> 4;   // descriptors count 16 bytes
        uint32_t un = 0, phase = 0;
        uint32_t group = 0;   // (split) kAhead stages sharing a scale slot
        int j = 0;
        bool ok = true;
        auto next_of = [&](uint32_t& unit, uint32_t& parity) {
            if (++unit == n_units) {
                unit = 0;
                parity ^= 1u;
            }
        };
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int n = __shfl_sync(0xFFFFFFFFu, (t.t1 - t.t0 + 15) & ~15, 0);
            const uint32_t id0 = idesc_mxf4(n, 0u), id2 = idesc_mxf4(n, 2u);
            const int ab = j % kAcc;
            if (j >= kAcc)
                ok = mbar_wait_for(&acc_empty[ab], static_cast<uint32_t>(j / kAcc - 1) & 1u,
                                   kWaitMx);
            fence_after_mx();
            const uint32_t d = tmem + ab * a.tn;
            // four MMAs of K = 64 a stage and the unit's release; the last stage of a row may
            // hold fewer
            auto issue = [&](int s0, uint32_t unit) {
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    const int s = s0 + i;
                    if (i > 0 && s >= s_hi) break;
                    const uint32_t stage = unit * kP + i;
                    const uint32_t sfa = sf_cols + stage * sf_stage, sfb = sfa + 8u;
                    const uint32_t sfb2 = sfb + 4u * NB;
                    const uint64_t ad = op0 + stage * stage16, bd = ad + (kABytes >> 4);
                    const int kk_end = (a.gpr - s * kGroupsStage + 1) / 2;
                    umma_mxf4(d, ad, bd, id0, sfa, sfb, s > s_lo ? 1u : 0u);
                    if (kk_end > 1) umma_mxf4(d, ad + 2, bd + 2, id2, sfa, sfb, 1u);
                    if (kk_end > 2) umma_mxf4(d, ad + 4, bd + 4, id0, sfa + 4u, sfb2, 1u);
                    if (kk_end > 3) umma_mxf4(d, ad + 6, bd + 6, id2, sfa + 4u, sfb2, 1u);
                }
                umma_commit_mx(&empty[unit]);
            };
            for (int s = s_lo; s < s_hi && ok;) {
                const uint32_t u0 = un, phase0 = phase;
                next_of(un, phase);
                if constexpr (kSplit) {
                    const uint32_t q = static_cast<uint32_t>(s - s_lo) % kAhead, slot = group & 1u;
                    if (q == 0) ok = mbar_wait_for(&sf_full[slot], (group >> 1) & 1u, kWaitMx);
                    ok = ok && mbar_wait_for(&full[u0], phase0, kWaitMx);
                    if (!ok) break;
                    fence_after_mx();
                    const bool last = q + kP == kAhead || s + kP >= s_hi;
                    if (leader) {
#pragma unroll
                        for (int i = 0; i < kP; ++i)
                            if (i == 0 || s + i < s_hi)
                                scales_to_tmem<NB>(
                                    sf_cols + (u0 * kP + i) * sf_stage,
                                    sf0 + ((slot * kSfSlot + (q + i) * kSfStage) >> 4));
                        issue(s, u0);
                        if (last) umma_commit_mx(&sf_empty[slot]);
                    }
                    __syncwarp();
                    group += last ? 1u : 0u;
                    s += kP;
                } else if constexpr (kP > 1) {
                    ok = mbar_wait_for(&full[u0], phase0, kWaitMx);
                    if (!ok) break;
                    fence_after_mx();
                    if (leader) issue(s, u0);
                    __syncwarp();
                    s += kP;
                } else {
                    // two stages at a time where the second is there too: their polls overlap
                    const uint32_t u1 = un, phase1 = phase;
                    bool both = s + 1 < s_hi;
                    const bool there = mbar_ready(&full[u1], phase1);
                    ok = mbar_wait_for(&full[u0], phase0, kWaitMx);
                    if (!ok) break;
                    both = __all_sync(0xFFFFFFFFu, both && there);
                    fence_after_mx();
                    if (both) {
                        next_of(un, phase);
                        if (leader) {
                            issue(s, u0);
                            issue(s + 1, u1);
                        }
                        s += 2;
                    } else {
                        if (leader) issue(s, u0);
                        ++s;
                    }
                    __syncwarp();
                }
            }
            if (ok && leader) umma_commit_mx(&acc_full[ab]);
            ok = ok && !*abort_flag;
        }
        if (!ok) {
            fail();
            if (leader) umma_commit_mx(&drain);
            mbar_wait_for(&drain, 0u, kWaitMx);
        }
        __syncwarp();
    } else if (!kSplit && warp == Roles<kSplit>::kToTmem) {
        // --- scales from shared to tensor memory, as far ahead as the ring goes
        const bool leader = elect_one();
        const uint64_t sf0 = scale_desc(smem_u32(sf_buf));
        uint32_t un = 0, phase = 1, group = 0;
        bool ok = true;
        auto copy = [&](uint32_t unit, uint32_t slot, int q, int n_q) {
#pragma unroll
            for (int i = 0; i < kP; ++i)
                if (i == 0 || q + i < n_q)
                    scales_to_tmem<NB>(sf_cols + (unit * kP + i) * sf_stage,
                                       sf0 + ((slot * kSfSlot + (q + i) * kSfStage) >> 4));
            umma_commit_mx(&full[unit]);
        };
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            for (int s0 = s_lo; s0 < s_hi && ok; s0 += kAhead, ++group) {
                const uint32_t slot = group & 1u;
                const int n_q = min(kAhead, s_hi - s0);
                ok = mbar_wait_for(&sf_full[slot], (group >> 1) & 1u, kWaitMx);
                for (int q = 0; q < n_q && ok;) {   // two units at a time, as the MMAs
                    const uint32_t u0 = un, phase0 = phase;
                    if (++un == n_units) {
                        un = 0;
                        phase ^= 1u;
                    }
                    bool both = mbar_ready(&empty[un], phase);
                    ok = mbar_wait_for(&empty[u0], phase0, kWaitMx);
                    if (!ok) break;
                    both = __all_sync(0xFFFFFFFFu, both && q + kP < n_q);
                    fence_after_mx();
                    if (leader) {
                        copy(u0, slot, q, n_q);
                        if (both) copy(un, slot, q + kP, n_q);
                        if (q + (both ? 2 * kP : kP) >= n_q) umma_commit_mx(&sf_empty[slot]);
                    }
                    __syncwarp();
                    if (both && ++un == n_units) {
                        un = 0;
                        phase ^= 1u;
                    }
                    q += both ? 2 * kP : kP;
                }
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
        __syncwarp();
    } else if (warp >= 2 && warp < 3 + NB) {
        // --- scales of W (warp 2) or of 128 tokens of X (warps 3, 4), loaded four to eight
        // stages ahead of their use and across tiles
        const bool is_w = warp == 2;
        const int block = is_w ? 0 : warp - 3;
        const uint32_t second = kSfChunk * static_cast<uint32_t>(is_w ? 1 : NB);
        const uint32_t slots = smem_u32(sf_buf) + (is_w ? 0u : (2u + block) * kSfChunk);
        int f_tile = tile0, f_step = s_lo;   // what to load next
        Tile ft{};
        if (f_tile < n_tiles) ft = tile_at(f_tile, 0);
        int f_count = 0;
        uint32_t group = 0;
        bool ok = true;
        auto fetch = [&](Scales<kAhead>& r) {
            if (f_tile >= n_tiles || !ok) return;
            const int row0 = is_w ? ft.r0 : ft.t0, row_end = is_w ? a.rows : ft.t1;
            const int g0 = f_step * kGroupsStage;
            if (!kSplit && a.n_sc > 0) {
                const int buf = f_count % 2;
                if (f_step == 0)
                    ok = __all_sync(0xFFFFFFFFu,
                                    mbar_wait_for(&sc_full[buf],
                                              static_cast<uint32_t>(f_count / 2) & 1u, kWaitMx));
                if (!ok) return;
                const uint8_t* rows = sc_buf + static_cast<size_t>(buf) * a.sc_bytes;
                if (!is_w)
                    rows += a.sc_w +
                            (static_cast<uint32_t>(static_cast<size_t>(ft.t0) * a.gpr) & 15u);
                load_scales<true>(r, rows, a.gpr, g0, 128 * block, row_end - row0, lane);
            } else {
                const uint8_t* plane =
                    is_w ? a.w_scales + static_cast<size_t>(ft.e) * a.bank_stride : a.x_scales;
                load_scales<false>(r, plane, a.gpr, g0, row0 + 128 * block, row_end, lane);
            }
            f_step += kAhead;
            if (f_step >= s_hi) {
                if (!kSplit && a.n_sc > 0) {   // the tile's rows are in registers
                    __syncwarp();
                    if (lane == 0) mbar_arrive_m(&sc_empty[f_count % 2]);
                }
                ++f_count;
                f_step = s_lo;
                f_tile += tile_step;
                if (f_tile < n_tiles) ft = tile_at(f_tile, f_count);
            }
        };
        Scales<kAhead> cur, nxt;
        fetch(cur);
        for (int tile = tile0; tile < n_tiles && ok; tile += tile_step) {
            for (int s0 = s_lo; s0 < s_hi && ok; s0 += kAhead) {
                fetch(nxt);
                const uint32_t slot = group & 1u;
                ok = ok && __all_sync(0xFFFFFFFFu,
                                      mbar_wait_for(&sf_empty[slot], ((group >> 1) & 1u) ^ 1u,
                                                    kWaitMx));
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < kAhead; ++q)   // (stages past the tile's end: not read)
                    store_scales(cur, q, slots + slot * kSfSlot + q * kSfStage, second, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_m(&sf_full[slot]);
                ++group;
                cur = nxt;
            }
            ok = ok && !*abort_flag;
        }
        if (!ok) fail();
    } else if (warp >= Roles<kSplit>::kEpi) {
        // --- epilogue
        const int quarter = warp & 3;   // TMEM lanes 32 * quarter .. + 31
        const int half = (warp - Roles<kSplit>::kEpi) >> 2;
        int j = 0;
        for (int tile = tile0; tile < n_tiles && !*abort_flag; tile += tile_step, ++j) {
            const Tile t = tile_at(tile, j);
            const int ab = j % kAcc;
            if (!__all_sync(0xFFFFFFFFu,
                            mbar_wait_for(&acc_full[ab], static_cast<uint32_t>(j / kAcc) & 1u,
                                      kWaitMx))) {
                fail();
                break;
            }
            fence_after_mx();
            const int n = t.t1 - t.t0;
            const uint32_t src =
                tmem + ab * a.tn + (static_cast<uint32_t>(quarter * 32) << 16);
            if constexpr (kSplit) {
                // [token][128 rows] partial sums of this rank
                float* part = reinterpret_cast<float*>(after);
                for (int c = 0; c < n; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(src + c, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        part[(c + i) * kM + quarter * 32 + lane] =
                            s_hi > s_lo ? __uint_as_float(v[i]) : 0.0f;
                }
            } else {
                store_tile(Y + static_cast<size_t>(t.t0) * a.rows + t.r0 + quarter * 32, a.rows,
                           min(32, a.rows - t.r0 - quarter * 32), 16 * half, n, src, lane);
            }
            fence_before_mx();
            __syncwarp();
            if (lane == 0) mbar_arrive_m(&acc_empty[ab]);
        }
    }

    __syncthreads();
    if constexpr (kSplit) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();   // every rank's partial sums are written
        const Tile t = tile_at(tile0, 0);
        float* part = reinterpret_cast<float*>(after);
        const int n_out = (t.t1 - t.t0) * kM;
        for (int i = rank * Roles<kSplit>::kThreads + tid; i < n_out && !*abort_flag;
             i += n_rank * Roles<kSplit>::kThreads) {
            const int r = t.r0 + (i & (kM - 1)), tok = t.t0 + i / kM;
            float v[kMaxSplit], sum = 0.0f;   // all loads on their way before the first sum
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                v[q] = cluster.map_shared_rank(part, q < n_rank ? q : rank)[i];
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                if (q < n_rank) sum += v[q];
            if (r < a.rows) Y[static_cast<size_t>(tok) * a.rows + r] = from_f32<T>(sum);
        }
        cluster.sync();   // no rank leaves while its sums are being read
    }
    __syncthreads();
    if (*abort_flag && tid == 0) {
        // a CTA that gave up: its copies in flight land long before this
        for (const long long t0 = clock64(); clock64() - t0 < kDrainMx;) __nanosleep(1000);
    }
    fence_before_mx();
    __syncthreads();
    if (warp == 1) {
        fence_after_mx();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(a.tmem_cols)
                     : "memory");
    }
}

// --- host side --------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Code planes of `experts` matrices [rows][cols/2] bytes, `stride` bytes apart; copies of
// 128 bytes x box_rows.
bool code_map(CUtensorMap* map, const void* base, int cols, int rows, int experts, size_t stride,
              int box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols / 2), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(experts)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols / 2),
                                   static_cast<cuuint64_t>(stride)};
    const cuuint32_t box[3] = {kK / 2, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, experts > 0 ? 3 : 2, const_cast<void*>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static PerDevice memo;
    return memo.get([] {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
            n = 1;
        return n;
    });
}

constexpr size_t kSmemMax = 227 * 1024, kSmemSlack = 2048;   // (the static arrays)

template <typename T, bool kSplit, int NB, int kP>
cudaError_t launch_k(const CUtensorMap& wmap, const CUtensorMap& xmap, const MxArgs& a, T* Y,
                     unsigned grid, unsigned cluster, size_t smem, cudaStream_t s) {
    static PerDevice memo;
    const cudaError_t attr_err = static_cast<cudaError_t>(memo.get([] {
        return static_cast<int>(cudaFuncSetAttribute(k_mx_mm<T, kSplit, NB, kP>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(kSmemMax - kSmemSlack)));
    }));
    if (attr_err != cudaSuccess) return attr_err;
    return launch_after(k_mx_mm<T, kSplit, NB, kP>, dim3(grid),
                        static_cast<unsigned>(Roles<kSplit>::kThreads), smem, s, cluster, wmap,
                        xmap, a, Y);
}

uint32_t tmem_columns(int need) {
    uint32_t c = 32;
    while (c < static_cast<uint32_t>(need)) c *= 2;
    return c;
}

}  // namespace

cudaError_t launch_mx_mm(const uint8_t* bank, int n_experts, int rows, int cols,
                         const uint8_t* xq, int n_rows, const int32_t* offsets, void* Y,
                         int y_type, cudaStream_t s) {
    const size_t w_codes = static_cast<size_t>(rows) * cols / 2;
    const size_t x_codes = static_cast<size_t>(n_rows) * cols / 2;
    const size_t stride = padded_nbytes(rows, cols);
    const int sms = sm_count();
    MxArgs a{};
    a.w_scales = bank + w_codes;
    a.bank_stride = stride;
    a.x_scales = xq + x_codes;
    a.offsets = offsets;
    a.n_experts = n_experts;
    a.rows = rows;
    a.gpr = cols / kGroup;
    a.n_rows = n_rows;
    a.n_steps = (cols + kK - 1) / kK;
    a.n_rt = (rows + kM - 1) / kM;
    int split = 1, per_sm = 1;
    if (offsets != nullptr) {
        const int mean = (n_rows + n_experts - 1) / n_experts;
        // widest tile near the mean: narrower ones read the weights again, wider ones leave
        // less room for copies in flight (64 experts 2880x2880, us: 2 rows each 38.8 at 16
        // columns, 39.4 at 32; 32 rows 51.8 at 32, 49.5 at 96; 64 rows 82.5 at 32, 53.2 at 96,
        // 56.5 at 160; 128 rows 70.6 at 96, 66.4 at 128, 68.3 at 160; 256 rows 104 at 128, 98 at
        // 160, 113 at 176).  Copies of 16 rows: a tile brings no rows that it does not use (128
        // rows 66.4, with copies of 64 68.0).
        a.tn = mean <= 8 ? 16 : mean <= 24 ? 32 : mean <= 80 ? 96 : mean <= 128 ? 128 : 160;
        a.box = 16;
        a.n_tt = 0;
    } else {
        a.tn = std::min((n_rows + 15) / 16 * 16, kMaxTokens);
        if (n_rows > 64) {
            // token tiles: the fewest rounds of tiles over the SMs x columns per tile (and 32
            // for what a tile costs by itself).  Within 4 % of the best width from 64 to 208 on
            // eleven shapes swept, e.g. 4096x4096, 512 tokens: 128 columns 9.6 us (64: 11.3,
            // 208: 11.7); 4096 tokens: 192 columns 37.5 us (128: 39.5)
            long best = -1;
            for (int tn = 32; tn <= kMaxTokens; tn += 16) {
                const long tiles = static_cast<long>(a.n_rt) * ((n_rows + tn - 1) / tn);
                const long cost = (tiles + sms - 1) / sms * (tn + 32);
                if (best < 0 || cost <= best) {
                    best = cost;
                    a.tn = tn;
                }
            }
        } else {
            // few tokens, and row tiles for less than two thirds of the SMs: slices of K over a
            // cluster, as many as two CTAs an SM hold (us, one token unless said: 4096x4096
            // 8.0 unsplit, 6.2 split by 4, 6.0 by 8; 2880x2880, 4 tokens 7.4, 6.8, 5.9;
            // 8192x8192, 16 tokens 12.6, 10.7 by 4, 16.2 by 8; with 112 row tiles, 14336x4096,
            // 8.4 unsplit, 9.4 by 2)
            while (split < kMaxSplit && 3 * a.n_rt < 2 * sms && a.n_rt * split * 2 <= 2 * sms &&
                   split * 2 <= a.n_steps)
                split *= 2;
            per_sm = std::min(4, (a.n_rt * split + sms - 1) / sms);
        }
        a.box = a.tn;
        a.n_tt = (n_rows + a.tn - 1) / a.tn;
    }
    const int sf_blocks = (a.tn + 127) / 128;
    a.stage_bytes = kABytes + static_cast<uint32_t>(a.tn) * 128u;
    const int n_acc = split > 1 ? 1 : 2;
    const size_t sf_bytes = 2u * (split > 1 ? 2 : 4) * 2u * kSfChunk * (1 + sf_blocks);
    const size_t extra =
        sf_bytes + (split > 1            ? static_cast<size_t>(a.tn) * kM * 4
                    : offsets != nullptr ? static_cast<size_t>(n_experts + 1) * 8
                                         : 0);
    // Whole scale rows of a tile by bulk copies, two tiles deep, where rows of a tile are short
    // enough; else (long rows, slices of a split tile) loads a few stages ahead.
    if (split == 1 && static_cast<long>(kM + a.tn) * a.gpr <= 32 * 1024 - 64) {
        a.n_sc = 2;
        a.sc_w = static_cast<uint32_t>(kM * a.gpr);
        a.sc_bytes = a.sc_w + (static_cast<uint32_t>(a.tn * a.gpr + 31 + 15) & ~15u);
    }
    const size_t budget = kSmemMax / (split > 1 ? per_sm : 1) - kSmemSlack - 1024 - extra -
                          static_cast<size_t>(a.n_sc) * a.sc_bytes;
    a.n_stages = std::min(kMaxStages, static_cast<int>(budget / a.stage_bytes));
    if (split > 1) a.n_stages = std::min(a.n_stages, (a.n_steps + 1) / 2 / split * 2 + 2);
    const int sf_cols = 8 + 8 * sf_blocks;
    a.n_stages = std::min(a.n_stages, (512 / (split > 1 ? per_sm : 1) - n_acc * a.tn) / sf_cols);
    // Units of two stages (one barrier each way for both) where three of them fit, or a slice
    // of a split tile has two (us: 4096x14336, 8 tokens 9.4, single stages 10.1; 4096x4096, 128
    // tokens 7.2, single 7.7; with one unit a slice, 4096x4096, one token, 5.4, single 5.15)
    const bool pairs = sf_blocks == 1 && (split > 1 ? a.n_stages >= 4 && a.n_steps >= 4 * split
                                                    : a.n_stages >= 6);
    if (pairs) a.n_stages &= ~1;
    a.tmem_cols = tmem_columns(n_acc * a.tn + a.n_stages * sf_cols);
    // As many units as copy warps at least: a warp asks about its next unit with one parity bit,
    // which must not answer for the round before.  (The shapes above leave three stages or more
    // unsplit.)
    const int copiers = split > 1 ? Roles<true>::kCopiers : Roles<false>::kCopiers;
    if (a.n_stages / (pairs ? 2 : 1) < copiers) return cudaErrorNotSupported;
    // A CTA that waits for tensor memory must not hold up a cluster: an unsplit CTA takes
    // its SM's whole shared memory (and all 512 columns), and a split CTA at least 40 KB,
    // so that the columns of those that fit an SM together never exceed 512 (2.2 columns
    // per KB at most) and none shares an SM with a kernel that takes them all.
    const size_t ring = static_cast<size_t>(a.n_stages) * a.stage_bytes +
                        static_cast<size_t>(a.n_sc) * a.sc_bytes + extra + 1024;
    const size_t smem =
        split > 1 ? std::max(ring, static_cast<size_t>(40 * 1024)) : kSmemMax - kSmemSlack;
    CUtensorMap wmap, xmap;
    if (!code_map(&wmap, bank, cols, rows, n_experts, stride, kM) ||
        !code_map(&xmap, xq, cols, n_rows, 0, 16, a.box))
        return cudaErrorNotSupported;
    const unsigned cluster = static_cast<unsigned>(split);
    const long tiles = static_cast<long>(a.n_rt) * (offsets != nullptr ? 1 : a.n_tt);
    const unsigned most = static_cast<unsigned>(sms) / cluster;
    const unsigned grid =
        cluster * (split > 1 ? static_cast<unsigned>(a.n_rt)
                   : offsets != nullptr || tiles > static_cast<long>(most)
                       ? most
                       : static_cast<unsigned>(tiles));
    auto go = [&](auto* y) {
        using T = std::remove_pointer_t<decltype(y)>;
        auto launch = [&](auto kernel_launch) {
            return kernel_launch(wmap, xmap, a, y, grid, cluster, smem, s);
        };
        if (split > 1)
            return pairs ? launch(launch_k<T, true, 1, 2>) : launch(launch_k<T, true, 1, 1>);
        if (sf_blocks == 2) return launch(launch_k<T, false, 2, 1>);
        return pairs ? launch(launch_k<T, false, 1, 2>) : launch(launch_k<T, false, 1, 1>);
    };
    return y_type == kTypeF32 ? go(static_cast<float*>(Y)) : go(static_cast<__nv_bfloat16*>(Y));
}

cudaError_t read_fault_mx(int* value, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_mx, sizeof(int));
    if (e != cudaSuccess || !reset) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_fault_mx, &zero, sizeof(int));
}

}  // namespace mxk
