// f8_quant.cu -- quantisation to E4M3 with a power-of-two scale for each block of 128
// (include/f8.h mxfp4_f8_quant: 1x128 of a row; mxfp4_f8_quant_weight: 128x128 of a matrix).
//
// With amax = 1.m * 2^(E-127) the block's largest magnitude, 448 = 1.75 * 2^8: the scale's
// exponent field is E - 8, and one more where 1.m > 1.75 (at least 1); code = E4M3 of x * 2^-k by
// the hardware pair conversion (nearest even).  A power of two makes the scaling exact, so that
// the code is the only rounding and the maximum of the block in integers is all that is reduced.
//
// Bound by HBM: each element is read once, its code (and rounded value) written.  A thread takes 16
// elements, eight lanes a block: 32 bytes a load where x, its rows and the values are all 32-byte
// aligned, else an element a load ([7996, 2880] bf16 with values 19 us; rows 2888 apart 35, values 16
// bytes off 33.  Matrix [14336, 4096] f32 76 us, 16 bytes off 138; bf16 44 and 69).
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "f8_kernels.h"
#include "kernels.h"
#include "pdl.cuh"

namespace mxk {
namespace {

// These kernels do not let the next launch start early, as the 4-bit quantisers do not.
constexpr int kQThreads = 256;
constexpr int kItem = 16;                      // elements a thread
constexpr int kLanes = kF8Block / kItem;       // threads a block's row

// Exponent field of the scale for the largest magnitude's bits; 255 (NaN) where not finite.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) {
    const uint32_t e = top >> 23;
    if (e == 255u) return 255u;
    const int f = static_cast<int>(e) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(max(f, 1));
}
__device__ __forceinline__ float scale_value(uint32_t field) {
    return __uint_as_float(field == 255u ? 0x7FC00000u : field << 23);
}

// Packed maximum of unsigned halves.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two floats -> two E4M3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    return f16x2_to_f32x2(h);
}

// A thread's 16 elements as they lie in memory: 16-bit ones stay packed until they are quantised
// (half the registers on the way, and their largest magnitude takes one operation a pair).
template <typename T>
struct Item {
    static constexpr int kWords = kItem * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // kVec: p is 32-byte aligned
    template <bool kVec>
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kVec) {
#pragma unroll
            for (int q = 0; q < kWords / 8; ++q) {
                uint32_t r[8];
                ld_dep_stream32(reinterpret_cast<const uint32_t*>(p) + 8 * q, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[8 * q + i] = r[i];
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kItem; ++i) w[i] = ld_dep(reinterpret_cast<const uint32_t*>(p) + i);
        } else {
#pragma unroll
            for (int i = 0; i < kItem / 2; ++i) {
                const uint16_t lo = ld_dep(reinterpret_cast<const uint16_t*>(p) + 2 * i);
                const uint16_t hi = ld_dep(reinterpret_cast<const uint16_t*>(p) + 2 * i + 1);
                w[i] = lo | (static_cast<uint32_t>(hi) << 16);
            }
        }
    }
    // The largest magnitude, as bits of T (two halves to be compared where T has 16).
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) m = max(m, w[i] & 0x7FFFFFFFu);
            else m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
        }
        return m;
    }
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else if constexpr (std::is_same_v<T, __half>) return f16x2_to_f32x2(w[i]);
        else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
};

template <typename T>
__device__ __forceinline__ uint32_t max_top(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return max_u16x2(a, b);
}
// Bits of the float that the largest magnitude is.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    else {
        const uint32_t h = max(m & 0xFFFFu, m >> 16);
        if constexpr (std::is_same_v<T, __half>) return __float_as_uint(f16x2_to_f32x2(h).x);
        else return h << 16;
    }
}

// The codes of 16 elements (0 in a NaN block), and what they stand for; kVec: values are
// 32-byte aligned, else 16.
template <typename T, bool kVec>
__device__ __forceinline__ void store16(const Item<T>& v, uint32_t field, uint8_t* codes,
                                        T* values) {
    const float inv = __uint_as_float((254u - field) << 23);
    uint32_t pair[kItem / 2];
#pragma unroll
    for (int i = 0; i < kItem / 2; ++i) {
        const float2 s = __fmul2_rn(v.pair(i), make_float2(inv, inv));
        pair[i] = field == 255u ? 0u : to_e4m3x2(s.x, s.y);
    }
    *reinterpret_cast<uint4*>(codes) =
        make_uint4(pair[0] | (pair[1] << 16), pair[2] | (pair[3] << 16), pair[4] | (pair[5] << 16),
                   pair[6] | (pair[7] << 16));
    if (values == nullptr) return;
    const float s = scale_value(field);
    constexpr int kN = (kVec ? 32 : 16) / static_cast<int>(sizeof(T));
#pragma unroll
    for (int q = 0; q < kItem / kN; ++q) {
        float f[kN];
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
            const float2 d = __fmul2_rn(from_e4m3x2(pair[(q * kN + i) / 2]), make_float2(s, s));
            f[i] = d.x;
            f[i + 1] = d.y;
        }
        Pack<T, kN> a;
        a.set(f);
        store_pack(reinterpret_cast<Pack<T, kN>*>(values) + q, a);
    }
}

// Items in the flat [rows][8 per block of 128] space; those past a row's end hold zeros.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kQThreads)
    k_f8_quant(const T* x, int x_rows, int cols, long long ld, const int32_t* row_of,
               uint32_t row0, uint32_t items, FastDiv per_row, int rows,
               uint8_t* __restrict__ codes, float* __restrict__ scales, T* __restrict__ values) {
    pdl_wait();
    const uint32_t i = blockIdx.x * kQThreads + threadIdx.x;
    const uint32_t r = per_row.of(i);
    const uint32_t unit = i - r * per_row.d;
    const uint32_t c = unit * kItem;
    const size_t row = static_cast<size_t>(row0) + r;
    const bool in = i < items && c < static_cast<uint32_t>(cols);
    Item<T> v;
    v.clear();
    if (in) {
        long long src = static_cast<long long>(row);
        if (row_of != nullptr) src = ld_dep(row_of + row);
        if (src >= 0 && src < x_rows) v.template load<kVec>(x + src * ld + c);
    }
    uint32_t top = v.top();
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1)
        top = max_top<T>(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (!in) return;
    const uint32_t field = scale_field(top_bits<T>(top));
    if (unit % kLanes == 0)
        scales[static_cast<size_t>(unit / kLanes) * rows + row] = scale_value(field);
    const size_t at = row * cols + c;
    store16<T, kVec>(v, field, codes + at, values != nullptr ? values + at : nullptr);
}

// A CTA a block of 128x128: a thread holds 16 columns of every 32nd row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kQThreads)
    k_f8_quant_weight(const T* w, int rows, int cols, int col_blocks, uint8_t* __restrict__ codes,
                      float* __restrict__ scales, T* __restrict__ values) {
    constexpr int kRows = kQThreads / kLanes, kU = kF8Block / kRows;
    __shared__ uint32_t tops[kQThreads / 32];
    pdl_wait();
    const int rb = blockIdx.x / col_blocks, cb = blockIdx.x - rb * col_blocks;
    const int r0 = rb * kF8Block + threadIdx.x / kLanes;
    const int c = cb * kF8Block + threadIdx.x % kLanes * kItem;
    const size_t base = static_cast<size_t>(blockIdx.z) * rows * cols;
    Item<T> v[kU];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        v[u].clear();
        const int r = r0 + u * kRows;
        if (r < rows && c < cols)
            v[u].template load<kVec>(w + base + static_cast<size_t>(r) * cols + c);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) top = max_top<T>(top, v[u].top());
    top = __reduce_max_sync(0xFFFFFFFFu, top_bits<T>(top));
    if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int i = 1; i < kQThreads / 32; ++i) top = max(top, tops[i]);
    const uint32_t field = scale_field(top);
    if (threadIdx.x == 0)
        scales[static_cast<size_t>(blockIdx.z) * gridDim.x + blockIdx.x] = scale_value(field);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int r = r0 + u * kRows;
        if (r >= rows || c >= cols) continue;
        const size_t at = base + static_cast<size_t>(r) * cols + c;
        store16<T, kVec>(v[u], field, codes + at, values != nullptr ? values + at : nullptr);
    }
}

template <typename T>
cudaError_t quant(const void* x, int x_rows, int cols, long long ld, const int32_t* row_of,
                  int rows, uint8_t* codes, float* scales, void* values, cudaStream_t s) {
    const bool vec = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(values) |
                      (static_cast<uintptr_t>(ld) * sizeof(T))) % 32 == 0;
    const FastDiv per_row(static_cast<uint32_t>(f8_blocks(cols)) * kLanes);
    return over_rows(rows, f8_blocks(cols) * kLanes, [&](uint32_t row0, uint32_t items) {
        auto go = [&](auto kernel) {
            return launch_after(kernel, dim3((items + kQThreads - 1) / kQThreads), kQThreads, 0, s,
                                1, static_cast<const T*>(x), x_rows, cols, ld, row_of, row0, items,
                                per_row, rows, codes, scales, static_cast<T*>(values));
        };
        return vec ? go(k_f8_quant<T, true>) : go(k_f8_quant<T, false>);
    });
}

template <typename T>
cudaError_t quant_weight(const void* w, int n, int rows, int cols, uint8_t* codes, float* scales,
                         void* values, cudaStream_t s) {
    const bool vec =
        (reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(values)) % 32 == 0;
    const int col_blocks = f8_blocks(cols);
    const dim3 grid(static_cast<unsigned>(f8_blocks(rows)) * static_cast<unsigned>(col_blocks), 1,
                    static_cast<unsigned>(n));
    auto go = [&](auto kernel) {
        return launch_after(kernel, grid, kQThreads, 0, s, 1, static_cast<const T*>(w), rows, cols,
                            col_blocks, codes, scales, static_cast<T*>(values));
    };
    return vec ? go(k_f8_quant_weight<T, true>) : go(k_f8_quant_weight<T, false>);
}

}  // namespace

cudaError_t launch_f8_quant(const void* x, int type, int x_rows, int cols, long long ld,
                            const int32_t* row_of, int rows, uint8_t* codes, float* scales,
                            void* values, cudaStream_t s) {
    auto go = [&](auto one) {
        return quant<decltype(one)>(x, x_rows, cols, ld, row_of, rows, codes, scales, values, s);
    };
    return type == kTypeF32 ? go(float{}) : type == kTypeBF16 ? go(__nv_bfloat16{}) : go(__half{});
}

cudaError_t launch_f8_quant_weight(const void* w, int type, int n_matrices, int rows, int cols,
                                   uint8_t* codes, float* scales, void* values, cudaStream_t s) {
    auto go = [&](auto one) {
        return quant_weight<decltype(one)>(w, n_matrices, rows, cols, codes, scales, values, s);
    };
    return type == kTypeF32 ? go(float{}) : type == kTypeBF16 ? go(__nv_bfloat16{}) : go(__half{});
}

}  // namespace mxk
