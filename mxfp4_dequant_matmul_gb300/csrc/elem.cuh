// elem.cuh -- element types of dense tensors (FP32, bfloat16, IEEE half): loads
// widened to FP32 and stores rounded once to nearest even.
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pdl.cuh"

namespace mxk {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements moved as one access (N * sizeof(T) = 2, 4, 8, 16 or 32 bytes).  The
// bits are held as integers: copies of element structs come out element by element.
struct alignas(32) Raw32 {
    uint32_t w[8];
};
template <int kBytes>
struct RawOf;
template <>
struct RawOf<2> { using type = uint16_t; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<16> { using type = uint4; };
template <>
struct RawOf<32> { using type = Raw32; };

template <typename T, int N>
struct Pack {
    using Elem = T;
    static constexpr int kN = N;
    typename RawOf<sizeof(T) * N>::type raw;
    __device__ __forceinline__ void get(float (&f)[N]) const {
        const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32(e[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[N]) {
        T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_f32<T>(f[i]);
    }
};

// One load (of what a kernel ahead may have written) or store of a pack; 32-byte units, each
// read once, do not stay in L1.
template <typename P>
__device__ __forceinline__ P load_pack(const P* p) {
    P v;
    if constexpr (sizeof(P) == 32) ld_dep_stream32(p, v.raw.w);
    else v.raw = ld_dep(&p->raw);
    return v;
}
template <typename P>
__device__ __forceinline__ void store_pack(P* p, const P& v) {
    if constexpr (sizeof(P) == 32)
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.raw.w[0]),
                     "r"(v.raw.w[1]), "r"(v.raw.w[2]), "r"(v.raw.w[3]), "r"(v.raw.w[4]),
                     "r"(v.raw.w[5]), "r"(v.raw.w[6]), "r"(v.raw.w[7])
                     : "memory");
    else
        p->raw = v.raw;
}

// i / d for 0 <= i < 2^32 as one multiplication (Granlund & Montgomery 1994): m =
// ceil(2^(32 + s) / d) with s = ceil(log2 d), one bit more than 32 bits hold.
struct FastDiv {
    uint32_t d, m, s;
    explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
        while ((1ull << s) < d) ++s;
        m = static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ uint32_t of(uint32_t i) const {
        if (d == 1) return i;
        const uint32_t t = __umulhi(i, m);
        return (t + ((i - t) >> 1)) >> (s - 1);
    }
};

// Calls go(row0, units) over n_rows rows of
// per_row units, in runs of rows whose units 32 bits can count.
template <class F>
cudaError_t over_rows(int n_rows, int per_row, F&& go) {
    const uint32_t most = static_cast<uint32_t>((1u << 31) / static_cast<uint32_t>(per_row));
    for (uint32_t row0 = 0; row0 < static_cast<uint32_t>(n_rows);) {
        const uint32_t rows = std::min(most, static_cast<uint32_t>(n_rows) - row0);
        const cudaError_t e = go(row0, rows * static_cast<uint32_t>(per_row));
        if (e != cudaSuccess) return e;
        row0 += rows;
    }
    return cudaSuccess;
}

}  // namespace mxk
