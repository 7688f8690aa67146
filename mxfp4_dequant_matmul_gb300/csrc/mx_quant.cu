// mx_quant.cu -- quantisation to MXFP4 (include/mx4.h mxfp4_quant,
// mxfp4_swiglu_quant).
//
// Per group of 32 elements with largest magnitude amax: scale byte k =
// max(0, E(amax) - 2), E the biased FP32 exponent (floor(log2 amax) + 127; 0 for
// zeros and subnormals), code = E2M1 of x * 2^(127-k) by the hardware pair
// conversion (nearest even, saturating at 6).  The scaling by a power of two is
// exact unless it underflows far below half of E2M1's smallest step, so the
// code is the only rounding.
//
// k_mx_quant takes any alignment.  Bound by HBM in FP32: each element is read once and 17/32
// byte (and the rounded value) written.  A thread takes 8 elements, four lanes a group: amax
// by two shuffles, one 32-bit word of codes per lane (128 bytes per warp) and the group's
// scale byte from the first of the four.  [14336, 4096] floats and their rounded values: 73.7 us,
// 6.8 TB/s; silu(gate) * up of [8192, 2880] floats 30.4 us, 6.6 TB/s, of
// bfloat16 rows aligned to an element 27.3 us, 3.9 TB/s.
#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mx4_kernels.h"
#include "pdl.cuh"

namespace mxk {
namespace {

// These kernels do not let the next launch start early: what they write may be the weights of
// an overlapped mxfp4_mv, which reads weights before it waits (and nothing was gained by it).
constexpr int kQThreads = 256;

// Two floats -> the byte of their E2M1 codes, `lo` in the low nibble; four such
// bytes -> a code word (elements 0..7 of v in nibbles 0..7).
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// 8 elements at p; kVec: p is 16-byte aligned.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (kVec) {
        constexpr int kN = 16 / sizeof(T);
#pragma unroll
        for (int q = 0; q < 8 / kN; ++q) {
            Pack<T, kN> a;
            a.raw = ld_dep_stream(reinterpret_cast<const uint4*>(p) + q);
            float f[kN];
            a.get(f);
#pragma unroll
            for (int i = 0; i < kN; ++i) v[q * kN + i] = f[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Pack<T, 1> a = load_pack(reinterpret_cast<const Pack<T, 1>*>(p + i));
            float f[1];
            a.get(f);
            v[i] = f[0];
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    constexpr int kN = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < 8 / kN; ++q) {
        float f[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] = v[q * kN + i];
        Pack<T, kN> a;
        a.set(f);
        *reinterpret_cast<uint4*>(p + q * kN) = a.raw;
    }
}

// silu(g) * u of two elements in FP32, u clamped to [-limit, limit] and g to at most limit where
// limit > 0.  silu(g) = g e^min(g,0) / (1 + e^-|g|): the denominator is in [1, 2], so nothing
// overflows on the way and rcp.approx holds it to 2^-23, far below the codes' 3 bits (the exact
// division costs as much as all the rest).
__device__ __forceinline__ float2 swiglu(float2 g, float2 u, float limit) {
    if (limit > 0.0f) {
        u.x = u.x < -limit ? -limit : (u.x > limit ? limit : u.x);
        u.y = u.y < -limit ? -limit : (u.y > limit ? limit : u.y);
        g.x = g.x > limit ? limit : g.x;   // (a NaN stays)
        g.y = g.y > limit ? limit : g.y;
    }
    const float2 e = make_float2(expf(-fabsf(g.x)), expf(-fabsf(g.y)));
    float2 r = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.y));
    const float2 top = make_float2(g.x < 0.0f ? e.x : 1.0f, g.y < 0.0f ? e.y : 1.0f);
    return __fmul2_rn(__fmul2_rn(__fmul2_rn(g, top), r), u);
}

// The 8 elements of one item (zeros past the end or for a row index out of range).
template <typename T, bool kAct, bool kVec>
__device__ __forceinline__ void load_item(float (&v)[8], const T* x, const T* up, int x_rows,
                                          long long ld, const int32_t* row_of, float limit,
                                          uint32_t row0, uint32_t i, uint32_t items,
                                          const FastDiv& per_row) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.0f;
    if (i >= items) return;
    const uint32_t r = per_row.of(i);
    const uint32_t c = (i - r * per_row.d) * 8;
    long long src = static_cast<long long>(row0) + r;
    if (row_of != nullptr) {
        src = ld_dep(row_of + src);
        if (src < 0 || src >= x_rows) return;
    }
    load8<T, kVec>(x + src * ld + c, v);
    if constexpr (kAct) {
        float u[8];
        load8<T, kVec>(up + src * ld + c, u);
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
            const float2 a =
                swiglu(make_float2(v[q], v[q + 1]), make_float2(u[q], u[q + 1]), limit);
            v[q] = a.x;
            v[q + 1] = a.y;
        }
    }
}

// Items of 8 elements in the flat [rows][cols / 8] space; a thread takes kU of them a block
// apart, all loaded before the first is quantised.
template <typename T, bool kAct, bool kVec, int kU>
__global__ void __launch_bounds__(kQThreads)
    k_mx_quant(const T* x, const T* up, int x_rows, long long ld,
               const int32_t* row_of, float limit, uint32_t row0, uint32_t items,
               FastDiv per_row, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
               T* __restrict__ values) {
    pdl_wait();
    const uint32_t i0 = blockIdx.x * (kQThreads * kU) + threadIdx.x;
    const size_t first = static_cast<size_t>(row0) * per_row.d;   // items of earlier launches
    float v[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u)
        load_item<T, kAct, kVec>(v[u], x, up, x_rows, ld, row_of, limit, row0,
                                 i0 + u * kQThreads, items, per_row);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        // largest magnitude as bits: a NaN or infinity has exponent 255
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[u][q]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t e = top >> 23;
        const bool bad = e == 255u;
        const uint32_t k = bad ? 255u : (e > 2u ? e - 2u : 0u);
        const float inv = __uint_as_float((254u - (bad ? 127u : k)) << 23);   // 2^(127-k)
#pragma unroll
        for (int q = 0; q < 8; ++q) v[u][q] = bad ? 0.0f : __fmul_rn(v[u][q], inv);
        const uint32_t word = f32x8_to_e2m1x8(v[u]);
        const uint32_t i = i0 + u * kQThreads;
        if (i >= items) continue;   // (a group's four lanes together)
        const size_t at = first + i;
        codes[at] = word;
        if ((i & 3) == 0) scales[at >> 2] = static_cast<uint8_t>(k);
        if (values != nullptr) {
            const float sc = e8m0_to_f32(k);
            e2m1x8_to_f32(word, v[u]);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[u][q] = __fmul_rn(v[u][q], sc);
            store8<T>(values + at * 8, v[u]);
        }
    }
}

// The same for aligned 16-bit rows, on the raw halves: with 16 bits an element the steps above
// issue about 160 instructions per 8 elements, twice what HBM leaves time for.  Here amax is a
// packed integer maximum of the magnitudes, and the rounded value is put together from the
// code.  For bfloat16: its two bytes by permutation out of a table of the eight magnitudes, x's
// sign, and one packed product with the scale (a power of two, exact); for half the hardware's
// E2M1 decode and two packed products, as 2^(k-127) alone may be below half's range although
// the value is not.  [7996, 2880] bfloat16 gathered from 1999 rows, with the rounded values:
// 12.6 us, 5.5 TB/s (the steps above took 24.6).
template <typename T>
__device__ __forceinline__ uint4 rounded_values(uint32_t word, const uint32_t (&raw)[4],
                                                uint32_t k);
template <>
__device__ __forceinline__ uint4 rounded_values<__nv_bfloat16>(uint32_t word,
                                                               const uint32_t (&raw)[4],
                                                               uint32_t k) {
    // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 as bfloat16: high bytes, low bytes
    constexpr uint32_t kHi0 = 0x3F3F3F00u, kHi1 = 0x40404040u;
    constexpr uint32_t kLo0 = 0xC0800000u, kLo1 = 0xC0804000u;
    const uint32_t m = word & 0x77777777u;
    // k << 7 is 2^(k-127) for 1 <= k <= 254; k = 0: the subnormal 2^-127; 255: NaN
    const uint32_t s16 = k == 0u ? 0x0040u : (k == 255u ? 0x7FC0u : k << 7);
    const uint32_t sc = s16 | (s16 << 16);
    uint32_t v[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sel = h == 0 ? m : m >> 16;
        const uint32_t hi = __byte_perm(kHi0, kHi1, sel), lo = __byte_perm(kLo0, kLo1, sel);
        v[2 * h] = __byte_perm(lo, hi, 0x5140);
        v[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] |= raw[i] & 0x80008000u;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(v[i]), "r"(sc));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ uint4 rounded_values<__half>(uint32_t word, const uint32_t (&)[4],
                                                        uint32_t k) {
    uint32_t v[4];
    e2m1x8_to_f16x2x4(word, v);
    // 2^(k-127) = 2^a 2^b, both normal halves: k - 127 is -26 .. 13 in a group that is not
    // all zeros (whose scale does not matter)
    const int e = max(static_cast<int>(k) - 127, -28);
    const int ea = e >> 1, eb = e - ea;
    uint32_t a16 = static_cast<uint32_t>(ea + 15) << 10, b16 = static_cast<uint32_t>(eb + 15) << 10;
    if (k == 255u) a16 = b16 = 0x7E00u;
    const uint32_t a2 = a16 | (a16 << 16), b2 = b16 | (b16 << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(v[i]), "r"(a2));
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(v[i]), "r"(b2));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// The halves of a register as floats.
template <typename T>
__device__ __forceinline__ float2 halves_to_f32(uint32_t h);
template <>
__device__ __forceinline__ float2 halves_to_f32<__nv_bfloat16>(uint32_t h) {
    return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 halves_to_f32<__half>(uint32_t h) { return f16x2_to_f32x2(h); }

// Packed maximum of unsigned halves.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ void stg32(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// An item is 16 elements (32 bytes, one access), two lanes a group.
template <typename T, int kU, bool kValues>
__global__ void __launch_bounds__(kQThreads)
    k_mx_quant16(const T* x, int x_rows, long long ld,
                 const int32_t* row_of, uint32_t row0, uint32_t items,
                 FastDiv per_row, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                 T* __restrict__ values) {
    pdl_wait();
    const uint32_t i0 = blockIdx.x * (kQThreads * kU) + threadIdx.x;
    const size_t first = static_cast<size_t>(row0) * per_row.d + i0;
    uint32_t raw[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint32_t i = i0 + u * kQThreads;
#pragma unroll
        for (int q = 0; q < 8; ++q) raw[u][q] = 0u;
        if (i < items) {
            const uint32_t r = per_row.of(i);
            int src = static_cast<int>(row0 + r);
            if (row_of != nullptr) src = ld_dep(row_of + src);
            if (src >= 0 && src < x_rows)
                ld_dep_stream32(x + src * ld + (i - r * per_row.d) * 16, raw[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        uint32_t top = raw[u][0] & 0x7FFF7FFFu;
#pragma unroll
        for (int q = 1; q < 8; ++q) top = max_u16x2(top, raw[u][q] & 0x7FFF7FFFu);
        top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top & 0xFFFFu, top >> 16);
        const uint32_t e = __float_as_uint(halves_to_f32<T>(top).x) >> 23;
        const bool bad = e == 255u;
        const uint32_t k = bad ? 255u : (e > 2u ? e - 2u : 0u);
        const float inv = __uint_as_float((254u - (bad ? 127u : k)) << 23);   // 2^(127-k)
        uint32_t word[2];
        uint4 val[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            const uint32_t r4[4] = {raw[u][4 * h], raw[u][4 * h + 1], raw[u][4 * h + 2],
                                    raw[u][4 * h + 3]};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = __fmul2_rn(halves_to_f32<T>(r4[q]), make_float2(inv, inv));
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            }
            word[h] = bad ? 0u : f32x8_to_e2m1x8(v);
            if (kValues) val[h] = rounded_values<T>(word[h], r4, k);
        }
        if (i0 + u * kQThreads >= items) continue;   // (a group's two lanes together)
        const size_t at = first + u * kQThreads;
        codes[at] = make_uint2(word[0], word[1]);
        if ((threadIdx.x & 1) == 0) scales[at >> 1] = static_cast<uint8_t>(k);
        if (kValues) stg32(values + at * 16, val[0], val[1]);
    }
}

// The larger magnitude of three, NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// silu(gate) * up of aligned 16-bit rows: items as k_mx_quant16's, the act in FP32.  Bound by
// issue (about 20 instructions an element, two of them on the special-function unit; HBM leaves
// time for 16): [8192, 2880] bfloat16 18.8 us, 5.7 TB/s (19.7 with the 36 registers it takes if
// it may; 24.2 with a limit), against 29.7 us with 8 elements a thread and exact divisions.
template <typename T, bool kValues>
__global__ void __launch_bounds__(kQThreads, 8)
    k_mx_swiglu16(const T* gate, const T* up, long long ld, float limit,
                  uint32_t row0, uint32_t items, FastDiv per_row, uint2* __restrict__ codes,
                  uint8_t* __restrict__ scales, T* __restrict__ values) {
    pdl_wait();
    const uint32_t i = blockIdx.x * kQThreads + threadIdx.x;
    uint32_t rg[8] = {}, ru[8] = {};
    if (i < items) {
        const uint32_t r = per_row.of(i);
        const size_t at = static_cast<size_t>(row0 + r) * ld + (i - r * per_row.d) * 16;
        ld_dep_stream32(gate + at, rg);
        ld_dep_stream32(up + at, ru);
    }
    float2 v[8];
    float top = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        v[q] = swiglu(halves_to_f32<T>(rg[q]), halves_to_f32<T>(ru[q]), limit);
        top = max_abs3(top, v[q].x, v[q].y);
    }
    const float other = __shfl_xor_sync(0xFFFFFFFFu, top, 1);
    const uint32_t e = __float_as_uint(max_abs3(top, other, other)) >> 23;
    const bool bad = e == 255u;
    const uint32_t k = bad ? 255u : (e > 2u ? e - 2u : 0u);
    const float inv = __uint_as_float((254u - (bad ? 127u : k)) << 23);   // 2^(127-k)
    uint32_t word[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float t[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = __fmul2_rn(v[4 * h + q], make_float2(inv, inv));
            t[2 * q] = f.x;
            t[2 * q + 1] = f.y;
        }
        word[h] = bad ? 0u : f32x8_to_e2m1x8(t);
    }
    if (i >= items) return;   // (a group's two lanes together)
    const size_t at = static_cast<size_t>(row0) * per_row.d + i;
    codes[at] = make_uint2(word[0], word[1]);
    if ((threadIdx.x & 1) == 0) scales[at >> 1] = static_cast<uint8_t>(k);
    if (kValues) {
        const float sc = e8m0_to_f32(k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t[8];
            e2m1x8_to_f32(word[h], t);
#pragma unroll
            for (int q = 0; q < 8; ++q) t[q] = __fmul_rn(t[q], sc);
            store8<T>(values + at * 16 + 8 * h, t);
        }
    }
}

template <typename T>
cudaError_t launch_typed(const void* x, const void* up, int x_rows, int cols, long long ld,
                         const int32_t* row_of, float limit, int rows, uint8_t* out, void* values,
                         cudaStream_t s) {
    auto* codes = reinterpret_cast<uint32_t*>(out);
    uint8_t* scales = out + static_cast<size_t>(rows) * cols / 2;
    const bool vec = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(up) |
                      (static_cast<uintptr_t>(ld) * sizeof(T))) % 16 == 0;
    if constexpr (sizeof(T) == 2) {
        if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(up) |
             reinterpret_cast<uintptr_t>(values) | (static_cast<uintptr_t>(ld) * sizeof(T))) % 32 ==
            0) {
            const FastDiv per16(static_cast<uint32_t>(cols / 16));
            if (up != nullptr)
                return over_rows(rows, cols / 16, [&](uint32_t row0, uint32_t items) {
                    auto go = [&](auto kernel) {
                        return launch_after(kernel, dim3((items + kQThreads - 1) / kQThreads),
                                            kQThreads, 0, s, 1, static_cast<const T*>(x),
                                            static_cast<const T*>(up), ld, limit, row0, items,
                                            per16, reinterpret_cast<uint2*>(codes), scales,
                                            static_cast<T*>(values));
                    };
                    return values != nullptr ? go(k_mx_swiglu16<T, true>)
                                             : go(k_mx_swiglu16<T, false>);
                });
            return over_rows(rows, cols / 16, [&](uint32_t row0, uint32_t items) {
                auto go = [&](auto kernel, uint32_t per_thread) {
                    const uint32_t per_block = kQThreads * per_thread;
                    return launch_after(kernel, dim3((items + per_block - 1) / per_block),
                                        kQThreads, 0, s, 1, static_cast<const T*>(x), x_rows, ld,
                                        row_of, row0, items, per16,
                                        reinterpret_cast<uint2*>(codes), scales,
                                        static_cast<T*>(values));
                };
                // two items a thread where that still leaves several blocks an SM (the sorted
                // prompt above: 12.6 us against 13.3; 1000 rows: 3.2 against 2.8)
                const bool two = items >= 2u * kQThreads * 152u * 8u;
                if (values != nullptr)
                    return two ? go(k_mx_quant16<T, 2, true>, 2) : go(k_mx_quant16<T, 1, true>, 1);
                return two ? go(k_mx_quant16<T, 2, false>, 2) : go(k_mx_quant16<T, 1, false>, 1);
            });
        }
    }
    const FastDiv per_row(static_cast<uint32_t>(cols / 8));
    return over_rows(rows, cols / 8, [&](uint32_t row0, uint32_t items) {
        auto go = [&](auto kernel, uint32_t per_thread) {
            const uint32_t per_block = kQThreads * per_thread;
            return launch_after(kernel, dim3((items + per_block - 1) / per_block), kQThreads, 0, s,
                                1, static_cast<const T*>(x), static_cast<const T*>(up), x_rows, ld,
                                row_of, limit, row0, items, per_row, codes, scales,
                                static_cast<T*>(values));
        };
        if (up != nullptr)
            return vec ? go(k_mx_quant<T, true, true, 1>, 1) : go(k_mx_quant<T, true, false, 1>, 1);
        if (!vec) return go(k_mx_quant<T, false, false, 1>, 1);
        // two items a thread as above ([14336, 4096] floats, codes alone: 39.4 us against 40.6)
        return items >= 2u * kQThreads * 152u * 8u ? go(k_mx_quant<T, false, true, 2>, 2)
                                                   : go(k_mx_quant<T, false, true, 1>, 1);
    });
}

}  // namespace

cudaError_t launch_mx_quant(const void* x, const void* up, int type, int x_rows, int cols,
                            long long ld, const int32_t* row_of, float limit, int rows,
                            uint8_t* out, void* values, cudaStream_t s) {
    if (type == kTypeF32)
        return launch_typed<float>(x, up, x_rows, cols, ld, row_of, limit, rows, out, values, s);
    if (type == kTypeBF16)
        return launch_typed<__nv_bfloat16>(x, up, x_rows, cols, ld, row_of, limit, rows, out,
                                           values, s);
    return launch_typed<__half>(x, up, x_rows, cols, ld, row_of, limit, rows, out, values, s);
}

}  // namespace mxk
