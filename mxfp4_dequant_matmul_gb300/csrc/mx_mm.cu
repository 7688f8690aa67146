// mx_mm.cu -- products of two MXFP4 matrices (include/mx4.h mxfp4_mm_mx,
// mxfp4_moe_mm_mx).
//
// Y[i][r] = sum_g 2^(kw-127) 2^(kx-127) sum_{c in g} e2m1(W[r][c]) e2m1(X[i][c]).
// A group's 32 products are multiples of 1/4 below 36, so their sum is exact in
// FP32; both scales are applied in one step, so that neither alone overflows.
//
// One warp per (weight row, 4 rows of X): lanes take groups, a warp tree adds.
#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mx4_kernels.h"

namespace mxk {
namespace {

constexpr int kTok = 4;

template <typename T>
__global__ void __launch_bounds__(256)
    k_mx_mm(const uint8_t* __restrict__ bank, size_t stride, int n_experts, int rows, int cols,
            const uint8_t* __restrict__ xq, int n_rows, const int32_t* __restrict__ offsets,
            T* __restrict__ Y) {
    const int gpr = cols / kGroup;
    const int lane = threadIdx.x & 31;
    const uint8_t* xs = xq + static_cast<size_t>(n_rows) * cols / 2;
    for (int e = blockIdx.y; e < n_experts; e += gridDim.y) {
        const int b0 = offsets == nullptr ? 0 : min(max(__ldg(offsets + e), 0), n_rows);
        const int b1 = offsets == nullptr ? n_rows : min(__ldg(offsets + e + 1), n_rows);
        const uint8_t* w = bank + static_cast<size_t>(e) * stride;
        const uint8_t* ws = w + static_cast<size_t>(rows) * cols / 2;
        const int n_tok = (b1 - b0 + kTok - 1) / kTok;
        const long long units = static_cast<long long>(rows) * max(n_tok, 0);
        for (long long u = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units;
             u += static_cast<long long>(gridDim.x) * 8) {
            const int r = static_cast<int>(u / n_tok);
            const int t0 = b0 + static_cast<int>(u % n_tok) * kTok;
            float acc[kTok] = {};
            for (int g = lane; g < gpr; g += 32) {
                const uint4 wc = __ldg(group_codes(w, gpr, r, g));
                const int kw = static_cast<int>(group_scale_byte(ws, gpr, r, g));
#pragma unroll
                for (int t = 0; t < kTok; ++t) {
                    const int row = min(t0 + t, b1 - 1);
                    const uint4 xc = __ldg(group_codes(xq, gpr, row, g));
                    const int kx = static_cast<int>(group_scale_byte(xs, gpr, row, g));
                    float d = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float a[8], b[8];
                        e2m1x8_to_f32(k == 0 ? wc.x : k == 1 ? wc.y : k == 2 ? wc.z : wc.w, a);
                        e2m1x8_to_f32(k == 0 ? xc.x : k == 1 ? xc.y : k == 2 ? xc.z : xc.w, b);
#pragma unroll
                        for (int q = 0; q < 8; ++q) d = fmaf(a[q], b[q], d);
                    }
                    acc[t] += kw == 255 || kx == 255 ? __uint_as_float(0x7FC00000u)
                                                     : ldexpf(d, kw + kx - 254);
                }
            }
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], m);
                if (lane == 0 && t0 + t < b1)
                    Y[static_cast<size_t>(t0 + t) * rows + r] = from_f32<T>(acc[t]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_mx_mm(const uint8_t* bank, int n_experts, int rows, int cols,
                         const uint8_t* xq, int n_rows, const int32_t* offsets, void* Y,
                         int y_type, cudaStream_t s) {
    const size_t stride = padded_nbytes(rows, cols);
    const dim3 grid(2048, static_cast<unsigned>(n_experts));
    if (y_type == kTypeF32)
        k_mx_mm<float><<<grid, 256, 0, s>>>(bank, stride, n_experts, rows, cols, xq, n_rows,
                                            offsets, static_cast<float*>(Y));
    else
        k_mx_mm<__nv_bfloat16><<<grid, 256, 0, s>>>(bank, stride, n_experts, rows, cols, xq,
                                                    n_rows, offsets,
                                                    static_cast<__nv_bfloat16*>(Y));
    return cudaGetLastError();
}

}  // namespace mxk
