// f8_api.cu -- the extern "C" boundary of include/f8.h: every entry point validates its
// arguments on the host, refuses with a status code (launching nothing) when they are
// wrong, and otherwise enqueues kernels on the caller's stream.
#include <cstdint>

#include "../../include/f8.h"
#include "f8_kernels.h"
#include "kernels.h"

namespace {

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return MXFP4_STATUS_OK;
    mxk::record_cuda_error(static_cast<int>(e));
    return MXFP4_STATUS_LAUNCH_FAILED;
}

bool aligned(const void* p, unsigned to) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1u)) == 0;
}

bool valid_type(int type) {
    return type == MXFP4_TYPE_F32 || type == MXFP4_TYPE_BF16 || type == MXFP4_TYPE_F16;
}

bool valid_out_type(int type) { return type == MXFP4_TYPE_F32 || type == MXFP4_TYPE_BF16; }

constexpr int kMaxSide = 1 << 24;   // of a product's matrices

// n matrices of codes.
bool valid_codes(int n, int rows, int cols) {
    return n >= 1 && rows >= 1 && cols >= 16 && cols % 16 == 0 &&
           static_cast<long long>(rows) * cols <= (1LL << 44) / n;
}

// What the four products share.  k: the terms of a sum, a row of X.
int f8_product(const void* bank, const float* bank_scales, int n_experts, int rows, int cols,
               const void* xq, const float* x_scales, int n_rows, bool grouped,
               const int32_t* offsets, void* y, int y_type, bool grad, cudaStream_t stream) {
    const int k = grad ? rows : cols;
    if (n_experts < 1 || n_experts > MXFP4_MOE_MAX_SORTED_EXPERTS ||
        !valid_codes(n_experts, rows, cols) || !valid_codes(1, n_rows, k) || rows > kMaxSide ||
        cols > kMaxSide || n_rows > kMaxSide ||
        static_cast<long long>(n_rows) * (grad ? cols : rows) > (1LL << 44) ||
        !valid_out_type(y_type))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(bank, 16) || !aligned(xq, 16) || !aligned(y, 16) || !aligned(bank_scales, 4) ||
        !aligned(x_scales, 4) || (grouped && !aligned(offsets, 4)))
        return MXFP4_STATUS_BAD_POINTER;
    mxk::F8Product p{};
    p.bank = static_cast<const uint8_t*>(bank);
    p.bank_scales = bank_scales;
    p.n_experts = n_experts;
    p.rows = rows;
    p.cols = cols;
    p.x = static_cast<const uint8_t*>(xq);
    p.x_scales = x_scales;
    p.n_rows = n_rows;
    p.offsets = grouped ? offsets : nullptr;
    p.y = y;
    p.y_type = y_type;
    p.grad = grad;
    return status_of(mxk::launch_f8_mm(p, stream));
}

int grad_w(const void* dy, const void* x, int type, int n_experts, int rows, int cols, int n_rows,
           bool grouped, const int32_t* offsets, void* dw, int dw_type, cudaStream_t stream) {
    if ((type != MXFP4_TYPE_BF16 && type != MXFP4_TYPE_F16) || !valid_out_type(dw_type) ||
        n_experts < 1 || n_experts > MXFP4_MOE_MAX_SORTED_EXPERTS || rows < 8 || cols < 8 ||
        rows % 8 != 0 || cols % 8 != 0 || n_rows < 1 || rows > kMaxSide || cols > kMaxSide ||
        n_rows > kMaxSide ||
        static_cast<long long>(rows) * cols > (1LL << 44) / n_experts ||
        static_cast<long long>(rows) * n_rows > (1LL << 44) ||
        static_cast<long long>(cols) * n_rows > (1LL << 44))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) ||
        (grouped && !aligned(offsets, 4)))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_mm_grad_w(dy, x, type, n_experts, rows, cols, n_rows,
                                           grouped ? offsets : nullptr, dw, dw_type, stream));
}

}  // namespace

extern "C" {

int mxfp4_f8_quant(const void* x, int type, int x_rows, int cols, long long ld,
                   const int32_t* row_of, int rows, void* codes, float* scales, void* values,
                   cudaStream_t stream) {
    if (!valid_type(type) || !valid_codes(1, rows, cols) || x_rows < 1 || ld < cols ||
        ld > (1LL << 40) || (row_of == nullptr && rows > x_rows))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(x, static_cast<unsigned>(mxk::type_bytes(type))) || !aligned(codes, 16) ||
        !aligned(scales, 4) || (row_of != nullptr && !aligned(row_of, 4)) ||
        (values != nullptr && !aligned(values, 16)))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_f8_quant(x, type, x_rows, cols, ld, row_of, rows,
                                          static_cast<uint8_t*>(codes), scales, values, stream));
}

int mxfp4_f8_quant_weight(const void* w, int type, int n_matrices, int rows, int cols, void* codes,
                          float* scales, void* values, cudaStream_t stream) {
    if (!valid_type(type) || n_matrices < 1 || n_matrices > MXFP4_MOE_MAX_SORTED_EXPERTS ||
        !valid_codes(n_matrices, rows, cols))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4) ||
        (values != nullptr && !aligned(values, 16)))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_f8_quant_weight(w, type, n_matrices, rows, cols,
                                                 static_cast<uint8_t*>(codes), scales, values,
                                                 stream));
}

int mxfp4_f8_mm(const void* w, const float* w_scales, int rows, int cols, const void* xq,
                const float* x_scales, int nb, void* Y, int y_type, cudaStream_t stream) {
    return f8_product(w, w_scales, 1, rows, cols, xq, x_scales, nb, false, nullptr, Y, y_type,
                      false, stream);
}

int mxfp4_f8_moe_mm(const void* bank, const float* bank_scales, int n_experts, int rows, int cols,
                    const void* xq, const float* x_scales, int n_rows, const int32_t* offsets,
                    void* Y, int y_type, cudaStream_t stream) {
    return f8_product(bank, bank_scales, n_experts, rows, cols, xq, x_scales, n_rows, true,
                      offsets, Y, y_type, false, stream);
}

int mxfp4_f8_mm_grad(const void* w, const float* w_scales, int rows, int cols, const void* dyq,
                     const float* dy_scales, int nb, void* dX, int dx_type, cudaStream_t stream) {
    return f8_product(w, w_scales, 1, rows, cols, dyq, dy_scales, nb, false, nullptr, dX, dx_type,
                      true, stream);
}

int mxfp4_f8_moe_mm_grad(const void* bank, const float* bank_scales, int n_experts, int rows,
                         int cols, const void* dyq, const float* dy_scales, int n_rows,
                         const int32_t* offsets, void* dX, int dx_type, cudaStream_t stream) {
    return f8_product(bank, bank_scales, n_experts, rows, cols, dyq, dy_scales, n_rows, true,
                      offsets, dX, dx_type, true, stream);
}

int mxfp4_mm_grad_w(const void* dy, const void* x, int type, int rows, int cols, int n_rows,
                    void* dW, int dw_type, cudaStream_t stream) {
    return grad_w(dy, x, type, 1, rows, cols, n_rows, false, nullptr, dW, dw_type, stream);
}

int mxfp4_moe_mm_grad_w(const void* dy, const void* x, int type, int n_experts, int rows, int cols,
                        int n_rows, const int32_t* offsets, void* dW, int dw_type,
                        cudaStream_t stream) {
    return grad_w(dy, x, type, n_experts, rows, cols, n_rows, true, offsets, dW, dw_type, stream);
}

}  // extern "C"
