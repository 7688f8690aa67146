// mx4_api.cu -- the extern "C" boundary of include/mx4.h: every entry point
// validates its arguments on the host, refuses with a status code (launching
// nothing) when they are wrong, and otherwise enqueues kernels on the caller's
// stream.
#include <cstdint>

#include "../../include/mx4.h"
#include "kernels.h"
#include "mx4_kernels.h"

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

// An MXFP4 matrix: as mxfp4.h's weight buffers.
bool valid_matrix(int rows, int cols) {
    return rows >= 1 && cols >= 32 && cols % 32 == 0 &&
           static_cast<long long>(rows) * cols <= (1LL << 46);
}

// P = n_tokens * top_k pairs.
bool valid_pairs(int n_tokens, int top_k) {
    return n_tokens >= 1 && top_k >= 1 &&
           static_cast<long long>(n_tokens) * top_k <= (1 << 22);
}

// The arguments the four row-moving entry points share.
int check_rows(const void* a, const void* b, int type, int n_tokens, int top_k, int width,
               const int32_t* index) {
    if (!valid_type(type) || !valid_pairs(n_tokens, top_k) || width < 1 || width > (1 << 24))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(index, 4)) return MXFP4_STATUS_BAD_POINTER;
    return MXFP4_STATUS_OK;
}

}  // namespace

extern "C" {

int mxfp4_quant(const void* x, int type, int x_rows, int cols, long long ld,
                const int32_t* row_of, int rows, void* out, void* values, cudaStream_t stream) {
    if (!valid_type(type) || !valid_matrix(rows, cols) || x_rows < 1 || ld < cols ||
        ld > (1LL << 40) || (row_of == nullptr && rows > x_rows))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(x, static_cast<unsigned>(mxk::type_bytes(type))) || !aligned(out, 16) ||
        (row_of != nullptr && !aligned(row_of, 4)) || (values != nullptr && !aligned(values, 16)))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_mx_quant(x, nullptr, type, x_rows, cols, ld, row_of, 0.0f, rows,
                                          static_cast<uint8_t*>(out), values, stream));
}

int mxfp4_swiglu_quant(const void* gate, const void* up, int type, int rows, int cols,
                       long long ld, float swiglu_limit, void* out, void* values,
                       cudaStream_t stream) {
    if (!valid_type(type) || !valid_matrix(rows, cols) || ld < cols || ld > (1LL << 40) ||
        !(swiglu_limit == swiglu_limit) || swiglu_limit > 3.0e38f)
        return MXFP4_STATUS_INVALID_ARGUMENT;
    const unsigned size = static_cast<unsigned>(mxk::type_bytes(type));
    if (!aligned(gate, size) || !aligned(up, size) || !aligned(out, 16) ||
        (values != nullptr && !aligned(values, 16)))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_mx_quant(gate, up, type, rows, cols, ld, nullptr,
                                          swiglu_limit > 0.0f ? swiglu_limit : 0.0f, rows,
                                          static_cast<uint8_t*>(out), values, stream));
}

int mxfp4_mm_mx(const void* w, int rows, int cols, const void* xq, int nb, void* Y, int y_type,
                cudaStream_t stream) {
    if (!valid_matrix(rows, cols) || nb < 1 || nb > (1 << 24) || !valid_matrix(nb, cols) ||
        (y_type != MXFP4_TYPE_F32 && y_type != MXFP4_TYPE_BF16))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(w, 16) || !aligned(xq, 16) || !aligned(Y, 16)) return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_mx_mm(static_cast<const uint8_t*>(w), 1, rows, cols,
                                       static_cast<const uint8_t*>(xq), nb, nullptr, Y, y_type,
                                       stream));
}

int mxfp4_moe_mm_mx(const void* bank, int n_experts, int rows, int cols, const void* xq,
                    int n_rows, const int32_t* offsets, void* Y, int y_type,
                    cudaStream_t stream) {
    if (!valid_matrix(rows, cols) || n_experts < 1 || n_experts > MXFP4_MOE_MAX_SORTED_EXPERTS ||
        static_cast<long long>(n_experts) * rows * cols > (1LL << 46) || n_rows < 1 ||
        n_rows > (1 << 24) || !valid_matrix(n_rows, cols) ||
        (y_type != MXFP4_TYPE_F32 && y_type != MXFP4_TYPE_BF16))
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(bank, 16) || !aligned(xq, 16) || !aligned(Y, 16) || !aligned(offsets, 4))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_mx_mm(static_cast<const uint8_t*>(bank), n_experts, rows, cols,
                                       static_cast<const uint8_t*>(xq), n_rows, offsets, Y, y_type,
                                       stream));
}

int mxfp4_moe_sort(const int32_t* expert_ids, int n_tokens, int top_k, int n_experts,
                   int32_t* token_at, int32_t* pos_of, int32_t* offsets, cudaStream_t stream) {
    if (!valid_pairs(n_tokens, top_k) || n_experts < 1 ||
        n_experts > MXFP4_MOE_MAX_SORTED_EXPERTS)
        return MXFP4_STATUS_INVALID_ARGUMENT;
    if (!aligned(expert_ids, 4) || !aligned(token_at, 4) || !aligned(pos_of, 4) ||
        !aligned(offsets, 4))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_moe_sort(expert_ids, n_tokens * top_k, top_k, n_experts, token_at,
                                          pos_of, offsets, stream));
}

int mxfp4_moe_dispatch(const void* x, int type, int n_tokens, int top_k, int width,
                       const int32_t* token_at, void* xs, cudaStream_t stream) {
    const int st = check_rows(x, xs, type, n_tokens, top_k, width, token_at);
    if (st != MXFP4_STATUS_OK) return st;
    return status_of(mxk::launch_moe_dispatch(x, type, n_tokens, n_tokens * top_k, width, token_at,
                                              xs, stream));
}

int mxfp4_moe_dispatch_grad(const void* dxs, int type, int n_tokens, int top_k, int width,
                            const int32_t* pos_of, void* dx, cudaStream_t stream) {
    const int st = check_rows(dxs, dx, type, n_tokens, top_k, width, pos_of);
    if (st != MXFP4_STATUS_OK) return st;
    return status_of(mxk::launch_moe_gather_sum(dxs, type, n_tokens, top_k, width, pos_of, nullptr,
                                                dx, stream));
}

int mxfp4_moe_combine(const void* o, int type, int n_tokens, int top_k, int width,
                      const int32_t* pos_of, const float* route_w, void* y,
                      cudaStream_t stream) {
    const int st = check_rows(o, y, type, n_tokens, top_k, width, pos_of);
    if (st != MXFP4_STATUS_OK) return st;
    if (!aligned(route_w, 4)) return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_moe_gather_sum(o, type, n_tokens, top_k, width, pos_of, route_w,
                                                y, stream));
}

int mxfp4_moe_combine_grad(const void* dy, const void* o, int type, int n_tokens, int top_k,
                           int width, const int32_t* pos_of, const float* route_w, void* d_o,
                           float* d_route_w, cudaStream_t stream) {
    const int st = check_rows(dy, o, type, n_tokens, top_k, width, pos_of);
    if (st != MXFP4_STATUS_OK) return st;
    if (!aligned(route_w, 4) || !aligned(d_o, 16) || !aligned(d_route_w, 4))
        return MXFP4_STATUS_BAD_POINTER;
    return status_of(mxk::launch_moe_combine_grad(dy, o, type, n_tokens, top_k, width, pos_of,
                                                  route_w, d_o, d_route_w, stream));
}

}  // extern "C"
