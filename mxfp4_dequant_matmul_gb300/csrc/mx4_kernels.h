// mx4_kernels.h -- host-side launchers behind include/mx4.h (internal).  The C ABI in
// mx4_api.cu validates every argument before calling these.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace mxk {

// Element type codes of include/mx4.h.
constexpr int kTypeF32 = 0, kTypeBF16 = 1, kTypeF16 = 2;

inline int type_bytes(int type) { return type == kTypeF32 ? 4 : 2; }

// mx_quant.cu.  up == nullptr: x quantised; else silu(x) * up.
cudaError_t launch_mx_quant(const void* x, const void* up, int type, int x_rows, int cols,
                            long long ld, const int32_t* row_of, float limit, int rows,
                            uint8_t* out, void* values, cudaStream_t s);

// mx_mm.cu.  offsets == nullptr: one matrix, all n_rows rows of X.
cudaError_t launch_mx_mm(const uint8_t* bank, int n_experts, int rows, int cols,
                         const uint8_t* xq, int n_rows, const int32_t* offsets, void* Y,
                         int y_type, cudaStream_t s);

// moe_route.cu
cudaError_t launch_moe_sort(const int32_t* ids, int n_pairs, int top_k, int n_experts,
                            int32_t* token_at, int32_t* pos_of, int32_t* offsets,
                            cudaStream_t s);
cudaError_t launch_moe_dispatch(const void* x, int type, int n_tokens, int n_rows, int width,
                                const int32_t* token_at, void* xs, cudaStream_t s);
// route_w == nullptr: plain sums.
cudaError_t launch_moe_gather_sum(const void* o, int type, int n_tokens, int top_k, int width,
                                  const int32_t* pos_of, const float* route_w, void* y,
                                  cudaStream_t s);
cudaError_t launch_moe_combine_grad(const void* dy, const void* o, int type, int n_tokens,
                                    int top_k, int width, const int32_t* pos_of,
                                    const float* route_w, void* d_o, float* d_route_w,
                                    cudaStream_t s);

}  // namespace mxk
