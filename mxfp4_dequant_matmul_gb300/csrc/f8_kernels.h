// f8_kernels.h -- host-side launchers behind include/f8.h (internal).  The C ABI in
// f8_api.cu validates every argument before calling these.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "mx4_kernels.h"

namespace mxk {

constexpr int kF8Block = 128;   // elements that share a scale

// (n + 127 would overflow for the last sides that an int holds.)
inline int f8_blocks(int n) { return n / kF8Block + (n % kF8Block != 0); }

// f8_quant.cu
cudaError_t launch_f8_quant(const void* x, int type, int x_rows, int cols, long long ld,
                            const int32_t* row_of, int rows, uint8_t* codes, float* scales,
                            void* values, cudaStream_t s);
cudaError_t launch_f8_quant_weight(const void* w, int type, int n_matrices, int rows, int cols,
                                   uint8_t* codes, float* scales, void* values, cudaStream_t s);

// f8_mm.cu.  grad: the matrices' columns are the outputs and their rows the sum's terms.
// offsets == nullptr: one matrix, all n_rows rows of X.
struct F8Product {
    const uint8_t* bank;
    const float* bank_scales;
    int n_experts, rows, cols;
    const uint8_t* x;
    const float* x_scales;
    int n_rows;
    const int32_t* offsets;
    void* y;
    int y_type;
    bool grad;
};
cudaError_t launch_f8_mm(const F8Product& p, cudaStream_t s);

// grad_w.cu.  offsets == nullptr: one matrix, all n_rows rows.
cudaError_t launch_mm_grad_w(const void* dy, const void* x, int type, int n_experts, int rows,
                             int cols, int n_rows, const int32_t* offsets, void* dw, int dw_type,
                             cudaStream_t s);

}  // namespace mxk
