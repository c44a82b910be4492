// rlk_train_int8.h -- launchers of the cross entropy and of the kernels on 8-bit integers (not
// part of the public C ABI; see include/rlk.h for that).
#pragma once

#include "rlk_internal.h"
#include "rlk_logits_w4.h"

namespace rlk {

// Cross entropy: the rows' records (and sum_z, with smoothing) to log-sum-exps and losses.
// row_losses [T] gets each row's weighted loss; total the weights' sum; loss (unless null) the
// rows' sum, divided by total with `mean`.
cudaError_t launch_cross_entropy(const void* partials, const float* sum_z, const int32_t* targets,
                                 const float* weights, int64_t T, int64_t V, float smoothing,
                                 float z_loss, bool mean, float* row_losses, float* lse,
                                 float* loss, float* total, cudaStream_t stream);
// Reads and clears the per-device count of rows whose target was >= V.  Synchronous.
cudaError_t cross_entropy_take_range_rows(unsigned long long* out);

// 8-bit integers with a scale per row (rlk_quantize_int8, rlk_dequantize_int8).
cudaError_t launch_quantize_int8(const void* x, ElemType type, int64_t rows, int64_t K,
                                 int8_t* codes, float* scales, cudaStream_t stream);
cudaError_t launch_dequantize_int8(const int8_t* codes, const float* scales, int64_t N, int64_t K,
                                   void* out, ElemType out_type, cudaStream_t stream);
// y [T][N] from x's codes (rlk_linear_int8).
cudaError_t launch_linear_int8(const int8_t* x, const float* x_scales, const int8_t* codes,
                               const float* scales, int64_t T, int64_t N, int64_t K, void* y,
                               ElemType y_type, int num_sms, cudaStream_t stream);

}  // namespace rlk
