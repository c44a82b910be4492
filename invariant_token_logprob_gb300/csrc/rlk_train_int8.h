// rlk_train_int8.h -- launchers of the cross entropy and of the kernels on 8-bit integers (not
// part of the public C ABI; see include/rlk.h for that).
#pragma once

#include "rlk_internal.h"
#include "rlk_logits_w4.h"

namespace rlk {

// Cross entropy: what launch_lmhead_loss leaves (sum_z with smoothing, else null) to log-sum-exps
// and losses.  row_losses [T] gets each row's weighted loss; total the weights' sum; loss (unless
// null) the rows' sum, divided by total with `mean`; done is the counter launch_lmhead_loss zeroes.
cudaError_t launch_cross_entropy(const float2* records, const float* zt, const float* sum_z,
                                 const int32_t* targets, const float* weights, int64_t T, int64_t V,
                                 float smoothing, float z_loss, bool mean, float* row_losses,
                                 float* lse, float* loss, float* total, unsigned int* done,
                                 cudaStream_t stream);

// What the gradient of the cross entropy depends on.  With a = g w (/ total):
//   dz[v] = a (p[v] (1 + 2 z_loss lse) - (1 - smoothing) [v == target] - smoothing / V)
struct CeTerms {
    const int32_t* targets;
    const float* weights;  // [T], or null: 1
    const float* lse;
    const float* grad;     // [T], or one value
    const float* total;    // where the loss is a mean; else null
    int per_row;           // grad is [T]
    int V;
    float smoothing, z_loss, inv_temp;
};
// The rows of the backward with tops [T], whose largest is `top` (see CeRow), and, unless h_fp16 is
// null, h in fp16.
cudaError_t launch_cross_entropy_rows(const CeTerms& terms, const void* h, const void* W, int64_t T,
                                      int64_t H, CeRow* rows, void* h_fp16, int* tops,
                                      cudaStream_t stream);
// Reads and clears the per-device count of rows whose target was >= V.  Synchronous.
cudaError_t cross_entropy_take_range_rows(unsigned long long* out);

// 8-bit integers with a scale per row (rlk_quantize_int8, rlk_dequantize_int8).
cudaError_t launch_quantize_int8(const void* x, ElemType type, int64_t rows, int64_t K,
                                 int8_t* codes, float* scales, cudaStream_t stream);
cudaError_t launch_dequantize_int8(const int8_t* codes, const float* scales, int64_t N, int64_t K,
                                   void* out, ElemType out_type, cudaStream_t stream);
// The same codes as fp16 whole numbers, an operand of the product: of x quantised, or of given codes.
cudaError_t launch_quantize_fp16(const void* x, ElemType type, int64_t rows, int64_t K, void* codes,
                                 float* scales, cudaStream_t stream);
cudaError_t launch_widen_int8(const int8_t* codes, int64_t count, void* out, cudaStream_t stream);
// y [T][N] from x's codes as fp16 (rlk_linear_int8).
cudaError_t launch_linear_int8(const void* x_fp16, const float* x_scales, const int8_t* codes,
                               const float* scales, int64_t T, int64_t N, int64_t K, void* y,
                               ElemType y_type, int num_sms, cudaStream_t stream);
// Its bounded-wait self-test (T = 1, N = 128, K = 512); mode 1: no copy is issued, 2: no stage is
// consumed.
cudaError_t launch_linear_int8_stall_selftest(const void* x_fp16, const float* x_scales,
                                              const int8_t* codes, const float* scales, float* y,
                                              int mode, int num_sms, cudaStream_t stream);
// Reads and clears its per-device error word (bit 0: a bounded wait ran out; bit 1: a teardown
// wait ran out).
cudaError_t linear_int8_take_error(unsigned int* out);

}  // namespace rlk
