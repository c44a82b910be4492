// rlk_logits_w4.h -- launchers of the kernels on logits and on 4-bit weights (not part of the
// public C ABI; see include/rlk.h for that).
#pragma once

#include "rlk_internal.h"

namespace rlk {

// Log probabilities from logits (rlk_token_logprobs) and their gradient; the
// arguments are those of the entry points, T >= 1.
enum class ElemType { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
constexpr int kMaxTopK = 32;
cudaError_t launch_token_logprobs(const void* logits, ElemType type, int64_t row_stride,
                                  const int32_t* targets, const uint32_t* allowed,
                                  int64_t allowed_stride, int64_t T, int64_t V, float inv_temp,
                                  int top_k, float* out_logp, float* out_lse, float* out_entropy,
                                  int32_t* out_ids, float* out_top, int num_sms, cudaStream_t stream);
cudaError_t launch_token_logprobs_backward(const void* logits, ElemType type, int64_t row_stride,
                                           const int32_t* targets, const uint32_t* allowed,
                                           int64_t allowed_stride, int64_t T, int64_t V,
                                           float inv_temp, const float* lse, const float* entropy,
                                           const float* g_logp, const float* g_lse,
                                           const float* g_entropy, const int32_t* top_ids,
                                           const float* g_top, int top_k, void* grad,
                                           int64_t grad_stride, int num_sms, cudaStream_t stream);
// Reads and clears the per-device count of rows whose target was >= V.
// Synchronous on the current device.
cudaError_t token_logprobs_take_range_rows(unsigned long long* out);

// 4-bit weights (rlk_linear_w4, rlk_quantize_w4, rlk_dequantize_w4); zeros may be
// null (every zero point is 8); x, scales and W have the 16-bit type `type`.
cudaError_t launch_linear_w4(const void* x, ElemType type, const uint32_t* codes,
                             const void* scales, const uint8_t* zeros, int64_t T, int64_t N,
                             int64_t K, int group, void* y, ElemType y_type, int num_sms,
                             cudaStream_t stream);
// Its bounded-wait self-test (T = 1, N = 128, K = 1024, group 128, bf16, fp32 output); mode 1:
// no copy is issued, 2: no stage is consumed.
cudaError_t launch_linear_w4_stall_selftest(const void* x, const uint32_t* codes,
                                            const void* scales, float* y, int mode, int num_sms,
                                            cudaStream_t stream);
// Reads and clears the product kernel's per-device error word (bit 0: a bounded wait ran
// out; bit 1: a teardown wait ran out).
cudaError_t linear_w4_take_error(unsigned int* out);
cudaError_t launch_quantize_w4(const void* W, ElemType type, int64_t N, int64_t K, int group,
                               uint32_t* codes, void* scales, uint8_t* zeros, cudaStream_t stream);
cudaError_t launch_dequantize_w4(const uint32_t* codes, const void* scales, const uint8_t* zeros,
                                 ElemType type, int64_t N, int64_t K, int group, void* W,
                                 ElemType w_type, cudaStream_t stream);

}  // namespace rlk
