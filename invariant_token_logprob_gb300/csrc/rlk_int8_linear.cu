// rlk_int8_linear.cu -- y [T][N] = x . W^T for both in 8-bit whole numbers (rlk_int8.cu):
//   y[t][n] = float(sum_k qx[t][k] qw[n][k]) * sx[t] * sw[n]
// the sum exact in 32 bits (K <= 131056), so no order of it can change a bit.
//
// One warp takes a row of W and eight rows of x at a time, four products per instruction; the
// lanes' sums meet in a butterfly.  Bounded by the instructions of the products.
#include "rlk_logits.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train_int8.h"

namespace rlk {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 8;  // rows of x at a time

template <typename Out>
__global__ void __launch_bounds__(kWarps * 32)
    linear_int8_kernel(const uint4* __restrict__ x, const float* __restrict__ x_scales,
                       const uint4* __restrict__ codes, const float* __restrict__ scales,
                       int64_t T, int64_t N, int vecs, Out* __restrict__ y) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t n = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (n >= N) return;
    const int lane = threadIdx.x % 32;
    const uint4* w = codes + n * vecs;
    for (int64_t t0 = int64_t(blockIdx.y) * kCols; t0 < T; t0 += int64_t(gridDim.y) * kCols) {
        int sum[kCols] = {};
        for (int i = lane; i < vecs; i += 32) {
            const uint4 a = __ldg(w + i);
#pragma unroll
            for (int t = 0; t < kCols; ++t)
                if (t0 + t < T) {
                    const uint4 b = __ldg(x + (t0 + t) * vecs + i);
                    sum[t] = __dp4a(int(a.x), int(b.x), sum[t]);
                    sum[t] = __dp4a(int(a.y), int(b.y), sum[t]);
                    sum[t] = __dp4a(int(a.z), int(b.z), sum[t]);
                    sum[t] = __dp4a(int(a.w), int(b.w), sum[t]);
                }
        }
#pragma unroll
        for (int t = 0; t < kCols; ++t) {
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], off);
            if (lane == t && t0 + t < T)
                y[(t0 + t) * N + n] = from_float<Out>(
                    __fmul_rn(__fmul_rn(float(sum[t]), __ldg(x_scales + t0 + t)), __ldg(scales + n)));
        }
    }
}

template <typename Out>
cudaError_t launch(const int8_t* x, const float* x_scales, const int8_t* codes, const float* scales,
                   int64_t T, int64_t N, int64_t K, void* y, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t chunks = (T + kCols - 1) / kCols;
    cfg.gridDim = dim3(unsigned((N + kWarps - 1) / kWarps), unsigned(chunks < 1024 ? chunks : 1024), 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, linear_int8_kernel<Out>,
                                       reinterpret_cast<const uint4*>(x), x_scales,
                                       reinterpret_cast<const uint4*>(codes), scales, T, N,
                                       int(K / 16), static_cast<Out*>(y));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_int8(const int8_t* x, const float* x_scales, const int8_t* codes,
                               const float* scales, int64_t T, int64_t N, int64_t K, void* y,
                               ElemType y_type, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    if (y_type == ElemType::kBf16)
        return launch<__nv_bfloat16>(x, x_scales, codes, scales, T, N, K, y, stream);
    if (y_type == ElemType::kFp16)
        return launch<__half>(x, x_scales, codes, scales, T, N, K, y, stream);
    return launch<float>(x, x_scales, codes, scales, T, N, K, y, stream);
}

}  // namespace rlk
