// rlk_cross_entropy.cu -- what the cross entropy does behind the LM-head kernel: from each row's
// records of the vocabulary's tiles {max, exp-sum, ., target's logit} to its log-sum-exp and loss
//   loss = lse - (1 - e) z[target] - (e / V) sum_v z[v] + l lse^2       (e smoothing, l z loss)
// and from the rows' losses to their weighted sum or mean.
//
// The row kernel is the merge kernel's shape, one warp per row with its fixed tree, so the lse is
// the log probability's bit for bit and, without smoothing and z loss, a loss of weight 1 is minus
// the log probability.  sum z comes from one fp32 number per tile: a lane adds its tiles in order,
// then the lanes meet in a butterfly.  Both orders follow from V alone.
//
// The sum over rows is one CTA: thread i adds rows i, i + 1024, ... in order, then a fixed tree.
// Two small kernels next to the LM-head GEMM's 2 T H V operations: latency-bound, a few us each.
#include "rlk_merge_row.cuh"
#include "rlk_sm103.cuh"
#include "rlk_train_int8.h"

namespace rlk {
namespace {

constexpr int kRowWarps = 8;
constexpr int kSumThreads = 1024;

// Rows whose target was >= V, counted since the last read.
__device__ unsigned long long g_ce_range_rows;

struct LossArgs {
    const float4* partials;
    const float* sum_z;  // [T][nvt], with smoothing
    const int32_t* targets;
    const float* weights;  // [T], or null: 1
    float* row_losses;
    float* lse;
    float* loss;  // or null
    float* total;
    int64_t T;
    int V, nvt;
    float smoothing, z_loss;
    int mean;
};

// The weight a row counts with: 0 where its target lies outside the vocabulary.
__device__ __forceinline__ float row_weight(const LossArgs& p, int64_t row, int32_t target) {
    if (target < 0 || target >= p.V) return 0.0f;
    return p.weights ? __ldg(p.weights + row) : 1.0f;
}

template <bool kSmooth>
__global__ void __launch_bounds__(kRowWarps * 32) row_loss_kernel(const LossArgs p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (row >= p.T) return;  // whole warp leaves together
    const int lane = threadIdx.x & 31;
    float sum_z = 0.0f;
    if constexpr (kSmooth) {
        for (int j = lane; j < p.nvt; j += 32) sum_z += __ldg(p.sum_z + row * p.nvt + j);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum_z += __shfl_xor_sync(0xffffffffu, sum_z, off);
    }
    const MergedRow r = merge_records<false, false>(p.partials, nullptr, p.targets, row, p.T, p.V,
                                                    p.nvt, 0);
    if (lane == 0) {
        const float lse = r.m + logf(r.s);
        const float w = row_weight(p, row, r.target);
        float loss = 0.0f;
        if (w != 0.0f) {
            loss = -(r.zt - lse);
            if constexpr (kSmooth) loss = fmaf(p.smoothing, r.zt - sum_z / float(p.V), loss);
            loss = fmaf(p.z_loss * lse, lse, loss) * w;
        }
        if (r.target >= p.V) atomicAdd(&g_ce_range_rows, 1ull);
        p.lse[row] = lse;
        p.row_losses[row] = loss;
    }
}

__global__ void __launch_bounds__(kSumThreads) sum_loss_kernel(const LossArgs p) {
    __shared__ float2 warps[kSumThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    float2 v = make_float2(0.0f, 0.0f);  // losses, weights
    for (int64_t row = threadIdx.x; row < p.T; row += kSumThreads) {
        v.x += p.row_losses[row];
        v.y += row_weight(p, row, __ldg(p.targets + row));
    }
    auto meet = [&]() {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
        }
    };
    meet();
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = warps[threadIdx.x];
        meet();
        if (threadIdx.x == 0) {
            *p.total = v.y;
            if (p.loss) *p.loss = !p.mean ? v.x : v.y > 0.0f ? v.x / v.y : 0.0f;
        }
    }
}

}  // namespace

cudaError_t launch_cross_entropy(const void* partials, const float* sum_z, const int32_t* targets,
                                 const float* weights, int64_t T, int64_t V, float smoothing,
                                 float z_loss, bool mean, float* row_losses, float* lse,
                                 float* loss, float* total, cudaStream_t stream) {
    const LossArgs p = {static_cast<const float4*>(partials), sum_z, targets, weights, row_losses,
                        lse, loss, total, T, int(V), int((V + kVocabTile - 1) / kVocabTile),
                        smoothing, z_loss, mean ? 1 : 0};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned((T + kRowWarps - 1) / kRowWarps), 1, 1);
    cfg.blockDim = dim3(kRowWarps * 32, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = sum_z ? cudaLaunchKernelEx(&cfg, row_loss_kernel<true>, p)
                          : cudaLaunchKernelEx(&cfg, row_loss_kernel<false>, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(kSumThreads, 1, 1);
    e = cudaLaunchKernelEx(&cfg, sum_loss_kernel, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t cross_entropy_take_range_rows(unsigned long long* out) {
    unsigned long long v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_ce_range_rows, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) e = cudaMemcpyToSymbol(g_ce_range_rows, &zero, sizeof zero);
    *out = v;
    return e;
}

}  // namespace rlk
