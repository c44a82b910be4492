// rlk_cross_entropy.cu -- what the cross entropy does around the LM-head kernel.
//
// Loss: from each row's records {m, sum 2^(z log2 e - m)} of the vocabulary's half tiles (m whole) and
// its target's z to
//   loss = lse - (1 - e) z[target] - (e / V) sum_v z[v] + l lse^2       (e smoothing, l z loss)
// and from the rows' losses to their weighted sum or mean.  One warp per row: the largest maximum
// first, then sum_j s_j 2^(m_j - M), a lane's records in order, the lanes in a butterfly; the sum
// of z likewise.  These orders follow from V alone.  The rows' sum is the last CTA's, in an order
// fixed by T, whichever CTA that is.
//
// Gradient: what each row's gradient with respect to its logits is made of (CeRow), and h in fp16.
// One warp per row (a CTA, where rows are few) reads h and its target's row of W, for the target's
// probability.
//
// Small kernels next to the LM-head products' 2 T H V operations: latency-bound, a few us each, at
// T = 4096, H = 4096 bounded by HBM (39 MB of records for the loss, 100 MB for the gradient's rows).
// The sum over rows as the last CTA's work instead of a launch of its own: 2.5 us a call.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "rlk_logits.cuh"
#include "rlk_lse.cuh"
#include "rlk_sm103.cuh"
#include "rlk_train_int8.h"

namespace rlk {
namespace {

constexpr int kRowWarps = 8;

// Rows whose target was >= V, counted since the last read.
__device__ unsigned long long g_ce_range_rows;

// The weight a row counts with: 0 where its target lies outside the vocabulary.
__device__ __forceinline__ float row_weight(const float* weights, int64_t row, int32_t target, int V) {
    if (target < 0 || target >= V) return 0.0f;
    return weights ? __ldg(weights + row) : 1.0f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

struct LossArgs {
    const float2* records;  // [T][n]
    const float* zt;
    const float* sum_z;     // [T][n], with smoothing
    const int32_t* targets;
    const float* weights;   // [T], or null: 1
    float* row_losses;
    float* lse;
    float* loss;  // or null
    float* total;
    int64_t T;
    int V, n;
    float smoothing, z_loss;
    int mean;
    unsigned int* done;  // CTAs whose rows are written; the LM-head kernel before has set it to 0
};

// By one warp.
template <bool kSmooth>
__device__ __forceinline__ void row_loss(const LossArgs& p, int64_t row, int lane) {
    const float2* records = p.records + row * p.n;
    const int32_t target = __ldg(p.targets + row);
    float top = -INFINITY, sum = 0.0f, sum_z = 0.0f;
#pragma unroll 8
    for (int j = lane; j < p.n; j += 32) top = fmaxf(top, __ldg(&records[j].x));
    top = warp_max(top);
#pragma unroll 8
    for (int j = lane; j < p.n; j += 32) {
        const float2 r = __ldg(records + j);
        sum += r.y * exp2f(r.x - top);
    }
    sum = warp_sum(sum);
    if constexpr (kSmooth) {
#pragma unroll 8
        for (int j = lane; j < p.n; j += 32) sum_z += __ldg(p.sum_z + row * p.n + j);
        sum_z = warp_sum(sum_z);
    }
    if (lane == 0) {
        // top log 2 in two numbers, the first times a whole number up to 2^9 exact
        const float top_log = top * 0.693145751953125f;
        const float log_sum = fmaf(top, 1.42860677e-6f, logf(sum));
        const float lse = top_log + log_sum;
        const float w = row_weight(p.weights, row, target, p.V);
        float loss = 0.0f;
        if (w != 0.0f) {
            const float zt = p.zt[row];
            loss = (top_log - zt) + log_sum;  // (the first difference is exact where they are near)
            if constexpr (kSmooth) loss = fmaf(p.smoothing, zt - sum_z / float(p.V), loss);
            if (p.z_loss != 0.0f) loss = fmaf(p.z_loss * lse, lse, loss);
            loss *= w;
        }
        if (target >= p.V) atomicAdd(&g_ce_range_rows, 1ull);
        p.lse[row] = lse;
        p.row_losses[row] = loss;
    }
}

template <bool kSmooth>
__global__ void __launch_bounds__(kRowWarps * 32) row_loss_kernel(const LossArgs p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (row < p.T) row_loss<kSmooth>(p, row, lane);
    // The last CTA to get here adds the rows up, thread i rows i, i + 256, ... in order.
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    __shared__ float2 warps[kRowWarps];
    float2 v = make_float2(0.0f, 0.0f);  // losses, weights
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < p.T; r += kRowWarps * 32) {
        v.x += __ldcg(p.row_losses + r);
        v.y += row_weight(p.weights, r, __ldg(p.targets + r), p.V);
    }
    v = make_float2(warp_sum(v.x), warp_sum(v.y));
    if (lane == 0) warps[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = warps[0];
        for (int w = 1; w < kRowWarps; ++w) v = make_float2(v.x + warps[w].x, v.y + warps[w].y);
        *p.total = v.y;
        if (p.loss) *p.loss = !p.mean ? v.x : v.y > 0.0f ? v.x / v.y : 0.0f;
    }
}

// The exponent e of the least power of two that |x| (finite) lies below: |x| < 2^e.
__device__ __forceinline__ int exponent_above(float x) {
    return int((__float_as_uint(x) >> 23) & 255u) - 126;
}

// kWarps warps per row (1 or 8).
template <int kWarps>
__global__ void __launch_bounds__(kRowWarps * 32)
    gradient_rows_kernel(const CeTerms p, const uint4* __restrict__ h, const uint4* __restrict__ W,
                         int64_t T, int vecs, CeRow* __restrict__ rows, uint4* __restrict__ h_fp16,
                         int* __restrict__ tops) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kLanes = 32 * kWarps;
    const int64_t row = (int64_t(blockIdx.x) * (kRowWarps * 32) + threadIdx.x) / kLanes;
    if (row >= T) return;  // (whole warps; with eight per row there is no such row)
    const int lane = threadIdx.x % kLanes;
    const int32_t target = __ldg(p.targets + row);
    const float w = row_weight(p.weights, row, target, p.V);
    float a = __ldg(p.grad + (p.per_row ? row : 0)) * w;
    if (p.total) {
        const float total = __ldg(p.total);
        a = total > 0.0f ? a / total : 0.0f;
    }
    const bool counts = w != 0.0f && a != 0.0f;
    const uint4* hr = h + row * vecs;
    const uint4* wr = W + int64_t(counts ? target : 0) * vecs;
    float dot = 0.0f, amax = 0.0f;
    if (counts) {
#pragma unroll 4
        for (int i = lane; i < vecs; i += kLanes) {
            const uint4 x = __ldg(hr + i), y = __ldg(wr + i);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = pair_to_float(xs[j], __nv_bfloat16());
                const float2 g = pair_to_float(ys[j], __nv_bfloat16());
                dot = fmaf(f.x, g.x, dot);
                dot = fmaf(f.y, g.y, dot);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        dot = warp_sum(dot);
        amax = warp_max(amax);
        if constexpr (kWarps > 1) {
            __shared__ float2 warps[kWarps];
            if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = make_float2(dot, amax);
            __syncthreads();
            dot = warps[0].x;
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                dot += warps[i].x;
                amax = fmaxf(amax, warps[i].y);
            }
            amax = fmaxf(amax, warps[0].y);
        }
    }
    const int h_exponent = max(exponent_above(amax), kCeLeastH);
    CeRow r = {};
    int top = INT_MIN;
    if (counts) {
        r.lse = __ldg(p.lse + row);
        r.p = a * fmaf(2.0f * p.z_loss, r.lse, 1.0f);
        r.target = a * (1.0f - p.smoothing);
        r.rest = a * (p.smoothing / float(p.V));
        const int most = exponent_above(fabsf(r.p) + fabsf(r.target) + fabsf(r.rest));
        // the target's element, and the factor that makes it a bf16 number
        const float at_target =
            fmaf(r.p, exp2f((dot * p.inv_temp - r.lse) * kLog2e), -r.rest) - r.target;
        const float rounded = __bfloat162float(__float2bfloat16_rn(at_target));
        float factor = rounded / at_target;
        if (!(factor > 0.99f && factor < 1.01f)) factor = 1.0f;  // (0, tiny, or not finite)
        r.p *= factor;
        r.target *= factor;
        r.rest *= factor;
        r.inv_factor = 1.0f / factor;
        r.h_exponent = h_exponent;
        if (amax > 0.0f)
            top = min(max(max(most, kCeTop - 127) + h_exponent, kCeLeastTop), kCeMostTop);
    }
    if (lane == 0) {
        rows[row] = r;
        tops[row] = top;
    }
    if (h_fp16) {
        // (rows that do not count as zeros, whatever they hold)
        const float scale = ce_power(kCeTop - h_exponent);
        uint4* out = h_fp16 + row * vecs;
#pragma unroll 4
        for (int i = lane; i < vecs; i += kLanes) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (counts) {
                const uint4 x = __ldg(hr + i);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = pair_to_float(xs[j], __nv_bfloat16());
                    const __half2 two = __floats2half2_rn(f.x * scale, f.y * scale);
                    o[j] = *reinterpret_cast<const uint32_t*>(&two);
                }
                v = make_uint4(o[0], o[1], o[2], o[3]);
            }
            out[i] = v;
        }
    }
}

cudaLaunchConfig_t config(int64_t blocks, int threads, cudaLaunchAttribute* attr,
                          cudaStream_t stream) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t launch_cross_entropy(const float2* records, const float* zt, const float* sum_z,
                                 const int32_t* targets, const float* weights, int64_t T, int64_t V,
                                 float smoothing, float z_loss, bool mean, float* row_losses,
                                 float* lse, float* loss, float* total, unsigned int* done,
                                 cudaStream_t stream) {
    const LossArgs p = {records, zt, sum_z, targets, weights, row_losses, lse, loss, total, T,
                        int(V), 2 * int((V + kVocabTile - 1) / kVocabTile), smoothing, z_loss,
                        mean ? 1 : 0, done};
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config((T + kRowWarps - 1) / kRowWarps, kRowWarps * 32, &attr, stream);
    cudaError_t e = sum_z ? cudaLaunchKernelEx(&cfg, row_loss_kernel<true>, p)
                          : cudaLaunchKernelEx(&cfg, row_loss_kernel<false>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cross_entropy_rows(const CeTerms& terms, const void* h, const void* W, int64_t T,
                                      int64_t H, CeRow* rows, void* h_fp16, int* tops,
                                      cudaStream_t stream) {
    cudaLaunchAttribute attr;
    // (long rows, and few of them: one CTA each)
    const bool wide = T <= 512 && H >= 1024;
    const cudaLaunchConfig_t cfg =
        config(wide ? T : (T + kRowWarps - 1) / kRowWarps, kRowWarps * 32, &attr, stream);
    auto kernel = wide ? gradient_rows_kernel<8> : gradient_rows_kernel<1>;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, terms, static_cast<const uint4*>(h),
                           static_cast<const uint4*>(W), T, int(H / 8), rows,
                           static_cast<uint4*>(h_fp16), tops);
    return e != cudaSuccess ? e : cudaGetLastError();
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
