// rlk_token_logprobs.cu -- log probabilities of given tokens from logits, with
// the log-sum-exp, the entropy and the top alternatives, and their gradient.
//
// Per row, with z = x * inv_temp over the tokens that are allowed and above -inf:
//   m = max z, S = sum exp(z - m), U = sum exp(z - m) (z - m)
//   lse = m + log S, entropy = log S - U / S, logp = z[target] - lse
// and the gradient of those outputs with respect to x (p = exp(z - lse)):
//   dx[v] = inv_temp * ( p[v] (g_lse - G - g_H (z[v] - lse + H))
//                        + [v == target] g_logp + sum_j [v == id_j] g_top_j ),
//   G = g_logp + sum_j g_top_j
// One CTA per row; every sum runs in a fixed order over the row's elements, so a
// row's bits depend on that row alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>

#include "rlk_internal.h"
#include "rlk_lse.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Rows whose target was >= V, counted since the last read on this device.
__device__ unsigned long long g_range_rows;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename Elem>
__device__ __forceinline__ Elem from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// Element v of a row as fp32, -inf where the row's allowed bits leave it out.
template <typename Elem>
__device__ __forceinline__ float load_logit(const Elem* row, const uint32_t* bits, int v) {
    if (bits && !((bits[v >> 5] >> (v & 31)) & 1u)) return -INFINITY;
    return to_float(row[v]);
}

// Sums about a reference m (a raw logit; -FLT_MAX, the identity, before any
// token): s = sum e^{c (x - m)}, u = sum e^{c (x - m)} (x - m) with c = inv_temp.
struct Sums {
    float m, s, u;
};

__device__ __forceinline__ Sums combine(Sums a, Sums b, float c2) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m - m, db = b.m - m;
    const float ea = a.s == 0.0f ? 0.0f : exp2f(da * c2), eb = b.s == 0.0f ? 0.0f : exp2f(db * c2);
    Sums r;
    r.m = m;
    r.s = a.s * ea + b.s * eb;
    // a vanished operand adds nothing, however far (even -inf) its m lies below
    r.u = (ea == 0.0f ? 0.0f : ea * fmaf(da, a.s, a.u)) +
          (eb == 0.0f ? 0.0f : eb * fmaf(db, b.s, b.u));
    return r;
}

template <typename Elem>
__global__ void __launch_bounds__(kThreads)
    token_logprobs_kernel(const Elem* __restrict__ logits, int64_t row_stride,
                          const int32_t* __restrict__ targets, const uint32_t* __restrict__ allowed,
                          int64_t allowed_stride, int V, float inv_temp, int top_k,
                          float* __restrict__ out_logp, float* __restrict__ out_lse,
                          float* __restrict__ out_entropy, int32_t* __restrict__ out_ids,
                          float* __restrict__ out_top) {
    __shared__ Sums part[kThreads];
    __shared__ float best_x[kWarps];
    __shared__ int best_i[kWarps];
    const int64_t t = blockIdx.x;
    const Elem* row = logits + t * row_stride;
    const uint32_t* bits = allowed ? allowed + t * allowed_stride : nullptr;
    const float c2 = inv_temp * kLog2e;

    Sums a = {-FLT_MAX, 0.0f, 0.0f};
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float x = load_logit(row, bits, v);
        if (x > a.m) a = combine(a, {x, 0.0f, 0.0f}, c2);
        const float d = x - a.m;
        const float e = exp2f(d * c2);
        a.s += e;
        a.u = fmaf(e, fmaxf(d, -FLT_MAX), a.u);
    }
    part[threadIdx.x] = a;
    __syncthreads();
    for (int w = kThreads / 2; w > 0; w >>= 1) {
        if (threadIdx.x < w) part[threadIdx.x] = combine(part[threadIdx.x], part[threadIdx.x + w], c2);
        __syncthreads();
    }
    a = part[0];
    const float logs = logf(a.s);
    const float lse = a.s == 0.0f ? -INFINITY : fmaf(a.m, inv_temp, logs);
    const bool empty = lse == -INFINITY;
    if (threadIdx.x == 0) {
        out_lse[t] = lse;
        out_entropy[t] = empty ? 0.0f : logs - inv_temp * (a.u / a.s);
        const int32_t tg = targets[t];
        float lp = 0.0f;
        if (tg >= 0 && tg < V) {
            const float x = load_logit(row, bits, tg);
            lp = x == -INFINITY || empty ? -INFINITY : (x - a.m) * inv_temp - logs;
        } else if (tg >= V) {
            atomicAdd(&g_range_rows, 1ull);
        }
        out_logp[t] = lp;
    }

    // The alternatives one after another: the best element behind the last one
    // in the order (larger x first, lower index first among equals).
    float last_x = INFINITY;
    int last_i = -1;
    for (int k = 0; k < top_k; ++k) {
        float bx = -INFINITY;
        int bi = INT_MAX;
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const float x = load_logit(row, bits, v);
            if ((x < last_x || (x == last_x && v > last_i)) && x > bx) {
                bx = x;
                bi = v;
            }
        }
        for (int off = 16; off > 0; off >>= 1) {
            const float ox = __shfl_xor_sync(0xffffffffu, bx, off);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
            if (ox > bx || (ox == bx && oi < bi)) {
                bx = ox;
                bi = oi;
            }
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            best_x[threadIdx.x >> 5] = bx;
            best_i[threadIdx.x >> 5] = bi;
        }
        __syncthreads();
        bx = best_x[0];
        bi = best_i[0];
        for (int w = 1; w < kWarps; ++w)
            if (best_x[w] > bx || (best_x[w] == bx && best_i[w] < bi)) {
                bx = best_x[w];
                bi = best_i[w];
            }
        if (threadIdx.x == 0) {
            out_ids[t * top_k + k] = bi == INT_MAX ? -1 : bi;
            out_top[t * top_k + k] = bi == INT_MAX || empty ? -INFINITY : (bx - a.m) * inv_temp - logs;
        }
        last_x = bx;
        last_i = bi;
    }
}

template <typename Elem>
__global__ void __launch_bounds__(kThreads)
    token_logprobs_backward_kernel(const Elem* logits, int64_t row_stride,
                                   const int32_t* __restrict__ targets,
                                   const uint32_t* __restrict__ allowed, int64_t allowed_stride,
                                   int V, float inv_temp, const float* __restrict__ lse_in,
                                   const float* __restrict__ entropy_in,
                                   const float* __restrict__ g_logp, const float* __restrict__ g_lse,
                                   const float* __restrict__ g_entropy,
                                   const int32_t* __restrict__ top_ids,
                                   const float* __restrict__ g_top, int top_k, Elem* grad,
                                   int64_t grad_stride) {
    const int64_t t = blockIdx.x;
    const Elem* row = logits + t * row_stride;
    Elem* out = grad + t * grad_stride;
    const uint32_t* bits = allowed ? allowed + t * allowed_stride : nullptr;
    const float lse = lse_in[t];
    const float H = entropy_in ? entropy_in[t] : 0.0f;
    const int32_t tg = targets[t];
    const bool inside = tg >= 0 && tg < V;
    const float gl = (inside && g_logp) ? g_logp[t] : 0.0f;
    const float gh = g_entropy ? g_entropy[t] : 0.0f;
    float total = gl;
    for (int k = 0; k < top_k; ++k)
        if (top_ids[t * top_k + k] >= 0) total += g_top[t * top_k + k];
    const float a = (g_lse ? g_lse[t] : 0.0f) - total;
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float x = load_logit(row, bits, v);
        float d = 0.0f;
        if (x != -INFINITY && lse != -INFINITY) {
            const float lp = fmaf(x, inv_temp, -lse);
            // e^-200 is 0 in fp32; without the floor 0 * inf could follow
            d = lp < -200.0f ? 0.0f : expf(lp) * (a - gh * (lp + H));
            if (inside && v == tg) d += gl;
            for (int k = 0; k < top_k; ++k)
                if (top_ids[t * top_k + k] == v) d += g_top[t * top_k + k];
        }
        out[v] = from_float<Elem>(d * inv_temp);
    }
}

}  // namespace

cudaError_t token_logprobs_take_range_rows(unsigned long long* out) {
    unsigned long long v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_range_rows, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) e = cudaMemcpyToSymbol(g_range_rows, &zero, sizeof zero);
    *out = v;
    return e;
}

cudaError_t launch_token_logprobs(const void* logits, ElemType type, int64_t row_stride,
                                  const int32_t* targets, const uint32_t* allowed,
                                  int64_t allowed_stride, int64_t T, int64_t V, float inv_temp,
                                  int top_k, float* out_logp, float* out_lse, float* out_entropy,
                                  int32_t* out_ids, float* out_top, int num_sms, cudaStream_t stream) {
    auto go = [&](auto elem) {
        using Elem = decltype(elem);
        token_logprobs_kernel<Elem><<<unsigned(T), kThreads, 0, stream>>>(
            static_cast<const Elem*>(logits), row_stride, targets, allowed, allowed_stride, int(V),
            inv_temp, top_k, out_logp, out_lse, out_entropy, out_ids, out_top);
        return cudaGetLastError();
    };
    if (type == ElemType::kBf16) return go(__nv_bfloat16());
    if (type == ElemType::kFp16) return go(__half());
    return go(float());
}

cudaError_t launch_token_logprobs_backward(const void* logits, ElemType type, int64_t row_stride,
                                           const int32_t* targets, const uint32_t* allowed,
                                           int64_t allowed_stride, int64_t T, int64_t V,
                                           float inv_temp, const float* lse, const float* entropy,
                                           const float* g_logp, const float* g_lse,
                                           const float* g_entropy, const int32_t* top_ids,
                                           const float* g_top, int top_k, void* grad,
                                           int64_t grad_stride, int num_sms, cudaStream_t stream) {
    auto go = [&](auto elem) {
        using Elem = decltype(elem);
        token_logprobs_backward_kernel<Elem><<<unsigned(T), kThreads, 0, stream>>>(
            static_cast<const Elem*>(logits), row_stride, targets, allowed, allowed_stride, int(V),
            inv_temp, lse, entropy, g_logp, g_lse, g_entropy, top_ids, g_top, top_k,
            static_cast<Elem*>(grad), grad_stride);
        return cudaGetLastError();
    };
    if (type == ElemType::kBf16) return go(__nv_bfloat16());
    if (type == ElemType::kFp16) return go(__half());
    return go(float());
}

}  // namespace rlk
