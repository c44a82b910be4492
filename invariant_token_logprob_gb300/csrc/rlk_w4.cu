// rlk_w4.cu -- weights in 4 bits with group scales: quantising and reading back (the
// product is in rlk_w4_linear.cu).
//
// Format: W [N][K] is cut along K into groups of `group` (32, 64 or 128) elements;
// the last group of a row is short where group does not divide K (K % 32 == 0).
// Element (n, k) of group g stands for scale[n][g] * (q - zero[n][g]), q in 0..15,
// with one 16-bit scale and one zero point (8 where no zero points are kept) per
// group.  Eight codes k = 8w .. 8w+7 make word w of a row: the even k in nibbles
// 0..3, the odd k in nibbles 4..7, so that (word >> 4i) & 0x000f000f is the pair
// (8w + 2i, 8w + 2i + 1) in the halves of a register.
#include "rlk_internal.h"
#include "rlk_logits.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;

// Bit position of code k of a word (k = 0..7).
__host__ __device__ constexpr int code_shift(int k) { return 4 * ((k & 1) * 4 + k / 2); }

// One group of kGroup elements is held by kGroup / 8 neighbouring lanes, eight
// elements (16 bytes of W, one word of codes) each.
template <typename Elem, int kGroup>
__global__ void __launch_bounds__(kThreads)
    quantize_w4_kernel(const Elem* __restrict__ W, int64_t N, int K, int num_groups,
                       uint32_t* __restrict__ codes, Elem* __restrict__ scales,
                       uint8_t* __restrict__ zeros) {
    constexpr int kLanes = kGroup / 8;
    const int64_t piece = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kLanes;  // (n, g)
    const int sub = threadIdx.x % kLanes;
    const bool act = piece < N * num_groups;
    const int64_t n = act ? piece / num_groups : 0;
    const int g = act ? int(piece - n * num_groups) : 0;
    const int k = g * kGroup + sub * 8;
    const bool in_row = act && k < K;
    float x[8];
    union {
        uint4 v;
        Elem e[8];
    } raw;
    raw.v = make_uint4(0u, 0u, 0u, 0u);
    if (in_row) raw.v = *reinterpret_cast<const uint4*>(W + n * K + k);
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = to_float(raw.e[i]);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    Elem s16 = from_float<Elem>(zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    if (to_float(s16) == 0.0f) s16 = from_float<Elem>(1.0f);
    const float s = to_float(s16);
    const float z = zeros ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 8.0f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = rintf(x[i] / s);
        const float q = zeros ? fminf(fmaxf(r + z, 0.0f), 15.0f) : fminf(fmaxf(r, -7.0f), 7.0f) + 8.0f;
        word |= uint32_t(int(q)) << code_shift(i);
    }
    if (in_row) codes[n * (K / 8) + k / 8] = word;
    if (act && sub == 0) {
        scales[piece] = s16;
        if (zeros) zeros[piece] = uint8_t(int(z));
    }
}

// One word of codes per thread.
template <typename Elem, typename Out>
__global__ void __launch_bounds__(kThreads)
    dequantize_w4_kernel(const uint32_t* __restrict__ codes, const Elem* __restrict__ scales,
                         const uint8_t* __restrict__ zeros, int64_t N, int K, int group,
                         int num_groups, Out* __restrict__ W) {
    const int words = K / 8;
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= N * words) return;
    const int64_t n = i / words;
    const int g = int(i - n * words) * 8 / group;
    const float s = to_float(scales[n * num_groups + g]);
    const int z = zeros ? zeros[n * num_groups + g] : 8;
    const uint32_t word = codes[i];
    union {
        uint4 v[sizeof(Out) / 2];
        Out e[8];
    } o;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        o.e[j] = from_float<Out>(float(int((word >> code_shift(j)) & 15u) - z) * s);
#pragma unroll
    for (int j = 0; j < int(sizeof(Out) / 2); ++j) reinterpret_cast<uint4*>(W + i * 8)[j] = o.v[j];
}

template <typename Elem>
cudaError_t quantize(const void* W, int64_t N, int64_t K, int group, uint32_t* codes, void* scales,
                     uint8_t* zeros, cudaStream_t stream) {
    const int G = int((K + group - 1) / group);
    const int64_t blocks = (N * G * (group / 8) + kThreads - 1) / kThreads;
    auto go = [&](auto kernel) {
        kernel<<<unsigned(blocks), kThreads, 0, stream>>>(static_cast<const Elem*>(W), N, int(K), G,
                                                          codes, static_cast<Elem*>(scales), zeros);
        return cudaGetLastError();
    };
    if (group == 32) return go(quantize_w4_kernel<Elem, 32>);
    if (group == 64) return go(quantize_w4_kernel<Elem, 64>);
    return go(quantize_w4_kernel<Elem, 128>);
}

template <typename Elem, typename Out>
cudaError_t dequantize(const uint32_t* codes, const void* scales, const uint8_t* zeros, int64_t N,
                       int64_t K, int group, void* W, cudaStream_t stream) {
    const int64_t blocks = (N * (K / 8) + kThreads - 1) / kThreads;
    dequantize_w4_kernel<Elem, Out><<<unsigned(blocks), kThreads, 0, stream>>>(
        codes, static_cast<const Elem*>(scales), zeros, N, int(K), group,
        int((K + group - 1) / group), static_cast<Out*>(W));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_w4(const void* W, ElemType type, int64_t N, int64_t K, int group,
                               uint32_t* codes, void* scales, uint8_t* zeros, cudaStream_t stream) {
    return type == ElemType::kBf16
               ? quantize<__nv_bfloat16>(W, N, K, group, codes, scales, zeros, stream)
               : quantize<__half>(W, N, K, group, codes, scales, zeros, stream);
}

cudaError_t launch_dequantize_w4(const uint32_t* codes, const void* scales, const uint8_t* zeros,
                                 ElemType type, int64_t N, int64_t K, int group, void* W,
                                 ElemType w_type, cudaStream_t stream) {
    const bool wide = w_type == ElemType::kFp32;
    if (type == ElemType::kBf16)
        return wide ? dequantize<__nv_bfloat16, float>(codes, scales, zeros, N, K, group, W, stream)
                    : dequantize<__nv_bfloat16, __nv_bfloat16>(codes, scales, zeros, N, K, group, W,
                                                               stream);
    return wide ? dequantize<__half, float>(codes, scales, zeros, N, K, group, W, stream)
                : dequantize<__half, __half>(codes, scales, zeros, N, K, group, W, stream);
}

}  // namespace rlk
