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
#include <float.h>

#include "rlk_logits.cuh"
#include "rlk_logits_w4.h"
#include "rlk_ptx.cuh"
#include "rlk_w4.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;

// Bit position of code k of a word (k = 0..7).
__host__ __device__ constexpr int code_shift(int k) { return 4 * ((k & 1) * 4 + k / 2); }

// Pieces of eight elements (16 bytes of W, one word of codes) per thread whose loads are in
// flight together: 64 KB per SM.
constexpr int kPieces = 4;

// a / b for a constant b with r = 1 / b rounded: t = a r is off by a unit of the last place
// at most, and the remainder a - t b, exact in a multiply-add, corrects it to the correctly
// rounded one (P. Markstein, IBM Journal of Research and Development 34, 1990).
__device__ __forceinline__ float divide(float a, float b, float r) {
    const float t = a * r;
    return fmaf(fmaf(-t, b, a), r, t);
}
__device__ __forceinline__ float reciprocal(float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

// Largest |x| of the four pairs of a piece.
__device__ __forceinline__ float max_abs(const uint4& v, __nv_bfloat16) {
    const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(w);
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    return fmaxf(m.x, m.y);
}
__device__ __forceinline__ float max_abs(const uint4& v, __half) {
    const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
    const __half2* p = reinterpret_cast<const __half2*>(w);
    const float2 m = __half22float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    return fmaxf(m.x, m.y);
}

// The smallest scale whose own rounding is a small part of it (and whose reciprocal and
// remainders stay inside fp32's range): from here on |x / scale| exceeds 7 (or a span 15) by
// less than half a code, so no code needs clamping at its end.
__device__ __forceinline__ float normal_scale(__nv_bfloat16) { return 7.8886090522101181e-31f; }  // 2^-100
__device__ __forceinline__ float normal_scale(__half) { return 1.220703125e-4f; }                 // 2^-13

// The word of eight codes.  2^23 + 2^22 + q has the whole number q in its low bits; adding the
// constant, which is even, rounds a half to the even code.  The words' constant part is
// subtracted at the end.
constexpr float kMagic = 12582912.0f;
constexpr uint32_t kMagicBits = 0x4b400000u;
__host__ __device__ constexpr uint32_t magic_word() {
    uint32_t c = 0;
    for (int j = 0; j < 8; ++j) c += kMagicBits * (1u << code_shift(j));
    return c;
}

// Quotients x / s, exactly rounded at ties: with an approximate reciprocal r, t = x r is off
// by some units of the last place; the remainder x - t s corrects it, so a quotient that is a
// whole number and a half comes out as that.  No other quotient of two numbers with 11
// significant bits lies closer to a half than 2^-13, far above what is left of the error.
template <bool kZeros>
__device__ __forceinline__ uint32_t code_word(const float2 (&x)[4], float s, float z) {
    const float r = reciprocal(s);
    const F2 rr = pack2(r, r), ss = pack2(-s, -s);
    const float add = kZeros ? kMagic : kMagic + 8.0f;
    const F2 magic = pack2(add, add);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const F2 v = pack2(x[j].x, x[j].y);
        const F2 t = mul2(v, rr);
        F2 q = add2(fma2(fma2(t, ss, v), rr, t), magic);
        if (kZeros) {  // the two ends' roundings may add up to one code more than 15
            const float2 f = unpack2(add2(q, pack2(z, z)));
            q = pack2(fminf(f.x, kMagic + 15.0f), fminf(f.y, kMagic + 15.0f));
        }
        const float2 f = unpack2(q);
        word += __float_as_uint(f.x) * (1u << code_shift(2 * j));
        word += __float_as_uint(f.y) * (1u << code_shift(2 * j + 1));
    }
    return word - magic_word();
}
// The same by division and with both ends clamped, for scales near the end of their range.
template <bool kZeros>
__device__ __noinline__ uint32_t code_word_small(float2 x0, float2 x1, float2 x2, float2 x3, float s,
                                                 float z) {
    const float x[8] = {x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
    uint32_t word = 0;
    for (int j = 0; j < 8; ++j) {
        const float q = rintf(x[j] / s);
        const float c = kZeros ? fminf(fmaxf(q + z, 0.0f), 15.0f) : fminf(fmaxf(q, -7.0f), 7.0f) + 8.0f;
        word |= uint32_t(int(c)) << code_shift(j);
    }
    return word;
}

// One group is held by kGroup / 8 neighbouring lanes, a piece each.  HBM-bound: reads W and
// writes a quarter of its bytes; a division per element would take longer than the bytes.
// kWhole: group divides K, so the pieces of W are dealt to the threads in memory order.
template <typename Elem, int kGroup, bool kZeros, bool kWhole>
__global__ void __launch_bounds__(kThreads, 4)
    quantize_w4_kernel(const Elem* __restrict__ W, int64_t N, int K, int num_groups,
                       uint32_t* __restrict__ codes, Elem* __restrict__ scales,
                       uint8_t* __restrict__ zeros) {
    constexpr int kLanes = kGroup / 8;
    const int64_t groups = N * num_groups;
    // (!kWhole) the row of the block's first group; the others by a 32-bit division from there
    const int64_t group0 = int64_t(blockIdx.x) * (kPieces * kThreads / kLanes);
    const int64_t row0 = kWhole ? 0 : group0 / num_groups;
    uint4 raw[kPieces];
    int64_t at[kPieces];  // piece of W, or -1 behind a row's end
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int64_t p = (int64_t(blockIdx.x) * kPieces + i) * kThreads + threadIdx.x;
        const int64_t group = p / kLanes;
        at[i] = -1;
        if (group < groups) {
            if (kWhole) {
                at[i] = p;
            } else {
                const uint32_t from_row0 = uint32_t(group - row0 * num_groups);
                const uint32_t rows = from_row0 / uint32_t(num_groups);
                const int k8 = int(from_row0 - rows * uint32_t(num_groups)) * kLanes + int(p % kLanes);
                if (k8 < K / 8) at[i] = (row0 + rows) * (K / 8) + k8;
            }
        }
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (at[i] >= 0) raw[i] = __ldcs(reinterpret_cast<const uint4*>(W) + at[i]);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float2 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pair_to_float(w[j], Elem());
        float lo = 0.0f, hi = 0.0f;
        if (kZeros) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo = fminf(fminf(lo, x[j].x), x[j].y);
                hi = fmaxf(fmaxf(hi, x[j].x), x[j].y);
            }
        } else {
            hi = max_abs(raw[i], Elem());
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) {
            if (kZeros) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        }
        Elem s16 = from_float<Elem>(kZeros ? divide(hi - lo, 15.0f, 1.0f / 15.0f)
                                           : divide(hi, 7.0f, 1.0f / 7.0f));
        if (kZeros && isinf(hi - lo)) s16 = from_float<Elem>(INFINITY);  // (bf16: a span beyond fp32)
        float s = to_float(s16);
        float z = 8.0f;
        uint32_t word;
        if (s >= normal_scale(Elem()) && s <= FLT_MAX) {
            if (kZeros) z = rintf(divide(-lo, s, reciprocal(s)));
            word = code_word<kZeros>(x, s, z);
        } else {
            if (s == 0.0f) {
                s = 1.0f;
                s16 = from_float<Elem>(1.0f);
            }
            if (kZeros) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
            word = code_word_small<kZeros>(x[0], x[1], x[2], x[3], s, z);
        }
        if (at[i] >= 0) {
            __stcs(codes + at[i], word);
            const int64_t p = (int64_t(blockIdx.x) * kPieces + i) * kThreads + threadIdx.x;
            if (p % kLanes == 0) {
                scales[p / kLanes] = s16;
                if (kZeros) zeros[p / kLanes] = uint8_t(int(z));
            }
        }
    }
}

// Words of codes per thread whose loads are in flight together.
constexpr int kWords = 8;

__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b, __half) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Values of a word, in order: scale * (q - zero) rounded once.  HBM-bound: writes four times
// what it reads.
template <typename Elem>
__device__ __forceinline__ void values(uint32_t word, Elem scale, uint32_t zero, Elem* out) {
    const Numbers<Elem> minus(zero);
    const Elem two[2] = {scale, scale};
    const Elem four = from_float<Elem>(1.0f / Numbers<Elem>::kUnit);
    const Elem fours[2] = {four, four};
    const uint32_t s = *reinterpret_cast<const uint32_t*>(two);
    const uint32_t f = *reinterpret_cast<const uint32_t*>(fours);
    uint32_t r[4];
    minus.pair(word, r[0], r[1]);
    minus.pair(word >> 8, r[2], r[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = times(times(r[j], f, Elem()), s, Elem());
    __stcs(reinterpret_cast<uint4*>(out), make_uint4(r[0], r[1], r[2], r[3]));
}
template <typename Elem>
__device__ __forceinline__ void values(uint32_t word, Elem scale, uint32_t zero, float* out) {
    const float s = to_float(scale);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = float(int((word >> code_shift(j)) & 15u) - int(zero)) * s;
    __stcs(reinterpret_cast<float4*>(out), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(out) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

template <typename Elem, typename Out, bool kWhole>
__global__ void __launch_bounds__(kThreads)
    dequantize_w4_kernel(const uint32_t* __restrict__ codes, const Elem* __restrict__ scales,
                         const uint8_t* __restrict__ zeros, int64_t N, int K, int group_shift,
                         int num_groups, Out* __restrict__ W) {  // groups of 2^group_shift words
    const int row_words = K / 8;
    const int64_t all = N * row_words;
    const int64_t block0 = int64_t(blockIdx.x) * (kWords * kThreads);
    const int64_t row0 = kWhole ? 0 : block0 / row_words;  // (!kWhole) of the block's first word
    const int64_t first = block0 + threadIdx.x;
    uint32_t word[kWords], zero[kWords];
    Elem scale[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int64_t w = first + i * kThreads;
        if (w < all) {
            word[i] = __ldcs(codes + w);
            int64_t g = w >> group_shift;
            if (!kWhole) {
                const uint32_t from_row0 = uint32_t(w - row0 * row_words);
                const uint32_t rows = from_row0 / uint32_t(row_words);
                g = (row0 + rows) * num_groups +
                    ((from_row0 - rows * uint32_t(row_words)) >> group_shift);
            }
            scale[i] = scales[g];
            zero[i] = zeros ? zeros[g] : 8u;
        }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int64_t w = first + i * kThreads;
        if (w < all) values(word[i], scale[i], zero[i], W + w * 8);
    }
}

template <typename Elem, int kGroup>
cudaError_t quantize(const void* W, int64_t N, int64_t K, uint32_t* codes, void* scales,
                     uint8_t* zeros, cudaStream_t stream) {
    const int64_t G = (K + kGroup - 1) / kGroup;
    const int64_t pieces = N * G * (kGroup / 8);
    const int64_t blocks = (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
    auto go = [&](auto kernel) {
        kernel<<<unsigned(blocks), kThreads, 0, stream>>>(static_cast<const Elem*>(W), N, int(K),
                                                          int(G), codes, static_cast<Elem*>(scales),
                                                          zeros);
        return cudaGetLastError();
    };
    if (K % kGroup == 0)
        return zeros ? go(quantize_w4_kernel<Elem, kGroup, true, true>)
                     : go(quantize_w4_kernel<Elem, kGroup, false, true>);
    return zeros ? go(quantize_w4_kernel<Elem, kGroup, true, false>)
                 : go(quantize_w4_kernel<Elem, kGroup, false, false>);
}

template <typename Elem>
cudaError_t quantize_group(const void* W, int64_t N, int64_t K, int group, uint32_t* codes,
                           void* scales, uint8_t* zeros, cudaStream_t stream) {
    if (group == 32) return quantize<Elem, 32>(W, N, K, codes, scales, zeros, stream);
    if (group == 64) return quantize<Elem, 64>(W, N, K, codes, scales, zeros, stream);
    return quantize<Elem, 128>(W, N, K, codes, scales, zeros, stream);
}

template <typename Elem, typename Out>
cudaError_t dequantize(const uint32_t* codes, const void* scales, const uint8_t* zeros, int64_t N,
                       int64_t K, int group, void* W, cudaStream_t stream) {
    const int64_t blocks = (N * (K / 8) + kThreads * kWords - 1) / (kThreads * kWords);
    auto go = [&](auto kernel) {
        kernel<<<unsigned(blocks), kThreads, 0, stream>>>(
            codes, static_cast<const Elem*>(scales), zeros, N, int(K),
            group == 32 ? 2 : group == 64 ? 3 : 4,
            int((K + group - 1) / group), static_cast<Out*>(W));
        return cudaGetLastError();
    };
    return K % group == 0 ? go(dequantize_w4_kernel<Elem, Out, true>)
                          : go(dequantize_w4_kernel<Elem, Out, false>);
}

}  // namespace

cudaError_t launch_quantize_w4(const void* W, ElemType type, int64_t N, int64_t K, int group,
                               uint32_t* codes, void* scales, uint8_t* zeros, cudaStream_t stream) {
    return type == ElemType::kBf16
               ? quantize_group<__nv_bfloat16>(W, N, K, group, codes, scales, zeros, stream)
               : quantize_group<__half>(W, N, K, group, codes, scales, zeros, stream);
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
