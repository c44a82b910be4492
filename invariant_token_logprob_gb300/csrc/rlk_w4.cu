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
// flight together: 96 KB per SM.
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

// The larger of the halves of (a, b) each: the largest of a's pair and of b's.
template <typename Pair>
__device__ __forceinline__ uint32_t max_halves(Pair a, Pair b) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(&a), y = *reinterpret_cast<const uint32_t*>(&b);
    const uint32_t low = __byte_perm(x, y, 0x5410), high = __byte_perm(x, y, 0x7632);
    const Pair m = max_pair(*reinterpret_cast<const Pair*>(&low), *reinterpret_cast<const Pair*>(&high));
    return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename Elem>
__device__ __forceinline__ typename PairOf<Elem>::type max_of_pairs(const uint4& v, uint32_t keep,
                                                                    uint32_t flip, Elem) {
    using Pair = typename PairOf<Elem>::type;
    const uint32_t w[4] = {(v.x & keep) ^ flip, (v.y & keep) ^ flip, (v.z & keep) ^ flip,
                           (v.w & keep) ^ flip};
    const Pair* p = reinterpret_cast<const Pair*>(w);
    return max_pair(max_pair(p[0], p[1]), max_pair(p[2], p[3]));
}
// The largest |x| of two pieces (NaN counts as nothing).
template <typename Elem>
__device__ __forceinline__ uint32_t max_abs_pair(const uint4& a, const uint4& b, Elem e) {
    return max_halves(max_of_pairs(a, 0x7fff7fffu, 0u, e), max_of_pairs(b, 0x7fff7fffu, 0u, e));
}
// The largest x and the largest -x of a piece.
template <typename Elem>
__device__ __forceinline__ uint32_t max_both(const uint4& a, Elem e) {
    return max_halves(max_of_pairs(a, 0xffffffffu, 0u, e), max_of_pairs(a, 0xffffffffu, 0x80008000u, e));
}

// The smallest scale whose own rounding is a small part of it (and whose reciprocal and
// remainders stay inside fp32's range): from here on |x / scale| exceeds 7 (or a span 15) by
// less than half a code, so no code needs clamping at its end.
__device__ __forceinline__ float normal_scale(__nv_bfloat16) { return 7.8886090522101181e-31f; }  // 2^-100
__device__ __forceinline__ float normal_scale(__half) { return 1.220703125e-4f; }                 // 2^-13

// The word of eight codes.  2^23 + 2^22 + q has the whole number q in its low bits; adding the
// constant, which is even, rounds a half to the even code.  Four codes become 16 bits of one
// such number by exact multiply-adds, the even and the odd ones side by side.
constexpr float kMagic = 12582912.0f;

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
    const F2 off = pack2(-kMagic, -kMagic);
    F2 four = magic;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const F2 v = pack2(x[j].x, x[j].y);
        const F2 t = mul2(v, rr);
        F2 q = add2(fma2(fma2(t, ss, v), rr, t), magic);
        if (kZeros) {  // the two ends' roundings may add up to one code more than 15
            const float2 f = unpack2(add2(q, pack2(z, z)));
            q = pack2(fminf(f.x, kMagic + 15.0f), fminf(f.y, kMagic + 15.0f));
        }
        const float place = float(1 << 4 * j);
        four = j == 0 ? q : fma2(add2(q, off), pack2(place, place), four);
    }
    const float2 f = unpack2(four);
    return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x5410);
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
// writes a quarter of its bytes.  A division per element would take longer than the bytes;
// the arithmetic is kept to packed pairs, and the groups' maxima go across lanes together
// (N = 151936, K = 4096, bf16, group 128: 233 us, 6.7 TB/s; with zero points 279 us).
// kWhole: group divides K, so the pieces of W are dealt to the threads in memory order, six
// CTAs to an SM (five: 241 us); the rows' places otherwise would spill with six.
template <typename Elem, int kGroup, bool kZeros, bool kWhole>
__global__ void __launch_bounds__(kThreads, kWhole ? 6 : 5)
    quantize_w4_kernel(const Elem* __restrict__ W, int64_t N, int K, int num_groups,
                       uint32_t* __restrict__ codes, Elem* __restrict__ scales,
                       uint8_t* __restrict__ zeros) {
    constexpr int kLanes = kGroup / 8;
    const int64_t first = int64_t(blockIdx.x) * (kPieces * kThreads) + threadIdx.x;
    const int left = int(min(N * num_groups * kLanes - first, int64_t(kPieces * kThreads)));
    // (!kWhole) the row of the block's first group, and the thread's first group from there;
    // its other groups lie kStep apart
    constexpr uint32_t kStep = kThreads / kLanes;
    const int64_t group0 = int64_t(blockIdx.x) * (kPieces * kStep);
    const uint32_t per_row = uint32_t(num_groups);
    const int64_t row0 = kWhole ? 0
                         : N * num_groups <= UINT32_MAX ? int64_t(uint32_t(group0) / per_row)
                                                        : group0 / num_groups;
    uint32_t col = uint32_t(group0 - row0 * num_groups) + threadIdx.x / kLanes;
    uint32_t row = kWhole ? 0 : col / per_row;
    col -= row * per_row;
    const uint32_t step_rows = kWhole ? 0 : kStep / per_row, step_cols = kStep - step_rows * per_row;
    const uint4* src = reinterpret_cast<const uint4*>(W) + (kWhole ? first : row0 * (K / 8));
    codes += kWhole ? first : row0 * (K / 8);
    scales += first / kLanes;
    if (kZeros) zeros += first / kLanes;
    uint4 raw[kPieces];
    int at[kPieces];  // piece of W from src on, or -1 behind a row's end
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        at[i] = i * kThreads < left ? i * kThreads : -1;
        if (!kWhole) {
            const int k8 = int(col) * kLanes + int(threadIdx.x % kLanes);
            at[i] = at[i] >= 0 && k8 < K / 8 ? int(row) * (K / 8) + k8 : -1;
            row += step_rows;
            col += step_cols;
            if (col >= per_row) {
                col -= per_row;
                ++row;
            }
        }
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (at[i] >= 0) raw[i] = __ldcs(src + at[i]);
    }
    // Every piece's largest element and largest negated one, or two pieces' largest |x|, as a
    // pair of the elements' own type: exact, and all groups' steps across lanes run together.
    using Pair = typename PairOf<Elem>::type;
    constexpr int kPairs = kZeros ? kPieces : kPieces / 2;
    uint32_t most[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        most[i] = kZeros ? max_both(raw[i], Elem()) : max_abs_pair(raw[2 * i], raw[2 * i + 1], Elem());
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, most[i], off);
            const Pair m = max_pair(*reinterpret_cast<const Pair*>(&most[i]),
                                    *reinterpret_cast<const Pair*>(&o));
            most[i] = *reinterpret_cast<const uint32_t*>(&m);
        }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float2 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pair_to_float(w[j], Elem());
        const float2 both = pair_to_float(most[kZeros ? i : i / 2], Elem());
        const float hi = kZeros ? fmaxf(both.x, 0.0f) : i % 2 ? both.y : both.x;
        const float lo = kZeros ? fminf(-both.y, 0.0f) : 0.0f;
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
            if (threadIdx.x % kLanes == 0) {
                scales[i * (kThreads / kLanes)] = s16;
                if (kZeros) zeros[i * (kThreads / kLanes)] = uint8_t(int(z));
            }
        }
    }
}

// Words of codes per thread whose loads are in flight together.  HBM-bound on what it writes
// (N = 151936, K = 4096, bf16, group 128: 226 us, 6.9 TB/s).
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
