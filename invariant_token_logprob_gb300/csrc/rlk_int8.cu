// rlk_int8.cu -- a matrix in 8-bit whole numbers with an fp32 scale per row, and back:
//   s = max|x| / 127 (1 for a row of zeros),  q = clamp(rint(x / s), -127, 127),  x ~ s q
// with fp32 divisions, for weights (a scale per channel) and for tokens (a scale per token).
//
// The quotient decides a code at its ties, so it has to be the IEEE one: from the correctly
// rounded reciprocal r, q = x r, its remainder e = fma(-q, s, x) and the correction fma(e, r, q)
// (Markstein's step).  Where s is tiny (below 2^-64; r, and products with it, could leave the
// range of normal numbers) the division itself is taken.  rint is the addition of 1.5 2^23,
// which leaves the whole number in the low bits, in two's complement.
//
// What bounds it: HBM, 3 bytes per 16-bit element.  A row stays in registers between the
// maximum and the codes (16 vectors of 16 bytes per lane): in one warp's where rows are many, in
// eight warps' where they are few or long.
// Measured for N = 151936, K = 4096, bf16: codes and scales 259 us (7.2 TB/s, 1.06 of a copy, whose
// bytes are written by half, not by a third), read back as bf16 266 us.
#include "rlk_logits.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train_int8.h"

namespace rlk {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 16;  // vectors of 16 bytes that a lane holds
constexpr float kSmallScale = 5.421010862427522e-20f;  // 2^-64
constexpr float kRint = 12582912.0f;                   // 1.5 2^23

__device__ __forceinline__ float scale_of(float amax) {
    const float s = __fdiv_rn(amax, 127.0f);
    return s > 0.0f ? s : 1.0f;
}

__device__ __forceinline__ uint32_t pack_pair(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&two);
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b, __half) {
    const __half2 two = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&two);
}

// A vector's elements as fp32.
template <typename Elem>
__device__ __forceinline__ void to_floats(const uint4& v, float (&f)[kVecElems<Elem>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(Elem) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else {
            const float2 two = pair_to_float(w[i], Elem());
            f[2 * i] = two.x;
            f[2 * i + 1] = two.y;
        }
    }
}

// The largest magnitude of elements, as they lie in memory: of 16-bit ones by pairs, which keeps
// their fp32 values out of the registers until the codes (146 registers, one row's warps fewer per
// SM, 371 us for N = 151936, K = 4096 otherwise).
template <typename Elem>
struct MaxAbs {
    using Pair = typename PairOf<Elem>::type;
    uint32_t w = 0;
    __device__ __forceinline__ void add(uint32_t x) {
        const uint32_t a = x & 0x7fff7fffu;
        const Pair m = max_pair(*reinterpret_cast<const Pair*>(&w), *reinterpret_cast<const Pair*>(&a));
        w = *reinterpret_cast<const uint32_t*>(&m);
    }
    __device__ __forceinline__ float value() const {
        const float2 f = pair_to_float(w, Elem());
        return fmaxf(f.x, f.y);
    }
};
template <>
struct MaxAbs<float> {
    float m = 0.0f;
    __device__ __forceinline__ void add(uint32_t x) { m = fmaxf(m, fabsf(__uint_as_float(x))); }
    __device__ __forceinline__ float value() const { return m; }
};
template <typename Elem>
__device__ __forceinline__ void add_vector(MaxAbs<Elem>& m, const uint4& v) {
    m.add(v.x);
    m.add(v.y);
    m.add(v.z);
    m.add(v.w);
}

// Two quotients x / s, rounded to whole numbers that stand in the low bits.
template <bool kFast>
__device__ __forceinline__ void two_codes(float a, float b, float s, float r, uint32_t (&q)[2]) {
    float2 v;
    if constexpr (kFast) {
        const F2 x = pack2(a, b), rr = pack2(r, r);
        const F2 q0 = mul2(x, rr);
        const F2 e = fma2(q0, pack2(-s, -s), x);
        v = unpack2(fma2(e, rr, q0));
    } else {
        v = make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s));
    }
    // (|x| <= 127 s (1 + 2^-24), but for scales that were rounded in the range of subnormal numbers)
    q[0] = __float_as_uint(fminf(fmaxf(v.x, -127.0f), 127.0f) + kRint);
    q[1] = __float_as_uint(fminf(fmaxf(v.y, -127.0f), 127.0f) + kRint);
}

// The codes of a vector, as bytes or as fp16 numbers.
template <typename Elem, bool kFast>
__device__ __forceinline__ void store_codes(const uint4& v, float s, float r, __half* dst) {
    constexpr int n = kVecElems<Elem>;
    float f[n];
    to_floats<Elem>(v, f);
    uint32_t words[n / 2];
#pragma unroll
    for (int i = 0; i < n; i += 2) {
        uint32_t q[2];
        two_codes<kFast>(f[i], f[i + 1], s, r, q);
        words[i / 2] = pack_pair(__uint_as_float(q[0]) - kRint, __uint_as_float(q[1]) - kRint, __half());
    }
    if constexpr (n == 8)
        *reinterpret_cast<uint4*>(dst) = make_uint4(words[0], words[1], words[2], words[3]);
    else
        *reinterpret_cast<uint2*>(dst) = make_uint2(words[0], words[1]);
}
template <typename Elem, bool kFast>
__device__ __forceinline__ void store_codes(const uint4& v, float s, float r, int8_t* dst) {
    constexpr int n = kVecElems<Elem>;
    float f[n];
    to_floats<Elem>(v, f);
    uint32_t words[n / 4];
#pragma unroll
    for (int i = 0; i < n; i += 4) {
        uint32_t lo[2], hi[2];
        two_codes<kFast>(f[i], f[i + 1], s, r, lo);
        two_codes<kFast>(f[i + 2], f[i + 3], s, r, hi);
        words[i / 4] = __byte_perm(__byte_perm(lo[0], lo[1], 0x0040),
                                   __byte_perm(hi[0], hi[1], 0x0040), 0x5410);
    }
    if constexpr (n == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(words[0], words[1]);
    else
        *reinterpret_cast<uint32_t*>(dst) = words[0];
}

// kWarps warps per row (1, 2, 4 or 8).  kHeld: the row fits in their registers; else it is read twice.
template <typename Elem, typename Code, int kWarps, bool kHeld>
__global__ void __launch_bounds__(kThreads, sizeof(Elem) == 2 ? 3 : 2)
    quantize_int8_kernel(const uint4* __restrict__ x, int64_t rows, int vecs,
                         Code* __restrict__ codes, float* __restrict__ scales) {
    constexpr int kRows = kThreads / 32 / kWarps;  // per CTA
    constexpr int kLanes = 32 * kWarps;
    constexpr int n = kVecElems<Elem>;
    __shared__ float warp_max[kThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes;
    if (kWarps == 1 && row >= rows) return;
    if (row >= rows) vecs = 0;  // (its warps are there for the barrier)
    const int at = threadIdx.x % kLanes;
    const uint4* src = x + row * vecs;
    uint4 v[kHeld ? kVecs : 1];
    MaxAbs<Elem> largest;
    if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            v[i] = at + i * kLanes < vecs ? __ldg(src + at + i * kLanes) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) add_vector(largest, v[i]);
    } else {
#pragma unroll 8
        for (int i = at; i < vecs; i += kLanes) add_vector(largest, __ldg(src + i));
    }
    float amax = largest.value();
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if constexpr (kWarps > 1) {
        if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            amax = fmaxf(amax, warp_max[threadIdx.x / kLanes * kWarps + w]);
    }
    const float s = scale_of(amax);
    if (at == 0 && row < rows) scales[row] = s;
    Code* dst = codes + row * vecs * n;
    auto store = [&](auto fast) {
        constexpr bool kFast = decltype(fast)::value;
        const float r = kFast ? __frcp_rn(s) : 0.0f;
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (at + i * kLanes < vecs)
                    store_codes<Elem, kFast>(v[i], s, r, dst + (at + i * kLanes) * n);
        } else {
#pragma unroll 4
            for (int i = at; i < vecs; i += kLanes)
                store_codes<Elem, kFast>(__ldg(src + i), s, r, dst + int64_t(i) * n);
        }
    };
    if (s >= kSmallScale)
        store(std::true_type());
    else
        store(std::false_type());
}

// Byte j of `codes`, which hold codes plus 128, as fp32: under the exponent of 2^23, less 2^23 + 128.
__device__ __forceinline__ float code_to_float(uint32_t codes, int j) {
    return __uint_as_float(__byte_perm(codes, 0x4b000000u, 0x7440 + j)) - 8388736.0f;
}

// One warp per row, sixteen vectors of 8 codes per lane in flight, so that a 16-bit output's stores
// are whole lines (16 codes per lane leave half lines per store: 325 us for N = 151936, K = 4096).
template <typename Out>
__global__ void __launch_bounds__(kThreads)
    dequantize_int8_kernel(const uint2* __restrict__ codes, const float* __restrict__ scales,
                           int64_t rows, int vecs, Out* __restrict__ out) {
    const int64_t row = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    if (row >= rows) return;
    const float s = __ldg(scales + row);
    const uint2* src = codes + row * vecs;
    Out* dst = out + row * vecs * 8;
    constexpr int kFlight = 16;
    for (int i0 = threadIdx.x % 32; i0 < vecs; i0 += 32 * kFlight) {
        uint2 v[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
            if (i0 + 32 * f < vecs) v[f] = __ldg(src + i0 + 32 * f);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            if (i0 + 32 * f >= vecs) break;
            const uint32_t w[2] = {v[f].x ^ 0x80808080u, v[f].y ^ 0x80808080u};
            constexpr int kWords = 2 * sizeof(Out);
            uint32_t r[kWords];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float a = __fmul_rn(code_to_float(w[j / 4], j % 4), s);
                const float b = __fmul_rn(code_to_float(w[j / 4], j % 4 + 1), s);
                if constexpr (sizeof(Out) == 4) {
                    r[j] = __float_as_uint(a);
                    r[j + 1] = __float_as_uint(b);
                } else {
                    r[j / 2] = pack_pair(a, b, Out());
                }
            }
            uint4* to = reinterpret_cast<uint4*>(dst + int64_t(i0 + 32 * f) * 8);
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j)
                to[j] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        }
    }
}

// Codes as fp16 numbers, 16 per thread.
__global__ void __launch_bounds__(kThreads)
    widen_int8_kernel(const uint4* __restrict__ codes, int64_t vecs, uint4* __restrict__ out) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= vecs) return;
    const uint4 v = __ldg(codes + i);
    const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u,
                           v.w ^ 0x80808080u};
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 16; j += 2)
        r[j / 2] = pack_pair(code_to_float(w[j / 4], j % 4), code_to_float(w[j / 4], j % 4 + 1), __half());
    out[2 * i] = make_uint4(r[0], r[1], r[2], r[3]);
    out[2 * i + 1] = make_uint4(r[4], r[5], r[6], r[7]);
}

cudaLaunchConfig_t config(int64_t blocks, cudaLaunchAttribute* attr, cudaStream_t stream) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename Elem, typename Code>
cudaError_t quantize(const void* x, int64_t rows, int64_t K, Code* codes, float* scales,
                     cudaStream_t stream) {
    const int vecs = int(K / kVecElems<Elem>);
    // The fewest warps that hold a row have the most bytes in flight each (N = 100000, K = 5152:
    // two warps 231 us, eight 526); eight warps fill the GPU where rows are fewer than some thousands.
    int warps = 1;
    while (warps < 8 && (rows < 2048 || vecs > 32 * kVecs * warps)) warps *= 2;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config((rows * warps + 7) / 8, &attr, stream);
    auto kernel = warps == 1                 ? quantize_int8_kernel<Elem, Code, 1, true>
                  : warps == 2               ? quantize_int8_kernel<Elem, Code, 2, true>
                  : warps == 4               ? quantize_int8_kernel<Elem, Code, 4, true>
                  : vecs <= kThreads * kVecs ? quantize_int8_kernel<Elem, Code, 8, true>
                                             : quantize_int8_kernel<Elem, Code, 8, false>;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint4*>(x), rows, vecs,
                                       codes, scales);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename Code>
cudaError_t quantize_typed(const void* x, ElemType type, int64_t rows, int64_t K, Code* codes,
                           float* scales, cudaStream_t stream) {
    if (type == ElemType::kBf16) return quantize<__nv_bfloat16>(x, rows, K, codes, scales, stream);
    if (type == ElemType::kFp16) return quantize<__half>(x, rows, K, codes, scales, stream);
    return quantize<float>(x, rows, K, codes, scales, stream);
}

}  // namespace

cudaError_t launch_quantize_int8(const void* x, ElemType type, int64_t rows, int64_t K,
                                 int8_t* codes, float* scales, cudaStream_t stream) {
    return quantize_typed(x, type, rows, K, codes, scales, stream);
}

cudaError_t launch_quantize_fp16(const void* x, ElemType type, int64_t rows, int64_t K, void* codes,
                                 float* scales, cudaStream_t stream) {
    return quantize_typed(x, type, rows, K, static_cast<__half*>(codes), scales, stream);
}

cudaError_t launch_widen_int8(const int8_t* codes, int64_t count, void* out, cudaStream_t stream) {
    const int64_t vecs = count / 16;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config((vecs + kThreads - 1) / kThreads, &attr, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, widen_int8_kernel, reinterpret_cast<const uint4*>(codes),
                                       vecs, static_cast<uint4*>(out));
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_dequantize_int8(const int8_t* codes, const float* scales, int64_t N, int64_t K,
                                   void* out, ElemType out_type, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config((N + 7) / 8, &attr, stream);
    const uint2* c = reinterpret_cast<const uint2*>(codes);
    const int vecs = int(K / 8);
    cudaError_t e;
    if (out_type == ElemType::kBf16)
        e = cudaLaunchKernelEx(&cfg, dequantize_int8_kernel<__nv_bfloat16>, c, scales, N, vecs,
                               static_cast<__nv_bfloat16*>(out));
    else if (out_type == ElemType::kFp16)
        e = cudaLaunchKernelEx(&cfg, dequantize_int8_kernel<__half>, c, scales, N, vecs,
                               static_cast<__half*>(out));
    else
        e = cudaLaunchKernelEx(&cfg, dequantize_int8_kernel<float>, c, scales, N, vecs,
                               static_cast<float*>(out));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rlk
