// rlk_logits.cuh -- reading rows of logits (bf16, fp16 or fp32) eight elements at a
// time with 16-byte loads, whatever the row's alignment.
//
// A row starts some elements behind a 16-byte boundary (an odd vocabulary puts rows at
// every alignment).  Which elements a lane handles must not depend on that -- the order of
// the sums, hence a row's bits, would -- so eight elements e0 .. e0 + 7 with e0 a multiple
// of 8 are always taken together: from the aligned vectors that cover them, one more than
// they fill where the row is not aligned (its line is the neighbouring lane's, so it costs
// an L1 hit, no memory traffic), shifted in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace rlk {

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

__device__ __forceinline__ float2 pair_to_float(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_to_float(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Elements in 16 bytes.
template <typename Elem>
constexpr int kVecElems = 16 / int(sizeof(Elem));

__device__ __forceinline__ __nv_bfloat162 max_pair(__nv_bfloat162 a, __nv_bfloat162 b) {
    return __hmax2(a, b);
}
__device__ __forceinline__ __half2 max_pair(__half2 a, __half2 b) { return __hmax2(a, b); }
template <typename Elem>
struct PairOf;
template <>
struct PairOf<__nv_bfloat16> {
    using type = __nv_bfloat162;
};
template <>
struct PairOf<__half> {
    using type = __half2;
};

// The pattern of -inf, twice for a 16-bit type.
__device__ __forceinline__ uint32_t minus_inf(float) { return 0xff800000u; }
__device__ __forceinline__ uint32_t minus_inf(__half) { return 0xfc00fc00u; }
__device__ __forceinline__ uint32_t minus_inf(__nv_bfloat16) { return 0xff80ff80u; }

// Eight elements as they lie in memory.
template <typename Elem>
struct Packed8 {
    static constexpr int kWords = 2 * int(sizeof(Elem));
    uint32_t w[kWords];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < kWords; ++j) w[j] = minus_inf(Elem());
    }
    // Elements e0 .. of a row of V, -inf behind its end, one load each.
    __device__ __forceinline__ void load_single(const Elem* row, int64_t e0, int64_t V) {
        clear();
        if constexpr (sizeof(Elem) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < V) w[j] = __float_as_uint(row[e0 + j]);
        } else {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < V) {
                    const uint32_t h = r[e0 + j];
                    w[j / 2] = j & 1 ? (w[j / 2] & 0xffffu) | (h << 16) : (w[j / 2] & 0xffff0000u) | h;
                }
        }
    }
    // -inf where the bit of `bits` is not set.
    __device__ __forceinline__ void keep(uint32_t bits) {
        if constexpr (sizeof(Elem) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = (bits >> j) & 1u ? w[j] : minus_inf(Elem());
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = (bits >> (2 * j)) & 3u;
                const uint32_t mask = (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
                w[j] = (w[j] & mask) | (minus_inf(Elem()) & ~mask);
            }
        }
    }
    __device__ __forceinline__ float2 pair(int j) const {
        if constexpr (sizeof(Elem) == 4)
            return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        else
            return pair_to_float(w[j], Elem());
    }
    // The largest that is not a NaN (-inf or a NaN if there is none).
    __device__ __forceinline__ float max() const {
        if constexpr (sizeof(Elem) == 4) {
            const float a = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                                  __uint_as_float(w[2]));
            const float b = fmaxf(fmaxf(__uint_as_float(w[3]), __uint_as_float(w[4])),
                                  __uint_as_float(w[5]));
            return fmaxf(fmaxf(fmaxf(a, b), __uint_as_float(w[6])), __uint_as_float(w[7]));
        } else {
            using P = typename PairOf<Elem>::type;
            const P* p = reinterpret_cast<const P*>(w);
            const P m = max_pair(max_pair(p[0], p[1]), max_pair(p[2], p[3]));
            const float2 f = pair_to_float(*reinterpret_cast<const uint32_t*>(&m), Elem());
            return fmaxf(f.x, f.y);
        }
    }
};

// The aligned vectors that cover eight elements e0 .. e0 + 7 of a row that starts `shift`
// elements behind a 16-byte boundary (not kShifted: shift is 0).
template <typename Elem, bool kShifted>
struct Vectors {
    static constexpr int E = kVecElems<Elem>;
    static constexpr int kVecs = 8 / E + (kShifted ? 1 : 0);
    uint4 v[kVecs];

    // Whether they lie inside a row of V elements.
    static __device__ __forceinline__ bool inside(int64_t e0, int shift, int64_t V) {
        return !kShifted ? e0 + 8 <= V : (e0 >= shift && e0 - shift + kVecs * E <= V);
    }
    __device__ __forceinline__ void load(const Elem* row, int64_t e0, int shift) {
        const uint4* q = reinterpret_cast<const uint4*>(row + e0 - (kShifted ? shift : 0));
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = q[i];
    }
    __device__ __forceinline__ uint32_t word(int i) const {  // i-th 32-bit word of the vectors
        const uint4& u = v[i / 4];
        return i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w;
    }
    template <int A>
    __device__ __forceinline__ void get(Packed8<Elem>& r) const {
        if constexpr (sizeof(Elem) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.w[j] = word(A + j);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r.w[j] = (A & 1) ? __funnelshift_r(word(A / 2 + j), word(A / 2 + j + 1), 16)
                                 : word(A / 2 + j);
        }
    }
};

// The eight elements of each of N groups out of their vectors (kShifted: any shift, 0 too).
// The amount of the shift
// picks one of a few short pieces of code that only move registers, not a copy of the
// caller: an odd vocabulary has rows of every shift on an SM at once, and copies of a whole
// loop for each would not stay in the instruction cache.
template <typename Elem, bool kShifted, int N>
__device__ __forceinline__ void unshift(const Vectors<Elem, kShifted> (&in)[N], int shift,
                                        Packed8<Elem> (&x)[N]) {
    auto all = [&](auto a) {
#pragma unroll
        for (int i = 0; i < N; ++i) in[i].template get<decltype(a)::value>(x[i]);
    };
    if constexpr (!kShifted) {
        all(std::integral_constant<int, 0>());
    } else if constexpr (sizeof(Elem) == 4) {
        switch (shift) {
            case 0: all(std::integral_constant<int, 0>()); break;
            case 1: all(std::integral_constant<int, 1>()); break;
            case 2: all(std::integral_constant<int, 2>()); break;
            default: all(std::integral_constant<int, 3>()); break;
        }
    } else {
        switch (shift) {
            case 0: all(std::integral_constant<int, 0>()); break;
            case 1: all(std::integral_constant<int, 1>()); break;
            case 2: all(std::integral_constant<int, 2>()); break;
            case 3: all(std::integral_constant<int, 3>()); break;
            case 4: all(std::integral_constant<int, 4>()); break;
            case 5: all(std::integral_constant<int, 5>()); break;
            case 6: all(std::integral_constant<int, 6>()); break;
            default: all(std::integral_constant<int, 7>()); break;
        }
    }
}

// The larger of a and the elements of one vector that are not NaN.
template <typename Elem>
__device__ __forceinline__ float max_of(float a, const uint4& v) {
    if constexpr (sizeof(Elem) == 4) {
        return fmaxf(fmaxf(fmaxf(a, __uint_as_float(v.x)), fmaxf(__uint_as_float(v.y), __uint_as_float(v.z))),
                     __uint_as_float(v.w));
    } else {
        using P = typename PairOf<Elem>::type;
        const P* p = reinterpret_cast<const P*>(&v);
        const P m = max_pair(max_pair(p[0], p[1]), max_pair(p[2], p[3]));
        const float2 f = pair_to_float(*reinterpret_cast<const uint32_t*>(&m), Elem());
        return fmaxf(a, fmaxf(f.x, f.y));
    }
}

// Elements a row lies behind a 16-byte boundary.
template <typename Elem>
__device__ __forceinline__ int row_shift(const Elem* row) {
    return int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(Elem));
}

}  // namespace rlk
