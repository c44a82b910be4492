// rlk_w4.cuh -- codes of a 4-bit weight as numbers (the format: rlk_w4.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace rlk {

// (a & mask) | set in one instruction: with both constants as immediates it would be two,
// and this is the instruction the whole kernel waits for.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t set) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(mask), "r"(set));
    return r;
}

// Eight codes as pairs of numbers kUnit (q - z) in 16 bits, exactly.  A code in the low places
// of a constant's pattern adds its value to the constant: the multiply-add that subtracts the
// constant and the zero point brings the unit along.  A code four places higher needs no shift:
// fp16's 1024 has room for it too (16 q).  (For fp16, with the even codes apart from the odd
// ones, a published method: Y. J. Kim et al., Who Says Elephants Can't Run, 2022.)  In bf16
// the bare bits are a subnormal number, 16 q * 2^-133, that 2^127 brings to q / 4.  So a
// word takes one shift and four cuts; the integer pipe's time goes into nothing else.
template <typename Elem>
struct Numbers;
template <>
struct Numbers<__nv_bfloat16> {
    static constexpr float kUnit = 0.25f;
    uint32_t less_low, less_high;  // -(32 + z / 4) and -z / 4, twice
    __device__ __forceinline__ explicit Numbers(uint32_t zero) {
        less_low = 0xc200c200u + zero * 0x00010001u;  // (the last place of 32 is 1/4)
        less_high = fma(0x43004300u + zero * 0x00010001u, 0xbe80be80u, 0x42004200u);  // 32 - (128 + z)/4
    }
    static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    __device__ __forceinline__ void pair(uint32_t v, uint32_t& low, uint32_t& high) const {
        low = fma(and_or(v, 0x000f000fu, 0x43004300u), 0x3e803e80u, less_low);  // (128 + q) / 4
        high = fma(v & 0x00f000f0u, 0x7f007f00u, less_high);                    // times 2^127
    }
};
template <>
struct Numbers<__half> {
    static constexpr float kUnit = 1.0f;
    uint32_t less_low, less_high;  // -(1024 + z) and -(64 + z), twice
    __device__ __forceinline__ explicit Numbers(uint32_t zero) {
        less_low = 0xe400e400u + zero * 0x00010001u;
        less_high = 0xd400d400u + zero * 0x00100010u;  // (that of 64 is 1/16)
    }
    static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    __device__ __forceinline__ void pair(uint32_t v, uint32_t& low, uint32_t& high) const {
        low = fma(and_or(v, 0x000f000fu, 0x64006400u), 0x3c003c00u, less_low);    // 1024 + q
        high = fma(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, less_high);  // (1024 + 16 q) / 16
    }
};

}  // namespace rlk
