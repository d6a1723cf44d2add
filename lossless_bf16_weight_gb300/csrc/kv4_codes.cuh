// 4-bit codes as operands of BF16 matrix products.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace uw {

// A value the compiler does not know, so that it stays in a register: the
// logic operations below take their masks from registers.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes as pairs of BF16: bits 0..7 of a BF16 on their own are the integer n
// they spell, times 2^-133 (subnormal below 128, the first normal binade
// from there).  So a code in bits 0..3 of a half is c, one in bits 4..7 is 16 c,
// in units of 2^-133, with no shift and no conversion; the queries and
// probabilities they meet are scaled up by kQUp and kPUp.
struct Codes {
    uint32_t mask0 = opaque(0x000f000fu), mask4 = opaque(0x00f000f0u);
    uint32_t mid0 = opaque(0x00080008u), mid4 = opaque(0x00800080u);
    // c and 16 c
    __device__ __forceinline__ uint32_t low(uint32_t w) const { return w & mask0; }
    __device__ __forceinline__ uint32_t high(uint32_t w) const { return w & mask4; }
    // c - 8 and 16 (c - 8), exact
    __device__ __forceinline__ uint32_t low_mid(uint32_t w) const { return sub2(w & mask0, mid0); }
    __device__ __forceinline__ uint32_t high_mid(uint32_t w) const { return sub2(w & mask4, mid4); }
};
constexpr uint32_t kQUpLow = 0x57805780u, kQUpHigh = 0x55805580u;  // 2^48, and 2^44 for the codes times 16
constexpr float kQDown = 3.8685626e25f;                            // 2^85 = 2^133 / 2^48
constexpr float kPUp = 1.8446744e19f;                              // 2^64
constexpr float kPDownLow = 5.9029581e20f, kPDownHigh = 3.6893488e19f;  // 2^69 = 2^133 / 2^64, 2^65

}  // namespace uw
