// 8-bit cache codes on their way to the 16-bit operands of a product: every code
// from -128 to 127 is exact in fp16 and in bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <stdint.h>

namespace moeq4k {

// Two codes of `x` (bytes A and B) as a pair of T.
template <typename T>
struct CodePair;

// fp16: 0x64uu is 1024 + u; with u = code + 128 (its top bit turned) less 1152.
template <>
struct CodePair<__half> {
    uint32_t u;
    __device__ __forceinline__ explicit CodePair(uint32_t x) : u(x ^ 0x80808080u) {}
    template <int A, int B>
    __device__ __forceinline__ uint32_t take() const {
        const uint32_t v = __byte_perm(u, 0x64646464u, A | 4 << 4 | B << 8 | 4 << 12), off = 0x64806480u;
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&off));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

// bf16 has 8 bits of significand: 0x43mm is 128 + m for the code's lower seven bits m, and
// with its sign bit alone (the exponent's last) 128 or 256, which is what is taken off.
template <>
struct CodePair<__nv_bfloat16> {
    uint32_t low, sign;
    __device__ __forceinline__ explicit CodePair(uint32_t x) : low(x & 0x7f7f7f7fu), sign(x & 0x80808080u) {}
    template <int A, int B>
    __device__ __forceinline__ uint32_t take() const {
        constexpr uint32_t sel = A | 4 << 4 | B << 8 | 4 << 12;
        const uint32_t v = __byte_perm(low, 0x43434343u, sel), off = __byte_perm(sign, 0x43434343u, sel);
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&off));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

// Weights times the values' scales, the product's operands, would leave fp16's range.  Each row
// takes them over 2^(e - kLift) of its own, which its sums are multiplied by at the end: 2^e is at or above the
// largest of them (over the row's reference maximum) that the row has seen, so that neither a scale that it does
// not see nor one without weight costs it anything.  As the maximum does, e follows only growth past 2^kGrowth: an
// operand is at most 2^(kLift + 8) = 2^14.
//
// The largest product of a tile is bounded by the largest weight times the largest scale where the scales are
// within 2^4 of one another, and else looked for key by key.  With the roundings up to powers of two e is at most
// 6.1 above it, so what an operand loses below 2^-14, half a step of 2^-24, is at most 2^-24 of the row's largest.
constexpr float kLift = 6.f;
constexpr float kRefLeast = -112.f, kRefMost = 126.f;  // of e: the factors stay normal
constexpr uint32_t kSpread = 4u << 23;                 // as a difference of scales' bits
// The bits of a scale, which rise with it: those of -0.0, the largest otherwise, are 0's.
__device__ __forceinline__ uint32_t scale_bits(float scale) { return __float_as_uint(scale) & 0x7fffffffu; }
constexpr uint32_t kInfinity = 0x7f800000u;  // bits of scales from there on are of an infinity or a NaN
// The exponent of the power of two above a scale (its bits), -inf for 0.
__device__ __forceinline__ float scale_log2(uint32_t bits) {
    return bits == 0u ? -CUDART_INF_F : float(int(bits >> 23) - 126);
}
// e of a row whose largest product and reference maximum have these logarithms.
__device__ __forceinline__ float ref_exponent(float product, float base) {
    return fminf(fmaxf(ceilf(product - base), kRefLeast), kRefMost);
}
// 2^e of an integer e from -126 to 127.
__device__ __forceinline__ float power_of_2(float e) { return __int_as_float((int(e) + 127) << 23); }

}  // namespace moeq4k
