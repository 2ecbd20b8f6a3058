// 8-bit cache codes on their way to the 16-bit operands of a product: every code
// from -128 to 127 is exact in fp16 and in bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

// fp16 weights times the values' scales would leave the type's range: they are taken
// over a power of two near the largest scale so far, which the sums are multiplied by at the end.
constexpr uint32_t kRefLeast = 0x00800000u, kRefMost = 0x7e800000u;  // 2^-126, 2^126
// The bits of a scale, which rise with it: those of -0.0, the largest otherwise, are 0's.
__device__ __forceinline__ uint32_t scale_bits(float scale) { return __float_as_uint(scale) & 0x7fffffffu; }
// The power of two at or below a scale (its bits), in that range.
__device__ __forceinline__ uint32_t ref_bits(uint32_t scale_bits) {
    return min(max(scale_bits & 0x7f800000u, kRefLeast), kRefMost);
}
__device__ __forceinline__ float over_ref(uint32_t bits) { return __uint_as_float(0x7f000000u - bits); }

}  // namespace moeq4k
