// Residual addition, RMSNorm and Q8_K quantisation in one pass over a row
// (moe_add_rmsnorm):
//   s = x + r,  y = s gamma / sqrt(mean(s^2) + eps),  q = rne(y 127 / amax)
// One CTA per row; each warp owns whole blocks of 256 values (lane L holds
// values 8L..8L+7, the arrangement of the Q8_K quantiser, whose steps it
// repeats on the same fp32 values), so the block maximum is a warp reduction
// and the row's values stay in registers between the two reductions.
//
// Bytes bound: each input is read and each output written once, some 6 flops a
// value.  4096 rows of 4096 (fp32 in, sum and bf16 out) take 34.7 us = 6.8 TB/s, the
// rate of a plain copy.  Few rows are bound by a chain of launch, load, barrier and
// store: one row of 2048 with Q8_K 2.1 us, 333 rows of 4096 5.6 us (3.7 TB/s).
#include <algorithm>

#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.cuh"

namespace moeq4k {
namespace arn {

constexpr int kMaxWarps = 16;

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename TX, typename TY, int kBlocks>  // kBlocks: blocks of 256 a warp holds
__global__ void add_rmsnorm_kernel(const AddNormArgs a) {
    pdl_enter();
    __shared__ float part[kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const size_t row = size_t(blockIdx.x) * a.H;
    const TX *x = static_cast<const TX *>(a.x) + row;
    // gamma with the rest, not after the reduction's barrier, where the registers do not cost
    // occupancy (333 rows of 4096 with Q8_K 6.6 -> 5.7 us; rows of 16384 would lose a tenth)
    constexpr bool kEarly = kBlocks == 1;
    float v[kBlocks][8], g[kBlocks][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int c = (warp + i * nw) * kQK + lane * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (c < a.H) {
            load8(x + c, v[i]);
            if (kEarly) load8(a.gamma + c, g[i]);
            if (a.residual != nullptr) {
                float r[8];
                load8(a.residual + row + c, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    if (a.sum_out != nullptr) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const int c = (warp + i * nw) * kQK + lane * 8;
            if (c < a.H) store8(a.sum_out + row + c, v[i]);
        }
    }
    if (a.y == nullptr && a.q == nullptr) return;
    ss = warp_sum(ss);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    __syncwarp();
    float total = 0.f;
    for (int w = 0; w < nw; ++w) total += part[w];
    const float inv = 1.0f / sqrtf(total / float(a.H) + a.eps);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int b = warp + i * nw;
        const int c = b * kQK + lane * 8;
        if (b * kQK >= a.H) break;
        if (c < a.H) {
            if (!kEarly) load8(a.gamma + c, g[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * g[i][j] * inv;
            if (a.y != nullptr) store8(static_cast<TY *>(a.y) + row + c, v[i]);
        }
        if (a.q == nullptr) continue;
        // the block's Q8_K codes (here H is a multiple of 256, no lane is idle)
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const size_t gb = size_t(blockIdx.x) * (a.H / kQK) + b;
        uint32_t w0 = 0, w1 = 0;
        int sum = 0;
        if (amax != 0.f) {
            const float s = __fdiv_rn(127.f, amax);
            int code[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                code[j] = __float2int_rn(__fmul_rn(v[i][j], s));
                sum += code[j];
            }
            w0 = (uint32_t(code[0]) & 255u) | (uint32_t(code[1]) & 255u) << 8 |
                 (uint32_t(code[2]) & 255u) << 16 | (uint32_t(code[3]) & 255u) << 24;
            w1 = (uint32_t(code[4]) & 255u) | (uint32_t(code[5]) & 255u) << 8 |
                 (uint32_t(code[6]) & 255u) << 16 | (uint32_t(code[7]) & 255u) << 24;
        }
        if (lane == 0) a.d[gb] = amax != 0.f ? __fdiv_rn(amax, 127.f) : 0.f;
        *reinterpret_cast<uint2 *>(a.q + row + c) = make_uint2(w0, w1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if ((lane & 3) == 0) a.sums[gb * (kQK / 32) + (lane >> 2)] = sum;
    }
}

template <typename TX, typename TY>
cudaError_t launch_typed(const AddNormArgs &a, cudaStream_t s) {
    const int blocks = (a.H + kQK - 1) / kQK;
    const int warps = std::min(blocks, blocks <= 8 ? 8 : kMaxWarps);
    const int per = (blocks + warps - 1) / warps;
    const dim3 grid(a.T), block(32 * warps);
    if (per <= 1)
        return launch_pdl(add_rmsnorm_kernel<TX, TY, 1>, grid, block, size_t(0), s, a);
    if (per <= 2)
        return launch_pdl(add_rmsnorm_kernel<TX, TY, 2>, grid, block, size_t(0), s, a);
    return launch_pdl(add_rmsnorm_kernel<TX, TY, 4>, grid, block, size_t(0), s, a);
}

template <typename TX>
cudaError_t launch_x(const AddNormArgs &a, cudaStream_t s) {
    switch (a.y == nullptr ? MOE_F32 : a.y_type) {
        case MOE_F16: return launch_typed<TX, __half>(a, s);
        case MOE_BF16: return launch_typed<TX, __nv_bfloat16>(a, s);
        default: return launch_typed<TX, float>(a, s);
    }
}

}  // namespace arn

cudaError_t launch_add_rmsnorm(const AddNormArgs &a, cudaStream_t s) {
    switch (a.x_type) {
        case MOE_F16: return arn::launch_x<__half>(a, s);
        case MOE_BF16: return arn::launch_x<__nv_bfloat16>(a, s);
        default: return arn::launch_x<float>(a, s);
    }
}

}  // namespace moeq4k
