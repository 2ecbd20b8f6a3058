// Attention of new tokens over a paged cache (moe_attention_paged), the plain
// kernel: one warp per (row, query head), lanes over the channels, one pass
// over the keys with the running maximum and sum of the softmax.
#include <algorithm>

#include <math_constants.h>

#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace moeq4k {
namespace attnr {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) attention_rows_kernel(const AttnArgs a) {
    pdl_enter();
    constexpr int kPer = D / 32;  // channels a lane holds: 2 or 4
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.b.B; b += gridDim.x * blockDim.x)
        seq_view(a.b, b, a.hdr, true);
    const int end = a.b.offs[a.b.B];
    const long items = long(a.b.N) * a.b.Hq;
    for (long it = long(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
         it += long(gridDim.x) * kWarps) {
        const int row = int(it / a.b.Hq), h = int(it % a.b.Hq);
        if (row >= end) break;
        int lo = 0, hi = a.b.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.b.offs[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        const SeqView sv = seq_view(a.b, lo, a.hdr, false);
        if (!sv.ok || row < sv.first || row >= sv.first + sv.n) continue;
        const int t = sv.len - sv.n + (row - sv.first);
        const int first = a.window > 0 ? max(0, t - a.window + 1) : 0;
        const int kh = h / (a.b.Hq / a.b.Hkv);
        float q[kPer], o[kPer];
        const uint32_t *qp = reinterpret_cast<const uint32_t *>(
            static_cast<const T *>(a.q) + (size_t(row) * a.b.Hq + h) * D + lane * kPer);
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) {
            const float2 f = Pair<T>::load(qp[i]);
            q[2 * i] = f.x * a.scale, q[2 * i + 1] = f.y * a.scale;
            o[2 * i] = o[2 * i + 1] = 0.f;
        }
        float m = -CUDART_INF_F, l = 0.f;
        int pg = -1;
        for (int j = first; j <= t; ++j) {
            if (j == first || j % a.b.page == 0) pg = page_of(a.b, lo, j, a.hdr);
            if (pg < 0) continue;
            const size_t at = ((size_t(pg) * a.b.Hkv + kh) * a.b.page + j % a.b.page) * D + lane * kPer;
            const uint32_t *kp = reinterpret_cast<const uint32_t *>(static_cast<const T *>(a.k) + at);
            const uint32_t *vp = reinterpret_cast<const uint32_t *>(static_cast<const T *>(a.v) + at);
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) {
                const float2 f = Pair<T>::load(kp[i]);
                z = fmaf(q[2 * i], f.x, z);
                z = fmaf(q[2 * i + 1], f.y, z);
            }
            z = warp_sum(z);
            if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
            const float mn = fmaxf(m, z), c = expf(m - mn), e = expf(z - mn);
            m = mn;
            l = l * c + e;
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) {
                const float2 f = Pair<T>::load(vp[i]);
                o[2 * i] = fmaf(o[2 * i], c, e * f.x);
                o[2 * i + 1] = fmaf(o[2 * i + 1], c, e * f.y);
            }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        uint32_t *op = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) +
                                                    (size_t(row) * a.b.Hq + h) * D + lane * kPer);
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) op[i] = Pair<T>::make(o[2 * i] * inv, o[2 * i + 1] * inv);
        if (a.lse != nullptr && lane == 0)
            a.lse[size_t(row) * a.b.Hq + h] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
    }
}

}  // namespace attnr

cudaError_t launch_attention_rows(const AttnArgs &a, int num_sms, cudaStream_t s) {
    using namespace attnr;
    const long items = long(a.b.N) * a.b.Hq;
    const dim3 grid(unsigned(std::min<long>((items + kWarps - 1) / kWarps, long(num_sms) * 64)));
    const dim3 block(kWarps * 32);
    if (a.type == MOE_F16)
        return a.b.D == 64
                   ? launch_pdl(attention_rows_kernel<__half, 64>, grid, block, size_t(0), s, a)
                   : launch_pdl(attention_rows_kernel<__half, 128>, grid, block, size_t(0), s, a);
    return a.b.D == 64
               ? launch_pdl(attention_rows_kernel<__nv_bfloat16, 64>, grid, block, size_t(0), s, a)
               : launch_pdl(attention_rows_kernel<__nv_bfloat16, 128>, grid, block, size_t(0), s, a);
}

}  // namespace moeq4k
