// Attention over a cache of 16-bit values or of 8-bit codes, with sinks and trees
// (moe_attention_cache), in its plainest form: a CTA per row and query head, a warp
// per key, the softmax's running maximum and sum in fp32.
#include "attention_stream.cuh"

namespace moeq4k {
namespace attn {

constexpr int kPlainWarps = 4;

template <typename T, int D, bool kCodes>
__global__ void __launch_bounds__(32 * kPlainWarps) attention_plain_kernel(const AttnArgs a) {
    constexpr int kPer = D / 32;
    __shared__ float sv[kPlainWarps][D], sm[kPlainWarps], sl[kPlainWarps];
    pdl_enter();
    const int row = blockIdx.x, head = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b = -1;
    SeqView s = {};
    for (int i = 0; i < a.b.B; ++i) {
        const SeqView v = seq_view(a.b, i, a.hdr, threadIdx.x == 0);
        if (v.ok && row >= v.first && row < v.first + v.n) {
            b = i;
            s = v;
        }
    }
    if (b < 0) return;
    const int base = s.len - s.n, own = base + row - s.first, kh = head / (a.b.Hq / a.b.Hkv);
    const uint32_t *bits = a.tree != nullptr ? a.tree + size_t(row) * a.words : nullptr;
    int at = own;
    if (bits != nullptr) {
        int m = 0;
        for (int i = 0; i < min(s.n, 32 * a.words); ++i) m += bits[i >> 5] >> (i & 31) & 1;
        at = base + max(m, 1) - 1;
    }
    float q[kPer], o[kPer], top = -CUDART_INF_F, sum = 0.f;
    for (int c = 0; c < kPer; ++c) {
        q[c] = float(static_cast<const T *>(a.q)[(size_t(row) * a.b.Hq + head) * D + lane * kPer + c]);
        o[c] = 0.f;
    }
    for (int key = warp; own >= 0 && key < s.len; key += kPlainWarps) {
        bool sees = key <= (bits != nullptr ? base - 1 : at);
        if (a.window > 0 && at - key >= a.window && key >= a.sinks) sees = false;
        if (bits != nullptr && key >= base) {
            const int i = key - base;
            sees = i < 32 * a.words && (bits[i >> 5] >> (i & 31) & 1) != 0;
        }
        if (!sees) continue;
        const int pg = page_of(a.b, b, key, a.hdr);
        if (pg < 0) continue;
        const size_t at_row = (size_t(pg) * a.b.Hkv + kh) * a.b.page + key % a.b.page;
        float k[kPer], v[kPer], ks = 1.f, vs = 1.f;
        for (int c = 0; c < kPer; ++c) {
            const size_t i = at_row * D + lane * kPer + c;
            if (kCodes) {
                k[c] = float(static_cast<const int8_t *>(a.k)[i]);
                v[c] = float(static_cast<const int8_t *>(a.v)[i]);
            } else {
                k[c] = float(static_cast<const T *>(a.k)[i]);
                v[c] = float(static_cast<const T *>(a.v)[i]);
            }
        }
        if (kCodes) ks = a.ks[at_row], vs = a.vs[at_row];
        float z = 0.f;
        for (int c = 0; c < kPer; ++c) z = fmaf(q[c], k[c], z);
        for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
        z *= ks * a.scale;
        if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
        const float up = fmaxf(top, z), f = expf(top - up), p = expf(z - up);
        top = up;
        sum = fmaf(sum, f, p);
        for (int c = 0; c < kPer; ++c) o[c] = fmaf(p * vs, v[c], o[c] * f);
    }
    for (int c = 0; c < kPer; ++c) sv[warp][lane * kPer + c] = o[c];
    if (lane == 0) sm[warp] = top, sl[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < kPlainWarps; ++w) top = fmaxf(top, sm[w]);
    sum = 0.f;
    for (int c = 0; c < kPer; ++c) o[c] = 0.f;
    for (int w = 0; w < kPlainWarps; ++w) {
        const float f = top == -CUDART_INF_F ? 0.f : expf(sm[w] - top);
        sum = fmaf(sl[w], f, sum);
        for (int c = 0; c < kPer; ++c) o[c] = fmaf(sv[w][lane * kPer + c], f, o[c]);
    }
    const size_t out = size_t(row) * a.b.Hq + head;
    for (int c = 0; c < kPer; ++c) static_cast<T *>(a.out)[out * D + lane * kPer + c] = T(o[c] * over_sum(sum));
    if (a.lse != nullptr && lane == 0) a.lse[out] = sum == 0.f ? -CUDART_INF_F : top + logf(sum);
}

}  // namespace attn

cudaError_t launch_attention_cache(const AttnArgs &a, int max_new, int num_sms, cudaStream_t s) {
    using namespace attn;
    if (a.ks == nullptr)
        return launch_attention(a, max_new, num_sms, s);
    if (long(max_new) * (a.b.Hq / a.b.Hkv) <= kMaxRows) return launch_stream_codes(a, make_params(a), num_sms, s);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(a.b.N, a.b.Hq), dim3(32 * kPlainWarps), size_t(0), s, a);
    };
    auto of = [&](auto type) {
        using T = decltype(type);
        if (a.ks != nullptr)
            return a.b.D == 64 ? go(attention_plain_kernel<T, 64, true>) : go(attention_plain_kernel<T, 128, true>);
        return a.b.D == 64 ? go(attention_plain_kernel<T, 64, false>) : go(attention_plain_kernel<T, 128, false>);
    };
    return a.type == MOE_F16 ? of(__half()) : of(__nv_bfloat16());
}

}  // namespace moeq4k
