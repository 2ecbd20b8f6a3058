// Per-head RMSNorm, rotary positions and the append to a paged cache
// (moe_rope_append).  Pair (a, b) of channel j turns by the angle
// pos[axis[j]] * inv_freq[j]:  (a cos - b sin, b cos + a sin).
//
// The angle is kept in turns as a 64-bit binary fraction: F_j = inv_freq_j /
// 2 pi mod 1, times 2^64, and pos * F_j wraps modulo 2^64, which is the exact
// reduction modulo a turn: the error is that of F_j (an fp64 product) times
// pos, as in fp64, at a 64-bit integer product a pair.  F_j is worked out once per
// CTA, sine and cosine once per token and channel, for all its heads.
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace moeq4k {
namespace rope {

constexpr int kMaxPairs = 64;  // D / 2
constexpr int kMaxThreads = 512;

// 2^64 times the fraction of a turn per position.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    double t = f * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    // 63 bits fit the conversion whatever t rounds to (t = 1 wraps to 0)
    return static_cast<unsigned long long>(__double2ll_rn(t * 4611686018427387904.0)) << 2;
}

// Thread: 16 channels of one head at a time (chunk c of D / 16): 8 pairs of a
// rotated chunk, or 16 plain channels.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) rope_append_kernel(const RopeArgs a) {
    pdl_enter();
    __shared__ unsigned long long frac[kMaxPairs];
    __shared__ int axis_sh[kMaxPairs];
    __shared__ float2 cs[kMaxPairs];  // (cos, sin)
    const int half = a.rot / 2, D = a.b.D, per = D / 16, heads = a.b.Hq + 2 * a.b.Hkv;
    for (int j = threadIdx.x; j < half; j += blockDim.x) {
        frac[j] = turn_fraction(a.inv_freq[j]);
        int ax = a.axis != nullptr ? a.axis[j] : 0;
        if (ax < 0 || ax >= a.axes) {
            if (blockIdx.x == 0) record_status(a.hdr, MOE_ERR_CACHE_RANGE, ax);
            ax = 0;
        }
        axis_sh[j] = ax;
    }
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.b.B; b += gridDim.x * blockDim.x)
        seq_view(a.b, b, a.hdr, true);  // records sequences out of range
    const int end = a.b.offs[a.b.B];
    for (int row = blockIdx.x; row < a.b.N; row += gridDim.x) {
        if (row >= end) break;  // rows of no sequence
        // the last sequence that starts at or before the row
        int lo = 0, hi = a.b.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.b.offs[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        const SeqView sv = seq_view(a.b, lo, a.hdr, false);
        if (!sv.ok || row < sv.first || row >= sv.first + sv.n) continue;
        const int at = sv.len - sv.n + (row - sv.first);  // cache index
        const int pg = at >= 0 ? page_of(a.b, lo, at, a.hdr) : -1;
        __syncthreads();  // frac written; the last row's cs read
        for (int j = threadIdx.x; j < half; j += blockDim.x) {
            const long long pos = a.pos[size_t(axis_sh[j]) * a.b.N + row];
            const long long turn = static_cast<long long>(static_cast<unsigned long long>(pos) * frac[j]);
            // the top 32 bits (rounded): a signed fraction of a turn, in half turns for sincospi
            const int top = static_cast<int>((turn + 0x80000000ll) >> 32);
            float c, s;
            sincospif(float(top) * 4.6566128730773926e-10f, &s, &c);  // * 2^-31
            cs[j] = make_float2(c, s);
        }
        __syncthreads();
        const T *src_row = static_cast<const T *>(a.qkv) + size_t(row) * heads * D;
        const int tasks = heads * per;
        // whole groups of D / 16 lanes take a head each; every lane of a warp
        // runs the same number of turns, so the shuffles below are complete
        const int turns = (tasks + blockDim.x - 1) / blockDim.x;
        for (int u = 0; u < turns; ++u) {
            const int task = u * blockDim.x + threadIdx.x;
            const bool live = task < tasks;
            const int head = live ? task / per : 0, c = task % per;
            // first and second 8 channels of this thread's 16
            int c0 = 16 * c, c1 = 16 * c + 8;
            const bool turned = head < a.b.Hq + a.b.Hkv && 16 * c < a.rot;
            if (!a.interleaved && 16 * c < a.rot) {
                c0 = 8 * c;
                c1 = 8 * c + half;
            }
            float v[16];
            uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
            if (live) {
                w0 = *reinterpret_cast<const uint4 *>(src_row + size_t(head) * D + c0);
                w1 = *reinterpret_cast<const uint4 *>(src_row + size_t(head) * D + c1);
            }
            const uint32_t in[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = Pair<T>::load(in[i]);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
                ss = fmaf(f.x, f.x, ss);
                ss = fmaf(f.y, f.y, ss);
            }
            const float *nw = head < a.b.Hq ? a.qw : head < a.b.Hq + a.b.Hkv ? a.kw : nullptr;
            for (int o = per >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (nw != nullptr) {
                const float inv = 1.0f / sqrtf(ss / float(D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = v[i] * nw[c0 + i] * inv;
                    v[8 + i] = v[8 + i] * nw[c1 + i] * inv;
                }
            }
            if (turned) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 t = cs[8 * c + i];
                    float &x = a.interleaved ? v[2 * i] : v[i];
                    float &y = a.interleaved ? v[2 * i + 1] : v[8 + i];
                    const float p = x * t.x - y * t.y, q = y * t.x + x * t.y;
                    x = p;
                    y = q;
                }
            }
            T *dst = nullptr;
            if (head < a.b.Hq) {
                dst = static_cast<T *>(a.q_out) + (size_t(row) * a.b.Hq + head) * D;
            } else if (pg >= 0) {
                const bool key = head < a.b.Hq + a.b.Hkv;
                const int kh = head - a.b.Hq - (key ? 0 : a.b.Hkv);
                dst = static_cast<T *>(key ? a.k : a.v) +
                      ((size_t(pg) * a.b.Hkv + kh) * a.b.page + at % a.b.page) * D;
            }
            if (live && dst != nullptr) {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = Pair<T>::make(v[2 * i], v[2 * i + 1]);
                *reinterpret_cast<uint4 *>(dst + c0) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(dst + c1) = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

}  // namespace rope

cudaError_t launch_rope_append(const RopeArgs &a, int num_sms, cudaStream_t s) {
    using namespace rope;
    const int tasks = (a.b.Hq + 2 * a.b.Hkv) * (a.b.D / 16);
    const int turns = (tasks + kMaxThreads - 1) / kMaxThreads;
    const int threads = ((tasks + turns - 1) / turns + 31) / 32 * 32;
    const dim3 grid(std::min(a.b.N, num_sms * 8)), block(std::max(threads, 64));
    if (a.type == MOE_F16)
        return launch_pdl(rope_append_kernel<__half>, grid, block, size_t(0), s, a);
    return launch_pdl(rope_append_kernel<__nv_bfloat16>, grid, block, size_t(0), s, a);
}

}  // namespace moeq4k
