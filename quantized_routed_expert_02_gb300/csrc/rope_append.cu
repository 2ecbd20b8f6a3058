// Per-head RMSNorm, rotary positions and the append to a paged cache
// (moe_rope_append).  Pair (a, b) of channel j turns by the angle
// pos[axis[j]] * inv_freq[j]:  (a cos - b sin, b cos + a sin).
//
// The angle is kept in turns as a 64-bit binary fraction: F_j = inv_freq_j /
// 2 pi mod 1, times 2^64, and pos * F_j wraps modulo 2^64, which is the exact
// reduction modulo a turn: the error is that of F_j (an fp64 product) times
// pos, as in fp64, at a 64-bit integer product a pair.
//
// Bytes bound (every row read once and written once) as long as the arithmetic
// stays small: a warp takes a row (or, with few rows, a share of its heads),
// works out the row's sines once and keeps each lane's eight pairs in registers
// for all the row's heads, so that a head costs its loads, packed fp32 arithmetic
// and its stores, with no barrier.
#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace moeq4k {
namespace rope {

constexpr int kMaxPairs = 64;  // D / 2
constexpr int kWarps = 4;
constexpr int kCtas = 4;       // on an SM
constexpr int kBatch = 4;      // heads' chunks that a lane has in flight

// 2^64 times the fraction of a turn per position.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    double t = f * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    // 63 bits fit the conversion whatever t rounds to (t = 1 wraps to 0)
    return static_cast<unsigned long long>(__double2ll_rn(t * 4611686018427387904.0)) << 2;
}

// The last sequence that starts at or before `row`, found by a whole warp in
// steps of 32 ways.
__device__ __forceinline__ int find_seq(const PagedBatch &p, int row, int lane) {
    int lo = 0, n = p.B;  // among [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const unsigned before = __ballot_sync(0xffffffffu, b < lo + n && p.offs[b] <= row);
        const int last = before == 0u ? 0 : 31 - __clz(before);
        const int at = lo + last * step;
        n = min(step, lo + n - at);
        lo = at;
    }
    return lo;
}

// A warp takes units of (row, share of its heads): `shares` of `share` heads
// each.  Lane: chunk c = lane % (D / 16) of a head at a time, kBatch of them
// loaded together: the channels 8 c .. 8 c + 7 and the 8 they pair with (rotated
// halves), or 16 in a row.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, kCtas) rope_append_kernel(const RopeArgs a, int shares, int share) {
    __shared__ __align__(16) float co_sh[kWarps][kMaxPairs], si_sh[kWarps][kMaxPairs];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = a.rot / 2, D = a.b.D, per = D / 16;
    const int Hq = a.b.Hq, Hkv = a.b.Hkv, heads = Hq + 2 * Hkv;
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.b.B; b += gridDim.x * blockDim.x)
        seq_view(a.b, b, a.hdr, true);  // records sequences out of range
    // this lane's two angles of a row
    unsigned long long frac[2];
    int axis[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = lane + 32 * k;
        frac[k] = j < half ? turn_fraction(a.inv_freq[j]) : 0ull;
        axis[k] = a.axis != nullptr && j < half ? a.axis[j] : 0;
        if (axis[k] < 0 || axis[k] >= a.axes) {
            if (blockIdx.x == 0) record_status(a.hdr, MOE_ERR_CACHE_RANGE, axis[k]);
            axis[k] = 0;
        }
    }
    const int c = lane % per, sub = lane / per, step = 32 / per;
    const bool in_rot = 16 * c < a.rot, norms = a.qw != nullptr || a.kw != nullptr;
    const bool split = in_rot && !kInterleaved;
    const int c0 = split ? 8 * c : 16 * c, c1 = split ? 8 * c + half : 16 * c + 8;
    const long units = long(a.b.N) * shares;
    for (long un = long(blockIdx.x) * kWarps + warp; un < units; un += long(gridDim.x) * kWarps) {
        const int row = int(un / shares), h0 = int(un - long(row) * shares) * share, h1 = min(heads, h0 + share);
        const T *src = static_cast<const T *>(a.qkv) + size_t(row) * heads * D;
        uint4 in[kBatch][2];
        auto load = [&](int h) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int u = h + k * step + sub;
                in[k][0] = in[k][1] = make_uint4(0, 0, 0, 0);
                if (u < h1) {
                    in[k][0] = *reinterpret_cast<const uint4 *>(src + size_t(u) * D + c0);
                    in[k][1] = *reinterpret_cast<const uint4 *>(src + size_t(u) * D + c1);
                }
            }
        };
        load(h0);  // under way while the row's place and sines are worked out
        int pos[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) pos[k] = a.pos[size_t(axis[k]) * a.b.N + row];
        const int b = find_seq(a.b, row, lane);
        const SeqView sv = seq_view(a.b, b, a.hdr, false);
        if (!sv.ok || row < sv.first || row >= sv.first + sv.n) continue;  // a row of no sequence
        const int at = sv.len - sv.n + (row - sv.first);                    // cache index
        long cache = -1;  // the first key/value head's cache row
        if (at >= 0) {
            const int pg = page_of(a.b, b, at, a.hdr);
            if (pg >= 0) cache = long(pg) * Hkv * a.b.page + at % a.b.page;
        }
        __syncwarp();  // the unit before has read its sines
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long turn = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(pos[k])) * frac[k]);
            // the top 32 bits (rounded): a signed fraction of a turn, in half turns for sincospi
            const int top = static_cast<int>((turn + 0x80000000ll) >> 32);
            sincospif(float(top) * 4.6566128730773926e-10f, &si_sh[warp][lane + 32 * k], &co_sh[warp][lane + 32 * k]);  // * 2^-31
        }
        __syncwarp();
        // two pairs at a time: cosines, sines, negated sines
        unsigned long long co[4], si[4], ni[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = in_rot ? 8 * c + 4 * i : 0;
            const float4 x = *reinterpret_cast<const float4 *>(&co_sh[warp][j]);
            const float4 y = *reinterpret_cast<const float4 *>(&si_sh[warp][j]);
            co[2 * i] = pack2(x.x, x.y), co[2 * i + 1] = pack2(x.z, x.w);
            si[2 * i] = pack2(y.x, y.y), si[2 * i + 1] = pack2(y.z, y.w);
            ni[2 * i] = pack2(-y.x, -y.y), ni[2 * i + 1] = pack2(-y.z, -y.w);
        }
        for (int h = h0; h < h1; h += kBatch * step) {
            if (h > h0) load(h);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (h + k * step >= h1) break;
                const int head = min(h + k * step + sub, h1 - 1);  // no lane leaves before the sum of squares
                const bool mine = h + k * step + sub < h1;
                const uint32_t w[8] = {in[k][0].x, in[k][0].y, in[k][0].z, in[k][0].w,
                                       in[k][1].x, in[k][1].y, in[k][1].z, in[k][1].w};
                unsigned long long v[8];  // channels two at a time: c0 .., then c1 ..
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = Pair<T>::load(w[i]);
                    v[i] = pack2(f.x, f.y);
                }
                const bool query = head < Hq, value = head >= Hq + Hkv;
                if (norms) {
                    unsigned long long s2[2] = {0ull, 0ull};
#pragma unroll
                    for (int i = 0; i < 8; ++i) s2[i & 1] = fma2(v[i], v[i], s2[i & 1]);
                    float sa, sb;
                    unpack2(add2(s2[0], s2[1]), sa, sb);
                    float ss = sa + sb;
                    for (int o = per >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float *nw = query ? a.qw : value ? nullptr : a.kw;
                    if (nw != nullptr) {
                        const float inv = 1.0f / sqrtf(ss / float(D) + a.eps);
                        const unsigned long long inv2 = pack2(inv, inv);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float4 x = __ldg(reinterpret_cast<const float4 *>(nw + (i < 4 ? c0 + 2 * i : c1 + 2 * i - 8)));
                            v[i] = mul2(mul2(v[i], pack2(x.x, x.y)), inv2);
                            v[i + 1] = mul2(mul2(v[i + 1], pack2(x.z, x.w)), inv2);
                        }
                    }
                }
                if (in_rot && !value) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kInterleaved) {  // channels (4 i, 4 i + 1), (4 i + 2, 4 i + 3): pairs 2 i, 2 i + 1
                            float cx, cy, sx, sy, x, y;
                            unpack2(co[i], cx, cy);
                            unpack2(si[i], sx, sy);
                            unpack2(v[2 * i], x, y);
                            v[2 * i] = pack2(x * cx - y * sx, y * cx + x * sx);
                            unpack2(v[2 * i + 1], x, y);
                            v[2 * i + 1] = pack2(x * cy - y * sy, y * cy + x * sy);
                        } else {
                            const unsigned long long x = v[i], y = v[4 + i];
                            v[i] = fma2(y, ni[i], mul2(x, co[i]));
                            v[4 + i] = fma2(x, si[i], mul2(y, co[i]));
                        }
                    }
                }
                T *dst = nullptr;
                if (query) {
                    dst = static_cast<T *>(a.q_out) + (size_t(row) * Hq + head) * D;
                } else if (cache >= 0) {
                    const int kh = value ? head - Hq - Hkv : head - Hq;
                    dst = static_cast<T *>(value ? a.v : a.k) + (cache + long(kh) * a.b.page) * D;
                }
                if (mine && dst != nullptr) {
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float x, y;
                        unpack2(v[i], x, y);
                        o[i] = Pair<T>::make(x, y);
                    }
                    *reinterpret_cast<uint4 *>(dst + c0) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(dst + c1) = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
        }
    }
}

}  // namespace rope

cudaError_t launch_rope_append(const RopeArgs &a, int num_sms, cudaStream_t s) {
    using namespace rope;
    // few rows: a row's heads are shared out until every SM has its warps; a
    // share is whole steps of 512 / D heads (what a warp turns at a time)
    const int heads = a.b.Hq + 2 * a.b.Hkv, step = 512 / a.b.D, warps = num_sms * kCtas * kWarps;
    const int most = (heads + step - 1) / step;
    int shares = std::min(most, std::max(1, warps / a.b.N));
    const int share = (most + shares - 1) / shares * step;
    shares = (heads + share - 1) / share;
    const long units = long(a.b.N) * shares;
    const dim3 grid(unsigned(std::min<long>((units + kWarps - 1) / kWarps, long(num_sms) * kCtas))), block(kWarps * 32);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, size_t(0), s, a, shares, share); };
    if (a.type == MOE_F16) return a.interleaved ? go(rope_append_kernel<__half, true>) : go(rope_append_kernel<__half, false>);
    return a.interleaved ? go(rope_append_kernel<__nv_bfloat16, true>) : go(rope_append_kernel<__nv_bfloat16, false>);
}

}  // namespace moeq4k
