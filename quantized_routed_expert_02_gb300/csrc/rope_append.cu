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
// stays small: a warp works out a row's sines once and keeps each lane's eight
// pairs in registers for all the heads of the row that are its, so that a head
// costs its loads, packed fp32 arithmetic and its stores, with no barrier.
//
// Measured: 4100 rows of 64/4 heads of 128 with norms 31.3 us = 4.8 TB/s, of
// 32/4 heads 17.5 us, one row 3.1 us.  Between that and the bytes' 22.2 us lie the
// start (3 us) and the latency of 16 warps an SM at 128 registers; weights folded into
// the sines (fewer operations, more registers) took 33.4 us, a ring of bulk
// copies and more warps with fewer chunks in flight no less than this.
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
constexpr int kBatch = 3;      // heads' chunks that a lane has in flight

// 2^64 times the fraction of a turn per position.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    double t = f * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    // 63 bits fit the conversion whatever t rounds to (t = 1 wraps to 0)
    return static_cast<unsigned long long>(__double2ll_rn(t * 4611686018427387904.0)) << 2;
}

// The last sequence that starts at or before `row`: one thread alone, or a
// whole warp for one row in steps of 32 ways.
__device__ __forceinline__ int find_seq(const PagedBatch &p, int row) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.offs[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int find_seq_warp(const PagedBatch &p, int row, int lane) {
    int lo = 0, n = p.B;  // among [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const unsigned before = __ballot_sync(0xffffffffu, b < lo + n && p.offs[b] <= row);
        const int at = lo + (before == 0u ? 0 : 31 - __clz(before)) * step;
        n = min(step, lo + n - at);
        lo = at;
    }
    return lo;
}

// Whether every offset is in range and none falls; the whole warp calls it.
__device__ inline bool offsets_rise(const PagedBatch &p, int lane) {
    bool ok = true;
    for (int b = lane; b < p.B; b += 32) {
        const int lo = p.offs[b], hi = p.offs[b + 1];
        ok = ok && lo >= 0 && hi >= lo && hi <= p.N;
    }
    return __all_sync(0xffffffffu, ok);
}

// The work is a run of steps, 512 / D heads each (what a warp turns at a time),
// row after row; a warp takes `run` of them, whatever the number of rows.
// Lane: chunk c = lane % (D / 16) of a head at a time: the channels
// 8 c .. 8 c + 7 and the 8 they pair with (rotated halves), or 16 in a row.
// kBatch of them are loaded ahead, over the ends of rows too, each slot again
// as soon as it is used; the places in the cache of a warp's next 32 rows are looked
// up together, a row per lane, so that no row waits for the chain of table loads.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, kCtas) rope_append_kernel(const RopeArgs a, int run) {
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
    const float mean = 1.f / float(D);  // exact: D is a power of two
    const int c0 = split ? 8 * c : 16 * c, c1 = split ? 8 * c + half : 16 * c + 8;
    // the warp's steps [at_step, end): rows from row on, heads [h0, h1) of it
    const int row_steps = (heads + step - 1) / step, total = a.b.N * row_steps;
    const int begin = (blockIdx.x * kWarps + warp) * run, end = min(total, begin + run);
    if (begin >= end) return;
    const int row_first = begin / row_steps, row_last = (end - 1) / row_steps;
    auto heads_of = [&](int r, int &from, int &to) {  // an empty range past the last row
        from = r == row_first ? (begin - r * row_steps) * step : 0;
        to = r > row_last ? 0 : r == row_last ? min(heads, (end - r * row_steps) * step) : heads;
    };
    uint4 in[kBatch][2];
    auto fetch = [&](int k, int row, int h0, int h1) {  // slot k of the batch that starts at head h0
        const int u = h0 + k * step + sub;
        in[k][0] = in[k][1] = make_uint4(0, 0, 0, 0);
        if (u < h1) {
            const T *p = static_cast<const T *>(a.qkv) + (size_t(row) * heads + u) * D;
            in[k][0] = *reinterpret_cast<const uint4 *>(p + c0);
            in[k][1] = *reinterpret_cast<const uint4 *>(p + c1);
        }
    };
    int h0, h1;
    heads_of(row_first, h0, h1);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) fetch(k, row_first, h0, h1);
    int pos[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) pos[k] = a.pos[size_t(axis[k]) * a.b.N + row_first];
    bool live32 = false;
    long cache32 = -1;  // of this lane's row among the next 32: the first key/value head's cache row
    for (int row = row_first; row <= row_last; ++row) {
        const int turn = (row - row_first) & 31;
        if (turn == 0) {
            const int r = min(row + lane, row_last);
            int b = row == row_last ? find_seq_warp(a.b, row, lane) : find_seq(a.b, r);
            SeqView sv = seq_view(a.b, b, a.hdr, false);
            auto has_row = [&]() { return sv.ok && r >= sv.first && r < sv.first + sv.n; };
            live32 = has_row();
            // A row of no sequence, or one that the search missed over offsets that do not rise: then
            // every sequence is looked at, so that a bad offset costs no other sequence its rows.
            if (!__all_sync(0xffffffffu, live32) && !offsets_rise(a.b, lane)) {
                for (int i = 0; !live32 && i < a.b.B; ++i) {
                    sv = seq_view(a.b, b = i, a.hdr, false);
                    live32 = has_row();
                }
                __syncwarp();
            }
            cache32 = -1;
            const int at = sv.len - sv.n + (r - sv.first);  // cache index
            if (live32 && at >= 0) {
                const int pg = page_of(a.b, b, at, a.hdr);
                if (pg >= 0) cache32 = long(pg) * Hkv * a.b.page + at % a.b.page;
            }
        }
        __syncwarp();
        const bool live = __shfl_sync(0xffffffffu, int(live32), turn) != 0;  // else a row of no sequence
        const long cache = __shfl_sync(0xffffffffu, cache32, turn);
        const int nrow = min(row + 1, row_last);
        int nh0, nh1;  // the next row's
        heads_of(row + 1, nh0, nh1);
        T *q_row = static_cast<T *>(a.q_out) + size_t(row) * Hq * D;
        T *k_row = static_cast<T *>(a.k) + max(cache, 0l) * D, *v_row = static_cast<T *>(a.v) + max(cache, 0l) * D;
        __syncwarp();  // the row before has read its sines
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long angle = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(pos[k])) * frac[k]);
            // the top 32 bits (rounded): a signed fraction of a turn, in half turns for sincospi
            const int top = static_cast<int>((angle + 0x80000000ll) >> 32);
            sincospif(float(top) * 4.6566128730773926e-10f, &si_sh[warp][lane + 32 * k], &co_sh[warp][lane + 32 * k]);  // * 2^-31
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) pos[k] = a.pos[size_t(axis[k]) * a.b.N + nrow];
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
            const bool more = h + kBatch * step < h1;  // of this row
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
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
                fetch(k, more ? row : nrow, more ? h + kBatch * step : nh0, more ? h1 : nh1);
                if (h + k * step >= h1) continue;
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
                        const float inv = rsqrtf(fmaf(ss, mean, a.eps));
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
                // heads are D apart in the queries, a page's rows apart in the cache
                T *dst = query ? q_row + head * D : value ? v_row + (head - Hq - Hkv) * (a.b.page * D)
                                                          : k_row + (head - Hq) * (a.b.page * D);
                if (mine && live && (query || cache >= 0)) {
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
        h0 = nh0;
        h1 = nh1;
    }
}

}  // namespace rope

cudaError_t launch_rope_append(const RopeArgs &a, int num_sms, cudaStream_t s) {
    using namespace rope;
    const int heads = a.b.Hq + 2 * a.b.Hkv, step = 512 / a.b.D, warps = num_sms * kCtas * kWarps;
    const int total = a.b.N * ((heads + step - 1) / step);  // at most 2^22 * 192
    const int run = (total + warps - 1) / warps;
    const int used = (total + run - 1) / run;
    const dim3 grid((used + kWarps - 1) / kWarps), block(kWarps * 32);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, size_t(0), s, a, run); };
    if (a.type == MOE_F16) return a.interleaved ? go(rope_append_kernel<__half, true>) : go(rope_append_kernel<__half, false>);
    return a.interleaved ? go(rope_append_kernel<__nv_bfloat16, true>) : go(rope_append_kernel<__nv_bfloat16, false>);
}

}  // namespace moeq4k
