// What the streaming attention kernels share: a CTA of four warps with a ring each, the
// instruction's operands, and the end of a segment.
#pragma once

#include <algorithm>

#include "attention.cuh"

namespace moeq4k {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 24 * 1024;          // bytes of a warp's ring: two CTAs' fill an SM
constexpr int kMaxRows = 16;              // of the instruction
// Floats of a row of the warps' meeting buffer.
__host__ __device__ constexpr int row_floats(int D) { return D + 8; }
// The least work of a CTA, in key tiles (1, 3, 5, 8: one token over 2000 9.1, 11.1, 12.7,
// 15.2 us), and an item's fixed cost (2, 3, 4: 48 tokens over 1500 34.0, 33.1, 34.1 us).
constexpr int kLeast = 1;
constexpr int kExtra = 3;
// What parting items costs, in key tiles: of one sequence, 300 tokens take 8.2 us whole
// and 8.9 in parts, 400 9.6 and 8.8; of 64 sequences, 300 10.0 and 14.9, 1000 27 and 31.
constexpr int kSplit = 9;
constexpr int kPartRows = 32;             // rows of a partial result (a multiple of 32)

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                 uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void put_vec(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put_vec(float *p, const float (&v)[2]) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
// A finished row: sums v (this lane's kPer channels) over the weights' sum; a
// row that saw nothing is 0, its logarithm -inf.
template <typename T, int kPer>
__device__ __forceinline__ void store_row(const Params &p, size_t row, int lane, float top, float sum,
                                          const float (&v)[kPer]) {
    const float inv = over_sum(sum);
    uint32_t w[kPer / 2];
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) w[c] = Pair<T>::make(v[2 * c] * inv, v[2 * c + 1] * inv);
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + (row * 32 + lane) * kPer);
    if (kPer == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[kPer / 2 - 1]);
    else dst[0] = w[0];
    if (p.lse != nullptr && lane == 0)
        p.lse[row] = log_sum(top, sum);
    __syncwarp();
}

// The end of a segment, by all threads: the warps' sums (rows of kOS floats at the start of
// each ring) and statistics become the item's rows or a part of them; parts are
// joined here where no second launch does it.
template <typename T, int D>
__device__ __forceinline__ void segment_result(const Params &p, const Run &run, int s0, int s1, uint8_t *smem,
                                               float (&sm_m)[kWarps][kMaxRows], float (&sm_l)[kWarps][kMaxRows],
                                               bool join_launch, bool &joins) {
    constexpr int kOS = row_floats(D);
    const Item &it = run.item;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.b.Hq / p.b.Hkv;
    const bool whole = s0 == 0 && s1 == it.tiles;
    const int rows = it.nt * G;
    constexpr int kPer = D / 32;  // channels a lane joins
    float *mine = p.part + size_t(part_slot(blockIdx.x, s0 == 0)) * part_floats(kPartRows, D);
    for (int r = warp; r < rows; r += kWarps) {
        float top = sm_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][r]);
        const float base = top == -CUDART_INF_F ? 0.f : top;
        float sum = 0.f, v[kPer];
#pragma unroll
        for (int c = 0; c < kPer; ++c) v[c] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_approx(sm_m[w][r] - base);
            sum = fmaf(sm_l[w][r], f, sum);
            const float *src = reinterpret_cast<const float *>(smem + w * kRing) + r * kOS + lane * kPer;
#pragma unroll
            for (int c = 0; c < kPer; ++c) v[c] = fmaf(src[c], f, v[c]);
        }
        if (whole) {
            store_row<T, kPer>(p, size_t(it.row0 + r / G) * p.b.Hq + it.kh * G + r % G, lane, top, sum, v);
        } else {
            put_vec(mine + part_at(r, lane * kPer, D), v);
            if (lane == 0) {
                mine[kPartRows * D + r] = top;
                mine[kPartRows * (D + 1) + r] = sum;
            }
            __syncwarp();
        }
    }
    if (join_launch) {
        if (tid == 0 && s0 == 0 && !whole) p.desc[blockIdx.x] = join_desc(p, run);
    } else if (!whole) {
        // the CTA that arrives last joins the parts (all are stored and seen then)
        const int first_cta = int(div_pos(run.item_u + p.extra, run.per));
        const JoinDesc d = join_desc(p, run);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            joins = atomicAdd(p.count + first_cta, 1u) + 1 == unsigned(d.parts);
            if (joins) p.count[first_cta] = 0u;  // for the next call
        }
        __syncthreads();
        __syncwarp();
        if (joins) {
            __threadfence();
            join_rows<T, D, kWarps>(p, d, first_cta, kPartRows, kPartRows, p.tt, 0, 1,
                                    reinterpret_cast<float *>(smem), &sm_m[0][0], &sm_l[0][0]);
        }
    }
}

Params make_params(const AttnArgs &a);

// Whether parted items are joined by a second launch.  Few items over many CTAs make many
// parts of each.  Up to kJoinInside of them the last CTA joins them on its way out (one
// token over 93: 9.6 us with the launch, 5.9 without); more take it longer than a second
// launch that spreads them over the GPU (one token over 600, 10 parts and more: 8.8 us with
// the launch, 9.4 without; over 131071, 76 parts: 52 and 56).
constexpr long kJoinInside = 10;
inline bool joins_by_launch(const PagedBatch &b, int grid, int tile, long inside) {
    const long items = long(b.B) * b.Hkv;
    const long tiles = (long(b.max_pages) * b.page + tile - 1) / tile + kExtra;  // of an item, at most
    return std::min(grid / items, tiles / kLeast) + 1 > inside;
}

// The same over a cache of 8-bit codes (any masks).
cudaError_t init_stream_codes();
cudaError_t launch_stream_codes(const AttnArgs &a, Params p, int max_new, int num_sms, cudaStream_t s);

}  // namespace attn
}  // namespace moeq4k
