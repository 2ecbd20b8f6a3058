// Attention of few query rows per key/value head over a paged cache: single
// tokens, drafted tokens (moe_attention_paged up to 16 rows).
//
// Bytes bound: every cached key and value is read once, 4 D bytes for 4 D
// flops per row.  So the keys stream through the SM and everything else stays
// in registers: each of a CTA's four warps owns a ring of its own, filled by
// TMA boxes of 16 keys (a box never crosses a page), and walks its pieces
// with no barrier but its ring's: S = Q K^T and O += P V by mma.sync m16n8k16 on
// 16-bit operands with fp32 sums, the running maximum and sum of the softmax in
// between.  The instruction's 16 rows are one tile of query rows (the G heads of a
// group times the tokens); a tcgen05 tile would be 128 rows, seven eighths of
// it padding, for work that the memory bounds anyway.  The four warps'
// results meet at the end of a segment.
//
// Measured (32/4 heads of 128, bf16): 64 sequences of 4000 tokens 89 us
// = 5.9 TB/s, eight of 20000 with 16/16 heads 207 us = 6.3 TB/s; a bare loop of the
// same copies over 268 MB reaches 6.3 to 6.6 TB/s whatever its box.  Short
// batches pay for the chain from the launch to the first keys (offsets, the search for the
// run, page table, keys: four dependent reads; of one token over 93, 6.0 us, nearly all, of a
// ragged batch some 7 us) and, with many parts, 4 us for the joining launch: one
// token over 131071 53 us, over 2000 9.1.  A cap's polynomial costs batches that the
// bytes do not fill 1.5 us (48 tokens over 1500 30.1 -> 31.8) and the others nothing.
#include <algorithm>

#include <cuda.h>

#include "attention.cuh"

namespace moeq4k {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kPiece = 16;                // keys of a piece
constexpr int kTile = kWarps * kPiece;    // keys of a tile: a piece for every warp
constexpr int kRing = 24 * 1024;          // bytes of a warp's ring: two CTAs' fill an SM
constexpr int kMaxRows = 16;              // of the instruction
// The least work of a CTA, in key tiles (1, 3, 5, 8: one token over 2000 9.1, 11.1, 12.7,
// 15.2 us), and an item's fixed cost (2, 3, 4: 48 tokens over 1500 34.0, 33.1, 34.1 us).
constexpr int kLeast = 1;
constexpr int kExtra = 3;
// What parting items costs, in key tiles: of one sequence, 300 tokens take 8.2 us whole
// and 8.9 in parts, 400 9.6 and 8.8; of 64 sequences, 300 10.0 and 14.9, 1000 27 and 31.
constexpr int kSplit = 9;
constexpr int kPartRows = 32;             // rows of a partial result (a multiple of 32)

struct StreamParams {
    CUtensorMap mk, mv;
    Params p;
    bool join_launch;  // split items are joined by a second launch
};

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

// Box of 64 channels x 16 cache rows of page-head z; out-of-range z reads as zeros.
__device__ __forceinline__ void tma_box(void *dst, const CUtensorMap *map, int ch, int row, int z,
                                        uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(ch), "r"(row), "r"(z), "r"(smem_addr(bar))
        : "memory");
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

template <typename T, int D, bool kCap>
__global__ void __launch_bounds__(kThreads, 2) attention_stream_kernel(const __grid_constant__ StreamParams sp) {
    constexpr int kHalves = D / 64;                      // boxes of a row
    constexpr int kBox = kPiece * 128;                   // bytes of a box
    constexpr int kStage = 2 * kHalves * kBox;           // K and V of a piece
    constexpr int kStages = kRing / kStage;
    constexpr int kRows = kMaxRows;
    constexpr int kOS = D + 8;                           // floats of a row of the warps' meeting buffer
    static_assert(kRows * kOS * 4 <= kRing, "a warp's sums fit its ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ unsigned failed;
    __shared__ bool joins;
    __shared__ Run run_sh;
    const Params &p = sp.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    const int G = p.b.Hq / p.b.Hkv;
    uint8_t *ring = smem + warp * kRing;
    if (tid == 0) {
        failed = 0;
        prefetch_map(&sp.mk);
        prefetch_map(&sp.mv);
    }
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1 + withheld(p));
    __syncwarp();
    fence_mbar_init();
    pdl_enter();
    if (sp.join_launch && tid == 0) p.desc[blockIdx.x].parts = 0;
    // Single-token calls of the experts leave tags where the parts are counted: the header says
    // whether there were any (read beside the search, looked at after it).
    const bool looks = !sp.join_launch && blockIdx.x == 0 && tid == 0;
    const unsigned long long tags = looks ? p.hdr->cta_calls : 0ull;
    Run run;
    const bool work = run_begin<kTile>(p, kLeast, kSplit, reinterpret_cast<long *>(smem), &run_sh, run);
    if (tags != 0) record_status(p.hdr, MOE_ERR_WORKSPACE, 0);
    if (!work) return;
    fence_proxy_async_smem();  // the prefix sums (generic) before the copies into the ring
    __syncthreads();

    uint32_t done = 0, issued = 0;  // pieces of this warp, over all segments
    while (run.u < run.end) {
        int s0, s1;
        if (!run_segment(p, run, s0, s1)) break;
        const Item it = run.item;
        const int key_first = (it.t0 + s0) * kTile + warp * kPiece;  // this warp's first piece
        const int last = it.pos0 + it.nt - 1;                       // the last key any row sees
        int n = s1 - s0;  // pieces of this warp that hold such keys
        n = max(0, min(n, last >= key_first ? (last - key_first) / kTile + 1 : 0));
        // the pages of 32 pieces at a time, and of the 32 after them
        auto page_at = [&](int i) {
            if (i >= n) return 0;
            // past the tensor, read as zeros: a piece before every row's window (its page may be
            // gone already) and a bad page
            const int key = key_first + i * kTile;
            const int pg = key + kPiece <= it.seen ? -1 : page_of(p.b, it.b, key, p.hdr);
            return pg < 0 ? p.b.num_pages : pg;
        };
        int pages = page_at(lane), pages_next = n > 32 ? page_at(32 + lane) : 0;
        // this thread's rows: gid, gid + 8 of each 16; their position, -1 for rows past the tile
        int pos[2];
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + gid;
            const int tok = r / G;
            const bool live = tok < it.nt;
            pos[h] = live ? it.pos0 + tok : -1;
            const T *row = static_cast<const T *>(p.q) +
                           (size_t(it.row0 + (live ? tok : 0)) * p.b.Hq + it.kh * G + r % G) * D;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(row + 16 * k + 2 * tig);
                qa[k][h] = live ? w[0] : 0u;
                qa[k][2 + h] = live ? w[4] : 0u;
            }
        }
        __syncwarp();
        int sent = 0;  // pieces of this segment issued
        auto issue = [&]() {
            if (sent > 0 && (sent & 31) == 0) {
                pages = pages_next;
                pages_next = page_at(sent + 32 + lane);
                __syncwarp();
            }
            const int z = __shfl_sync(0xffffffffu, pages, sent & 31) * p.b.Hkv + it.kh;
            if (lane == 0) {
                const uint32_t st = issued % kStages;
                uint8_t *dst = ring + st * kStage;
                uint64_t *bar = &full[warp][st];
                const int row = (key_first + sent * kTile) & (p.b.page - 1);
                mbar_arrive_expect_tx(bar, kStage);
#pragma unroll
                for (int c = 0; c < kHalves; ++c) tma_box(dst + c * kBox, &sp.mk, c * 64, row, z, bar);
#pragma unroll
                for (int c = 0; c < kHalves; ++c)
                    tma_box(dst + (kHalves + c) * kBox, &sp.mv, c * 64, row, z, bar);
            }
            __syncwarp();
            ++sent;
            ++issued;
        };
        for (int i = 0; i < kStages && i < n; ++i) issue();

        float o[D / 8][4], mx[2], l[2];
        mx[0] = mx[1] = -CUDART_INF_F;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const uint32_t st = done % kStages;
            if (!__all_sync(0xffffffffu, wait_phase(&full[warp][st], (done / kStages) & 1u, p.wait_ns))) {
                ok = false;
                break;
            }
            const int key0 = key_first + i * kTile;
            const uint32_t kb = smem_addr(ring + st * kStage), vb = kb + kHalves * kBox;
            float s[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
            // S: matrices (keys 0-7, channels lo/hi), (keys 8-15, lo/hi) of each 16 channels
            const int krow = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                const int ch = (2 * k + kc) & 7;
                ldsm4(b, kb + (k / 4) * kBox + krow * 128 + ((ch ^ (krow & 7)) << 4));
                mma16816<T>(s[0], qa[k], b[0], b[1]);
                mma16816<T>(s[1], qa[k], b[2], b[3]);
            }
            const bool edge = key0 + kPiece - 1 > it.pos0 || (p.window > 0 && key0 <= last - p.window);
            uint32_t pa[4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[j][c] = score<kCap>(s[j][c], p);
                    if (edge) {
                        const int key = key0 + 8 * j + 2 * tig + (c & 1), at = pos[c >> 1];
                        if (key > at || (p.window > 0 && at - key >= p.window))
                            s[j][c] = -CUDART_INF_F;
                    }
                }
            float cor[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]),
                                fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                v = fmaxf(v, mx[h]);
                const float base = v == -CUDART_INF_F ? 0.f : v;  // nothing seen yet
                cor[h] = exp2_approx(mx[h] - base);
                mx[h] = v;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[j][2 * h + c] = exp2_approx(s[j][2 * h + c] - base);
                l[h] = l[h] * cor[h] + ((s[0][2 * h] + s[0][2 * h + 1]) +
                                              (s[1][2 * h] + s[1][2 * h + 1]));
            }
            // the weights rounded to the 16-bit type for the product: its two operands have one type, and
            // the values beside them were rounded to it by the same half step; the sum l keeps them whole
            pa[0] = Pair<T>::make(s[0][0], s[0][1]);
            pa[1] = Pair<T>::make(s[0][2], s[0][3]);
            pa[2] = Pair<T>::make(s[1][0], s[1][1]);
            pa[3] = Pair<T>::make(s[1][2], s[1][3]);
            if (__any_sync(0xffffffffu, cor[0] != 1.f || cor[1] != 1.f)) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][0] *= cor[0], o[j][1] *= cor[0];
                    o[j][2] *= cor[1], o[j][3] *= cor[1];
                }
            }
            // O: matrices (keys 0-7, channel chunk c), (keys 8-15, c), then c + 1, transposed;
            // rows past the sequence's end hold anything: their weights are 0, and so must they be
            const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
            const bool tail = key0 + kPiece > it.len;
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if (tail)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + 8 * h + 2 * tig;
                    keep[h] = (key < it.len ? 0xffffu : 0u) | (key + 1 < it.len ? 0xffff0000u : 0u);
                }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t b[4];
                const int ch = (2 * j + vc) & 7;
                ldsm4_trans(b, vb + (j / 4) * kBox + vrow * 128 + ((ch ^ (vrow & 7)) << 4));
                if (tail) {
                    b[0] &= keep[0], b[1] &= keep[1];
                    b[2] &= keep[0], b[3] &= keep[1];
                }
                mma16816<T>(o[2 * j], pa, b[0], b[1]);
                mma16816<T>(o[2 * j + 1], pa, b[2], b[3]);
            }
            ++done;
            // every lane's reads of the stage (generic) are over before the copy (async proxy) into it:
            // none of 13500 calls differed without the fence, which costs 0.5 us at most
            if (sent < n) fence_proxy_async_smem();
            __syncwarp();
            if (sent < n) issue();
        }
        if (!ok) {
            record_status(p.hdr, MOE_ERR_TIMEOUT, 40 + warp);
            failed = 1;
        }
        // copies still in flight after a time-out land before the ring is written
        for (; done < issued; ++done)
            wait_phase(&full[warp][done % kStages], (done / kStages) & 1u, kDrainNs);

        // the warps' sums into their rings, the rows' statistics beside them
        float *so = reinterpret_cast<float *>(ring);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v = l[h];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            const int r = 8 * h + gid;
            if (tig == 0) {
                sm_m[warp][r] = mx[h];
                sm_l[warp][r] = v;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<float2 *>(so + r * kOS + 8 * j + 2 * tig) =
                    make_float2(o[j][2 * h], o[j][2 * h + 1]);
        }
        __syncthreads();
        __syncwarp();
        if (failed != 0) return;
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
        if (sp.join_launch) {
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
        run_next<kTile>(p, run);
        if (run.u < run.end) {
            fence_proxy_async_smem();  // the sums in the rings (generic) before the next copies
            __syncthreads();
        }
    }
}

constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) attention_join_kernel(const Params p, int rows, int half, int tth) {
    pdl_enter();
    __shared__ __align__(16) float sv[kJoinWarps * D * kJoinRows];
    __shared__ float sm[kJoinWarps * kJoinRows], sl[kJoinWarps * kJoinRows];
    const JoinDesc d = p.desc[blockIdx.x];
    if (d.parts == 0) return;
    join_rows<T, D, kJoinWarps>(p, d, blockIdx.x, rows, half, tth, blockIdx.y, gridDim.y, sv, sm, sl);
}

constexpr int kStreamSmem = kWarps * kRing;

// f on every form of the kernel, until one fails.
template <typename F>
cudaError_t each_stream(F f) {
    cudaError_t e = cudaSuccess;
    auto of = [&](auto type) {
        using T = decltype(type);
        if (e == cudaSuccess) e = f(attention_stream_kernel<T, 64, false>);
        if (e == cudaSuccess) e = f(attention_stream_kernel<T, 64, true>);
        if (e == cudaSuccess) e = f(attention_stream_kernel<T, 128, false>);
        if (e == cudaSuccess) e = f(attention_stream_kernel<T, 128, true>);
    };
    of(__half());
    of(__nv_bfloat16());
    return e;
}

template <typename T, int D>
cudaError_t launch_stream(const StreamParams &sp, int grid, cudaStream_t s) {
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(grid), dim3(kThreads), size_t(kStreamSmem), s, sp);
    };
    return sp.p.cap_in != 0.f ? go(attention_stream_kernel<T, D, true>) : go(attention_stream_kernel<T, D, false>);
}

Params make_params(const AttnArgs &a) {
    Params p = {};
    constexpr float kLog2e = 1.4426950408889634f;
    p.b = a.b;
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.scale_log2 = a.scale * kLog2e;
    p.cap_in = a.softcap > 0.f ? 2.f * kLog2e * a.scale / a.softcap : 0.f;
    p.cap_y = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
    p.cap_log2 = a.softcap * kLog2e;
    p.window = a.window;
    p.hdr = a.hdr;
    p.count = reinterpret_cast<unsigned *>(a.scratch);
    p.desc = reinterpret_cast<JoinDesc *>(a.scratch + kCountBytes);
    p.part = reinterpret_cast<float *>(a.scratch + kCountBytes + kDescBytes);
    p.wait_ns = a.wait_ns;
    p.withhold = a.withhold;
    return p;
}

cudaError_t launch_join(const Params &p, moe_dtype type, int grid, int rows, int half, int tth, cudaStream_t s) {
    const dim3 blocks(grid, std::min(rows / kJoinRows, 8)), threads(kJoinWarps * 32);
    auto go = [&](auto kernel) { return launch_pdl(kernel, blocks, threads, size_t(0), s, p, rows, half, tth); };
    if (type == MOE_F16)
        return p.b.D == 64 ? go(attention_join_kernel<__half, 64>) : go(attention_join_kernel<__half, 128>);
    return p.b.D == 64 ? go(attention_join_kernel<__nv_bfloat16, 64>)
                       : go(attention_join_kernel<__nv_bfloat16, 128>);
}

}  // namespace attn

size_t attention_part_bytes(int D) {
    using namespace attn;
    return kCountBytes + kDescBytes +
           std::max(size_t(2) * kMaxCtas * part_floats(kPartRows, D) * sizeof(float), tc_part_bytes(D));
}

cudaError_t init_attention() {
    using namespace attn;
    const cudaError_t e = each_stream([](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
    });
    return e != cudaSuccess ? e : init_tc();
}

cudaError_t launch_attention(const AttnArgs &a, int max_new, int num_sms, cudaStream_t s) {
    using namespace attn;
    const int G = a.b.Hq / a.b.Hkv;
    const Params base = make_params(a);
    // More than 16 rows are faster on the tensor cores' own tile, although most of its rows are
    // padding (32 rows over 6000 keys of 32 sequences 75 us, with a second instruction tile here
    // 84; 32 over 900 of one 11.8 and 18.3; 24 over 2000 of eight 18.8 and 24.8); up to 16 this
    // kernel is (16 rows over 2000 keys of eight 16.7 and 18.7; 8 over 12000 and less of 48
    // 57.5 and 58.3; 8 over 93 of one 5.5 and 9.7).
    if (long(max_new) * G > kMaxRows) return launch_tc(a, base, num_sms, s);
    StreamParams sp = {};
    sp.p = base;
    sp.p.tt = kMaxRows / G;
    sp.p.tt_magic = 0xffffffffu / unsigned(sp.p.tt) + 1;
    sp.p.extra = kExtra;
    if (!encode_pages_map(&sp.mk, a.k, a.b, a.type, kPiece) || !encode_pages_map(&sp.mv, a.v, a.b, a.type, kPiece))
        return cudaErrorInvalidValue;
    const int grid = std::min(2 * num_sms, kMaxCtas);
    // Few items over many CTAs make many parts of each.  Up to kJoinInside of them the last
    // CTA joins them on its way out (one token over 93: 9.6 us with the launch, 5.9 without);
    // more take it longer than a second launch that spreads them over the GPU (one token
    // over 600, 10 parts and more: 8.8 us with the launch, 9.4 without; over 131071, 76
    // parts: 52 and 56).
    constexpr long kJoinInside = 10;
    const long items = long(a.b.B) * a.b.Hkv;
    const long tiles = (long(a.b.max_pages) * a.b.page + kTile - 1) / kTile + kExtra;  // of an item, at most
    sp.join_launch = std::min(grid / items, tiles / kLeast) + 1 > kJoinInside;
    cudaError_t e;
    if (a.type == MOE_F16)
        e = a.b.D == 64 ? launch_stream<__half, 64>(sp, grid, s) : launch_stream<__half, 128>(sp, grid, s);
    else
        e = a.b.D == 64 ? launch_stream<__nv_bfloat16, 64>(sp, grid, s)
                        : launch_stream<__nv_bfloat16, 128>(sp, grid, s);
    if (e != cudaSuccess || !sp.join_launch) return e;
    return launch_join(sp.p, a.type, grid, kPartRows, kPartRows, sp.p.tt, s);
}

}  // namespace moeq4k
