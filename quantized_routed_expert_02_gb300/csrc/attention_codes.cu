// Attention of few query rows per key/value head over a paged cache of 8-bit codes
// (moe_attention_cache with scales, up to 16 rows): the streaming kernel for half the bytes.
//
// A key is k_scale * code, so a score is k_scale * (q . code), the product by
// mma.sync m16n8k16 on codes made 16-bit operands in registers (exact), the scale in
// fp32 behind it; a weight takes its value's scale before it is rounded for the product with V.
//
// Bytes bound as the 16-bit kernel is, at twice the keys per byte, so a piece is 32
// keys and what is done once a piece (maxima, rescales, waits) costs as much per byte as
// there.  The fragments need no shuffles: ldmatrix gives a lane four channels in a row of a
// key's codes, which as two pairs are an operand of the instruction for some order of the
// channels, and the queries are read in the same order; transposed it gives two channels of
// two keys, whose even and odd channels are two tiles of the output.
#include <cuda.h>
#include <type_traits>

#include "attention_stream.cuh"
#include "codes.cuh"

namespace moeq4k {
namespace attn {

constexpr int kCodePiece = 32;                      // keys of a piece
constexpr int kCodeTile = kWarps * kCodePiece;      // keys of a tile: as many bytes as the 16-bit kernel's

struct CodesParams {
    CUtensorMap mk, mv, mks, mvs;
    Params p;
    int boxes;         // of a piece: 1, or 2 where pages have 16 rows
    bool join_launch;  // split items are joined by a second launch
};

__device__ __forceinline__ void tma_codes(void *dst, const CUtensorMap *map, int row, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(0), "r"(row), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_scales(void *dst, const CUtensorMap *map, int row, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(row), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Byte of 16-byte chunk c of row r as the copy's swizzle places it.
template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) {
    return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

template <typename T, int D, bool kCap>
__global__ void __launch_bounds__(kThreads, 2) attention_codes_kernel(const __grid_constant__ CodesParams sp) {
    constexpr int kPiece = kCodePiece, kTile = kCodeTile;
    constexpr int kBytes = kPiece * D;                   // of a piece's keys, or values
    constexpr int kStages = kRing / (2 * kBytes);
    constexpr int kOS = row_floats(D);
    static_assert(kMaxRows * kOS * 4 <= kRing, "a warp's sums fit its ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    // of keys, of values; a box's begin on 128 bytes, as a copy's place has to
    __shared__ __align__(128) float scales[kWarps][kStages][2][2 * kPiece];
    __shared__ float sm_m[kWarps][kMaxRows], sm_l[kWarps][kMaxRows];
    __shared__ unsigned failed;
    __shared__ bool joins;
    __shared__ Run run_sh;
    const Params &p = sp.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    const int G = p.b.Hq / p.b.Hkv;
    const int nb = sp.boxes, box_rows = kPiece / nb;
    const int gap = nb == 2 ? 16 : 0;  // in the scales' places, ahead of a piece's key 16
    uint8_t *ring = smem + warp * kRing;
    if (tid == 0) {
        failed = 0;
        prefetch_map(&sp.mk);
        prefetch_map(&sp.mv);
        prefetch_map(&sp.mks);
        prefetch_map(&sp.mvs);
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
    const bool work = run_begin<kTile, true>(p, kLeast, kSplit, reinterpret_cast<long *>(smem), &run_sh, run);
    if (tags != 0) record_status(p.hdr, MOE_ERR_WORKSPACE, 0);
    if (!work) return;
    fence_proxy_async_smem();  // the prefix sums (generic) before the copies into the ring
    __syncthreads();

    uint32_t done = 0, issued = 0;  // pieces of this warp, over all segments
    while (run.u < run.end) {
        int s0, s1;
        if (!run_segment(p, run, s0, s1)) break;
        const Item it = run.item;
        auto key_of = [&](int i) { return tile_key<kTile, true>(it, s0 + i) + warp * kPiece; };  // this warp's pieces
        const int last = last_key<true>(p, it);
        int n = s1 - s0;  // pieces of this warp that hold keys that a row sees
        if (key_of(n - 1) > last) --n;
        // the pages of 32 boxes at a time, and of the 32 after them
        auto page_at = [&](int i) {
            const int piece = nb == 2 ? i >> 1 : i;
            if (piece >= n) return 0;
            // past the tensor, read as zeros: a box past the last key, one between the sinks and every row's
            // window (its page may be gone already) and a bad page
            const int key = key_of(piece) + (nb == 2 ? (i & 1) * box_rows : 0);
            const int pg = key > last || (key + box_rows <= it.seen && key >= p.sinks) ? -1
                                                                                        : page_of(p.b, it.b, key, p.hdr);
            return pg < 0 ? p.b.num_pages : pg;
        };
        int pages = page_at(lane), pages_next = n * nb > 32 ? page_at(32 + lane) : 0;
        Sight sight[2];  // of this thread's rows: gid, gid + 8
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + gid;
            const int tok = r / G;
            const bool live = tok < it.nt;
            sight[h] = row_sight(p, run.seq, live, it.row0 + tok, it.qt * p.tt + tok);
            const T *row = static_cast<const T *>(p.q) +
                           (size_t(it.row0 + (live ? tok : 0)) * p.b.Hq + it.kh * G + r % G) * D;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {  // four channels in a row, as the codes come
                const uint2 w = *reinterpret_cast<const uint2 *>(row + 16 * k + 4 * tig);
                qa[k][h] = live ? w.x : 0u;
                qa[k][2 + h] = live ? w.y : 0u;
            }
        }
        __syncwarp();
        int sent = 0;  // pieces of this segment issued
        auto issue = [&]() {
            if (sent > 0 && ((sent * nb) & 31) == 0) {
                pages = pages_next;
                pages_next = page_at(sent * nb + 32 + lane);
                __syncwarp();
            }
            const int box = lane >> 2;  // lanes 0 .. 4 nb - 1: box, and keys, values, scales of either
            const int z = __shfl_sync(0xffffffffu, pages, (sent * nb + box) & 31) * p.b.Hkv + it.kh;
            const uint32_t st = issued % kStages;
            uint64_t *bar = &full[warp][st];
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kBytes + 2 * kPiece * 4);
            __syncwarp();
            if (box < nb) {
                const int row = (key_of(sent) + box * box_rows) & (p.b.page - 1);
                uint8_t *dst = ring + st * (2 * kBytes) + box * box_rows * D;
                if ((lane & 3) == 0) tma_codes(dst, &sp.mk, row, z, bar);
                else if ((lane & 3) == 1) tma_codes(dst + kBytes, &sp.mv, row, z, bar);
                else if ((lane & 3) == 2) tma_scales(&scales[warp][st][0][box * kPiece], &sp.mks, row, z, bar);
                else tma_scales(&scales[warp][st][1][box * kPiece], &sp.mvs, row, z, bar);
            }
            __syncwarp();
            ++sent;
            ++issued;
        };
        for (int i = 0; i < kStages && i < n; ++i) issue();

        // sums of channels 16 c + 4 tig + 2 x (tile 2 c) and one after each (tile 2 c + 1)
        float o[D / 8][4], mx[2], l[2];
        uint32_t ref = kRefLeast;
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
            const int key0 = key_of(i);
            const uint32_t kb = smem_addr(ring + st * (2 * kBytes)), vb = kb + kBytes;
            const float *ks = scales[warp][st][0], *vs = scales[warp][st][1];
            float s[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
            // S: matrices of keys 8 j .. 8 j + 7, the same 16 channels of each
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                ldsm4(b, kb + code_chunk<D>(lane, k));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const CodePair<T> c(b[j]);
                    mma16816<T>(s[j], qa[k], c.template take<0, 1>(), c.template take<2, 3>());
                }
            }
            // keys that some row does not see
            const int all = p.tree != nullptr ? run.seq.len - run.seq.n - 1 : it.pos0;
            const bool edge = key0 + kPiece - 1 > all ||
                              (p.window > 0 && key0 <= last - p.window && key0 + kPiece > p.sinks);
            uint32_t sees[2] = {0u, 0u};
            if (edge) {
#pragma unroll
                for (int h = 0; h < 2; ++h) sees[h] = sight32(p, run.seq, sight[h], key0) >> (2 * tig);
                __syncwarp();
            }
            // the values' scales; those past the sequence's end hold anything, and a weight of 0 takes them
            const bool tail = key0 + kPiece > it.len;
            float w[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = *reinterpret_cast<const float2 *>(vs + 8 * j + (j >> 1) * gap + 2 * tig);
                w[j][0] = v.x;
                w[j][1] = v.y;
                if (tail) {
                    if (key0 + 8 * j + 2 * tig >= it.len) w[j][0] = 0.f;
                    if (key0 + 8 * j + 2 * tig + 1 >= it.len) w[j][1] = 0.f;
                }
            }
            float grown = 1.f;  // of the sums, where the scales' reference has grown
            if (ScaleRef<T>::kUsed) {
                const float mine = tail && key0 + lane >= it.len ? 0.f : vs[lane + (lane >> 4) * gap];
                const uint32_t top = ref_bits(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));
                if (top > ref) {
                    grown = __uint_as_float(ref) * over_ref(top);
                    ref = top;
                }
                const float over = over_ref(ref);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j][0] *= over, w[j][1] *= over;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 k = *reinterpret_cast<const float2 *>(ks + 8 * j + (j >> 1) * gap + 2 * tig);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[j][c] = score<kCap>(s[j][c] * ((c & 1) != 0 ? k.y : k.x), p);
                    if (edge && (sees[c >> 1] >> (8 * j + (c & 1)) & 1u) == 0u) s[j][c] = -CUDART_INF_F;
                }
            }
            float cor[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = mx[h];
#pragma unroll
                for (int j = 0; j < 4; ++j) v = fmaxf(v, fmaxf(s[j][2 * h], s[j][2 * h + 1]));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                const float base = v == -CUDART_INF_F ? 0.f : v;  // nothing seen yet
                cor[h] = exp2_approx(mx[h] - base);
                mx[h] = v;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[j][2 * h + c] = exp2_approx(s[j][2 * h + c] - base);
                    sum += s[j][2 * h] + s[j][2 * h + 1];
                }
                l[h] = l[h] * cor[h] + sum;
                cor[h] *= grown;
            }
            // the weights times the values' scales, rounded to the 16-bit type for the product (its two
            // operands have one type); the sum l keeps the weights whole
            uint32_t pa[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = 2 * t + (x >> 1), h = x & 1;
                    pa[t][x] = Pair<T>::make(s[j][2 * h] * w[j][0], s[j][2 * h + 1] * w[j][1]);
                }
            if (__any_sync(0xffffffffu, cor[0] != 1.f || cor[1] != 1.f)) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][0] *= cor[0], o[j][1] *= cor[0];
                    o[j][2] *= cor[1], o[j][3] *= cor[1];
                }
            }
            // O: matrices (keys 0-7 and 8-15 of 16, channel chunk c), then of chunk c + 1, transposed
            const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < D / 16; c += 2) {
                    uint32_t b[4];
                    ldsm4_trans(b, vb + code_chunk<D>(16 * t + vrow, c + vc));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const CodePair<T> lo(b[2 * x]), hi(b[2 * x + 1]);
                        mma16816<T>(o[2 * (c + x)], pa[t], lo.template take<0, 2>(), hi.template take<0, 2>());
                        mma16816<T>(o[2 * (c + x) + 1], pa[t], lo.template take<1, 3>(), hi.template take<1, 3>());
                    }
                }
            ++done;
            // every lane's reads of the stage (generic) are over before the copy (async proxy) into it
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
        const float unit = ScaleRef<T>::kUsed ? __uint_as_float(ref) : 1.f;
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
            for (int c = 0; c < D / 16; ++c)
                *reinterpret_cast<float4 *>(so + r * kOS + 16 * c + 4 * tig) =
                    make_float4(o[2 * c][2 * h] * unit, o[2 * c + 1][2 * h] * unit, o[2 * c][2 * h + 1] * unit,
                                o[2 * c + 1][2 * h + 1] * unit);
        }
        __syncthreads();
        __syncwarp();
        if (failed != 0) return;
        segment_result<T, D>(p, run, s0, s1, smem, sm_m, sm_l, sp.join_launch, joins);
        run_next<kTile, true>(p, run);
        if (run.u < run.end) {
            fence_proxy_async_smem();  // the sums in the rings (generic) before the next copies
            __syncthreads();
        }
    }
}

constexpr int kCodesSmem = kWarps * kRing;

cudaError_t init_stream_codes() {
    cudaError_t e = cudaSuccess;
    auto of = [&](auto kernel) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCodesSmem);
    };
    auto with = [&](auto type) {
        using T = decltype(type);
        of(attention_codes_kernel<T, 64, false>);
        of(attention_codes_kernel<T, 64, true>);
        of(attention_codes_kernel<T, 128, false>);
        of(attention_codes_kernel<T, 128, true>);
    };
    with(__half());
    with(__nv_bfloat16());
    return e;
}

cudaError_t launch_stream_codes(const AttnArgs &a, Params p, int num_sms, cudaStream_t s) {
    CodesParams sp = {};
    p.tt = kMaxRows / (a.b.Hq / a.b.Hkv);
    p.tt_magic = 0xffffffffu / unsigned(p.tt) + 1;
    p.extra = kExtra;
    sp.p = p;
    sp.boxes = a.b.page < kCodePiece ? 2 : 1;
    const int box_rows = kCodePiece / sp.boxes;
    if (!encode_codes_map(&sp.mk, a.k, a.b, box_rows, false) || !encode_codes_map(&sp.mv, a.v, a.b, box_rows, false) ||
        !encode_scales_map(&sp.mks, a.ks, a.b, box_rows) || !encode_scales_map(&sp.mvs, a.vs, a.b, box_rows))
        return cudaErrorInvalidValue;
    const int grid = std::min(2 * num_sms, kMaxCtas);
    sp.join_launch = joins_by_launch(a.b, grid, kCodeTile);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(grid), dim3(kThreads), size_t(kCodesSmem), s, sp);
    };
    auto of = [&](auto type, auto cap) {
        using T = decltype(type);
        constexpr bool kCap = decltype(cap)::value;
        return a.b.D == 64 ? go(attention_codes_kernel<T, 64, kCap>) : go(attention_codes_kernel<T, 128, kCap>);
    };
    auto with = [&](auto type) { return p.cap_in != 0.f ? of(type, std::true_type()) : of(type, std::false_type()); };
    const cudaError_t e = a.type == MOE_F16 ? with(__half()) : with(__nv_bfloat16());
    if (e != cudaSuccess || !sp.join_launch) return e;
    return launch_join(p, a.type, grid, kPartRows, kPartRows, p.tt, s);
}

}  // namespace attn
}  // namespace moeq4k
