// Attention of few query rows per key/value head over a paged cache of 8-bit codes
// (moe_attention_cache with scales, up to 16 rows): the streaming kernel for half the bytes.
//
// A key is k_scale * code, so a score is k_scale * (q . code), the product by
// mma.sync m16n8k16 on codes made fp16 operands in registers (exact), the scale in fp32
// behind it; a weight takes its value's scale before it is rounded for the product with V.
// bf16 queries become fp16 ones, each row by a power of two that puts its largest
// element below 2^15: a bf16 element within 2^-28 of that is exact, the others are off by less
// than 2^-39 of it, and fp16 codes cost 5 instructions for 4, bf16 ones 8.
//
// Bytes bound as the 16-bit kernel is, at twice the keys per byte, so what counts is the
// instructions per key.  The products are transposed, S^T = K Q^T and O^T = V^T P^T: keys, and
// channels, fill the instruction's 16 rows and the query rows its 8 columns, once or
// twice, so that up to 8 rows (a token of a group of 8) pay for no padding.  The fragments need no
// shuffles: ldmatrix gives a lane four channels in a row of a key's codes, which as two
// pairs are an operand of the instruction for some order of the channels, and the queries
// are read in the same order; transposed it gives two channels of two keys, an operand
// whose rows are the even and the odd channels.  The weights turn in registers (movmatrix).
//
// The first copies are under way before anything waits for the queries (48 of 2000 31.0 -> 29.2 us).
//
// Measured (32/4 heads of 128): 48 sequences of 150 to 12000 tokens 38.5 us (16-bit values 57.9), 128
// of 4000 98.7 us = 5.5 TB/s, one over 93 6.3, one over 100000 30.5.  With the rows where the keys
// are now (16 of them, half padding) and a rescale for every new maximum these took 42.9,
// 110.7, 6.5 and 33.7; without any arithmetic the copies take 33 and 89.  Beside those, three CTAs an SM
// with smaller rings (46.7 and 116), and the next piece's scores computed among a piece's softmax
// (45.3 and 116) were slower.
#include <cuda.h>
#include <type_traits>

#include "attention_stream.cuh"
#include "codes.cuh"
#include "f32x2.cuh"
#include "tcgen05.cuh"

namespace moeq4k {
namespace attn {

constexpr int kCodePiece = 32;                      // keys of a piece
constexpr long kCodeJoinInside = 10;                // parts that the last CTA joins (6, 10: 700 tokens of one 17.0, 12.7 us)
// What parting items costs, in key tiles (2, 5, 9: 200 tokens of one sequence 8.7, 7.4, 7.3 us, 700
// 10.4, 10.4, 12.7; 600 of 48 18.3, 14.3, 14.3; 2000 of 48 30.8, 30.8, 32.0).
constexpr int kCodeSplit = 5;
constexpr float kGrowth = 8.f;                      // log2 growth of a maximum that moves the reference
constexpr int kCodeTile = kWarps * kCodePiece;      // keys of a tile: as many bytes as the 16-bit kernel's

struct CodesParams {
    CUtensorMap mk, mv;
    Params p;
    int boxes;         // of a piece: 1, or 2 where pages have 16 rows
    bool join_launch;  // split items are joined by a second launch
};

// An 8 x 8 matrix of 16-bit values, a row's two in a lane, transposed.
__device__ __forceinline__ uint32_t turned(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two queries as the fp16 operand: a bf16 pair times its row's factor.
__device__ __forceinline__ uint32_t query_pair(__half, uint32_t w, float) { return w; }
__device__ __forceinline__ uint32_t query_pair(__nv_bfloat16, uint32_t w, float f) {
    const float2 x = Pair<__nv_bfloat16>::load(w);
    return Pair<__half>::make(x.x * f, x.y * f);
}

__device__ __forceinline__ void tma_codes(void *dst, const CUtensorMap *map, int row, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(0), "r"(row), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
// Byte of 16-byte chunk c of row r as the copy's swizzle places it.
template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) {
    return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// kN: tiles of 8 query rows.
template <typename T, int D, bool kCap, int kN>
__global__ void __launch_bounds__(kThreads, 2) attention_codes_kernel(const __grid_constant__ CodesParams sp) {
    constexpr int kPiece = kCodePiece, kTile = kCodeTile;
    constexpr int kBytes = kPiece * D;                   // of a piece's keys, or values
    constexpr int kStages = kRing / (2 * kBytes);
    constexpr bool kScaleQ = std::is_same_v<T, __nv_bfloat16>;
    constexpr int kOS = row_floats(D);
    static_assert(kMaxRows * kOS * 4 <= kRing, "a warp's sums fit its ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ __align__(16) float scales[kWarps][kStages][2][kPiece];  // of keys, of values
    __shared__ float sm_m[kWarps][kMaxRows], sm_l[kWarps][kMaxRows];
    __shared__ unsigned failed;
    __shared__ bool joins;
    __shared__ Run run_sh;
    const Params &p = sp.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    const int G = p.b.Hq / p.b.Hkv;
    const int nb = sp.boxes, box_rows = kPiece / nb;
    uint8_t *ring = smem + warp * kRing;
    if (tid == 0) {
        failed = 0;
        prefetch_map(&sp.mk);
        prefetch_map(&sp.mv);
    }
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1 + 32 + withheld(p));
    __syncwarp();
    fence_mbar_init();
    pdl_enter();
    if (sp.join_launch && tid == 0) p.desc[blockIdx.x].parts = 0;
    // Single-token calls of the experts leave tags where the parts are counted: the header says
    // whether there were any (read beside the search, looked at after it).
    const bool looks = !sp.join_launch && blockIdx.x == 0 && tid == 0;
    const unsigned long long tags = looks ? p.hdr->cta_calls : 0ull;
    Run run;
    const bool work = run_begin<kTile, true>(p, kLeast, kCodeSplit, reinterpret_cast<long *>(smem), &run_sh, run);
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
        // the queries: row 8 x + gid, four channels in a row as the codes come
        uint2 w[kN][D / 16];
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int r = 8 * x + gid, tok = r / G;
            const bool live = tok < it.nt;
            const T *row = static_cast<const T *>(p.q) +
                           (size_t(it.row0 + (live ? tok : 0)) * p.b.Hq + it.kh * G + r % G) * D;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                w[x][k] = live ? *reinterpret_cast<const uint2 *>(row + 16 * k + 4 * tig) : make_uint2(0u, 0u);
        }
        __syncwarp();
        int sent = 0;  // pieces of this segment issued
        auto issue = [&]() {
            if (sent > 0 && ((sent * nb) & 31) == 0) {
                pages = pages_next;
                pages_next = page_at(sent * nb + 32 + lane);
                __syncwarp();
            }
            const uint32_t st = issued % kStages;
            uint64_t *bar = &full[warp][st];
            const int row0 = key_of(sent) & (p.b.page - 1);
            // the scales, four keys a lane, by copies of the lanes' own
            const int kind = (lane >> 3) & 1, key = 4 * (lane & 7), box = key / box_rows;
            const int pg = __shfl_sync(0xffffffffu, pages, (sent * nb + box) & 31);
            if (lane < 16) {
                const bool there = pg < p.b.num_pages;
                // (boxes of a piece are of different pages, and begin at their first row)
                const size_t at = (size_t(there ? pg : 0) * p.b.Hkv + it.kh) * p.b.page +
                                  ((row0 + box * box_rows) & (p.b.page - 1)) + key % box_rows;
                tc::cp_async_16_zfill(&scales[warp][st][kind][key], (kind == 0 ? p.ks : p.vs) + at, there);
            }
            cp_async_arrive_noinc(bar);
            if (lane == 0) {
                uint8_t *dst = ring + st * (2 * kBytes);
                mbar_arrive_expect_tx(bar, 2 * kBytes);
                tma_codes(dst, &sp.mk, row0, pg * p.b.Hkv + it.kh, bar);
                tma_codes(dst + kBytes, &sp.mv, row0, pg * p.b.Hkv + it.kh, bar);
            }
            if (nb == 2 && lane == 4) {  // (whose keys are the second box's)
                uint8_t *dst = ring + st * (2 * kBytes) + box_rows * D;
                const int row = (row0 + box_rows) & (p.b.page - 1);
                tma_codes(dst, &sp.mk, row, pg * p.b.Hkv + it.kh, bar);
                tma_codes(dst + kBytes, &sp.mv, row, pg * p.b.Hkv + it.kh, bar);
            }
            __syncwarp();
            ++sent;
            ++issued;
        };
        for (int i = 0; i < kStages && i < n; ++i) issue();  // ahead of what has to wait for the queries

        uint32_t qb[kN][D / 16][2];
        float unit[kN][2];  // what the scores of this thread's rows (8 x + 2 tig, + 1) take back
        Sight sight[kN][2];
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            float factor = 1.f;
            if (kScaleQ) {
                float most = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const float2 a = Pair<T>::load(w[x][k].x), b = Pair<T>::load(w[x][k].y);
                    most = fmaxf(fmaxf(most, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                // 2^14 over the largest's power of two, at most 2^126
                factor = __uint_as_float(min(268u - (__float_as_uint(most) >> 23), 253u) << 23);
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qb[x][k][0] = query_pair(T(), w[x][k].x, factor);
                qb[x][k][1] = query_pair(T(), w[x][k].y, factor);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int t = (8 * x + 2 * tig + c) / G;
                // (over a power of two: the exponent's complement)
                const float f = __shfl_sync(0xffffffffu, factor, 8 * tig + 4 * c);
                unit[x][c] = kScaleQ ? __uint_as_float(0x7f000000u - __float_as_uint(f)) : 1.f;
                sight[x][c] = row_sight(p, run.seq, t < it.nt, it.row0 + t, it.qt * p.tt + t);
                __syncwarp();
            }
        }

        // sums of channels 16 c + 2 gid (o[][c][0 .. 1]) and the one after (o[][c][2 .. 3]) of this thread's rows
        float o[kN][D / 16][4], mx[kN][2], l[kN][2];
        float re[kN][2], rf[kN][2];  // the rows' e, and 2^(kLift - e)
        float enough[kN][2];         // scores up to here move no reference
        // the scales that the pieces so far had, from `range` (their bits) to kSpread above it, and the logarithm
        // of a power of two above those
        uint32_t range = 0x80000000u;  // none
        float range_log2 = 0.f;
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            mx[x][0] = mx[x][1] = -CUDART_INF_F;
            l[x][0] = l[x][1] = 0.f;
            re[x][0] = re[x][1] = 0.f;
            rf[x][0] = rf[x][1] = 1.f;
            enough[x][0] = enough[x][1] = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.f;
        }
        auto bounded = [&](int x, int c) { enough[x][c] = mx[x][c] + fminf(kGrowth, re[x][c] + kGrowth - range_log2); };

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
            // S^T: matrices of keys 8 j .. 8 j + 7, the same 16 channels of each; s[][t]: keys 16 t + gid, + 8
            float s[kN][2][4];
#pragma unroll
            for (int x = 0; x < kN; ++x)
#pragma unroll
                for (int t = 0; t < 2; ++t) s[x][t][0] = s[x][t][1] = s[x][t][2] = s[x][t][3] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                ldsm4(b, kb + code_chunk<D>(lane, k));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const CodePair<__half> lo(b[2 * t]), hi(b[2 * t + 1]);
                    const uint32_t a[4] = {lo.template take<0, 1>(), hi.template take<0, 1>(), lo.template take<2, 3>(),
                                           hi.template take<2, 3>()};
#pragma unroll
                    for (int x = 0; x < kN; ++x) mma16816<__half>(s[x][t], a, qb[x][k][0], qb[x][k][1]);
                }
            }
            // keys that some row does not see
            const int all = p.tree != nullptr ? run.seq.len - run.seq.n - 1 : it.pos0;
            const bool edge = key0 + kPiece - 1 > all ||
                              (p.window > 0 && key0 <= last - p.window && key0 + kPiece > p.sinks);
            // the scales of keys 8 j + gid; the values' past the sequence's end hold anything, and a weight of 0
            // takes them
            const bool tail = key0 + kPiece > it.len;
            float kf[4], vf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kf[j] = ks[8 * j + gid];
                vf[j] = tail && key0 + 8 * j + gid >= it.len ? 0.f : vs[8 * j + gid];
            }
            bool apart = false;  // the piece's scales are: the rows' products are looked for key by key
            const uint32_t mine = scale_bits(vs[lane]);
            if (!__all_sync(0xffffffffu, mine - range <= kSpread)) {
                // (of keys that some row may see)
                bool none = edge && (key0 + lane >= it.len || (key0 + lane >= p.sinks && key0 + lane < it.seen));
                const uint32_t odd = __ballot_sync(0xffffffffu, mine >= kInfinity);
                if (odd != 0u) {
                    // values that are not finite make the rows that see them NaN; the others' weights are 0, and
                    // so must those be
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (scale_bits(vf[j]) >= kInfinity) vf[j] = 0.f;
#pragma unroll
                    for (int x = 0; x < kN; ++x)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if ((sight32(p, run.seq, sight[x][c], key0) & odd) != 0u) l[x][c] = CUDART_NAN_F;
                    none = none || mine >= kInfinity;
                    __syncwarp();
                }
                const uint32_t hi = __reduce_max_sync(0xffffffffu, none ? 0u : mine);
                const uint32_t lo = min(hi, __reduce_min_sync(0xffffffffu, none ? 0xffffffffu : mine));
                apart = hi - lo > kSpread;
                if (!apart && (lo < range || hi - range > kSpread)) {
                    range = min(lo - min(lo, (kSpread - (hi - lo)) / 2), kInfinity - 1 - kSpread);
                    range_log2 = scale_log2(range + kSpread);
#pragma unroll
                    for (int x = 0; x < kN; ++x) bounded(x, 0), bounded(x, 1);
                }
            }
            // The rows' reference maxima, and with them the sums, follow the scores only where one has grown by
            // more than 2^kGrowth since (weights up to that are as exact in 16 bits as those up to 1, and
            // the sums are fp32): in a short range new maxima are frequent.  So do the references of the products.
            float v[kN][2];  // the rows' largest scores
            bool grows = apart;
#pragma unroll
            for (int x = 0; x < kN; ++x)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t sees = 0xffffffffu;
                    if (edge) sees = sight32(p, run.seq, sight[x][c], key0) >> gid;
                    float top = -CUDART_INF_F;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float &z = s[x][j >> 1][2 * (j & 1) + c];
                        z = score<kCap>(z * (kScaleQ ? kf[j] * unit[x][c] : kf[j]), p);
                        if (edge && (sees >> (8 * j) & 1u) == 0u) z = -CUDART_INF_F;
                        top = fmaxf(top, z);
                    }
                    __syncwarp();
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                    v[x][c] = top;
                    grows = grows || top > enough[x][c];
                }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int x = 0; x < kN; ++x) {
                    float cor[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float up = fmaxf(mx[x][c], v[x][c]), base = up == -CUDART_INF_F ? 0.f : up;
                        float product = v[x][c] + range_log2;  // the row's largest of the piece (log2)
                        if (apart) {
                            product = -CUDART_INF_F;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                product = fmaxf(product, s[x][j >> 1][2 * (j & 1) + c] + scale_log2(scale_bits(vf[j])));
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1)
                                product = fmaxf(product, __shfl_xor_sync(0xffffffffu, product, w));
                        }
                        const float e = ref_exponent(fmaxf(mx[x][c] + re[x][c], product), base);
                        l[x][c] *= exp2_approx(mx[x][c] - base);  // -inf: nothing seen yet
                        cor[c] = exp2_approx((mx[x][c] - base) + (re[x][c] - e));
                        mx[x][c] = up;
                        re[x][c] = e;
                        rf[x][c] = power_of_2(kLift - e);
                        bounded(x, c);
                    }
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[x][j][0] *= cor[0], o[x][j][1] *= cor[1];
                        o[x][j][2] *= cor[0], o[x][j][3] *= cor[1];
                    }
                }
            }
            // the weights times the values' scales, rounded to fp16 for the product (its two operands have one
            // type); the sum l keeps the weights whole
            uint32_t pb[kN][2][2];
#pragma unroll
            for (int x = 0; x < kN; ++x) {
                const unsigned long long rf2 = pack2(rf[x][0], rf[x][1]);
                float base[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) base[c] = mx[x][c] == -CUDART_INF_F ? 0.f : mx[x][c];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = exp2_approx(s[x][j >> 1][2 * (j & 1)] - base[0]);
                    const float b = exp2_approx(s[x][j >> 1][2 * (j & 1) + 1] - base[1]);
                    l[x][0] += a;
                    l[x][1] += b;
                    float wa, wb;
                    unpack2(mul2(mul2(pack2(a, b), rf2), pack2(vf[j], vf[j])), wa, wb);
                    pb[x][j >> 1][j & 1] = turned(Pair<__half>::make(wa, wb));
                }
            }
            // O^T: matrices (keys 0-7 and 8-15 of 16, channel chunk c), then of chunk c + 1, transposed
            const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < D / 16; c += 2) {
                    uint32_t b[4];
                    ldsm4_trans(b, vb + code_chunk<D>(16 * t + vrow, c + vc));
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const CodePair<__half> lo(b[2 * y]), hi(b[2 * y + 1]);
                        const uint32_t a[4] = {lo.template take<0, 2>(), lo.template take<1, 3>(),
                                               hi.template take<0, 2>(), hi.template take<1, 3>()};
#pragma unroll
                        for (int x = 0; x < kN; ++x) mma16816<__half>(o[x][c + y], a, pb[x][t][0], pb[x][t][1]);
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
        __syncwarp();
#pragma unroll
        for (int x = 0; x < kN; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float sum = l[x][c];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                const int r = 8 * x + 2 * tig + c;
                const float back = power_of_2(re[x][c] - kLift);
                if (gid == 0) {
                    sm_m[warp][r] = mx[x][c];
                    sm_l[warp][r] = sum;
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    *reinterpret_cast<float2 *>(so + r * kOS + 16 * j + 2 * gid) =
                        make_float2(o[x][j][c] * back, o[x][j][2 + c] * back);
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

// f on every form of the kernel for a type.
template <typename T, typename F>
void each_codes(F f) {
    f(attention_codes_kernel<T, 64, false, 1>);
    f(attention_codes_kernel<T, 64, false, 2>);
    f(attention_codes_kernel<T, 64, true, 1>);
    f(attention_codes_kernel<T, 64, true, 2>);
    f(attention_codes_kernel<T, 128, false, 1>);
    f(attention_codes_kernel<T, 128, false, 2>);
    f(attention_codes_kernel<T, 128, true, 1>);
    f(attention_codes_kernel<T, 128, true, 2>);
}

cudaError_t init_stream_codes() {
    cudaError_t e = cudaSuccess;
    auto set = [&](auto kernel) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCodesSmem);
    };
    each_codes<__half>(set);
    each_codes<__nv_bfloat16>(set);
    return e;
}

cudaError_t launch_stream_codes(const AttnArgs &a, Params p, int max_new, int num_sms, cudaStream_t s) {
    CodesParams sp = {};
    const int G = a.b.Hq / a.b.Hkv, tiles = long(max_new) * G <= 8 ? 1 : 2;
    p.tt = 8 * tiles / G;
    p.tt_magic = 0xffffffffu / unsigned(p.tt) + 1;
    p.extra = kExtra;
    sp.p = p;
    sp.boxes = a.b.page < kCodePiece ? 2 : 1;
    const int box_rows = kCodePiece / sp.boxes;
    if (!encode_codes_map(&sp.mk, a.k, a.b, box_rows, false) || !encode_codes_map(&sp.mv, a.v, a.b, box_rows, false))
        return cudaErrorInvalidValue;
    const int grid = std::min(2 * num_sms, kMaxCtas);
    sp.join_launch = joins_by_launch(a.b, grid, kCodeTile, kCodeJoinInside);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(grid), dim3(kThreads), size_t(kCodesSmem), s, sp);
    };
    auto of = [&](auto type, auto cap, auto n) {
        using T = decltype(type);
        constexpr bool kCap = decltype(cap)::value;
        constexpr int kN = decltype(n)::value;
        return a.b.D == 64 ? go(attention_codes_kernel<T, 64, kCap, kN>) : go(attention_codes_kernel<T, 128, kCap, kN>);
    };
    auto rows = [&](auto type, auto cap) {
        return tiles == 1 ? of(type, cap, std::integral_constant<int, 1>()) : of(type, cap, std::integral_constant<int, 2>());
    };
    auto with = [&](auto type) { return p.cap_in != 0.f ? rows(type, std::true_type()) : rows(type, std::false_type()); };
    const cudaError_t e = a.type == MOE_F16 ? with(__half()) : with(__nv_bfloat16());
    if (e != cudaSuccess || !sp.join_launch) return e;
    return launch_join(p, a.type, grid, kPartRows, kPartRows, p.tt, s);
}

}  // namespace attn
}  // namespace moeq4k
