// Attention of many query rows per key/value head (chunks of prompts) on the
// tensor cores: S = Q K^T and O += P V by tcgen05 with Q, K, V in shared
// memory and S, P, O in tensor memory.
//
// An item is two halves of 128 query rows (tokens x the group's heads) that
// share every key tile of 128 keys.  Nineteen warps (24 over codes): for each half eight
// softmax warps (two threads per row, half the keys each), a warp that issues the
// MMAs, and two that copy (K tiles with the queries, V tiles; TMA boxes of
// one page at most).  The two halves take turns on the tensor pipe: while one
// half's P V and next Q K^T run, the other half's softmax does.  P overwrites S
// in tensor memory and is the A operand from there; a thread's first 32 keys
// are handed over as soon as they are written.  O is rescaled only when a row's
// maximum has grown by more than 2^8 since the last rescale (weights up to 2^8
// are as exact in 16 bits as those up to 1, and sums are fp32), so most
// tiles leave O alone.  Tensor memory: S/P of half h at column 128 h, O of half h
// at 256 + 128 h.
//
// What bounds it: without a cap shared memory (each of the two products reads
// its 32 KB tile from there once per half, next to the copies' writes) and the tensor
// pipe: a chunk of 2048 rows over 16384 keys, 32/4 heads of 128, takes 337 us
// = 1.53 PFLOP/s.  With a cap the exponentials and reciprocals, 10 cycles a
// warp for 32 scores, and their arithmetic do: 448 us.  Short ranges pay for
// their segments' ends (the last softmax, the result, the first softmax: 3 tiles'
// time): a prompt of 4096, 117 us = 1.18 PFLOP/s.  One thread per row
// (four warps a half) was slower by the latency of its chain: the capped chunk 613
// against 465 us, the prompt 2 us faster.
//
// Three forms are built of it.  kPaged: chains in a window.  kMasked: trees and sinks too; a
// tile that some row does not see whole takes a bit a key from its row's mask, the others are
// as before (16 trees of 48 to 64 nodes over 900 to 8100 keys, 64/4 heads: 104 us = 1.02
// PFLOP/s).  kCodes: the same over 8-bit codes.  Their copies land in a ring of their own, six
// more warps spread them to the 16-bit tiles that the products read (every code is exact
// there), and the scales come in the softmax: K's as a factor of the scores, in fp32, V's as
// one of the weights before those are rounded.  80 registers a thread are left for that, so
// each warp's run lies in shared memory.  The chunk of 2048 over 16384 takes 529 us = 0.97
// PFLOP/s (fp16, whose rows have references of their own for V's scales: 545), with a cap 697:
// the memory's bytes are half, but the issue slots (62 % used) and the path to shared memory
// (57 %, beside the products' own reads) now carry the codes' conversion and 768 loads of scales a
// tile; when it took 583 us it took 465 without the conversion, when 529 (an earlier form) 493
// without the softmax's scales.
#pragma once

#include <algorithm>
#include <type_traits>

#include <cuda.h>

#include "attention.cuh"
#include "codes.cuh"
#include "f32x2.cuh"
#include "tcgen05.cuh"

namespace moeq4k {
namespace attn {
namespace tc5 {

constexpr int kHalf = 128;                 // rows of a half
constexpr int kKeys = 128;                 // keys of a tile
constexpr int kSoftmaxWarps = 16;
constexpr int kCopyWarps = 2;               // K tiles, V tiles
constexpr int kMmaWarp = kSoftmaxWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kCopyWarps);
// Over 8-bit codes: a copying warp, and six that spread the codes, a piece of a tile each in turn.
constexpr int kConvertWarp = kCopyWarp + 1, kConvertWarps = 6;
constexpr int kPieceRows = 32;
constexpr int kCodesThreads = 32 * (kConvertWarp + kConvertWarps);
constexpr int kMaxGrid = kMaxCtas / 2;     // one CTA per SM
// The least work of a CTA, and an item's fixed cost, in key tiles (a cost of 1, 2, 3:
// a prompt of 4096 139, 117, 118 us, four of 1024 64, 52.5, 55 us).
constexpr int kLeast = 2;
constexpr int kExtra = 2;
// What parting items costs, in key tiles: 64 tokens over 500 of eight sequences take 17.3 us
// whole and 20.7 in parts, a prompt of 300 12.8 and 15.2, of 1200 26.2 and 28.1; 8 tokens over
// 500 of eight 14.5 and 13.2.
constexpr int kSplit = 5;
constexpr float kGrowth = 8.f;             // log2 growth of the maximum that forces a rescale
constexpr float kTanhOne = 30.f;           // 2^-30 from 1 is 1 in fp32
constexpr float kTanhMinusOne = -64.f;     // 1 + 2^-64 is 1, and the tangent -1

// What a kernel is built for: chains in a window (moe_attention_paged), trees and sinks, or
// both over 8-bit codes.
enum Form { kPaged, kMasked, kCodes };
constexpr int form_threads(int form) { return form == kCodes ? kCodesThreads : kThreads; }

struct TcParams {
    CUtensorMap mq, mk, mv;
    CUtensorMap mks, mvs;  // the scales of codes
    Params p;          // p.tt: tokens of an item (both halves)
    int tth;           // tokens of a half
    int box_rows;      // rows of a K/V box
    uint32_t idesc_qk, idesc_pv;
};

template <int D, int kForm>
struct Cfg {
    static constexpr int kCh = D / 64;                 // 64-channel slabs of a row
    static constexpr int kSlab = 128 * 128;            // bytes of a 128-row slab
    static constexpr int kTileB = kCh * kSlab;         // a tile of K, of V, or of a half's Q
    static constexpr bool kQ8 = kForm == kCodes;
    static constexpr int kStages = kQ8 ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
    static constexpr int kQAt = kStages * kTileB;
    // Results on their way out, 32 rows x 32 channels of each softmax warp (over codes, whose form has
    // no room for them, only what two warps exchange).
    static constexpr int kStageOut = kQ8 ? 256 : 32 * 64;
    static constexpr int kOutAt = kQAt + 2 * kTileB;
    // Codes: the ring of tiles as they are copied, their scales (of each box on 128 bytes), and the scales as
    // the softmax reads them, K's and V's of a tile.  Those are written when the tile kStages before has
    // been used: for the keys' that says that the softmax is done with the tile kScaleTiles before.
    static constexpr int kSlots = 3;
    static constexpr int kCodesAt = kOutAt + kSoftmaxWarps * kStageOut;
    static constexpr int kCodeScalesAt = kCodesAt + (kQ8 ? kSlots * kKeys * D : 0);
    static constexpr int kScalesAt = kCodeScalesAt + (kQ8 ? kSlots * 1024 : 0);
    static constexpr int kScaleTiles = D == 128 ? 2 : 4;
    static constexpr int kSmem = kScalesAt + (kQ8 ? kScaleTiles * 2 * kKeys * 4 : 0);
    // A converting warp sees every use of the slots and places that it uses.
    static_assert(!kQ8 || (kStages * (kKeys / kPieceRows) % kConvertWarps == 0 &&
                           kSlots * (kKeys / kPieceRows) % kConvertWarps == 0), "the warps' pieces repeat with the rings");
};

__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_box2(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A holds two 16-bit values of a row per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}

// Descriptor of an operand whose rows of 64 values are its K (here: V's keys)
// and whose columns, contiguous, are its N: 128-byte swizzle, 8-row groups
// 1024 B apart, the next 64 columns `slab` bytes on.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t slab) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFF);
    d |= uint64_t((slab >> 4) & 0x3FFF) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

#define R4(a, i) "=f"(a[i]), "=f"(a[i + 1]), "=f"(a[i + 2]), "=f"(a[i + 3])
#define W4(a, i) "+f"(a[i]), "+f"(a[i + 1]), "+f"(a[i + 2]), "+f"(a[i + 3])
#define F4(a, i) "f"(a[i]), "f"(a[i + 1]), "f"(a[i + 2]), "f"(a[i + 3])
#define S4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
// 32 consecutive columns of this thread's lane; the values are there after wait_ld32.
__device__ __forceinline__ void tmem_ld32(uint32_t t, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : R4(v, 0), R4(v, 4), R4(v, 8), R4(v, 12), R4(v, 16), R4(v, 20), R4(v, 24), R4(v, 28)
        : "r"(t));
}
__device__ __forceinline__ void wait_ld32(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : W4(v, 0), W4(v, 4), W4(v, 8), W4(v, 12), W4(v, 16), W4(v, 20), W4(v, 24), W4(v, 28)
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16};" ::"r"(t),
        S4(v, 0), S4(v, 4), S4(v, 8), S4(v, 12)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), S4(v, 0), S4(v, 4)
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        F4(v, 0), F4(v, 4), F4(v, 8), F4(v, 12), F4(v, 16), F4(v, 20), F4(v, 24), F4(v, 28)
        : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t t, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
        "[%16];"
        : R4(v, 0), R4(v, 4), R4(v, 8), R4(v, 12)
        : "r"(t));
}
__device__ __forceinline__ void wait_ld16(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : W4(v, 0), W4(v, 4), W4(v, 8), W4(v, 12) : : "memory");
}
#undef R4
#undef W4
#undef S4
#undef F4

__device__ __forceinline__ bool elect_one() {
    uint32_t is = 0;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(is));
    return is != 0u;
}

// The whole warp waits for a phase; recorded when it runs out.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Params &p, int who,
                                          uint64_t limit_ns) {
    const bool ok = __all_sync(0xffffffffu, wait_phase(bar, parity, limit_ns));
    if (!ok) record_status(p.hdr, MOE_ERR_TIMEOUT, who);
    return ok;
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Params &p, int who) {
    return warp_wait(bar, parity, p, who, p.wait_ns);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The larger and the smaller of two, a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four values times four scales (16-byte aligned).
__device__ __forceinline__ void scaled(const float *v, const float *scales, float *r) {
    const float4 f = *reinterpret_cast<const float4 *>(scales);
    unpack2(mul2(pack2(v[0], v[1]), pack2(f.x, f.y)), r[0], r[1]);
    unpack2(mul2(pack2(v[2], v[3]), pack2(f.z, f.w)), r[2], r[3]);
}

// The CTA's run in registers, or in shared memory as each warp's own.
template <bool kShared>
__device__ __forceinline__ Run &run_place(Run &found, Run &mine) {
    if (!kShared) return found;
    if ((threadIdx.x & 31) == 0) mine = found;
    __syncwarp();
    return mine;
}

// The copies of a segment's tiles in the form over codes, by one warp: a lane for each box's codes
// and one for its scales.  `g`: tiles (K, V, K, ..) of the segments before.
template <int D>
__device__ __forceinline__ bool copy_codes(const TcParams &tp, const Item &it, int s0, int n, uint32_t &g, uint8_t *smem,
                                           uint64_t *landed, uint64_t *taken) {
    using C = Cfg<D, kCodes>;
    const Params &p = tp.p;
    const int lane = threadIdx.x & 31, box = lane >> 1, rows = tp.box_rows, boxes = kKeys / rows;
    auto page_z = [&](int j) {  // page-head of this lane's box of tile j
        if (j >= n || box >= boxes) return 0;
        // past the tensor, read as zeros: a box past the end, one between the sinks and every row's
        // window (its page may be gone already) and a bad page
        const int key = tile_key<kKeys, true>(it, s0 + j) + box * rows;
        const int pg = key >= it.len || (key + rows <= it.seen && key >= p.sinks) ? -1 : page_of(p.b, it.b, key, p.hdr);
        return (pg < 0 ? p.b.num_pages : pg) * p.b.Hkv + it.kh;
    };
    int z_next = page_z(0);
    for (int j = 0; j < n; ++j) {
        const int z = z_next, row = (tile_key<kKeys, true>(it, s0 + j) + box * rows) & (p.b.page - 1);
        z_next = page_z(j + 1);
        for (int kv = 0; kv < 2; ++kv, ++g) {
            const uint32_t slot = g % C::kSlots;
            if (g >= uint32_t(C::kSlots) && !warp_wait(&taken[slot], (g / C::kSlots - 1) & 1u, p, 51 + kv)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&landed[slot], kKeys * D + kKeys * 4);
            __syncwarp();
            if (box < boxes) {
                if ((lane & 1) == 0)
                    tma_box3(smem_addr(smem) + C::kCodesAt + slot * (kKeys * D) + box * rows * D,
                             kv == 0 ? &tp.mk : &tp.mv, 0, row, z, &landed[slot]);
                else
                    tma_box2(smem_addr(smem) + C::kCodeScalesAt + slot * 1024 + box * max(rows * 4, 128),
                             kv == 0 ? &tp.mks : &tp.mvs, row, z, &landed[slot]);
            }
            __syncwarp();
        }
    }
    return true;
}

// A converting warp of the form over codes.  The pieces of the tiles, 32 rows each, go round the
// warps.  A warp spreads its piece to the 16-bit tile that the products read (8-row groups
// of 1024 bytes, 128 a row, swizzled), once that place is free, and puts the scales where
// the softmax reads them (K's times `k_unit`).  A thread has 16 codes of a row at a time, which
// become two chunks of 16 bytes.  Eight lanes have four chunks of one row and the same four
// of another, of the other parity (r and r ^ 5 where rows are 128 bytes of codes, which the copy
// swizzles by the row), so that their loads and their stores go to different banks.
//
// The products wait for the place's release and then for these warps, so what can be done
// ahead of the release is: the codes are in registers, half of them as operands.  (Where these
// warps also made the copies, a piece took them 3900 cycles, a third of it in the copies'
// issue.)
template <typename T, int D, typename F>
__device__ __forceinline__ void convert_tiles(const TcParams &tp, float k_unit, const Run &run, F next, uint8_t *smem,
                                              uint64_t *landed, uint64_t *taken, uint64_t *empty, uint64_t *conv,
                                              volatile int *odd) {
    using C = Cfg<D, kCodes>;
    constexpr int kRowsAtOnce = 512 / D, kSteps = kPieceRows / kRowsAtOnce;  // of a piece
    constexpr int kAhead = kSteps / 2, kTilePieces = kKeys / kPieceRows;
    const Params &p = tp.p;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kConvertWarp;
    // this thread's chunk of its row, and its row of step k
    const int c = D == 128 ? (lane & 3) + ((lane >> 3) & 1) * 4 : lane & 3;
    auto row_of = [&](int k) {
        if (D == 64) return k * kRowsAtOnce + (lane >> 2);
        const int r = (k & 1) * 2 + (lane >> 4);
        return k / 2 * 8 + ((lane & 4) != 0 ? r ^ 5 : r);
    };
    uint32_t piece = warp, g0 = 0;  // of all pieces; tiles of the segments before
    bool ok = true;
    while (ok && run.u < run.end) {
        int s0, s1;
        if (!run_segment(p, run, s0, s1)) break;
        const uint32_t end = g0 + 2 * (s1 - s0);
        const int len = run.item.len, ts = run.item.ts, t0 = run.item.t0, seen = run.item.seen;
        for (; piece / kTilePieces < end; piece += kConvertWarps) {
            const uint32_t g = piece / kTilePieces, quarter = piece % kTilePieces;
            const uint32_t st = g % C::kStages, slot = g % C::kSlots;
            const bool value = (g & 1) != 0;
            if (!(ok = warp_wait(&landed[slot], (g / C::kSlots) & 1u, p, 67))) break;
            const uint8_t *codes = smem + C::kCodesAt + slot * (kKeys * D) + quarter * kPieceRows * D;
            uint4 x[kSteps];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int r = row_of(k);
                x[k] = *reinterpret_cast<const uint4 *>(codes + r * D + ((D == 128 ? c ^ (r & 7) : c) << 4));
            }
            const int key_in = quarter * kPieceRows + lane;
            const int spread = tp.box_rows == 16 ? (key_in >> 4) * 32 + (key_in & 15) : key_in;
            const float f = reinterpret_cast<const float *>(smem + C::kCodeScalesAt + slot * 1024)[spread];
            fence_proxy_async_smem();  // these reads before the next copy into their place
            __syncwarp();
            if (lane == 0) mbar_arrive(&taken[slot]);
            __syncwarp();
            auto wide = [&](const uint4 &v, uint4 &first, uint4 &second) {
                const CodePair<T> a(v.x), b(v.y), d(v.z), e(v.w);
                first = make_uint4(a.template take<0, 1>(), a.template take<2, 3>(), b.template take<0, 1>(),
                                   b.template take<2, 3>());
                second = make_uint4(d.template take<0, 1>(), d.template take<2, 3>(), e.template take<0, 1>(),
                                    e.template take<2, 3>());
            };
            uint4 w[kAhead][2];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) wide(x[k], w[k][0], w[k][1]);
            if (g >= uint32_t(C::kStages) && !(ok = warp_wait(&empty[st], (g / C::kStages - 1) & 1u, p, 68))) break;
            uint8_t *tile = smem + st * C::kTileB + quarter * kPieceRows * 128 + (c >> 2) * C::kSlab;
            auto store = [&](int k, const uint4 &first, const uint4 &second) {
                const int r = row_of(k), chunk = 2 * (c & 3);
                *reinterpret_cast<uint4 *>(tile + r * 128 + ((chunk ^ (r & 7)) << 4)) = first;
                *reinterpret_cast<uint4 *>(tile + r * 128 + (((chunk + 1) ^ (r & 7)) << 4)) = second;
            };
#pragma unroll
            for (int k = 0; k < kAhead; ++k) store(k, w[k][0], w[k][1]);
#pragma unroll
            for (int k = kAhead; k < kSteps; ++k) {
                uint4 first, second;
                wide(x[k], first, second);
                store(k, first, second);
            }
            // past the sequence's end the scales may be anything.  A key's is above 0: a hidden score is an
            // infinity, which 0 would make a NaN (the codes of a scale of 0 are 0 themselves).  For the same reason one
            // that is not finite becomes an infinity: times the codes 0 it gives NaN to the rows that see it.
            // A value's of a key that no row sees is -0.0, and so is one that is not finite: what it makes NaN is found
            // at the segment's end, where `odd` says that there is any.  All others are positive or 0.
            const int i = s0 + int((g - g0) >> 1), key = (i < ts ? i : t0 - ts + i) * kKeys + key_in;
            const bool past = key >= len;
            const float kf = fminf(f, CUDART_INF_F) * k_unit;  // (of a NaN an infinity)
            float vf = past || (key >= p.sinks && key < seen) ? -0.f : fabsf(f);
            if (value && scale_bits(vf) >= kInfinity) {
                vf = -0.f;
                *odd = 1;
            }
            reinterpret_cast<float *>(smem + C::kScalesAt)[((g >> 1) % C::kScaleTiles) * (2 * kKeys) +
                                                           (value ? kKeys : 0) + key_in] =
                value  ? vf
                : past ? 1.f
                       : (kf <= 1.4e-45f ? 1.4e-45f : kf);
            fence_proxy_async_smem();  // these stores before the products' reads of them
            __syncwarp();
            if (lane == 0) mbar_arrive(&conv[st]);
            __syncwarp();
        }
        g0 = end;
        next();
    }
}

// Whether the row sees one of a segment's keys whose value's scale is not finite, in 64 keys of each tile from
// `at` on; the whole warp calls it.
static __device__ __noinline__ bool sees_odd(const Params &p, const SeqView &s, const Item &it, const Sight &sight,
                                             int s0, int s1, int at) {
    const int lane = threadIdx.x & 31;
    bool sees = false;
    for (int i = 2 * s0; i < 2 * s1; ++i) {
        const int key0 = tile_key<kKeys, true>(it, i >> 1) + at + 32 * (i & 1), key = key0 + lane;
        bool is = false;
        if (key < it.len && (key < p.sinks || key >= it.seen)) {
            const int pg = page_of(p.b, it.b, key, p.hdr);
            is = pg >= 0 && scale_bits(p.vs[(size_t(pg) * p.b.Hkv + it.kh) * p.b.page + key % p.b.page]) >= kInfinity;
        }
        const uint32_t odd = __ballot_sync(0xffffffffu, is);
        sees = sees || (odd != 0u && (sight32(p, s, sight, key0) & odd) != 0u);
        __syncwarp();
    }
    return sees;
}

// How a score follows from q.k: by a positive scale, capped after a positive
// scale, or in any other way (negative and zero scales, caps past kCapNear).
enum Mode { kScaled, kCapped, kAny };

// kCapped takes the tangent from 1 - 2 / (1 + e^2y) alone: its error is at most
// 2^-21 of the cap, up to this cap 2^-15, a few fp32 steps of the scores that the cap
// lets through.  Caps beyond go to kAny, whose scores are score()'s (2048 rows over 16384
// keys: 448 us, by kAny 550; 939 before scores far below the cap left out the exponential).
constexpr float kCapNear = 64.f;

template <typename T, int D, int kMode, int kForm>
__global__ void __launch_bounds__(form_threads(kForm), 1) attention_tc_kernel(const __grid_constant__ TcParams tp) {
    using C = Cfg<D, kForm>;
    constexpr bool kMasks = kForm != kPaged, kQ8 = kForm == kCodes, kRef = kQ8 && std::is_same_v<T, __half>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], q_full, q_empty, s_full[2], p_ready[2][2],
        o_full[2], drain, conv[kQ8 ? C::kStages : 1], landed[C::kSlots], taken[C::kSlots];
    __shared__ int odd;  // values that are not finite have been met
    __shared__ uint32_t tmem_base;
    __shared__ Run run_sh;
    __shared__ Run run_of[kQ8 ? kCodesThreads / 32 : 1];  // each warp's own, where registers are few
    const Params &p = tp.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.b.Hq / p.b.Hkv;
    uint8_t *q_smem = smem + C::kQAt;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(&s_full[h], 1), mbar_init(&o_full[h], 1);
            mbar_init(&p_ready[h][0], 8 + withheld(p)), mbar_init(&p_ready[h][1], 8);
        }
        mbar_init(&drain, 1);
        if (kQ8) {
            for (int i = 0; i < C::kStages; ++i) mbar_init(&conv[i], kKeys / kPieceRows);
            for (int i = 0; i < C::kSlots; ++i) mbar_init(&landed[i], 1), mbar_init(&taken[i], kKeys / kPieceRows);
        }
        odd = 0;
        prefetch_map(&tp.mq);
        prefetch_map(&tp.mk);
        prefetch_map(&tp.mv);
        if (kQ8) prefetch_map(&tp.mks), prefetch_map(&tp.mvs);
    }
    __syncwarp();
    fence_mbar_init();
    pdl_enter();
    if (tid == kCopyWarp * 32) p.desc[blockIdx.x].parts = 0;
    __syncwarp();
    Run found;
    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, 512);  // beside the search
    tc::fence_before_sync();
    const bool work = run_begin<kKeys, kMasks>(p, kLeast, kSplit, reinterpret_cast<long *>(smem), &run_sh, found);
    Run &run = run_place<kQ8>(found, run_of[kQ8 ? warp : 0]);
    auto next = [&]() {
        if (kQ8) {
            __syncwarp();
            if (lane == 0) run_next<kKeys, kMasks>(p, run);
            __syncwarp();
        } else {
            run_next<kKeys, kMasks>(p, run);
        }
    };
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base;
    if (!work) {
        if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
        return;
    }
    fence_proxy_async_smem();  // the sequences' costs (generic) before the copies into the ring
    __syncthreads();

    if (kQ8 && warp >= kConvertWarp) {
        const float k_unit = kMode == kScaled ? p.scale_log2 : kMode == kCapped ? p.cap_in : 1.f;
        convert_tiles<T, D>(tp, k_unit, run, next, smem, landed, taken, empty, conv, &odd);
    } else if (warp >= kCopyWarp && warp < kCopyWarp + (kQ8 ? 1 : kCopyWarps)) {
        // ---- Q of each segment and its K tiles, or its V tiles
        const int me = warp - kCopyWarp;
        const int nbox = kKeys / tp.box_rows;  // boxes of a tile, one lane each
        uint32_t g = 0, seg = 0;               // tiles copied, segments
        bool ok = true;
        while (ok && run.u < run.end) {
            int s0, s1;
            if (!run_segment(p, run, s0, s1)) break;
            const std::conditional_t<kQ8, const Item &, const Item> it = run.item;
            const int halves = it.nt > tp.tth ? 2 : 1;
            if (me == 0 && seg > 0 && !(ok = warp_wait(&q_empty, (seg - 1) & 1u, p, 50))) break;
            if (me == 0 && lane == 0) {
                mbar_arrive_expect_tx(&q_full, uint32_t(halves) * C::kCh * G * tp.tth * 128);
                for (int h = 0; h < halves; ++h)
                    for (int c = 0; c < C::kCh; ++c)
                        tma_box3(smem_addr(q_smem) + h * C::kTileB + c * C::kSlab, &tp.mq, c * 64, it.kh * G,
                                 it.row0 + h * tp.tth, &q_full);
            }
            ++seg;
            if (me == 0 && lane == 0 && s0 == 0 && s1 < it.tiles) p.desc[blockIdx.x] = join_desc(p, run);
            __syncwarp();
            if constexpr (kQ8) {
                ok = copy_codes<D>(tp, it, s0, s1 - s0, g, smem, landed, taken);
                next();
                continue;
            }
            auto page_z = [&](int j) {  // page-head of this lane's box of tile j
                const int key = tile_key<kKeys, kMasks>(it, s0 + j) + lane * tp.box_rows;
                if (j >= s1 - s0 || lane >= nbox || key >= it.len) return 0;
                // past the tensor, read as zeros: a box before every row's window (its page may be
                // gone already) and a bad page
                const int pg = key + tp.box_rows <= it.seen && (!kMasks || key >= p.sinks)
                                   ? -1
                                   : page_of(p.b, it.b, key, p.hdr);
                return (pg < 0 ? p.b.num_pages : pg) * p.b.Hkv + it.kh;
            };
            int z_next = page_z(0);
            for (int j = 0; ok && j < s1 - s0; ++j) {
                const int z = z_next;
                z_next = page_z(j + 1);
                const int key0 = tile_key<kKeys, kMasks>(it, s0 + j);
                const int key = key0 + lane * tp.box_rows, row = key & (p.b.page - 1);
                const bool mine = lane < nbox && key < it.len;
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
                for (int kv = 0; kv < 2; ++kv, ++g) {
                    // a ring slot has one copying warp (K tiles the first, V tiles the second): the
                    // parity of its phases says something only to who waits for each of them
                    if (kv != me) continue;
                    const uint32_t st = g % C::kStages;
                    if (g >= uint32_t(C::kStages) &&
                        !(ok = warp_wait(&empty[st], (g / C::kStages - 1) & 1u, p, 51 + kv)))
                        break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], boxes * C::kCh * tp.box_rows * 128);
                    __syncwarp();
                    if (mine) {
                        const uint32_t dst = smem_addr(smem) + st * C::kTileB + lane * tp.box_rows * 128;
#pragma unroll
                        for (int c = 0; c < C::kCh; ++c)
                            tma_box3(dst + c * C::kSlab, kv == 0 ? &tp.mk : &tp.mv, c * 64, row, z, &full[st]);
                    }
                    __syncwarp();
                }
            }
            next();
        }
        // this warp's last copies land before the CTA exits, whoever else gave up on what: the MMA
        // warp may have left by a time-out of its own and not waited for them
        if (kQ8)
            for (uint32_t i = 0; i < uint32_t(C::kSlots) && i < g; ++i)
                warp_wait(&landed[(g - 1 - i) % C::kSlots], ((g - 1 - i) / C::kSlots) & 1u, p, 53, kDrainNs);
        for (uint32_t i = 0; !kQ8 && i < uint32_t(C::kStages) && i < g; ++i) {
            const uint32_t gg = g - 1 - i;
            if (int(gg % 2) == me) warp_wait(&full[gg % C::kStages], (gg / C::kStages) & 1u, p, 53, kDrainNs);
        }
        if (me == 0 && seg > 0) warp_wait(&q_full, (seg - 1) & 1u, p, 54, kDrainNs);
    } else if (warp == kMmaWarp) {
        // ---- the MMAs; the whole warp walks the loop, one lane issues
        const bool leader = elect_one();
        uint32_t g = 0, seg = 0, np[2] = {0, 0};  // ring tiles, segments, P tiles of each half
        const uint32_t ring = smem_addr(smem), qs = smem_addr(q_smem);
        bool ok = true;
        uint64_t *tiles = kQ8 ? conv : full;  // a tile of the ring is there
        auto qk = [&](int h, uint32_t st) {
            if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_f16(tmem + 128u * h,
                                tc::smem_desc_sw128(qs + h * C::kTileB + (k / 4) * C::kSlab) + uint64_t(2 * (k % 4)),
                                tc::smem_desc_sw128(ring + st * C::kTileB + (k / 4) * C::kSlab) + uint64_t(2 * (k % 4)),
                                tp.idesc_qk, k > 0);
                tc::commit_arrive(&s_full[h]);
            }
        };
        auto pv = [&](int h, uint32_t st, int chunk, bool acc) {  // 32 keys
            if (leader) {
                const uint64_t dv = desc_mn_sw128(ring + st * C::kTileB, C::kSlab);
#pragma unroll
                for (int k = 0; k < 2; ++k)  // 16 keys: 8 columns of P, 2048 bytes of V
                    mma_ts(tmem + 256u + 128u * h, tmem + 128u * h + 32u * chunk + 8u * k,
                           dv + uint64_t(128 * (2 * chunk + k)), tp.idesc_pv, acc || k > 0);
            }
        };
        while (ok && run.u < run.end) {
            int s0, s1;
            if (!run_segment(p, run, s0, s1)) break;
            const std::conditional_t<kQ8, const Item &, const Item> it = run.item;
            const int n = s1 - s0, halves = it.nt > tp.tth ? 2 : 1;
            uint32_t ks = g % C::kStages;
            if (!(ok = warp_wait(&q_full, seg & 1u, p, 55)) ||
                !(ok = warp_wait(&tiles[ks], (g / C::kStages) & 1u, p, 56)))
                break;
            tc::fence_after_sync();
            for (int h = 0; h < halves; ++h) qk(h, ks);
            if (leader) {
                tc::commit_arrive(&empty[ks]);
                if (n == 1) tc::commit_arrive(&q_empty);
            }
            for (int j = 0; ok && j < n; ++j) {
                const uint32_t vs = (g + 2 * j + 1) % C::kStages, vph = ((g + 2 * j + 1) / C::kStages) & 1u;
                if (!(ok = warp_wait(&tiles[vs], vph, p, 57))) break;
                const int key0 = tile_key<kKeys, kMasks>(it, s0 + j);
                if (!kQ8 && key0 + kKeys > it.len) {  // (any code is finite)
                    // rows at or past the sequence's end hold anything (or an earlier tile's
                    // values): their weights are 0, and so must they be
                    const int first = max(0, it.len - key0);
                    for (int i = first * 8 + lane; i < kKeys * 8; i += 32)
#pragma unroll
                        for (int c = 0; c < C::kCh; ++c)
                            *reinterpret_cast<uint4 *>(smem + vs * C::kTileB + c * C::kSlab + i * 16) =
                                make_uint4(0, 0, 0, 0);
                    __syncwarp();
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (j + 1 < n) {
                    ks = (g + 2 * j + 2) % C::kStages;
                    if (!(ok = warp_wait(&tiles[ks], ((g + 2 * j + 2) / C::kStages) & 1u, p, 58))) break;
                }
                for (int h = 0; ok && h < halves; ++h) {
                    if (!(ok = warp_wait(&p_ready[h][0], np[h] & 1u, p, 59))) break;
                    tc::fence_after_sync();
                    pv(h, vs, 0, j > 0);
                    pv(h, vs, 2, true);
                    __syncwarp();
                    if (!(ok = warp_wait(&p_ready[h][1], np[h] & 1u, p, 59))) break;
                    ++np[h];
                    tc::fence_after_sync();
                    pv(h, vs, 1, true);
                    pv(h, vs, 3, true);
                    if (j + 1 < n) qk(h, ks);
                    else if (leader) tc::commit_arrive(&o_full[h]);
                }
                if (leader) {
                    tc::commit_arrive(&empty[vs]);
                    if (j + 1 < n) tc::commit_arrive(&empty[ks]);
                    if (j + 2 == n) tc::commit_arrive(&q_empty);
                }
                __syncwarp();
            }
            g += 2 * n;
            ++seg;
            next();
        }
        // every MMA complete before the tensor memory is released
        if (leader) tc::commit_arrive(&drain);
        __syncwarp();
        warp_wait(&drain, 0, p, 60, kDrainNs);
    } else if (warp < kSoftmaxWarps) {
        // ---- softmax: half h, rows 32 q4 + lane, keys 64 ch .. of each tile (and of the
        // result the channels D/2 ch ..)
        const int q4 = warp & 3, h = (warp >> 2) & 1, ch = warp >> 3, row = 32 * q4 + lane;
        const uint32_t lanes = uint32_t(32 * q4) << 16;
        const uint32_t ts = tmem + 128u * h + 64u * ch + lanes, to = tmem + 256u + 128u * h + uint32_t(D / 2) * ch + lanes;
        const int tok_h = row / G, head = row % G;
        const bool capped = kMode == kCapped || (kMode == kAny && p.cap_in != 0.f);
        const float sign = kMode == kAny && (capped ? p.cap_in : p.scale_log2) < 0.f ? -1.f : 1.f;
        // The q.k of a key that a row does not see, and the least (by sign) of one that it does: what
        // is less, an infinity too, has the same capped score, and is not taken for hidden
        const float hidden = -CUDART_INF_F * sign;
        constexpr bool kInCap = kQ8 && kMode == kCapped;  // the scores come over the cap: a factor of K's scales
        const float cap_in = kInCap ? 1.f : p.cap_in;
        const float lowest = kMode == kCapped ? kTanhMinusOne / cap_in : -CUDART_MAX_NORMAL_F;
        uint32_t ns = 0, no = 0, nx = 0;  // S tiles and O results taken, exchanges
        uint32_t gt = 0;                  // tiles of all segments (kQ8)
        bool ok = true;  // after a time-out: no more waits, but every barrier still met
        // a value of the row's other thread, through the space of the results on their way out
        uint8_t *stage = smem + C::kOutAt + warp * C::kStageOut;
        float *mine_x = reinterpret_cast<float *>(stage) + lane;  // in turns at 0 and 32
        const float *other_x = reinterpret_cast<float *>(stage + ((warp ^ 8) - warp) * C::kStageOut) + lane;
        auto meet = [&]() { named_bar_sync(1 + (warp & 7), 64); };
        auto exchange = [&](float mine) {
            const uint32_t o = (nx++ & 1) * 32;
            mine_x[o] = mine;
            meet();
            return other_x[o];
        };
        while (run.u < run.end) {
            int s0, s1;
            if (!run_segment(p, run, s0, s1)) break;
            const std::conditional_t<kQ8, const Item &, const Item> it = run.item;
            const int nth = min(tp.tth, it.nt - h * tp.tth);  // this half's tokens
            if (nth > 0) {
                const int first = it.pos0 + h * tp.tth;  // position of the half's first token
                const bool live = tok_h < nth;
                const int at = live ? first + tok_h : -1;
                Sight sight;
                if (kMasks)
                    sight = row_sight(p, run.seq, live, it.row0 + h * tp.tth + tok_h,
                                      it.qt * p.tt + h * tp.tth + tok_h);
                __syncwarp();
                // what every row of the half sees, and the last token's key or one after it
                const bool tree = kMasks && p.tree != nullptr;
                const int all = tree ? run.seq.len - run.seq.n - 1 : first, late = tree ? it.len - 1 : first + nth - 1;
                float top = -CUDART_INF_F, sum = 0.f;  // reference maximum (log2), sum of weights
                // kRef: the row's e; the scales that the tiles so far had, as in the streaming kernel
                float re = 0.f;
                uint32_t range = 0x80000000u;
                for (int j = 0; j < s1 - s0; ++j) {
                    ok = ok && warp_wait(&s_full[h], ns & 1u, p, 61 + h);
                    ++ns;
                    // S is there, so the tiles before this one's V are spread: of the barrier of its stage only
                    // that phase is to come
                    const uint32_t vg = 2 * (gt + j) + 1, vst = vg % C::kStages;
                    if (kQ8) ok = ok && warp_wait(&conv[vst], (vg / C::kStages) & 1u, p, 65 + h);
                    const float *ks = reinterpret_cast<const float *>(smem + C::kScalesAt) +
                                      ((gt + j) % C::kScaleTiles) * (2 * kKeys) + 64 * ch;
                    const float *vs = ks + kKeys;
                    tc::fence_after_sync();
                    const int key0 = tile_key<kKeys, kMasks>(it, s0 + j);
                    const bool edge = key0 + kKeys - 1 > all ||
                                      (p.window > 0 && key0 <= late - p.window && (!kMasks || key0 + kKeys > p.sinks));
                    // a tile that some row does not see whole: what it does not see becomes the
                    // score of weight 0, in place, so that the passes below (whose code is long)
                    // exist once and pay for no comparisons
                    if (edge) {
                        const int hi = at - key0 - 64 * ch, lo = p.window > 0 ? hi - p.window : -1;  // sees lo < i <= hi
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t sees = 0u;
                            if (kMasks) {
                                sees = sight32(p, run.seq, sight, key0 + 64 * ch + 32 * c);
                                __syncwarp();
                            }
                            float u[32];
                            tmem_ld32(ts + 32 * c, u);
                            wait_ld32(u);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (kMode == kCapped && !kQ8) u[i] = max_nan(u[i], lowest);
                                if (kMode == kAny && !kQ8 && capped && u[i] == hidden) u[i] = lowest * sign;
                                if (kMasks ? (sees >> i & 1u) == 0u : 32 * c + i > hi || 32 * c + i <= lo) u[i] = hidden;
                            }
                            tmem_st32(ts + 32 * c, u);
                        }
                        wait_st();
                    }
                    // first pass: the row's maximum (the score grows with sign * q.k, so the maximum
                    // of those gives the maximum of the scores)
                    float v[2][16];
                    float mt, most = 0.f;  // the largest, and the largest magnitude of this thread's keys
                    {
                        float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                        float a4[4] = {0.f, 0.f, 0.f, 0.f};
                        auto larger = [&](const float (&u)[32]) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2)
                                m4[(i >> 1) & 3] = kMode == kAny ? max3(m4[(i >> 1) & 3], u[i] * sign, u[i + 1] * sign)
                                                                 : max3(m4[(i >> 1) & 3], u[i], u[i + 1]);
                            if (kMode == kAny && capped)
#pragma unroll
                                for (int i = 0; i < 32; i += 2)
                                    a4[(i >> 1) & 3] = max3(a4[(i >> 1) & 3], fabsf(u[i]), fabsf(u[i + 1]));
                        };
                        if (kQ8) {  // (both at once leave no registers for the scales)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float u[32];
                                tmem_ld32(ts + 32 * c, u);
                                wait_ld32(u);
#pragma unroll
                                for (int i = 0; i < 32; i += 4) scaled(u + i, ks + 32 * c + i, u + i);
                                larger(u);
                            }
                        } else {
                            float u[2][32];
                            tmem_ld32(ts, u[0]);
                            tmem_ld32(ts + 32, u[1]);
                            wait_ld32(u[0]);
                            wait_ld32(u[1]);
                            larger(u[0]);
                            larger(u[1]);
                        }
                        mt = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
                        if (kMode == kAny && capped) most = max3(fmaxf(a4[0], a4[1]), a4[2], a4[3]);
                    }
                    tmem_ld16(ts, v[0]);  // for the second pass
                    if (kRef) {
                        // Where a wait has run out for one of the two warps, both know from here on: what follows meets
                        // only where the scales say so, and only while both have seen the same ones.
                        const float other = exchange(ok ? mt : CUDART_NAN_F);
                        ok = ok && other == other;
                        mt = fmaxf(mt, other);
                    } else {
                        mt = fmaxf(mt, exchange(mt));
                    }
                    if (capped && !edge) mt = fmaxf(mt, lowest);
                    // a row of no token holds what was in shared memory, or another sequence's query:
                    // it has no say in the warp's choices below, which show in the live rows' roundings
                    if (!live) mt = -CUDART_INF_F, most = 0.f;
                    // kCapped: a tile that every row sees whole and whose tangents stay off 1; kAny: one
                    // whose scores all are far below the cap (a hidden score's magnitude is infinite)
                    const bool plain =
                        kMode == kCapped ? !edge && !__any_sync(0xffffffffu, mt * cap_in > kTanhOne)
                        : kMode == kAny && capped ? __all_sync(0xffffffffu, most * fabsf(p.cap_y) < kTanhNear)
                                                  : false;
                    if (mt != -CUDART_INF_F)
                        mt = kMode == kCapped            ? capped_far(mt, cap_in, p)
                             : capped                    ? score<true>(mt * sign, p)
                             : kQ8 && kMode == kScaled   ? mt
                                                         : score<false>(mt * sign, p);
                    float product = -CUDART_INF_F;  // the row's largest of the tile (log2)
                    if (kRef) {
                        // the tile's scales, four a lane (-0.0 is the least as a signed number, and above all others as
                        // an unsigned one)
                        const uint4 x = *reinterpret_cast<const uint4 *>(vs - 64 * ch + 4 * lane);
                        const int hi = max(max(int(x.x), int(x.y)), max(int(x.z), int(x.w)));
                        const uint32_t lo = min(min(x.x, x.y), min(x.z, x.w));
                        bool apart = false;
                        if (!__all_sync(0xffffffffu, lo >= range && hi <= int(range + kSpread))) {
                            const uint32_t hi_all = max(__reduce_max_sync(0xffffffffu, hi), 0);
                            const uint32_t lo_all = min(__reduce_min_sync(0xffffffffu, lo), hi_all);
                            apart = hi_all - lo_all > kSpread;
                            if (!apart) range = lo_all - min(lo_all, (kSpread - (hi_all - lo_all)) / 2);
                        }
                        if (apart && ok) {
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                float u[16];
                                tmem_ld16(ts + 16 * c, u);
                                wait_ld16(u);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float x = u[i] * ks[16 * c + i];
                                    const float z = kMode == kCapped            ? capped_far(fmaxf(x, lowest), cap_in, p)
                                                    : capped                    ? score<true>(x, p)
                                                    : kMode == kScaled          ? x
                                                                                : score<false>(x, p);
                                    if (x != hidden) product = fmaxf(product, z + scale_log2(scale_bits(vs[16 * c + i])));
                                }
                            }
                            product = fmaxf(product, exchange(product));
                        } else {
                            product = mt + scale_log2(range + kSpread);
                        }
                        if (!live) product = -CUDART_INF_F;
                    }
                    if (j == 0) {
                        top = mt;
                        if (kRef) re = ref_exponent(product, top == -CUDART_INF_F ? 0.f : top);
                    } else if (__any_sync(0xffffffffu, mt - top > kGrowth || (kRef && product - top - re > kGrowth))) {
                        // this half's P V of the tile before is complete: its S came after it
                        const float up = fmaxf(top, mt), base = up == -CUDART_INF_F ? 0.f : up;
                        float f = exp2_approx(top - base);
                        sum *= f;
                        if (kRef) {
                            const float e = ref_exponent(fmaxf(top + re, product), base);
                            f = exp2_approx((top - base) + (re - e));
                            re = e;
                        }
                        top = up;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[16];
                            tmem_ld16(to + 16 * c, o);
                            wait_ld16(o);
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * f);
                            tmem_st16(to + 16 * c, w);
                        }
                    }
                    // second pass: the weights
                    const float base = top == -CUDART_INF_F ? 0.f : top;
                    unsigned long long s2[2] = {0ull, 0ull};  // pairs of sums
                    const float scale = kMode == kCapped ? p.cap_in : p.scale_log2;
                    const float b = kMode == kCapped ? p.cap_log2 - base : -base, k2 = -2.f * p.cap_log2;
                    const unsigned long long scale2 = pack2(scale, scale), base2 = pack2(b, b);
                    const unsigned long long one2 = pack2(1.f, 1.f), near2 = pack2(p.cap_y, p.cap_y);
                    const float from = edge ? -CUDART_INF_F : kTanhMinusOne;
                    const float rf = kRef ? power_of_2(kLift - re) : 1.f;
                    const unsigned long long hide2 = pack2(0x1p-100f, 0x1p-100f);
                    auto take = [&](auto is_plain, int c, const float (&raw)[16]) {
                        constexpr bool kPlain = decltype(is_plain)::value;
                        uint32_t w[8];
                        constexpr bool kFused = kQ8 && kMode == kScaled;  // the scale is a factor of K's scales
                        float u[16];
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            float4 ksc = make_float4(1.f, 1.f, 1.f, 1.f);
                            if (kFused) ksc = *reinterpret_cast<const float4 *>(ks + 16 * c + i);
                            if (kQ8 && !kFused) {
                                scaled(raw + i, ks + 16 * c + i, u + i);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k) u[i + k] = raw[i + k];
                            }
                            unsigned long long e2[2] = {pack2(u[i], u[i + 1]), pack2(u[i + 2], u[i + 3])};
                            if (kMode == kAny && kPlain) {  // score()'s polynomial, less the base
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const unsigned long long y = mul2(e2[k], near2), t = mul2(y, y);
                                    unsigned long long r = fma2(t, pack2(kTanh5, kTanh5), pack2(kTanh4, kTanh4));
                                    r = fma2(t, r, pack2(kTanh3, kTanh3));
                                    r = fma2(t, r, pack2(kTanh2, kTanh2));
                                    r = fma2(t, r, pack2(kTanh1, kTanh1));
                                    r = fma2(t, r, one2);
                                    e2[k] = fma2(mul2(e2[k], scale2), r, base2);
                                }
                            } else if (kMode == kAny && capped) {
                                float z[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) z[k] = score<true>(u[i + k], p) - base;
                                e2[0] = pack2(z[0], z[1]);
                                e2[1] = pack2(z[2], z[3]);
                            } else if (kMode == kCapped) {
                                // the score less the base: d = 1 + e^2x, and the four reciprocals from that
                                // of their product (a reciprocal takes twice an exponential's time; d is
                                // kept below 2^30 for it, where the tangent is 1 in fp32: by the tile's
                                // maxima where it is plain)
                                unsigned long long d2[2], x2[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    float x, y;
                                    unpack2(kInCap ? e2[k] : mul2(e2[k], scale2), x, y);
                                    if (!kPlain) {
                                        x = min_nan(max_nan(x, from), kTanhOne);
                                        y = min_nan(max_nan(y, from), kTanhOne);
                                        x2[k] = pack2(x, y);
                                    }
                                    d2[k] = add2(pack2(exp2_approx(x), exp2_approx(y)), one2);
                                }
                                float x, y;
                                unpack2(mul2(d2[0], d2[1]), x, y);
                                const float r = rcp_approx(x * y) * k2;
                                const unsigned long long r2 = mul2(pack2(r, r), pack2(y, x));
                                // a hidden score (an infinity, the only one left) is brought back by a
                                // product that is nothing beside any other score
                                e2[0] = fma2(r2, d2[1], kPlain ? base2 : fma2(x2[0], hide2, base2));
                                e2[1] = fma2(r2, d2[0], kPlain ? base2 : fma2(x2[1], hide2, base2));
                            } else {
                                e2[0] = fma2(e2[0], kFused ? pack2(ksc.x, ksc.y) : scale2, base2);
                                e2[1] = fma2(e2[1], kFused ? pack2(ksc.z, ksc.w) : scale2, base2);
                            }
                            // codes: the values' scales join the weights
                            float4 vsc = make_float4(1.f, 1.f, 1.f, 1.f);
                            if (kQ8) vsc = *reinterpret_cast<const float4 *>(vs + 16 * c + i);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float x, y;
                                unpack2(e2[k], x, y);
                                x = exp2_approx(x);
                                y = exp2_approx(y);
                                if (kMode == kAny && !kPlain && edge) {  // times 0 an infinity does not give weight 0 by itself
                                    if (u[i + 2 * k] == hidden) x = 0.f;
                                    if (u[i + 2 * k + 1] == hidden) y = 0.f;
                                }
                                s2[k] = add2(s2[k], pack2(x, y));
                                // rounded for the product, whose operands have one type (V's values were
                                // rounded to it by the same half step); the sum keeps the weight whole
                                if (kQ8) {
                                    unsigned long long w2 = pack2(x, y);
                                    if (kRef) w2 = mul2(w2, pack2(rf, rf));
                                    unpack2(mul2(w2, k == 0 ? pack2(vsc.x, vsc.y) : pack2(vsc.z, vsc.w)), x, y);
                                }
                                w[i / 2 + k] = Pair<T>::make(x, y);
                            }
                        }
                        // over the chunk's own scores: 32 keys' weights side by side
                        tmem_st8(ts + 32 * (c >> 1) + 8 * (c & 1), w);
                    };
                    auto ready = [&](uint64_t *bar) {
                        wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0 && ok) mbar_arrive(bar);
                        __syncwarp();
                    };
                    auto weights = [&](auto is_plain) {
                        wait_ld16(v[0]);
                        tmem_ld16(ts + 16, v[1]);
                        take(is_plain, 0, v[0]);
                        wait_ld16(v[1]);
                        tmem_ld16(ts + 32, v[0]);
                        take(is_plain, 1, v[1]);
                        ready(&p_ready[h][0]);  // the product of this thread's first 32 keys can begin
                        wait_ld16(v[0]);
                        tmem_ld16(ts + 48, v[1]);
                        take(is_plain, 2, v[0]);
                        wait_ld16(v[1]);
                        take(is_plain, 3, v[1]);
                        ready(&p_ready[h][1]);
                    };
                    if (plain) weights(std::true_type());
                    else weights(std::false_type());
                    float sa, sb;
                    unpack2(add2(s2[0], s2[1]), sa, sb);
                    sum += sa + sb;
                }
                if (kQ8 && *static_cast<volatile int *>(&odd) != 0 && sees_odd(p, run.seq, it, sight, s0, s1, 64 * ch))
                    sum = CUDART_NAN_F;
                __syncwarp();
                // ---- the half's result: this warp's channels
                sum += exchange(sum);
                meet();  // both have read: the space is free for the results
                ok = ok && warp_wait(&o_full[h], no & 1u, p, 63 + h);
                ++no;
                tc::fence_after_sync();
                const bool whole = s0 == 0 && s1 == it.tiles;
                const int out_row = live ? (it.row0 + h * tp.tth + tok_h) * p.b.Hq + it.kh * G + head : -1;
                float *mine = p.part + size_t(part_slot(blockIdx.x, s0 == 0)) * part_floats(2 * kHalf, D);
                const int prow = h * kHalf + row;
                const float unit = kRef ? power_of_2(re - kLift) : 1.f, inv = over_sum(sum) * unit;
#pragma unroll 1
                for (int c = 0; ok && c < D / 64; ++c) {
                    const int ch0 = D / 2 * ch + 32 * c;  // first of 32 channels
                    float o[32];
                    tmem_ld32(to + 32 * c, o);
                    wait_ld32(o);
                    if (whole && kQ8) {
                        if (live) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + size_t(out_row) * D + ch0);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float *x = &o[8 * k];
                                dst[k] = make_uint4(Pair<T>::make(x[0] * inv, x[1] * inv), Pair<T>::make(x[2] * inv, x[3] * inv),
                                                    Pair<T>::make(x[4] * inv, x[5] * inv), Pair<T>::make(x[6] * inv, x[7] * inv));
                            }
                        }
                    } else if (whole) {
                        // through shared memory: a row per lane in (16-byte chunks, swizzled),
                        // 64-byte runs of eight rows at a time out
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float *x = &o[8 * k];
                            *reinterpret_cast<uint4 *>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
                                make_uint4(Pair<T>::make(x[0] * inv, x[1] * inv), Pair<T>::make(x[2] * inv, x[3] * inv),
                                           Pair<T>::make(x[4] * inv, x[5] * inv), Pair<T>::make(x[6] * inv, x[7] * inv));
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + (lane >> 2), k = lane & 3;
                            const int dst = __shfl_sync(0xffffffffu, out_row, r);
                            const uint4 w = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((k ^ ((r >> 1) & 3)) << 4));
                            if (dst >= 0)
                                *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + size_t(dst) * D + ch0 + 8 * k) = w;
                        }
                    } else if (live) {
                        if (kRef)
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= unit;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            tc::st_global_v8(mine + part_at(prow, ch0 + i, D),
                                             {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6],
                                              o[i + 7]});
                    }
                    __syncwarp();  // the next load of tensor memory wants the warp together
                }
                if (ok && live && ch == 0) {
                    if (!whole) {
                        mine[size_t(2 * kHalf) * D + prow] = top;
                        mine[size_t(2 * kHalf) * (D + 1) + prow] = sum;
                    } else if (p.lse != nullptr) {
                        p.lse[out_row] = log_sum(top, sum);
                    }
                }
                __syncwarp();
                tc::fence_before_sync();
            }
            gt += s1 - s0;
            next();
            // Each warp reads the lengths for itself.  Should they change under the call (a missing stream order), the
            // two of a row could count their tiles differently, and a barrier has no limit: they go on only together.
            const unsigned turn = unsigned(run.item.tiles) * 512u + unsigned(run.item.nt) +
                                  (p.withhold == kCountApart && blockIdx.x == 0 ? ch : 0);
            if (run.u < run.end && __float_as_uint(exchange(__uint_as_float(turn))) != turn) {
                record_status(p.hdr, MOE_ERR_CACHE_RANGE, run.seq.len);
                break;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int kForm, typename T, int D>
cudaError_t launch(const TcParams &tp, bool near_cap, int grid, cudaStream_t s) {
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(grid), dim3(form_threads(kForm)), size_t(Cfg<D, kForm>::kSmem), s, tp);
    };
    if (tp.p.cap_in > 0.f && near_cap) return go(attention_tc_kernel<T, D, kCapped, kForm>);
    if (tp.p.cap_in == 0.f && tp.p.scale_log2 > 0.f) return go(attention_tc_kernel<T, D, kScaled, kForm>);
    return go(attention_tc_kernel<T, D, kAny, kForm>);
}

template <int kForm, typename T, int D>
cudaError_t init() {
    auto set = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, kForm>::kSmem);
    };
    cudaError_t e = set(attention_tc_kernel<T, D, kScaled, kForm>);
    if (e == cudaSuccess) e = set(attention_tc_kernel<T, D, kAny, kForm>);
    if (e == cudaSuccess) e = set(attention_tc_kernel<T, D, kCapped, kForm>);
    return e;
}

// Every kernel of a form, until one fails.
template <int kForm>
cudaError_t init_form() {
    cudaError_t e = init<kForm, __half, 64>();
    if (e == cudaSuccess) e = init<kForm, __half, 128>();
    if (e == cudaSuccess) e = init<kForm, __nv_bfloat16, 64>();
    if (e == cudaSuccess) e = init<kForm, __nv_bfloat16, 128>();
    return e;
}

template <int kForm>
cudaError_t launch_form(const AttnArgs &a, const Params &p, int num_sms, cudaStream_t s) {
    const int G = a.b.Hq / a.b.Hkv;
    TcParams tp = {};
    tp.p = p;
    tp.tth = kHalf / G;
    tp.p.tt = 2 * tp.tth;
    tp.p.tt_magic = 0xffffffffu / unsigned(tp.p.tt) + 1;
    tp.p.extra = kExtra;
    tp.box_rows = std::min(a.b.page, kKeys);
    const uint32_t fmt = a.type == MOE_BF16 ? (1u << 7) | (1u << 10) : 0u;  // A and B bf16
    tp.idesc_qk = tc::idesc_f16_f32(kHalf, kKeys) | fmt;
    tp.idesc_pv = tc::idesc_f16_f32(kHalf, a.b.D) | fmt | (1u << 16);       // B: N contiguous
    auto pages = [&](CUtensorMap *map, const void *base) {
        return kForm == kCodes ? encode_codes_map(map, base, a.b, tp.box_rows, a.b.D == 64)
                               : encode_pages_map(map, base, a.b, a.type, tp.box_rows);
    };
    if (!pages(&tp.mk, a.k) || !pages(&tp.mv, a.v) || !encode_rows_map(&tp.mq, a.q, a.b, a.type, tp.tth))
        return cudaErrorInvalidValue;
    if (kForm == kCodes &&
        (!encode_scales_map(&tp.mks, a.ks, a.b, tp.box_rows) || !encode_scales_map(&tp.mvs, a.vs, a.b, tp.box_rows)))
        return cudaErrorInvalidValue;
    const int grid = std::min(num_sms, kMaxGrid);
    const bool near_cap = a.softcap <= kCapNear && p.cap_in > 1e-30f;  // kCapped: kTanhMinusOne / cap_in is finite
    auto of = [&](auto type) {
        using T = decltype(type);
        return a.b.D == 64 ? launch<kForm, T, 64>(tp, near_cap, grid, s) : launch<kForm, T, 128>(tp, near_cap, grid, s);
    };
    const cudaError_t e = a.type == MOE_F16 ? of(__half()) : of(__nv_bfloat16());
    if (e != cudaSuccess) return e;
    // nothing is parted where even the most and longest items that the arguments allow are taken
    // whole (a prompt of 100 in a table of its length: 9.5 us, with the joining launch 12.0)
    const long items = long(a.b.B) * a.b.Hkv * ((a.b.N + tp.p.tt - 1) / tp.p.tt);
    const long tiles = (long(a.b.max_pages) * a.b.page + kKeys - 1) / kKeys;
    if (items <= grid && tiles + kExtra <= kSplit) return cudaSuccess;
    return launch_join(tp.p, a.type, grid, 2 * kHalf, kHalf, tp.tth, s);
}

}  // namespace tc5
}  // namespace attn
}  // namespace moeq4k
