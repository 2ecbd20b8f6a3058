// What the attention kernels share: the split of the work over the CTAs and
// the joining of split key ranges.
//
// An item is a tile of query rows of one sequence and one key/value head: tt
// tokens times the G query heads that read the head.  Its work is the run of
// key tiles (KT keys) that any of its rows sees, at least one, and a fixed cost
// of `extra` tiles (queries in, results out).  All items' work, laid end to end,
// is cut into equal runs, one per CTA, whatever the sequences' lengths: a CTA's
// run is a few segments, each a range of key tiles of one item.  An item
// inside one run is finished there; one that crosses a cut leaves a partial
// result (unnormalised sums, running maximum and sum) per segment, and a
// second launch joins them in key order over the whole GPU.  So the order of
// every sum depends on the shapes alone and results repeat bit for bit.
#pragma once

#include <math_constants.h>

#include "async_copy.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace moeq4k {
namespace attn {

constexpr int kMaxCtas = 304;  // 2 per SM

// An item that starts in a CTA's run and does not end there (parts > 1), or
// none (parts = 0).  One per CTA, written by every call.
struct JoinDesc {
    int parts, row0, nt, kh;
};
constexpr size_t kDescBytes = (kMaxCtas * sizeof(JoinDesc) + 255) / 256 * 256;

struct Params {
    PagedBatch b;
    const void *q;
    void *out;
    float *lse;
    float scale_log2;   // scale * log2(e), or without softcap's scale: see score()
    float cap_in;       // softcap: 2 log2(e) scale / cap; 0: none
    float cap_log2;     // softcap * log2(e)
    int window;
    int tt;             // tokens of a query tile
    int extra;          // fixed cost of an item, in key tiles
    WsHeader *hdr;
    JoinDesc *desc;     // [kMaxCtas]
    float *part;
    unsigned long long wait_ns;
};

// Bring a tensor map (a kernel parameter) into the cache of such descriptors.
__device__ __forceinline__ void prefetch_map(const void *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The score in units of log2: scale q.k log2(e), or cap tanh(scale q.k / cap)
// log2(e) with tanh(x) = 1 - 2 / (1 + e^2x).  Its error is about 2^-22 of the
// cap, whatever the score: the absolute error is what the softmax feels.
template <bool kCap>
__device__ __forceinline__ float score(float s, const Params &p) {
    if (!kCap) return s * p.scale_log2;
    return fmaf(__fdividef(-2.f, 1.f + exp2_approx(s * p.cap_in)), p.cap_log2, p.cap_log2);
}

struct Item {
    int b, qt, kh;
    int row0;    // first row (token) of the tile
    int nt;      // tokens in it
    int pos0;    // cache index of the first
    int len;     // cached tokens
    int t0;      // first key tile
    int tiles;   // key tiles, at least 1 (a tile whose rows see nothing has one, all masked)
};

template <int KT>
__device__ __forceinline__ void item_tiles(int window, int tt, const SeqView &s, int qt, int &nt,
                                           int &pos0, int &t0, int &tiles) {
    nt = min(tt, s.n - qt * tt);
    pos0 = s.len - s.n + qt * tt;
    const int last = pos0 + nt - 1;
    const int kb = window > 0 && pos0 >= window ? pos0 - window + 1 : 0;
    t0 = kb / KT;
    tiles = last >= kb ? last / KT + 1 - t0 : 1;
}

// The CTA's run: positions [u, end) of the whole work; u is inside `item`,
// which starts at item_u with `extra` positions before its first tile.
struct Run {
    long per;  // positions of a run
    long u, end, item_u;
    SeqView seq;  // item's sequence
    Item item;
};

// The work of a sequence: its query tiles' key tiles and fixed costs, of one
// key/value head.
template <int KT>
__device__ __forceinline__ long tile_cost(const Params &p, const SeqView &s, int qt) {
    int nt, pos0, t0, tiles;
    item_tiles<KT>(p.window, p.tt, s, qt, nt, pos0, t0, tiles);
    return tiles + p.extra;
}

// a / b for a >= 0, b > 0: as 32 bits where they fit (64-bit division is long).
__device__ __forceinline__ long div_pos(long a, long b) {
    if (((a | b) >> 31) == 0) return long(unsigned(a) / unsigned(b));
    return a / b;
}

// Every thread of the CTA calls it; `scratch`: B longs of shared memory (free
// again at the next barrier).  A run is at least `least` long.  False: nothing
// to do.  A thread per sequence where its tiles are few (decode), a warp where
// they are many, then each warp sums and searches by itself: at 64 sequences this
// takes 2 us of the kernel's start where a warp per sequence took 10.
template <int KT>
__device__ inline bool run_begin(const Params &p, int least, long *scratch, Run &r) {
    constexpr int kFew = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int B = p.b.B, Hkv = p.b.Hkv;
    for (int base = warp * 32; base < B; base += nw * 32) {
        const int b = base + lane;
        int nq = 0;
        long total = 0;
        if (b < B) {
            const SeqView s = seq_view(p.b, b, p.hdr, blockIdx.x == 0);
            nq = (s.n + p.tt - 1) / p.tt;
            if (nq <= kFew) {
                for (int qt = 0; qt < nq; ++qt) total += tile_cost<KT>(p, s, qt);
                scratch[b] = total * Hkv;
            }
        }
        for (unsigned many = __ballot_sync(0xffffffffu, nq > kFew); many != 0; many &= many - 1) {
            const int src = __ffs(many) - 1, nqs = __shfl_sync(0xffffffffu, nq, src);
            const SeqView s = seq_view(p.b, base + src, p.hdr, false);
            total = 0;
            for (int qt = lane; qt < nqs; qt += 32) total += tile_cost<KT>(p, s, qt);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (lane == 0) scratch[base + src] = total * Hkv;
        }
    }
    __syncthreads();
    long U = 0;
    for (int b = lane; b < B; b += 32) U += scratch[b];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) U += __shfl_xor_sync(0xffffffffu, U, o);
    r.per = max(long(least), div_pos(U + gridDim.x - 1, gridDim.x));
    r.u = r.per * blockIdx.x;
    r.end = min(U, r.u + r.per);
    if (r.u >= r.end) return false;
    // the first position past which a prefix sum over steps of 32 goes
    auto locate = [&](int n, long at, auto cost, int &which, long &start) {
        for (int base = 0; base < n; base += 32) {
            long v = base + lane < n ? cost(base + lane) : 0;
            const long mine = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long w = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += w;
            }
            const unsigned past = __ballot_sync(0xffffffffu, at + v > r.u);
            if (past != 0u) {
                const int src = __ffs(past) - 1;
                which = base + src;
                start = at + __shfl_sync(0xffffffffu, v - mine, src);
                return;
            }
            at += __shfl_sync(0xffffffffu, v, 31);
        }
    };
    Item &it = r.item;
    it.b = 0;
    it.qt = 0;
    long at = 0, first = 0;
    locate(B, 0, [&](int b) { return scratch[b]; }, it.b, at);
    r.seq = seq_view(p.b, it.b, p.hdr, false);
    const int nq = (r.seq.n + p.tt - 1) / p.tt;
    if (nq > 1)
        locate(nq, at, [&](int qt) { return tile_cost<KT>(p, r.seq, qt) * Hkv; }, it.qt, first);
    else
        first = at;
    it.len = r.seq.len;
    it.row0 = r.seq.first + it.qt * p.tt;
    item_tiles<KT>(p.window, p.tt, r.seq, it.qt, it.nt, it.pos0, it.t0, it.tiles);
    const long each = it.tiles + p.extra;
    it.kh = int(div_pos(r.u - first, each));
    r.item_u = first + it.kh * each;
    return true;
}

// The CTA's segment of r.item: tiles [s0, s1); false when the run ends before them.
__device__ __forceinline__ bool run_segment(const Params &p, const Run &r, int &s0, int &s1) {
    const long first = r.item_u + p.extra;
    s0 = int(max(0l, r.u - first));
    s1 = int(min(long(r.item.tiles), r.end - first));
    return s1 > s0;
}

// On to the item after r.item, if the run reaches it.
template <int KT>
__device__ inline void run_next(const Params &p, Run &r) {
    Item &it = r.item;
    r.u = r.item_u = r.item_u + p.extra + it.tiles;
    if (r.u >= r.end || ++it.kh < p.b.Hkv) return;
    it.kh = 0;
    ++it.qt;
    while (it.qt * p.tt >= r.seq.n && it.b + 1 < p.b.B) {
        ++it.b;
        it.qt = 0;
        r.seq = seq_view(p.b, it.b, p.hdr, false);
    }
    it.len = r.seq.len;
    it.row0 = r.seq.first + it.qt * p.tt;
    item_tiles<KT>(p.window, p.tt, r.seq, it.qt, it.nt, it.pos0, it.t0, it.tiles);
}

// A partial result: `rows` (a multiple of 32) rows of D sums, then their maxima,
// then their sums of weights.  The sums of 32 rows x 8 channels are
// together, so that a warp with a row per lane stores 1 KB runs.
__host__ __device__ constexpr size_t part_floats(int rows, int D) { return size_t(rows) * (D + 2); }
__device__ __forceinline__ int part_at(int row, int ch, int D) {
    return ((row >> 5) * (D / 8) + (ch >> 3)) * 256 + (row & 31) * 8 + (ch & 7);
}

// Its slot: a CTA has at most one segment that goes on from the CTA before
// (its first) and one that it leaves to the next (its last).
__device__ __forceinline__ int part_slot(int cta, bool starts_here) { return 2 * cta + (starts_here ? 1 : 0); }

// The parts of r.item: consecutive CTAs from the one with its first tile on.
__device__ __forceinline__ JoinDesc join_desc(const Params &p, const Run &r) {
    const long first = r.item_u + p.extra;
    JoinDesc d;
    d.parts = int(div_pos(first + r.item.tiles - 1, r.per) - div_pos(first, r.per)) + 1;
    d.row0 = r.item.row0;
    d.nt = r.item.nt;
    d.kh = r.item.kh;
    return d;
}

// Joins the partial results of items of up to `rows` rows; query row r of an item
// is token r / half * tth + r % half / G, head r % half % G.
cudaError_t launch_join(const Params &p, moe_dtype type, int grid, int rows, int half, int tth, cudaStream_t s);

// The tensor-core kernel (many rows per key/value head).
size_t tc_part_bytes(int D);
cudaError_t init_tc();
cudaError_t launch_tc(const AttnArgs &a, const Params &p, int num_sms, cudaStream_t s);

}  // namespace attn
}  // namespace moeq4k
