// What the attention kernels share: the split of the work over the CTAs and
// the joining of split key ranges.
//
// An item is a tile of query rows of one sequence and one key/value head: tt
// tokens times the G query heads that read the head.  Its work is the run of
// key tiles (KT keys) that any of its rows sees, at least one, and a fixed cost
// of `extra` tiles (queries in, results out).  All items' work, laid end to end,
// is cut into equal runs, one per CTA, whatever the sequences' lengths (but a CTA
// takes an item whole where that is as fast): a CTA's
// run is a few segments, each a range of key tiles of one item.  An item
// inside one run is finished there; one that crosses a cut leaves a partial
// result (unnormalised sums, running maximum and sum) per segment.  These are
// joined in a fixed order, by the CTA that arrives last (few rows in few parts) or by
// a second launch over the whole GPU (many parts, many rows), so that the order of
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
// Arrivals at each CTA's item, ahead of the descriptors: zero before the first
// call (moe_workspace_init) and after every call.
constexpr size_t kCountBytes = 2048;
static_assert(kMaxCtas * sizeof(unsigned) <= kCountBytes && kCountBytes <= sizeof(unsigned long long) * kSyncWords,
              "one per CTA, zeroed by moe_workspace_init");

struct Params {
    PagedBatch b;
    const void *q;
    void *out;
    float *lse;
    float scale_log2;   // scale * log2(e), or without softcap's scale: see score()
    float cap_in;       // softcap: 2 log2(e) scale / cap; 0: none
    float cap_y;        // scale / cap
    float cap_log2;     // softcap * log2(e)
    int window;
    int tt;             // tokens of a query tile
    unsigned tt_magic;  // ceil(2^32 / tt), tt > 1: n / tt as a high product (n < 2^23)
    int extra;          // fixed cost of an item, in key tiles
    WsHeader *hdr;
    unsigned *count;    // [kMaxCtas]
    JoinDesc *desc;     // [kMaxCtas]
    float *part;
    unsigned long long wait_ns;
    int withhold;       // test hook: CTA 0's waits run out
};

// The arrivals that CTA 0's barriers expect and never get (moe_debug_withhold_arrivals).
__device__ __forceinline__ int withheld(const Params &p) { return p.withhold != 0 && blockIdx.x == 0 ? 1 : 0; }

// Bring a tensor map (a kernel parameter) into the cache of such descriptors.
__device__ __forceinline__ void prefetch_map(const void *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The score in units of log2: scale q.k log2(e), or cap tanh(y) log2(e) with
// y = scale q.k / cap.  tanh(y) = 1 - 2 / (1 + e^2y) has an error of about 2^-22
// of the cap, whatever the score, so below kTanhNear the score is z (tanh(y) / y)
// with a polynomial in y^2 (interpolated at Chebyshev's nodes, 4e-9 off): the
// error is some 2^-21 of the score, however far the cap is.
constexpr float kTanhNear = 0.55f;
constexpr float kTanh1 = -0.33333331f, kTanh2 = 0.13333113f, kTanh3 = -0.053909428f, kTanh4 = 0.021309389f,
                kTanh5 = -0.0066102277f;  // of y^2, y^4, ...
__device__ __forceinline__ float capped_far(float s, const Params &p) {
    return fmaf(__fdividef(-2.f, 1.f + exp2_approx(s * p.cap_in)), p.cap_log2, p.cap_log2);
}
template <bool kCap>
__device__ __forceinline__ float score(float s, const Params &p) {
    if (!kCap) return s * p.scale_log2;
    const float far = capped_far(s, p);  // always: a branch costs more (48 tokens over 1500 35.4 us, so 31.8)
    const float y = s * p.cap_y, t = y * y;
    float r = fmaf(t, kTanh5, kTanh4);
    r = fmaf(t, r, kTanh3);
    r = fmaf(t, r, kTanh2);
    r = fmaf(t, r, kTanh1);
    r = fmaf(t, r, 1.f);
    return t < kTanhNear * kTanhNear ? s * p.scale_log2 * r : far;
}

// 1 / the weights' sum, 0 for a row that saw nothing, and the natural logarithm
// of the sum over the scores themselves (a NaN stays one in both).
__device__ __forceinline__ float over_sum(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float log_sum(float top, float sum) {
    return sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.693147180559945f;
}

struct Item {
    int b, qt, kh;
    int row0;    // first row (token) of the tile
    int nt;      // tokens in it
    int pos0;    // cache index of the first
    int len;     // cached tokens
    int seen;    // first key that a row sees
    int t0;      // first key tile
    int tiles;   // key tiles, at least 1 (a tile whose rows see nothing has one, all masked)
};

// Query tiles of a sequence with n new rows.
__device__ __forceinline__ int query_tiles(const Params &p, int n) {
    return p.tt == 1 ? n : int(__umulhi(unsigned(n + p.tt - 1), p.tt_magic));
}

template <int KT>
__device__ __forceinline__ void item_tiles(int window, int tt, const SeqView &s, int qt, int &nt,
                                           int &pos0, int &seen, int &t0, int &tiles) {
    nt = min(tt, s.n - qt * tt);
    pos0 = s.len - s.n + qt * tt;
    const int last = pos0 + nt - 1;
    seen = window > 0 && pos0 >= window ? pos0 - window + 1 : 0;
    t0 = seen / KT;
    tiles = last >= seen ? last / KT + 1 - t0 : 1;
}

// The CTA's run: positions [u, end) of the whole work; u is inside `item`,
// which starts at item_u with `extra` positions before its first tile.
struct Run {
    long per;  // positions of a run
    int pad;   // every item's cost where each CTA takes one whole, else 0
    long u, end, item_u;
    SeqView seq;  // item's sequence
    Item item;
};

// The work of a sequence: its query tiles' key tiles and fixed costs, of one
// key/value head.
template <int KT>
__device__ __forceinline__ long tile_cost(const Params &p, const SeqView &s, int qt) {
    int nt, pos0, seen, t0, tiles;
    item_tiles<KT>(p.window, p.tt, s, qt, nt, pos0, seen, t0, tiles);
    return tiles + p.extra;
}

// a / b for a >= 0, b > 0: as 32 bits where they fit (64-bit division is long).
__device__ __forceinline__ long div_pos(long a, long b) {
    if (((a | b) >> 31) == 0) return long(unsigned(a) / unsigned(b));
    return a / b;
}

// Beside a sequence's cost: its items (of all key/value heads) and their largest cost.
struct Items {
    int n, top;
};

// The run of this CTA from the sequences' costs and items, by one warp.  The
// lengths are read again for the item that is found: should the caller change them
// under the call (a missing stream order) they need not fit the costs any more, so
// what is derived from both, here and in join_desc, is bounded by the buffers.
template <int KT>
__device__ inline void run_find(const Params &p, int least, int split, const long *scratch, const Items *items,
                                Run &r) {
    const int lane = threadIdx.x & 31, B = p.b.B, Hkv = p.b.Hkv;
    // the sum of the lanes' values, each below 2^58, by 32-bit reductions
    auto total = [&](long v) {
        const unsigned lo = __reduce_add_sync(0xffffffffu, unsigned(v) & 0x3ffffffu);
        const unsigned mid = __reduce_add_sync(0xffffffffu, unsigned(v >> 26) & 0x3ffffffu);
        const unsigned hi = __reduce_add_sync(0xffffffffu, unsigned(v >> 52));
        return long(lo) + (long(mid) << 26) + (long(hi) << 52);
    };
    // the first of n entries past which the prefix sum from `at` goes beyond u: steps of 32
    // by their totals, then within the step
    auto locate = [&](int n, long at, auto cost, int &which, long &start) {
        for (int base = 0; base < n; base += 32) {
            const long mine = base + lane < n ? cost(base + lane) : 0;
            const long step = total(mine);
            if (at + step <= r.u) {
                at += step;
                continue;
            }
            long v = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long w = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += w;
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, at + v > r.u)) - 1;
            which = base + src;
            start = at + __shfl_sync(0xffffffffu, v - mine, src);
            return;
        }
    };
    long U = 0;
    unsigned n = 0, top = 0;
    for (int b = lane; b < B; b += 32) {
        U += scratch[b];
        n = min(n + unsigned(items[b].n), 1u << 26);
        top = max(top, unsigned(items[b].top));
    }
    U = total(U);
    n = __reduce_add_sync(0xffffffffu, n);
    top = __reduce_max_sync(0xffffffffu, top);
    const long even = div_pos(U, gridDim.x);
    // (a little more where memory is busy: 48 sequences of 1500 30 us whole, 33 in parts)
    r.pad = n <= gridDim.x && long(top) <= even + min(even, 16l) / 8 + split ? int(top) : 0;
    if (r.pad != 0) {
        U = long(n) * r.pad;
        r.per = r.pad;
    } else {
        r.per = max(long(least), even * gridDim.x == U ? even : even + 1);
    }
    r.u = r.per * blockIdx.x;
    r.end = min(U, r.u + r.per);
    if (r.u >= r.end) return;
    Item &it = r.item;
    it.b = 0;
    it.qt = 0;
    long at = 0, first = 0;
    if (B > 1) locate(B, 0, [&](int b) { return r.pad != 0 ? long(items[b].n) * r.pad : scratch[b]; }, it.b, at);
    r.seq = seq_view(p.b, it.b, p.hdr, false);
    const int nq = query_tiles(p, r.seq.n);
    if (nq > 1)
        locate(nq, at, [&](int qt) { return (r.pad != 0 ? long(r.pad) : tile_cost<KT>(p, r.seq, qt)) * Hkv; }, it.qt,
               first);
    else
        first = at;
    it.len = r.seq.len;
    it.row0 = r.seq.first + it.qt * p.tt;
    item_tiles<KT>(p.window, p.tt, r.seq, it.qt, it.nt, it.pos0, it.seen, it.t0, it.tiles);
    const long each = r.pad != 0 ? r.pad : it.tiles + p.extra;
    // the head, of few: a quotient in fp32, put right
    const long in = r.u - first;
    it.kh = min(int(__fdividef(float(in), float(each))), Hkv - 1);
    while (it.kh * each > in) --it.kh;
    while (it.kh + 1 < Hkv && (it.kh + 1) * each <= in) ++it.kh;
    r.item_u = first + it.kh * each;
}

// Every thread of the CTA calls it; `scratch`: 16 B bytes of shared memory, `out`:
// the run that the first warp finds.  A run is at least `least` long.  It is one
// item where there are no more of them than CTAs and the longest takes no longer
// than an even share and `split`, the time (in key tiles) of leaving parts and
// joining them.  False: nothing to do.  A thread per sequence where its tiles are
// few (decode), a warp where they are many, then one warp sums and searches.
template <int KT>
__device__ inline bool run_begin(const Params &p, int least, int split, long *scratch, Run *out, Run &run) {
    constexpr int kFew = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int B = p.b.B, Hkv = p.b.Hkv;
    Items *items = reinterpret_cast<Items *>(scratch + B);
    for (int base = warp * 32; base < B; base += nw * 32) {
        const int b = base + lane;
        int nq = 0;
        long total = 0, top = 0;
        if (b < B) {
            const SeqView s = seq_view(p.b, b, p.hdr, blockIdx.x == 0);
            nq = query_tiles(p, s.n);
            if (nq <= kFew) {
                for (int qt = 0; qt < nq; ++qt) {
                    const long c = tile_cost<KT>(p, s, qt);
                    total += c;
                    top = max(top, c);
                }
                scratch[b] = total * Hkv;
                items[b] = {nq * Hkv, int(top)};
            }
        }
        __syncwarp();
        for (unsigned many = __ballot_sync(0xffffffffu, nq > kFew); many != 0; many &= many - 1) {
            const int src = __ffs(many) - 1, nqs = __shfl_sync(0xffffffffu, nq, src);
            const SeqView s = seq_view(p.b, base + src, p.hdr, false);
            total = 0;
            unsigned most = 0;
            for (int qt = lane; qt < nqs; qt += 32) {
                const long c = tile_cost<KT>(p, s, qt);
                total += c;
                most = max(most, unsigned(c));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) {
                scratch[base + src] = total * Hkv;
                items[base + src] = {nqs * Hkv, int(most)};
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 0) {
        // A warp that left a branch lane by lane stays apart, at a multiple of the time, until it is
        // brought together (the search took 6000 cycles that way, 2000 so); so wherever
        // single lanes have just worked, here and in the kernels.
        __syncwarp();
        Run r;
        run_find<KT>(p, least, split, scratch, items, r);
        if (lane == 0) *out = r;
    }
    __syncthreads();
    __syncwarp();
    run = *out;
    return run.u < run.end;
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
    r.u = r.item_u = r.item_u + (r.pad != 0 ? r.pad : p.extra + it.tiles);
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
    item_tiles<KT>(p.window, p.tt, r.seq, it.qt, it.nt, it.pos0, it.seen, it.t0, it.tiles);
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

__device__ __forceinline__ float ld_l2(const float *p) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 ld_l2_v4(const float *p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p));
    return v;
}

// The parts of r.item: consecutive CTAs from the one with its first tile on.
__device__ __forceinline__ JoinDesc join_desc(const Params &p, const Run &r) {
    const long first = r.item_u + p.extra;
    JoinDesc d;
    const long cta = div_pos(first, r.per);
    d.parts = int(min(div_pos(first + r.item.tiles - 1, r.per), long(gridDim.x) - 1) - cta) + 1;
    d.row0 = r.item.row0;
    d.nt = r.item.nt;
    d.kh = r.item.kh;
    return d;
}

// Joins parts first_cta .. of an item of `rows` rows: row r is token
// r / half * tth + r % half / G of the item, head r % half % G.  All threads of a
// CTA of W warps call it, for the blocks of rows blk, blk + step, ...; `sv`, `sm`,
// `sl`: W * D * 4, W * 4 and W * 4 floats of shared memory.
//
// What bounds it is the latency of dependent loads, so their chain is kept
// short: a group of S warps (S by the number of parts) takes four consecutive
// rows, each warp every S-th part, four at a time with all their loads in
// flight together; the warps' results meet in shared memory.  Lane l holds
// row l / 2 % 4, of each 32 channels the four from 8 (l / 8) + 4 (l % 2).
constexpr int kJoinRows = 4;
constexpr int kJoinParts = 4;

template <typename T, int D, int W>
__device__ inline void join_rows(const Params &p, const JoinDesc &d, int first_cta, int rows, int half, int tth,
                                 int blk0, int step, float *sv_mem, float *sm, float *sl) {
    constexpr int kVec = D / 32;
    float4 *sv = reinterpret_cast<float4 *>(sv_mem);  // [W][kVec][32]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.b.Hq / p.b.Hkv;
    const size_t stride = part_floats(rows, D);
    const int S = d.parts <= kJoinParts ? 1 : d.parts <= 4 * kJoinParts ? 4 : W;
    const int group = warp / S, w0 = warp % S, groups = W / S;
    const int sub = (lane >> 1) & 3, ch0 = 8 * (lane >> 3) + 4 * (lane & 1);
    const int used = half == rows ? min(rows, d.nt * G) : rows;  // rows past the tokens' end
    const int blocks = (used + kJoinRows * groups - 1) / (kJoinRows * groups);
    for (int blk = blk0; blk < blocks; blk += step) {
        const int row = (blk * groups + group) * kJoinRows + sub;
        const int tok_h = row % half / G, tok = row / half * tth + tok_h;
        const bool live = row < rows && tok_h < tth && tok < d.nt;  // rows of no token have no sums
        float top = -CUDART_INF_F, sum = 0.f;
        float4 v[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = w0; live && i0 < d.parts; i0 += S * kJoinParts) {
            float m[kJoinParts], l[kJoinParts];
            float4 x[kJoinParts][kVec];
#pragma unroll
            for (int u = 0; u < kJoinParts; ++u) {
                const int i = i0 + S * u;
                m[u] = -CUDART_INF_F;
                l[u] = 0.f;
#pragma unroll
                for (int c = 0; c < kVec; ++c) x[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < d.parts) {
                    // part 0 is the item's start, the others go on in the CTAs after it; read where
                    // other CTAs' stores are (not in L1)
                    const float *q = p.part + size_t(part_slot(first_cta + i, i == 0)) * stride;
                    m[u] = ld_l2(q + rows * D + row);
                    l[u] = ld_l2(q + rows * (D + 1) + row);
#pragma unroll
                    for (int c = 0; c < kVec; ++c) x[u][c] = ld_l2_v4(q + part_at(row, 32 * c + ch0, D));
                }
            }
            float up = top;
#pragma unroll
            for (int u = 0; u < kJoinParts; ++u) up = fmaxf(up, m[u]);
            const float base = up == -CUDART_INF_F ? 0.f : up, old = exp2_approx(top - base);
            top = up;
            sum *= old;
#pragma unroll
            for (int c = 0; c < kVec; ++c) v[c].x *= old, v[c].y *= old, v[c].z *= old, v[c].w *= old;
#pragma unroll
            for (int u = 0; u < kJoinParts; ++u) {
                const float f = exp2_approx(m[u] - base);
                sum = fmaf(l[u], f, sum);
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    v[c].x = fmaf(x[u][c].x, f, v[c].x);
                    v[c].y = fmaf(x[u][c].y, f, v[c].y);
                    v[c].z = fmaf(x[u][c].z, f, v[c].z);
                    v[c].w = fmaf(x[u][c].w, f, v[c].w);
                }
            }
        }
        bool mine[kVec];  // the vectors this warp finishes
#pragma unroll
        for (int c = 0; c < kVec; ++c) mine[c] = S == 1 || c % S == w0;
        if (S > 1) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < kVec; ++c) sv[(warp * kVec + c) * 32 + lane] = v[c];
            if (ch0 == 0) {
                sm[warp * kJoinRows + sub] = top;
                sl[warp * kJoinRows + sub] = sum;
            }
            __syncthreads();
            const int first = group * S;
            for (int w = 0; w < S; ++w) top = fmaxf(top, sm[(first + w) * kJoinRows + sub]);
            const float base = top == -CUDART_INF_F ? 0.f : top;
            sum = 0.f;
#pragma unroll
            for (int c = 0; c < kVec; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < S; ++w) {
                const float f = exp2_approx(sm[(first + w) * kJoinRows + sub] - base);
                sum = fmaf(sl[(first + w) * kJoinRows + sub], f, sum);
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    if (!mine[c]) continue;
                    const float4 y = sv[((first + w) * kVec + c) * 32 + lane];
                    v[c].x = fmaf(y.x, f, v[c].x);
                    v[c].y = fmaf(y.y, f, v[c].y);
                    v[c].z = fmaf(y.z, f, v[c].z);
                    v[c].w = fmaf(y.w, f, v[c].w);
                }
            }
        }
        __syncwarp();
        if (!live) continue;
        const size_t at = size_t(d.row0 + tok) * p.b.Hq + d.kh * G + row % half % G;
        const float inv = over_sum(sum);
#pragma unroll
        for (int c = 0; c < kVec; ++c)
            if (mine[c])
                *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + at * D + 32 * c + ch0) =
                    make_uint2(Pair<T>::make(v[c].x * inv, v[c].y * inv), Pair<T>::make(v[c].z * inv, v[c].w * inv));
        if (p.lse != nullptr && ch0 == 0 && w0 == 0)
            p.lse[at] = log_sum(top, sum);
    }
}

// The second launch: joins the items that start in each CTA's run.
cudaError_t launch_join(const Params &p, moe_dtype type, int grid, int rows, int half, int tth, cudaStream_t s);

// The tensor-core kernel (many rows per key/value head).
size_t tc_part_bytes(int D);
cudaError_t init_tc();
cudaError_t launch_tc(const AttnArgs &a, const Params &p, int num_sms, cudaStream_t s);

}  // namespace attn
}  // namespace moeq4k
