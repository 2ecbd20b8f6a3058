// Device-side reading of a paged batch: which sequence a row belongs to, its
// cache index, and the checks that keep a bad table inside the buffers.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.cuh"

namespace moeq4k {

struct SeqView {
    int first;  // first row
    int n;      // new rows
    int len;    // cached tokens, the new ones included
    bool ok;    // lengths and offsets are in range
};

// Sequence b of the batch; one that is out of range comes back empty, with
// the offending value recorded (`report`: one thread of the grid's that look).
__device__ inline SeqView seq_view(const PagedBatch &p, int b, WsHeader *hdr, bool report) {
    SeqView s;
    const int lo = p.offs[b], hi = p.offs[b + 1], len = p.lens[b];
    const bool offs_ok = lo >= 0 && hi >= lo && hi <= p.N;
    const bool len_ok = len >= 0 && int64_t(len) <= int64_t(p.max_pages) * p.page;
    s.ok = offs_ok && len_ok;
    s.first = s.ok ? lo : 0;
    s.n = s.ok ? hi - lo : 0;
    s.len = s.ok ? len : 0;
    if (!s.ok && report) record_status(hdr, MOE_ERR_CACHE_RANGE, offs_ok ? len : (lo < 0 || lo > p.N ? lo : hi));
    return s;
}

// The page of cache index j of sequence b, or -1 (recorded) when the table
// names none of the cache's.
__device__ inline int page_of(const PagedBatch &p, int b, int j, WsHeader *hdr) {
    const int pg = p.table[size_t(b) * p.max_pages + j / p.page];
    if (pg < 0 || pg >= p.num_pages) {
        record_status(hdr, MOE_ERR_CACHE_RANGE, pg);
        return -1;
    }
    return pg;
}

// The 16-bit types: pairs to fp32 and back (round to nearest even).
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    static __device__ __forceinline__ float2 load(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ uint32_t make(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 load(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t make(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

}  // namespace moeq4k
