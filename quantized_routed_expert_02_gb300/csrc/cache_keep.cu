// The accepted ones of a tree's drafted tokens move together in the paged
// cache (moe_cache_keep): row base + keep[d] -> base + d.
//
// A CTA moves the rows of one sequence and head, keys or values.  keep rises
// strictly, so keep[d] >= d: a step's rows are all read before any is written,
// and what it writes lies before every row that a later step reads.  Bytes bound
// for many rows; few take the chain of dependent reads (lengths, keep, table, row): five rows of one
// sequence 2.4 us, up to 24 of each of 64 sequences 5.0 us.
#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace moeq4k {
namespace keep {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) cache_keep_kernel(const KeepArgs a) {
    __shared__ bool bad;
    pdl_enter();
    const int b = blockIdx.x, kh = blockIdx.y, tid = threadIdx.x;
    const bool first = blockIdx.y == 0 && blockIdx.z == 0;  // the CTA that records
    const SeqView s = seq_view(a.b, b, a.hdr, first && tid == 0);
    if (tid == 0) bad = false;
    __syncthreads();
    const int kept = a.kept[b], base = s.len - s.n;
    const int32_t *keep = a.keep + size_t(b) * a.most;
    if (!s.ok || kept == 0) return;
    if (kept < 0 || kept > a.most || kept > s.n || base < 0) {
        if (first && tid == 0) record_status(a.hdr, MOE_ERR_CACHE_RANGE, base < 0 ? base : kept);
        return;
    }
    // every entry and every page, before anything is written
    for (int d = tid; d < kept; d += kThreads) {
        const int i = keep[d], before = d > 0 ? keep[d - 1] : -1;
        if (i <= before || i >= s.n) {
            if (first) record_status(a.hdr, MOE_ERR_CACHE_RANGE, i);
            bad = true;
        } else if (page_of(a.b, b, base + i, a.hdr) < 0 || page_of(a.b, b, base + d, a.hdr) < 0) {
            bad = true;
        }
    }
    __syncthreads();
    if (bad) return;
    const int row_bytes = a.b.D * a.elem, chunks = row_bytes / 16, rows = kThreads / chunks;
    uint8_t *data = static_cast<uint8_t *>(blockIdx.z == 0 ? a.k : a.v);
    float *scales = blockIdx.z == 0 ? a.ks : a.vs;
    auto place = [&](int j) {  // the cache row of cached token j
        const int pg = a.b.table[size_t(b) * a.b.max_pages + j / a.b.page];
        return (size_t(pg) * a.b.Hkv + kh) * a.b.page + j % a.b.page;
    };
    for (int d0 = 0; d0 < kept; d0 += rows) {
        const int d = d0 + tid / chunks, c = tid % chunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        float f = 0.f;
        const bool moves = d < kept && keep[d] != d;
        if (moves) {
            const size_t from = place(base + keep[d]);
            v = *reinterpret_cast<const uint4 *>(data + from * row_bytes + c * 16);
            if (scales != nullptr && c == 0) f = scales[from];
        }
        __syncthreads();
        if (moves) {
            const size_t to = place(base + d);
            *reinterpret_cast<uint4 *>(data + to * row_bytes + c * 16) = v;
            if (scales != nullptr && c == 0) scales[to] = f;
        }
    }
}

}  // namespace keep

cudaError_t launch_cache_keep(const KeepArgs &a, cudaStream_t s) {
    return launch_pdl(keep::cache_keep_kernel, dim3(a.b.B, a.b.Hkv, 2), dim3(keep::kThreads), size_t(0), s, a);
}

}  // namespace moeq4k
