// C ABI of the attention half of a decoder block: argument checks and launches
// of moe_add_rmsnorm, moe_rope_append and moe_attention_paged.
#include "abi_checks.cuh"
#include "common.cuh"
#include "kernels.cuh"

using namespace moeq4k;

namespace {

constexpr int kMaxRows = 1 << 22;
constexpr int kMaxNormH = 16384;
constexpr int kMaxSeqs = 4096;
constexpr int kMaxHeads = 256;
constexpr int kMaxGroup = 128;
constexpr int kMaxAxes = 8;
constexpr int64_t kMaxIndex = int64_t(1) << 30;  // page-heads of a cache, tokens of a sequence

bool known_type(moe_dtype t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }
bool type16(moe_dtype t) { return t == MOE_F16 || t == MOE_BF16; }

moe_status check_heads(int Hq, int Hkv, int D) {
    if (Hkv < 1 || Hq < Hkv || Hq > kMaxHeads || Hq % Hkv != 0 || Hq / Hkv > kMaxGroup)
        return MOE_ERR_INVALID_SHAPE;
    if (D != 64 && D != 128) return MOE_ERR_INVALID_SHAPE;
    return MOE_OK;
}

moe_status check_batch(const PagedBatch &p, moe_dtype type) {
    if (p.N < 1 || p.N > kMaxRows || p.B < 1 || p.B > kMaxSeqs) return MOE_ERR_INVALID_SHAPE;
    if (p.max_pages < 1 || p.num_pages < 1) return MOE_ERR_INVALID_SHAPE;
    if (p.page != 16 && p.page != 32 && p.page != 64 && p.page != 128 && p.page != 256)
        return MOE_ERR_INVALID_SHAPE;
    MOE_TRY(check_heads(p.Hq, p.Hkv, p.D));
    if (int64_t(p.num_pages) * p.Hkv > kMaxIndex || int64_t(p.max_pages) * p.page > kMaxIndex)
        return MOE_ERR_INVALID_SHAPE;
    if (!type16(type)) return MOE_ERR_INVALID_SHAPE;
    return MOE_OK;
}

moe_status check_batch_ptrs(const PagedBatch &p, const void *k, const void *v, const void *ws) {
    MOE_TRY(check_ptr(k, 16));
    MOE_TRY(check_ptr(v, 16));
    MOE_TRY(check_ptr(p.table, 4));
    MOE_TRY(check_ptr(p.offs, 4));
    MOE_TRY(check_ptr(p.lens, 4));
    return check_ptr(ws, 256);
}

}  // namespace

extern "C" {

moe_status moe_add_rmsnorm(const void *x, moe_dtype x_type, const float *residual,
                           const float *gamma, float eps, int T, int H, float *sum_out, void *y,
                           moe_dtype y_type, int8_t *q, float *d, int32_t *sums, void *stream) {
    if (T < 1 || T > kMaxRows || H < 8 || H % 8 != 0 || H > kMaxNormH) return MOE_ERR_INVALID_SHAPE;
    if (!known_type(x_type) || (y != nullptr && !known_type(y_type))) return MOE_ERR_INVALID_SHAPE;
    if (!(eps >= 0.f) || !finite_f(eps)) return MOE_ERR_INVALID_SHAPE;
    const bool any_q = q != nullptr || d != nullptr || sums != nullptr;
    if (any_q && H % kQK != 0) return MOE_ERR_INVALID_SHAPE;
    MOE_TRY(check_ptr(x, 16));
    MOE_TRY(check_opt(residual, 16));
    MOE_TRY(check_ptr(gamma, 16));
    MOE_TRY(check_opt(sum_out, 16));
    MOE_TRY(check_opt(y, 16));
    if (any_q) {
        MOE_TRY(check_ptr(q, 16));
        MOE_TRY(check_ptr(d, 4));
        MOE_TRY(check_ptr(sums, 4));
    }
    if (sum_out == nullptr && y == nullptr && !any_q) return MOE_ERR_NULL;
    if (stream == MOE_CHECK_ONLY) return MOE_OK;
    int sms = 0;
    MOE_TRY(device_info(&sms, nullptr));
    AddNormArgs a = {};
    a.x = x, a.residual = residual, a.gamma = gamma, a.sum_out = sum_out, a.y = y;
    a.q = q, a.d = d, a.sums = sums, a.eps = eps, a.T = T, a.H = H;
    a.x_type = x_type, a.y_type = y_type;
    return cuda_status(launch_add_rmsnorm(a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_rope_append(const void *qkv, const int32_t *pos, const double *inv_freq,
                           const int32_t *axis, int axes, int rot_dim, int interleaved,
                           const float *q_norm_w, const float *k_norm_w, float norm_eps,
                           void *q_out, void *k_pages, void *v_pages, const int32_t *page_table,
                           const int32_t *q_offs, const int32_t *kv_lens, int N, int B,
                           int max_pages, int num_pages, int page, int Hq, int Hkv, int D,
                           moe_dtype dtype, void *ws, size_t ws_bytes, void *stream) {
    const PagedBatch p = {page_table, q_offs, kv_lens, N, B, max_pages, num_pages, page, Hq, Hkv, D};
    MOE_TRY(check_batch(p, dtype));
    if (axes < 1 || axes > kMaxAxes || rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > D)
        return MOE_ERR_INVALID_SHAPE;
    if (!(norm_eps >= 0.f) || !finite_f(norm_eps)) return MOE_ERR_INVALID_SHAPE;
    MOE_TRY(check_ptr(qkv, 16));
    MOE_TRY(check_ptr(pos, 4));
    MOE_TRY(check_ptr(inv_freq, 8));
    MOE_TRY(check_opt(axis, 4));
    MOE_TRY(check_opt(q_norm_w, 16));
    MOE_TRY(check_opt(k_norm_w, 16));
    MOE_TRY(check_ptr(q_out, 16));
    MOE_TRY(check_batch_ptrs(p, k_pages, v_pages, ws));
    if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE;
    if (stream == MOE_CHECK_ONLY) return MOE_OK;
    int sms = 0;
    MOE_TRY(device_info(&sms, nullptr));
    RopeArgs a = {};
    a.qkv = qkv, a.pos = pos, a.inv_freq = inv_freq, a.axis = axis, a.qw = q_norm_w, a.kw = k_norm_w;
    a.q_out = q_out, a.k = k_pages, a.v = v_pages, a.b = p, a.axes = axes, a.rot = rot_dim;
    a.eps = norm_eps, a.interleaved = interleaved != 0, a.type = dtype;
    a.hdr = static_cast<WsHeader *>(ws);
    return cuda_status(launch_rope_append(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_attention_workspace_bytes(int Hq, int Hkv, int D) {
    if (check_heads(Hq, Hkv, D) != MOE_OK) return 0;
    return sizeof(WsHeader) + attention_part_bytes(D);
}

moe_status moe_attention_paged(const void *q, const void *k_pages, const void *v_pages,
                               const int32_t *page_table, const int32_t *q_offs,
                               const int32_t *kv_lens, int N, int B, int max_new, int max_pages,
                               int num_pages, int page, int Hq, int Hkv, int D, moe_dtype dtype,
                               float scale, float softcap, int window, void *out, float *lse,
                               void *ws, size_t ws_bytes, void *stream) {
    const PagedBatch p = {page_table, q_offs, kv_lens, N, B, max_pages, num_pages, page, Hq, Hkv, D};
    MOE_TRY(check_batch(p, dtype));
    if (max_new < 1 || window < 0 || !finite_f(scale) || !(softcap >= 0.f) || !finite_f(softcap))
        return MOE_ERR_INVALID_SHAPE;
    if (softcap > 0.f && !finite_f(4.f * scale / softcap)) return MOE_ERR_INVALID_SHAPE;
    MOE_TRY(check_ptr(q, 16));
    MOE_TRY(check_ptr(out, 16));
    MOE_TRY(check_opt(lse, 4));
    MOE_TRY(check_batch_ptrs(p, k_pages, v_pages, ws));
    if (ws_bytes < moe_attention_workspace_bytes(Hq, Hkv, D)) return MOE_ERR_WORKSPACE;
    if (stream == MOE_CHECK_ONLY) return MOE_OK;
    int sms = 0;
    MOE_TRY(attention_info(&sms));
    AttnArgs a = {};
    a.q = q, a.k = k_pages, a.v = v_pages, a.out = out, a.lse = lse, a.b = p;
    a.scale = scale, a.softcap = softcap, a.window = window, a.type = dtype;
    a.hdr = static_cast<WsHeader *>(ws);
    a.scratch = static_cast<uint8_t *>(ws) + sizeof(WsHeader);
    a.wait_ns = device_wait_ns();
    a.withhold = device_withhold();
    return cuda_status(launch_attention(a, max_new, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
