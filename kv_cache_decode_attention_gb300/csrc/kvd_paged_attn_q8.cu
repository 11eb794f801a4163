// kvd_paged_attn_q8.cu -- paged_attention over pages of 8-bit codes.

#include <cmath>
#include <cstring>

#include "kvd_q8.cuh"
#include "kvd_rope.cuh"

namespace kvd {
namespace {

struct QaArgs {
    const void *q;
    void *out;
    int64_t q_tok, q_head, out_tok, out_head;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *cu_new, *seq_len;
    const float *sinks;
    uint32_t *err;
    int64_t window;
    int32_t n_seq, n_tokens, n_q, n_kv, group, max_pages, n_pages, page_log2, hd;
    float scale, softcap;
};

// A warp for each new row and query head, a row of K and V at a time.
template <typename T, int HD>
__global__ void __launch_bounds__(128) rows_kernel(const __grid_constant__ QaArgs a) {
    constexpr int kPer = HD / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)  // requests that no row asks about are looked at too
        for (int b = threadIdx.x; b < a.n_seq; b += blockDim.x) {
            const int32_t q0 = a.cu_new[b], q1 = a.cu_new[b + 1], len = a.seq_len[b];
            if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 || len > (int64_t(a.max_pages) << a.page_log2)) set_error(a.err, kErrBounds);
        }
    const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int64_t tok = item / a.n_q;
    const int head = int(item - tok * a.n_q), kv = head / a.group;
    if (tok >= a.n_tokens || tok < a.cu_new[0] || tok >= a.cu_new[a.n_seq]) return;
    int b = 0, above = a.n_seq;
    while (above - b > 1) {
        const int mid = (b + above) / 2;
        if (a.cu_new[mid] <= tok) b = mid;
        else above = mid;
    }
    const int32_t q0 = a.cu_new[b], q1 = a.cu_new[b + 1], len = a.seq_len[b];
    if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 || len > (int64_t(a.max_pages) << a.page_log2)) {
        set_error(a.err, kErrBounds);
        return;
    }
    const int64_t pos = int64_t(len) - (q1 - q0) + (tok - q0);
    int64_t first = a.window > 0 ? pos - a.window + 1 : 0;
    if (first < 0) first = 0;
    float q[kPer], o[kPer] = {};
    const T *qp = static_cast<const T *>(a.q) + tok * a.q_tok + head * a.q_head + lane * kPer;
    for (int i = 0; i < kPer; ++i) q[i] = to_f32<T>(qp[i]) * a.scale;
    float top = -INFINITY, sum = 0.0f;
    for (int64_t p = first; p <= pos; ++p) {
        const int32_t page = a.block_table[int64_t(b) * a.max_pages + (p >> a.page_log2)];
        const bool there = page >= 0 && page < a.n_pages;
        if (!there) set_error(a.err, kErrBounds);
        const int64_t block = int64_t(there ? page : 0) * a.n_kv + kv;
        const int64_t at = ((block << a.page_log2) + (p & ((1 << a.page_log2) - 1))) * HD + lane * kPer;
        auto value = [&](const uint8_t *x) {
            return there ? __half2float(__half(__nv_cvt_fp8_to_halfraw(*x, __NV_E4M3))) : 0.0f;
        };
        float s = 0.0f;
        for (int i = 0; i < kPer; ++i) s += q[i] * value(a.k + at + i);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        s *= scale_of(a.k_scale[block], a.err);
        if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
        const float now = fmaxf(top, s), f = expf(top - now), w = expf(s - now);
        sum = sum * f + w;
        const float wv = w * scale_of(a.v_scale[block], a.err);
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + wv * value(a.v + at + i);
        top = now;
    }
    float g = 1.0f;
    if (a.sinks != nullptr && top != -INFINITY) {
        const float all = fmaxf(top, a.sinks[head]);
        g = expf(top - all);
        sum = sum * g + expf(a.sinks[head] - all);
    }
    g *= sum == 0.0f ? 0.0f : 1.0f / sum;
    T *op = static_cast<T *>(a.out) + tok * a.out_tok + head * a.out_head + lane * kPer;
    for (int i = 0; i < kPer; ++i) op[i] = from_f32<T>(o[i] * g);
}

bool shape_ok(int64_t n_tokens, int32_t n_q, int32_t n_kv, int32_t hd) {
    return n_tokens >= 0 && n_tokens <= kMaxTokens && n_kv >= 1 && n_kv <= 1024 && n_q >= n_kv && n_q % n_kv == 0 &&
           n_q / n_kv <= kMaxHpk && (hd == 64 || hd == 128);
}

// A [tokens][heads][hd] view whose rows a 16-byte access may touch (the stride of
// an axis with one entry is never used).
bool view_ok(const kvd_rows *r, int64_t tokens, int32_t heads) {
    const int64_t lim = int64_t(1) << 38;
    if (r == nullptr || (r->data == nullptr && tokens > 0) || (reinterpret_cast<uintptr_t>(r->data) & 15) != 0) return false;
    if (tokens == 0) return true;
    auto ok = [&](int64_t entries, int64_t stride) {
        return entries <= 1 || (stride >= 0 && stride < lim && stride % 8 == 0);
    };
    return ok(tokens, r->token_stride) && ok(heads, r->head_stride);
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status paged_attention_q8_workspace_bytes(int64_t n_tokens, int32_t n_q, int32_t n_kv, int32_t head_dim,
                                                         int64_t *bytes_out) {
    if (bytes_out == nullptr || !shape_ok(n_tokens, n_q, n_kv, head_dim)) return KVD_EINVAL;
    *bytes_out = 256;
    return KVD_OK;
}

extern "C" kvd_status paged_attention_q8(const kvd_rows *q, const kvd_rows *out, int64_t n_tokens, int32_t n_q, int32_t n_kv,
                                         int32_t head_dim, int32_t dtype, const void *k_pages, const void *v_pages,
                                         const float *k_scale, const float *v_scale, int64_t n_pages, int32_t page_size,
                                         const int32_t *block_table, int32_t max_pages, const int32_t *cu_new,
                                         const int32_t *seq_len, int32_t n_seq, float scale, int64_t window, float softcap,
                                         const float *sinks, void *workspace, int64_t workspace_bytes, uint32_t *err,
                                         void *stream) {
    KVD_NVTX_RANGE("paged_attention_q8");
    if (!shape_ok(n_tokens, n_q, n_kv, head_dim) || (dtype != KVD_T_F16 && dtype != KVD_T_BF16)) return KVD_EINVAL;
    if (!view_ok(q, n_tokens, n_q) || !view_ok(out, n_tokens, n_q)) return KVD_EINVAL;
    if (k_pages == nullptr || v_pages == nullptr ||
        ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15) != 0)
        return KVD_EINVAL;
    if (k_scale == nullptr || v_scale == nullptr ||
        ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3) != 0)
        return KVD_EINVAL;
    if ((page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) || n_pages < 1 || n_pages >= (int64_t(1) << 31) ||
        n_pages * page_size * n_kv >= (int64_t(1) << 31))
        return KVD_EINVAL;
    if (block_table == nullptr || cu_new == nullptr || seq_len == nullptr || err == nullptr || n_seq < 1 || n_seq > (1 << 20) || max_pages < 1 ||
        int64_t(max_pages) * page_size > (int64_t(1) << 31) - 1024)
        return KVD_EINVAL;
    if (!std::isfinite(scale) || scale <= 0.0f || window < 0 || !std::isfinite(softcap) || softcap < 0.0f) return KVD_EINVAL;
    const float log2e = 1.4426950408889634f;
    if (!std::isfinite(scale * log2e) || (softcap > 0.0f && (!std::isfinite(softcap * log2e) || !std::isfinite(2.0f * scale * log2e / softcap))))
        return KVD_EINVAL;
    if (sinks != nullptr && (reinterpret_cast<uintptr_t>(sinks) & 3) != 0) return KVD_EINVAL;
    if (n_tokens == 0) return KVD_OK;
    {
        const View o = view_of(out, n_tokens, n_q, head_dim, 2);
        const int64_t pages = n_pages * page_size * n_kv * head_dim, scales = n_pages * n_kv * 4;
        if (!rows_apart(o) || !views_apart(o, view_of(q, n_tokens, n_q, head_dim, 2)) || !views_apart(o, make_range(k_pages, pages)) ||
            !views_apart(o, make_range(v_pages, pages)) || !views_apart(o, make_range(k_scale, scales)) ||
            !views_apart(o, make_range(v_scale, scales)))
            return KVD_EINVAL;
    }
    int64_t need = 0;
    paged_attention_q8_workspace_bytes(n_tokens, n_q, n_kv, head_dim, &need);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < need) return KVD_EINVAL;
    QaArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q->data;
    a.q_tok = q->token_stride;
    a.q_head = q->head_stride;
    a.out = out->data;
    a.out_tok = out->token_stride;
    a.out_head = out->head_stride;
    a.k = static_cast<const uint8_t *>(k_pages);
    a.v = static_cast<const uint8_t *>(v_pages);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.block_table = block_table;
    a.cu_new = cu_new;
    a.seq_len = seq_len;
    a.sinks = sinks;
    a.err = err;
    a.window = window < (int64_t(1) << 31) ? window : 0;
    a.n_seq = n_seq;
    a.n_tokens = int32_t(n_tokens);
    a.n_q = n_q;
    a.n_kv = n_kv;
    a.group = n_q / n_kv;
    a.max_pages = max_pages;
    a.n_pages = int32_t(n_pages);
    a.page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    a.hd = head_dim;
    a.scale = scale;
    a.softcap = softcap;
    const auto kern = dtype == KVD_T_F16 ? (head_dim == 64 ? rows_kernel<__half, 64> : rows_kernel<__half, 128>)
                                         : (head_dim == 64 ? rows_kernel<__nv_bfloat16, 64> : rows_kernel<__nv_bfloat16, 128>);
    const cudaError_t e = launch_pdl(kern, dim3(unsigned(ceil_div(n_tokens * n_q, 4))), dim3(128), 0, as_stream(stream), a);
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}
