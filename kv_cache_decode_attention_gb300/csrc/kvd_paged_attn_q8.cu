// kvd_paged_attn_q8.cu -- paged_attention over pages of 8-bit codes.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "kvd_paged_attn_q8.cuh"

namespace kvd {
namespace {

// The driver's encoder, looked up once; nullptr if it is missing.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Codes as rows of head_dim bytes, a page of them to a box.
bool encode(CUtensorMap *m, const void *base, int32_t hd, int64_t rows, int32_t page_size) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    const cuuint64_t dims[2] = {cuuint64_t(hd), cuuint64_t(rows)}, strides[1] = {cuuint64_t(hd)};
    const cuuint32_t box[2] = {cuuint32_t(hd), cuuint32_t(page_size)}, ones[2] = {1, 1};
    return fn != nullptr && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, ones,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct WsLayout {
    int64_t cut, ml, o, total;
};
WsLayout ws_layout(int32_t hd) {
    WsLayout w;
    const int64_t rows = int64_t(2) * kQrMaxCtas * kQrRows;
    w.cut = 0;
    w.ml = round_up(int64_t(kQrMaxCtas) * int64_t(sizeof(QrCut)), 256);
    w.o = w.ml + round_up(rows * 8, 256);
    w.total = w.o + rows * hd * 4;
    return w;
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
    *bytes_out = ws_layout(head_dim).total;
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
    const WsLayout ws = ws_layout(head_dim);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < ws.total) return KVD_EINVAL;
    QrArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t pool_rows = n_pages * page_size * n_kv;
    if (!encode(&a.k, k_pages, head_dim, pool_rows, page_size) || !encode(&a.v, v_pages, head_dim, pool_rows, page_size)) return KVD_EINVAL;
    char *w = static_cast<char *>(workspace);
    a.cut = reinterpret_cast<QrCut *>(w + ws.cut);
    a.part_ml = reinterpret_cast<float2 *>(w + ws.ml);
    a.part_o = reinterpret_cast<float *>(w + ws.o);
    a.q = q->data;
    a.q_tok = q->token_stride;
    a.q_head = q->head_stride;
    a.out = out->data;
    a.out_tok = out->token_stride;
    a.out_head = out->head_stride;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.block_table = block_table;
    a.cu_new = cu_new;
    a.seq_len = seq_len;
    a.sinks = sinks;
    a.err = err;
    // every position is below 2^31, so a window from there on hides nothing
    a.window = window < (int64_t(1) << 31) ? window : 0;
    a.n_seq = n_seq;
    a.n_tokens = int32_t(n_tokens);
    a.n_kv = n_kv;
    a.group = n_q / n_kv;
    a.tile_tok = kQrRows / a.group;
    a.max_pages = max_pages;
    a.n_pages = int32_t(n_pages);
    a.page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    a.pool_rows = int32_t(pool_rows);
    a.give_up = -1;
    // A cap so far above the scale that their quotient is no normal number (a raw
    // score would have to pass 10^34 to feel it) is none.
    const bool cap = softcap > 0.0f && scale / softcap >= FLT_MIN;
    a.mul = cap ? float(2.0 * 1.4426950408889634 * double(scale) / softcap) : scale * log2e;
    a.cap = cap ? softcap * log2e : 0.0f;
    const bool bf16 = dtype == KVD_T_BF16;
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = head_dim == 64 ? (bf16 ? launch_qr<64, true>(a, st) : launch_qr<64, false>(a, st))
                                         : (bf16 ? launch_qr<128, true>(a, st) : launch_qr<128, false>(a, st));
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}
