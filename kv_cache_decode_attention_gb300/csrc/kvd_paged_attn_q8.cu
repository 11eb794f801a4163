// kvd_paged_attn_q8.cu -- paged_attention over pages of 8-bit codes.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>

#include "kvd_paged_attn_q8p.cuh"

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

// Rows of one piece of a large item.
int32_t piece_rows(int64_t n_tokens, int32_t group) {
    const int64_t rows = round_up(n_tokens * group, 8);
    return int32_t(rows < kQpMaxRows ? rows : kQpMaxRows);
}

struct WsLayout {
    int64_t cut[2], ml[2], o[2], total;  // of the launch for few rows, and of the one for many
};
WsLayout ws_layout(int64_t n_tokens, int32_t group, int32_t hd) {
    WsLayout w;
    const int64_t ctas[2] = {kQrMaxCtas, n_tokens * group > kQrRows ? kQpCtas : 0};
    const int64_t rows[2] = {kQrRows, piece_rows(n_tokens, group)};
    int64_t at = 0;
    for (int i = 0; i < 2; ++i) {
        w.cut[i] = at;
        w.ml[i] = w.cut[i] + round_up(ctas[i] * int64_t(sizeof(QrCut)), 256);
        w.o[i] = w.ml[i] + round_up(2 * ctas[i] * rows[i] * 8, 256);
        at = w.o[i] + 2 * ctas[i] * rows[i] * hd * 4;
    }
    w.total = at;
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

// What an item costs beside its tiles, in tiles: 10 us of 1.6 us (few rows), 8 of 1.2 to
// 1.7.  (Drafts took 70 us without, 57 with 2, 49 with 4, 47 with 6, 45 to 46 with 8 and
// 12, but a decode step 192 with 4, 194 with 6, 199 with 12; 4096 rows over 4096 took 218
// us without, 151 with 4, 158 with 6, 169 with 12.)
constexpr int kExtraFew = 6, kExtraMany = 5;

// Requests of up to kQrRows query rows a KV head and larger ones are taken by a kernel
// each; how many of either there are is known on the device only, so a call that may
// have both launches both.
template <int HD, bool BF16>
cudaError_t launch(const QrArgs &call, const WsLayout &ws, void *workspace, cudaStream_t st) {
    char *w = static_cast<char *>(workspace);
    QrJoin j;
    std::memset(&j, 0, sizeof(j));
    const bool many = int64_t(call.n_tokens) * call.group > kQrRows;
    // Eight columns where one token for each request is what there is, as in a decode
    // step; a request with more rows is then two items that read its K and V twice.
    const bool eight = call.group <= 8 && call.n_tokens <= call.n_seq;
    for (int i = 0; i < (many ? 2 : 1); ++i) {
        QrArgs &a = i == 0 ? j.few : j.many;
        a = call;
        a.cut = reinterpret_cast<QrCut *>(w + ws.cut[i]);
        a.part_ml = reinterpret_cast<float2 *>(w + ws.ml[i]);
        a.part_o = reinterpret_cast<float *>(w + ws.o[i]);
        a.part_rows = i == 0 ? kQrRows : piece_rows(call.n_tokens, call.group);
        a.run = i == 0 ? (eight ? 8 : kQrRows) / call.group : 2 * (kQrTile / call.group);
        a.extra = i == 0 ? kExtraFew : kExtraMany;
        a.more = i == 0 ? 0 : kQrRows;
        a.most = i == 0 ? kQrRows : INT64_MAX;
    }
    cudaError_t e = eight ? launch_qr<HD, BF16, 8>(j.few, st) : launch_qr<HD, BF16, 16>(j.few, st);
    if (e == cudaSuccess && many) {
        e = launch_qp<HD, BF16>(j.many, st);
        j.wide = int32_t(ceil_div(j.many.part_rows, 32));
    }
    return e == cudaSuccess ? launch_qr_join<HD, BF16>(j, st) : e;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status paged_attention_q8_workspace_bytes(int64_t n_tokens, int32_t n_q, int32_t n_kv, int32_t head_dim,
                                                         int64_t *bytes_out) {
    if (bytes_out == nullptr || !shape_ok(n_tokens, n_q, n_kv, head_dim)) return KVD_EINVAL;
    *bytes_out = ws_layout(n_tokens, n_q / n_kv, head_dim).total;
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
    const WsLayout ws = ws_layout(n_tokens, n_q / n_kv, head_dim);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < ws.total) return KVD_EINVAL;
    QrArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t pool_rows = n_pages * page_size * n_kv;
    if (!encode(&a.k, k_pages, head_dim, pool_rows, page_size) || !encode(&a.v, v_pages, head_dim, pool_rows, page_size)) return KVD_EINVAL;
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
    a.max_pages = max_pages;
    a.n_pages = int32_t(n_pages);
    a.page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    a.pool_rows = int32_t(pool_rows);
    const int64_t armed = paged_give_up();
    a.give_up = armed < 0 ? -1 : int32_t(armed >> 32);
    a.give_up_ns = uint32_t(armed);
    // A cap that q.k would have to pass 10^15 to feel is none.  The kernels' factor holds
    // the page's and the row's powers of two, too: with caps up to 16-bit pages' limit (10^34)
    // it fell below the normal numbers of f32 and took the scores' last bits with it.
    const bool cap = softcap > 0.0f && scale / softcap >= 5.421010862427522e-20f;  // 2^-64
    a.mul = cap ? float(2.0 * 1.4426950408889634 * double(scale) / softcap) : scale * log2e;
    a.cap = cap ? softcap * log2e : 0.0f;
    const bool bf16 = dtype == KVD_T_BF16;
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = head_dim == 64 ? (bf16 ? launch<64, true>(a, ws, workspace, st) : launch<64, false>(a, ws, workspace, st))
                                         : (bf16 ? launch<128, true>(a, ws, workspace, st) : launch<128, false>(a, ws, workspace, st));
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}
