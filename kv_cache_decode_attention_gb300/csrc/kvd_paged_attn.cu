// kvd_paged_attn.cu -- the entry points of paged_attention: checks, tensor
// maps, workspace and launches.  Kernels: kvd_paged_attn.cuh, compiled per head
// size in kvd_paged_attn64.cu and kvd_paged_attn128.cu.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "kvd_paged_attn.cuh"
#include "kvd_views.h"

namespace kvd {

cudaError_t launch_paged_attention_64(const PaArgs &a, bool bf16, bool cap, cudaStream_t st);
cudaError_t launch_paged_attention_128(const PaArgs &a, bool bf16, bool cap, cudaStream_t st);

namespace {

std::atomic<int64_t> g_give_up{-1};  // kvd_test_give_up: CTA << 32 | ns

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

bool encode(CUtensorMap *m, bool bf16, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn != nullptr &&
           fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void *>(base),
              dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool pow2_page(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }

// Rows of one piece in the workspace.
int32_t piece_rows(int64_t n_tokens, int32_t group) {
    const int32_t tile_tok = kPaTile / group;
    return n_tokens > tile_tok ? kPaMaxRows : int32_t(round_up(n_tokens * group, 8));
}

struct WsLayout {
    int64_t tickets, cut, ml, o, total;
};
WsLayout ws_layout(int64_t n_tokens, int32_t group, int32_t hd) {
    WsLayout w;
    const int64_t rows = int64_t(2) * kPaCtas * piece_rows(n_tokens, group);
    w.tickets = 0;
    w.cut = round_up(int64_t(kPaCtas) * 8, 256);
    w.ml = w.cut + round_up(int64_t(kPaCtas) * int64_t(sizeof(PaPiecesOf)), 256);
    w.o = w.ml + round_up(rows * 8, 256);
    w.total = w.o + rows * hd * 4;
    return w;
}

bool shape_ok(int64_t n_tokens, int32_t n_q, int32_t n_kv, int32_t hd) {
    return n_tokens >= 0 && n_tokens <= (int64_t(1) << 30) && n_kv >= 1 && n_kv <= 1024 && n_q >= n_kv &&
           n_q % n_kv == 0 && n_q / n_kv <= kMaxHpk && (hd == 64 || hd == 128);
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

// The capped score softcap tanh(y), y = score scale / softcap, in log2 units as a
// polynomial of the raw score.  Masked scores of such a tile become -10^4 cap_near,
// y = -5000, where the last term, softcap 0.017 y^9, leads by far and gives a
// weight of zero.  That holds only where f32 has every coefficient to full
// precision (one that fell to zero would leave the lead to one of the other sign)
// and the cap itself is no speck; a call without goes through pa_tanh throughout.
void set_cap(PaArgs *a, float scale, float softcap) {
    const double log2e = 1.4426950408889634, k = double(scale) / softcap;
    a->cap_in = float(2.0 * log2e * k);
    a->cap_mul = float(scale * log2e);
    bool whole = softcap >= 1e-20f;
    double power = scale * log2e;
    for (int i = 0; i < 4; ++i) {
        const double c = kPaTanh[i] * (power *= k * k);
        whole = whole && std::fabs(c) >= FLT_MIN && std::fabs(c) <= FLT_MAX;
        a->cap_c[i] = whole ? float(c) : 0.0f;
    }
    a->cap_near = whole ? float(0.5 / k) : -1.0f;
    a->cap_hidden = whole ? -1e4f * a->cap_near : -INFINITY;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status paged_attention_workspace_bytes(int64_t n_tokens, int32_t n_q, int32_t n_kv, int32_t head_dim,
                                                      int64_t *bytes_out) {
    if (bytes_out == nullptr || !shape_ok(n_tokens, n_q, n_kv, head_dim)) return KVD_EINVAL;
    *bytes_out = ws_layout(n_tokens, n_q / n_kv, head_dim).total;
    return KVD_OK;
}

extern "C" kvd_status paged_attention(const kvd_rows *q, const kvd_rows *out, int64_t n_tokens, int32_t n_q, int32_t n_kv,
                                      int32_t head_dim, int32_t dtype, const void *k_pages, const void *v_pages,
                                      int64_t n_pages, int32_t page_size, const int32_t *block_table, int32_t max_pages,
                                      const int32_t *cu_new, const int32_t *seq_len, int32_t n_seq, float scale,
                                      int64_t window, float softcap, const float *sinks, void *workspace,
                                      int64_t workspace_bytes, uint32_t *err, void *stream) {
    KVD_NVTX_RANGE("paged_attention");
    if (!shape_ok(n_tokens, n_q, n_kv, head_dim) || (dtype != KVD_T_F16 && dtype != KVD_T_BF16)) return KVD_EINVAL;
    if (!view_ok(q, n_tokens, n_q) || !view_ok(out, n_tokens, n_q)) return KVD_EINVAL;
    if (k_pages == nullptr || v_pages == nullptr ||
        ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15) != 0)
        return KVD_EINVAL;
    if (!pow2_page(page_size) || n_pages < 1 || n_pages * page_size >= (int64_t(1) << 31) ||
        n_pages >= (int64_t(1) << 31) || n_pages * page_size * n_kv >= (int64_t(1) << 31))
        return KVD_EINVAL;
    if (block_table == nullptr || cu_new == nullptr || seq_len == nullptr || err == nullptr || n_seq < 1 || n_seq > kPaMaxSeq || max_pages < 1 ||
        int64_t(max_pages) * page_size > (int64_t(1) << 31) - 1024)
        return KVD_EINVAL;
    if (!std::isfinite(scale) || scale <= 0.0f || window < 0 || !std::isfinite(softcap) || softcap < 0.0f) return KVD_EINVAL;
    const float log2e = 1.4426950408889634f;
    if (!std::isfinite(scale * log2e) || (softcap > 0.0f && (!std::isfinite(softcap * log2e) || !std::isfinite(2.0f * scale * log2e / softcap))))
        return KVD_EINVAL;
    if (sinks != nullptr && (reinterpret_cast<uintptr_t>(sinks) & 3) != 0) return KVD_EINVAL;
    const int32_t group = n_q / n_kv;
    const WsLayout ws = ws_layout(n_tokens, group, head_dim);
    if (n_tokens == 0) return KVD_OK;
    {
        const View o = make_view(out->data, out->token_stride, out->head_stride, n_tokens, n_q, head_dim, 2);
        const int64_t pages = n_pages * page_size * n_kv * head_dim * 2;
        if (!rows_apart(o) || !views_apart(o, make_view(q->data, q->token_stride, q->head_stride, n_tokens, n_q, head_dim, 2)) ||
            !views_apart(o, make_range(k_pages, pages)) || !views_apart(o, make_range(v_pages, pages)))
            return KVD_EINVAL;
    }
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < ws.total)
        return KVD_EINVAL;

    PaArgs a;
    std::memset(&a, 0, sizeof(a));
    const bool bf16 = dtype == KVD_T_BF16;
    a.tile_tok = kPaTile / group;
    {
        const cuuint64_t dims[4] = {cuuint64_t(head_dim), cuuint64_t(group), cuuint64_t(n_kv), cuuint64_t(n_tokens)};
        // strides of axes that have one entry are never used; give them a legal value
        const int64_t hs = n_q > 1 ? q->head_stride : head_dim, ts = n_tokens > 1 ? q->token_stride : hs * n_q;
        const cuuint64_t strides[3] = {cuuint64_t(hs) * 2, cuuint64_t(hs) * 2 * group, cuuint64_t(ts) * 2};
        const cuuint32_t box[4] = {64, cuuint32_t(group), 1, cuuint32_t(a.tile_tok)};
        if (!encode(&a.q, bf16, 4, q->data, dims, strides, box)) return KVD_EINVAL;
        const cuuint64_t kdims[2] = {cuuint64_t(head_dim), cuuint64_t(n_pages * page_size * n_kv)};
        const cuuint64_t kstrides[1] = {cuuint64_t(head_dim) * 2};
        const cuuint32_t kbox[2] = {64, cuuint32_t(page_size)};
        if (!encode(&a.k, bf16, 2, k_pages, kdims, kstrides, kbox) || !encode(&a.v, bf16, 2, v_pages, kdims, kstrides, kbox))
            return KVD_EINVAL;
    }
    char *w = static_cast<char *>(workspace);
    a.cut = reinterpret_cast<PaPiecesOf *>(w + ws.cut);
    a.join_here = n_tokens * group <= kPaJoinRows ? 1 : 0;
    const int64_t armed = g_give_up.load(std::memory_order_relaxed);
    a.give_up = armed < 0 ? -1 : int32_t(armed >> 32);
    a.give_up_ns = uint32_t(armed);
    a.tickets = reinterpret_cast<uint64_t *>(w + ws.tickets);
    static std::atomic<uint64_t> launches{0x9e3779b97f4a7cull};  // any start will do; 2^56 launches wrap
    a.nonce = launches.fetch_add(1, std::memory_order_relaxed) & ((uint64_t(1) << 56) - 1);
    a.part_ml = reinterpret_cast<float2 *>(w + ws.ml);
    a.part_o = reinterpret_cast<float *>(w + ws.o);
    a.part_rows = piece_rows(n_tokens, group);
    a.block_table = block_table;
    a.cu_new = cu_new;
    a.seq_len = seq_len;
    a.out = out->data;
    a.out_tok = out->token_stride;
    a.out_head = out->head_stride;
    a.sinks = sinks;
    a.err = err;
    // every position is below 2^31, so a window from there on hides nothing; as it
    // stands it would leave the 64-bit range below a negative position
    a.window = window < (int64_t(1) << 31) ? window : 0;
    a.n_seq = n_seq;
    a.n_tokens = int32_t(n_tokens);
    a.n_kv = n_kv;
    a.group = group;
    a.max_pages = max_pages;
    a.n_pages = int32_t(n_pages);
    a.page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    a.pool_rows = int32_t(n_pages * page_size * n_kv);
    // A cap so far above the scale that their quotient is no normal number (a raw
    // score would have to pass 10^34 to feel it) is none.
    const bool cap = softcap > 0.0f && scale / softcap >= FLT_MIN;
    a.scale_log2 = (cap ? softcap : scale) * log2e;
    if (cap) set_cap(&a, scale, softcap);
    const cudaError_t e = head_dim == 64 ? launch_paged_attention_64(a, bf16, cap, as_stream(stream))
                                         : launch_paged_attention_128(a, bf16, cap, as_stream(stream));
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}

extern "C" kvd_status kvd_test_give_up(int32_t cta, int64_t after_ns) {
    if (cta >= kPaCtas || after_ns < 0 || after_ns > 1000000000) return KVD_EINVAL;
    g_give_up.store(cta < 0 ? -1 : int64_t(cta) << 32 | after_ns);
    return KVD_OK;
}
