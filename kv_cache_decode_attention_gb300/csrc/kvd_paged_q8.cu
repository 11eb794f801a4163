// kvd_paged_q8.cu -- pages of 8-bit codes: rows quantised as they are written, and
// rows of pages read back.
//
// A block is one page of one KV head, of K or of V; it has e4m3 codes and one f32
// scale s, and stands for code * s.  The writer keeps s a power of two, the smallest
// with |x| <= 448 s for every row the block has taken since its row 0 was written:
//   x / s is exact, so a code is one rounding of x;
//   when a later row needs a larger s, the codes that stand move by a power of two,
//   which is exact for all that stay normal numbers of e4m3 (those that fall below
//   2^-6 s are rounded once more, to a multiple of 2^-9 s).
// What the power of two gives away is less than one of e4m3's 18 binades, no
// precision.  (With s = max|x| / 448 every growth would round every code anew.)
//
// Writing.  The rows of one page stand together in the packed batch, so a CTA takes
// the runs of rows that begin among its 16 tokens, for some heads of K or V: one
// pass over the rows for the largest value of each run and head, then the scales and
// the codes already there, then a second pass that writes the codes.  Nobody waits
// for another CTA, because a block's rows all lie in one.  The second pass finds its
// rows in L1 or L2.

#include <cfloat>
#include <cmath>

#include "kvd_q8.cuh"
#include "kvd_rope.cuh"

namespace kvd {
namespace {

constexpr int kStoreTok = 16;     // tokens whose runs a CTA takes
constexpr int kMaxPage = 128;
constexpr int kStoreHeads = 8;    // heads of one CTA at most

struct StoreArgs {
    RopeArgs r;               // g[1], g[2]: k and v with their pages
    float *scale[2];          // of K and V: [n_pages][n_kv]
    int32_t heads;            // of one CTA
};

// The smallest power of two s with top <= 448 s, within the limits: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = int(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
    return e <= 127 - 64 ? kScaleLow : e >= 127 + 64 ? kScaleHigh : __uint_as_float(uint32_t(e) << 23);
}
__device__ __forceinline__ bool pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// Runs of rows in one page that begin among the CTA's tokens.
struct Runs {
    int32_t slot[kStoreTok + kMaxPage];    // of token t0 + i, -1 = none
    int8_t run[kStoreTok + kMaxPage];      // -1: no row of this CTA's
    int32_t page[kStoreTok], row0[kStoreTok];
    int32_t end, n;
    uint32_t top[kStoreTok][kStoreHeads];  // largest finite |x|, as bits
    float scale[kStoreTok][kStoreHeads], ratio[kStoreTok][kStoreHeads];
};

__device__ __forceinline__ void find_runs(const RopeArgs &a, Runs &s, int64_t t0, bool report) {
    const int size = 1 << a.page_log2, span = kStoreTok + size;
    for (int i = threadIdx.x; i < span; i += blockDim.x) {
        const int64_t t = t0 + i;
        int32_t slot = t < a.n_tokens ? a.slots[t] : -1;
        if (slot >= a.n_slots) {
            if (report) set_error(a.err, kErrBounds);
            slot = -1;
        }
        s.slot[i] = slot < 0 ? -1 : slot;
        s.run[i] = -1;
    }
    for (int i = threadIdx.x; i < kStoreTok * kStoreHeads; i += blockDim.x) s.top[i / kStoreHeads][i % kStoreHeads] = 0;
    if (threadIdx.x == 0) s.end = span;
    __syncthreads();
    // a row that goes on where the one before it stands, in the same page
    auto goes_on = [&](int i) {
        const int32_t slot = s.slot[i];
        const int32_t last = i > 0 ? s.slot[i - 1] : t0 > 0 ? a.slots[t0 - 1] : -1;
        return slot >= 0 && last >= 0 && slot == last + 1 && (slot & (size - 1)) != 0;
    };
    for (int i = kStoreTok + int(threadIdx.x); i < span; i += blockDim.x)
        if (!goes_on(i)) atomicMin(&s.end, i);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int i = threadIdx.x;
        const bool there = i < kStoreTok && s.slot[i] >= 0, lead = there && !goes_on(i);
        const uint32_t leads = __ballot_sync(~0u, lead), upto = leads & (~0u >> (31 - i));
        const int run = __popc(upto) - 1;
        if (there && run >= 0) s.run[i] = int8_t(run);
        if (lead) {
            s.page[run] = s.slot[i] >> a.page_log2;
            s.row0[run] = s.slot[i] & (size - 1);
        }
        if (i == 0) s.n = __popc(leads);
    }
    __syncthreads();
    // rows past the sixteenth token belong to the run that its row is in
    const int8_t last = s.run[kStoreTok - 1];
    for (int i = kStoreTok + int(threadIdx.x); i < s.end; i += blockDim.x) s.run[i] = last;
    __syncthreads();
}

// The 16 channels of a row that a thread owns, rotated.  HALF: eight and their
// eight partners where they turn; else 16 neighbours.
template <typename TI, bool HALF, bool ANY>
struct Row16 {
    float c[ANY ? 16 : 8], s[ANY ? 16 : 8];
    int at0, at1;
    bool turn;

    __device__ __forceinline__ void place(const RopeArgs &a, int task) {
        turn = ANY ? task * 16 < 2 * a.pairs : task < a.n_pairs_task;
        at0 = !ANY && HALF && turn ? task * 8 : task * 16;
        at1 = !ANY && HALF && turn ? a.half + task * 8 : task * 16 + 8;
    }
    __device__ __forceinline__ void angles(const RopeArgs &a, int task, int64_t tok) {
        if (!turn) return;
        const uint64_t *turns = a.turns;
        asm volatile("" : "+l"(turns));  // an ordinary load, as fill_angles explains
        const int32_t pos = a.positions[tok];
#pragma unroll
        for (int i = 0; i < (ANY ? 16 : 8); ++i) {
            c[i] = a.factor;
            s[i] = 0.0f;
            int p = task * 8 + i;
            if (ANY) {
                const int ch = task * 16 + i;
                if (ch >= 2 * a.pairs) continue;
                p = HALF ? (ch < a.pairs ? ch : ch - a.pairs) : ch / 2;
            }
            if (pos >= 0) {
                float sn, cs;
                sincospif(float(int32_t((uint64_t(pos) * turns[p]) >> 32)) * 4.656612873077393e-10f, &sn, &cs);
                c[i] = cs * a.factor;
                s[i] = sn * a.factor;
            }
        }
    }
    __device__ __forceinline__ void load(const RopeArgs &a, const TI *in, int task, bool rotate, float *x) const {
        if constexpr (ANY) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int ch = task * 16 + i;
                x[i] = to_f32<TI>(in[ch]);
                if (!rotate || ch >= 2 * a.pairs) continue;
                const bool low = HALF ? ch < a.pairs : ch % 2 == 0;
                const float y = to_f32<TI>(in[HALF ? (low ? ch + a.pairs : ch - a.pairs) : ch ^ 1]);
                x[i] = low ? x[i] * c[i] - y * s[i] : x[i] * c[i] + y * s[i];
            }
        } else {
            load8<TI>(in + at0, x);
            load8<TI>(in + at1, x + 8);
            if (!rotate || !turn) return;
            if (HALF) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x[i] * c[i] - x[8 + i] * s[i], w = x[8 + i] * c[i] + x[i] * s[i];
                    x[i] = u;
                    x[8 + i] = w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
                    x[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
                    x[2 * i] = u;
                }
            }
        }
    }
};

template <typename TI, bool HALF, bool ANY>
__global__ void __launch_bounds__(256) store_kernel(const __grid_constant__ StoreArgs args) {
    __shared__ Runs sh;
    const RopeArgs &a = args.r;
    pdl_wait();
    const int64_t t0 = int64_t(blockIdx.x) * kStoreTok;
    const int kind = blockIdx.z, h0 = blockIdx.y * args.heads;
    const int heads = a.n_kv - h0 < args.heads ? a.n_kv - h0 : args.heads;
    const Group &g = a.g[1 + kind];
    const bool rotate = kind == 0 && a.pairs > 0;
    find_runs(a, sh, t0, blockIdx.y == 0 && kind == 0);
    if (sh.n == 0) return;
    const int size = 1 << a.page_log2;
    const int task = threadIdx.x % a.n_tasks, lane = threadIdx.x / a.n_tasks, lanes = blockDim.x / a.n_tasks;
    Row16<TI, HALF, ANY> row;
    row.place(a, task);

    // the largest value of each run and head
    for (int i0 = 0; i0 < sh.end; i0 += lanes) {
        const int i = i0 + lane;
        const int run = i < sh.end ? sh.run[i] : -1;
        if (run >= 0 && rotate) row.angles(a, task, t0 + i);
        for (int h = 0; h < heads; ++h) {
            float top = 0.0f;
            if (run >= 0) {
                float x[16];
                row.load(a, static_cast<const TI *>(g.in) + (t0 + i) * g.in_tok + (h0 + h) * g.in_head, task, rotate, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float v = fabsf(x[e]);
                    top = v <= FLT_MAX ? fmaxf(top, v) : top;
                }
            }
            for (int d = 1; d < a.n_tasks; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            if (run >= 0 && task == 0) atomicMax(&sh.top[run][h], __float_as_uint(top));
        }
    }
    __syncthreads();

    // the scales, which only grow while a block keeps rows
    for (int i = threadIdx.x; i < sh.n * heads; i += blockDim.x) {
        const int run = i / heads, h = i - run * heads;
        float *at = args.scale[kind] + int64_t(sh.page[run]) * a.n_kv + h0 + h;
        float s = scale_for(__uint_as_float(sh.top[run][h])), ratio = 1.0f;
        if (sh.row0[run] > 0) {
            const float old = *at;
            if (!scale_ok(old)) set_error(a.err, kErrBounds);
            else if (old >= s) s = old;
            else ratio = old / s;
        }
        *at = s;
        sh.scale[run][h] = s;
        sh.ratio[run][h] = ratio;
    }
    __syncthreads();

    uint8_t *pages = static_cast<uint8_t *>(g.out);
    auto block_of = [&](int run, int h) { return pages + ((int64_t(sh.page[run]) * a.n_kv + h0 + h) << a.page_log2) * a.hd; };
    // codes that stand before a run move to the new scale
    for (int run = 0; run < sh.n; ++run) {
        if (sh.row0[run] == 0) continue;
        for (int h = 0; h < heads; ++h) {
            const float ratio = sh.ratio[run][h];
            if (ratio == 1.0f) continue;
            uint4 *p = reinterpret_cast<uint4 *>(block_of(run, h));
            for (int i = threadIdx.x; i < sh.row0[run] * a.hd / 16; i += blockDim.x) {
                uint4 v = p[i];
                uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[4];
                    values4(w[e], x);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] *= ratio;
                    w[e] = codes4(x);
                }
                p[i] = v;
            }
        }
    }

    // the codes
    for (int i0 = 0; i0 < sh.end; i0 += lanes) {
        const int i = i0 + lane;
        const int run = i < sh.end ? sh.run[i] : -1;
        if (run < 0) continue;
        if (rotate) row.angles(a, task, t0 + i);
        for (int h = 0; h < heads; ++h) {
            float x[16];
            row.load(a, static_cast<const TI *>(g.in) + (t0 + i) * g.in_tok + (h0 + h) * g.in_head, task, rotate, x);
            const float s = sh.scale[run][h], inv = 1.0f / s;  // exact for a power of two
            const bool exact = pow2(s);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = exact ? x[e] * inv : x[e] / s;
            uint8_t *out = block_of(run, h) + (sh.slot[i] & (size - 1)) * a.hd;
            if (row.at1 == row.at0 + 8) {
                *reinterpret_cast<uint4 *>(out + row.at0) = make_uint4(codes4(x), codes4(x + 4), codes4(x + 8), codes4(x + 12));
            } else {
                *reinterpret_cast<uint2 *>(out + row.at0) = make_uint2(codes4(x), codes4(x + 4));
                *reinterpret_cast<uint2 *>(out + row.at1) = make_uint2(codes4(x + 8), codes4(x + 12));
            }
        }
    }
}

template <typename TI>
cudaError_t launch_store(StoreArgs &a, bool aligned, int layout, cudaStream_t st) {
    const bool any = !aligned || a.r.pairs % 8 != 0, half = layout == KVD_ROPE_HALF;
    // One head to a CTA while that leaves no more CTAs than the SMs hold at once;
    // two share the angles of a long prompt's rows.
    a.heads = ceil_div(a.r.n_tokens, kStoreTok) * a.r.n_kv <= 152 * 8 ? 1 : 2;
    const dim3 grid(unsigned(ceil_div(a.r.n_tokens, kStoreTok)), unsigned(ceil_div(a.r.n_kv, a.heads)), 2);
    const auto kern = any ? (half ? store_kernel<TI, true, true> : store_kernel<TI, false, true>)
                          : (half ? store_kernel<TI, true, false> : store_kernel<TI, false, false>);
    return launch_pdl(kern, grid, dim3(256), 0, st, a);
}

// ---------------------------------------------------------------- reading back

struct ReadArgs {
    const void *pages[2];
    const float *scale[2];
    void *out[2];
    int64_t out_tok[2], out_head[2];  // strides in elements
    const int32_t *block_table, *seq_len, *start, *cu_rows;
    uint32_t *err;
    int64_t n_rows, n_pages;
    int32_t n_seq, max_pages, page_log2, n_kv, hd;
};

constexpr int kReadRows = 32;  // rows of one CTA

// Where output row t comes from: its page and row there; page -1 = nothing stands
// there (zeros), -2 = no request asked for it (left alone).
__device__ __forceinline__ int2 read_place(const ReadArgs &a, int64_t t) {
    if (t >= a.n_rows || t < a.cu_rows[0] || t >= a.cu_rows[a.n_seq]) return make_int2(-2, 0);
    int lo = 0, hi = a.n_seq;  // cu_rows[lo] <= t < cu_rows[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.cu_rows[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int64_t pos = (a.start != nullptr ? int64_t(a.start[lo]) : 0) + t - a.cu_rows[lo];
    const int64_t p = pos >> a.page_log2;
    int32_t page = -1;
    if (pos >= 0 && pos < a.seq_len[lo] && p < a.max_pages) page = a.block_table[int64_t(lo) * a.max_pages + p];
    if (page < 0 || page >= a.n_pages) {
        set_error(a.err, kErrBounds);
        page = -1;
    }
    return make_int2(page, int32_t(pos & ((1 << a.page_log2) - 1)));
}

template <typename TP, typename TO>  // TP uint8_t: e4m3 codes with scales
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadArgs a) {
    __shared__ int2 place[kReadRows];
    pdl_wait();
    const int64_t t0 = int64_t(blockIdx.x) * kReadRows;
    if (threadIdx.x < kReadRows) place[threadIdx.x] = read_place(a, t0 + threadIdx.x);
    __syncthreads();
    const int chunks = a.hd / 16, per_head = kReadRows * chunks, h0 = blockIdx.y;
#pragma unroll 2
    for (int i = threadIdx.x; i < per_head * 2; i += blockDim.x) {
        const int kind = i / per_head, r = (i - kind * per_head) / chunks, at = (i % chunks) * 16;
        const int2 from = place[r];
        if (from.x == -2) continue;
        float x[16];
        if (from.x < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.0f;
        } else {
            const int64_t block = int64_t(from.x) * a.n_kv + h0;
            const TP *in = static_cast<const TP *>(a.pages[kind]) + ((block << a.page_log2) + from.y) * a.hd + at;
            if constexpr (sizeof(TP) == 1) {
                const uint4 v = *reinterpret_cast<const uint4 *>(in);
                const float s = scale_of(a.scale[kind][block], a.err);
                values4(v.x, x);
                values4(v.y, x + 4);
                values4(v.z, x + 8);
                values4(v.w, x + 12);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= s;
            } else {
                load8<TP>(in, x);
                load8<TP>(in + 8, x + 8);
            }
        }
        TO *out = static_cast<TO *>(a.out[kind]) + (t0 + r) * a.out_tok[kind] + int64_t(h0) * a.out_head[kind] + at;
        store8<TO>(out, x);
        store8<TO>(out + 8, x + 8);
    }
}

template <typename TP>
cudaError_t launch_read(const ReadArgs &a, int32_t out_dtype, cudaStream_t st) {
    const dim3 grid(unsigned(ceil_div(a.n_rows, kReadRows)), unsigned(a.n_kv));
    const auto kern = out_dtype == KVD_T_F32   ? read_kernel<TP, float>
                      : out_dtype == KVD_T_F16 ? read_kernel<TP, __half>
                                               : read_kernel<TP, __nv_bfloat16>;
    return launch_pdl(kern, grid, dim3(256), 0, st, a);
}

bool page_ok(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }
int32_t log2_of(int32_t p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }
bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kv_paged_append_q8(const kvd_rope *R, const kvd_rows *q, const kvd_rows *q_out, int32_t n_q,
                                         const kvd_rows *k, const kvd_rows *v, int32_t n_kv, int32_t head_dim,
                                         int32_t in_dtype, int32_t q_dtype, const int32_t *positions, const int32_t *slots,
                                         int64_t n_tokens, void *k_pages, void *v_pages, float *k_scale, float *v_scale,
                                         int64_t n_pages, int32_t page_size, uint32_t *err, void *stream) {
    KVD_NVTX_RANGE("kv_paged_append_q8");
    const Rope *r = checked_rope(R);
    const int ib = dtype_bytes(in_dtype), qb = dtype_bytes(q_dtype);
    if ((R != nullptr && r == nullptr) || ib == 0) return KVD_EINVAL;
    if (head_dim != 64 && head_dim != 128) return KVD_EINVAL;
    if (r != nullptr && r->rot_dim > head_dim) return KVD_EINVAL;
    if (!page_ok(page_size) || n_pages < 1 || n_pages >= (int64_t(1) << 31) || n_pages * page_size >= (int64_t(1) << 31)) return KVD_EINVAL;
    if (n_tokens < 0 || n_tokens > kMaxTokens || n_kv < 1 || n_kv > 1024) return KVD_EINVAL;
    if ((n_tokens > 0 && (positions == nullptr || slots == nullptr)) || err == nullptr || (q == nullptr) != (q_out == nullptr)) return KVD_EINVAL;
    if (k_pages == nullptr || v_pages == nullptr || !aligned_to(k_pages, 16) || !aligned_to(v_pages, 16)) return KVD_EINVAL;
    if (k_scale == nullptr || v_scale == nullptr || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4)) return KVD_EINVAL;
    if (!rows_ok(k, n_tokens, n_kv, ib) || !rows_ok(v, n_tokens, n_kv, ib)) return KVD_EINVAL;
    StoreArgs a;
    std::memset(&a, 0, sizeof(a));
    RopeArgs turn;
    std::memset(&turn, 0, sizeof(turn));
    if (q != nullptr) {
        if (qb != 2 || (in_dtype != KVD_T_F32 && in_dtype != q_dtype)) return KVD_EINVAL;
        if (n_q < 1 || n_q > 1024 || !rows_ok(q, n_tokens, n_q, ib) || !rows_ok(q_out, n_tokens, n_q, qb)) return KVD_EINVAL;
        turn.g[0] = group_of(q, q_out, n_q);
    }
    const kvd_rows kp = {k_pages, 0, 0}, vp = {v_pages, 0, 0};
    a.r.g[1] = group_of(k, &kp, n_kv);
    a.r.g[2] = group_of(v, &vp, n_kv);
    const bool aligned = aligned16(a.r.g[1], true, ib, 1) && aligned16(a.r.g[2], true, ib, 1);
    if (n_tokens == 0) return KVD_OK;
    {
        // q turns in place; else what is written shares memory with nothing else
        const int64_t pages = n_pages * page_size * n_kv * head_dim, scales = n_pages * n_kv * 4;
        const View in[2] = {view_of(k, n_tokens, n_kv, head_dim, ib), view_of(v, n_tokens, n_kv, head_dim, ib)};
        const View out[4] = {make_range(k_pages, pages), make_range(v_pages, pages), make_range(k_scale, scales), make_range(v_scale, scales)};
        bool ok = true;
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < i; ++j) ok = ok && views_apart(out[i], out[j]);
            for (const View &x : in) ok = ok && views_apart(out[i], x);
        }
        if (q != nullptr) {
            const View vq = view_of(q, n_tokens, n_q, head_dim, ib), vo = view_of(q_out, n_tokens, n_q, head_dim, qb);
            ok = ok && rows_apart(vo) && (same_rows(vq, vo) || views_apart(vq, vo)) && views_apart(vo, in[0]) && views_apart(vo, in[1]);
            for (const View &x : out) ok = ok && views_apart(x, vq) && views_apart(x, vo);
        }
        if (!ok) return KVD_EINVAL;
    }
    const int layout = r != nullptr ? r->layout : KVD_ROPE_HALF;
    cudaStream_t st = as_stream(stream);
    cudaError_t e = cudaSuccess;
    if (q != nullptr) {
        set_rope(&turn, r, head_dim);
        turn.positions = positions;
        turn.n_tokens = n_tokens;
        e = rotate_rows(turn, layout, in_dtype, q_dtype, st);
        if (e != cudaSuccess) return KVD_ECUDA;
    }
    set_rope(&a.r, r, head_dim);
    a.r.paged = 1;
    a.r.n_kv = n_kv;
    a.r.page_log2 = log2_of(page_size);
    a.r.n_slots = n_pages * page_size;
    a.r.positions = positions;
    a.r.slots = slots;
    a.r.n_tokens = n_tokens;
    a.r.err = err;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    e = in_dtype == KVD_T_F32   ? launch_store<float>(a, aligned, layout, st)
        : in_dtype == KVD_T_F16 ? launch_store<__half>(a, aligned, layout, st)
                                : launch_store<__nv_bfloat16>(a, aligned, layout, st);
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}

extern "C" kvd_status kv_paged_read(const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                                    int32_t page_dtype, int64_t n_pages, int32_t page_size, int32_t n_kv, int32_t head_dim,
                                    const int32_t *block_table, int32_t max_pages, const int32_t *seq_len, const int32_t *start,
                                    const int32_t *cu_rows, int32_t n_seq, const kvd_rows *k_out, const kvd_rows *v_out,
                                    int32_t out_dtype, int64_t n_rows, uint32_t *err, void *stream) {
    KVD_NVTX_RANGE("kv_paged_read");
    const int ob = dtype_bytes(out_dtype), pb = page_dtype == KVD_T_E4M3 ? 1 : page_dtype == KVD_T_F32 ? 0 : dtype_bytes(page_dtype);
    if (ob == 0 || pb == 0 || (head_dim != 64 && head_dim != 128) || n_kv < 1 || n_kv > 1024) return KVD_EINVAL;
    if (!page_ok(page_size) || n_pages < 1 || n_pages >= (int64_t(1) << 31) || n_pages * page_size >= (int64_t(1) << 31)) return KVD_EINVAL;
    if (k_pages == nullptr || v_pages == nullptr || !aligned_to(k_pages, 16) || !aligned_to(v_pages, 16)) return KVD_EINVAL;
    if (pb == 1 ? k_scale == nullptr || v_scale == nullptr || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4)
                : k_scale != nullptr || v_scale != nullptr)
        return KVD_EINVAL;
    if (block_table == nullptr || seq_len == nullptr || cu_rows == nullptr || err == nullptr || n_seq < 1 || n_seq > (1 << 20) || max_pages < 1)
        return KVD_EINVAL;
    if (n_rows < 0 || n_rows > kMaxTokens || !rows_ok(k_out, n_rows, n_kv, ob) || !rows_ok(v_out, n_rows, n_kv, ob)) return KVD_EINVAL;
    if (n_rows == 0) return KVD_OK;
    const kvd_rows *out[2] = {k_out, v_out};
    for (const kvd_rows *o : out)
        if (!aligned_to(o->data, 16) || (n_rows > 1 && o->token_stride * ob % 16 != 0) || (n_kv > 1 && o->head_stride * ob % 16 != 0)) return KVD_EINVAL;
    {
        const View vk = view_of(k_out, n_rows, n_kv, head_dim, ob), vv = view_of(v_out, n_rows, n_kv, head_dim, ob);
        const int64_t pages = n_pages * page_size * n_kv * head_dim * pb, scales = n_pages * n_kv * 4;
        bool ok = rows_apart(vk) && rows_apart(vv) && views_apart(vk, vv);
        for (const View &x : {vk, vv}) {
            ok = ok && views_apart(x, make_range(k_pages, pages)) && views_apart(x, make_range(v_pages, pages));
            if (pb == 1) ok = ok && views_apart(x, make_range(k_scale, scales)) && views_apart(x, make_range(v_scale, scales));
        }
        if (!ok) return KVD_EINVAL;
    }
    ReadArgs a;
    std::memset(&a, 0, sizeof(a));
    a.pages[0] = k_pages;
    a.pages[1] = v_pages;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    for (int i = 0; i < 2; ++i) {
        a.out[i] = out[i]->data;
        a.out_tok[i] = out[i]->token_stride;
        a.out_head[i] = out[i]->head_stride;
    }
    a.block_table = block_table;
    a.seq_len = seq_len;
    a.start = start;
    a.cu_rows = cu_rows;
    a.err = err;
    a.n_rows = n_rows;
    a.n_pages = n_pages;
    a.n_seq = n_seq;
    a.max_pages = max_pages;
    a.page_log2 = log2_of(page_size);
    a.n_kv = n_kv;
    a.hd = head_dim;
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = pb == 1                     ? launch_read<uint8_t>(a, out_dtype, st)
                          : page_dtype == KVD_T_F16 ? launch_read<__half>(a, out_dtype, st)
                                                    : launch_read<__nv_bfloat16>(a, out_dtype, st);
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}
