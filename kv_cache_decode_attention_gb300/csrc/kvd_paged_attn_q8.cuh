// kvd_paged_attn_q8.cuh -- attention over pages of e4m3 codes, a few query rows at a
// time, on the fifth-generation tensor cores.
//
// out_t = sum_p softmax_p(scale q_t . k_p) v_p with k_p = c_p s_K(p), v_p = d_p s_V(p):
// codes c, d and one scale for each page of a KV head.  Decode steps and drafts are
// bound by the bytes of K and V, so nothing is made of them but operands: the codes
// go from the TMA's tile straight into the MMAs (kind::f8f6f4), as their M side,
//   S^T [128 rows of K x N] = K Q^T,    O^T [head_dim x N] = V^T P^T,
// and what is not of 8 bits becomes several e4m3 terms beside one another in N, each
// with its own accumulator and so its own scale:
//   q, scaled by a power of two so that its row's largest lies in [128, 256), is
//   t0 + t1 / 16 (+ t2 / 256): eight significant bits for bf16, twelve for f16, down
//   to 2^-21 (2^-25) of the largest;
//   p, a weight with the scale of its V block, relative to the largest of its tile,
//   likewise, by way of f16: rounded by 2^-9 + 2^-11 of it at most for bf16, 2^-11 for f16.
// References are those of weights with their scales, the sum that of weights alone, and a
// weight that is nothing beside another's scale still counts there.  So once a part has met
// a scale of V past kScaleFar its weights are summed from the scores once more, and the
// factor between two references reaches the sum as two halves.
// So S is exact but for its f32 sums, and the weights are rounded to about q's type.
// (Converting the codes to 16 bits instead costs 48 KB of shared-memory traffic a tile of
// 16, which at the rate of HBM leaves no room for the MMAs' own.)
//
// An item is one (request, KV head, run of tokens): kQrRows query rows (token, head of
// the group) at most.  Items are cut into tiles of 128 rows and every CTA gets the
// same number of consecutive ones, however long the requests are; an item that is cut
// leaves its pieces (output, reference, sum) to qr_join_kernel.
//
// A CTA, of which an SM holds three (f16: two, with three stages each):
//   warps 0-3  softmax, a thread per row of K: its scales are the thread's own, masks
//              of single tokens a comparison; and the sum of the O^T over the tiles,
//              a thread per channel, in f32 registers (fresh accumulators each tile:
//              no rescaling in TMEM, a weight's range counts within its tile only);
//   warp 4     walks the work, looks up pages and scales, TMA loads of K and V;
//   warp 5     issues the MMAs: S^T of tile i + 1 before O^T of tile i.
// Barriers, all of one phase a tile (K, V: a ring of kStages): s_full, s_free (S is in
// registers), p_ready (P is in shared memory, O of the tile before in registers),
// o_full.  No warp can be two phases ahead of one that waits: S(i + 1) waits for
// s_free(i), P(i + 1) for o_full(i).  The softmax warps meet once an item, a tile and an
// item's end, and at their end, at a named barrier, whose wait knows no limit.  So all four
// come to every meeting, one whose wait was given up to the rest of its item's without doing
// anything else; it says so at the next item's first, where all leave.
// (tests/test_paged8_protocol_cpu.py has warps and barriers as a model.  Meetings at an
// mbarrier with a bounded wait cost a decode step 2%, 256 requests of 300 rows 10%; a reduction at
// every one of them 0 and 4%.)
//
// Measured (GPU time on one GB300; a copy runs at 6.77 TB/s): one new row for each of 64
// requests of up to 16384 rows, 32 heads over 8, 193 us, 6.1 TB/s, f16 217; 4 of 131072
// rows, 128 heads over 8, 184 to 186 us, 5.8 TB/s; four drafts for each of 32 requests 47 us;
// one row for each of 256 requests of 300 rows 52; one over 1023 rows 11.  With eight
// columns and bf16 a CTA waits for HBM (a tile in 4300 cycles, 2400 of them busy: 6.8 TB/s
// while all CTAs are at it; the rest is the first scores, some 5 us after the launch, the
// ends and the joining launch); with 16 columns in three terms, two CTAs to an SM, it is
// the softmax warps' chain: 3300 cycles a tile, 2700 of them busy.  An item costs some
// 5 us beside its tiles with eight columns and 10 with 16.
// Measured and not taken: 16 columns for single tokens (decode 253 us when eight took
// 211); three CTAs of two stages for 16 bf16 columns (drafts 80 us against 70: registers
// spill; eight columns spill 24 bytes in bf16 and some 145 in f16 for their third CTA); a reduction by instruction for each column's maximum (five instructions more a
// column); joining CTAs of 512 threads (decode 203 against 194); zeros for V's rows before
// a window, as for those behind the last (decode 203 against 193, without any window): rows
// that a request holds have to be finite.
#pragma once

#include <cfloat>

#include "kvd_paged_attn.cuh"
#include "kvd_q8.cuh"
#include "kvd_rope.cuh"

namespace kvd {

constexpr int kQrTile = 128;     // rows of K and V of a tile
constexpr int kQrRows = 16;      // query rows of an item
constexpr int kQrThreads = 192;
constexpr int kQrMaxCtas = 152 * 3;
constexpr int kQrJobs = 4;
// With scales of V up to here (2^8; f16 needs no larger ones) a weight that is lost beside
// another's scale is below 2^-54 of that one's.
constexpr float kScaleFar = 256.0f;

// A cut item as qr_join_kernel finds it; n = 0: none.
struct QrCut {
    int64_t unit0, total;
    int32_t tiles, rows, q_row, kv_head, n, pad;  // unit0: of its first tile
};

struct QrArgs {
    CUtensorMap k, v;
    const void *q;
    void *out;
    int64_t q_tok, q_head, out_tok, out_head;  // strides in elements
    const float *k_scale, *v_scale;
    const int32_t *block_table, *cu_new, *seq_len;
    const float *sinks;
    float *part_o;    // [2 * ctas][part_rows][hd]
    float2 *part_ml;  // [2 * ctas][part_rows]: reference (log2 units), sum
    QrCut *cut;       // [ctas]: the cut item that begins in each CTA
    uint32_t *err;
    int64_t window;   // below 2^31; 0 = none
    int32_t ctas, n_seq, n_tokens, n_kv, group, run, extra, max_pages, n_pages, page_log2, pool_rows;
    int64_t more, most;  // requests with more than `more` and at most `most` query rows a KV head are this launch's
    int32_t part_rows;
    int32_t give_up;  // for tests: the CTA (of qr_kernel every 152nd) whose waits end so many ns after it began, or -1
    uint32_t give_up_ns;
    float mul;        // scale * log2 e; with a cap 2 * scale * log2 e / softcap
    float cap;        // softcap * log2 e, or 0
};

// ---------------------------------------------------------------- tcgen05, 8 bits

__device__ __forceinline__ void tc_ld16(uint32_t addr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tc_mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Instruction descriptor of kind::f8f6f4, e4m3 both: f32 accumulator, M x N, operands MN-major or not.
__host__ __device__ constexpr uint32_t tc_idesc8(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// Shared-memory matrix descriptor; type 2: 128-byte swizzle, 4: 64-byte, 0: none.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t type) {
    return uint64_t((addr & 0x3ffffu) >> 4) | uint64_t(lbo >> 4) << 16 | uint64_t(sbo >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(type) << 61;
}

// ---------------------------------------------------------------- the work

// An item costs its CTA more than its tiles do (q, the first scores, its end): as much
// as `extra` tiles, which the cut counts before them.  A part without a tile of its own
// is none.
struct QrItem {
    int32_t count, first_pos, tile0, tiles, units;
};
__device__ __forceinline__ PaSeq qr_seq(const QrArgs &a, int b, bool report) {
    PaSeq s = {0, 0, 0};
    if (b >= a.n_seq) return s;
    const int32_t q0 = a.cu_new[b], q1 = a.cu_new[b + 1], len = a.seq_len[b];
    if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 || len > (int64_t(a.max_pages) << a.page_log2)) {
        if (report) set_error(a.err, kErrBounds);
        return s;
    }
    const int64_t rows = int64_t(q1 - q0) * a.group;
    if (rows <= a.more || rows > a.most) return s;
    s.q0 = q0;
    s.fresh = q1 - q0;
    s.len = len;
    return s;
}
__device__ __forceinline__ QrItem qr_item(const QrArgs &a, const PaSeq &s, int32_t tok) {
    QrItem it;
    const int32_t left = s.fresh - tok;
    it.count = left < a.run ? left : a.run;
    it.first_pos = s.len - s.fresh + tok;
    int64_t lo = a.window > 0 ? int64_t(it.first_pos) - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    int32_t hi = it.first_pos + it.count;
    if (hi < 0) hi = 0;
    it.tile0 = int32_t(lo) / kQrTile;
    const int32_t n = (hi + kQrTile - 1) / kQrTile - it.tile0;
    it.tiles = n > 1 ? n : 1;
    it.units = it.tiles + a.extra;
    return it;
}
// The next item in the order (request, KV head, token run).
__device__ __forceinline__ void qr_next(const QrArgs &a, PaWalk &w) {
    w.tok += a.run;
    if (w.tok < w.s.fresh) return;
    w.tok = 0;
    if (++w.h < a.n_kv) return;
    w.h = 0;
    do {
        ++w.b;
        w.s = qr_seq(a, w.b, false);
    } while (w.s.fresh == 0 && w.b < a.n_seq);
}

// CTA c takes units [c W / ctas, (c + 1) W / ctas) of the W there are.  All
// threads; the result is in shared memory.  (As pa_cut.)
template <int THREADS>
__device__ __forceinline__ void qr_cut(const QrArgs &a, PaStart *out, int64_t *warp_sums) {
    constexpr int kWarps = THREADS / 32;
    const int per = (a.n_seq + THREADS - 1) / THREADS;
    const int b0 = int(threadIdx.x) * per < a.n_seq ? int(threadIdx.x) * per : a.n_seq;
    const int b1 = b0 + per < a.n_seq ? b0 + per : a.n_seq;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t mine = 0, off = 0, u = 0, from = 0, to = 0;
    uint64_t total = 0;
    PaSeq s = {0, 0, 0};
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        int b = b0;
        if (turn == 0 || per > 1) {  // a thread's only request is still at hand
#pragma unroll 1
            for (; b < b1; ++b) {
                s = qr_seq(a, b, turn == 0 && blockIdx.x == 0);
                u = 0;
#pragma unroll 1
                for (int32_t tok = 0; tok < s.fresh; tok += a.run) u += qr_item(a, s, tok).units;
                if (turn == 0) mine += u * a.n_kv;
                else if (off < u * a.n_kv) break;
                else off -= u * a.n_kv;
            }
        }
        if (turn == 1) {
            int32_t h = 0, tok = 0;
#pragma unroll 1
            for (; off >= u; off -= u) ++h;
#pragma unroll 1
            for (;; tok += a.run) {
                const int32_t n = qr_item(a, s, tok).units;
                if (off < n) break;
                off -= n;
            }
            *out = PaStart{b, h, tok, int32_t(off), s, to - from, from, int64_t(total)};
            break;
        }
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) warp_sums[w] = x;
        if (threadIdx.x == 0) out->units = 0;
        __syncthreads();
        int64_t before = 0;
        total = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            before += i < w ? warp_sums[i] : 0;
            total += uint64_t(warp_sums[i]);
        }
        before += x - mine;
        from = total * blockIdx.x / gridDim.x;
        to = total * (blockIdx.x + 1) / gridDim.x;
        off = from - before;
        if (from >= to || off < 0 || off >= mine) break;
    }
    __syncthreads();
}

// The CTAs that hold pieces of a cut item.  A piece of CTA c is kept in slot 2 c + 1 if
// it begins its item, else in slot 2 c.
static __device__ __forceinline__ int32_t qr_cta_of(int64_t u, int64_t total, int32_t ctas) {
    return int32_t((uint64_t(u + 1) * ctas + total - 1) / uint64_t(total)) - 1;
}
struct QrPieces {
    int32_t first, n, ctas;
    int64_t unit0, sparse;  // sparse = units in all, if fewer than CTAs (each has one then), else 0
    __device__ __forceinline__ QrPieces(int64_t unit0_, int32_t tiles, int64_t total, int32_t ctas_) {
        ctas = ctas_;
        first = qr_cta_of(unit0_, total, ctas);
        sparse = total < ctas ? total : 0;
        unit0 = unit0_;
        n = sparse != 0 ? tiles : qr_cta_of(unit0_ + tiles - 1, total, ctas) - first + 1;
    }
    __device__ __forceinline__ int64_t slot(int32_t i) const {
        if (i == 0) return 2 * first + 1;
        return 2 * (sparse != 0 ? qr_cta_of(unit0 + i, sparse, ctas) : first + i);
    }
};

// ---------------------------------------------------------------- the kernel

// R: query rows of an item, 16 or 8 (half the columns, for half the work of the
// softmax warps).
template <int HD, bool BF16, int R>
struct QrShape {
    static constexpr int kTerms = BF16 ? 2 : 3;
    static constexpr int kN = (kTerms * R + 15) / 16 * 16;  // columns: a multiple of 16
    // what fits: the third terms of 16 rows take the third CTA's room
    static constexpr int kPerSm = R == 8 ? 3 : 2, kCtas = 152 * kPerSm;
    static constexpr int kStages = (R == 8 ? 2 : 3) * (HD == 128 ? 1 : 2);
    // Scales of tile t + kScales replace those of tile t once its K is asked for, for
    // which S of tile t + 2 is over, and so tile t's softmax has read its own.
    static constexpr int kScales = kStages + 2;
    static constexpr int kTileBytes = kQrTile * HD;
    static constexpr int kQBytes = (kN * HD + 1023) / 1024 * 1024, kPBytes = kN * kQrTile;
    static constexpr int kK = 0, kV = kStages * kTileBytes, kQ = 2 * kStages * kTileBytes, kP = kQ + kQBytes, kTotal = kP + kPBytes;
    static constexpr int kColumns = 2 * kN <= 32 ? 32 : 2 * kN <= 64 ? 64 : 128;  // of TMEM: S, then O
    static constexpr uint32_t kSwizzle = HD == 128 ? 2 : 4, kAtom = HD * 8;
    static constexpr int kRows = R;
};

struct QrJob {
    int32_t n, tile0, head, whole;  // tiles of this CTA's part of it, the first; begins here; begins and ends here
    int32_t q_row, count, kv_head, first_pos, len;
};

template <typename S>
struct QrShared {
    uint64_t k_full[S::kStages], k_empty[S::kStages], v_full[S::kStages], v_empty[S::kStages], sc_full[S::kScales];
    uint64_t s_full, s_free, p_ready, o_full, q_ready, job_full[kQrJobs], job_empty[kQrJobs], drain;
    QrJob job[kQrJobs];
    PaStart start;
    int64_t warp_sums[kQrThreads / 32];
    uint32_t tmem;
    int stop;
    uint64_t deadline;  // for tests: when every wait ends
    float4 scale[S::kScales][8];  // of a tile's pages: K's scale, log2 of V's, 1 / V's; in all alike: far ones since the part began
    float top[2][S::kRows][4];     // of a tile's columns, by warp
    float ref[4][S::kRows];        // the tile's reference less 8, by warp
    float2 fold[2][4][S::kRows];   // factors of old and new sums, by warp
    float col[S::kRows];
};

// Whether a test wants this CTA given up: one in 152 has the number that it names.
__device__ __forceinline__ bool qr_gives_up(const QrArgs &a) { return a.give_up == int32_t(blockIdx.x) % 152; }

// Waits end after two seconds, or once another wait of the CTA has, or at a test's wish,
// which the loading warp sees with every tile, too: nothing here waits for more than a
// tile's copies and MMAs.
template <typename SH>
static __device__ __noinline__ bool qr_wait_long(SH &sh, uint64_t *bar, uint32_t parity) {
    volatile int *stop = &sh.stop;
    const uint64_t since = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*stop != 0) return false;
        const uint64_t now = global_ns();
        if (now - since >= 2000000000ull || now >= sh.deadline) {
            *stop = 1;
            return false;
        }
    }
    return true;
}
template <typename SH>
__device__ __forceinline__ bool qr_wait(SH &sh, uint64_t *bar, uint32_t parity) {
    const bool ok = mbar_try_wait(bar, parity) || qr_wait_long(sh, bar, parity);
    return __all_sync(~0u, ok);
}
__device__ __forceinline__ void qr_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) pa_arrive(bar);
}
__device__ __forceinline__ void qr_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same; whether all four had what they waited for.
__device__ __forceinline__ bool qr_meet(bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(uint32_t(ok))
        : "memory");
    return all != 0;
}

// The largest of a warp's values of each of R columns; lane l gets that of column
// l % R.  Lanes pass on half of the columns that they still have, R - 1 exchanges in all,
// and go on in groups.
template <int R>
__device__ __forceinline__ float warp_tops(const float *x) {
    const int lane = threadIdx.x & 31;
    float y[R];
#pragma unroll
    for (int c = 0; c < R; ++c) y[c] = x[c];
#pragma unroll
    for (int n = R / 2; n >= 1; n /= 2) {
        const bool up = (lane & n) != 0;
#pragma unroll
        for (int c = 0; c < n; ++c) {
            const float keep = up ? y[c + n] : y[c], pass = up ? y[c] : y[c + n];
            y[c] = fmaxf(keep, __shfl_xor_sync(~0u, pass, n));
        }
    }
#pragma unroll
    for (int n = R; n < 32; n *= 2) y[0] = fmaxf(y[0], __shfl_xor_sync(~0u, y[0], n));
    return y[0];
}

// The factor of raw scores under a cap.  A raw score that is not zero is 2^-26 at least,
// with which a factor of 2^100 is past every cap's end; infinity would make a number of
// zero that is none.
__device__ __forceinline__ float qr_cap_factor(float k) { return k > 1.2676506e30f ? 1.2676506e30f : k; }

// x (two values) as e4m3 terms x = t0 + t1 / 16 (+ t2 / 256), packed in 16 bits each.
template <int TERMS>
__device__ __forceinline__ void split2(float x, float y, uint32_t *t) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        t[i] = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
        if (i + 1 == TERMS) break;
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(t[i]), __NV_E4M3)));
        x = (x - v.x) * 16.0f;
        y = (y - v.y) * 16.0f;
    }
}
// The same of two weights up to 256, by way of f16: three terms hold its eleven bits, two
// round them to nine, and what a term leaves to the next is exact in it.  Six instructions
// for two terms, ten for three, where f32 takes nine and seventeen.
template <int TERMS>
__device__ __forceinline__ void split2_weights(float x, float y, uint32_t *t) {
    __half2 v = __floats2half2_rn(x, y);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        t[i] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
        if (i + 1 == TERMS) break;
        v = __hmul2(__hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(t[i]), __NV_E4M3))), __float2half2_rn(16.0f));
    }
}
template <int TERMS, int R>
__device__ __forceinline__ float joined(const float *x, int c) {
    float v = fmaf(x[R + c], 1.0f / 16, x[c]);
    if constexpr (TERMS == 3) v = fmaf(x[2 * R + c], 1.0f / 256, v);
    return v;
}
template <int N>
__device__ __forceinline__ void tc_ld_columns(uint32_t addr, float *x) {
    if constexpr (N == 16) tc_ld16(addr, x);
    else tc_ld32(addr, x);
    if constexpr (N == 48) tc_ld16(addr + 32, x + 32);
}

template <int HD, bool BF16, int R>
__global__ void __launch_bounds__(kQrThreads, (QrShape<HD, BF16, R>::kPerSm)) qr_kernel(const __grid_constant__ QrArgs a) {
    using S = QrShape<HD, BF16, R>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr int kTerms = S::kTerms;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    QrShared<S> &sh = *reinterpret_cast<QrShared<S> *>(smem_raw + S::kTotal);
    const uint32_t smem = smem_addr(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int i = 0; i < S::kScales; ++i) mbar_init(&sh.sc_full[i], 1);
        for (int i = 0; i < kQrJobs; ++i) {
            mbar_init(&sh.job_full[i], 1);
            mbar_init(&sh.job_empty[i], 5);  // softmax warps and the MMAs'
        }
        mbar_init(&sh.s_full, 1);
        mbar_init(&sh.s_free, 4);
        mbar_init(&sh.p_ready, 4);
        mbar_init(&sh.o_full, 1);
        mbar_init(&sh.q_ready, 4);
        mbar_init(&sh.drain, 1);
        fence_mbar_init();
        sh.stop = 0;
        sh.deadline = qr_gives_up(a) ? global_ns() + a.give_up_ns : ~0ull;
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(S::kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_before();
    }
    if (warp == 4 && lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &a.k : &a.v) : "memory");
    pdl_wait();
    // The next launch may come: it waits for this one before it writes, and finds its
    // SM free when this one's CTAs leave.
    pdl_trigger();
    qr_cut<kQrThreads>(a, &sh.start, sh.warp_sums);  // synchronises the CTA
    tc_after();
    const uint32_t tmem = sh.tmem;
    const PaStart st = sh.start;
    uint32_t k_loads = 0, v_loads = 0;  // tiles asked for
    if (threadIdx.x == 128) a.cut[blockIdx.x].n = 0;  // whose thread writes a record, too

    if (st.units > 0) {
        if (warp == 4) {
            // -------------------------------------------------------- work and loads
            PaWalk w = {st.b, st.h, st.tok, st.s};
            int32_t unit = st.unit;
            int64_t left = st.units;
            const int ppt = kQrTile >> a.page_log2;
            const uint32_t box = uint32_t(HD) << a.page_log2;  // bytes of a page
            bool ok = true;
            for (uint32_t at = 0;;) {
                const bool over = left <= 0;
                QrItem it = {};
                int32_t have = 0, tile = 0, n = 0;
                if (!over) {
                    it = qr_item(a, w.s, w.tok);
                    have = it.units - unit;
                    const int32_t end = unit + (left < have ? int32_t(left) : have) - a.extra;
                    tile = unit > a.extra ? unit - a.extra : 0;
                    n = end > tile ? end - tile : 0;
                }
                const int32_t tile0 = it.tile0 + tile;
                if (over || n > 0) {
                    QrJob &job = sh.job[at % kQrJobs];
                    if (at >= kQrJobs) ok = qr_wait(sh, &sh.job_empty[at % kQrJobs], (at / kQrJobs & 1) ^ 1);
                    if (!ok) break;
                    if (lane == 0) {
                        const bool whole = n == it.tiles;
                        job = QrJob{n, tile0, tile == 0, whole, w.s.q0 + w.tok, it.count, w.h, it.first_pos, w.s.len};
                        if (!over && tile == 0 && !whole)
                            a.cut[blockIdx.x] = QrCut{st.from + (st.units - left) - unit + a.extra, st.total, it.tiles, it.count * a.group, w.s.q0 + w.tok, w.h, 1, 0};
                    }
                    qr_arrive(&sh.job_full[at % kQrJobs]);
                    ++at;
                }
                if (over) break;
                const int32_t held = (w.s.len + (1 << a.page_log2) - 1) >> a.page_log2;
                const int32_t *table = a.block_table + int64_t(w.b) * a.max_pages;
                const int32_t h = w.h;
                // Page numbers and scales of 32 pages at a time, lane by lane; the next 32 are
                // under way meanwhile.  (A tile's own, two and one ahead, held up pages of 16.)
                const int32_t page0 = tile0 * ppt, pages = n * ppt;
                auto lookup = [&](int32_t block) {
                    const int32_t p = block * 32 + lane;
                    int32_t page = -1;
                    if (p < pages && page0 + p < held) {
                        page = table[page0 + p];
                        if (uint32_t(page) >= uint32_t(a.n_pages)) {
                            set_error(a.err, kErrBounds);
                            page = -1;
                        }
                    }
                    return page;
                };
                auto scales = [&](int32_t page) {
                    float2 s = make_float2(1.0f, 1.0f);
                    if (page >= 0) s = make_float2(a.k_scale[int64_t(page) * a.n_kv + h], a.v_scale[int64_t(page) * a.n_kv + h]);
                    return s;
                };
                auto load = [&](const CUtensorMap *map, uint32_t dst, int32_t page, uint64_t *bar) {
                    if (lane == 0) mbar_arrive_expect_tx(bar, S::kTileBytes);
                    __syncwarp();
                    if (lane < ppt) tma_2d(dst + lane * box, map, 0, page < 0 ? a.pool_rows : (page * a.n_kv + h) << a.page_log2, bar);
                };
                const int32_t per_block = 32 / ppt;  // tiles
                int32_t block_pages = lookup(0), next_pages = lookup(1), v_page = -1;
                float2 block_scales = scales(block_pages), next_scales = make_float2(1.0f, 1.0f);
                bool far = false;
                // K runs a tile ahead of V
                for (int32_t t = 0; ok && t <= n; ++t) {
                    int32_t page = -1;
                    if (qr_gives_up(a) && global_ns() >= sh.deadline) {
                        *static_cast<volatile int *>(&sh.stop) = 1;
                        ok = false;
                        break;
                    }
                    if (t < n) {
                        const int32_t in = t % per_block;
                        if (t > 0 && in == 0) {
                            block_pages = next_pages;
                            block_scales = per_block > 1 ? next_scales : scales(block_pages);
                            next_pages = lookup(t / per_block + 1);
                        }
                        if (in == 1) next_scales = scales(next_pages);
                        const int from = in * ppt + lane % ppt;
                        page = __shfl_sync(~0u, block_pages, from);
                        const float ks = __shfl_sync(~0u, block_scales.x, from), vs = __shfl_sync(~0u, block_scales.y, from);
                        const uint32_t slot = k_loads % S::kStages, turn = k_loads / S::kStages, sc = k_loads % S::kScales;
                        if (turn > 0) ok = qr_wait(sh, &sh.k_empty[slot], (turn & 1) ^ 1);
                        if (!ok) break;
                        // (K first: the scales may still be on their way)
                        load(&a.k, smem + S::kK + slot * S::kTileBytes, page, &sh.k_full[slot]);
                        far = far || __any_sync(~0u, vs > kScaleFar && vs <= kScaleHigh);
                        if (lane < ppt) {
                            const float v = scale_of(vs, a.err);
                            sh.scale[sc][lane] = make_float4(scale_of(ks, a.err), log2f(v), 1.0f / v, far ? 1.0f : 0.0f);
                        }
                        qr_arrive(&sh.sc_full[sc]);
                        ++k_loads;
                    }
                    if (t > 0) {
                        const uint32_t slot = v_loads % S::kStages, turn = v_loads / S::kStages;
                        if (turn > 0) ok = qr_wait(sh, &sh.v_empty[slot], (turn & 1) ^ 1);
                        if (!ok) break;
                        load(&a.v, smem + S::kV + slot * S::kTileBytes, v_page, &sh.v_full[slot]);
                        ++v_loads;
                    }
                    v_page = page;
                }
                if (!ok) break;
                left -= have;
                unit = 0;
                if (left > 0) qr_next(a, w);
            }
        } else if (warp == 5) {
            // -------------------------------------------------------- MMAs
            uint32_t g = 0;  // tiles so far
            bool ok = true;
            auto score = [&](uint32_t i) {
                const uint32_t slot = i % S::kStages;
                ok = qr_wait(sh, &sh.k_full[slot], i / S::kStages & 1);
                if (ok && i > 0) ok = qr_wait(sh, &sh.s_free, (i - 1) & 1);
                if (!ok) return;
                tc_after();
                if (elect_one()) {
                    constexpr uint32_t id = tc_idesc8(128, S::kN, false, false);
                    const uint64_t kd = tc_desc(smem + S::kK + slot * S::kTileBytes, 16, S::kAtom, S::kSwizzle);
                    const uint64_t qd = tc_desc(smem + S::kQ, 16, S::kAtom, S::kSwizzle);
#pragma unroll
                    for (int kk = 0; kk < HD / 32; ++kk) tc_mma8(tmem, kd + kk * 2, qd + kk * 2, id, kk != 0);
                }
                __syncwarp();
                tc_commit(&sh.s_full);
                tc_commit(&sh.k_empty[slot]);
            };
            for (uint32_t at = 0;; ++at) {
                ok = qr_wait(sh, &sh.job_full[at % kQrJobs], at / kQrJobs & 1);
                if (!ok) break;
                const uint32_t n = uint32_t(sh.job[at % kQrJobs].n);
                qr_arrive(&sh.job_empty[at % kQrJobs]);
                if (n == 0) break;
                ok = qr_wait(sh, &sh.q_ready, at & 1);
                if (!ok) break;
                score(g);
                for (uint32_t i = g; ok && i < g + n; ++i) {
                    if (i + 1 < g + n) score(i + 1);
                    if (!ok) break;
                    const uint32_t slot = i % S::kStages;
                    ok = qr_wait(sh, &sh.v_full[slot], i / S::kStages & 1) && qr_wait(sh, &sh.p_ready, i & 1);
                    if (!ok) break;
                    tc_after();
                    if (elect_one()) {
                        constexpr uint32_t id = tc_idesc8(HD, S::kN, true, true);
                        const uint64_t vd = tc_desc(smem + S::kV + slot * S::kTileBytes, kQrTile * 128, S::kAtom, S::kSwizzle);
                        const uint64_t pd = tc_desc(smem + S::kP, 128, kQrTile * 16, 0);
#pragma unroll
                        for (int kk = 0; kk < kQrTile / 32; ++kk)
                            tc_mma8(tmem + S::kN, vd + kk * (32 * HD >> 4), pd + kk * (512 >> 4), id, kk != 0);
                    }
                    __syncwarp();
                    tc_commit(&sh.o_full);
                    tc_commit(&sh.v_empty[slot]);
                }
                if (!ok) break;
                g += n;
            }
            // nobody waits for the last v_empty, but the block must not end before it has come
            tc_commit(&sh.drain);
            if (!mbar_wait_bounded(&sh.drain, 0, 500000000ull)) *static_cast<volatile int *>(&sh.stop) = 1;
        } else {
            // -------------------------------------------------------- softmax and sums
            const int row = threadIdx.x;                 // of the tile
            const uint32_t t_row = tmem + (uint32_t(warp * 32) << 16);
            // the channel whose sums this thread keeps: rows of 64 lie in the first 16 lanes of each warp
            const int chan = HD == 128 ? row : warp * 16 + lane;
            const bool has_chan = HD == 128 || lane < 16;
            const int32_t per_256 = (256 + a.group - 1) / a.group;  // exact for 16 columns
            uint32_t g = 0;
            bool ok = true, met = true;
            for (uint32_t at = 0;; ++at) {
                ok = qr_wait(sh, &sh.job_full[at % kQrJobs], at / kQrJobs & 1);
                if (!ok) break;
                const QrJob job = sh.job[at % kQrJobs];
                qr_arrive(&sh.job_empty[at % kQrJobs]);
                if (job.n == 0) break;
                const int32_t live = job.count * a.group;  // query rows

                // q as e4m3 terms; every MMA that read the last item's has been waited for
                {
                    constexpr int kLanes = 128 / R, kPer = HD / kLanes;  // lanes of a row, channels of a lane
                    const int r = row / kLanes, part = row % kLanes;
                    float x[kPer], top = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) x[i] = 0.0f;
                    if (r < live) {
                        const int32_t tok = r / a.group;
                        const T *p = static_cast<const T *>(a.q) + (int64_t(job.q_row) + tok) * a.q_tok +
                                     int64_t(job.kv_head * a.group + r - tok * a.group) * a.q_head + part * kPer;
                        if constexpr (kPer >= 8) {
#pragma unroll
                            for (int i = 0; i < kPer; i += 8) load8<T>(p + i, x + i);
                        } else {
                            T y[4];
                            *reinterpret_cast<uint2 *>(y) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[i] = to_f32<T>(y[i]);
                        }
                    }
                    bool fine = true;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        fine = fine && fabsf(x[i]) <= FLT_MAX;
                        top = fmaxf(top, fabsf(x[i]));
                    }
#pragma unroll
                    for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    const uint32_t odd = __ballot_sync(~0u, !fine) >> (lane & ~(kLanes - 1)) & ((1u << kLanes) - 1);
                    int e = 134 - int(__float_as_uint(top) >> 23);
                    e = top == 0.0f ? 0 : e > 120 ? 120 : e < -120 ? -120 : e;
                    const float up = __uint_as_float(uint32_t(e + 127) << 23);
                    uint32_t t[kPer / 2][kTerms];
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i) split2<kTerms>(x[2 * i] * up, x[2 * i + 1] * up, t[i]);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) {
                        uint32_t to = (k * R + r) * HD + part * kPer;
                        to = smem + S::kQ + (to ^ (HD == 128 ? (to >> 7 & 7) << 4 : (to >> 7 & 3) << 4));
                        const uint32_t w0 = t[0][k] | t[1][k] << 16;
                        if constexpr (kPer == 16)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(w0), "r"(t[2][k] | t[3][k] << 16),
                                         "r"(t[4][k] | t[5][k] << 16), "r"(t[6][k] | t[7][k] << 16)
                                         : "memory");
                        else if constexpr (kPer == 8)
                            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(w0), "r"(t[2][k] | t[3][k] << 16) : "memory");
                        else
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(w0) : "memory");
                    }
                    // a row that is not finite is none of numbers
                    if (part == 0) sh.col[r] = odd != 0 ? __int_as_float(0x7fc00000) : a.mul * __uint_as_float(uint32_t(127 - e) << 23);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    qr_arrive(&sh.q_ready);
                    met = qr_meet(true);
                    if (!met) break;
                }

                float acc[R], sum[R];
#pragma unroll
                for (int c = 0; c < R; ++c) acc[c] = sum[c] = 0.0f;
                float m_run = -INFINITY;  // of column lane % R
                // the tile's part of the sums, once its O is there
                auto take = [&](float *o) {
                    tc_after();
                    tc_ld_columns<S::kN>(t_row + S::kN, o);
                    tc_wait_ld();
                    tc_before();
                };
                auto fold = [&](const float *o, uint32_t i) {
#pragma unroll
                    for (int c = 0; c < R; c += 2) {
                        const float4 f = *reinterpret_cast<const float4 *>(&sh.fold[i & 1][warp][c]);
                        acc[c] = fmaf(acc[c], f.x, joined<kTerms, R>(o, c) * f.y);
                        acc[c + 1] = fmaf(acc[c + 1], f.z, joined<kTerms, R>(o, c + 1) * f.w);
                    }
                };
                int32_t owed = 0;  // meetings to come of this item, before a wait
                for (int32_t i = 0; i < job.n; ++i, ++g) {
                    owed = job.n - i + 1;
                    ok = qr_wait(sh, &sh.sc_full[g % S::kScales], g / S::kScales & 1);
                    if (!ok) break;
                    const float4 sc = sh.scale[g % S::kScales][row >> a.page_log2];
                    ok = qr_wait(sh, &sh.s_full, g & 1);
                    if (!ok) break;
                    float x[R];
                    {
                        float s[S::kN];
                        tc_after();
                        tc_ld_columns<S::kN>(t_row, s);
                        tc_wait_ld();
                        tc_before();
                        qr_arrive(&sh.s_free);
                        // scores with the scale of V's block, log2 units
#pragma unroll
                        for (int c = 0; c < R; ++c) {
                            const float k = sh.col[c] * sc.x, y = joined<kTerms, R>(s, c);
                            if (a.cap > 0.0f) x[c] = fmaf(pa_tanh_of_any(y * qr_cap_factor(k)), a.cap, sc.y);
                            else x[c] = fmaf(y, k, sc.y);
                        }
                    }
                    // masks: rows behind a token, and before its window
                    const int32_t key = (job.tile0 + i) * kQrTile + row;
                    const int32_t key0 = key - row, last = job.first_pos + job.count - 1;
                    const int64_t lo = a.window > 0 ? int64_t(job.first_pos) - a.window + 1 : 0;  // of the first token
                    if (key0 + kQrTile - 1 > job.first_pos || (a.window > 0 && key0 < lo + job.count - 1)) {
#pragma unroll
                        for (int c = 0; c < R; ++c) {
                            const int32_t pos = job.first_pos + (c * per_256 >> 8);  // its token is c / group
                            const bool seen = key <= pos && pos <= last && (a.window == 0 || key > pos - a.window);
                            x[c] = seen ? x[c] : -INFINITY;
                        }
                    }
                    // the tile's reference: the largest weight with its block's scale
                    {
                        const float t = warp_tops<R>(x);
                        if (lane < R) sh.top[i & 1][lane][warp] = t;
                    }
                    qr_sync();
                    owed = job.n - i;
                    {
                        const int c = lane % R;
                        const float4 t = *reinterpret_cast<const float4 *>(sh.top[i & 1][c]);
                        const float ref = fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)), now = fmaxf(m_run, ref);
                        const float base = now == -INFINITY ? 0.0f : now;
                        // weights are held 2^8 higher
                        if (sc.w != 0.0f) {
                            const float half = ex2(0.5f * (m_run - base));
#pragma unroll
                            for (int e = 0; e < R; ++e) {
                                const float f = __shfl_sync(~0u, half, e);
                                sum[e] = fmaf(sum[e] * f, f, ex2(x[e] - sc.y - __shfl_sync(~0u, base, e)));
                            }
                        }
                        if (lane < R) {
                            sh.ref[warp][c] = ref == -INFINITY ? 0.0f : ref - 8.0f;
                            sh.fold[i & 1][warp][c] = make_float2(ex2(m_run - base), ex2(ref - base) * 0.00390625f);
                        }
                        m_run = now;
                        __syncwarp();
                    }
                    uint32_t p[R / 2][kTerms];
#pragma unroll
                    for (int c = 0; c < R; c += 2) {
                        const float2 ref = *reinterpret_cast<const float2 *>(&sh.ref[warp][c]);
                        const float4 f = *reinterpret_cast<const float4 *>(&sh.fold[i & 1][warp][c]);
                        const float w0 = ex2(x[c] - ref.x), w1 = ex2(x[c + 1] - ref.y);
                        if (sc.w == 0.0f) {
                            sum[c] = fmaf(sum[c], f.x, w0 * (sc.z * f.y));
                            sum[c + 1] = fmaf(sum[c + 1], f.z, w1 * (sc.z * f.w));
                        }
                        split2_weights<kTerms>(w0, w1, p[c / 2]);
                    }
                    // rows of V that nobody holds: their weights are zero, but zero times NaN is not
                    if (key0 + kQrTile > job.len) {
                        ok = qr_wait(sh, &sh.v_full[g % S::kStages], g / S::kStages & 1);
                        if (!ok) break;
                        if (key >= job.len) {
                            const uint32_t v = smem + S::kV + g % S::kStages * S::kTileBytes + row * HD;
#pragma unroll
                            for (int b = 0; b < HD; b += 16) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + b), "r"(0) : "memory");
                        }
                    }
                    float o[S::kN];
                    if (i > 0) {
                        ok = qr_wait(sh, &sh.o_full, (g - 1) & 1);
                        if (!ok) break;
                        take(o);
                    }
                    // 16 columns of a row lie together
#pragma unroll
                    for (int k = 0; k < (R == 16 ? kTerms : (kTerms + 1) / 2); ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int from = R == 16 ? k : k * 2 + e / 2, pair = R == 16 ? 2 * e : 2 * (e % 2);
                            w[e] = from < kTerms ? p[pair][from] | p[pair + 1][from] << 16 : 0u;
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(smem + S::kP + k * (kQrTile * 16) + row * 16), "r"(w[0]), "r"(w[1]),
                                     "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_before();
                    qr_arrive(&sh.p_ready);
                    if (i > 0) fold(o, uint32_t(i - 1));
                }
                if (ok) {
                    float o[S::kN];
                    owed = 1;
                    ok = qr_wait(sh, &sh.o_full, (g - 1) & 1);
                    if (ok) {
                        take(o);
                        fold(o, uint32_t(job.n - 1));
                    }
                }
                if (!ok) {
                    for (; owed > 0; --owed) qr_sync();
                    break;
                }
                // the sums over the tile's rows, by way of the maxima's buffer that is not the last tile's
                float(*const sums)[4] = sh.top[job.n & 1];
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    float s = sum[c];
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
                    if (lane == c) sums[c][warp] = s;
                }
                qr_sync();
                const int64_t slot = int64_t(blockIdx.x) * 2 + job.head;
                // what column lane % R is multiplied by
                float f;
                {
                    const int c = lane % R;
                    const float4 s4 = *reinterpret_cast<const float4 *>(sums[c]);
                    float s = (s4.x + s4.y) + (s4.z + s4.w);
                    f = 1.0f;
                    if (job.whole != 0 && a.sinks != nullptr && c < live && m_run != -INFINITY) {
                        const float sink = a.sinks[job.kv_head * a.group + c % a.group] * 1.4426950408889634f, all = fmaxf(m_run, sink);
                        f = ex2(m_run - all);
                        s = s * f + ex2(sink - all);
                    }
                    f *= s == 0.0f ? 0.0f : rcp(s);
                    // Of a piece the outputs over the sum, whose logarithm joins the reference: pieces meet as weights, without V's
                    // scales.  (By approximate instructions, whose errors are 2^-22 of a weight: what rcp is off by stays in s * f.)
                    if (job.whole == 0 && row < live) a.part_ml[slot * a.part_rows + c] = make_float2(s == 0.0f ? -INFINITY : m_run + __log2f(s), s * f);
                }
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    if (c >= live) break;
                    const float y = acc[c] * __shfl_sync(~0u, f, c);
                    if (!has_chan) continue;
                    const int32_t tok = c / a.group, head = job.kv_head * a.group + c - tok * a.group;
                    if (job.whole == 0) a.part_o[(slot * a.part_rows + c) * HD + chan] = y;
                    else static_cast<T *>(a.out)[(int64_t(job.q_row) + tok) * a.out_tok + int64_t(head) * a.out_head + chan] = from_f32<T>(y);
                }
                // (the next item's sums are written behind qr_sync calls that every warp passes after this)
            }
            // behind the last item, or with a wait given up: the others are on their way to this meeting
            if (met) qr_meet(ok);
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (*static_cast<volatile int *>(&sh.stop) != 0) {
        // given up: no copy may be in flight into this CTA's memory
        if (threadIdx.x == 0) set_error(a.err, kErrTimeout);
        if (warp == 4)
            for (uint32_t i = 0; i < uint32_t(S::kStages); ++i) {
                if (k_loads > i) mbar_wait_bounded(&sh.k_full[(k_loads - 1 - i) % S::kStages], (k_loads - 1 - i) / S::kStages & 1, 500000000ull);
                if (v_loads > i) mbar_wait_bounded(&sh.v_full[(v_loads - 1 - i) % S::kStages], (v_loads - 1 - i) / S::kStages & 1, 500000000ull);
            }
        tc_before();
        __syncthreads();
        tc_after();
    }
    if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kColumns) : "memory");
}

template <int HD, bool BF16, int R>
cudaError_t launch_qr(QrArgs &a, cudaStream_t st) {
    using S = QrShape<HD, BF16, R>;
    constexpr int smem = S::kTotal + int(sizeof(QrShared<S>));
    static_assert(S::kPerSm * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
    const auto kern = qr_kernel<HD, BF16, R>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    a.ctas = S::kCtas;
    return launch_pdl(kern, dim3(S::kCtas), dim3(kQrThreads), smem, st, a);
}

struct QrJoin {
    QrArgs few, many;  // of the launches whose pieces these are; ctas 0 = none
    int32_t wide;      // CTAs for each record of `many`
};

// Joins the rows of cut items, by warps whose lanes stand for channels, four pieces
// under way at a time: one CTA for a record of `few`, whose warps share the pieces of its
// rows, `wide` for one of `many`.  (A token over 131072 rows leaves 57 pieces of a row.)
constexpr int kJoinThreads = 256;
template <int HD, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) qr_join_kernel(const __grid_constant__ QrJoin j) {
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr int kPer = HD / 32, kWarps = kJoinThreads / 32, kDeep = 4;
    __shared__ float parts[kWarps][HD + 2];
    pdl_wait();
    const bool is_few = int32_t(blockIdx.x) < j.few.ctas;
    const int32_t at_cta = int32_t(blockIdx.x) - (is_few ? 0 : j.few.ctas);
    const QrArgs &a = is_few ? j.few : j.many;
    const int32_t share = is_few ? 1 : j.wide;
    const QrCut cut = a.cut[at_cta / share];
    if (cut.n == 0) return;
    const QrPieces pieces(cut.unit0, cut.tiles, cut.total, a.ctas);
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane * kPer;
    int32_t at_once = kWarps;  // rows
    if (is_few)
        while (at_once / 2 >= cut.rows) at_once /= 2;
    const int32_t split = kWarps / at_once, part = warp / at_once;  // warps of a row
    for (int32_t r = at_cta % share * at_once + warp % at_once; r < cut.rows || split > 1; r += share * at_once) {
        float top = -INFINITY, sum = 0.0f, o[kPer] = {};
#pragma unroll 1
        for (int32_t i0 = part; i0 < pieces.n && r < cut.rows; i0 += kDeep * split) {
            float2 ml[kDeep];
            float v[kDeep][kPer] = {};
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                ml[i] = make_float2(-INFINITY, 0.0f);
                if (i0 + i * split >= pieces.n) continue;
                const int64_t at = pieces.slot(i0 + i * split) * a.part_rows + r;
                ml[i] = __ldcg(&a.part_ml[at]);
                const float *p = a.part_o + at * HD + col;
                if constexpr (kPer == 4) *reinterpret_cast<float4 *>(v[i]) = __ldcg(reinterpret_cast<const float4 *>(p));
                else *reinterpret_cast<float2 *>(v[i]) = __ldcg(reinterpret_cast<const float2 *>(p));
            }
            float now = top;
#pragma unroll
            for (int i = 0; i < kDeep; ++i) now = fmaxf(now, ml[i].x);
            const float base = now == -INFINITY ? 0.0f : now, f0 = ex2(top - base);
            sum *= f0;
#pragma unroll
            for (int c = 0; c < kPer; ++c) o[c] *= f0;
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const float f = ex2(ml[i].x - base);
                sum += ml[i].y * f;
#pragma unroll
                for (int c = 0; c < kPer; ++c) o[c] += v[i][c] * f;
            }
            top = now;
        }
        if (split > 1) {  // the warps' parts of a row, in their order
            if (lane == 0) parts[warp][HD] = top, parts[warp][HD + 1] = sum;
#pragma unroll
            for (int c = 0; c < kPer; ++c) parts[warp][col + c] = o[c];
            __syncthreads();
            if (part > 0 || r >= cut.rows) return;
            for (int32_t w = warp; w < kWarps; w += at_once) top = fmaxf(top, parts[w][HD]);
            const float base = top == -INFINITY ? 0.0f : top;
            sum = 0.0f;
#pragma unroll
            for (int c = 0; c < kPer; ++c) o[c] = 0.0f;
            for (int32_t w = warp; w < kWarps; w += at_once) {
                const float f = ex2(parts[w][HD] - base);
                sum += parts[w][HD + 1] * f;
#pragma unroll
                for (int c = 0; c < kPer; ++c) o[c] += parts[w][col + c] * f;
            }
        }
        const int32_t tok = r / a.group, head = cut.kv_head * a.group + r - tok * a.group;
        float f = 1.0f;
        if (a.sinks != nullptr && top != -INFINITY) {
            const float sink = a.sinks[head] * 1.4426950408889634f, all = fmaxf(top, sink);
            f = ex2(top - all);
            sum = sum * f + ex2(sink - all);
        }
        f *= sum == 0.0f ? 0.0f : 1.0f / sum;
        T *dst = static_cast<T *>(a.out) + (int64_t(cut.q_row) + tok) * a.out_tok + int64_t(head) * a.out_head + col;
#pragma unroll
        for (int c = 0; c < kPer; c += 2) *reinterpret_cast<uint32_t *>(dst + c) = pack2<BF16>(o[c] * f, o[c + 1] * f);
        if (split > 1) return;  // all rows were at once
    }
}

template <int HD, bool BF16>
cudaError_t launch_qr_join(const QrJoin &j, cudaStream_t st) {
    return launch_pdl(qr_join_kernel<HD, BF16>, dim3(unsigned(j.few.ctas + j.many.ctas * j.wide)), dim3(kJoinThreads), 0, st, j);
}

}  // namespace kvd
