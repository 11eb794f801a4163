// kvd_paged_attn.cuh -- attention of new rows over a paged cache, on the
// fifth-generation tensor cores.
//
// out_t = sum_p softmax_p(scale q_t . k_p) v_p over the rows p that t sees, in
// one pass over K and V with a running maximum and sum.
//
// Query rows.  The query heads of one KV head share its K and V, so a tile's
// 128 rows are (token, head of the group) pairs: 128 / group tokens.  An item
// of work is one (request, KV head, run of up to two tiles' tokens):
//   two tiles ("dual", prompts): both tiles meet the same KV tile, whose 64 KB
//     then serve 256 query rows;
//   one tile ("single", decode steps and drafts): the two streams of the
//     pipeline take the even and the odd KV tiles and are joined at the end, so
//     a single token still keeps two softmax groups and the copies busy.
// Work is cut into units (one KV tile of a dual item, two of a single one) and
// every CTA gets the same number of consecutive units, however long the
// requests are; an item that is cut leaves its pieces (unnormalised output,
// maximum, sum) in the workspace and paged_merge_kernel joins them.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax of stream 0 and 1, a thread per query row;
//   warp 8          TMA loads: Q, and K / V tiles of 128 rows into a ring, page
//                   by page (a page that does not exist reads as zeros);
//   warp 9          the MMAs: S = Q K^T and O += P V, P read from TMEM.
// TMEM: S0 S1 (128 columns each; P overwrites the first 64) O0 O1.
// MMAs of one thread run in order, so S of a stream's next tile may be issued
// behind P V of its last one without a wait, and S being complete says that P V
// before it is: the softmax group may then rescale O in place.  It does so only
// when a row's maximum grew by more than 2^kSlack; until then the old one is
// as good a reference.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvd_internal.cuh"

namespace kvd {

constexpr int kPaCtas = 152;       // one per SM; also fixes the cut of the work
constexpr int kPaThreads = 384;    // warps 10 and 11 only fill their warpgroup
// Registers a thread: the launch gives 384 x 168; the softmax warpgroups trade up.
constexpr int kPaRegs = 168, kPaSoftRegs = 208, kPaLoadRegs = 88;
static_assert(2 * kPaSoftRegs + kPaLoadRegs <= 3 * kPaRegs, "setmaxnreg shares");
constexpr int kPaTile = 128;       // query rows of a tile, and KV rows of a tile
constexpr int kPaQBytes = 2 * kPaTile * 256;
constexpr int kPaMaxRows = 2 * kPaTile;

struct PaArgs {
    CUtensorMap q, k, v;
    const int32_t *block_table, *cu_new, *seq_len;
    void *out;
    int64_t out_tok, out_head;
    const float *sinks;
    float *part_o;     // [2 * kPaCtas][part_rows][hd]
    float2 *part_ml;   // [2 * kPaCtas][part_rows]: reference maximum (log2 units), sum
    int32_t *meta;     // [kPaCtas][8]
    uint32_t *err;
    int64_t window;    // 0 = none
    int32_t n_seq, n_tokens, n_kv, group, tile_tok, max_pages, n_pages, page_log2;
    int32_t part_rows, pool_rows;
    float scale_log2;  // scale * log2 e (softcap 0), or softcap * log2 e
    float cap_in;      // softcap > 0: 2 * scale * log2 e / softcap
};

// Piece records in PaArgs::meta.
enum { kPmTail = 0, kPmSeq = 1, kPmHead = 2, kPmTok = 3, kPmFirst = 4 };
// kPmTail: 1 = this CTA holds the head piece of a cut item (slot 2 c + 1).
// kPmFirst: 0 = starts on an item boundary, 1 = its first piece continues the
// item of the CTA before and ends it, 2 = continues and does not end it,
// 3 = this CTA has no work.

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_ld32(uint32_t addr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const float *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]),
        "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]),
        "f"(r[17]), "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]),
        "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major operands: sbo =
// bytes between groups of eight rows.  MN-major: lbo = bytes between runs of 64
// MN elements, sbo = bytes between groups of eight K rows.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return uint64_t((addr & 0x3ffffu) >> 4) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Instruction descriptor of kind::f16: f32 accumulator, M x N, B MN-major or not.
__host__ __device__ constexpr uint32_t tc_idesc(bool bf16, int m, int n, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrive once on bar when every MMA this thread has issued so far is complete.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void pa_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, int32_t w,
                                       uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two f32 operations in one issue slot.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A wait that gives up: bounded in time, and ended early once another warp of
// the CTA has given up.  The whole warp gets one answer.
__device__ __forceinline__ bool pa_wait(uint64_t *bar, uint32_t parity, volatile int *stop) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        for (int i = 0; i < 256 && !ok; ++i) ok = mbar_try_wait(bar, parity);
        if (!ok) {
            const uint64_t t0 = global_ns();
            while (!(ok = mbar_try_wait(bar, parity)))
                if (*stop != 0 || global_ns() - t0 > 2000000000ull) break;
        }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *stop = 1;
    return ok;
}

// ---------------------------------------------------------------- the work

struct PaSeq {
    int32_t q0, fresh, len;  // first packed row, new rows (0 = skip), rows held
};
__device__ __forceinline__ PaSeq pa_seq(const PaArgs &a, int b, bool report) {
    PaSeq s = {0, 0, 0};
    if (b >= a.n_seq) return s;
    const int32_t q0 = a.cu_new[b], q1 = a.cu_new[b + 1], len = a.seq_len[b];
    if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 || len > (int64_t(a.max_pages) << a.page_log2)) {
        if (report) set_error(a.err, kErrBounds);
        return s;
    }
    s.q0 = q0;
    s.fresh = q1 - q0;
    s.len = len;
    return s;
}

// One item: tokens [tok, tok + count) of a request for one KV head.
struct PaItem {
    int32_t count;         // tokens
    int32_t first_pos;     // position of the first (may be negative)
    int32_t tile0, tiles;  // its KV tiles
    bool dual;
    int32_t units;
};
__device__ __forceinline__ PaItem pa_item(const PaArgs &a, const PaSeq &s, int32_t tok) {
    PaItem it;
    const int32_t left = s.fresh - tok, most = 2 * a.tile_tok;
    it.count = left < most ? left : most;
    it.first_pos = s.len - s.fresh + tok;
    int64_t lo = a.window > 0 ? int64_t(it.first_pos) - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    int32_t hi = it.first_pos + it.count;
    if (hi < 0) hi = 0;
    it.tile0 = int32_t(lo) / kPaTile;
    const int32_t n = (hi + kPaTile - 1) / kPaTile - it.tile0;
    it.tiles = n > 1 ? n : 1;
    it.dual = it.count > a.tile_tok;
    it.units = it.dual ? it.tiles : (it.tiles + 1) / 2;
    return it;
}

// Position in the order (request, KV head, token run); every role walks it alike.
struct PaWalk {
    int32_t b, h, tok;
    PaSeq s;
};
__device__ __forceinline__ void pa_next(const PaArgs &a, PaWalk &w) {
    w.tok += 2 * a.tile_tok;
    if (w.tok < w.s.fresh) return;
    w.tok = 0;
    if (++w.h < a.n_kv) return;
    w.h = 0;
    do {
        ++w.b;
        w.s = pa_seq(a, w.b, false);
    } while (w.s.fresh == 0 && w.b < a.n_seq);
}

struct PaStart {
    int32_t b, h, tok, unit;  // first item and the unit in it
    int64_t units;            // units of this CTA
};

// The cut: CTA c of n takes units [c W / n, (c + 1) W / n) of the W there are.
// All threads; the result is in shared memory.
__device__ __forceinline__ void pa_cut(const PaArgs &a, PaStart *out, int64_t *warp_sums) {
    const int per = (a.n_seq + kPaThreads - 1) / kPaThreads;
    const int b0 = threadIdx.x * per < a.n_seq ? threadIdx.x * per : a.n_seq;
    const int b1 = b0 + per < a.n_seq ? b0 + per : a.n_seq;
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const PaSeq s = pa_seq(a, b, blockIdx.x == 0);
        int64_t u = 0;
        for (int32_t tok = 0; tok < s.fresh; tok += 2 * a.tile_tok) u += pa_item(a, s, tok).units;
        mine += u * a.n_kv;
    }
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    if (threadIdx.x == 0) out->units = 0;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kPaThreads / 32; ++i) {
        const int64_t v = warp_sums[i];
        before += i < w ? v : 0;
        total += v;
    }
    before += x - mine;
    const int64_t from = total * blockIdx.x / gridDim.x, to = total * (blockIdx.x + 1) / gridDim.x;
    if (from < to && before <= from && from < before + mine) {
        int64_t off = from - before;
        int b = b0;
        PaSeq s;
        int64_t u;
        for (;; ++b) {
            s = pa_seq(a, b, false);
            u = 0;
            for (int32_t tok = 0; tok < s.fresh; tok += 2 * a.tile_tok) u += pa_item(a, s, tok).units;
            if (off < u * a.n_kv) break;
            off -= u * a.n_kv;
        }
        const int32_t h = int32_t(off / u);
        off -= h * u;
        int32_t tok = 0;
        for (;; tok += 2 * a.tile_tok) {
            const int32_t n = pa_item(a, s, tok).units;
            if (off < n) break;
            off -= n;
        }
        out->b = b;
        out->h = h;
        out->tok = tok;
        out->unit = int32_t(off);
        out->units = to - from;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- the kernel

template <int HD>
struct PaShape {
    static constexpr int kHalves = HD / 64;
    static constexpr int kStageBytes = kPaTile * HD * 2;
    static constexpr int kStages = HD == 128 ? 5 : 10;
    static constexpr int kQTileBytes = kPaTile * HD * 2;
    static constexpr int kTiles = 2 * kQTileBytes + kStages * kStageBytes;
};

struct PaShared {
    uint64_t q_full, q_empty;
    uint64_t kv_full[10], kv_empty[10];
    uint64_t s_full[2], p_ready[2], o_full[2], o_empty[2];
    uint64_t ml_full[2], drain;
    PaStart start;
    int64_t warp_sums[kPaThreads / 32];
    uint32_t tmem;
    int stop;
    float2 ml[2][kPaTile];  // stream 1's maximum and sum of a single item, by item parity
};

// The part of an item that this CTA does: KV tiles [first, first + n) of it.
struct PaPart {
    int32_t first, n;
    bool head, tail;  // begins / ends the item
};
__device__ __forceinline__ PaPart pa_part(const PaItem &it, int32_t unit, int64_t units_left) {
    PaPart p;
    const int32_t have = it.units - unit;
    const int32_t take = units_left < have ? int32_t(units_left) : have;
    p.head = unit == 0;
    p.tail = unit + take == it.units;
    if (it.dual) {
        p.first = unit;
        p.n = take;
    } else {
        p.first = 2 * unit;
        const int32_t end = 2 * (unit + take) < it.tiles ? 2 * (unit + take) : it.tiles;
        p.n = end - p.first;
    }
    return p;
}

template <int HD, bool BF16, bool CAP>
__global__ void __launch_bounds__(kPaThreads, 1) paged_attention_kernel(const __grid_constant__ PaArgs a) {
    using S = PaShape<HD>;
    // tiles on 1024-byte boundaries: the swizzle pattern is one of addresses
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PaShared &sh = *reinterpret_cast<PaShared *>(smem_raw + S::kTiles);
    const uint32_t q_smem = smem_addr(smem_raw);
    const uint32_t kv_smem = q_smem + 2 * S::kQTileBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t kO = 256;  // TMEM column of O0; O1 follows

    if (threadIdx.x == 0) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i], 4);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.o_empty[i], 4);
            mbar_init(&sh.ml_full[i], 4);
        }
        mbar_init(&sh.drain, 1);
        fence_mbar_init();
        sh.stop = 0;
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_before();
    }
    if (warp == 9 && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &a.q : lane == 1 ? &a.k : &a.v;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    pdl_wait();
    pa_cut(a, &sh.start, sh.warp_sums);  // synchronises the CTA
    tc_after();
    const uint32_t tmem = sh.tmem;
    volatile int *stop = &sh.stop;
    const PaStart st = sh.start;
    int32_t issued = 0;  // loader: ring entries issued, for the clean-up below

    if (threadIdx.x == 0) {
        int32_t *m = a.meta + blockIdx.x * 8;
        m[kPmTail] = 0;
        m[kPmFirst] = st.units == 0 ? 3 : st.unit == 0 ? 0 : 2;
    }
    if (st.units > 0) {
        PaWalk w;
        w.b = st.b;
        w.h = st.h;
        w.tok = st.tok;
        w.s = pa_seq(a, w.b, false);
        int32_t unit = st.unit;
        int64_t left = st.units;

        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaLoadRegs));
            if (warp == 8) {
                // ------------------------------------------------------ loads
                const int ppt = kPaTile >> a.page_log2;          // pages of a tile
                const uint32_t box = (128u << a.page_log2);      // bytes of one page's half
                uint32_t items = 0;
                bool ok = true;
                while (ok && left > 0) {
                    const PaItem it = pa_item(a, w.s, w.tok);
                    const PaPart pt = pa_part(it, unit, left);
                    const int32_t held = (w.s.len + (1 << a.page_log2) - 1) >> a.page_log2;
                    const int32_t *table = a.block_table + int64_t(w.b) * a.max_pages;
                    // the tensor-map row of lane's page of a tile; past the pool = zeros
                    auto page_row = [&](int32_t tile) {
                        const int32_t p = tile * ppt + lane;
                        int32_t row = a.pool_rows;
                        if (lane < ppt && p < held) {
                            const int32_t page = table[p];
                            if (uint32_t(page) < uint32_t(a.n_pages)) row = (page * a.n_kv + w.h) << a.page_log2;
                            else set_error(a.err, kErrBounds);
                        }
                        return row;
                    };
                    auto load = [&](const CUtensorMap *map, int32_t row) {
                        const int stage = issued % S::kStages;
                        if (issued >= S::kStages) ok = pa_wait(&sh.kv_empty[stage], ((issued / S::kStages) & 1) ^ 1, stop);
                        if (!ok) return;
                        if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[stage], S::kStageBytes);
                        __syncwarp();
                        if (lane < ppt) {
                            const uint32_t dst = kv_smem + stage * S::kStageBytes + lane * box;
#pragma unroll
                            for (int i = 0; i < S::kHalves; ++i)
                                tma_2d(dst + i * (kPaTile * 128), map, i * 64, row, &sh.kv_full[stage]);
                        }
                        ++issued;
                    };
                    const int32_t t0 = it.tile0 + pt.first;
                    // Q once the MMAs of the item before have read theirs
                    if (items > 0) ok = pa_wait(&sh.q_empty, (items - 1) & 1, stop);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t bytes = uint32_t(a.tile_tok * a.group) * 128u * S::kHalves;
                        mbar_arrive_expect_tx(&sh.q_full, it.dual ? 2 * bytes : bytes);
                        for (int d = 0; d < (it.dual ? 2 : 1); ++d)
                            for (int i = 0; i < S::kHalves; ++i)
                                tma_4d(q_smem + d * S::kQTileBytes + i * (kPaTile * 128), &a.q, i * 64, 0, w.h,
                                       w.s.q0 + w.tok + d * a.tile_tok, &sh.q_full);
                    }
                    __syncwarp();
                    ++items;
                    // K and V in the order the MMAs use them: dual K0 V0 K1 V1 ..,
                    // single K0 K1 V0 K2 V1 .. (K runs one tile further ahead)
                    const int ahead = it.dual ? 1 : 2;
                    int32_t row_k = page_row(t0), row_v = row_k;
                    load(&a.k, row_k);
                    int32_t row_k1 = 0;
                    if (ahead == 2 && pt.n > 1) {
                        row_k1 = page_row(t0 + 1);
                        if (ok) load(&a.k, row_k1);
                    }
                    for (int32_t i = 0; ok && i < pt.n; ++i) {
                        const int32_t next = i + ahead;
                        const int32_t row_n = next < pt.n ? page_row(t0 + next) : 0;
                        load(&a.v, row_v);
                        if (ok && next < pt.n) load(&a.k, row_n);
                        if (ahead == 1) {
                            row_v = row_n;
                        } else {
                            row_v = row_k1;
                            row_k1 = row_n;
                        }
                    }
                    left -= it.units - unit < left ? it.units - unit : left;
                    unit = 0;
                    if (left > 0) pa_next(a, w);
                }
            } else if (warp == 9) {
                // ------------------------------------------------------ MMAs
                constexpr uint32_t id_s = tc_idesc(BF16, 128, 128, false), id_o = tc_idesc(BF16, 128, HD, true);
                uint32_t items = 0, ring = 0, p_phase[2] = {0, 0}, o_items[2] = {0, 0};
                bool ok = true;
                auto stage_full = [&](uint32_t at) {
                    return pa_wait(&sh.kv_full[at % S::kStages], (at / S::kStages) & 1, stop);
                };
                while (ok && left > 0) {
                    const PaItem it = pa_item(a, w.s, w.tok);
                    const PaPart pt = pa_part(it, unit, left);
                    const int32_t steps = it.dual ? 2 * pt.n : pt.n;
                    auto at_k = [&](int32_t t) {
                        return ring + uint32_t(it.dual ? 2 * t : t < 2 ? t : 2 * t - 1);
                    };
                    auto at_v = [&](int32_t t) {
                        return ring + uint32_t(it.dual ? 2 * t + 1 : t < pt.n - 1 ? 2 * t + 2 : 2 * pt.n - 1);
                    };
                    // the last rows of the last page hold nothing the request wrote:
                    // rows [cut0, cut1) of that tile are cleared in V before use
                    const int32_t end_tile = w.s.len / kPaTile;
                    const int32_t cut0 = w.s.len % kPaTile;
                    const int32_t cut1 = ((cut0 + (1 << a.page_log2) - 1) >> a.page_log2) << a.page_log2;
                    auto issue_s = [&](int32_t j) {  // S of step j
                        const int d = j & 1;
                        const int32_t t = it.dual ? j >> 1 : j;
                        const uint32_t at = at_k(t);
                        ok = stage_full(at);
                        if (!ok) return;
                        tc_after();
                        if (lane == 0) {
                            const uint32_t qa = q_smem + (it.dual ? d : 0) * S::kQTileBytes;
                            const uint32_t ka = kv_smem + (at % S::kStages) * S::kStageBytes;
#pragma unroll
                            for (int kk = 0; kk < HD / 16; ++kk) {
                                const uint32_t off = (kk / 4) * (kPaTile * 128) + (kk % 4) * 32;
                                tc_mma_ss(tmem + d * 128, tc_desc(qa + off, 16, 1024), tc_desc(ka + off, 16, 1024), id_s,
                                          kk != 0);
                            }
                            if (!it.dual || d == 1) tc_commit(&sh.kv_empty[at % S::kStages]);
                            tc_commit(&sh.s_full[d]);
                            if (j == steps - 1) tc_commit(&sh.q_empty);
                        }
                        __syncwarp();
                    };
                    ok = pa_wait(&sh.q_full, items & 1, stop);
                    if (!ok) break;
                    ++items;
                    issue_s(0);
                    if (ok && steps > 1) issue_s(1);
                    for (int32_t j = 0; ok && j < steps; ++j) {
                        const int d = j & 1;
                        const int32_t t = it.dual ? j >> 1 : j;
                        const uint32_t at = at_v(t);
                        ok = stage_full(at);
                        if (!ok) break;
                        if (it.tile0 + pt.first + t == end_tile && cut0 < cut1 && (!it.dual || d == 0)) {
                            const uint32_t va = kv_smem + (at % S::kStages) * S::kStageBytes;
                            const int32_t pieces = (cut1 - cut0) * 8;
                            for (int h = 0; h < S::kHalves; ++h)
                                for (int32_t i = lane; i < pieces; i += 32)
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(va + h * (kPaTile * 128) + cut0 * 128 + i * 16),
                                                 "r"(0)
                                                 : "memory");
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                        }
                        ok = pa_wait(&sh.p_ready[d], p_phase[d], stop);
                        if (!ok) break;
                        p_phase[d] ^= 1;
                        if (j < 2) {  // the first write to O of this item: the one before must have been read
                            if (o_items[d] > 0) ok = pa_wait(&sh.o_empty[d], (o_items[d] - 1) & 1, stop);
                            if (!ok) break;
                        }
                        tc_after();
                        if (lane == 0) {
                            const uint32_t va = kv_smem + (at % S::kStages) * S::kStageBytes;
#pragma unroll
                            for (int kk = 0; kk < kPaTile / 16; ++kk)
                                tc_mma_ts(tmem + kO + d * HD, tmem + d * 128 + kk * 8,
                                          tc_desc(va + kk * 2048, kPaTile * 128, 1024), id_o, j >= 2 || kk != 0);
                            if (!it.dual || d == 1) tc_commit(&sh.kv_empty[at % S::kStages]);
                            if (j + 2 >= steps) tc_commit(&sh.o_full[d]);
                        }
                        __syncwarp();
                        if (j + 2 < steps) issue_s(j + 2);
                    }
                    ++o_items[0];
                    ++o_items[1];
                    ring += 2 * pt.n;
                    left -= it.units - unit < left ? it.units - unit : left;
                    unit = 0;
                    if (left > 0) pa_next(a, w);
                }
                if (!ok && lane == 0) tc_commit(&sh.drain);
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPaSoftRegs));
            // ------------------------------------------------------ softmax
            const int d = warp >> 2;                       // stream
            const int row = (warp & 3) * 32 + lane;        // row of the tile
            const uint32_t t_row = tmem + (uint32_t((warp & 3) * 32) << 16);
            const uint32_t t_s = t_row + d * 128;
            // f16 weights are scaled up so that small ones stay normal; a row's
            // weights then reach 2^(kLift + kSlack)
            constexpr float kLift = BF16 ? 0.0f : 8.0f, kSlack = BF16 ? 8.0f : 4.0f;
            const int32_t rtok = row / a.group, rhead = row - rtok * a.group;
            const bool in_tile = rtok < a.tile_tok;
            uint32_t s_phase = 0, o_phase[2] = {0, 0}, ml_phase = 0, ml_items = 0;
            bool ok = true;
            while (ok && left > 0) {
                const PaItem it = pa_item(a, w.s, w.tok);
                const PaPart pt = pa_part(it, unit, left);
                const int32_t tok = w.tok + (it.dual ? d * a.tile_tok : 0) + rtok;  // of the request
                const bool valid = in_tile && tok < w.s.fresh;
                const int32_t pos = w.s.len - w.s.fresh + tok;
                int64_t lo64 = a.window > 0 ? int64_t(pos) - a.window + 1 : 0;
                const int32_t lo = lo64 > 0 ? int32_t(lo64) : 0;
                const bool busy = __any_sync(0xffffffffu, valid);
                const int32_t n = it.dual ? pt.n : (pt.n - d + 1) / 2;  // tiles of this stream
                float ref = -INFINITY;  // reference maximum, log2 units, less kLift
                float2 sum2 = make_float2(0.0f, 0.0f);
                for (int32_t i = 0; i < n; ++i) {
                    const int32_t t = it.tile0 + pt.first + (it.dual ? i : 2 * i + d);
                    ok = pa_wait(&sh.s_full[d], s_phase, stop);
                    if (!ok) break;
                    s_phase ^= 1;
                    if (busy) {
                        tc_after();
                        float x[128];
#pragma unroll
                        for (int c = 0; c < 4; ++c) tc_ld32(t_s + c * 32, x + c * 32);
                        tc_wait_ld();
                        if (CAP) {
                            // softcap * tanh(s / softcap), with tanh(y) = 1 - 2 / (e^2y + 1)
#pragma unroll
                            for (int c = 0; c < 128; ++c) x[c] = 1.0f - __fdividef(2.0f, ex2(x[c] * a.cap_in) + 1.0f);
                        }
                        const int32_t key0 = t * kPaTile, hi_c = pos - key0, lo_c = lo - key0;
                        if (__any_sync(0xffffffffu, hi_c < kPaTile - 1 || lo_c > 0)) {
#pragma unroll
                            for (int c = 0; c < 128; ++c) x[c] = c <= hi_c && c >= lo_c ? x[c] : -INFINITY;
                        }
                        float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[2], x[3]), m2 = fmaxf(x[4], x[5]), m3 = fmaxf(x[6], x[7]);
#pragma unroll
                        for (int c = 8; c < 128; c += 8) {
                            m0 = fmaxf(m0, fmaxf(x[c], x[c + 1]));
                            m1 = fmaxf(m1, fmaxf(x[c + 2], x[c + 3]));
                            m2 = fmaxf(m2, fmaxf(x[c + 4], x[c + 5]));
                            m3 = fmaxf(m3, fmaxf(x[c + 6], x[c + 7]));
                        }
                        const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * a.scale_log2 - kLift;
                        // move the reference when a row grew past the slack
                        if (__any_sync(0xffffffffu, top > ref + kSlack || (ref == -INFINITY && top > -INFINITY))) {
                            const float now = fmaxf(ref, top);
                            if (i > 0) {
                                const float f = now == -INFINITY ? 1.0f : ex2(ref - now);
                                const float2 f2 = make_float2(f, f), z2 = make_float2(0.0f, 0.0f);
                                sum2 = fma2(sum2, f2, z2);
#pragma unroll
                                for (int c = 0; c < HD; c += 32) {
                                    float o[32];
                                    tc_ld32(t_row + kO + d * HD + c, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] *= f;
                                    tc_st32(t_row + kO + d * HD + c, o);
                                }
                            }
                            ref = now;
                        }
                        const float base = ref == -INFINITY ? 0.0f : ref;
                        const float2 sc = make_float2(a.scale_log2, a.scale_log2), nb = make_float2(-base, -base);
                        float2 acc[4] = {sum2, make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t p[32];
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                float2 v = fma2(make_float2(x[half * 64 + 2 * c], x[half * 64 + 2 * c + 1]), sc, nb);
                                v.x = ex2(v.x);
                                v.y = ex2(v.y);
                                acc[c & 3] = add2(acc[c & 3], v);
                                p[c] = pack2<BF16>(v.x, v.y);
                            }
                            tc_st32(t_s + half * 32, p);
                        }
                        sum2 = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
                        tc_wait_st();
                        tc_before();
                    }
                    __syncwarp();
                    if (lane == 0) pa_arrive(&sh.p_ready[d]);
                }
                if (!ok) break;
                float sum = sum2.x + sum2.y;

                // ---- the end of the item, or of this CTA's piece of it
                float other_ref = -INFINITY, other_sum = 0.0f;
                const bool two = !it.dual && pt.n > 1;  // a single item with a second stream
                if (two) {
                    if (d == 1) {
                        sh.ml[ml_items & 1][row] = make_float2(ref, sum);
                        __syncwarp();
                        if (lane == 0) pa_arrive(&sh.ml_full[ml_items & 1]);
                    } else {
                        ok = pa_wait(&sh.ml_full[ml_items & 1], ml_phase >> (ml_items & 1) & 1, stop);
                        if (!ok) break;
                        ml_phase ^= 1u << (ml_items & 1);
                        const float2 v = sh.ml[ml_items & 1][row];
                        other_ref = v.x;
                        other_sum = v.y;
                    }
                    ++ml_items;
                }
                if (it.dual || d == 0) {
                    ok = pa_wait(&sh.o_full[d], o_phase[d], stop);
                    if (!ok) break;
                    if (two) {
                        ok = pa_wait(&sh.o_full[1], o_phase[1], stop);
                        if (!ok) break;
                    }
                    if (busy) {
                        tc_after();
                        const float top = fmaxf(ref, other_ref), base = top == -INFINITY ? 0.0f : top;
                        float f0 = ex2(ref - base), f1 = two ? ex2(other_ref - base) : 0.0f;
                        sum = sum * f0 + other_sum * f1;
                        const bool whole = pt.head && pt.tail;
                        if (whole) {
                            if (a.sinks != nullptr && valid) {
                                // the sink joins the maximum and the sum (a row without rows stays zero)
                                const float sink = a.sinks[w.h * a.group + rhead] * 1.4426950408889634f;
                                const float all = fmaxf(top, sink), g = ex2(base - all);
                                if (top != -INFINITY) {
                                    sum = sum * g + ex2(sink - all);
                                    f0 *= g;
                                    f1 *= g;
                                }
                            }
                            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                            f0 *= inv;
                            f1 *= inv;
                        }
                        const int32_t slot = blockIdx.x * 2 + (pt.head ? 1 : 0);
                        const int32_t prow = (it.dual ? d * a.tile_tok * a.group : 0) + row;
                        if (!whole && valid) a.part_ml[int64_t(slot) * a.part_rows + prow] = make_float2(top, sum);
                        uint8_t *dst = static_cast<uint8_t *>(a.out) +
                                       ((int64_t(w.s.q0) + tok) * a.out_tok + int64_t(w.h * a.group + rhead) * a.out_head) * 2;
                        float *pdst = a.part_o + (int64_t(slot) * a.part_rows + prow) * HD;
#pragma unroll
                        for (int c = 0; c < HD; c += 32) {
                            float y[32];
                            __syncwarp();
                            tc_ld32(t_row + kO + d * HD + c, y);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] *= f0;
                            if (two) {
                                float z[32];
                                tc_ld32(t_row + kO + HD + c, z);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) y[e] += z[e] * f1;
                            }
                            if (valid && whole) {
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
                                    *reinterpret_cast<uint4 *>(dst + (c + e) * 2) =
                                        make_uint4(pack2<BF16>(y[e], y[e + 1]), pack2<BF16>(y[e + 2], y[e + 3]),
                                                   pack2<BF16>(y[e + 4], y[e + 5]), pack2<BF16>(y[e + 6], y[e + 7]));
                            } else if (valid) {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<float4 *>(pdst + c + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                            }
                        }
                        __syncwarp();
                        tc_before();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        // O1 first: the MMA warp takes O0 of a single item as a sign for both
                        if (!it.dual) pa_arrive(&sh.o_empty[1]);
                        pa_arrive(&sh.o_empty[d]);
                    }
                    if (threadIdx.x == 0) {
                        int32_t *m = a.meta + blockIdx.x * 8;
                        if (pt.head && !pt.tail) {
                            m[kPmTail] = 1;
                            m[kPmSeq] = w.b;
                            m[kPmHead] = w.h;
                            m[kPmTok] = w.tok;
                        }
                        if (!pt.head && pt.tail) m[kPmFirst] = 1;
                    }
                }
                o_phase[0] ^= 1;
                if (it.dual || two) o_phase[1] ^= 1;
                left -= it.units - unit < left ? it.units - unit : left;
                unit = 0;
                if (left > 0) pa_next(a, w);
            }
        }
    }
    // ---- the end: nothing may still be in flight into this CTA's memory
    __syncwarp();
    if (*stop != 0) {
        if (threadIdx.x == 0) set_error(a.err, kErrTimeout);
        if (warp == 8)
            for (int32_t i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
                mbar_wait_bounded(&sh.kv_full[i % S::kStages], (i / S::kStages) & 1, 500000000ull);
        if (warp == 9) mbar_wait_bounded(&sh.drain, 0, 500000000ull);
    }
    tc_before();
    __syncthreads();
    tc_after();
    pdl_trigger();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the pieces of a cut item: CTA (c, y) those of the item whose head piece
// CTA c of the attention left, a warp per query row.
template <int HD, bool BF16>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PaArgs a) {
    pdl_wait();
    const int c0 = blockIdx.x;
    const int32_t *m = a.meta + c0 * 8;
    if (m[kPmTail] == 0) return;
    const PaSeq s = pa_seq(a, m[kPmSeq], false);
    const int32_t h = m[kPmHead], tok0 = m[kPmTok];
    const PaItem it = pa_item(a, s, tok0);
    const int32_t rows = it.count * a.group;
    // slots of its pieces, in the order of the CTAs up to the one that ends it
    __shared__ int32_t slots[kPaCtas];
    __shared__ int32_t n_slots, last;
    const int32_t c = threadIdx.x;
    const int32_t first = c < kPaCtas ? a.meta[c * 8 + kPmFirst] : 3;
    if (c == 0) last = kPaCtas - 1;
    __syncthreads();
    if (c > c0 && first == 1) atomicMin(&last, c);
    __syncthreads();
    const bool mine = c == c0 || (c > c0 && c <= last && first != 3);
    __shared__ int32_t counts[8];
    const uint32_t vote = __ballot_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = __popc(vote);
    __syncthreads();
    int32_t rank = __popc(vote & ((1u << (threadIdx.x & 31)) - 1u));
    for (int i = 0; i < (threadIdx.x >> 5); ++i) rank += counts[i];
    if (mine) slots[rank] = c == c0 ? 2 * c + 1 : 2 * c;
    if (c == last) n_slots = rank + 1;
    __syncthreads();
    const int32_t n = n_slots;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kPer = HD / 32;
    for (int32_t r = blockIdx.y * 8 + warp; r < rows; r += gridDim.y * 8) {
        float top = -INFINITY;
        for (int32_t i = lane; i < n; i += 32) top = fmaxf(top, a.part_ml[int64_t(slots[i]) * a.part_rows + r].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, o[kPer] = {};
#pragma unroll 4
        for (int32_t i = 0; i < n; ++i) {
            const int64_t at = int64_t(slots[i]) * a.part_rows + r;
            const float2 ml = a.part_ml[at];
            const float f = ex2(ml.x - base);
            sum += ml.y * f;
            const float *p = a.part_o + at * HD + lane * kPer;
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] += p[e] * f;
        }
        const int32_t rtok = r / a.group, rhead = r - rtok * a.group;
        float g = 1.0f;
        if (a.sinks != nullptr && top != -INFINITY) {
            const float sink = a.sinks[h * a.group + rhead] * 1.4426950408889634f;
            const float all = fmaxf(top, sink);
            g = ex2(base - all);
            sum = sum * g + ex2(sink - all);
        }
        g *= sum == 0.0f ? 0.0f : 1.0f / sum;
        uint32_t *dst = reinterpret_cast<uint32_t *>(
            static_cast<uint8_t *>(a.out) +
            ((int64_t(s.q0) + tok0 + rtok) * a.out_tok + int64_t(h * a.group + rhead) * a.out_head + lane * kPer) * 2);
#pragma unroll
        for (int i = 0; i < kPer; i += 2) dst[i / 2] = pack2<BF16>(o[i] * g, o[i + 1] * g);
    }
}

template <int HD, bool BF16, bool CAP>
cudaError_t launch_paged_one(const PaArgs &a, cudaStream_t st) {
    constexpr int smem = PaShape<HD>::kTiles + int(sizeof(PaShared));
    static_assert(smem <= 227 * 1024, "shared memory of an SM");
    const auto kern = paged_attention_kernel<HD, BF16, CAP>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(kPaCtas), dim3(kPaThreads), smem, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_merge_kernel<HD, BF16>, dim3(kPaCtas, unsigned(ceil_div(a.part_rows, 64))), dim3(256), 0, st, a);
}

template <int HD>
cudaError_t launch_paged(const PaArgs &a, bool bf16, bool cap, cudaStream_t st) {
    if (bf16) return cap ? launch_paged_one<HD, true, true>(a, st) : launch_paged_one<HD, true, false>(a, st);
    return cap ? launch_paged_one<HD, false, true>(a, st) : launch_paged_one<HD, false, false>(a, st);
}

}  // namespace kvd
