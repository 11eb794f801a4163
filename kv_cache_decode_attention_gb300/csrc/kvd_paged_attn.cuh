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
// maximum, sum) in the workspace.  A call of at most kPaJoinRows query rows a KV
// head has them joined by the CTA that finishes the last of them (nobody waits
// for another CTA, and there is no second launch); larger calls, whose joins
// are work for more than one CTA, by paged_join_kernel.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax of stream 0 and 1, a thread per query row;
//   warps 8, 12     TMA loads of Q and K, and of V: tiles of 128 rows into one
//                   ring, page by page (a page that does not exist reads as
//                   zeros); small pages take many copies, hence two warps;
//   warps 9, 14     issue the MMAs of stream 0 and 1: S = Q K^T and O += P V, P
//                   from TMEM;
//   warp 10         clears the rows of V behind a request's last one;
//   warp 11         walks the CTA's share of the work and hands the items on;
//   warp 13         ends every wait if the CTA stops making steps.
// TMEM: S0 S1 (128 columns each; P overwrites the first 64) O0 O1.
// MMAs of one thread run in order, so S of a stream's next tile may be issued
// behind P V of its last one without a wait, and S being complete says that P V
// before it is: the softmax group may then rescale O in place.  It does so only
// when a row's maximum grew by more than 2^kSlack; until then the old one is
// as good a reference.
//
// Roundings.  Scores, maxima, sums, weights and O are f32.  The weights are
// rounded once to the pages' type, because the second product's operands have one
// type; the sum is taken of the weights before that, so each row's error is that
// of independent half steps.  f16 weights are held 2^8 higher: without that a
// weight below 2^-14 of the largest would lose bits.
//
// Bounds, and what was measured (GPU time on one GB300; a copy runs at 6.69 TB/s, a
// large bf16 product at 1934 TFLOP/s, 1753 after seconds at the power limit):
//   one new row for each of 64 requests of up to 16384 rows, 32 heads over 8: HBM;
//     346-350 us for 2.31 GB, 6.6-6.7 TB/s.  4 of 131072, 128 heads over 8: 306-311
//     us, 6.9-7.0 TB/s.  64 KB tiles, five 32 KB stages and equal shares of units
//     are what that takes: any two of K, V and the next K are under way.
//   4096 new rows of a prompt over 32768, 32 heads over 8: tensor cores; 1405-1420
//     us, 1450-1467 TFLOP/s, at the power limit (1510 us in passes that go on for
//     seconds).  A unit takes 1.8 us where its MMAs
//     alone need 1.1: a warp's looks at barriers and the hand-over of P are what is
//     left between them.  Head size 64 takes 1.6 us a unit for half the MMAs.
//   short requests: an item costs some 3 us beside its copies (from its first S to
//     its rows stored 2.6), and a CTA has its first scores some 4.5 us after it began:
//     barriers and TMEM 0.5, lengths and the cut 1.1, the first item, its page numbers
//     and the request for K 2, the copy and S 1.  A second kernel that joins takes 3
//     to 4 us more, 9.6 where seven chunks of up to 700 rows are cut.  One row over
//     1023 rows takes 14 us, one for each of 256 requests of 300 rows 96 (up to 300
//     rows: 72), for 64 busy of 4096 places 9 more than for 64 alone.
// Measured and not taken: two softmax groups for each stream, half a tile each
// (prompts -5%, drafts +7%, windows +11%); P handed over in halves (prompts +6%); a
// third buffer for S at head size 64 (long requests -1%, windows +4%); short items
// each on one stream (one-tile items -24%, drafts +2%, windows and prompts of 2000
// +2%); one warp for both streams' MMAs (requests of up to 300 rows +16%, mixed prompts +3%,
// windows -1%, 2000-row prompts at head size 64 -2%).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kvd_internal.cuh"

namespace kvd {

constexpr int kPaCtas = 152;       // one per SM; also fixes the cut of the work
constexpr int kPaThreads = 512;    // warp 15 only fills its warpgroup
// Registers a thread: the launch gives 512 x 128; the softmax warpgroups trade up.
constexpr int kPaRegs = 128, kPaSoftRegs = 184, kPaLoadRegs = 72;
static_assert(2 * kPaSoftRegs + 2 * kPaLoadRegs <= 4 * kPaRegs, "setmaxnreg shares");
constexpr int kPaTile = 128;       // query rows of a tile, and KV rows of a tile
constexpr int kPaMaxRows = 2 * kPaTile;
// A CTA passes requests without new rows one after another.  So many take 2.8 ms,
// well below the two seconds without a step after which it would give up.
constexpr int kPaMaxSeq = 1 << 20;
// Joining 16 rows of 19 pieces takes one CTA some 3 us, as long as a second
// launch; 256 rows of 2 pieces took it 20 us, and the kernel 3 to 4.
constexpr int kPaJoinRows = 16;

// A cut item as paged_join_kernel finds it; n = 0: none.
struct PaPiecesOf {
    int64_t unit0, total;
    int32_t units, rows, q_row, kv_head, n, pad;
};

struct PaArgs {
    CUtensorMap q, k, v;
    const int32_t *block_table, *cu_new, *seq_len;
    void *out;
    int64_t out_tok, out_head;
    const float *sinks;
    float *part_o;     // [2 * kPaCtas][part_rows][hd]
    float2 *part_ml;   // [2 * kPaCtas][part_rows]: reference maximum (log2 units), sum
    uint64_t *tickets; // [kPaCtas]: of the cut item that begins in the CTA, nonce << 8 | pieces done
    uint64_t nonce;    // of the launch, below 2^56
    PaPiecesOf *cut;   // [kPaCtas]: the cut item that begins in each CTA
    int32_t join_here; // by the last finisher
    int32_t give_up;   // for tests: the CTA whose watch gives up so many ns after it began, or -1
    uint32_t give_up_ns;
    uint32_t *err;
    int64_t window;    // below 2^31; 0 = none
    int32_t n_seq, n_tokens, n_kv, group, tile_tok, max_pages, n_pages, page_log2;
    int32_t part_rows, pool_rows;
    float scale_log2;  // scale * log2 e (softcap 0), or softcap * log2 e
    float cap_in;      // softcap > 0: 2 * scale * log2 e / softcap
    float cap_mul;     // scale * log2 e: the polynomial's first coefficient
    float cap_near;    // below it in size, a score's tanh is the polynomial (negative: never)
    float cap_hidden;  // what a masked score becomes before it is capped
    float cap_c[4];    // its other coefficients, in powers of the score
};

// A ticket that carries another nonce counts as zero, so the workspace needs no
// initialisation; whoever joins the pieces sets it to 0 for a graph's next
// replay, which comes with the same nonce.  (So every piece has its ticket taken,
// those of a CTA that gave up too.)  A piece of CTA c is kept in slot 2 c + 1 if it
// begins its item, else in slot 2 c.

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


__device__ __forceinline__ void tc_st32(uint32_t addr, const float *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const float *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]) : "memory");
}

// Instruction descriptor of kind::f16: f32 accumulator, M x N, B MN-major or not.
__host__ __device__ constexpr uint32_t tc_idesc(bool bf16, int m, int n, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// One lane of a converged warp; always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
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
// Arrive once on bar when every MMA the elected lane has issued so far is complete.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    if (elect_one())
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
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
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// tanh(y) / y in powers of y^2, fitted to a relative error of 1.3e-8 up to |y| = 1/2.
constexpr double kPaTanh[4] = {-0.3333306908607483, 0.13324779272079468, -0.05298607423901558, 0.017135001718997955};

// tanh(y) of x = 2 y log2 e, as 1 - 2 / (e^2y + 1): two special-function
// instructions, right to some 2^-23 of 1.
__device__ __forceinline__ float pa_tanh(float x) { return fmaf(rcp(ex2(x) + 1.0f), -2.0f, 1.0f); }
// The same to some 2^-21 of the result: the polynomial where y is small.  (As all
// scores are to a cap far out of reach, of which 2^-23 is more than they are.)
__device__ __forceinline__ float pa_tanh_of_any(float x) {
    const float y = x * 0.34657359027997264f, z = y * y;
    const float p = fmaf(fmaf(fmaf(fmaf(float(kPaTanh[3]), z, float(kPaTanh[2])), z, float(kPaTanh[1])), z, float(kPaTanh[0])), z, 1.0f) * y;
    return fabsf(y) < 0.5f ? p : pa_tanh(x);
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

// A wait that gives up once *stop is set, which the watching warp does when the
// CTA has made no step for two seconds.  Small on purpose: it stands in twenty
// places, and code that does not stay in the instruction caches is paid again
// for every item.
__device__ __forceinline__ bool pa_wait_one(uint64_t *bar, uint32_t parity, volatile int *stop) {
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (*stop != 0) return false;
    return true;
}
// Looks at three barriers at once; a bit for each whose phase is over.  While the tensor
// cores read both operands from shared memory they leave little of its
// bandwidth, and one such look takes some 200 cycles: the MMA warps take their
// looks together.
__device__ __forceinline__ uint32_t pa_test3(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, uint64_t *b2, uint32_t p2) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b, c;\n\t.reg .b32 x, y, z;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 a, [%1], %2;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 b, [%3], %4;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 c, [%5], %6;\n\t"
        "selp.u32 x, 1, 0, a;\n\tselp.u32 y, 2, 0, b;\n\tselp.u32 z, 4, 0, c;\n\t"
        "or.b32 x, x, y;\n\tor.b32 %0, x, z;\n\t}"
        : "=r"(r)
        : "r"(smem_addr(b0)), "r"(p0), "r"(smem_addr(b1)), "r"(p1), "r"(smem_addr(b2)), "r"(p2)
        : "memory");
    return __reduce_and_sync(0xffffffffu, r);
}
// A wait with one answer for a whole warp.
__device__ __forceinline__ bool pa_wait(uint64_t *bar, uint32_t parity, volatile int *stop) {
    return __all_sync(0xffffffffu, pa_wait_one(bar, parity, stop));
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Bits lo .. hi of 32 (none if lo > hi or both lie outside): the columns a row sees.
__device__ __forceinline__ uint32_t pa_seen(int32_t lo, int32_t hi) {
    const uint32_t to = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1u;
    const uint32_t from = lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
    return to & from;
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
    PaSeq s;                  // its request
    int64_t units;            // units of this CTA
    int64_t from, total;      // its first unit, and all units
};

// The cut: CTA c of kPaCtas takes units [c W / kPaCtas, (c + 1) W / kPaCtas) of
// the W there are.  All threads; the result is in shared memory.
__device__ __forceinline__ void pa_cut(const PaArgs &a, PaStart *out, int64_t *warp_sums) {
    const int per = (a.n_seq + kPaThreads - 1) / kPaThreads;
    const int b0 = threadIdx.x * per < a.n_seq ? threadIdx.x * per : a.n_seq;
    const int b1 = b0 + per < a.n_seq ? b0 + per : a.n_seq;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    // first turn: this thread's units; second, for the thread whose requests
    // hold the CTA's first unit: where it is in them
    int64_t mine = 0, off = 0, u = 0, from = 0, to = 0;
    uint64_t total = 0;
    PaSeq s = {0, 0, 0};
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        int b = b0;
        if (turn == 0 || per > 1) {  // a thread's only request is still at hand
#pragma unroll 1
            for (; b < b1; ++b) {
                s = pa_seq(a, b, turn == 0 && blockIdx.x == 0);
                u = 0;
#pragma unroll 1
                for (int32_t tok = 0; tok < s.fresh; tok += 2 * a.tile_tok) u += pa_item(a, s, tok).units;
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
            for (;; tok += 2 * a.tile_tok) {
                const int32_t n = pa_item(a, s, tok).units;
                if (off < n) break;
                off -= n;
            }
            *out = PaStart{b, h, tok, int32_t(off), s, to - from, from, int64_t(total)};
            break;
        }
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) warp_sums[w] = x;
        if (threadIdx.x == 0) out->units = 0;
        __syncthreads();
        constexpr int kWarps = kPaThreads / 32;
        int64_t before = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
        for (int d = 1; d < kWarps; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += y;
        }
        total = __shfl_sync(0xffffffffu, before, kWarps - 1);
        before = __shfl_sync(0xffffffffu, before, w > 0 ? w - 1 : 0);
        before = (w > 0 ? before : 0) + x - mine;
        from = total * blockIdx.x / kPaCtas;
        to = total * (blockIdx.x + 1) / kPaCtas;
        off = from - before;
        if (from >= to || off < 0 || off >= mine) break;
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

// One item as the other warps see it; n = 0 ends the work.
struct PaJob {
    int32_t n;                 // KV tiles of this CTA's part of it
    int32_t tile0;             // the first of them
    int32_t tail;              // which of them holds the request's short last page, or -1
    int32_t dual, head, whole; // two query tiles; begins here; begins and ends here
    int32_t seq, kv_head, tok; // request, KV head, first token in its new rows
    int32_t q0, fresh, len;    // as PaSeq
    int32_t count, units;      // tokens and units of the whole item
    int64_t unit0;             // its first unit of all
};
constexpr int kPaJobs = 4;

struct PaShared {
    uint64_t job_full[kPaJobs], job_empty[kPaJobs];
    PaJob job[kPaJobs];
    uint64_t q_full, q_empty;
    uint64_t kv_full[10], kv_empty[10];
    uint64_t s_full[2], p_ready[2], o_full[2], o_empty[2];
    uint64_t ml_full[2], tail_go[2], tail_ready[2], pace[2], piece_done, verdict, all_done, drain[2];
    PaStart start;
    int64_t warp_sums[kPaThreads / 32];
    uint32_t tmem;
    int join;         // the verdict: this CTA joins the pieces
    int tickets;      // that the CTA has taken
    int stop, steps;  // the watch: give up; changes with every K tile that is loaded
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

// What the MMA thread keeps: the ring's cursor (loads are used in their order,
// dual K0 V0 K1 V1 .., single K0 K1 V0 K2 V1 ..) and the operands' bases.
template <int HD, bool BF16>
struct PaIssue {
    using S = PaShape<HD>;
    PaShared &sh;
    const uint32_t tmem, q, kv;
    volatile int *stop;
    uint32_t stage = 0, phase = 0;
    __device__ PaIssue(PaShared &s, uint32_t q_smem, uint32_t kv_smem, uint32_t t, volatile int *st)
        : sh(s), tmem(uni(t)), q(uni((q_smem & 0x3ffffu) >> 4)), kv(uni((kv_smem & 0x3ffffu) >> 4)), stop(st) {}
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) { return pa_wait(bar, parity, stop); }
    __device__ __forceinline__ bool wait_stage() { return pa_wait(&sh.kv_full[stage], phase, stop); }
    __device__ __forceinline__ uint32_t take() {
        const uint32_t at = stage;
        if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1;
        }
        return at;
    }
    // A tile of the other stream's: let go of behind this one's own, so that stages
    // become empty in the ring's order, which the loading warps count on.
    __device__ __forceinline__ bool skip() {
        if (!wait_stage()) return false;
        tc_commit(&sh.kv_empty[take()]);
        return true;
    }
    // the stage after the next one
    __device__ __forceinline__ uint32_t after() const { return stage + 1 == S::kStages ? 0 : stage + 1; }
    __device__ __forceinline__ uint32_t phase_after() const { return stage + 1 == S::kStages ? phase ^ 1 : phase; }
    // Shared-memory matrix descriptor, 128-byte swizzle, groups of eight rows
    // 1024 bytes apart; for MN-major operands lbo = bytes between runs of 64.
    static __device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t lbo) {
        constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
        return (uint64_t(hi) << 32) | (uint64_t(lbo >> 4) << 16) | lo;
    }
    // S of stream d = Q tile qt x K in stage k
    __device__ __forceinline__ void score(int d, int qt, uint32_t k) const {
        constexpr uint32_t id = tc_idesc(BF16, 128, 128, false);
        const uint64_t qd = desc(uni(q + qt * (S::kQTileBytes >> 4)), 16), kd = desc(uni(kv + k * (S::kStageBytes >> 4)), 16);
        tc_after();
        if (!elect_one()) return;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
            constexpr uint32_t kHalf = kPaTile * 128 >> 4;
            const uint32_t off = (kk / 4) * kHalf + (kk % 4) * 2;
            tc_mma_ss(tmem + d * 128, qd + off, kd + off, id, kk != 0);
        }
    }
    // O of stream d (+)= P x V in stage v
    __device__ __forceinline__ void value(int d, uint32_t v, bool more) const {
        constexpr uint32_t id = tc_idesc(BF16, 128, HD, true);
        const uint64_t vd = desc(uni(kv + v * (S::kStageBytes >> 4)), kPaTile * 128);
        tc_after();
        if (!elect_one()) return;
#pragma unroll
        for (int kk = 0; kk < kPaTile / 16; ++kk)
            tc_mma_ts(tmem + 256 + d * HD, tmem + d * 128 + kk * 8, vd + kk * (2048 >> 4), id, more || kk != 0);
    }
};
// The part's tile in which the request's last page ends short, or -1.
__device__ __forceinline__ int32_t pa_tail_tile(const PaArgs &a, const PaSeq &s, const PaItem &it, const PaPart &pt) {
    const int32_t t = s.len / kPaTile - it.tile0 - pt.first;
    return t >= 0 && t < pt.n && (s.len & ((1 << a.page_log2) - 1)) != 0 ? t : -1;
}

// The CTAs that hold pieces of a cut item.  With W units in all, unit u lies in
// CTA ceil((u + 1) kPaCtas / W) - 1; with fewer units than CTAs every unit has
// one of its own, else every CTA between the first and the last has a piece.
static __device__ __noinline__ int32_t pa_cta_of(int64_t u, int64_t total) {
    return int32_t((uint64_t(u + 1) * kPaCtas + total - 1) / uint64_t(total)) - 1;
}
struct PaPieces {
    int32_t first, n, sparse, unit0;  // sparse = units in all, if fewer than CTAs, else 0
    __device__ __forceinline__ PaPieces(int64_t unit0_, int32_t units, int64_t total) {
        first = pa_cta_of(unit0_, total);
        sparse = total < kPaCtas ? int32_t(total) : 0;
        unit0 = int32_t(unit0_);
        n = sparse != 0 ? units : pa_cta_of(unit0_ + units - 1, total) - first + 1;
    }
    __device__ __forceinline__ int64_t slot(int32_t i) const {
        if (i == 0) return 2 * first + 1;
        const int32_t c = sparse != 0 ? (uint32_t(unit0 + i + 1) * kPaCtas + sparse - 1) / uint32_t(sparse) - 1 : first + i;
        return 2 * c;
    }
};

// One more piece of the item is done: whether it was the last.  `old` is what
// the ticket was a while ago; a wrong guess costs one more turn.
static __device__ __noinline__ bool pa_ticket(uint64_t *word, uint64_t nonce, int32_t n, uint64_t old) {
    uint64_t now;
    for (;;) {
        now = (old >> 8 == nonce ? old : nonce << 8) + 1;
        // n <= 152 pieces fit the low byte; the last one leaves 0 for a replay
        uint64_t got;
        asm volatile("atom.acq_rel.gpu.global.cas.b64 %0, [%1], %2, %3;"
                     : "=l"(got)
                     : "l"(word), "l"(old), "l"(int32_t(now & 255u) == n ? uint64_t(0) : now)
                     : "memory");
        if (got == old) break;
        old = got;
    }
    return int32_t(now & 255u) == n;
}

// Take the tickets that a CTA that gave up still owes, all but its first `taken`:
// nobody joins for it (the error word tells), but the words come to their 0.
static __device__ __noinline__ void pa_owed_tickets(const PaArgs &a, const PaStart &st, int32_t taken) {
    PaWalk w = {st.b, st.h, st.tok, st.s};
    int32_t unit = st.unit;
    for (int64_t left = st.units; left > 0;) {
        const PaItem it = pa_item(a, w.s, w.tok);
        const PaPart pt = pa_part(it, unit, left);
        if (!(pt.head && pt.tail) && --taken < 0) {
            const PaPieces pieces(st.from + (st.units - left) - unit, it.units, st.total);
            pa_ticket(a.tickets + pieces.first, a.nonce, pieces.n, 0);
        }
        left -= it.units - unit;
        unit = 0;
        if (left > 0) pa_next(a, w);
    }
}

// Row r of a cut item from its pieces, by a warp whose lanes stand for columns,
// four pieces under way at a time.
template <int HD, bool BF16>
__device__ __forceinline__ void pa_join_row(const PaArgs &a, const PaPieces &pieces, int32_t r, int32_t q_row, int32_t kv_head) {
    constexpr int kPer = HD / 32;
    const int32_t col = int32_t(threadIdx.x & 31) * kPer;
    float top = -INFINITY, sum = 0.0f, o[kPer] = {};
#pragma unroll 1
    for (int32_t i0 = 0; i0 < pieces.n; i0 += 4) {
        float2 ml[4];
        float v[4][kPer] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ml[i] = make_float2(-INFINITY, 0.0f);
            if (i0 + i >= pieces.n) continue;
            const int64_t at = pieces.slot(i0 + i) * a.part_rows + r;
            ml[i] = __ldcg(&a.part_ml[at]);
            const float *p = a.part_o + at * HD + col;
            if constexpr (kPer == 4) *reinterpret_cast<float4 *>(v[i]) = __ldcg(reinterpret_cast<const float4 *>(p));
            else *reinterpret_cast<float2 *>(v[i]) = __ldcg(reinterpret_cast<const float2 *>(p));
        }
        const float now = fmaxf(max3(top, ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), base = now == -INFINITY ? 0.0f : now;
        const float f0 = ex2(top - base);
        sum *= f0;
#pragma unroll
        for (int c = 0; c < kPer; ++c) o[c] *= f0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = ex2(ml[i].x - base);
            sum += ml[i].y * f;
#pragma unroll
            for (int c = 0; c < kPer; ++c) o[c] += v[i][c] * f;
        }
        top = now;
    }
    const int32_t rtok = r / a.group, head = kv_head * a.group + r - rtok * a.group;
    float g = 1.0f;
    if (a.sinks != nullptr && top != -INFINITY) {
        const float sink = a.sinks[head] * 1.4426950408889634f, all = fmaxf(top, sink);
        g = ex2(top - all);
        sum = sum * g + ex2(sink - all);
    }
    g *= sum == 0.0f ? 0.0f : 1.0f / sum;
    uint8_t *dst = static_cast<uint8_t *>(a.out) + ((int64_t(q_row) + rtok) * a.out_tok + int64_t(head) * a.out_head + col) * 2;
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<BF16>(o[0] * g, o[1] * g), pack2<BF16>(o[2] * g, o[3] * g));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack2<BF16>(o[0] * g, o[1] * g);
}

// CTA (c, y) joins rows of the cut item that begins in CTA c.
template <int HD, bool BF16>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PaArgs a) {
    pdl_wait();
    const PaPiecesOf cut = a.cut[blockIdx.x];
    if (cut.n == 0) return;
    const PaPieces pieces(cut.unit0, cut.units, cut.total);
    for (int32_t r = blockIdx.y * 8 + (threadIdx.x >> 5); r < cut.rows; r += gridDim.y * 8)
        pa_join_row<HD, BF16>(a, pieces, r, cut.q_row, cut.kv_head);
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
        mbar_init(&sh.q_empty, 2);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i], 4);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.o_empty[i], 4);
            mbar_init(&sh.ml_full[i], 4);
            mbar_init(&sh.tail_go[i], 1);
            mbar_init(&sh.pace[i], 1);
            mbar_init(&sh.tail_ready[i], 1);
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < kPaJobs; ++i) {
            mbar_init(&sh.job_full[i], 1);
            mbar_init(&sh.job_empty[i], 13);  // two of loads, two of MMAs, ends of V, eight softmax warps
        }
        mbar_init(&sh.piece_done, 4);
        mbar_init(&sh.verdict, 1);
        mbar_init(&sh.all_done, 14);  // every warp but 13 and 15
        fence_mbar_init();
        sh.stop = 0;
        sh.steps = 0;
        sh.tickets = 0;
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
    // copies asked for, for the clean-up below: bits of the stages (bit 16: Q) and the parities of their last ones
    uint32_t loaded = 0, parity = 0;

    if (a.join_here == 0 && warp == 11 && lane == 0) a.cut[blockIdx.x].n = 0;
    if (st.units > 0) {
        // the next item: its record, read in place until job_empty is told
        uint32_t job_at = 0;
        auto next_job = [&](bool &ok) -> const PaJob & {
            ok = pa_wait(&sh.job_full[job_at % kPaJobs], job_at / kPaJobs & 1, stop);
            return sh.job[job_at++ % kPaJobs];
        };
        auto done_job = [&]() {
            __syncwarp();
            if (lane == 0) pa_arrive(&sh.job_empty[(job_at - 1) % kPaJobs]);
        };

        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaLoadRegs));
            if (warp == 8 || warp == 12) {
                // ------------------------------------------------------ loads
                const int ppt = kPaTile >> a.page_log2;          // pages of a tile
                const uint32_t box = 128u << a.page_log2;        // bytes of one page's half
                const bool v_warp = warp == 12;
                const CUtensorMap *map = v_warp ? &a.v : &a.k;
                uint32_t items = 0, ring = 0;
                bool ok = true;
                for (;;) {
                    const PaJob &job = next_job(ok);
                    if (!ok || job.n == 0) break;
                    const int32_t n = job.n, t0 = job.tile0, h = job.kv_head;
                    const bool dual = job.dual != 0;
                    const int32_t held = (job.len + (1 << a.page_log2) - 1) >> a.page_log2, q_row = job.q0 + job.tok;
                    const int32_t *table = a.block_table + int64_t(job.seq) * a.max_pages;
                    done_job();
                    // the tensor-map row of lane's page of a tile; past the pool = zeros
                    auto page_row = [&](int32_t tile) {
                        const int32_t p = tile * ppt + lane;
                        int32_t row = a.pool_rows;
                        if (lane < ppt && p < held) {
                            const int32_t page = table[p];
                            if (uint32_t(page) < uint32_t(a.n_pages)) row = (page * a.n_kv + h) << a.page_log2;
                            else set_error(a.err, kErrBounds);
                        }
                        return row;
                    };
                    // places in the ring, in the order the MMAs use them: dual K0 V0 K1
                    // V1 .., single K0 K1 V0 K2 V1 .. (K runs one tile further ahead)
                    int32_t row = page_row(t0);
                    for (int32_t t = 0; t < n; ++t) {
                        const int32_t now = row;
                        if (t + 1 < n) row = page_row(t0 + t + 1);  // looked up while this one waits
                        const uint32_t at = ring + uint32_t(v_warp ? (dual ? 2 * t + 1 : t < n - 1 ? 2 * t + 2 : 2 * n - 1)
                                                                   : (dual ? 2 * t : t < 2 ? t : 2 * t - 1));
                        const uint32_t stage = at % S::kStages, turn = at / S::kStages;
                        if (turn > 0) ok = pa_wait(&sh.kv_empty[stage], (turn & 1) ^ 1, stop);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[stage], S::kStageBytes);
                        __syncwarp();
                        if (lane < ppt) {
                            const uint32_t dst = kv_smem + stage * S::kStageBytes + lane * box;
#pragma unroll 1
                            for (int i = 0; i < S::kHalves; ++i)
                                tma_2d(dst + i * (kPaTile * 128), map, i * 64, now, &sh.kv_full[stage]);
                        }
                        loaded |= 1u << stage;
                        if (lane == 0 && !v_warp) *static_cast<volatile int *>(&sh.steps) = int(ring) + t;
                        parity = (parity & ~(1u << stage)) | (turn & 1) << stage;
                        if (t == 0 && !v_warp) {
                            // Q once the MMAs of the item before have read theirs
                            if (items > 0) ok = pa_wait(&sh.q_empty, (items - 1) & 1, stop);
                            if (!ok) break;
                            if (lane == 0) {
                                const uint32_t bytes = uint32_t(a.tile_tok * a.group) * 128u * S::kHalves;
                                mbar_arrive_expect_tx(&sh.q_full, dual ? 2 * bytes : bytes);
#pragma unroll 1
                                for (int i = 0; i < (dual ? 2 * S::kHalves : S::kHalves); ++i)
                                    tma_4d(q_smem + i * (kPaTile * 128), &a.q, i % S::kHalves * 64, 0, h,
                                           q_row + i / S::kHalves * a.tile_tok, &sh.q_full);
                            }
                            __syncwarp();
                            loaded |= 1u << 16;
                            parity = (parity & ~(1u << 16)) | (items & 1) << 16;
                            ++items;
                        }
                    }
                    ring += 2 * n;
                    if (!ok) break;
                }
            } else if (warp == 9 || warp == 14) {
                // ------------------------------------------------------ MMAs
                // A warp for each stream.  Between two batches of MMAs come looks at
                // barriers, which queue up behind the batch: the other warp's batches
                // fill that time.
                PaIssue<HD, BF16> mma(sh, q_smem, kv_smem, tmem, stop);
                const uint32_t d = uni(warp == 14 ? 1 : 0);
                uint32_t items = 0, uses = 0, tails = 0, p_phase = 0, pairs = 0;  // uses: items with a tile for this stream
                bool ok = true;
                for (;;) {
                    ok = mma.wait(&sh.job_full[job_at % kPaJobs], job_at / kPaJobs & 1);
                    if (!ok) break;
                    const PaJob &job = sh.job[job_at % kPaJobs];
                    const int32_t n = uni(job.n), tail = uni(job.tail);
                    const bool dual = uni(job.dual) != 0;
                    ++job_at;
                    done_job();
                    if (n == 0) break;
                    ok = mma.wait(&sh.q_full, items & 1);
                    if (!ok) break;
                    // Step j: P V of tile j, then S of this stream's next tile.  Of a single
                    // item's tiles a stream uses every other one; it waits for the rest and
                    // lets go of them, so that it sees every turn of the ring.
                    const int32_t next = dual ? 1 : 2;
                    for (int32_t j = -next; j < n; ++j) {
                        const bool more = j + next < n;
                        if (!dual && (uint32_t(j) & 1) != d) {
                            if (j >= 0) ok = mma.skip();
                            if (ok && more) ok = mma.skip();
                            if (!ok) break;
                            continue;
                        }
                        uint32_t is = 0, v = 0;  // bits: V there, P there, next K there
                        if (j >= 0) {
                            is = pa_test3(&sh.kv_full[mma.stage], mma.phase, &sh.p_ready[d], p_phase, &sh.kv_full[mma.after()], mma.phase_after());
                            if ((is & 1) == 0) ok = mma.wait_stage();
                            // it ends short: cleared first.  (Of a dual item at stream 0's wish,
                            // after whose turn stream 1's comes.)
                            if (ok && j == tail && (!dual || d == 0)) {
                                if (elect_one()) pa_arrive(&sh.tail_go[d]);
                                ok = mma.wait(&sh.tail_ready[d], tails++ & 1);
                            }
                            v = mma.take();
                            // before the first write to O the last item's must have been read
                            if (ok && j < next && uses > 0) ok = mma.wait(&sh.o_empty[d], (uses - 1) & 1);
                            if (ok && (is & 2) == 0) ok = mma.wait(&sh.p_ready[d], p_phase);
                            // the streams of a dual item take turns: one that ran ahead would
                            // leave the other to end the item alone
                            if (ok && dual && (d == 1 || pairs > 0)) ok = mma.wait(&sh.pace[d ^ 1], (pairs - (d ^ 1)) & 1);
                            if (!ok) break;
                            p_phase ^= 1;
                            mma.value(d, v, j >= next);
                            if (!more) tc_commit(&sh.o_full[d]);
                        }
                        if (more) {
                            if ((is & 4) == 0) ok = mma.wait_stage();
                            if (!ok) break;
                            const uint32_t k = mma.take();
                            mma.score(d, dual ? d : 0, k);
                            tc_commit(&sh.s_full[d]);
                            tc_commit(&sh.kv_empty[k]);
                            if (j + 2 * next >= n) tc_commit(&sh.q_empty);
                        }
                        if (j >= 0) tc_commit(&sh.kv_empty[v]);
                        if (dual && j >= 0) {
                            if (elect_one()) pa_arrive(&sh.pace[d]);
                            ++pairs;
                        }
                    }
                    if (!ok) break;
                    if (!dual && n == 1 && d == 1) {  // no tile for this stream
                        if (elect_one()) pa_arrive(&sh.q_empty);
                    } else {
                        ++uses;
                    }
                    ++items;
                }
            } else if (warp == 10) {
                // ------------------------------------------------------ ends of V
                // Rows of a request's last page behind its last row hold nothing;
                // their weights are zero, but zero times NaN is not: they are
                // cleared after the copy and before the MMA, whose thread says when.
                uint32_t ring = 0, tails = 0;  // bits: parity of each stream's next one
                bool ok = true;
                for (;;) {
                    const PaJob &job = next_job(ok);
                    if (!ok || job.n == 0) break;
                    const int32_t t = job.tail, n = job.n, row0 = job.len % kPaTile;
                    const bool dual = job.dual != 0;
                    done_job();
                    if (t >= 0) {
                        const int s = dual ? 0 : t & 1;
                        ok = pa_wait(&sh.tail_go[s], tails >> s & 1, stop);
                        if (!ok) break;
                        tails ^= 1u << s;
                        const uint32_t stage = (ring + uint32_t(dual ? 2 * t + 1 : t < n - 1 ? 2 * t + 2 : 2 * n - 1)) % S::kStages;
                        const int32_t row1 = ((row0 + (1 << a.page_log2) - 1) >> a.page_log2) << a.page_log2;
                        const uint32_t va = kv_smem + stage * S::kStageBytes + row0 * 128;
                        for (int h = 0; h < S::kHalves; ++h)
                            for (int32_t i = lane; i < (row1 - row0) * 8; i += 32)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(va + h * (kPaTile * 128) + i * 16), "r"(0)
                                             : "memory");
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) pa_arrive(&sh.tail_ready[s]);
                    }
                    ring += 2 * n;
                }
            } else if (warp == 13 && lane == 0) {
                // ------------------------------------------------------ watch
                volatile int *steps = &sh.steps;
                int last = 0;
                uint64_t since = global_ns();
                const bool early = a.give_up == int32_t(blockIdx.x);
                const uint64_t limit = early ? a.give_up_ns : 2000000000ull;
                while (!mbar_try_wait(&sh.all_done, 0)) {
                    const uint64_t now = global_ns();
                    if (*steps != last) {
                        last = *steps;
                        if (!early) since = now;
                    } else if (now - since >= limit) {
                        *stop = 1;
                        break;
                    }
                }
            } else if (warp == 11 && lane == 0) {
                // ------------------------------------------------------ items
                PaWalk w = {st.b, st.h, st.tok, st.s};
                int32_t unit = st.unit;
                int64_t left = st.units;
                bool ok = true;
                for (;; ++job_at) {
                    const uint32_t slot = job_at % kPaJobs;
                    if (job_at >= kPaJobs) ok = pa_wait_one(&sh.job_empty[slot], (job_at / kPaJobs & 1) ^ 1, stop);
                    if (!ok) break;
                    PaJob &job = sh.job[slot];
                    job.n = 0;
                    int64_t step = 0;
                    if (left > 0) {
                        const PaItem it = pa_item(a, w.s, w.tok);
                        const PaPart pt = pa_part(it, unit, left);
                        job = PaJob{pt.n, it.tile0 + pt.first, pa_tail_tile(a, w.s, it, pt), it.dual, pt.head, pt.head && pt.tail,
                                    w.b, w.h, w.tok, w.s.q0, w.s.fresh, w.s.len,
                                    it.count, it.units, st.from + (st.units - left) - unit};
                        step = it.units - unit;
                        if (a.join_here == 0 && pt.head && !pt.tail)
                            a.cut[blockIdx.x] = PaPiecesOf{job.unit0, st.total, it.units, it.count * a.group, w.s.q0 + w.tok, w.h, 1, 0};
                    }
                    pa_arrive(&sh.job_full[slot]);
                    if (left <= 0) break;
                    left -= step;
                    unit = 0;
                    if (left > 0) pa_next(a, w);
                }
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
            uint32_t s_phase = 0, o_phase[2] = {0, 0}, ml_phase = 0, ml_items = 0, cuts = 0;
            bool ok = true;
            for (;;) {
                const PaJob &job = next_job(ok);
                if (!ok || job.n == 0) break;
                const bool dual = job.dual != 0;
                const int32_t tok = job.tok + (dual ? d * a.tile_tok : 0) + rtok;  // of the request
                const bool valid = in_tile && tok < job.fresh;
                const int32_t pos = job.len - job.fresh + tok;
                int64_t lo64 = a.window > 0 ? int64_t(pos) - a.window + 1 : 0;
                const int32_t lo = lo64 > 0 ? int32_t(lo64) : 0;
                const bool busy = __any_sync(0xffffffffu, valid);
                const int32_t n = dual ? job.n : (job.n - d + 1) / 2;  // tiles of this stream
                const int32_t step = dual ? kPaTile : 2 * kPaTile;
                int32_t key0 = (job.tile0 + (dual ? 0 : d)) * kPaTile;
                float ref = -INFINITY;  // reference maximum, log2 units, less kLift
                float2 sum2 = make_float2(0.0f, 0.0f);
                for (int32_t i = 0; i < n; ++i, key0 += step) {
                    ok = pa_wait(&sh.s_full[d], s_phase, stop);
                    if (!ok) break;
                    s_phase ^= 1;
                    if (busy) {
                        tc_after();
                        // first pass: the maximum, 64 scores at a time; masked ones go
                        // back to TMEM as such, so that the second finds them.  Capping
                        // keeps the order, so it is left to the second pass; there a
                        // masked score is one so low that its polynomial is lower still
                        // (and -infinity in a call that has no polynomial).
                        float m0 = -INFINITY, m1 = -INFINITY, low0 = INFINITY, low1 = INFINITY;
                        const float hidden = CAP ? a.cap_hidden : -INFINITY;
                        const int32_t hi_c = pos - key0, lo_c = lo - key0;
                        const bool edge = __any_sync(0xffffffffu, hi_c < kPaTile - 1 || lo_c > 0);
#pragma unroll 1
                        for (int c0 = 0; c0 < kPaTile; c0 += 64) {
                            float x[64];
                            tc_ld32(t_s + c0, x);
                            tc_ld32(t_s + c0 + 32, x + 32);
                            tc_wait_ld();
                            if (edge) {
#pragma unroll
                                for (int e = 0; e < 64; e += 32) {
                                    const uint32_t seen = pa_seen(lo_c - c0 - e, hi_c - c0 - e);
#pragma unroll
                                    for (int c = 0; c < 32; ++c) {
                                        if (CAP) low0 = fminf(low0, (seen >> c & 1u) != 0 ? x[e + c] : INFINITY);
                                        x[e + c] = (seen >> c & 1u) != 0 ? x[e + c] : hidden;
                                    }
                                }
                                tc_st32(t_s + c0, x);
                                tc_st32(t_s + c0 + 32, x + 32);
                            } else if (CAP) {
#pragma unroll
                                for (int c = 0; c < 64; c += 4) {
                                    low0 = min3(low0, x[c], x[c + 1]);
                                    low1 = min3(low1, x[c + 2], x[c + 3]);
                                }
                            }
#pragma unroll
                            for (int c = 0; c < 64; c += 4) {
                                m0 = max3(m0, x[c], x[c + 1]);
                                m1 = max3(m1, x[c + 2], x[c + 3]);
                            }
                        }
                        if (edge) tc_wait_st();
                        float top = fmaxf(m0, m1);
                        // (Rows that are no row of the request have no say in what its
                        // rows do, nor have scores that no row sees: the same bits come
                        // out whatever lies there.)
                        bool near = false;  // all of the warp's scores are small beside the cap
                        if (CAP) {
                            near = a.cap_near > 0.0f && __all_sync(0xffffffffu, !valid || (top <= a.cap_near && fminf(low0, low1) >= -a.cap_near));
                            const bool some = hi_c >= 0 && lo_c < kPaTile && lo_c <= hi_c;
                            top = some ? pa_tanh_of_any(top * a.cap_in) : -INFINITY;
                        }
                        top = valid ? top * a.scale_log2 - kLift : -INFINITY;
                        // move the reference when a row grew past the slack
                        if (__any_sync(0xffffffffu, top > ref + kSlack || (ref == -INFINITY && top > -INFINITY))) {
                            const float now = fmaxf(ref, top);
                            if (i > 0) {
                                const float f = now == -INFINITY ? 1.0f : ex2(ref - now);
                                sum2.x *= f;
                                sum2.y *= f;
#pragma unroll 1
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
                        // second pass: the weights, 32 at a time, the next scores on
                        // their way; P takes the place of scores already read
                        const float base = ref == -INFINITY ? 0.0f : ref;
                        const float2 sc = make_float2(a.scale_log2, a.scale_log2), nb = make_float2(-base, -base);
                        float2 acc = make_float2(0.0f, 0.0f);
                        // weights of 32 scores from their exponents, and P
                        auto weigh = [&](const float *x, int q, auto exponent, uint32_t seen) {
                            float p[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                float2 v = exponent(make_float2(x[2 * c], x[2 * c + 1]));
                                v.x = ex2(v.x);
                                v.y = ex2(v.y);
                                if (seen != ~0u) {  // known to be ~0 where nothing is masked
                                    v.x = (seen >> (2 * c) & 1u) != 0 ? v.x : 0.0f;
                                    v.y = (seen >> (2 * c + 1) & 1u) != 0 ? v.y : 0.0f;
                                }
                                if (c & 1) acc = add2(acc, v);
                                else sum2 = add2(sum2, v);
                                p[c] = __uint_as_float(pack2<BF16>(v.x, v.y));
                            }
                            tc_st16(t_s + q * 16, p);
                        };
                        // tanh(y) = y (1 + c1 y^2 + .. + c4 y^8), in powers of the score and
                        // log2 units
                        auto near_cap = [&](float2 v) {
                            const float2 zero = make_float2(0.0f, 0.0f);
                            const float2 z = fma2(v, v, zero);
                            float2 t = fma2(z, make_float2(a.cap_c[3], a.cap_c[3]), make_float2(a.cap_c[2], a.cap_c[2]));
                            t = fma2(t, z, make_float2(a.cap_c[1], a.cap_c[1]));
                            t = fma2(t, z, make_float2(a.cap_c[0], a.cap_c[0]));
                            t = fma2(t, z, make_float2(a.cap_mul, a.cap_mul));
                            return fma2(t, v, nb);
                        };
                        if (!CAP || near) {
                            float x[4][32];
                            tc_ld32(t_s, x[0]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                tc_wait_ld();
                                if (q < 3) tc_ld32(t_s + (q + 1) * 32, x[q + 1]);
                                if constexpr (CAP) weigh(x[q], q, near_cap, ~0u);
                                else weigh(x[q], q, [&](float2 v) { return fma2(v, sc, nb); }, ~0u);
                            }
                        } else {
                            // scores that come near the cap: rare, and small code.  (Seven
                            // chunks with a window: special functions throughout 64 us, with
                            // the care for small scores 72, the polynomial 51.)
#pragma unroll 1
                            for (int q = 0; q < 4; ++q) {
                                float x[32];
                                tc_ld32(t_s + q * 32, x);
                                tc_wait_ld();
                                const uint32_t seen = pa_seen(lo_c - q * 32, hi_c - q * 32);
                                if (a.cap_near > 0.0f)
                                    weigh(x, q, [&](float2 v) {
                                        return fma2(make_float2(pa_tanh(v.x * a.cap_in), pa_tanh(v.y * a.cap_in)), sc, nb);
                                    }, seen);
                                else
                                    weigh(x, q, [&](float2 v) {
                                        return fma2(make_float2(pa_tanh_of_any(v.x * a.cap_in), pa_tanh_of_any(v.y * a.cap_in)), sc, nb);
                                    }, seen);
                            }
                        }
                        sum2 = add2(sum2, acc);
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
                const bool two = !dual && job.n > 1;  // a single item with a second stream
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
                if (dual || d == 0) {
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
                        const bool whole = job.whole != 0;
                        if (whole) {
                            if (a.sinks != nullptr && valid) {
                                // the sink joins the maximum and the sum (a row without rows stays zero)
                                const float sink = a.sinks[job.kv_head * a.group + rhead] * 1.4426950408889634f;
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
                        const int32_t slot = blockIdx.x * 2 + job.head;
                        const int32_t prow = (dual ? d * a.tile_tok * a.group : 0) + row;
                        if (!whole && valid) a.part_ml[int64_t(slot) * a.part_rows + prow] = make_float2(top, sum);
                        uint8_t *dst = static_cast<uint8_t *>(a.out) +
                                       ((int64_t(job.q0) + tok) * a.out_tok + int64_t(job.kv_head * a.group + rhead) * a.out_head) * 2;
                        float *pdst = a.part_o + (int64_t(slot) * a.part_rows + prow) * HD;
#pragma unroll 1
                        for (int c = 0; c < HD; c += 32) {
                            float y[32], z[32];
                            __syncwarp();
                            tc_ld32(t_row + kO + d * HD + c, y);
                            if (two) tc_ld32(t_row + kO + HD + c, z);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = two ? y[e] * f0 + z[e] * f1 : y[e] * f0;
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
                        if (two) pa_arrive(&sh.o_empty[1]);
                        pa_arrive(&sh.o_empty[d]);
                    }
                }
                o_phase[0] ^= 1;
                if (dual || two) o_phase[1] ^= 1;
                if (a.join_here != 0 && job.whole == 0 && d == 0) {
                    // (a call so small has single items only.)  The CTA's piece is in
                    // the workspace once its four warps say so; then one thread takes a
                    // ticket, and the holder of the last one has the pieces joined.
                    __syncwarp();
                    if (lane == 0) pa_arrive(&sh.piece_done);
                    const PaPieces pieces(job.unit0, job.units, st.total);
                    if (warp == 0) {
                        uint64_t *word = a.tickets + pieces.first;
                        const uint64_t old = *static_cast<volatile uint64_t *>(word);
                        ok = pa_wait(&sh.piece_done, cuts & 1, stop);
                        if (!ok) break;
                        if (lane == 0) {
                            sh.join = pa_ticket(word, a.nonce, pieces.n, old) ? 1 : 0;
                            sh.tickets = int(cuts) + 1;
                            pa_arrive(&sh.verdict);
                        }
                    }
                    ok = pa_wait(&sh.verdict, cuts & 1, stop);
                    if (!ok) break;
                    ++cuts;
                    if (sh.join != 0) {
                        const int32_t rows = job.count * a.group;
                        for (int32_t r = warp; r < rows; r += 4) pa_join_row<HD, BF16>(a, pieces, r, job.q0 + job.tok, job.kv_head);
                    }
                }
                done_job();
            }
            if (!ok && a.join_here != 0 && threadIdx.x == 0) pa_owed_tickets(a, sh.start, sh.tickets);
        }
        // (13 goes on watching until every warp is here)
        __syncwarp();
        if (lane == 0 && warp != 13 && warp != 15) pa_arrive(&sh.all_done);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (*stop != 0) {
        // Given up, and every warp knows: nothing may still be in flight into this
        // CTA's memory.  Of the copies each stage's last may be, and Q's last.  (Of
        // the two loading warps' last ones for a stage the newer counts; the wait for
        // the older may run out, its parity having come round again.)
        if (threadIdx.x == 0) set_error(a.err, kErrTimeout);
        if (warp == 9 || warp == 14) {
            uint64_t *drain = &sh.drain[warp == 9 ? 0 : 1];
            tc_commit(drain);
            mbar_wait_bounded(drain, 0, 500000000ull);
        }
#pragma unroll 1
        for (int i = 0; i <= 16; ++i)
            if (loaded >> i & 1) mbar_wait_bounded(i < 16 ? &sh.kv_full[i] : &sh.q_full, parity >> i & 1, 5000000ull);
        tc_before();
        __syncthreads();
        tc_after();
    }
    pdl_trigger();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int HD, bool BF16, bool CAP>
cudaError_t launch_paged_one(const PaArgs &a, cudaStream_t st) {
    constexpr int smem = PaShape<HD>::kTiles + int(sizeof(PaShared));
    static_assert(smem <= 227 * 1024, "shared memory of an SM");
    const auto kern = paged_attention_kernel<HD, BF16, CAP>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(kPaCtas), dim3(kPaThreads), smem, st, a);
    if (e != cudaSuccess || a.join_here != 0) return e;
    return launch_pdl(paged_join_kernel<HD, BF16>, dim3(kPaCtas, unsigned(ceil_div(a.part_rows, 32))), dim3(256), 0, st, a);
}

template <int HD>
cudaError_t launch_paged(const PaArgs &a, bool bf16, bool cap, cudaStream_t st) {
    if (bf16) return cap ? launch_paged_one<HD, true, true>(a, st) : launch_paged_one<HD, true, false>(a, st);
    return cap ? launch_paged_one<HD, false, true>(a, st) : launch_paged_one<HD, false, false>(a, st);
}

}  // namespace kvd
