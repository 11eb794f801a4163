// kvd_paged_attn_q8p.cuh -- attention of many query rows over pages of e4m3 codes.
//
// The same sums as kvd_paged_attn_q8.cuh, for requests with more query rows a KV head
// than its 16: prompts, whose bound is the tensor cores.  A tile of 128 rows is (token,
// head of the group) pairs, and an item is one (request, KV head, run of up to two
// tiles' tokens): both tiles ("streams") meet the same KV tile.
//
//   S = Q K^T   kind::f8f6f4.  q, scaled by a power of two so that its row's largest lies
//               in [128, 256), is the sum of two e4m3 numbers (f16: three), each of which
//               multiplies the codes of K as they lie in the pages: two products at
//               twice the rate of 16 bits, from half the bytes.  Eight significant bits
//               of bf16 are two times four; 2^-17 of the row's largest is left out.
//   O += P V    kind::f16.  V's codes become f16 by four warps between the copy and the
//               MMA, times their block's power of two over the largest that the part of the
//               item has met: exactly, if that is within 2^22 of it, else to 2^-32 of the
//               largest number there.  P in f16, whatever q's type, with what is left of the
//               block's scale, a number in [1, 2), in it.  So references and sums know no more
//               of V's scales; a part that meets a larger one rescales O, as for a reference
//               that grew.  P in e4m3 terms would do without the conversion, but a sum over a
//               whole prompt meets weights far below 2^-17 of the largest, and five instructions
//               a weight cost the softmax warps more than it, of which 256 rows share one.
//
// One CTA per SM:
//   warps 0-3, 4-7   softmax of stream 0 and 1, a thread per query row; they make q's
//                    terms, too;
//   warp 8           walks the work, looks up pages and scales, TMA loads of K and V;
//   warps 9, 14      issue the MMAs of stream 0 and 1;
//   warps 10-13      V to f16, zeros for rows that nobody holds;
//   warp 15          ends every wait if the CTA stops making steps.
// TMEM: S0 S1 (128 columns each) O0 O1.  A stream's S is two halves of 64 columns: its
// softmax works on one (P in f16 takes its first 32 columns) while P V of the other and S
// of that half's next 64 rows are made, so neither waits for the other.  MMAs run in the
// order in which a thread issues them: S of a half's next rows stands behind P V of its
// last ones, whose P it overwrites.  O is rescaled only where a row's reference grew by
// more than 2^kSlack, once P V of the half before is done.
//
// Barriers of a ring (k_full, k_empty; c_full, c_empty: codes of V; v_full, v_empty:
// V in f16) turn once a slot; s_full, p_ready, o_step once a tile for each stream and
// half.  A stream without rows lets go of what it does not use only once it is there, so
// it sees every turn; o_step of a half is one phase ahead at most of what the softmax
// warps know of it (their last s_full of that half stands behind the one before).
//
// Measured (GPU time on one GB300): 4096 new rows of a prompt over 32768, 32 heads over
// 8, 1480 to 1515 us, 1360 to 1390 TFLOP/s at the power limit, in f16 1.77 ms; 4096 over 4096
// 158, in f16 178; seven chunks of up to 700 rows with a window, 60 with capped scores, 40
// without.  A unit (a KV tile of both streams) takes some 1.15 us, 1.7 at the power limit,
// and its MMAs alone 1.1; an item 8 us beside its units (q, the first scores, the last P V,
// its rows).  (Some 50 to 90 bytes of registers spill.)
// Measured and not taken: S in one piece of 128 columns, as wide as the tile (prompt 1.99
// ms: a stream's softmax, 2500 cycles, and its MMAs with their barriers, 2100, one after
// the other); S only once P V has been seen done (1.61 ms against 1.48); the maximum
// before the weights (no difference beside that); a slack of 2^4 (below); all of V's scale
// in P, and the weights summed once more from the scores where scales lie far apart (prompt
// 1.57 to 1.71 ms, from the larger code alone).
#pragma once

#include "kvd_paged_attn_q8.cuh"

namespace kvd {

constexpr int kQpThreads = 512;
constexpr int kQpCtas = 152;
constexpr int kQpRegs = 128, kQpSoftRegs = 184, kQpLoadRegs = 72;
static_assert(2 * kQpSoftRegs + 2 * kQpLoadRegs <= 4 * kQpRegs, "setmaxnreg shares");
constexpr int kQpMaxRows = 2 * kQrTile;
constexpr int kVUp = 7;  // codes, 448 at most, times 2^kVUp are numbers of f16
constexpr float kTanh1 = float(kPaTanh[0]), kTanh2 = float(kPaTanh[1]), kTanh3 = float(kPaTanh[2]), kTanh4 = float(kPaTanh[3]);

template <int HD, bool BF16>
struct QpShape {
    static constexpr int kTerms = BF16 ? 2 : 3;
    static constexpr int kCodeBytes = kQrTile * HD, kWideBytes = 2 * kCodeBytes;
    static constexpr int kStages = BF16 ? 3 : 2;                  // of K's codes
    static constexpr int kCodes = BF16 ? 2 : 1, kWide = 2;        // of V's codes, of V in f16
    static constexpr int kScales = kStages + 2;
    static constexpr int kQBytes = kTerms * kCodeBytes;           // of one stream: a term after another
    static constexpr int kQ = 0, kK = 2 * kQBytes, kC = kK + kStages * kCodeBytes, kV = kC + kCodes * kCodeBytes,
                         kTotal = kV + kWide * kWideBytes;
    static constexpr uint32_t kSwizzle = HD == 128 ? 2 : 4, kAtom = HD * 8;
};

template <typename S>
struct QpShared {
    uint64_t k_full[S::kStages], k_empty[S::kStages], c_full[S::kCodes], c_empty[S::kCodes], v_full[S::kWide], v_empty[S::kWide], sc_full[S::kScales];
    uint64_t s_full[2][2], p_ready[2][2], o_step[2][2], q_ready[2], job_full[kQrJobs], job_empty[kQrJobs], drain[2];
    QrJob job[kQrJobs];
    PaStart start;
    int64_t warp_sums[kQpThreads / 32];
    uint32_t tmem;
    int stop, steps;  // the watch: give up; changes with every tile that is loaded
    uint64_t all_done;
    float4 scale[S::kScales][8];  // of a tile's pages: K's scale; V's over its power of two, m: log2 m, 1 / m; the largest power's exponent
    uint32_t v_up[S::kScales][8];  // what V's codes are multiplied by, f16 twice
};

template <int HD, bool BF16, bool CAP>
__global__ void __launch_bounds__(kQpThreads, 1) qp_kernel(const __grid_constant__ QrArgs a) {
    using S = QpShape<HD, BF16>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr int kTerms = S::kTerms;
    constexpr uint32_t kO = 256;  // TMEM column of O0; O1 follows
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    QpShared<S> &sh = *reinterpret_cast<QpShared<S> *>(smem_raw + S::kTotal);
    const uint32_t smem = smem_addr(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 2);
        }
        for (int i = 0; i < S::kCodes; ++i) {
            mbar_init(&sh.c_full[i], 1);
            mbar_init(&sh.c_empty[i], 4);
        }
        for (int i = 0; i < S::kWide; ++i) {
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.v_empty[i], 2);
        }
        for (int i = 0; i < S::kScales; ++i) mbar_init(&sh.sc_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.s_full[i][b], 1);
                mbar_init(&sh.p_ready[i][b], 4);
                mbar_init(&sh.o_step[i][b], 1);
            }
            mbar_init(&sh.q_ready[i], 4);
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < kQrJobs; ++i) {
            mbar_init(&sh.job_full[i], 1);
            mbar_init(&sh.job_empty[i], 14);  // eight softmax warps, two of MMAs, four that convert
        }
        mbar_init(&sh.all_done, 15);  // every warp but 15
        fence_mbar_init();
        sh.stop = 0;
        sh.steps = 0;
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_before();
    }
    if (warp == 8 && lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &a.k : &a.v) : "memory");
    // The launch before has let this one come early: what it cuts is older than both.
    qr_cut<kQpThreads>(a, &sh.start, sh.warp_sums);  // synchronises the CTA
    pdl_wait();
    pdl_trigger();
    tc_after();
    const uint32_t tmem = sh.tmem;
    volatile int *stop = &sh.stop;
    const PaStart st = sh.start;
    const int32_t tile_tok = a.run / 2;    // tokens of a stream
    uint32_t k_loads = 0, v_loads = 0;     // tiles asked for
    if (threadIdx.x == 256) a.cut[blockIdx.x].n = 0;  // whose thread writes a record, too

    if (st.units > 0) {
        bool ok = true;
        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQpLoadRegs));
            if (warp == 8) {
                // ---------------------------------------------------- work and loads
                PaWalk w = {st.b, st.h, st.tok, st.s};
                int32_t unit = st.unit;
                int64_t left = st.units;
                const int ppt = kQrTile >> a.page_log2;
                const uint32_t box = uint32_t(HD) << a.page_log2;  // bytes of a page
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
                        if (at >= kQrJobs) ok = pa_wait(&sh.job_empty[at % kQrJobs], (at / kQrJobs & 1) ^ 1, stop);
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
                        if (lane == 0) mbar_arrive_expect_tx(bar, S::kCodeBytes);
                        __syncwarp();
                        if (lane < ppt) tma_2d(dst + lane * box, map, 0, page < 0 ? a.pool_rows : (page * a.n_kv + h) << a.page_log2, bar);
                    };
                    const int32_t per_block = 32 / ppt;  // tiles
                    int32_t block_pages = lookup(0), next_pages = lookup(1), v_page = -1;
                    float2 block_scales = scales(block_pages), next_scales = make_float2(1.0f, 1.0f);
                    int32_t most = -64;  // exponent of V's largest scale so far
                    // K runs a tile ahead of V
                    for (int32_t t = 0; ok && t <= n; ++t) {
                        int32_t page = -1;
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
                            if (turn > 0) ok = pa_wait(&sh.k_empty[slot], (turn & 1) ^ 1, stop);
                            if (!ok) break;
                            // (K first: the scales may still be on their way)
                            load(&a.k, smem + S::kK + slot * S::kCodeBytes, page, &sh.k_full[slot]);
                            const uint32_t v = __float_as_uint(scale_ok(vs) ? vs : scale_of(vs, lane < ppt ? a.err : nullptr));
                            const int32_t e = page >= 0 ? int32_t(v >> 23) - 127 : -64;
                            most = max(most, __reduce_max_sync(~0u, e));
                            if (lane < ppt) {
                                const float m = __uint_as_float((v & 0x7fffffu) | 0x3f800000u);
                                sh.scale[sc][lane] = make_float4(scale_of(ks, a.err), log2f(m), 1.0f / m, float(most));
                                const int32_t up = e - most + kVUp;  // f16's normal numbers begin at 2^-14, its others at 2^-24
                                sh.v_up[sc][lane] = 0x10001u * (up >= -14 ? uint32_t(up + 15) << 10 : up >= -24 ? 1u << (up + 24) : 0u);
                            }
                            qr_arrive(&sh.sc_full[sc]);
                            ++k_loads;
                            if (lane == 0) *static_cast<volatile int *>(&sh.steps) = int(k_loads);
                    }
                        if (t > 0) {
                            const uint32_t slot = v_loads % S::kCodes, turn = v_loads / S::kCodes;
                            if (turn > 0) ok = pa_wait(&sh.c_empty[slot], (turn & 1) ^ 1, stop);
                            if (!ok) break;
                            load(&a.v, smem + S::kC + slot * S::kCodeBytes, v_page, &sh.c_full[slot]);
                            ++v_loads;
                        }
                        v_page = page;
                    }
                    if (!ok) break;
                    left -= have;
                    unit = 0;
                    if (left > 0) qr_next(a, w);
                }
            } else if (warp == 9 || warp == 14) {
                // ---------------------------------------------------- MMAs
                const int d = warp == 14 ? 1 : 0;
                uint32_t g = 0, mine = 0, items = 0;  // tiles, tiles and items of this stream
                // S of half b of tile i: 64 rows of K
                auto score = [&](uint32_t i, int b) {
                    const uint32_t slot = i % S::kStages;
                    if (b == 0) ok = pa_wait(&sh.k_full[slot], i / S::kStages & 1, stop);
                    if (!ok) return;
                    tc_after();
                    if (elect_one()) {
                        constexpr uint32_t id = tc_idesc8(128, 64, false, false);
                        const uint64_t kd = tc_desc(smem + S::kK + slot * S::kCodeBytes + b * (S::kCodeBytes / 2), 16, S::kAtom, S::kSwizzle);
                        const uint64_t qd = tc_desc(smem + S::kQ + d * S::kQBytes, 16, S::kAtom, S::kSwizzle);
#pragma unroll
                        for (int t = 0; t < kTerms; ++t)
#pragma unroll
                            for (int kk = 0; kk < HD / 32; ++kk)
                                tc_mma8(tmem + d * 128 + b * 64, qd + t * (S::kCodeBytes >> 4) + kk * 2, kd + kk * 2, id, t != 0 || kk != 0);
                    }
                    __syncwarp();
                    tc_commit(&sh.s_full[d][b]);
                    if (b == 1) tc_commit(&sh.k_empty[slot]);
                };
                for (uint32_t at = 0;; ++at) {
                    ok = pa_wait(&sh.job_full[at % kQrJobs], at / kQrJobs & 1, stop);
                    if (!ok) break;
                    const uint32_t n = uint32_t(sh.job[at % kQrJobs].n);
                    const bool busy = d == 0 || sh.job[at % kQrJobs].count > tile_tok;
                    qr_arrive(&sh.job_empty[at % kQrJobs]);
                    if (n == 0) break;
                    if (!busy) {
                        for (uint32_t i = g; ok && i < g + n; ++i) {
                            ok = pa_wait(&sh.k_full[i % S::kStages], i / S::kStages & 1, stop);
                            if (!ok) break;
                            qr_arrive(&sh.k_empty[i % S::kStages]);
                            ok = pa_wait(&sh.v_full[i % S::kWide], i / S::kWide & 1, stop);
                            if (!ok) break;
                            qr_arrive(&sh.v_empty[i % S::kWide]);
                        }
                        if (!ok) break;
                        g += n;
                        continue;
                    }
                    // (q_ready says, too, that O of the item before has been read)
                    ok = pa_wait(&sh.q_ready[d], items++ & 1, stop);
                    if (!ok) break;
                    score(g, 0);
                    if (ok) score(g, 1);
                    for (uint32_t i = g; ok && i < g + n; ++i, ++mine) {
                        const uint32_t slot = i % S::kWide;
                        ok = pa_wait(&sh.v_full[slot], i / S::kWide & 1, stop);
#pragma unroll 1
                        for (int b = 0; ok && b < 2; ++b) {
                            ok = pa_wait(&sh.p_ready[d][b], mine & 1, stop);
                            if (!ok) break;
                            tc_after();
                            if (elect_one()) {
                                constexpr uint32_t id = tc_idesc(false, 128, HD, true);
                                const uint64_t vd = tc_desc(smem + S::kV + slot * S::kWideBytes + b * (64 * 128), kQrTile * 128, 1024, 2);
#pragma unroll
                                for (int kk = 0; kk < 64 / 16; ++kk)
                                    tc_mma_ts(tmem + kO + d * HD, tmem + d * 128 + b * 64 + kk * 8, vd + kk * (2048 >> 4), id, i != g || b != 0 || kk != 0);
                            }
                            __syncwarp();
                            tc_commit(&sh.o_step[d][b]);
                            if (b == 1) tc_commit(&sh.v_empty[slot]);
                            if (i + 1 < g + n) {
                                // S takes the place of P once P V has read it
                                score(i + 1, b);
                            }
                        }
                    }
                    if (!ok) break;
                    g += n;
                }
                // nobody waits for the last v_empty, but the block must not end before it has come
                tc_commit(&sh.drain[d]);
                if (!mbar_wait_bounded(&sh.drain[d], 0, 500000000ull)) *stop = 1;
            } else if (warp >= 10 && warp < 14) {
                // ---------------------------------------------------- V to f16
                // A lane takes 16 codes; eight neighbouring lanes those of eight rows, whose
                // places the swizzle spreads over all banks, read and written.
                constexpr int kChunks = HD / 16;
                const int r0 = (warp - 10) * 32 + lane % 8, c0 = lane / 8;
                uint32_t g = 0;
                for (uint32_t at = 0;; ++at) {
                    ok = pa_wait(&sh.job_full[at % kQrJobs], at / kQrJobs & 1, stop);
                    if (!ok) break;
                    const int32_t n = sh.job[at % kQrJobs].n, tile0 = sh.job[at % kQrJobs].tile0, len = sh.job[at % kQrJobs].len;
                    qr_arrive(&sh.job_empty[at % kQrJobs]);
                    if (n == 0) break;
                    for (int32_t i = 0; i < n; ++i, ++g) {
                        const uint32_t from = g % S::kCodes, to = g % S::kWide;
                        ok = pa_wait(&sh.c_full[from], g / S::kCodes & 1, stop);
                        uint32_t up[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) up[k] = sh.v_up[g % S::kScales][(r0 + k * 8) >> a.page_log2];
                        if (ok && g >= uint32_t(S::kWide)) ok = pa_wait(&sh.v_empty[to], (g / S::kWide & 1) ^ 1, stop);
                        if (!ok) break;
                        const uint32_t src = smem + S::kC + from * S::kCodeBytes, dst = smem + S::kV + to * S::kWideBytes;
                        const int32_t held = len - (tile0 + i) * kQrTile;  // rows of the tile
#pragma unroll
                        for (int k = 0; k < kChunks; ++k) {
                            const int r = r0 + k % 4 * 8, c = c0 + k / 4 * 4;
                            uint32_t at8 = r * HD + c * 16;
                            at8 ^= HD == 128 ? (r & 7) << 4 : (at8 >> 7 & 3) << 4;
                            uint32_t w[4];
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src + at8));
                            if (held < kQrTile && r >= held) w[0] = w[1] = w[2] = w[3] = 0;
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __half2 v = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[e / 2] >> (16 * (e % 2))), __NV_E4M3));
                                const __half2 y = __hmul2(v, *reinterpret_cast<const __half2 *>(&up[k % 4]));
                                x[e] = *reinterpret_cast<const uint32_t *>(&y);
                            }
                            // channel 16 c of a row lies in half c / 4, 16-byte piece 2 (c % 4)
                            const uint32_t to16 = dst + (c / 4) * (kQrTile * 128) + r * 128;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to16 + (((2 * (c % 4) + j) ^ (r & 7)) << 4)), "r"(x[4 * j]),
                                             "r"(x[4 * j + 1]), "r"(x[4 * j + 2]), "r"(x[4 * j + 3])
                                             : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        qr_arrive(&sh.c_empty[from]);
                        qr_arrive(&sh.v_full[to]);
                    }
                    if (!ok) break;
                }
            } else if (warp == 15 && lane == 0) {
                // ---------------------------------------------------- watch
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
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQpSoftRegs));
            // -------------------------------------------------------- softmax
            const int d = warp >> 2;                       // stream
            const int row = (warp & 3) * 32 + lane;        // row of the tile
            const uint32_t t_row = tmem + (uint32_t((warp & 3) * 32) << 16);
            const uint32_t t_s = t_row + d * 128, t_o = t_row + kO + d * HD;
            // Weights reach 2^(kLift + kSlack), the most that f16 holds, before the reference
            // moves, and keep 11 bits down to 2^-17 of it, some down to 2^-27.  (With a slack of
            // 2^4 4096 rows over 4096 took 18 us longer: the maximum grows often while a
            // row has seen little.)
            constexpr float kLift = 3.0f, kSlack = 12.0f;
            const int32_t rtok = row / a.group, rhead = row - rtok * a.group;
            // Rows travel between global memory and the threads by way of the first two
            // terms' places of the warp's own rows, a row's 2 HD bytes by neighbouring
            // lanes: a lane that read or wrote its own row in 16-byte pieces would take a
            // sector of 32 rows each time, 2 us an item for q and again for O.
            constexpr int kPieces = HD / 8, kRowsAtOnce = 32 / kPieces;
            auto place = [&](int r, int piece) {  // of 16 bytes of tile row r
                uint32_t at = r * HD + piece % (HD / 16) * 16;
                at ^= HD == 128 ? (r & 7) << 4 : (at >> 7 & 3) << 4;
                return smem + S::kQ + d * S::kQBytes + piece / (HD / 16) * S::kCodeBytes + at;
            };
            uint32_t g = 0, mine = 0;  // tiles, and halves of this stream's
            for (uint32_t at = 0;; ++at) {
                ok = pa_wait(&sh.job_full[at % kQrJobs], at / kQrJobs & 1, stop);
                if (!ok) break;
                const QrJob job = sh.job[at % kQrJobs];
                qr_arrive(&sh.job_empty[at % kQrJobs]);
                if (job.n == 0) break;
                if (d == 1 && job.count <= tile_tok) {
                    g += job.n;
                    continue;
                }
                const int32_t tok = d * tile_tok + rtok;  // of the item
                const bool valid = rtok < tile_tok && tok < job.count;
                const int32_t head = job.kv_head * a.group + rhead, pos = job.first_pos + tok;
                // q as e4m3 terms; every MMA that read the last item's has been waited for
                float mul;
                {
                    uint4 x[HD / 8];
                    const T *mine_q = static_cast<const T *>(a.q) + (int64_t(job.q_row) + tok) * a.q_tok + int64_t(head) * a.q_head;
                    // (a row before its request's start sees nothing, whatever q is there)
                    const uint64_t src = valid && pos >= 0 ? reinterpret_cast<uint64_t>(mine_q) : 0;
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) {
                        const int r = k * kRowsAtOnce + lane / kPieces;
                        const uint64_t from = __shfl_sync(~0u, src, r);
                        x[k] = from != 0 ? reinterpret_cast<const uint4 *>(from)[lane % kPieces] : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int k = 0; k < kPieces; ++k)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place((warp & 3) * 32 + k * kRowsAtOnce + lane / kPieces, lane % kPieces)),
                                     "r"(x[k].x), "r"(x[k].y), "r"(x[k].z), "r"(x[k].w)
                                     : "memory");
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kPieces; ++k)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[k].x), "=r"(x[k].y), "=r"(x[k].z), "=r"(x[k].w) : "r"(place(row, k)) : "memory");
                    __syncwarp();
                    auto two = [](uint32_t w) {
                        float2 v;
                        if constexpr (BF16) v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                        else v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                        return v;
                    };
                    // the largest, by the bits of the type, which are ordered; what is not finite has all bits of the exponent
                    uint32_t big = 0;
#pragma unroll
                    for (int i = 0; i < HD / 2; ++i) big = __vmaxu2(big, reinterpret_cast<const uint32_t *>(x)[i] & 0x7fff7fffu);
                    big = max(big >> 16, big & 0xffffu);
                    const bool fine = big < (BF16 ? 0x7f80u : 0x7c00u);
                    const float top = BF16 ? __uint_as_float(big << 16) : __half2float(__ushort_as_half(uint16_t(big)));
                    int e = 134 - int(__float_as_uint(top) >> 23);
                    e = top == 0.0f ? 0 : e > 120 ? 120 : e < -120 ? -120 : e;
                    const float up = __uint_as_float(uint32_t(e + 127) << 23);
                    // a row that is not finite is none of numbers
                    mul = fine ? a.mul * __uint_as_float(uint32_t(127 - e) << 23) : __int_as_float(0x7fc00000);
#pragma unroll
                    for (int c = 0; c < HD / 16; ++c) {
                        uint32_t t[kTerms][4];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float2 v = two(reinterpret_cast<const uint32_t *>(x)[c * 8 + i]);
                            // f16 holds the scaled values and what the terms leave of them, but for 2^-25
                            __half2 y = __floats2half2_rn(v.x * up, v.y * up);
#pragma unroll
                            for (int k = 0; k < kTerms; ++k) {
                                const uint32_t b = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(y), __NV_SATFINITE, __NV_E4M3);
                                t[k][i / 2] = i % 2 ? t[k][i / 2] | b << 16 : b;
                                if (k + 1 < kTerms) y = __hsub2(y, __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(b), __NV_E4M3)));
                            }
                        }
                        uint32_t to = row * HD + c * 16;
                        to ^= HD == 128 ? (row & 7) << 4 : (to >> 7 & 3) << 4;
#pragma unroll
                        for (int k = 0; k < kTerms; ++k)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(smem + S::kQ + d * S::kQBytes + k * S::kCodeBytes + to), "r"(t[k][0]),
                                         "r"(t[k][1]), "r"(t[k][2]), "r"(t[k][3])
                                         : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_before();
                    qr_arrive(&sh.q_ready[d]);
                }
                const int64_t lo64 = a.window > 0 ? int64_t(pos) - a.window + 1 : 0;
                const int32_t lo = lo64 > 0 ? int32_t(lo64) : 0;
                const bool busy = __any_sync(~0u, valid);
                int32_t key0 = job.tile0 * kQrTile;
                float ref = -INFINITY;  // reference, log2 units, less kLift
                float unit = 0.0f;      // O's: 2^(unit - kVUp)
                float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll 1
                for (int32_t i = 0; i < 2 * job.n; ++i, ++mine, key0 += 64) {
                    const int b = i & 1;  // the tile's first or second half, 64 rows of K
                    const uint32_t tile = g + uint32_t(i / 2);
                    if (b == 0) ok = pa_wait(&sh.sc_full[tile % S::kScales], tile / S::kScales & 1, stop);
                    ok = ok && pa_wait(&sh.s_full[d][b], mine >> 1 & 1, stop);
                    if (!ok) break;
                    if (busy) {
                        const float4 *sc = sh.scale[tile % S::kScales];
                        const float most = sc[0].w;
                        if (i == 0) unit = most;
                        const uint32_t t_h = t_s + b * 64;
                        const int col0 = b * 64;
                        tc_after();
                        const int32_t hi_c = pos - key0, lo_c = lo - key0;
                        float x[64];
                        tc_ld32(t_h, x);
                        tc_ld32(t_h + 32, x + 32);
                        tc_wait_ld();
                        float size = 0.0f;  // CAP: the largest score that is seen, by size
                        if (__any_sync(~0u, hi_c < 63 || lo_c > 0)) {
#pragma unroll
                            for (int e = 0; e < 64; e += 16) {
                                const uint32_t seen = pa_seen(lo_c - e, hi_c - e);
                                float m = 0.0f;
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    if (CAP) m = fmaxf(m, (seen >> c & 1u) != 0 ? fabsf(x[e + c]) : 0.0f);
                                    x[e + c] = (seen >> c & 1u) != 0 ? x[e + c] : -INFINITY;
                                }
                                if (CAP) size = fmaxf(size, m * sc[(col0 + e) >> a.page_log2].x);
                            }
                        } else if (CAP) {
#pragma unroll
                            for (int u = 0; u < 64; u += 16) {
                                float m0 = fabsf(x[u]), m1 = fabsf(x[u + 1]);
#pragma unroll
                                for (int c = 2; c < 16; c += 2) {
                                    m0 = fmaxf(m0, fabsf(x[u + c]));
                                    m1 = fmaxf(m1, fabsf(x[u + c + 1]));
                                }
                                size = fmaxf(size, fmaxf(m0, m1) * sc[(col0 + u) >> a.page_log2].x);
                            }
                        }
                        // 2 log2 e y = the score's tanh argument; the polynomial holds to y = 1/2.
                        // (Rows that are no row of the request have no say in what its rows do.)
                        const bool near = CAP && __all_sync(~0u, !valid || size * mul <= 1.4426950f);
                        // Weights relative to the reference as it stands, and the largest score
                        // beside them: where a row grew past the slack they are taken once
                        // more with a new one.
#pragma unroll 1
                        for (;;) {
                            const float base = ref == -INFINITY ? 0.0f : ref;
                            float top = -INFINITY;
                            float2 sums = sum2;
                            // `exponent` of two scores, their factor k and what is added to them
                            auto weigh = [&](auto exponent) {
#pragma unroll
                                for (int q = 0; q < 64; q += 32) {
                                    float p[16];
#pragma unroll
                                    for (int u = q; u < q + 32; u += 16) {
                                        const float4 f = sc[(col0 + u) >> a.page_log2];
                                        float m0 = fmaxf(x[u], x[u + 1]), m1 = fmaxf(x[u + 2], x[u + 3]);
#pragma unroll
                                        for (int c = 4; c < 16; c += 4) {
                                            m0 = max3(m0, x[u + c], x[u + c + 1]);
                                            m1 = max3(m1, x[u + c + 2], x[u + c + 3]);
                                        }
                                        // Never zero, for which what is hidden, -infinity, would be no
                                        // number: scores are below 2^-100 where this is not their factor.
                                        float k = f.x * mul;
                                        k = k < FLT_MIN ? FLT_MIN : k;  // (no number stays none)
                                        if constexpr (CAP) k = qr_cap_factor(k);
                                        const float b0 = f.y - base;
                                        if constexpr (CAP) {
                                            const float m = fmaxf(m0, m1) * k;
                                            top = fmaxf(top, (m == -INFINITY ? m : pa_tanh_of_any(m) * a.cap) + f.y);
                                        } else {
                                            top = fmaxf(top, fmaf(fmaxf(m0, m1), k, f.y));
                                        }
                                        float2 acc[2];
#pragma unroll
                                        for (int c = 0; c < 8; ++c) {
                                            float2 v = exponent(make_float2(x[u + 2 * c], x[u + 2 * c + 1]), k, b0);
                                            v.x = ex2(v.x);
                                            v.y = ex2(v.y);
                                            acc[c & 1] = c < 2 ? v : add2(acc[c & 1], v);
                                            p[(u - q) / 2 + c] = __uint_as_float(pack2<false>(v.x, v.y));
                                        }
                                        sums = fma2(add2(acc[0], acc[1]), make_float2(f.z, f.z), sums);
                                    }
                                    tc_st16(t_h + q / 2, p);
                                }
                            };
                            if constexpr (!CAP) {
                                weigh([](float2 v, float k, float b0) { return fma2(v, make_float2(k, k), make_float2(b0, b0)); });
                            } else if (near) {
                                // cap tanh(y) = cap y (1 + c1 y^2 + .. + c4 y^8); what is masked stays -infinity
                                weigh([&](float2 v, float k, float b0) {
                                    const float ky = k * 0.34657359027997264f;  // y of a raw score
                                    const float2 y = fma2(v, make_float2(ky, ky), make_float2(0.0f, 0.0f)), z = fma2(y, y, make_float2(0.0f, 0.0f));
                                    float2 w = fma2(z, make_float2(kTanh4, kTanh4), make_float2(kTanh3, kTanh3));
                                    w = fma2(w, z, make_float2(kTanh2, kTanh2));
                                    w = fma2(w, z, make_float2(kTanh1, kTanh1));
                                    w = fma2(w, z, make_float2(1.0f, 1.0f));
                                    return fma2(fma2(y, make_float2(a.cap, a.cap), make_float2(0.0f, 0.0f)), w, make_float2(b0, b0));
                                });
                            } else {
                                weigh([&](float2 v, float k, float b0) {
                                    return make_float2(v.x == -INFINITY ? v.x : fmaf(pa_tanh_of_any(v.x * k), a.cap, b0),
                                                       v.y == -INFINITY ? v.y : fmaf(pa_tanh_of_any(v.y * k), a.cap, b0));
                                });
                            }
                            top = valid ? top - kLift : -INFINITY;
                            if (!__any_sync(~0u, top > ref + kSlack || (ref == -INFINITY && top > -INFINITY) || unit != most)) {
                                sum2 = sums;
                                break;
                            }
                            tc_wait_st();  // P is written once more
                            const float now = fmaxf(ref, top);
                            if (i > 0) {
                                // O is the warps' own once P V of the half before is done
                                ok = pa_wait(&sh.o_step[d][b ^ 1], (mine - 1) >> 1 & 1, stop);
                                if (!ok) break;
                                tc_after();
                                float f = now == -INFINITY ? 1.0f : ex2(ref - now);
                                sum2.x *= f;
                                sum2.y *= f;
                                f *= ex2(unit - most);
#pragma unroll 1
                                for (int c = 0; c < HD; c += 32) {
                                    float o[32];
                                    tc_ld32(t_o + c, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] *= f;
                                    tc_st32(t_o + c, o);
                                }
                            }
                            ref = now;
                            unit = most;
                        }
                        if (!ok) break;
                        tc_wait_st();
                        tc_before();
                    }
                    qr_arrive(&sh.p_ready[d][b]);
                }
                g += uint32_t(job.n);
                if (!ok) break;
                // ---- the end of the item, or of this CTA's piece of it
                ok = pa_wait(&sh.o_step[d][0], (mine - 2) >> 1 & 1, stop) && pa_wait(&sh.o_step[d][1], (mine - 1) >> 1 & 1, stop);
                if (!ok) break;
                if (busy) {
                    tc_after();
                    const float sum = sum2.x + sum2.y;
                    const bool whole = job.whole != 0;
                    float f = 1.0f;
                    const float to_v = __uint_as_float(uint32_t(127 - kVUp + int32_t(unit)) << 23);
                    if (whole) {
                        float s = sum;
                        if (a.sinks != nullptr && valid && ref != -INFINITY) {
                            // the sink joins the reference and the sum (a row without rows stays zero)
                            const float sink = a.sinks[head] * 1.4426950408889634f, all = fmaxf(ref, sink);
                            f = ex2(ref - all);
                            s = s * f + ex2(sink - all);
                        }
                        f *= s == 0.0f ? 0.0f : 1.0f / s;
                    }
                    f *= to_v;
                    const int64_t slot = int64_t(blockIdx.x) * 2 + job.head;
                    const int32_t prow = d * tile_tok * a.group + row;
                    if (!whole && valid) a.part_ml[slot * a.part_rows + prow] = make_float2(ref, sum);
                    const uint64_t dst = !valid ? 0
                                         : whole ? reinterpret_cast<uint64_t>(static_cast<T *>(a.out) + (int64_t(job.q_row) + tok) * a.out_tok + int64_t(head) * a.out_head)
                                                 : reinterpret_cast<uint64_t>(a.part_o + (slot * a.part_rows + prow) * HD);
                    // 2 HD bytes of each of the warp's rows to `skip` bytes behind their dst
                    auto send = [&](int skip) {
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < kPieces; ++k) {
                            const int r = k * kRowsAtOnce + lane / kPieces;
                            const uint64_t to = __shfl_sync(~0u, dst, r);
                            uint4 v;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(place((warp & 3) * 32 + r, lane % kPieces)) : "memory");
                            if (to != 0) *reinterpret_cast<uint4 *>(to + skip + lane % kPieces * 16) = v;
                        }
                        __syncwarp();
                    };
#pragma unroll
                    for (int c = 0; c < HD; c += 32) {
                        float y[32];
                        tc_ld32(t_o + c, y);
                        tc_wait_ld();
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(row, (c + e) / 8)), "r"(pack2<BF16>(y[e] * f, y[e + 1] * f)),
                                             "r"(pack2<BF16>(y[e + 2] * f, y[e + 3] * f)), "r"(pack2<BF16>(y[e + 4] * f, y[e + 5] * f)),
                                             "r"(pack2<BF16>(y[e + 6] * f, y[e + 7] * f))
                                             : "memory");
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(row, (c + e) % (HD / 2) / 4)), "f"(y[e] * f), "f"(y[e + 1] * f),
                                             "f"(y[e + 2] * f), "f"(y[e + 3] * f)
                                             : "memory");
                            if ((c + 32) % (HD / 2) == 0) send((c + 32 - HD / 2) * 4);
                        }
                    }
                    if (whole) send(0);
                    __syncwarp();
                    tc_before();
                }
            }
        }
        // (15 goes on watching until every warp is here)
        if (warp != 15) qr_arrive(&sh.all_done);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (*stop != 0) {
        // given up: no copy may be in flight into this CTA's memory
        if (threadIdx.x == 0) set_error(a.err, kErrTimeout);
        if (warp == 8) {
            for (uint32_t i = 0; i < uint32_t(S::kStages); ++i)
                if (k_loads > i) mbar_wait_bounded(&sh.k_full[(k_loads - 1 - i) % S::kStages], (k_loads - 1 - i) / S::kStages & 1, 500000000ull);
            for (uint32_t i = 0; i < uint32_t(S::kCodes); ++i)
                if (v_loads > i) mbar_wait_bounded(&sh.c_full[(v_loads - 1 - i) % S::kCodes], (v_loads - 1 - i) / S::kCodes & 1, 500000000ull);
        }
        tc_before();
        __syncthreads();
        tc_after();
    }
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int HD, bool BF16>
cudaError_t launch_qp(QrArgs &a, cudaStream_t st) {
    using S = QpShape<HD, BF16>;
    constexpr int smem = S::kTotal + int(sizeof(QpShared<S>));
    static_assert(smem <= 227 * 1024, "shared memory of an SM");
    const auto kern = a.cap > 0.0f ? qp_kernel<HD, BF16, true> : qp_kernel<HD, BF16, false>;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    a.ctas = kQpCtas;
    return launch_pdl(kern, dim3(kQpCtas), dim3(kQpThreads), smem, st, a);
}

}  // namespace kvd
