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
// the runs of rows in one page that begin among its tokens, for some heads of K or one of
// V: it holds up to 128 rows of a head in registers, takes the largest value of each run,
// settles the scales and the codes already there, and writes the codes.  Nobody waits for
// another CTA, because a block's rows all lie in one, and every row is read once.
//
// Measured (GPU time on one GB300; a copy runs at 6.77 TB/s): 8192 tokens of a prompt, 32
// + 8 + 8 heads, bf16, written in 47 us (184 MB; 3.9 TB/s), 9000 of chunks in f32 in 25.5,
// one token for each of 256 requests in 5.4; 373000 rows of 48 requests read back to bf16
// in 368 us, 6.23 TB/s (32 rows and one head to a CTA, a binary search each: 470).  Writing
// is bound by latency: a run's rows, their largest value, the scale, the codes, one after
// another, with some 30 warps to an SM.

#include <cfloat>
#include <cmath>

#include "kvd_q8.cuh"
#include "kvd_rope.cuh"

namespace kvd {
namespace {

constexpr int kWindow = 128;      // rows in registers: any run fits

struct StoreArgs {
    RopeArgs r;               // g[0]: q; g[1], g[2]: k and v with their pages
    float *scale[2];          // of K and V: [n_pages][n_kv]
    int32_t tok;              // tokens whose runs a CTA takes: at most 128, and with a page's rows at most 256
    int32_t k_heads, k_ctas;  // heads of a CTA of K; CTAs of K's heads
    int32_t q_tok, q_ctas;    // tokens of a CTA of q; CTAs of q
    int32_t q_f16;            // q_out's type
};

// The smallest power of two s with top <= 448 s, within the limits: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = int(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
    return e <= 127 - 64 ? kScaleLow : e >= 127 + 64 ? kScaleHigh : __uint_as_float(uint32_t(e) << 23);
}
__device__ __forceinline__ bool pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// Runs of rows in one page that begin among the CTA's tokens; row i is token t0 + i.
struct Runs {
    int32_t slot[256];
    int16_t run[256];           // -1: no row of this CTA's
    int32_t first[129], page[128];        // a run's first row, its page,
    int32_t row0[128];                    // and the row of it in that page
    int32_t end, leads[8];
    uint32_t top[128];                    // largest finite |x|, as bits
    float scale[128], ratio[128];
};

// How many there are.
__device__ __forceinline__ int find_runs(const StoreArgs &args, Runs &s, int64_t t0, bool report) {
    const RopeArgs &a = args.r;
    const int size = 1 << a.page_log2, span = args.tok + size, i = threadIdx.x, warp = i >> 5;
    const bool in = i < 256;  // a thread for each row
    const int64_t t = t0 + i;
    int32_t slot = i < span && t < a.n_tokens ? a.slots[t] : -1, last = -1;
    if (i == 0 && t0 > 0) last = a.slots[t0 - 1];
    if (slot >= a.n_slots) {
        if (report) set_error(a.err, kErrBounds);
        slot = -1;
    }
    if (slot < 0) slot = -1;
    if (in) s.slot[i] = slot;
    if (i < 128) s.top[i] = 0;
    if (i == 0) s.end = int32_t(a.n_tokens - t0 < span ? a.n_tokens - t0 : span);  // no row behind the batch
    __syncthreads();
    if (in && i > 0) last = s.slot[i - 1];
    // a row that goes on where the one before it stands, in the same page
    const bool on = slot >= 0 && last >= 0 && slot == last + 1 && (slot & (size - 1)) != 0;
    const bool lead = i < args.tok && slot >= 0 && !on;
    if (i >= args.tok && i < span && !on) atomicMin(&s.end, i);
    const uint32_t leads = __ballot_sync(~0u, lead);
    if (in && (i & 31) == 0) s.leads[warp] = __popc(leads);
    __syncthreads();
    int before = __popc(leads & (~0u >> (31 - (i & 31)))), n = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        before += w < warp ? s.leads[w] : 0;
        n += s.leads[w];
    }
    // rows past the CTA's tokens are those of a run that goes on
    if (in) s.run[i] = int16_t(slot >= 0 && i < s.end ? before - 1 : -1);
    if (lead) {
        s.first[before - 1] = i;
        s.page[before - 1] = slot >> a.page_log2;
        s.row0[before - 1] = slot & (size - 1);
    }
    if (i == 0) s.first[n] = s.end;
    __syncthreads();
    return n;
}

// cos and sin of rows t0 .. t0 + n - 1 into cs[row][pair]; a row without a position stays.
template <int THREADS>
__device__ __forceinline__ void find_angles(const RopeArgs &a, float2 *cs, int64_t t0, int n) {
    const uint64_t *turns = a.turns;
    asm volatile("" : "+l"(turns));  // an ordinary load: of constant memory every lane's own would take a turn
    // a thread has one pair; no pairs, no angles, and rot_dim is at most 128
    const int at_once = a.pairs > 0 ? THREADS / a.pairs : 0;  // rows
    const int r0 = at_once > 0 ? threadIdx.x / a.pairs : 0, p = at_once > 0 ? threadIdx.x % a.pairs : 0;
    if (r0 >= at_once) return;
    const uint64_t step = turns[p];
    for (int r = r0; r < n; r += at_once) {
        const int32_t pos = a.positions[t0 + r];
        float sn = 0.0f, c = 1.0f;
        if (pos >= 0) {
            // The angle, a fraction of a turn, in two parts: 24 bits that f32 holds, and the
            // next ones by the first terms of sine and cosine.  (One f32 would move the
            // result by 2^-23: more rows would fall on the other side of a code's border.)
            const uint64_t frac = uint64_t(pos) * step;
            const int32_t hi = int32_t(uint32_t(frac >> 32) & 0xffffff00u);
            const float rest = float(uint32_t(frac >> 8)) * 8.71967124502158e-17f;  // 2 pi 2^-56: radians
            float s0, c0;
            sincospif(float(hi) * 4.656612873077393e-10f, &s0, &c0);
            c = fmaf(-rest, s0, c0);
            sn = fmaf(rest, c0, s0);
        }
        cs[r * a.pairs + p] = make_float2(c * a.factor, sn * a.factor);
    }
}

// The 16 channels of a row that a thread owns, rotated.  HALF: eight and their
// eight partners where they turn; else 16 neighbours.  ANY: of any alignment and
// rot_dim, element by element.
template <typename TI, bool HALF, bool ANY>
struct Row16 {
    int at0, at1;
    bool turn;

    __device__ __forceinline__ void place(const RopeArgs &a, int task, bool rotate) {
        turn = rotate && (ANY ? task * 16 < 2 * a.pairs : task < a.n_pairs_task);
        at0 = !ANY && HALF && turn ? task * 8 : task * 16;
        at1 = !ANY && HALF && turn ? a.half + task * 8 : task * 16 + 8;
    }
    __device__ __forceinline__ void load(const TI *in, float *x) const {
        load8<TI>(in + at0, x);
        load8<TI>(in + at1, x + 8);
    }
    // cs: the row's pairs
    __device__ __forceinline__ void rotate(const float2 *cs, int task, float *x) const {
        if (!turn) return;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 v = reinterpret_cast<const float4 *>(cs + task * 8)[i / 2];
            const float c[2] = {v.x, v.z}, s[2] = {v.y, v.w};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int p = HALF ? i + k : 2 * (i + k), q = HALF ? 8 + i + k : 2 * (i + k) + 1;
                const float u = x[p] * c[k] - x[q] * s[k], w = x[q] * c[k] + x[p] * s[k];
                x[p] = u;
                x[q] = w;
            }
        }
    }
    __device__ __forceinline__ void load_any(const RopeArgs &a, const float2 *cs, const TI *in, int task, float *x) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int ch = task * 16 + i;
            x[i] = to_f32<TI>(in[ch]);
            if (!turn || ch >= 2 * a.pairs) continue;
            const bool low = HALF ? ch < a.pairs : ch % 2 == 0;
            const float y = to_f32<TI>(in[HALF ? (low ? ch + a.pairs : ch - a.pairs) : ch ^ 1]);
            const float2 v = cs[HALF ? (low ? ch : ch - a.pairs) : ch / 2];
            x[i] = low ? x[i] * v.x - y * v.y : x[i] * v.x + y * v.y;
        }
    }
};

// q's rows t0 .. t0 + n - 1, all heads; n at most 16.
template <typename TI, int HD, bool HALF, bool ANY, int THREADS>
__device__ __forceinline__ void turn_rows(const StoreArgs &args, float2 *cs, int64_t t0, int n) {
    constexpr int kTasks = HD / 16, kLanes = THREADS / kTasks;
    const RopeArgs &a = args.r;
    const Group &g = a.g[0];
    const int task = threadIdx.x % kTasks, lane = threadIdx.x / kTasks;
    const int at_once = kLanes / n, r = lane % n, first = lane / n;  // heads at once
    Row16<TI, HALF, ANY> row;
    row.place(a, task, a.pairs > 0);
    find_angles<THREADS>(a, cs, t0, n);
    __syncthreads();
    const int64_t t = t0 + r;
    const bool there = first < at_once && a.positions[t] >= 0;
    const TI *in = static_cast<const TI *>(g.in) + t * g.in_tok;
    float x[2][16];  // rows of this turn and of the next
    if (!ANY && there && first < g.heads) row.load(in + first * g.in_head, x[0]);
#pragma unroll 2
    for (int k = 0; k * at_once < g.heads; ++k) {
        const int h = k * at_once + first;
        const bool mine = there && h < g.heads;
        float *y = x[k & 1];
        if constexpr (ANY) {
            if (mine) row.load_any(a, cs + r * a.pairs, in + h * g.in_head, task, y);
            __syncwarp();  // in place, no channel is written before its partner's thread has it
        } else {
            if (there && h + at_once < g.heads) row.load(in + (h + at_once) * g.in_head, x[(k + 1) & 1]);
            if (mine) row.rotate(cs + r * a.pairs, task, y);
        }
        if (!mine) continue;
        const int64_t at = t * g.out_tok + h * g.out_head;
        auto put = [&](auto *out) {
            using TO = std::remove_pointer_t<decltype(out)>;
            if constexpr (ANY) {
#pragma unroll
                for (int e = 0; e < 16; ++e) out[at + task * 16 + e] = from_f32<TO>(y[e]);
            } else {
                store8<TO>(out + at + row.at0, y);
                store8<TO>(out + at + row.at1, y + 8);
            }
        };
        if (args.q_f16 != 0) put(static_cast<__half *>(g.out));
        else put(static_cast<__nv_bfloat16 *>(g.out));
    }
}

template <typename TI, int HD, bool HALF, bool ANY, int THREADS>
__global__ void __launch_bounds__(THREADS, 2) store_kernel(const __grid_constant__ StoreArgs args) {
    constexpr int kTasks = HD / 16, kLanes = THREADS / kTasks;  // of a row; rows at once
    constexpr int kTurns = kWindow / kLanes;
    extern __shared__ __align__(16) float2 cs[];  // of the rows at hand
    __shared__ Runs sh;
    const RopeArgs &a = args.r;
    pdl_wait();
    int64_t t0 = int64_t(blockIdx.x) * args.tok;
    // q's CTAs, which only copy, between those of K and V, which mostly wait
    const int y = int(blockIdx.y), kv = args.k_ctas + a.n_kv, both = args.q_ctas < kv ? args.q_ctas : kv;
    const bool is_q = y < 2 * both ? y % 2 == 0 : args.q_ctas > kv;
    const int place = y < 2 * both ? y / 2 : y - both;
    if (is_q) {
        t0 += int64_t(place) * args.q_tok;
        const int64_t end = int64_t(blockIdx.x + 1) * args.tok < a.n_tokens ? int64_t(blockIdx.x + 1) * args.tok : a.n_tokens;
        const int n = int(end - t0 < args.q_tok ? end - t0 : args.q_tok);
        if (n > 0) turn_rows<TI, HD, HALF, ANY, THREADS>(args, cs, t0, n);
        return;
    }
    const int kind = place < args.k_ctas ? 0 : 1, h0 = kind == 0 ? place * args.k_heads : place - args.k_ctas;
    const int heads = kind == 1 ? 1 : a.n_kv - h0 < args.k_heads ? a.n_kv - h0 : args.k_heads;
    const Group &g = a.g[1 + kind];
    const int n = find_runs(args, sh, t0, place == 0);
    if (n == 0) return;
    const int size = 1 << a.page_log2;
    const int task = threadIdx.x % kTasks, lane = threadIdx.x / kTasks;
    Row16<TI, HALF, ANY> row;
    row.place(a, task, kind == 0 && a.pairs > 0);
    uint8_t *pages = static_cast<uint8_t *>(g.out);

    // as many runs at a time as the registers hold
    for (int ra = 0, rb; ra < n; ra = rb) {
        const int w0 = sh.first[ra];
        rb = n;
        if (sh.first[n] - w0 > kWindow)
            for (rb = ra + 1; rb < n && sh.first[rb + 1] - w0 <= kWindow; ++rb) {
            }
        const int w1 = sh.first[rb];
        if (kind == 0 && a.pairs > 0) {
            if (ra > 0) __syncthreads();
            find_angles<THREADS>(a, cs, t0 + w0, w1 - w0);
            __syncthreads();
        }
        int run[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int i = w0 + k * kLanes + lane;
            run[k] = i < w1 ? sh.run[i] : -1;
        }
        for (int h = h0; h < h0 + heads; ++h) {
            auto block_of = [&](int r) { return pages + ((int64_t(sh.page[r]) * a.n_kv + h) << a.page_log2) * HD; };
            // the scale that stands, for the thread that settles its run's
            const int my = ra + int(threadIdx.x);
            float *scale_at = nullptr, old = 0.0f;
            if (my < rb) {
                scale_at = args.scale[kind] + int64_t(sh.page[my]) * a.n_kv + h;
                if (sh.row0[my] > 0) old = *scale_at;
            }
            float x[kTurns][16];
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                if (ANY || run[k] < 0) continue;
                row.load(static_cast<const TI *>(g.in) + (t0 + w0 + k * kLanes + lane) * g.in_tok + h * g.in_head, x[k]);
            }
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                if (w0 + k * kLanes >= w1) break;
                const int i = k * kLanes + lane;  // row of the window
                float top = 0.0f;
                if (run[k] >= 0) {
                    if constexpr (ANY) row.load_any(a, cs + i * a.pairs, static_cast<const TI *>(g.in) + (t0 + w0 + i) * g.in_tok + h * g.in_head, task, x[k]);
                    else row.rotate(cs + i * a.pairs, task, x[k]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float v = fabsf(x[k][e]);
                        top = v <= FLT_MAX ? fmaxf(top, v) : top;
                    }
                }
#pragma unroll
                for (int d = 1; d < kTasks; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                if (run[k] >= 0 && task == 0) atomicMax(&sh.top[run[k]], __float_as_uint(top));
            }
            __syncthreads();
            if (my < rb) {  // scales only grow while a block keeps rows
                float s = scale_for(__uint_as_float(sh.top[my])), ratio = 1.0f;
                sh.top[my] = 0;  // for the next head
                if (sh.row0[my] > 0) {
                    if (!scale_ok(old)) set_error(a.err, kErrBounds);
                    else if (old >= s) s = old;
                    else ratio = old / s;
                }
                *scale_at = s;
                sh.scale[my] = s;
                sh.ratio[my] = ratio;
            }
            __syncthreads();
            // codes that stand before a run move to the new scale: a warp for each run
            for (int r = ra + int(threadIdx.x >> 5); r < rb; r += THREADS / 32) {
                const float ratio = sh.ratio[r];
                if (ratio == 1.0f) continue;
                uint4 *p = reinterpret_cast<uint4 *>(block_of(r));
#pragma unroll 4
                for (int i = threadIdx.x & 31; i < sh.row0[r] * HD / 16; i += 32) {
                    uint4 v = p[i];
                    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float y[4];
                        values4(w[e], y);
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] *= ratio;
                        w[e] = codes4(y);
                    }
                    p[i] = v;
                }
            }
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                if (run[k] < 0) continue;
                const float s = sh.scale[run[k]], inv = 1.0f / s;  // exact for a power of two
                if (pow2(s)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[k][e] *= inv;
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[k][e] /= s;
                }
                uint8_t *out = block_of(run[k]) + (sh.slot[w0 + k * kLanes + lane] & (size - 1)) * HD;
                if (row.at1 == row.at0 + 8) {
                    *reinterpret_cast<uint4 *>(out + row.at0) = make_uint4(codes4(x[k]), codes4(x[k] + 4), codes4(x[k] + 8), codes4(x[k] + 12));
                } else {
                    *reinterpret_cast<uint2 *>(out + row.at0) = make_uint2(codes4(x[k]), codes4(x[k] + 4));
                    *reinterpret_cast<uint2 *>(out + row.at1) = make_uint2(codes4(x[k] + 8), codes4(x[k] + 12));
                }
            }
        }
    }
}

template <typename TI, int HD, int THREADS>
cudaError_t launch_store(const StoreArgs &a, dim3 grid, bool any, bool half, int smem, cudaStream_t st) {
    const auto kern = any ? (half ? store_kernel<TI, HD, true, true, THREADS> : store_kernel<TI, HD, false, true, THREADS>)
                          : (half ? store_kernel<TI, HD, true, false, THREADS> : store_kernel<TI, HD, false, false, THREADS>);
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem);
    return e != cudaSuccess ? e : launch_pdl(kern, grid, dim3(THREADS), size_t(smem), st, a);
}

template <typename TI, int HD>
cudaError_t launch_store(StoreArgs &a, bool aligned, int layout, cudaStream_t st) {
    const bool any = !aligned || a.r.pairs % 8 != 0, half = layout == KVD_ROPE_HALF;
    // Many tokens: 128 to a CTA of 512 threads, which hold their rows, and four heads of K
    // for the angles.  Few: 16 tokens, one head, 256 threads, for more CTAs.  (8192 tokens
    // of 32 + 8 + 8 heads into pages of 128: 47 us, in the small form 91; 256 tokens: 5.4,
    // in the large form 13 to 20.  K and V alone take 24, q alone 32; kvd_rope_apply's
    // kernel turns q in 25.5, which in a launch of its own comes to 49 in all.)
    const bool many = a.r.n_tokens >= 2048;
    const int32_t size = 1 << a.r.page_log2;
    a.tok = many ? 128 : 16;
    a.k_heads = many ? 4 : 1;
    a.k_ctas = int32_t(ceil_div(a.r.n_kv, a.k_heads));
    a.q_tok = many ? 16 : 4;
    a.q_ctas = a.r.g[0].heads > 0 ? a.tok / a.q_tok : 0;
    const dim3 grid(unsigned(ceil_div(a.r.n_tokens, a.tok)), unsigned(a.k_ctas + a.r.n_kv + a.q_ctas));
    const int32_t rows = a.tok + size < kWindow ? a.tok + size : kWindow;
    const int smem = int(sizeof(float2)) * a.r.pairs * rows;
    return many ? launch_store<TI, HD, 512>(a, grid, any, half, smem, st) : launch_store<TI, HD, 256>(a, grid, any, half, smem, st);
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
    int32_t n_seq, max_pages, page_log2, n_kv, hd, heads;
};

constexpr int kReadRows = 32;  // rows of one CTA

// The last request b with cu_rows[b] <= t, by a warp: 32 places looked at at once.
__device__ __forceinline__ int32_t request_of(const ReadArgs &a, int64_t t) {
    int32_t lo = 0, hi = a.n_seq;  // cu_rows[lo] <= t, cu_rows[hi] > t
    const int32_t lane = threadIdx.x & 31;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool below = at < hi && (lane == 0 || a.cu_rows[at] <= t);
        const int32_t k = 31 - __clz(__ballot_sync(~0u, below));
        hi = lo + (k + 1) * step < hi ? lo + (k + 1) * step : hi;
        lo += k * step;
    }
    return lo;
}

// Where output row t of a request between lo and hi comes from: its page and row there;
// page -1 = nothing stands there (zeros), -2 = no request asked for it (left alone).
__device__ __forceinline__ int2 read_place(const ReadArgs &a, int64_t t, int32_t lo, int32_t hi) {
    if (t >= a.n_rows || t < a.cu_rows[0] || t >= a.cu_rows[a.n_seq]) return make_int2(-2, 0);
    while (hi > lo) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (a.cu_rows[mid] <= t) lo = mid;
        else hi = mid - 1;
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

// x s, which may have 28 bits, cut to 24 whose last one says, too, whether anything was cut
// off: rounding that to 22 bits or fewer rounds x s itself.  (Rounded to f32 first, a
// product just beside the middle of two values of 16 bits would lie on it.)
__device__ __forceinline__ float times_to_odd(float x, float s) {
    const float p = __fmul_rz(x, s);
    return fmaf(x, s, -p) != 0.0f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// HD / 16 threads for a row of a head, 16 channels each; a warp's rows follow one
// another in a page and in the output.  (Six CTAs to an SM: with the registers that the
// compiler would take, and five, a long read takes 397 us instead of 368.)
template <typename TP, typename TO, int HD>  // TP uint8_t: e4m3 codes with scales
__global__ void __launch_bounds__(256, 6) read_kernel(const __grid_constant__ ReadArgs a) {
    constexpr int kChunks = HD / 16;
    __shared__ int2 place[kReadRows];
    pdl_wait();
    const int64_t t0 = int64_t(blockIdx.x) * kReadRows;
    if (threadIdx.x < kReadRows) {
        const int64_t t1 = t0 + kReadRows - 1 < a.n_rows ? t0 + kReadRows - 1 : a.n_rows - 1;
        const int32_t lo = request_of(a, t0), hi = request_of(a, t1);
        place[threadIdx.x] = read_place(a, t0 + threadIdx.x, lo, hi);
    }
    __syncthreads();
    const int h0 = blockIdx.y * a.heads, heads = a.n_kv - h0 < a.heads ? a.n_kv - h0 : a.heads;
#pragma unroll 4
    for (int i = threadIdx.x; i < kReadRows * kChunks * 2 * heads; i += 256) {
        const int at = i % kChunks * 16, r = i / kChunks % kReadRows, kind = i / (kChunks * kReadRows) % 2, h = h0 + i / (kChunks * kReadRows * 2);
        const int2 from = place[r];
        if (from.x == -2) continue;
        float x[16];
        if (from.x < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.0f;
        } else {
            const int64_t block = int64_t(from.x) * a.n_kv + h;
            const TP *in = static_cast<const TP *>(a.pages[kind]) + ((block << a.page_log2) + from.y) * HD + at;
            if constexpr (sizeof(TP) == 1) {
                const uint4 v = *reinterpret_cast<const uint4 *>(in);
                const float s = scale_of(a.scale[kind][block], a.err);
                values4(v.x, x);
                values4(v.y, x + 4);
                values4(v.z, x + 8);
                values4(v.w, x + 12);
                if (sizeof(TO) == 4 || pow2(s)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] *= s;
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = times_to_odd(x[e], s);
                }
            } else {
                load8<TP>(in, x);
                load8<TP>(in + 8, x + 8);
            }
        }
        TO *out = static_cast<TO *>(a.out[kind]) + (t0 + r) * a.out_tok[kind] + int64_t(h) * a.out_head[kind] + at;
        store8<TO>(out, x);
        store8<TO>(out + 8, x + 8);
    }
}

template <typename TP, int HD>
cudaError_t launch_read(ReadArgs &a, int32_t out_dtype, cudaStream_t st) {
    // all heads to a CTA once that leaves CTAs enough for every SM several times
    a.heads = ceil_div(a.n_rows, kReadRows) >= 152 * 8 ? a.n_kv : 1;
    const dim3 grid(unsigned(ceil_div(a.n_rows, kReadRows)), unsigned(ceil_div(a.n_kv, a.heads)));
    const auto kern = out_dtype == KVD_T_F32   ? read_kernel<TP, float, HD>
                      : out_dtype == KVD_T_F16 ? read_kernel<TP, __half, HD>
                                               : read_kernel<TP, __nv_bfloat16, HD>;
    return launch_pdl(kern, grid, dim3(256), 0, st, a);
}
template <typename TP>
cudaError_t launch_read(ReadArgs &a, int32_t out_dtype, cudaStream_t st) {
    return a.hd == 64 ? launch_read<TP, 64>(a, out_dtype, st) : launch_read<TP, 128>(a, out_dtype, st);
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
    bool aligned = true;
    if (q != nullptr) {
        if (qb != 2 || (in_dtype != KVD_T_F32 && in_dtype != q_dtype)) return KVD_EINVAL;
        if (n_q < 1 || n_q > 1024 || !rows_ok(q, n_tokens, n_q, ib) || !rows_ok(q_out, n_tokens, n_q, qb)) return KVD_EINVAL;
        a.r.g[0] = group_of(q, q_out, n_q);
        aligned = aligned16(a.r.g[0], false, ib, qb);
        a.q_f16 = q_dtype == KVD_T_F16 ? 1 : 0;
    }
    const kvd_rows kp = {k_pages, 0, 0}, vp = {v_pages, 0, 0};
    a.r.g[1] = group_of(k, &kp, n_kv);
    a.r.g[2] = group_of(v, &vp, n_kv);
    aligned = aligned && aligned16(a.r.g[1], true, ib, 1) && aligned16(a.r.g[2], true, ib, 1);
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
    const auto go = [&](auto type) {
        using TI = decltype(type);
        return head_dim == 64 ? launch_store<TI, 64>(a, aligned, layout, st) : launch_store<TI, 128>(a, aligned, layout, st);
    };
    const cudaError_t e = in_dtype == KVD_T_F32 ? go(float()) : in_dtype == KVD_T_F16 ? go(__half()) : go(__nv_bfloat16());
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
