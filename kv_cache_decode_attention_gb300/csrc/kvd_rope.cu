// kvd_rope.cu -- rotary positions: the frequency tables, the rotation of q and
// k rows, and the paged append that rotates and writes K and V to their slots.
//
// Pair i of a head turns by position * f_i.  The table holds f_i / 2 pi as a
// 64-bit fraction of a turn, so position * table is the angle modulo one turn
// in one wrapping integer product.  The table is computed in f64 and right to 2^-54
// turns, and the product adds nothing: position * 2^-54 turns (an f32 angle of 10^6
// radians would be off by 0.03, this one by 4e-10).  Its top 32 bits, 2^-32 of a
// turn, become an f32 between -1 and 1: 2^-26 turns.
//
// Bound by HBM: every row is read and written once.  A CTA computes the cos
// and sin of its tokens once into shared memory and each thread keeps the
// eight pairs of its place in the head in registers while it walks the heads,
// so the trigonometry is paid once per (token, pair) and not per head.
//
// Measured: 8192 tokens of 40 bf16 heads of 128 30.5 us, 5.5 TB/s (a copy runs at
// 6.7); an append of 7800 tokens, f32 in, f16 pages, 31.1 us, 5.8 TB/s; of 256
// tokens 3.2 us and one token 2.8, where an empty launch takes 2.

#include <cmath>

#include "kvd_rope.cuh"

namespace kvd {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTok = 4;       // tokens of one CTA

// cos and sin of the CTA's tokens into cs[token][pair].
__device__ __forceinline__ void fill_angles(const RopeArgs &a, float2 *cs, int64_t tok0, int n_tok) {
    // The table lies in the kernel's parameters.  Read through a plain pointer:
    // a load that the compiler knows to be of constant memory takes a turn for
    // every different address of a warp, an ordinary one takes the line at once.
    const uint64_t *turns = a.turns;
    asm volatile("" : "+l"(turns));
    for (int i = threadIdx.x; i < n_tok * a.pairs; i += blockDim.x) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        const int32_t pos = a.positions[tok0 + t];
        float s = 0.0f, c = 1.0f;
        if (pos >= 0) {
            const uint64_t frac = uint64_t(pos) * turns[p];
            // signed top 32 bits: the turn in [-1/2, 1/2), as half turns for sincospi
            sincospif(float(int32_t(frac >> 32)) * 4.656612873077393e-10f, &s, &c);
        }
        cs[t * a.pairs + p] = make_float2(c * a.factor, s * a.factor);
    }
}

// Where the rows of one token go: its position (negative = leave the outputs
// of kvd_rope_apply and q alone) and its slot (negative or past the pool =
// leave the pages alone).
struct Place {
    int32_t pos, slot;
};
__device__ __forceinline__ Place place_of(const RopeArgs &a, int64_t tok) {
    Place p = {a.positions[tok], -1};
    if (a.paged) {
        p.slot = a.slots[tok];
        if (p.slot >= a.n_slots) {
            set_error(a.err, kErrBounds);
            p.slot = -1;
        }
    }
    return p;
}
template <typename TO>
__device__ __forceinline__ TO *row_out(const RopeArgs &a, int gi, int64_t tok, int head, const Place &p) {
    const Group &g = a.g[gi];
    TO *out = static_cast<TO *>(g.out);
    if (gi == 0 || !a.paged) return p.pos < 0 ? nullptr : out + tok * g.out_tok + head * g.out_head;
    if (p.slot < 0) return nullptr;
    const int64_t page = p.slot >> a.page_log2, row = p.slot & ((1 << a.page_log2) - 1);
    return out + (((page * a.n_kv + head) << a.page_log2) + row) * a.hd;
}

// Vector form: a thread owns 16 channels of a head -- eight pairs, or 16
// channels that only pass through -- and walks the heads of one token.
// Needs 16-byte aligned rows, head_dim % 16 == 0 and rot_dim % 16 == 0.
template <typename TI, typename TO, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const __grid_constant__ RopeArgs a, int tok_per_cta) {
    extern __shared__ float2 cs[];
    pdl_wait();
    const int64_t tok0 = int64_t(blockIdx.x) * tok_per_cta;
    const int n_tok = int(a.n_tokens - tok0 < tok_per_cta ? a.n_tokens - tok0 : tok_per_cta);
    fill_angles(a, cs, tok0, n_tok);
    __syncthreads();
    const int lanes = blockDim.x / a.n_tasks;           // rows in flight
    const int task = threadIdx.x % a.n_tasks, lane = threadIdx.x / a.n_tasks;
    const int per_tok = lanes / tok_per_cta;            // of them for one token
    const int t = lane / per_tok, first = lane - t * per_tok;
    if (t >= n_tok || lane >= per_tok * tok_per_cta) return;
    const int64_t tok = tok0 + t;
    const Place place = place_of(a, tok);
    const bool turn = task < a.n_pairs_task;
    float c[8], s[8];
    if (turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = cs[t * a.pairs + task * 8 + i];
            c[i] = v.x;
            s[i] = v.y;
        }
    }
    // where this thread's two runs of eight channels start
    const int at0 = turn && HALF ? task * 8 : task * 16;
    const int at1 = turn && HALF ? a.half + task * 8 : task * 16 + 8;
    const int total = a.g[0].heads + a.g[1].heads + a.g[2].heads;
    for (int h = first; h < total; h += per_tok) {
        int gi = 0, head = h;
        if (head >= a.g[0].heads) head -= a.g[0].heads, gi = 1;
        if (gi == 1 && head >= a.g[1].heads) head -= a.g[1].heads, gi = 2;
        const Group &g = a.g[gi];
        TO *out = row_out<TO>(a, gi, tok, head, place);
        if (out == nullptr) continue;
        const TI *in = static_cast<const TI *>(g.in) + tok * g.in_tok + head * g.in_head;
        float x[8], y[8];
        load8<TI>(in + at0, x);
        load8<TI>(in + at1, y);
        if (turn && gi < 2) {
            if (HALF) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x[i] * c[i] - y[i] * s[i], w = y[i] * c[i] + x[i] * s[i];
                    x[i] = u;
                    y[i] = w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
                    x[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
                    x[2 * i] = u;
                    const float w = y[2 * i] * c[4 + i] - y[2 * i + 1] * s[4 + i];
                    y[2 * i + 1] = y[2 * i + 1] * c[4 + i] + y[2 * i] * s[4 + i];
                    y[2 * i] = w;
                }
            }
        }
        store8<TO>(out + at0, x);
        store8<TO>(out + at1, y);
    }
}

// A rot_dim that is no multiple of 16, in rows that allow 16-byte accesses: a
// thread owns eight neighbouring channels.  Interleaved partners are its own;
// the other layout's lie in other threads of the row, which is one warp's
// (head_dim 64, 128 or 256), and come through shared memory.  Bound by issue, not by
// memory (8192 tokens of 40 heads of 128, 70 rotated: 69 us, issue slots 69% busy,
// DRAM 22%): eight angles from shared memory for every head and channel-wise
// choices, half of the shared-memory wavefronts bank conflicts.
template <typename TI, typename TO, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_part_kernel(const __grid_constant__ RopeArgs a, int tok_per_cta) {
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float row[HALF ? kRopeThreads : 1][9];  // 9: a thread's eight values start in another bank
    pdl_wait();
    const int64_t tok0 = int64_t(blockIdx.x) * tok_per_cta;
    const int n_tok = int(a.n_tokens - tok0 < tok_per_cta ? a.n_tokens - tok0 : tok_per_cta);
    fill_angles(a, cs, tok0, n_tok);
    __syncthreads();
    const int chunks = a.hd / 8, lanes = kRopeThreads / chunks;
    const int chunk = threadIdx.x % chunks, lane = threadIdx.x / chunks, base = threadIdx.x - chunk;
    const int total = a.g[0].heads + a.g[1].heads + a.g[2].heads, rot = 2 * a.pairs;
    for (int t = 0; t < n_tok; ++t) {
        const int64_t tok = tok0 + t;
        const Place place = place_of(a, tok);
        const float2 *angle = cs + t * a.pairs;
        for (int h0 = 0; h0 < total; h0 += lanes) {
            int gi = 0, head = h0 + lane;
            const bool there = head < total;
            if (head >= a.g[0].heads) head -= a.g[0].heads, gi = 1;
            if (gi == 1 && head >= a.g[1].heads) head -= a.g[1].heads, gi = 2;
            if (!there) gi = 0, head = 0;
            const Group &g = a.g[gi];
            TO *out = there ? row_out<TO>(a, gi, tok, head, place) : nullptr;
            float x[8], y[8];
            if (out != nullptr) load8<TI>(static_cast<const TI *>(g.in) + tok * g.in_tok + head * g.in_head + chunk * 8, x);
            const bool turn = gi < 2 && chunk * 8 < rot;
            if (HALF) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) row[threadIdx.x][i] = x[i];
                __syncwarp();
            }
            if (out == nullptr) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ch = chunk * 8 + i;
                y[i] = x[i];
                if (!turn || ch >= rot) continue;
                if (HALF) {
                    const bool low = ch < a.pairs;
                    const int other = low ? ch + a.pairs : ch - a.pairs;
                    const float2 v = angle[low ? ch : other];
                    const float z = row[base + other / 8][other % 8];
                    y[i] = low ? x[i] * v.x - z * v.y : x[i] * v.x + z * v.y;
                } else {
                    const float2 v = angle[ch / 2];
                    y[i] = i % 2 == 0 ? x[i] * v.x - x[i | 1] * v.y : x[i] * v.x + x[i & 6] * v.y;
                }
            }
            store8<TO>(out + chunk * 8, y);
        }
    }
}

// Any other size, stride or alignment: one thread per pair or plain channel.
// (8192 tokens of 40 heads of 128, 70 rotated channels: 120 us, rope_part_kernel 69;
// 256 tokens: 8.7 and 4.8.  Issue slots 68% busy with index arithmetic and accesses
// of one element.)
template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const __grid_constant__ RopeArgs a, int interleaved) {
    extern __shared__ float2 cs[];
    pdl_wait();
    const int64_t tok = blockIdx.x;
    fill_angles(a, cs, tok, 1);
    __syncthreads();
    const Place place = place_of(a, tok);
    const int rot = 2 * a.pairs, per_row = a.hd - a.pairs;  // pairs, then the channels past rot_dim
    const int total = a.g[0].heads + a.g[1].heads + a.g[2].heads;
    for (int i = threadIdx.x; i < total * per_row; i += blockDim.x) {
        const int h = i / per_row, e = i - h * per_row;
        int gi = 0, head = h;
        if (head >= a.g[0].heads) head -= a.g[0].heads, gi = 1;
        if (gi == 1 && head >= a.g[1].heads) head -= a.g[1].heads, gi = 2;
        const Group &g = a.g[gi];
        TO *out = row_out<TO>(a, gi, tok, head, place);
        if (out == nullptr) continue;
        const TI *in = static_cast<const TI *>(g.in) + tok * g.in_tok + head * g.in_head;
        if (e >= a.pairs) {
            const int at = rot + e - a.pairs;
            out[at] = from_f32<TO>(to_f32<TI>(in[at]));
            continue;
        }
        const int p = interleaved ? 2 * e : e, r = interleaved ? 2 * e + 1 : e + a.pairs;
        const float x = to_f32<TI>(in[p]), y = to_f32<TI>(in[r]);
        const float2 v = gi < 2 ? cs[e] : make_float2(1.0f, 0.0f);
        out[p] = from_f32<TO>(gi < 2 ? x * v.x - y * v.y : x);
        out[r] = from_f32<TO>(gi < 2 ? y * v.x + x * v.y : y);
    }
}

template <typename TI, typename TO>
cudaError_t launch_rope(const RopeArgs &a, bool aligned, int layout, cudaStream_t st) {
    const bool vec = aligned && a.hd % 16 == 0 && a.pairs % 8 == 0;
    if (!vec && aligned && (a.hd == 64 || a.hd == 128 || a.hd == 256)) {
        const int tok = a.n_tokens >= 152 * 2 * kMaxTok ? kMaxTok : a.n_tokens >= 152 * 4 ? 2 : 1;
        const dim3 grid(unsigned(ceil_div(a.n_tokens, tok)));
        const size_t smem = sizeof(float2) * size_t(a.pairs) * tok;
        return layout == KVD_ROPE_HALF ? launch_pdl(rope_part_kernel<TI, TO, true>, grid, dim3(kRopeThreads), smem, st, a, tok)
                                       : launch_pdl(rope_part_kernel<TI, TO, false>, grid, dim3(kRopeThreads), smem, st, a, tok);
    }
    if (!vec) {
        const size_t smem = sizeof(float2) * size_t(a.pairs);
        return launch_pdl(rope_any_kernel<TI, TO>, dim3(unsigned(a.n_tokens)), dim3(kRopeThreads), smem, st, a,
                          layout == KVD_ROPE_INTERLEAVED ? 1 : 0);
    }
    // Several tokens to a CTA amortise its prologue once there are CTAs enough
    // for every SM twice over; fewer tokens than that spread wider.  (8192 tokens of
    // 40 heads: four to a CTA 30.4 us, one 41.3; 1500: four 6.1, one 7.3; 64: four
    // 4.0, one 2.5.  Two from four CTAs an SM on: 900 tokens 4.2, one 5.8, four 5.0;
    // 608: 3.8, 3.8, 4.1; 1215: 4.9, 6.5, 5.1; appends alike.  rope_part_kernel takes
    // the same: 900 tokens two 9.4, one 10.1, four 14.2; 608: 7.9, 6.6, 12.8.)
    const int lanes = kRopeThreads / a.n_tasks;
    int tok = a.n_tokens >= 152 * 2 * kMaxTok ? kMaxTok : a.n_tokens >= 152 * 4 ? 2 : 1;
    while (tok > lanes) tok >>= 1;
    const dim3 grid(unsigned(ceil_div(a.n_tokens, tok)));
    const size_t smem = sizeof(float2) * size_t(a.pairs) * tok;
    return layout == KVD_ROPE_HALF
               ? launch_pdl(rope_vec_kernel<TI, TO, true>, grid, dim3(kRopeThreads), smem, st, a, tok)
               : launch_pdl(rope_vec_kernel<TI, TO, false>, grid, dim3(kRopeThreads), smem, st, a, tok);
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_rope_init(kvd_rope *R, const kvd_rope_config *c) {
    if (R == nullptr || c == nullptr) return KVD_EINVAL;
    if (c->rot_dim < 2 || c->rot_dim > 2 * kMaxPairs || c->rot_dim % 2 != 0) return KVD_EINVAL;
    if (c->layout != KVD_ROPE_INTERLEAVED && c->layout != KVD_ROPE_HALF) return KVD_EINVAL;
    if (c->scaling < KVD_ROPE_NONE || c->scaling > KVD_ROPE_BANDS) return KVD_EINVAL;
    if (!std::isfinite(c->base) || c->base <= 1.0) return KVD_EINVAL;
    if (!std::isfinite(c->attention_factor) || c->attention_factor < 0.0) return KVD_EINVAL;
    const bool scaled = c->scaling != KVD_ROPE_NONE;
    const double factor = scaled ? c->factor : 1.0;
    if (!std::isfinite(factor) || factor < 1.0) return KVD_EINVAL;
    if (c->scaling == KVD_ROPE_NTK && c->rot_dim == 2) return KVD_EINVAL;
    if (c->scaling == KVD_ROPE_YARN || c->scaling == KVD_ROPE_BANDS)
        if (!std::isfinite(c->original_len) || c->original_len < 1.0) return KVD_EINVAL;
    if (c->scaling == KVD_ROPE_YARN)
        if (!std::isfinite(c->beta_fast) || !(c->beta_fast > c->beta_slow) || !(c->beta_slow > 0.0)) return KVD_EINVAL;
    if (c->scaling == KVD_ROPE_BANDS)
        if (!std::isfinite(c->high_freq_factor) || !(c->high_freq_factor > c->low_freq_factor) || !(c->low_freq_factor >= 0.0))
            return KVD_EINVAL;
    const double two_pi = 6.283185307179586476925286766559;
    const double rot = c->rot_dim;
    const double base = c->scaling == KVD_ROPE_NTK ? c->base * std::pow(factor, rot / (rot - 2.0)) : c->base;
    if (!std::isfinite(base)) return KVD_EINVAL;
    double low = 0.0, high = 0.0;
    if (c->scaling == KVD_ROPE_YARN) {
        const double per_turn = rot / (2.0 * std::log(base));
        low = std::fmax(std::floor(per_turn * std::log(c->original_len / (c->beta_fast * two_pi))), 0.0);
        high = std::fmin(std::ceil(per_turn * std::log(c->original_len / (c->beta_slow * two_pi))), rot - 1.0);
    }
    Rope r;
    std::memset(&r, 0, sizeof(r));
    r.magic = kRopeMagic;
    r.rot_dim = c->rot_dim;
    r.layout = c->layout;
    const double mul = c->attention_factor > 0.0 ? c->attention_factor
                       : c->scaling == KVD_ROPE_YARN ? 0.1 * std::log(factor) + 1.0
                                                     : 1.0;
    r.factor = float(mul);
    for (int i = 0; i < c->rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (c->scaling == KVD_ROPE_LINEAR) f /= factor;
        if (c->scaling == KVD_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 1e-3), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        if (c->scaling == KVD_ROPE_BANDS) {
            const double turns = c->original_len * f / two_pi;
            const double mix = std::fmin(
                std::fmax((turns - c->low_freq_factor) / (c->high_freq_factor - c->low_freq_factor), 0.0), 1.0);
            f = f / factor * (1.0 - mix) + f * mix;
        }
        r.turns[i] = uint64_t(std::ldexp(f / two_pi, 64));  // f <= 1, so the product is below 2^62
    }
    std::memcpy(R, &r, sizeof(r));
    return KVD_OK;
}

extern "C" kvd_status kvd_rope_apply(const kvd_rope *R, const kvd_rows *q, const kvd_rows *q_out, int32_t n_q,
                                     const kvd_rows *k, const kvd_rows *k_out, int32_t n_kv, int32_t head_dim,
                                     int32_t dtype, const int32_t *positions, int64_t n_tokens, void *stream) {
    KVD_NVTX_RANGE("kvd_rope_apply");
    const Rope *r = checked_rope(R);
    const int bytes = dtype_bytes(dtype);
    if (r == nullptr || bytes == 0 || (positions == nullptr && n_tokens > 0) || n_tokens < 0 || n_tokens > kMaxTokens) return KVD_EINVAL;
    if (head_dim < r->rot_dim || head_dim > 512) return KVD_EINVAL;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (q == nullptr && k == nullptr))
        return KVD_EINVAL;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    bool aligned = true;
    const kvd_rows *in[2] = {q, k}, *out[2] = {q_out, k_out};
    const int32_t heads[2] = {n_q, n_kv};
    for (int i = 0; i < 2; ++i) {
        if (in[i] == nullptr) continue;
        if (heads[i] < 1 || heads[i] > 1024) return KVD_EINVAL;
        if (!rows_ok(in[i], n_tokens, heads[i], bytes) || !rows_ok(out[i], n_tokens, heads[i], bytes)) return KVD_EINVAL;
        a.g[i] = group_of(in[i], out[i], heads[i]);
        aligned = aligned && aligned16(a.g[i], false, bytes, bytes);
    }
    if (n_tokens == 0) return KVD_OK;
    // Rows turn in place, one by one; an output shares memory with nothing else.
    View vi[2], vo[2];
    for (int i = 0; i < 2; ++i) {
        if (in[i] == nullptr) continue;
        vi[i] = view_of(in[i], n_tokens, heads[i], head_dim, bytes);
        vo[i] = view_of(out[i], n_tokens, heads[i], head_dim, bytes);
        if (!rows_apart(vo[i]) || !(same_rows(vi[i], vo[i]) || views_apart(vi[i], vo[i]))) return KVD_EINVAL;
    }
    if (q != nullptr && k != nullptr &&
        !(views_apart(vo[0], vo[1]) && views_apart(vo[0], vi[1]) && views_apart(vo[1], vi[0])))
        return KVD_EINVAL;
    set_rope(&a, r, head_dim);
    a.positions = positions;
    a.n_tokens = n_tokens;
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = dtype == KVD_T_F32   ? launch_rope<float, float>(a, aligned, r->layout, st)
                          : dtype == KVD_T_F16 ? launch_rope<__half, __half>(a, aligned, r->layout, st)
                                               : launch_rope<__nv_bfloat16, __nv_bfloat16>(a, aligned, r->layout, st);
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}

extern "C" kvd_status kv_paged_append(const kvd_rope *R, const kvd_rows *q, const kvd_rows *q_out, int32_t n_q,
                                      const kvd_rows *k, const kvd_rows *v, int32_t n_kv, int32_t head_dim,
                                      int32_t in_dtype, int32_t page_dtype, const int32_t *positions,
                                      const int32_t *slots, int64_t n_tokens, void *k_pages, void *v_pages,
                                      int64_t n_pages, int32_t page_size, uint32_t *err, void *stream) {
    KVD_NVTX_RANGE("kv_paged_append");
    const Rope *r = checked_rope(R);
    const int ib = dtype_bytes(in_dtype), ob = dtype_bytes(page_dtype);
    if (R != nullptr && r == nullptr) return KVD_EINVAL;
    if (ib == 0 || ob != 2 || (in_dtype != KVD_T_F32 && in_dtype != page_dtype)) return KVD_EINVAL;
    if (head_dim != 64 && head_dim != 128) return KVD_EINVAL;
    if (r != nullptr && r->rot_dim > head_dim) return KVD_EINVAL;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return KVD_EINVAL;
    if (n_pages < 1 || n_pages * page_size >= (int64_t(1) << 31) || n_pages >= (int64_t(1) << 31)) return KVD_EINVAL;
    if (n_tokens < 0 || n_tokens > kMaxTokens || n_kv < 1 || n_kv > 1024) return KVD_EINVAL;
    if ((n_tokens > 0 && (positions == nullptr || slots == nullptr)) || err == nullptr || (q == nullptr) != (q_out == nullptr)) return KVD_EINVAL;
    if (k_pages == nullptr || v_pages == nullptr ||
        ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15) != 0)
        return KVD_EINVAL;
    if (!rows_ok(k, n_tokens, n_kv, ib) || !rows_ok(v, n_tokens, n_kv, ib)) return KVD_EINVAL;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    bool aligned = true;
    if (q != nullptr) {
        if (n_q < 1 || n_q > 1024 || !rows_ok(q, n_tokens, n_q, ib) || !rows_ok(q_out, n_tokens, n_q, ob)) return KVD_EINVAL;
        a.g[0] = group_of(q, q_out, n_q);
        aligned = aligned16(a.g[0], false, ib, ob);
    }
    const kvd_rows kp = {k_pages, 0, 0}, vp = {v_pages, 0, 0};
    a.g[1] = group_of(k, &kp, n_kv);
    a.g[2] = group_of(v, &vp, n_kv);
    aligned = aligned && aligned16(a.g[1], true, ib, ob) && aligned16(a.g[2], true, ib, ob);
    if (n_tokens == 0) return KVD_OK;
    {
        // q turns in place; else what is written shares memory with nothing else
        const int64_t pages = n_pages * page_size * n_kv * head_dim * ob;
        const View vk = view_of(k, n_tokens, n_kv, head_dim, ib), vv = view_of(v, n_tokens, n_kv, head_dim, ib);
        const View pk = make_range(k_pages, pages), pv = make_range(v_pages, pages);
        bool ok = views_apart(pk, pv) && views_apart(vk, pk) && views_apart(vk, pv) && views_apart(vv, pk) && views_apart(vv, pv);
        if (q != nullptr) {
            const View vq = view_of(q, n_tokens, n_q, head_dim, ib), vo = view_of(q_out, n_tokens, n_q, head_dim, ob);
            ok = ok && rows_apart(vo) && (same_rows(vq, vo) || views_apart(vq, vo)) && views_apart(vo, vk) && views_apart(vo, vv) &&
                 views_apart(vo, pk) && views_apart(vo, pv) && views_apart(vq, pk) && views_apart(vq, pv);
        }
        if (!ok) return KVD_EINVAL;
    }
    set_rope(&a, r, head_dim);
    a.paged = 1;
    a.n_kv = n_kv;
    a.page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    a.n_slots = n_pages * page_size;
    a.positions = positions;
    a.slots = slots;
    a.n_tokens = n_tokens;
    a.err = err;
    const int layout = r != nullptr ? r->layout : KVD_ROPE_HALF;
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (page_dtype == KVD_T_F16)
        e = in_dtype == KVD_T_F32 ? launch_rope<float, __half>(a, aligned, layout, st)
                                  : launch_rope<__half, __half>(a, aligned, layout, st);
    else
        e = in_dtype == KVD_T_F32 ? launch_rope<float, __nv_bfloat16>(a, aligned, layout, st)
                                  : launch_rope<__nv_bfloat16, __nv_bfloat16>(a, aligned, layout, st);
    return e == cudaSuccess ? KVD_OK : KVD_ECUDA;
}
