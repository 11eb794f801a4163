// kvd_rope.cuh -- frequency tables, row access and angles, shared by the rotation
// and by the appends that rotate.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "kvd_internal.cuh"
#include "kvd_views.h"

namespace kvd {

constexpr int kMaxPairs = 256;   // rot_dim <= 512
constexpr int32_t kRopeMagic = 0x4b564452;  // "KVDR"

struct Rope {
    int32_t magic, rot_dim, layout;
    float factor;                // multiplies cos and sin
    uint64_t turns[kMaxPairs];   // f_i / 2 pi in units of 2^-64 turns
};
static_assert(sizeof(Rope) <= sizeof(kvd_rope), "kvd_rope too small");

// One launch: up to three groups of heads (q, k, v) with their outputs.
struct Group {
    const void *in;
    void *out;
    int64_t in_tok, in_head, out_tok, out_head;  // strides in elements
    int32_t heads;
};
struct RopeArgs {
    Group g[3];          // q, k, v; heads 0 = absent
    int32_t paged;       // k and v outputs are pages addressed by slot
    int32_t hd, pairs, half, n_pairs_task, n_tasks;
    int32_t page_log2, n_kv;
    int64_t n_slots, n_tokens;
    const int32_t *positions, *slots;
    uint32_t *err;
    float factor;
    uint64_t turns[kMaxPairs];
};

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight values in 16-byte pieces.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float *x) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            T t[2];
            memcpy(t, &w[i], 4);
            x[2 * i] = to_f32<T>(t[0]);
            x[2 * i + 1] = to_f32<T>(t[1]);
        }
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float *x) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T t[2] = {from_f32<T>(x[2 * i]), from_f32<T>(x[2 * i + 1])};
            memcpy(&w[i], t, 4);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

inline int dtype_bytes(int32_t t) { return t == KVD_T_F32 ? 4 : (t == KVD_T_F16 || t == KVD_T_BF16) ? 2 : 0; }

inline bool rows_ok(const kvd_rows *r, int64_t tokens, int32_t heads, int bytes) {
    if (r == nullptr || (r->data == nullptr && tokens > 0) || (reinterpret_cast<uintptr_t>(r->data) % bytes) != 0) return false;
    const int64_t lim = int64_t(1) << 40;
    return (tokens <= 1 || (r->token_stride >= 0 && r->token_stride < lim)) &&
           (heads <= 1 || (r->head_stride >= 0 && r->head_stride < lim));
}

inline bool aligned16(const Group &g, bool paged_out, int in_bytes, int out_bytes) {
    if (g.heads == 0) return true;
    if ((reinterpret_cast<uintptr_t>(g.in) | reinterpret_cast<uintptr_t>(g.out)) & 15) return false;
    if ((g.in_tok * in_bytes) & 15 || (g.in_head * in_bytes) & 15) return false;
    return paged_out || !((g.out_tok * out_bytes) & 15 || (g.out_head * out_bytes) & 15);
}

inline const Rope *checked_rope(const kvd_rope *R) {
    const Rope *r = reinterpret_cast<const Rope *>(R);
    return r != nullptr && r->magic == kRopeMagic ? r : nullptr;
}

inline void set_rope(RopeArgs *a, const Rope *r, int32_t hd) {
    a->hd = hd;
    a->pairs = r != nullptr ? r->rot_dim / 2 : 0;
    a->half = a->pairs;
    a->n_tasks = hd / 16;
    a->n_pairs_task = a->pairs / 8;
    a->factor = r != nullptr ? r->factor : 1.0f;
    if (r != nullptr) std::memcpy(a->turns, r->turns, sizeof(uint64_t) * size_t(a->pairs));
}

inline Group group_of(const kvd_rows *in, const kvd_rows *out, int32_t heads) {
    Group g = {};
    g.in = in->data;
    g.in_tok = in->token_stride;
    g.in_head = in->head_stride;
    g.out = out->data;
    g.out_tok = out->token_stride;
    g.out_head = out->head_stride;
    g.heads = heads;
    return g;
}

inline View view_of(const kvd_rows *r, int64_t tokens, int32_t heads, int32_t hd, int bytes) {
    return make_view(r->data, r->token_stride, r->head_stride, tokens, heads, hd, bytes);
}

constexpr int64_t kMaxTokens = int64_t(1) << 30;

}  // namespace kvd
