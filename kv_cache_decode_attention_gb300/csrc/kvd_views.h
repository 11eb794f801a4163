// kvd_views.h -- which [token][head][row] views of memory share bytes (host only).
//
// A view is the set of bytes at + i token + j head + [0, row), i < tokens, j < heads.
// The checks prove that views are apart or they say that they may not be: exact for
// the views that slices and transpositions of contiguous arrays make, and on the
// safe side for any other strides.
#pragma once

#include <cstdint>
#include <numeric>

namespace kvd {

struct View {
    uintptr_t at;
    int64_t token, head;    // strides in bytes, >= 0; 0 for an axis with one entry
    int64_t tokens, heads;  // >= 1
    int64_t row;            // bytes
};

inline View make_view(const void *data, int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t heads, int64_t hd,
                      int64_t bytes) {
    return {reinterpret_cast<uintptr_t>(data), tokens > 1 ? token_stride * bytes : 0, heads > 1 ? head_stride * bytes : 0,
            tokens, heads, hd * bytes};
}
inline View make_range(const void *data, int64_t bytes) { return {reinterpret_cast<uintptr_t>(data), 0, 0, 1, 1, bytes}; }

// No two rows of the view share a byte: one axis' rows lie side by side and the
// other axis steps over all of them.
inline bool rows_apart(const View &v) {
    using Wide = __int128;
    const auto nested = [&](int64_t inner, int64_t n_inner, int64_t outer, int64_t n_outer) {
        return (n_inner == 1 || inner >= v.row) && (n_outer == 1 || Wide(outer) >= Wide(inner) * (n_inner - 1) + v.row);
    };
    return nested(v.head, v.heads, v.token, v.tokens) || nested(v.token, v.tokens, v.head, v.heads);
}

// No byte belongs to both views.  Either their ranges are apart, or they are modulo
// the greatest common divisor of some of the strides (heads or channels of one
// array beside one another).
inline bool views_apart(const View &a, const View &b) {
    using Wide = __int128;
    for (int mask = 0; mask < 4; ++mask) {
        uint64_t g = 0;
        Wide ea = a.row, eb = b.row;  // what the axes that are left span
        const auto axis = [&](bool modulo, int64_t stride, int64_t n, Wide &extent) {
            if (modulo) g = std::gcd(g, uint64_t(stride));
            else extent += Wide(stride) * (n - 1);
        };
        axis(mask & 1, a.token, a.tokens, ea);
        axis(mask & 2, a.head, a.heads, ea);
        axis(mask & 1, b.token, b.tokens, eb);
        axis(mask & 2, b.head, b.heads, eb);
        if (mask == 0) {
            if (Wide(a.at) + ea <= Wide(b.at) || Wide(b.at) + eb <= Wide(a.at)) return true;
        } else if (g != 0) {
            const uint64_t d = b.at >= a.at ? (b.at - a.at) % g : (g - (a.at - b.at) % g) % g;
            if (Wide(d) >= ea && Wide(d) + eb <= Wide(g)) return true;
        }
    }
    return false;
}

// The same rows in the same places (in place, row by row).
inline bool same_rows(const View &a, const View &b) {
    return a.at == b.at && a.token == b.token && a.head == b.head && a.row == b.row;
}

}  // namespace kvd
