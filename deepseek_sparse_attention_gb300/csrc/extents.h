// extents.h -- whether tensors of rows share memory: the host's check of outputs
// against the other tensors of a call.
#pragma once

#include <stdint.h>

namespace dsa {

using wide = __int128;                                   // strides of any caller's, times counts

// n intervals of `width` bytes, `stride` >= width apart.
struct Rows {
    wide at, n, stride, width;
    wide end() const { return at + (n - 1) * stride + width; }
};
inline Rows make_rows(const void* p, wide n, wide stride, wide width) {
    // overlapping intervals: all between the first and the last
    if (n > 1 && stride < width) { width += (n - 1) * stride; n = 1; }
    return Rows{(wide)reinterpret_cast<uintptr_t>(p), n, n > 1 ? stride : width, width};
}

inline wide floor_div(wide a, wide b) { return a / b - (a % b < 0 ? 1 : 0); }   // b > 0

// The least x >= 0 with l <= a x mod m <= r, or -1 (0 < l <= r < m, 0 <= a < m).  Where no
// multiple of a lies in [l, r] itself, a x = m y + [l, r] for the least y with m y mod a in
// [-r mod a, -l mod a]: Euclid's steps.
inline wide first_hit(wide a, wide m, wide l, wide r) {
    if (a == 0) return -1;
    const wide x = (l + a - 1) / a;
    if (a * x <= r) return x;
    const wide y = first_hit(m % a, a, a - r % a, a - l % a);
    return y < 0 ? -1 : (l + m * y + a - 1) / a;
}

// Whether an interval of a and one of b have a byte in common.
inline bool rows_meet(const Rows& a, const Rows& b) {
    if (a.end() <= b.at || b.end() <= a.at) return false;
    const wide most = (wide)1 << 62;                     // more than memory has
    if (a.end() - a.at > most || b.end() - b.at > most) return true;
    // a's intervals between b's first and last byte
    wide i0 = floor_div(b.at - a.at - a.width, a.stride) + 1, i1 = floor_div(b.end() - 1 - a.at, a.stride);
    if (i0 < 0) i0 = 0;
    if (i1 > a.n - 1) i1 = a.n - 1;
    if (i0 > i1) return false;
    // i meets one of b's where (a.at + i a.stride - b.at + a.width - 1) mod b.stride < either width's sum less 1
    const wide hit = a.width + b.width - 1;
    const wide c = (a.at + i0 * a.stride - b.at + a.width - 1) % b.stride;
    if (c < hit) return true;
    const wide x = first_hit(a.stride % b.stride, b.stride, b.stride - c, b.stride - c + hit - 1);
    return x >= 0 && i0 + x <= i1;
}

// The heads of tokens: intervals with two strides, the larger outermost.
struct Heads {
    wide at, outer, n_outer, inner, n_inner, width;
    wide span() const { return (n_inner - 1) * inner + width; }      // of the inner ones
    Rows rows() const {
        Rows r = make_rows(nullptr, n_outer, outer, span());
        r.at = at;
        return r;
    }
};
inline Heads make_heads(const void* p, wide tok, wide n_tok, wide head, wide heads, wide width) {
    const wide at = (wide)reinterpret_cast<uintptr_t>(p);
    if (n_tok == 1) tok = 0;
    if (heads == 1) head = 0;
    return tok >= head ? Heads{at, tok, n_tok, head, heads, width} : Heads{at, head, heads, tok, n_tok, width};
}

// Whether heads of a and b (whose own do not overlap) have a byte in common.  Exact where both have the same
// strides or each outer stride's whole span is apart; else spans that meet are taken to.
inline bool heads_meet(const Heads& a, const Heads& b) {
    if (!rows_meet(a.rows(), b.rows())) return false;
    if (a.outer != b.outer || a.inner != b.inner || a.n_outer != b.n_outer || a.n_inner != b.n_inner) return true;
    if ((a.n_outer > 1 && a.span() > a.outer) || (a.n_inner > 1 && a.width > a.inner)) return true;
    // a.at - b.at + k outer + j inner within a width of 0, for |k| < n_outer and |j| < n_inner
    for (int e = 0; e < 2; ++e) {
        const wide k = a.n_outer > 1 ? floor_div(b.at - a.at, a.outer) + e : 0;
        if (k <= -a.n_outer || k >= a.n_outer) continue;
        const wide rest = a.at - b.at + k * a.outer;
        for (int f = 0; f < 2; ++f) {
            const wide j = a.n_inner > 1 ? floor_div(-rest, a.inner) + f : 0;
            const wide d = rest + j * a.inner;
            if (j > -a.n_inner && j < a.n_inner && d > -a.width && d < a.width) return true;
        }
    }
    return false;
}

}  // namespace dsa
