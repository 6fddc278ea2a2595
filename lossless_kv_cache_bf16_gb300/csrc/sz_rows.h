// sz_rows.h -- whether two sets of rows share memory.  Host code, of the C ABI
// and of the Python binding.
#pragma once

#include <algorithm>
#include <cstdint>

namespace sz {

// bf16 rows [tokens][heads] by their strides in elements.
struct RowSet {
    const void* base;
    int64_t token_stride, head_stride;
    uint64_t tokens, heads;
};

// Whether a and b are the same rows at the same addresses.
inline bool same_rows(const RowSet& a, const RowSet& b) {
    return a.base == b.base && a.tokens == b.tokens && a.heads == b.heads &&
           (a.tokens <= 1 || a.token_stride == b.token_stride) && (a.heads <= 1 || a.head_stride == b.head_stride);
}

// Whether a row of a and a row of b, of `dim` contiguous channels each, share
// memory.  Exact where the sets have their strides in common (views of one
// buffer); sets of other strides count as overlapping where their address
// ranges do.
inline bool rows_overlap(const RowSet& a, const RowSet& b, uint64_t dim) {
    using Int = __int128;
    if (a.tokens == 0 || a.heads == 0 || b.tokens == 0 || b.heads == 0 || dim == 0) return false;
    const Int width = 2 * (Int)dim;
    struct Set {
        Int first;            // lowest address
        Int count[2], step[2];  // tokens, heads; steps in bytes, not negative
        Int reach() const { return (count[0] - 1) * step[0] + (count[1] - 1) * step[1]; }
    };
    auto set_of = [](const RowSet& r) {
        Set s{(Int)reinterpret_cast<uintptr_t>(r.base), {(Int)r.tokens, (Int)r.heads}, {2 * (Int)r.token_stride, 2 * (Int)r.head_stride}};
        for (int k = 0; k < 2; k++) {
            if (s.count[k] == 1) s.step[k] = 0;
            if (s.step[k] < 0) {
                s.first += (s.count[k] - 1) * s.step[k];
                s.step[k] = -s.step[k];
            }
        }
        return s;
    };
    const Set x = set_of(a), y = set_of(b);
    if (x.first + x.reach() + width <= y.first || y.first + y.reach() + width <= x.first) return false;
    // A dimension of one entry has the other set's step.
    Int step[2];
    for (int k = 0; k < 2; k++) {
        if (x.count[k] > 1 && y.count[k] > 1 && x.step[k] != y.step[k]) return true;
        step[k] = std::max(x.step[k], y.step[k]);
    }
    // Rows start at multiples of the steps from the first: the starts' distance
    // is gap - i * step[0] - j * step[1], i from 1 - y.count[0] to x.count[0] - 1
    // and j likewise.
    const Int gap = y.first - x.first;
    const int wide = step[0] >= step[1] ? 0 : 1, narrow = 1 - wide;
    if (step[wide] > 0) {
        // Sets of one packed buffer: each within its part of every wide step.
        Int off = gap % step[wide];
        if (off < 0) off += step[wide];
        const Int x_span = (x.count[narrow] - 1) * step[narrow] + width, y_span = (y.count[narrow] - 1) * step[narrow] + width;
        if (off >= x_span && off + y_span <= step[wide]) return false;
    }
    // Over the dimension of fewer entries; the other's nearest one is known.
    const int loop = x.count[0] + y.count[0] <= x.count[1] + y.count[1] ? 0 : 1, other = 1 - loop;
    for (Int j = 1 - y.count[loop]; j < x.count[loop]; j++) {
        const Int d = gap - j * step[loop];
        const Int below = step[other] > 0 ? d / step[other] - (d % step[other] < 0 ? 1 : 0) : 0;
        for (Int i = below; i <= below + 1; i++) {
            const Int in = std::min(std::max(i, 1 - y.count[other]), x.count[other] - 1), left = d - in * step[other];
            if (left < width && -left < width) return true;
        }
    }
    return false;
}

}  // namespace sz
