// Whether two sets of rows share a byte (host only).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace patchk {

// `count` rows of `width` bytes, `stride` >= `width` bytes apart, from `begin` up
// to `end`.  Null, or no rows: nothing (begin = end).
struct ByteRows {
    int64_t count = 0, stride = 0, width = 0;
    uintptr_t begin = 0, end = 0;
    ByteRows() = default;
    ByteRows(const void *at, int64_t count, int64_t stride, int64_t width)
        : count(count), stride(stride), width(width), begin(reinterpret_cast<uintptr_t>(at)), end(begin) {
        if (!at || count < 1 || width < 1) return;
        // (128 bits: a stride may be any 64-bit number)
        const __int128 last = static_cast<__int128>(count - 1) * stride + width + begin;
        end = last > static_cast<__int128>(UINTPTR_MAX) ? UINTPTR_MAX : static_cast<uintptr_t>(last);
    }
};

inline bool rows_meet(ByteRows a, ByteRows b);

// most pairs are apart as a whole
inline bool overlap(const ByteRows &a, const ByteRows &b) {
    return a.begin < b.end && b.begin < a.end && a.begin < a.end && b.begin < b.end && rows_meet(a, b);
}

// the rows of two sets whose ranges meet
inline bool rows_meet(ByteRows a, ByteRows b) {
    using wide = __int128;
    if (a.count > b.count) std::swap(a, b);
    const wide a0 = a.begin, b0 = b.begin;
    auto floor_div = [](wide n, wide d) { return n / d - (n % d < 0 ? 1 : 0); };  // d > 0
    if (a.count == 1) {
        // the first row of b that ends behind a's start
        const wide j = std::max<wide>(0, floor_div(a0 - b0 - b.width, b.stride) + 1);
        return j < b.count && b0 + j * b.stride < a0 + a.width;
    }
    if (a.stride == b.stride) {
        // rows i of a and j of b are (b0 - a0) + (j - i) * stride apart: the
        // least j - i that ends behind a's row
        const wide k = std::max<wide>(-(a.count - 1), floor_div(a0 - b0 - b.width, b.stride) + 1);
        return k < b.count && b0 - a0 + k * b.stride < a.width;
    }
    for (int64_t i = 0; i < a.count; ++i) {
        const wide r = a0 + static_cast<wide>(i) * a.stride;
        const wide j = std::max<wide>(0, floor_div(r - b0 - b.width, b.stride) + 1);
        if (j < b.count && b0 + j * b.stride < r + a.width) return true;
    }
    return false;
}

}  // namespace patchk
