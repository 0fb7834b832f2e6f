// Whether two sets of rows share a byte (host only).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace patchk {

// `count` rows of `width` bytes, `stride` >= `width` bytes apart.  No rows: nothing.
struct ByteRows {
    const void *at = nullptr;
    int64_t count = 0, stride = 0, width = 0;
};

inline bool overlap(ByteRows a, ByteRows b) {
    using wide = __int128;  // a stride may be any 64-bit number
    if (!a.at || !b.at || a.count < 1 || b.count < 1 || a.width < 1 || b.width < 1) return false;
    if (a.count > b.count) std::swap(a, b);
    const wide a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
    auto end = [](wide at, const ByteRows &r) { return at + static_cast<wide>(r.count - 1) * r.stride + r.width; };
    if (end(a0, a) <= b0 || end(b0, b) <= a0) return false;
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
