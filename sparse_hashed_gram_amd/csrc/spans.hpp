// Host checks of where a call's buffers lie.
#pragma once

#include <stdint.h>

namespace spans {

// `rows` rows of `len` bytes, `ld` bytes apart (one row: a plain range).
struct Span {
    const void *p;
    uint64_t len;
    uint64_t rows = 1;
    uint64_t ld = 0;

    bool empty() const { return !p || len == 0 || rows == 0; }
    uint64_t extent() const { return len + (rows - 1) * ld; }
};

// True if the two share a byte, or (rows of different distances, interleaved)
// might.
inline bool meet(const Span &a, const Span &b)
{
    if (a.empty() || b.empty())
        return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (x + a.extent() <= y || y + b.extent() <= x)
        return false;
    if (a.rows > 1 && b.rows > 1 && a.ld == b.ld) {   // columns of one array
        const uint64_t d = (y > x ? y - x : x - y) % a.ld, near = y > x ? a.len : b.len, far = y > x ? b.len : a.len;
        return d < near || a.ld - d < far;
    }
    return true;
}

}   // namespace spans
