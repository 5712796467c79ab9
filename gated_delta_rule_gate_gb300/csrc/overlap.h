// overlap.h -- whether two operands share memory (host side, from addresses alone).
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace gdn {

// `rows` rows of `width` bytes, `stride` (at least width) apart.
struct Span {
    const void *at;
    int64_t rows, stride, width;
};
inline Span block_of(const void *at, int64_t bytes) { return {at, 1, bytes, bytes}; }

// A row of `a`, which begins at 0, and the bytes from `begin` to `end` (above begin).
inline bool row_in(const Span &a, int64_t begin, int64_t end) {
    const int64_t i = begin < a.width ? 0 : (begin - a.width) / a.stride + 1;  // the first that ends behind `begin`
    return i < a.rows && i * a.stride < end;
}

inline bool overlap(Span a, Span b) {
    if (!a.at || !b.at || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    for (Span *s : {&a, &b})
        if (s->rows == 1 || s->stride == s->width) *s = block_of(s->at, s->rows * s->width);
    if (reinterpret_cast<uintptr_t>(b.at) < reinterpret_cast<uintptr_t>(a.at)) {
        const Span t = a;
        a = b, b = t;
    }
    // b begins d bytes behind a
    const uintptr_t far = reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at);
    const int64_t extent = (a.rows - 1) * a.stride + a.width;
    if (far >= (uintptr_t)extent) return false;
    const int64_t d = (int64_t)far;
    if (a.rows == 1) return true;  // b's first byte is in it
    if (b.rows == 1) return row_in(a, d, d + b.width);
    if (a.stride == b.stride) {
        // columns side by side, or not: b's rows begin in row q of a at r, and go on into the next
        const int64_t q = d / a.stride, r = d - q * a.stride;
        return r < a.width || (r + b.width > a.stride && q + 1 < a.rows);
    }
    // rows at unequal distances among one another: one by one
    for (int64_t j = 0; j < b.rows && d + j * b.stride < extent; ++j)
        if (row_in(a, d + j * b.stride, d + j * b.stride + b.width)) return true;
    return false;
}

}  // namespace gdn
