// overlap.hpp -- whether two buffers of rows share a byte (host code).
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <utility>

namespace archead {

// rows of `width` bytes, one every `stride` >= width; nothing where at is null
struct Span {
    const void *at;
    int64_t rows, width, stride;
};
inline Span vector_span(const void *at, int64_t bytes) { return {at, 1, bytes, bytes}; }
inline Span matrix_span(const void *at, int64_t rows, int64_t cols, int64_t ld, int64_t element)
{
    return {at, rows, cols * element, ld * element};
}

// Exact: rows between the other's rows (columns of one wider matrix) are apart.  Constant
// time but for two matrices that lie within each other with different strides: then a
// step for each row of the one with fewer.
inline bool overlap(Span a, Span b)
{
    typedef __int128 Wide; // rows times strides pass 64 bits
    if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1)
        return false;
    if ((uintptr_t)b.at < (uintptr_t)a.at)
        std::swap(a, b);
    const Wide gap = (Wide)(uintptr_t)b.at - (Wide)(uintptr_t)a.at; // >= 0
    if (gap >= (Wide)(a.rows - 1) * a.stride + a.width)
        return false;
    const int64_t stride = b.rows > 1 ? b.stride : a.rows > 1 ? a.stride : a.width; // a single row has any
    if (a.rows == 1 || a.stride == stride) {
        if (a.rows == 1)
            return true; // b begins inside a's only row
        const Wide into = gap % stride; // b's first row begins at a's row gap / stride or behind it
        return into < a.width || into + b.width > stride;
    }
    const bool fewer = a.rows <= b.rows;
    const Span &one = fewer ? a : b, &other = fewer ? b : a;
    const Wide from = fewer ? -gap : gap; // of one's first row from other's
    for (int64_t i = 0; i < one.rows; ++i) {
        const Wide first = from + (Wide)i * one.stride, last = first + one.width - 1;
        if (last < 0)
            continue;
        const Wide row = std::min(last / other.stride, (Wide)(other.rows - 1)); // the last that begins by then
        if (row * other.stride + other.width > first)
            return true;
    }
    return false;
}

// any of these with any of those
inline bool overlap(std::initializer_list<Span> these, std::initializer_list<Span> those)
{
    for (const Span &a : these)
        for (const Span &b : those)
            if (overlap(a, b))
                return true;
    return false;
}
// two of these
inline bool overlap(std::initializer_list<Span> these)
{
    for (const Span *a = these.begin(); a != these.end(); ++a)
        for (const Span *b = a + 1; b != these.end(); ++b)
            if (overlap(*a, *b))
                return true;
    return false;
}
// a result that may be this input itself, with its stride
inline bool overlap_but_itself(const Span &result, const Span &input)
{
    return !(result.at == input.at && (result.stride == input.stride || result.rows <= 1)) && overlap(result, input);
}

} // namespace archead
