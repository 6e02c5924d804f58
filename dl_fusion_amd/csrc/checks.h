// Argument checks shared by the C-ABI translation units of the decode operators.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace dlf {

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// One operand's bytes: [p, p + n); a null pointer or no bytes overlaps nothing.
struct Span {
    const void* p;
    size_t n;
};

inline bool overlaps(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Does an output overlap an input or another output?
inline bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (overlaps(*o, i)) return true;
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (overlaps(*o, *q)) return true;
    }
    return false;
}

// Bytes from the first to past the last element of `rows` rows of `width` elements, `stride` apart.
inline size_t rows_bytes(int64_t rows, int64_t stride, int64_t width, size_t elem) {
    return rows > 0 ? static_cast<size_t>((rows - 1) * stride + width) * elem : 0;
}

}  // namespace dlf
