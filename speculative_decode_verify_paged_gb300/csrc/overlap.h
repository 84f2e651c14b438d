// Do two buffers of a call share a byte?  Host only, exact for rows at any
// strides: views of one fused projection, or K and V pages in one allocation,
// lie between each other without touching.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace spec_attn {

// n rows of `width` bytes, `step` apart (at least `width` where n > 1).
struct ByteRows {
    const void* at;
    uint64_t width, step, n;
};

inline ByteRows bytes_at(const void* at, uint64_t n) { return {at, n, n, 1}; }

// sum over i < n of floor((a i + b) / m): Euclid's algorithm on the line's slope (the count of the lattice points below it).
inline unsigned __int128 sum_of_floors(uint64_t n, uint64_t m, uint64_t a, unsigned __int128 b) {
    unsigned __int128 total = 0;
    while (n > 0) {
        total += static_cast<unsigned __int128>(n) * (n - 1) / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const unsigned __int128 top = static_cast<unsigned __int128>(a) * n + b;
        if (top < m) break;
        n = static_cast<uint64_t>(top / m);
        b = top % m;
        const uint64_t t = m;
        m = a;
        a = t;
    }
    return total;
}

inline bool overlap(const ByteRows& a, const ByteRows& b) {
    if (!a.n || !b.n || !a.width || !b.width || !a.at || !b.at) return false;
    const uint64_t a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
    const uint64_t sa = a.n > 1 ? a.step : a.width, sb = b.n > 1 ? b.step : b.width;
    const uint64_t a1 = a0 + (a.n - 1) * sa + a.width, b1 = b0 + (b.n - 1) * sb + b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    // a's rows i0 .. i1 - 1 reach into [b0, b1).  Each of them meets a row of b if and only if it meets one of b's rows
    // continued without end: a row that reaches past an end of b holds the byte at that end, which is b's own.
    const uint64_t i0 = a0 + a.width > b0 ? 0 : (b0 - a0 - a.width) / sa + 1;
    const uint64_t i1 = b1 <= a0 ? 0 : (b1 - a0 - 1) / sa + 1 < a.n ? (b1 - a0 - 1) / sa + 1 : a.n;
    if (i0 >= i1) return false;
    // Row i at x_i meets the rows j with x_i - width_b < b0 + j sb < x_i + width_a.  Their number is
    // floor((x_i + width_a - 1 - b0) / sb) - floor((x_i - width_b - b0) / sb), summed over i; both shifted by a
    // few rows of b, since x_i may lie below b0.
    const uint64_t pad = (a.width + b.width) / sb + 1;
    const unsigned __int128 first = static_cast<unsigned __int128>(pad) * sb + a0 + static_cast<unsigned __int128>(i0) * sa - b0;
    return sum_of_floors(i1 - i0, sb, sa, first + a.width - 1) != sum_of_floors(i1 - i0, sb, sa, first - b.width);
}

// Does an output meet another output or an input?  (An input that an output may be, and is, is left out by the caller:
// it meets what the output meets.)
template <size_t O, size_t I>
bool outputs_overlap(const ByteRows (&out)[O], const ByteRows (&in)[I]) {
    for (size_t i = 0; i < O; ++i) {
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
        for (size_t j = 0; j < I; ++j)
            if (overlap(out[i], in[j])) return true;
    }
    return false;
}

}  // namespace spec_attn
