// Whether two views share memory.  Plain host code, which the tests compile by themselves.
#pragma once
#include <cstdint>

namespace h3fp4 {

// Places of memory: rows of heads of `width` bytes each; strides in bytes, not below zero.
struct Span {
    const void* p;
    int64_t rows, row, heads, head;
    uint64_t width;
};

// Whether some j + a i with 0 <= i < n lies in [lo, hi).
inline bool any_between(int64_t a, int64_t n, int64_t j, int64_t lo, int64_t hi)
{
    if (a == 0) return j >= lo && j < hi;
    const int64_t i = j >= lo ? 0 : (lo - j + a - 1) / a;
    return i < n && j + a * i < hi;
}

// Whether two of them share a byte.  Views may lie between one another, as Q, K and V of one projection do: those have
// equal strides, and a loop over their heads (or rows, where there are fewer) tells.  Others whose ranges cross are compared
// head by head; where that would be more than 2^22 comparisons they count as sharing one.
inline bool overlap(Span a, Span b)
{
    if (!a.p || !b.p || a.width == 0 || b.width == 0 || a.rows <= 0 || b.rows <= 0) return false;
    for (Span* s : {&a, &b}) {   // a stride that is never taken says nothing
        if (s->rows == 1) s->row = 0;
        if (s->heads == 1) s->head = 0;
    }
    using Wide = unsigned __int128;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const Wide ea = Wide(pa) + Wide(a.rows - 1) * Wide(a.row) + Wide(a.heads - 1) * Wide(a.head) + a.width;
    const Wide eb = Wide(pb) + Wide(b.rows - 1) * Wide(b.row) + Wide(b.heads - 1) * Wide(b.head) + b.width;
    if (Wide(pa) >= eb || Wide(pb) >= ea) return false;
    if (ea > Wide(1) << 60 || eb > Wide(1) << 60) return false;   // (no such memory: below, 64 bits do)
    // a head of a at x meets one of b at y where -b.width < y - x < a.width
    const int64_t from = (int64_t)(pa - pb), wa = (int64_t)a.width, wb = (int64_t)b.width;
    if (a.row == b.row && a.head == b.head) {
        const bool by_rows = (a.rows < b.rows ? b.rows : a.rows) < (a.heads < b.heads ? b.heads : a.heads);
        const int64_t na = by_rows ? a.rows : a.heads, nb = by_rows ? b.rows : b.heads, step = by_rows ? a.row : a.head;
        const int64_t ma = by_rows ? a.heads : a.rows, mb = by_rows ? b.heads : b.rows, inner = by_rows ? a.head : a.row;
        for (int64_t d = 1 - na; d < nb; ++d)
            if (any_between(inner, ma + mb - 1, d * step - (ma - 1) * inner, from - wb + 1, from + wa)) return true;
        return false;
    }
    if (Wide(a.rows) * Wide(a.heads) * Wide(b.heads) > Wide(1) << 22) return true;
    for (int64_t r = 0; r < a.rows; ++r)
        for (int64_t h = 0; h < a.heads; ++h)
            for (int64_t k = 0; k < b.heads; ++k) {
                const int64_t x = from + r * a.row + h * a.head;
                if (any_between(b.row, b.rows, k * b.head, x - wb + 1, x + wa)) return true;
            }
    return false;
}

}  // namespace h3fp4
