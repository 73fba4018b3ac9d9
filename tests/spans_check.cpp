// Pairs of views from standard input (address, rows, row stride, heads, head stride, width each, in bytes): for each 1
// where they share a byte by spans.h, else 0.
#include <cstdint>
#include <iostream>

#include "spans.h"

int main()
{
    auto read = [](h3fp4::Span& s) {
        unsigned long long p;
        if (!(std::cin >> p >> s.rows >> s.row >> s.heads >> s.head >> s.width)) return false;
        s.p = reinterpret_cast<const void*>((uintptr_t)p);
        return true;
    };
    h3fp4::Span a, b;
    while (read(a) && read(b)) std::cout << (h3fp4::overlap(a, b) ? 1 : 0) << "\n";
}
