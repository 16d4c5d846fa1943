// Do two strided arrays share memory?  Host checks of the entry points.
#pragma once

#include <cstdint>

namespace bspo {

// rows pieces of `len` bytes, `stride` apart.
struct Rows {
    const void* at;
    int64_t rows, len, stride;
};

// True unless the two are apart: no byte of one lies between the first and
// the last of the other, or they step by the same stride through different
// bytes of it (two slices of one tensor's rows).
inline bool meet(const Rows& a, const Rows& b)
{
    if (a.rows <= 0 || b.rows <= 0 || a.len <= 0 || b.len <= 0) return false;
    const int64_t end_a = (a.rows - 1) * (a.rows > 1 ? a.stride : 0) + a.len;
    const int64_t end_b = (b.rows - 1) * (b.rows > 1 ? b.stride : 0) + b.len;
    const int64_t off = (int64_t)((uintptr_t)a.at - (uintptr_t)b.at);  // of a in b
    if (off >= end_b || -off >= end_a) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
    const int64_t s = a.rows > 1 ? a.stride : b.stride;
    if ((a.rows < 2 && b.rows < 2) || a.len > s || b.len > s) return true;
    const int64_t r = ((off % s) + s) % s;  // where a piece of a begins in a step of b
    return r < b.len || r + a.len > s;
}

}  // namespace bspo
