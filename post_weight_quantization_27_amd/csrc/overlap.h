// Whether the memory of two arguments of a call overlaps, from their sizes and strides: host code, no
// HIP, so that it can be compiled and checked alone.
#pragma once

#include <stdint.h>

namespace pwq {

// `rows` pieces of `len` bytes, `pitch` bytes apart (pitch >= len where there are several)
struct Rows {
    uint64_t p, rows, len, pitch;
};

inline Rows rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    return p ? Rows{(uint64_t)(uintptr_t)p, (uint64_t)rows, (uint64_t)(cols * size), (uint64_t)(ld * size)} : Rows{0, 0, 0, 0};
}
inline Rows bytes_of(const void* p, int64_t n) { return rows_of(p, 1, n, n, 1); }

// True where a row of a and a row of b share a byte.  Matrices whose rows lie between each other's
// (columns of one wider matrix, records of several arrays) do not.
inline bool overlap(const Rows& a, const Rows& b) {
    if (a.rows == 0 || a.len == 0 || b.rows == 0 || b.len == 0) return false;
    if (a.p + (a.rows - 1) * a.pitch + a.len <= b.p || b.p + (b.rows - 1) * b.pitch + b.len <= a.p) return false;
    if (a.rows > 1 && b.rows > 1 && a.pitch == b.pitch) {
        // row i of a and row i + k of b: the first k whose row of b ends behind the start of a's row
        const int64_t pitch = (int64_t)a.pitch, d = (int64_t)(b.p - a.p);
        const int64_t lo = -(int64_t)b.len - d;               // k pitch > lo
        int64_t k = (lo >= 0 ? lo / pitch : -((pitch - 1 - lo) / pitch)) + 1;
        if (k < 1 - (int64_t)a.rows) k = 1 - (int64_t)a.rows;
        return k < (int64_t)b.rows && d + k * pitch < (int64_t)a.len;
    }
    // other strides: through both in order, past all of one's rows that end before the other's at once
    uint64_t i = 0, j = 0;
    while (i < a.rows && j < b.rows) {
        const uint64_t x = a.p + i * a.pitch, y = b.p + j * b.pitch;
        if (x + a.len <= y) {
            if (a.rows == 1) return false;
            i += (y - x - a.len) / a.pitch + 1;
        } else if (y + b.len <= x) {
            if (b.rows == 1) return false;
            j += (x - y - b.len) / b.pitch + 1;
        } else {
            return true;
        }
    }
    return false;
}

// True where an output overlaps an input or another output
template <int NO, int NI>
inline bool outputs_overlap(const Rows (&out)[NO], const Rows (&in)[NI]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int i = o + 1; i < NO; ++i)
            if (overlap(out[o], out[i])) return true;
    }
    return false;
}

}  // namespace pwq
