// What the entry points' argument checks share.
#pragma once
#include <cstddef>
#include <cstdint>

#include "mhc.h"

namespace mhc {

inline size_t size_of(mhc_dtype d) { return d == MHC_F32 ? 4 : 2; }
inline bool dtype_ok(mhc_dtype d) { return d == MHC_F32 || d == MHC_BF16 || d == MHC_F16; }
inline bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A byte range an entry point reads or writes (n == 0: none).
struct Span {
    const void *p;
    size_t n;
};
inline bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}
// Any output over an input (but `same`, an output that may be that input) or another output.
inline bool aliased(const Span *outs, int no, const Span *ins, int ni, int same_out, int same_in) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j) {
            if (i == same_out && j == same_in && outs[i].p == ins[j].p && outs[i].n == ins[j].n) continue;
            if (overlap(outs[i], ins[j])) return true;
        }
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

// Rows `stride` elements apart: the range that they lie in. False when it
// would not fit 63 bits.
inline bool rows_span(const void *p, int64_t stride, int64_t T, int H, size_t elem, Span *s) {
    const __int128 n = (static_cast<__int128>(T - 1) * stride + H) * static_cast<__int128>(elem);
    if (n > (static_cast<__int128>(1) << 62)) return false;
    *s = {p, static_cast<size_t>(n)};
    return true;
}
inline bool size_fits(int64_t T, int H) { return T <= (int64_t(1) << 61) / H / 4; }

}  // namespace mhc
