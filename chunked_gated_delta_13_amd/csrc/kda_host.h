// Argument checks shared by the host sources of libkda.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

inline bool mul_ok(long long a, long long b, long long* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > (1LL << 62) / a) return false;
    *out = a * b;
    return true;
}

// The same for the entry points beside KDA, whose inputs may be strided rows.
namespace host {

using kda::Range;
using kda::aligned;
using kda::mul_ok;
using kda::overlap;
using kda::range_of;

constexpr long long kMaxGridYZ = 65535;   // blocks of a launch along y or z
// Workgroups of a launch along x: up to 512 threads each, and fewer than 2^32 threads in all.
constexpr long long kMaxUnits = 1LL << 22;

inline size_t elem_size(kda_dtype_t dt) { return dt == KDA_BF16 ? 2 : 4; }

// The bytes spanned by `rows` rows of `width` elements whose starts lie `stride` elements apart.
inline Range rows_range(const void* p, long long rows, long long width, long long stride, size_t esz) {
    if (rows <= 0 || width <= 0 || !p) return range_of(p, 0);
    return range_of(p, ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * esz);
}

// rows * stride elements stay far inside 63 bits, and a stride is at least a row's width.
inline bool stride_ok(long long rows, long long width, long long stride) {
    long long n = 0;
    if (rows <= 1) return stride >= 0;
    return stride >= width && mul_ok(rows, stride, &n) && n < (1LL << 58);
}

// A strided row input that is read in 16-byte pieces.
inline bool wide_rows_ok(const void* ptr, long long rows, long long width, long long stride, size_t esz) {
    if (!stride_ok(rows, width, stride)) return false;
    return aligned(ptr, 16) && (rows <= 1 || ((size_t)stride * esz) % 16 == 0);
}

// The kernels take exponentials of base 2: scale log2(e) has to be a finite number too.
inline bool scale_ok(float scale) { return scale > 0.0f && scale <= 2.3e38f; }

// Compute units of the current device (256 where the runtime does not say).
int cu_count();

}  // namespace host

}  // namespace kda
