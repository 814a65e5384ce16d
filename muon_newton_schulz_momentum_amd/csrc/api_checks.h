// Argument checks shared by the entry points of the expert layers (host only).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "plan_internal.h"

namespace muon {
namespace checks {

constexpr int64_t MAX_I32 = 0x7fffffff;

inline muon_status fail(muon_status s, const char* who, const char* what) {
    return set_error(s, std::string(who) + ": " + what);
}

inline muon_status launched(hipError_t e, const char* who) {
    return e == hipSuccess ? MUON_OK : set_error(MUON_ERR_HIP, std::string(who) + ": " + hipGetErrorString(e));
}

inline bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// The bytes of a buffer from the first that a call may touch to the last.  Rows and matrices lie a stride apart and the last
// of them ends with its own columns: what follows belongs to someone else.
struct Extent {
    const void* p;
    double bytes;                         // (sizes are products that may pass 64 bits)
    uint64_t step = 0, width = 0;         // rows of `width` bytes, `step` bytes apart; 0: no gaps
};
inline Extent extent(const void* p, double bytes) { return {p, bytes}; }
// `count` matrices of `rows` x `cols` elements
inline Extent extent(const void* p, int64_t count, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t size = 1) {
    if (count < 1 || rows < 1) return {p, 0};
    Extent e{p, ((double)(count - 1) * (double)stride + (double)(rows - 1) * (double)ld + (double)cols) * (double)size};
    if (ld > cols && (count == 1 || stride % ld == 0)) {
        e.step = (uint64_t)(ld * size);
        e.width = (uint64_t)(cols * size);
    }
    return e;
}
inline bool overlap(const Extent& a, const Extent& b) {
    const double x = (double)(uintptr_t)a.p, y = (double)(uintptr_t)b.p;
    if (!(a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes)) return false;
    if (a.step == 0 || a.step != b.step) return true;
    // b's rows in the gaps between a's: two column ranges of one matrix
    const uint64_t d = ((uintptr_t)b.p % a.step + a.step - (uintptr_t)a.p % a.step) % a.step;
    return d < a.width || d + b.width > a.step;
}

// Whether an output overlaps an input or another output.
template <int N, int M>
bool collide(const Extent (&out)[N], const Extent (&in)[M]) {
    for (int i = 0; i < N; ++i) {
        for (const Extent& e : in)
            if (overlap(out[i], e)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

inline bool is_dtype(int32_t d) { return d == MUON_DTYPE_F32 || d == MUON_DTYPE_BF16; }

}  // namespace checks
}  // namespace muon
