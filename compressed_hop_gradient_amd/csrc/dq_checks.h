// dq_checks.h -- argument checks that the stateless entry points share (host code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "dq.h"

namespace dq {
namespace {

constexpr size_t kAlign = 256;

bool is_kind(int32_t kind) { return kind == DQ_BF16 || kind == DQ_F32; }
uintptr_t elem_bytes(int32_t kind) { return kind == DQ_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

dq_status hip_status(hipError_t e) { return e == hipSuccess ? DQ_OK : DQ_EHIP; }

// The bytes of an operand: windows of one width at one stride (rows that touch
// or overlap are one window).
struct Span {
    uint64_t lo, hi;                     // first byte, and past the last; lo = hi: nothing
    uint64_t stride, width;              // stride 0: one window
    bool out;
};
Span span(const void *p, int64_t rows, int64_t stride, int64_t cols, int64_t es, bool out) {
    const uint64_t lo = reinterpret_cast<uintptr_t>(p);
    if (!p || rows <= 0 || cols <= 0) return Span{lo, lo, 0, 0, out};
    typedef unsigned __int128 wide;
    const wide hi = lo + ((wide)(rows - 1) * (uint64_t)stride + (uint64_t)cols) * (uint64_t)es;
    const bool windows = rows > 1 && stride > cols;
    return Span{lo, hi > UINT64_MAX ? UINT64_MAX : (uint64_t)hi, windows ? (uint64_t)stride * es : 0,
                (uint64_t)cols * es, out};
}
// An input of `many` such matrices, `apart` elements apart: from the first element to the last.
Span span_all(const void *p, int64_t many, int64_t apart, int64_t rows, int64_t stride, int64_t cols, int64_t es) {
    const uint64_t lo = reinterpret_cast<uintptr_t>(p);
    typedef unsigned __int128 wide;
    const wide hi = lo + ((wide)(many - 1) * (uint64_t)apart + (wide)(rows - 1) * (uint64_t)stride + (uint64_t)cols) *
                             (uint64_t)es;
    return Span{lo, hi > UINT64_MAX ? UINT64_MAX : (uint64_t)hi, 0, 0, false};
}
Span bytes(const void *p, size_t n, bool out) { return span(p, 1, 0, (int64_t)n, 1, out); }

// Whether two of them meet.  Windows of equal stride may interleave (two halves of
// one wide tensor); at two strides it goes by the first and the last byte.
bool meet(const Span &a, const Span &b) {
    if (a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo) return false;
    const uint64_t s = a.stride ? a.stride : b.stride;
    if (!s || (a.stride && b.stride && a.stride != b.stride)) return true;
    const uint64_t d = b.lo >= a.lo ? (b.lo - a.lo) % s : (s - (a.lo - b.lo) % s) % s;
    // a window that is the only one of its operand is as wide as all of it
    const uint64_t wa = a.stride ? a.width : a.hi - a.lo, wb = b.stride ? b.width : b.hi - b.lo;
    return d < wa || wb > s - d;
}

// The operands of a call.  clash(): an output among them meets an input or another
// output.  In order of their first bytes, almost all are told apart by the last
// byte so far; only where that fails (windows that interleave) all pairs are tried.
class Spans {
    static constexpr size_t kFew = 64;
    Span few[kFew];
    std::unique_ptr<Span[]> many;
    Span *at = few;
    size_t n = 0;

public:
    // room for `most`; false if there is none
    bool reserve(size_t most) {
        if (most <= kFew) return true;
        many.reset(new (std::nothrow) Span[most]);
        at = many.get();
        return at != nullptr;
    }
    void add(const Span &s) {
        if (s.lo != s.hi) at[n++] = s;
    }
    bool clash() {
        std::sort(at, at + n, [](const Span &a, const Span &b) { return a.lo < b.lo; });
        uint64_t any = 0, out = 0;
        size_t i = 0;
        for (; i < n && at[i].lo >= (at[i].out ? any : out); i++) {
            any = std::max(any, at[i].hi);
            if (at[i].out) out = std::max(out, at[i].hi);
        }
        if (i == n) return false;
        for (; i < n; i++)
            for (size_t j = 0; j < i; j++)
                if ((at[i].out || at[j].out) && meet(at[i], at[j])) return true;
        return false;
    }
};

}  // namespace
}  // namespace dq
