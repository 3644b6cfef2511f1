// ssm_check.hpp -- host-side argument checks shared by the C-ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "ssm.h"

namespace ssm {
namespace check {

// True when p is not a multiple of `align` bytes (NULL is never misaligned).
inline bool misaligned(const void *p, uintptr_t align)
{
    return p && (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0;
}

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Span span(const void *p, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}

inline bool overlaps(const void *p, size_t pb, const void *q, size_t qb)
{
    if (!p || !q || pb == 0 || qb == 0) return false;
    const Span a = span(p, pb), b = span(q, qb);
    return a.lo < b.hi && b.lo < a.hi;
}

// A strided tensor in bytes: runs of `run` bytes (one step), `step` apart,
// batch entries `batch` apart, `bytes` from the first to the last.  Of a
// time-major tensor `step` and `batch` are the other way round.
struct Steps {
    const void *p;
    size_t bytes, run;
    long long step, batch;
};

// With one step a batch entry the entries are the steps: the step stride of
// such a tensor says nothing.
inline Steps one_step(const Steps &a, int seqlen)
{
    return seqlen == 1 ? Steps{a.p, a.bytes, a.run, a.batch, 0} : a;
}

// overlaps(), except that two tensors with the same strides whose runs lie
// beside each other in every step (slices of one buffer) do not overlap.
inline bool overlaps(const Steps &a, const Steps &b)
{
    if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.step != b.step || a.batch != b.batch || a.step <= 0 || a.batch % a.step) return true;
    const size_t step = size_t(a.step);
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const size_t d = pb >= pa ? (pb - pa) % step : (step - (pa - pb) % step) % step;
    return d < a.run || d + b.run > step;
}

// The value of an enum argument as the int a C caller passed: its bits are
// read without loading the argument as the enum type, so a value outside the
// enumeration (an error the validation reports) is not undefined behaviour.
template <typename E>
inline int enum_bits(const E &e)
{
    static_assert(sizeof(E) == sizeof(int), "C enums are int-sized");
    int v = 0;
    memcpy(&v, &e, sizeof v);
    return v;
}

inline bool valid_dtype(int t) { return t == SSM_F32 || t == SSM_BF16; }
inline size_t dsize(int t) { return t == SSM_BF16 ? 2 : 4; }

// Product of positive ints as size_t, or 0 on overflow past 2^62.
inline size_t mul3(long long a, long long b, long long c)
{
    const unsigned __int128 r = (unsigned __int128)a * (unsigned __int128)b * (unsigned __int128)c;
    if (r > ((unsigned __int128)1 << 62)) return 0;
    return size_t(r);
}

}  // namespace check
}  // namespace ssm
