// ssm_stride.hpp -- host-side checks of tensors of batch x steps x heads rows
// with free strides, shared by the C-ABI sources of the multi-head recurrences.
#pragma once

#include "delta_launch.hpp"
#include "ssm_check.hpp"

namespace ssm {
namespace check {

// Strides with defaults filled in and the span in elements of a tensor of
// batch x steps x heads x row elements: false when a stride is negative, two
// elements share a place, or the span reaches 2^56.
inline bool delta_stride(long long given_t, long long given_h, long long given_b, int batch, int steps, int heads,
                         int row, ssm::DeltaStride &s, size_t &sp)
{
    if (given_t < 0 || given_h < 0 || given_b < 0) return false;
    constexpr __int128 most = (__int128)1 << 56;
    const __int128 dh = given_h ? given_h : row;
    const __int128 dt = given_t ? (__int128)given_t : heads * dh;
    const __int128 db = given_b ? (__int128)given_b : steps * dt;
    if (dh >= most || dt >= most || db >= most) return false;
    struct Dim {
        __int128 stride;
        int n;
    } d[3] = {{dh, heads}, {dt, steps}, {db, batch}};
    for (int i = 0; i < 2; ++i)  // smallest stride first; dimensions of one entry do not count
        for (int j = 0; j < 2 - i; ++j)
            if (d[j].n == 1 ? d[j + 1].n != 1 : (d[j + 1].n != 1 && d[j].stride > d[j + 1].stride)) {
                const Dim t = d[j];
                d[j] = d[j + 1];
                d[j + 1] = t;
            }
    __int128 span = row;  // of everything inside the dimension
    for (const Dim &x : d) {
        if (x.n == 1) continue;
        if (x.stride < span) return false;
        span += x.stride * (x.n - 1);
        if (span >= most) return false;
    }
    // the kernels bound a buffer of rows by rows x step: one step's is a row, whatever the
    // stride that leads to no second one
    s = {steps == 1 ? row : (long long)dt, (long long)dh, (long long)db};
    sp = size_t(span);
    return true;
}

// A tensor for the overlap check, element strides given: runs of one step's
// heads, and the strides from run to run, the smaller first (the batch's in
// time-major tensors; one that leads nowhere is 0).  Where the heads do not lie
// inside a run, the range alone counts.
inline Steps steps_of(const void *p, size_t span, size_t es, const ssm::DeltaStride &s, int heads, int row, int seqlen,
                      int batch)
{
    const long long run = (heads - 1) * s.h + row, t = seqlen > 1 ? s.t : 0, b = batch > 1 ? s.b : 0;
    const bool time_major = !t || (b && b < t);
    const long long inner = time_major ? b : t, outer = time_major ? t : b;
    if (run > inner) return {p, span * es, span * es, 0, 0};
    return {p, span * es, size_t(run) * es, (long long)(inner * es), (long long)(outer * es)};
}
inline Steps range_of(const void *p, size_t bytes) { return {p, bytes, bytes, 0, 0}; }

}  // namespace check
}  // namespace ssm
