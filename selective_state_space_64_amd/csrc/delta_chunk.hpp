// delta_chunk.hpp -- what the chunked delta rule's kernels agree on: the
// workspace, the number of bf16 terms, and the launch parameters.
#pragma once

#include <type_traits>

#include "delta_mfma.hpp"
#include "ssm_launch.hpp"

namespace ssm {

// Padded key size of the kernels' tiles.
inline int delta_kd(int K) { return K <= 64 ? 64 : K <= 128 ? 128 : 256; }
inline int delta_vp(int V) { return (V + 63) / 64 * 64; }

// bf16 terms of the inputs (kIn) and of what the kernels form from them
// (kSum: states, U, T, P, ...).  Two terms leave 2^-17 of a value's size,
// below what the fp32 sums of a chain of products lose by some factor 10 but
// 200 times under the rounding of a bf16 output; fp32 inputs take three, except where
// K > 128 leaves no LDS for them.
template <typename T, int KD> struct Terms {
    static constexpr int kIn = sizeof(T) == 2 ? 1 : KD > 128 ? 2 : 3;
    static constexpr int kSum = sizeof(T) == 2 ? 2 : kIn;
};

struct DeltaWs {
    float *vec;
    uint16_t *T, *P, *Tt, *Pt;
    float *S0, *U, *dS1, *dX;
};

inline DeltaWs delta_ws(void *workspace, long long recs, int K, int V, bool bwd, size_t *bytes)
{
    const size_t n = size_t(recs), state = size_t(delta_kd(K)) * delta_vp(V), step = size_t(64) * delta_vp(V);
    char *p = static_cast<char *>(workspace);
    size_t at = 0;
    auto take = [&](size_t each) {
        char *r = p ? p + at : nullptr;
        at += n * each;
        return r;
    };
    DeltaWs w{};
    const size_t tri = kTriFrags * 3 * 512 * sizeof(uint16_t);  // three terms at most
    w.vec = reinterpret_cast<float *>(take(256 * sizeof(float)));
    w.T = reinterpret_cast<uint16_t *>(take(tri));
    w.P = reinterpret_cast<uint16_t *>(take(tri));
    if (bwd) {
        w.Tt = reinterpret_cast<uint16_t *>(take(tri));
        w.Pt = reinterpret_cast<uint16_t *>(take(tri));
        w.S0 = reinterpret_cast<float *>(take(state * sizeof(float)));
        w.U = reinterpret_cast<float *>(take(step * sizeof(float)));
        w.dS1 = reinterpret_cast<float *>(take(state * sizeof(float)));
        w.dX = reinterpret_cast<float *>(take(step * sizeof(float)));
    }
    if (bytes) *bytes = at;
    return w;
}

// 16-byte accesses fit every row of a tensor with n elements a row.
inline bool delta_vec(const void *p, const DeltaStride &s, int n, int esize, const DeltaArgs &a, int heads)
{
    const long long per = 16 / esize;
    return n % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.seqlen == 1 || s.t % per == 0) &&
           (heads == 1 || s.h % per == 0) && (a.batch == 1 || s.b % per == 0);
}

// Sum of the first l + 1 log decays of a chunk, for lane l of one wave; in
// double: a step that clears the state (-110) must not cost the later steps'
// differences their low bits.
__device__ inline double decay_sums(float g)
{
    double sum = g < -110.0f ? -110.0f : g;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const double v = __shfl_up(sum, o);
        if (int(threadIdx.x & 63) >= o) sum += v;
    }
    return sum;
}

// f(T{}, TG{}, padded K) for the call's types.
template <typename F>
hipError_t delta_dispatch(bool in_bf16, bool g_bf16, int K, F &&f)
{
    const int kd = delta_kd(K);
    auto sized = [&](auto t, auto tg) {
        return kd == 64 ? f(t, tg, std::integral_constant<int, 64>{})
             : kd == 128 ? f(t, tg, std::integral_constant<int, 128>{})
                         : f(t, tg, std::integral_constant<int, 256>{});
    };
    if (in_bf16) return g_bf16 ? sized(bf16_t{}, bf16_t{}) : sized(bf16_t{}, 0.0f);
    return g_bf16 ? sized(0.0f, bf16_t{}) : sized(0.0f, 0.0f);
}

// Matrices of every chunk (delta_fwd.hip); both: the transposes too.
hipError_t launch_delta_prep(const DeltaArgs &a, const DeltaWs &ws, bool both, hipStream_t stream);
// The recurrence over the chunks; with ws.S0 the states entering them and U
// are kept.
hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaWs &ws, hipStream_t stream);

}  // namespace ssm
