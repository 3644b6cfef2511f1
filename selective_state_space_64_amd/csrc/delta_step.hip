// delta_step.hip -- the gated delta rule one step at a time, for gfx950: the
// decode step on persistent states, and the same loop over short sequences.
//
// Per head, with the decayed state D = e^g S (K x V):
//     u = beta (v - D^T k),   S' = D + k u^T,
//     y = scale S'^T q = scale (D^T q + (k . q) u)
// so one pass over the state gives both products that need a sum over K, and
// the state is read once and written once.  A workgroup owns a tile of
// columns (V) of one head's state and all K rows, in registers: a thread 4
// neighbouring columns of every 256 / (tile / 4)-th row.  The sums over K go
// through lane moves inside a wave and LDS across the four waves.  A decode
// step is bound by the state's bytes (2 x 4 K V per head).
#include "delta_launch.hpp"
#include "ssm_device.hpp"
#include "ssm_launch.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct StepParams {
    int seqlen, rep, h, K, V, nslots;
    float scale;
    const void *q, *k, *v;
    const float *g, *beta, *s0;
    void *y;
    float *s1;
    const int *slots, *cu;
    DeltaStride sq, sk, sv, sy, sg, sbeta;
};

// (a NaN stays one)
__device__ inline float delta_decay(float g) { return exp2_hw((g < -110.0f ? -110.0f : g) * kLog2e); }

// kCols columns a tile; kRows rows a thread (K <= kRows * 1024 / kCols).
// kVec: 16-byte state accesses (V a multiple of 4).
template <typename T, typename TOut, int kCols, int kRows, bool kVec>
__global__ __launch_bounds__(kThreads) void delta_steps_kernel(const StepParams p)
{
    constexpr int kAcross = kCols / 4;             // threads along the columns
    constexpr int kDown = kThreads / kAcross;      // threads along the rows
    constexpr int kWaveDown = 64 / kAcross;        // of them in one wave
    __shared__ float sums[2][4][2][kCols];         // [step parity][wave][D^T k, D^T q][column]
    __shared__ float kq[2][2][kDeltaMaxK];         // [step parity][k, q]
    const int tid = int(threadIdx.x), wave = tid >> 6;
    const int across = tid % kAcross, down = tid / kAcross;
    const int head = int(blockIdx.y), seq = int(blockIdx.z), qk_head = head / p.rep;
    const int c0 = int(blockIdx.x) * kCols + across * 4;  // the thread's first column
    const int K = p.K, V = p.V;

    long long t0 = 0, bi = seq;
    int len = p.seqlen;
    if (p.cu) {
        const int lo = min(max(p.cu[seq], 0), p.seqlen);
        len = min(max(p.cu[seq + 1], lo), p.seqlen) - lo;
        t0 = lo;
        bi = 0;
    }
    long long slot = seq;
    bool live = true;
    if (p.slots) {
        slot = p.slots[seq];
        live = slot >= 0 && slot < p.nslots;
    }
    const T *q = static_cast<const T *>(p.q) + bi * p.sq.b + t0 * p.sq.t + qk_head * p.sq.h;
    const T *k = static_cast<const T *>(p.k) + bi * p.sk.b + t0 * p.sk.t + qk_head * p.sk.h;
    const T *v = static_cast<const T *>(p.v) + bi * p.sv.b + t0 * p.sv.t + head * p.sv.h;
    const float *g = p.g + bi * p.sg.b + t0 * p.sg.t + head * p.sg.h;
    const float *beta = p.beta + bi * p.sbeta.b + t0 * p.sbeta.t + head * p.sbeta.h;
    TOut *y = static_cast<TOut *>(p.y) + bi * p.sy.b + t0 * p.sy.t + head * p.sy.h;
    if (!live) {  // uniform over the workgroup
        if (down == 0)
            for (int i = 0; i < 4; ++i)
                if (c0 + i < V) {
                    if constexpr (sizeof(TOut) == 4) y[c0 + i] = 0.0f;
                    else y[c0 + i].bits = 0;
                }
        return;
    }

    const long long at = (slot * p.h + head) * (long long)K * V;
    f32x4 S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = down + i * kDown;
        S[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (p.s0 && row < K) {
            const float *s = p.s0 + at + (long long)row * V + c0;
            if (kVec) {
                if (c0 < V) S[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(s));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c0 + e < V) S[i][e] = s[e];
            }
        }
    }

    for (int t = 0; t < len; ++t) {
        const int par = t & 1;
        // the step's key and query, zero behind K
        if (tid < kDeltaMaxK) {
            kq[par][0][tid] = tid < K ? io<T>::load1(k + tid) : 0.0f;
            kq[par][1][tid] = tid < K ? io<T>::load1(q + tid) : 0.0f;
        }
        const float a = delta_decay(*g), b = *beta;
        float vv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = c0 + e < V ? io<T>::load1(v + c0 + e) : 0.0f;
        __syncthreads();
        float sk[4] = {0, 0, 0, 0}, sq[4] = {0, 0, 0, 0}, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float kr = kq[par][0][down + i * kDown], qr = kq[par][1][down + i * kDown];
            dot = __builtin_fmaf(kr, qr, dot);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S[i][e] *= a;
                sk[e] = __builtin_fmaf(S[i][e], kr, sk[e]);
                sq[e] = __builtin_fmaf(S[i][e], qr, sq[e]);
            }
        }
        // over the wave's rows, then over the waves
#pragma unroll
        for (int off = kAcross; off < 64; off *= 2) {
            dot += __shfl_xor(dot, off);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sk[e] += __shfl_xor(sk[e], off);
                sq[e] += __shfl_xor(sq[e], off);
            }
        }
        __shared__ float dots[2][4];
        if (down % kWaveDown == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sums[par][wave][0][across * 4 + e] = sk[e];
                sums[par][wave][1][across * 4 + e] = sq[e];
            }
            if (across == 0) dots[par][wave] = dot;
        }
        __syncthreads();
        dot = dots[par][0] + dots[par][1] + dots[par][2] + dots[par][3];
        float u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = across * 4 + e;
            const float dk = sums[par][0][0][c] + sums[par][1][0][c] + sums[par][2][0][c] + sums[par][3][0][c];
            const float dq = sums[par][0][1][c] + sums[par][1][1][c] + sums[par][2][1][c] + sums[par][3][1][c];
            u[e] = b * (vv[e] - dk);
            const float out = p.scale * __builtin_fmaf(dot, u[e], dq);
            if (down == 0 && c0 + e < V) {
                if constexpr (sizeof(TOut) == 4) y[c0 + e] = out;
                else y[c0 + e].bits = uint16_t(pack_bf16x2(out, out));
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float kr = kq[par][0][down + i * kDown];
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][e] = __builtin_fmaf(kr, u[e], S[i][e]);
        }
        q += p.sq.t;
        k += p.sk.t;
        v += p.sv.t;
        g += p.sg.t;
        beta += p.sbeta.t;
        y += p.sy.t;
    }

    if (!p.s1) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = down + i * kDown;
        if (row < K) {
            float *s = p.s1 + at + (long long)row * V + c0;
            if (kVec) {
                if (c0 < V) __builtin_nontemporal_store(S[i], reinterpret_cast<f32x4 *>(s));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c0 + e < V) s[e] = S[i][e];
            }
        }
    }
}

template <typename T, typename TOut, int kCols, int kRows>
hipError_t launch_rows(const StepParams &p, int nseq, bool vec, hipStream_t stream)
{
    const dim3 grid((p.V + kCols - 1) / kCols, p.h, nseq);
    if (log_enabled())
        log_line("delta_steps: delta_steps_kernel<in %s, out %s, columns %d, rows a thread %d, vec %d>, "
                 "grid (%u, %u, %u) x %d threads", type_tag<T>(), type_tag<TOut>(), kCols, kRows, int(vec),
                 grid.x, grid.y, grid.z, kThreads);
    if (vec) delta_steps_kernel<T, TOut, kCols, kRows, true><<<grid, dim3(kThreads), 0, stream>>>(p);
    else delta_steps_kernel<T, TOut, kCols, kRows, false><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, typename TOut, int kCols>
hipError_t launch_cols(const StepParams &p, int nseq, bool vec, hipStream_t stream)
{
    constexpr int down = kThreads / (kCols / 4);
    if (p.K <= down) return launch_rows<T, TOut, kCols, 1>(p, nseq, vec, stream);
    if (p.K <= 2 * down) return launch_rows<T, TOut, kCols, 2>(p, nseq, vec, stream);
    if (p.K <= 4 * down) return launch_rows<T, TOut, kCols, 4>(p, nseq, vec, stream);
    if constexpr (down * 4 < kDeltaMaxK) return launch_rows<T, TOut, kCols, 8>(p, nseq, vec, stream);
    return hipErrorInvalidValue;
}

template <typename T, typename TOut>
hipError_t launch_typed(const StepParams &p, int nseq, bool vec, hipStream_t stream)
{
    // Tiles of 32 columns move the most bytes a second; 16 where those would
    // leave compute units without work.  64 states of 40 heads of 128 x 128, out
    // of memory: 16 columns 119 us, 32 67.5, 64 91, 128 69 (336 MB; a copy of as
    // many bytes 69 us); 74 us with 32 columns and ordinary in place of
    // nontemporal accesses.
    const long long wide = (long long)((p.V + 31) / 32) * p.h * nseq;
    return wide >= 1024 ? launch_cols<T, TOut, 32>(p, nseq, vec, stream)
                        : launch_cols<T, TOut, 16>(p, nseq, vec, stream);
}

hipError_t launch_steps(const DeltaArgs &a, const float *s0, float *s1, const int *slots, int nslots,
                        hipStream_t stream)
{
    StepParams p{a.seqlen, a.h / a.hk, a.h, a.K, a.V, nslots, a.scale, a.q, a.k, a.v, a.g, a.beta, s0,
                 a.y, s1, slots, a.cu, a.sq, a.sk, a.sv, a.sy, a.sg, a.sbeta};
    const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(s0) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(s1) % 16 == 0;
    if (a.in_bf16 && a.out_bf16) return launch_typed<bf16_t, bf16_t>(p, a.nseq, vec, stream);
    if (a.in_bf16) return launch_typed<bf16_t, float>(p, a.nseq, vec, stream);
    if (a.out_bf16) return launch_typed<float, bf16_t>(p, a.nseq, vec, stream);
    return launch_typed<float, float>(p, a.nseq, vec, stream);
}

}  // namespace

hipError_t launch_delta_steps(const DeltaArgs &a, hipStream_t stream)
{
    return launch_steps(a, a.h0, a.hL, nullptr, 0, stream);
}

hipError_t launch_delta_update(const DeltaUpdateArgs &a, hipStream_t stream)
{
    return launch_steps(a.f, a.state, a.state, a.slots, a.num_slots, stream);
}

}  // namespace ssm
