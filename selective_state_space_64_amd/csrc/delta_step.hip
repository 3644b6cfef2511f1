// delta_step.hip -- the gated delta rule's decode step on persistent states,
// for gfx950.
//
// Per head, with the decayed state D = e^g S (K x V):
//     u = beta (v - D^T k),   S' = D + k u^T,
//     y = scale S'^T q = scale (D^T q + (k . q) u)
// so one pass over the state gives both products that need a sum over K, and
// the state is read once and written once.  A workgroup owns a tile of
// columns (V) of one head's state and all K rows, in registers: a thread 4
// neighbouring columns of every 256 / (tile / 4)-th row.  The sums over K go
// through lane moves inside a wave and LDS across the four waves.  A decode
// step is bound by the state's bytes (2 x 4 K V per head): 64 sequences of 40
// heads, 128 x 128, take 70.4 us a call for 336 MB (4.8 TB/s, a large copy's
// rate), one sequence 11 us, the host's part of the call.
#include "delta_launch.hpp"
#include "ssm_device.hpp"
#include "ssm_launch.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct StepParams {
    int rep, h, K, V, nslots;
    float scale;
    const void *q, *k, *v;
    const float *g, *beta;
    void *y;
    float *state;
    const int *slots;
    DeltaStride sq, sk, sv, sy, sg, sbeta;
};

// (a NaN stays one)
__device__ inline float delta_decay(float g) { return exp2_hw((g < -110.0f ? -110.0f : g) * kLog2e); }

// kCols columns a tile; kRows rows a thread (K <= kRows * 1024 / kCols).
// kVec: 16-byte state accesses (V a multiple of 4).
template <typename T, typename TOut, int kCols, int kRows, bool kVec>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(const StepParams p)
{
    constexpr int kAcross = kCols / 4;          // threads along the columns
    constexpr int kDown = kThreads / kAcross;   // threads along the rows
    constexpr int kWaveDown = 64 / kAcross;     // of them in one wave
    __shared__ float sums[4][2][kCols];         // [wave][D^T k, D^T q][column]
    __shared__ float kq[2][kDeltaMaxK], dots[4];  // [k, q]; k . q by wave
    const int tid = int(threadIdx.x), wave = tid >> 6;
    const int across = tid % kAcross, down = tid / kAcross;
    const int head = int(blockIdx.y), row = int(blockIdx.z), qk_head = head / p.rep;
    const int c0 = int(blockIdx.x) * kCols + across * 4;  // the thread's first column
    const int K = p.K, V = p.V;

    long long slot = row;
    bool live = true;
    if (p.slots) {
        slot = p.slots[row];
        live = slot >= 0 && slot < p.nslots;
    }
    const T *q = static_cast<const T *>(p.q) + row * p.sq.b + qk_head * p.sq.h;
    const T *k = static_cast<const T *>(p.k) + row * p.sk.b + qk_head * p.sk.h;
    const T *v = static_cast<const T *>(p.v) + row * p.sv.b + head * p.sv.h;
    TOut *y = static_cast<TOut *>(p.y) + row * p.sy.b + head * p.sy.h;
    auto put = [&](int c, float x) {
        if constexpr (sizeof(TOut) == 4) y[c] = x;
        else y[c].bits = uint16_t(pack_bf16x2(x, x));
    };
    if (!live) {  // uniform over the workgroup
        if (down == 0)
            for (int e = 0; e < 4; ++e)
                if (c0 + e < V) put(c0 + e, 0.0f);
        return;
    }

    // read once and written once: neither stays in a cache
    float *state = p.state + (slot * p.h + head) * (long long)K * V + c0;
    f32x4 S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int n = down + i * kDown;
        S[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (n < K) {
            const float *s = state + (long long)n * V;
            if (kVec) {
                if (c0 < V) S[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(s));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c0 + e < V) S[i][e] = s[e];
            }
        }
    }
    kq[0][tid] = tid < K ? io<T>::load1(k + tid) : 0.0f;  // kThreads == kDeltaMaxK
    kq[1][tid] = tid < K ? io<T>::load1(q + tid) : 0.0f;
    const float a = delta_decay(p.g[row * p.sg.b + head * p.sg.h]);
    const float b = p.beta[row * p.sbeta.b + head * p.sbeta.h];
    float vv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) vv[e] = c0 + e < V ? io<T>::load1(v + c0 + e) : 0.0f;
    __syncthreads();
    float sk[4] = {0, 0, 0, 0}, sq[4] = {0, 0, 0, 0}, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float kr = kq[0][down + i * kDown], qr = kq[1][down + i * kDown];
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
    if (down % kWaveDown == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sums[wave][0][across * 4 + e] = sk[e];
            sums[wave][1][across * 4 + e] = sq[e];
        }
        if (across == 0) dots[wave] = dot;
    }
    __syncthreads();
    dot = dots[0] + dots[1] + dots[2] + dots[3];
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = across * 4 + e;
        const float dk = sums[0][0][c] + sums[1][0][c] + sums[2][0][c] + sums[3][0][c];
        const float dq = sums[0][1][c] + sums[1][1][c] + sums[2][1][c] + sums[3][1][c];
        u[e] = b * (vv[e] - dk);
        if (down == 0 && c0 + e < V) put(c0 + e, p.scale * __builtin_fmaf(dot, u[e], dq));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int n = down + i * kDown;
        const float kr = kq[0][n];
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][e] = __builtin_fmaf(kr, u[e], S[i][e]);
        if (n < K) {
            float *s = state + (long long)n * V;
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
hipError_t launch_rows(const StepParams &p, int batch, bool vec, hipStream_t stream)
{
    const dim3 grid((p.V + kCols - 1) / kCols, p.h, batch);
    if (log_enabled())
        log_line("delta_update: delta_step_kernel<in %s, out %s, columns %d, rows a thread %d, vec %d>, "
                 "grid (%u, %u, %u) x %d threads", type_tag<T>(), type_tag<TOut>(), kCols, kRows, int(vec),
                 grid.x, grid.y, grid.z, kThreads);
    if (vec) delta_step_kernel<T, TOut, kCols, kRows, true><<<grid, dim3(kThreads), 0, stream>>>(p);
    else delta_step_kernel<T, TOut, kCols, kRows, false><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, typename TOut, int kCols>
hipError_t launch_cols(const StepParams &p, int batch, bool vec, hipStream_t stream)
{
    constexpr int down = kThreads / (kCols / 4);  // 16 columns: 64, and K is over 64 (launch_typed)
    if constexpr (kCols == 32)
        if (p.K <= down) return launch_rows<T, TOut, kCols, 1>(p, batch, vec, stream);
    if (p.K <= 2 * down) return launch_rows<T, TOut, kCols, 2>(p, batch, vec, stream);
    if (p.K <= 4 * down) return launch_rows<T, TOut, kCols, 4>(p, batch, vec, stream);
    if constexpr (down * 4 < kDeltaMaxK) return launch_rows<T, TOut, kCols, 8>(p, batch, vec, stream);
    return hipErrorInvalidValue;
}

template <typename T, typename TOut>
hipError_t launch_typed(const StepParams &p, int batch, bool vec, hipStream_t stream)
{
    // Tiles of 32 columns move the most bytes a second; 16 give twice the workgroups,
    // each with half as long a column of the state to a thread, where the card is far from
    // full.  us a step in a graph, states out of memory, 32 against 16 columns, by tiles of
    // 32: K = 64 3.65 / 4.02 at 64 tiles, 3.9 / 5.1 at 256; K = 128 5.7 / 4.4 at 64, 5.9 / 5.5 at
    // 192, 6.0 / 6.0 at 256, 6.5 / 7.2 at 384, 8.0 / 12.6 at 960, 35 / 55 at 5120; K = 256 9.1 / 6.5
    // at 64, 9.6 / 8.4 at 256, 11.1 / 12.7 at 512, 20.0 / 18.4 at 768, 21.1 / 24.5 at 1024.
    const long long tiles = (long long)((p.V + 31) / 32) * p.h * batch;
    return p.K <= 64 || tiles >= 2 * p.K ? launch_cols<T, TOut, 32>(p, batch, vec, stream)
                                         : launch_cols<T, TOut, 16>(p, batch, vec, stream);
}

}  // namespace

hipError_t launch_delta_update(const DeltaUpdateArgs &u, hipStream_t stream)
{
    const DeltaArgs &a = u.f;
    const StepParams p{a.h / a.hk, a.h, a.K, a.V, u.num_slots, a.scale, a.q, a.k, a.v, a.g, a.beta, a.y, u.state,
                       u.slots, a.sq, a.sk, a.sv, a.sy, a.sg, a.sbeta};
    const bool vec = a.V % 4 == 0;  // the state itself is aligned to 16 bytes
    if (a.in_bf16 && a.out_bf16) return launch_typed<bf16_t, bf16_t>(p, a.batch, vec, stream);
    if (a.in_bf16) return launch_typed<bf16_t, float>(p, a.batch, vec, stream);
    if (a.out_bf16) return launch_typed<float, bf16_t>(p, a.batch, vec, stream);
    return launch_typed<float, float>(p, a.batch, vec, stream);
}

}  // namespace ssm
