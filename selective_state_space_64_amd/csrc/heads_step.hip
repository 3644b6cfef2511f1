// heads_step.hip -- the decode step of the selective scan with one decay a
// head, on persistent states, for gfx950.
//
// Per head, with D = softplus(dt + dt_bias) and the state S (N x P):
//     S' = e^{D A} S + (D B) x^T,   y = S'^T C + Dskip x
// The state is read once and written once, which is what bounds the step (2 x
// 4 N P bytes a head).  A workgroup owns a tile of columns (P) of one head's
// state and all N rows: a thread 4 neighbouring columns of every 256 /
// (tile / 4)-th row.  An element is stored as soon as it is updated; only y waits
// for the sum over N, which goes through lane moves inside a wave and LDS across
// the four.  64 sequences of 80 heads of 128 x 64, bf16 inputs: 58.1 us, 5.8 TB/s; with their
// states in a pool of 80 slots 61.3 us, 5.5 TB/s; one sequence 4 us of kernel in a call of 12.
#include "heads_launch.hpp"
#include "ssm_device.hpp"
#include "ssm_launch.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct HeadsStep {
    int rep, h, N, P, nslots;
    const void *x, *dt, *B, *C;
    const float *A, *bias, *D;
    void *y;
    float *state;
    const int *slots;
    DeltaStride sx, sdt, sB, sC, sy;
};

// kCols columns a tile; kRows rows a thread (N <= kRows * 1024 / kCols).
// kVec: 16-byte state accesses (P a multiple of 4).
template <typename T, typename TOut, int kCols, int kRows, bool kVec>
__global__ __launch_bounds__(kThreads) void heads_step_kernel(const HeadsStep p)
{
    constexpr int kAcross = kCols / 4;         // threads along the columns
    constexpr int kDown = kThreads / kAcross;  // threads along the rows
    __shared__ float sums[4][kCols];           // [wave][column]
    __shared__ float in[2][kHeadsMaxN];        // B, C
    static_assert(kThreads == kHeadsMaxN, "a thread an entry");
    const int tid = int(threadIdx.x), wave = tid >> 6;
    const int across = tid % kAcross, down = tid / kAcross;
    const int head = int(blockIdx.y), row = int(blockIdx.z), group = head / p.rep;
    const int c0 = int(blockIdx.x) * kCols + across * 4;  // the thread's first column
    const int N = p.N, P = p.P;

    long long slot = row;
    bool live = true;
    if (p.slots) {
        slot = p.slots[row];
        live = slot >= 0 && slot < p.nslots;
    }
    const T *x = static_cast<const T *>(p.x) + row * p.sx.b + head * p.sx.h;
    const T *B = static_cast<const T *>(p.B) + row * p.sB.b + group * p.sB.h;
    const T *C = static_cast<const T *>(p.C) + row * p.sC.b + group * p.sC.h;
    TOut *y = static_cast<TOut *>(p.y) + row * p.sy.b + head * p.sy.h;
    auto put = [&](int c, float v) {
        if constexpr (sizeof(TOut) == 4) y[c] = v;
        else y[c].bits = uint16_t(pack_bf16x2(v, v));
    };
    if (!live) {  // uniform over the workgroup
        if (down == 0)
            for (int e = 0; e < 4; ++e)
                if (c0 + e < P) put(c0 + e, 0.0f);
        return;
    }

    // One buffer is the head's state: rows behind N and columns behind P read as 0 and
    // are not stored, without a branch.  Read once and written once: neither stays in a
    // cache (kNt).
    constexpr int kNt = 2;
    const auto buf = __builtin_amdgcn_make_buffer_rsrc(p.state + (slot * p.h + head) * (long long)N * P, 0, N * P * 4,
                                                       0x00020000);
    uint32_t at[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e] = c0 + e < P ? uint32_t(down * P + c0 + e) * 4u : 0x80000000u;
    const uint32_t rows = uint32_t(kDown * P) * 4u;
    f32x4 S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if constexpr (kVec) {
            S[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, at[0] + i * rows, 0, kNt));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[i][e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, at[e] + i * rows, 0, kNt));
        }
    }
    in[0][tid] = tid < N ? io<T>::load1(B + tid) : 0.0f;  // kThreads == kHeadsMaxN
    in[1][tid] = tid < N ? io<T>::load1(C + tid) : 0.0f;
    const float raw = io<T>::load1(static_cast<const T *>(p.dt) + row * p.sdt.b + head * p.sdt.h);
    const float dt = softplus(raw + (p.bias ? p.bias[head] : 0.0f)), la = dt * p.A[head];
    const float a = exp2_hw((la < -110.0f ? -110.0f : la) * kLog2e);  // (a NaN stays one)
    const float D = p.D ? p.D[head] : 0.0f;
    float v[4], sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c0 + e < P ? io<T>::load1(x + c0 + e) : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float b = dt * in[0][down + i * kDown], c = in[1][down + i * kDown];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = __builtin_fmaf(a, S[i][e], b * v[e]);
            sum[e] = __builtin_fmaf(S[i][e], c, sum[e]);
        }
        if constexpr (kVec) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[i]), buf, at[0] + i * rows, 0, kNt);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][e]), buf, at[e] + i * rows, 0, kNt);
        }
    }
    // over the wave's rows, then over the waves
#pragma unroll
    for (int off = kAcross; off < 64; off *= 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], off);
    if ((tid & 63) < kAcross)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][across * 4 + e] = sum[e];
    __syncthreads();
    if (down == 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = across * 4 + e;
            if (c0 + e < P) put(c0 + e, __builtin_fmaf(D, v[e], (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c])));
        }
}

template <typename T, typename TOut, int kCols, int kRows, bool kVec>
hipError_t launch_rows(const HeadsStep &p, int batch, hipStream_t stream)
{
    const dim3 grid((p.P + kCols - 1) / kCols, p.h, batch);
    if (log_enabled())
        log_line("head_scan_update: heads_step_kernel<in %s, out %s, columns %d, rows a thread %d, vec %d>, "
                 "grid (%u, %u, %u) x %d threads", type_tag<T>(), type_tag<TOut>(), kCols, kRows, int(kVec),
                 grid.x, grid.y, grid.z, kThreads);
    heads_step_kernel<T, TOut, kCols, kRows, kVec><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

// Tiles of 64 columns where they leave no lane idle, else of 32.  Measured in one
// run, 80 heads of 128 x 64, bf16 inputs, tiles of 64, 32 and 16 columns: 64 sequences 58.1,
// 60.0 and 97.6 us (fp32 inputs 54.5, 57.6 and 99.9), in a pool of 80 slots 61.3, 63.5 and
// 108.3; one sequence 12.0 with each (the host's call).
template <typename T, typename TOut>
hipError_t launch_typed(const HeadsStep &p, int batch, bool vec, hipStream_t stream)
{
    if (p.P % 64 == 0) {
        if (p.N <= 32) return launch_rows<T, TOut, 64, 2, true>(p, batch, stream);
        if (p.N <= 64) return launch_rows<T, TOut, 64, 4, true>(p, batch, stream);
        if (p.N <= 128) return launch_rows<T, TOut, 64, 8, true>(p, batch, stream);
        return launch_rows<T, TOut, 64, 16, true>(p, batch, stream);
    }
    auto sized = [&](auto v) {
        constexpr bool kVec = decltype(v)::value;
        if (p.N <= 32) return launch_rows<T, TOut, 32, 1, kVec>(p, batch, stream);
        if (p.N <= 64) return launch_rows<T, TOut, 32, 2, kVec>(p, batch, stream);
        if (p.N <= 128) return launch_rows<T, TOut, 32, 4, kVec>(p, batch, stream);
        return launch_rows<T, TOut, 32, 8, kVec>(p, batch, stream);
    };
    return vec ? sized(std::true_type{}) : sized(std::false_type{});
}

}  // namespace

hipError_t launch_heads_update(const HeadsUpdateArgs &u, hipStream_t stream)
{
    const HeadsArgs &a = u.f;
    const HeadsStep p{a.h / a.groups, a.h, a.N, a.P, u.num_slots, a.x, a.dt, a.B, a.C, a.A, a.dt_bias, a.Dskip, a.y,
                      u.state, u.slots, a.sx, a.sdt, a.sB, a.sC, a.sy};
    const bool vec = a.P % 4 == 0;  // the state itself is aligned to 16 bytes
    if (a.in_bf16 && a.out_bf16) return launch_typed<bf16_t, bf16_t>(p, a.batch, vec, stream);
    if (a.in_bf16) return launch_typed<bf16_t, float>(p, a.batch, vec, stream);
    if (a.out_bf16) return launch_typed<float, bf16_t>(p, a.batch, vec, stream);
    return launch_typed<float, float>(p, a.batch, vec, stream);
}

}  // namespace ssm
