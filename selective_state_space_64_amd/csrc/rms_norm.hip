// rms_norm.hip -- root-mean-square norm with the residual's addition and an
// 8-bit output with block scales, and its gradients, for gfx950 (C ABI in
// include/ssm_rms.h).
//
// Per row of n channels:
//     h = x + residual,  r = (mean(h^2) + eps)^(-1/2),  y = h r w
// and for l = sum dy . y + sum dh . h, with u = dy w:
//     dh' = r (u - h r^2 mean(u h)) + dh,   dw = sum dy h r over the rows
// Both sums of a row's gradient (h^2 and u h) are taken in one pass, so that a
// row is read once and waits for one sum over the workgroup.  Each input is read
// once and each output written once: the calls are bound by HBM bandwidth.
// 4 x 2048 rows of 2560, bf16 x, fp32 stream, 8-bit output: 45 us for 231 MB (5.1
// TB/s); gradients with an fp32 stream 76 us for 336 MB (4.4 TB/s).
//
// A row is held in registers by one wave (up to 512 channels) or by a
// workgroup of just as many waves as it takes; a thread keeps the same channels
// from row to row, so that the weight stays in registers and dw is summed there,
// written once a thread, and added in a fixed order by a second small kernel.
// Channels go to lanes in runs: 8 neighbours a lane where 16-byte accesses fit,
// so that 16 lanes hold the 128 channels of a scale; otherwise lane l of a wave
// holds l and l + 64 of 128.  Rows beyond the registers of 1024 threads are read
// a second time.
#include "ssm_rms.h"

#include "ssm_device.hpp"
#include "ssm_launch.hpp"
#include "ssm_stride.hpp"

namespace ssm {
namespace {

constexpr int kMaxThreads = 1024, kWaveRows = 4;

struct e4m3_t {
    uint8_t bits;
};
template <typename T> constexpr bool kIs8 = sizeof(T) == 1;

struct RmsParams {
    int seqlen, n;
    unsigned rows, splits;  // splits rows are in work at once
    float eps, inv_n;
    // x, residual, residual_out, y | h, dy, dh, dx, dresidual
    const void *in[3];
    void *out[2];
    const float *weight;
    float *scales, *pw;  // pw: dw's partial sums [splits][n], or NULL
    long long step[5], batch[5];
    DeltaStride ss;  // of the scales; h: from block to block
};

// ------------------------------------------------------------ runs of a row
// E elements a run; run c of a thread starts at first + c * stride, its
// elements lie kGap apart.
template <bool kVec> struct Runs {
    static constexpr int E = kVec ? 8 : 2, kGap = kVec ? 1 : 64;
    int first, stride;
    // tid of the `threads` that hold a row
    __device__ inline Runs(int tid, int threads)
    {
        first = kVec ? tid * 8 : (tid >> 6) * 128 + (tid & 63);
        stride = threads * E;
    }
};

// Whole runs are there or not (n % 8 == 0); others are checked by element.
template <typename T, bool kVec> __device__ inline void get(const T *p, int i, int n, float *v)
{
    constexpr int E = Runs<kVec>::E;
    if constexpr (kVec) {
        if (i < n) {
#pragma unroll
            for (int w = 0; w < E / io<T>::kVec; ++w)
                io<T>::unpack(reinterpret_cast<const u32x4 *>(p + i)[w], v + w * io<T>::kVec);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = 0.0f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = i + 64 * e < n ? io<T>::load1(p + i + 64 * e) : 0.0f;
    }
}

__device__ inline uint32_t e4m3x4(float a, float b, float c, float d)
{
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true));
}

template <typename T, bool kVec> __device__ inline void put(T *p, int i, int n, const float *v)
{
    if constexpr (kVec) {
        if (i >= n) return;
        if constexpr (kIs8<T>) {
            typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u32x2 *>(p + i) = u32x2{e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7])};
        } else if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<u32x4 *>(p + i) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        } else {
            reinterpret_cast<f32x4 *>(p + i)[0] = f32x4{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4 *>(p + i)[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int at = i + 64 * e;
            if (at >= n) continue;
            if constexpr (kIs8<T>) p[at].bits = uint8_t(e4m3x4(v[e], 0.0f, 0.0f, 0.0f));
            else if constexpr (sizeof(T) == 2) p[at].bits = uint16_t(pack_bf16x2(v[e], v[e]));
            else p[at] = v[e];
        }
    }
}

// ------------------------------------------------------------ sums
template <int kCtrl> __device__ inline uint32_t dpp_u32(uint32_t v)
{
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), kCtrl, 0xf, 0xf, true));
}
// f over 16 lanes, to all of them (each step takes in a lane of the other half)
template <typename F> __device__ inline uint32_t over16(uint32_t v, F &&f)
{
    v = f(v, dpp_u32<0xB1>(v));   // quad_perm 1,0,3,2
    v = f(v, dpp_u32<0x4E>(v));   // quad_perm 2,3,0,1
    v = f(v, dpp_u32<0x141>(v));  // row_half_mirror
    return f(v, dpp_u32<0x140>(v));  // row_mirror
}
__device__ inline float wave_sum(float v)
{
    auto add = [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
    v = __uint_as_float(over16(__float_as_uint(v), add));
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
// Sums over the threads that hold a row, to all of them.  `part` is the half of
// this row's parity: the barrier between two rows keeps its last readers apart.
template <int K, bool kWave> __device__ inline void row_sums(float (&v)[K], float (*part)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (!kWave) {
        const int waves = int(blockDim.x) >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) part[threadIdx.x >> 6][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
            for (int w = 0; w < waves; ++w) s += part[w][k];
            v[k] = s;
        }
    }
}

// ------------------------------------------------------------ forward
// The run's values in 8 bits and their block's scale.  Magnitudes are compared
// as integers, where a NaN is above infinity.  The quotient is rounded once: t
// is off by an ulp at most, and with the rounded reciprocal the remainder's
// correction gives the nearest float.
template <bool kVec> __device__ inline float block_scale(const float *y)
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < Runs<kVec>::E; ++e) m = max(m, __float_as_uint(y[e]) & 0x7fffffffu);
    m = over16(m, [](uint32_t a, uint32_t b) { return max(a, b); });
    if constexpr (!kVec) {
        m = max(m, uint32_t(__shfl_xor(int(m), 16)));
        m = max(m, uint32_t(__shfl_xor(int(m), 32)));
    }
    const float s = __uint_as_float(m) / 448.0f;
    return s < 0x1p-126f ? 0x1p-126f : s;  // (a NaN stays one)
}
template <bool kVec> __device__ inline void to_scale(float *y, float scale)
{
    const float inv = 1.0f / scale;
#pragma unroll
    for (int e = 0; e < Runs<kVec>::E; ++e) {
        const float t = y[e] * inv, rest = __builtin_fmaf(-t, scale, y[e]);
        // an infinite scale: 0, and NaN for what made it so
        y[e] = scale < __builtin_inff() ? __builtin_fmaf(rest, inv, t) : t;
    }
}

// CH runs a thread; 0: rows of any length, read twice.  kWave: a wave a row.
template <typename T, typename S, typename TOut, bool kVec, int CH, bool kWave>
__global__ __launch_bounds__(kWave ? 64 * kWaveRows : kMaxThreads) void rms_fwd_kernel(const RmsParams p)
{
    constexpr int E = Runs<kVec>::E, M = (CH ? CH : 1) * E;
    __shared__ float part[2][kWave ? 1 : kMaxThreads / 64][1];
    const int tid = kWave ? int(threadIdx.x) & 63 : int(threadIdx.x), threads = kWave ? 64 : int(blockDim.x);
    const unsigned split = kWave ? blockIdx.x * kWaveRows + (threadIdx.x >> 6) : blockIdx.x;
    const Runs<kVec> runs(tid, threads);
    const int n = p.n;
    float w[M];
    auto weights = [&](int i, float *to) {
        if (p.weight) get<float, kVec>(p.weight, i, n, to);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) to[e] = 1.0f;
    };
    if constexpr (CH > 0)
#pragma unroll
        for (int c = 0; c < CH; ++c) weights(runs.first + c * runs.stride, w + c * E);
    int parity = 0;
    for (unsigned row = split; row < p.rows; row += p.splits, parity ^= 1) {
        const unsigned bi = row / unsigned(p.seqlen), t = row - bi * unsigned(p.seqlen);
        auto at = [&](int i) { return (long long)bi * p.batch[i] + (long long)t * p.step[i]; };
        const T *px = static_cast<const T *>(p.in[0]) + at(0);
        const S *pr = p.in[1] ? static_cast<const S *>(p.in[1]) + at(1) : nullptr;
        S *ph = p.out[0] ? static_cast<S *>(p.out[0]) + at(2) : nullptr;
        TOut *py = static_cast<TOut *>(p.out[1]) + at(3);
        float *ps = kIs8<TOut> ? p.scales + (long long)bi * p.ss.b + (long long)t * p.ss.t : nullptr;
        auto input = [&](int i, float *h) {
            get<T, kVec>(px, i, n, h);
            if (pr) {
                float r[E];
                get<S, kVec>(pr, i, n, r);
#pragma unroll
                for (int e = 0; e < E; ++e) h[e] += r[e];
            }
        };
        auto output = [&](int i, const float *h, const float *wt, float r) {
            if (ph) put<S, kVec>(ph, i, n, h);
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = h[e] * r * wt[e];
            if constexpr (kIs8<TOut>) {
                const float s = block_scale<kVec>(y);
                to_scale<kVec>(y, s);
                // one lane of the block's 16 (64)
                if ((tid & (kVec ? 15 : 63)) == 0 && i < n) ps[(i >> 7) * p.ss.h] = s;
            }
            put<TOut, kVec>(py, i, n, y);
        };
        float sum[1] = {0.0f};
        if constexpr (CH > 0) {
            float h[M];
#pragma unroll
            for (int c = 0; c < CH; ++c) input(runs.first + c * runs.stride, h + c * E);
#pragma unroll
            for (int i = 0; i < M; ++i) sum[0] = __builtin_fmaf(h[i], h[i], sum[0]);
            row_sums<1, kWave>(sum, part[parity]);
            const float r = 1.0f / __builtin_sqrtf(sum[0] * p.inv_n + p.eps);
#pragma unroll
            for (int c = 0; c < CH; ++c) output(runs.first + c * runs.stride, h + c * E, w + c * E, r);
        } else {
            // whole waves stay together (a block's lanes are compared): by the run's first lane
            const int lane_off = runs.first - (kVec ? (tid & ~63) * 8 : (tid >> 6) * 128);
            for (int i = runs.first; i - lane_off < n; i += runs.stride) {
                float h[E];
                input(i, h);
#pragma unroll
                for (int e = 0; e < E; ++e) sum[0] = __builtin_fmaf(h[e], h[e], sum[0]);
            }
            row_sums<1, kWave>(sum, part[parity]);
            const float r = 1.0f / __builtin_sqrtf(sum[0] * p.inv_n + p.eps);
            for (int i = runs.first; i - lane_off < n; i += runs.stride) {
                float h[E], wt[E];
                input(i, h);
                weights(i, wt);
                output(i, h, wt, r);
            }
        }
    }
}

// ------------------------------------------------------------ gradients
template <typename S, typename G, bool kVec, int CH, bool kWave>
__global__ __launch_bounds__(kWave ? 64 * kWaveRows : kMaxThreads) void rms_bwd_kernel(const RmsParams p)
{
    constexpr int E = Runs<kVec>::E, M = (CH ? CH : 1) * E;
    __shared__ float part[2][kWave ? 1 : kMaxThreads / 64][2];
    const int tid = kWave ? int(threadIdx.x) & 63 : int(threadIdx.x), threads = kWave ? 64 : int(blockDim.x);
    const unsigned split = kWave ? blockIdx.x * kWaveRows + (threadIdx.x >> 6) : blockIdx.x;
    if (split >= p.splits) return;  // whole rows' threads leave together
    const Runs<kVec> runs(tid, threads);
    const int n = p.n;
    float w[M], dw[M];
    auto weights = [&](int i, float *to) {
        if (p.weight) get<float, kVec>(p.weight, i, n, to);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) to[e] = 1.0f;
    };
#pragma unroll
    for (int i = 0; i < M; ++i) dw[i] = 0.0f;
    if constexpr (CH > 0)
#pragma unroll
        for (int c = 0; c < CH; ++c) weights(runs.first + c * runs.stride, w + c * E);
    int parity = 0;
    for (unsigned row = split; row < p.rows; row += p.splits, parity ^= 1) {
        const unsigned bi = row / unsigned(p.seqlen), t = row - bi * unsigned(p.seqlen);
        auto at = [&](int i) { return (long long)bi * p.batch[i] + (long long)t * p.step[i]; };
        const S *ph = static_cast<const S *>(p.in[0]) + at(0);
        const G *pdy = static_cast<const G *>(p.in[1]) + at(1);
        const S *pdh = p.in[2] ? static_cast<const S *>(p.in[2]) + at(2) : nullptr;
        G *pdx = p.out[0] ? static_cast<G *>(p.out[0]) + at(3) : nullptr;
        S *pdr = p.out[1] ? static_cast<S *>(p.out[1]) + at(4) : nullptr;
        // r u - h r^3 mean(u h) + dh
        auto output = [&](int i, const float *h, const float *u, const float *dh, float r, float k) {
            float d[E];
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = __builtin_fmaf(r, u[e] - h[e] * k, dh[e]);
            if (pdx) put<G, kVec>(pdx, i, n, d);
            if (pdr) put<S, kVec>(pdr, i, n, d);
        };
        auto stream_grad = [&](int i, float *dh) {
            if (pdh) get<S, kVec>(pdh, i, n, dh);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) dh[e] = 0.0f;
        };
        float sum[2] = {0.0f, 0.0f};
        if constexpr (CH > 0) {
            float h[M], dy[M], dh[M];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = runs.first + c * runs.stride;
                get<S, kVec>(ph, i, n, h + c * E);
                get<G, kVec>(pdy, i, n, dy + c * E);
                stream_grad(i, dh + c * E);
            }
#pragma unroll
            for (int i = 0; i < M; ++i) {
                sum[0] = __builtin_fmaf(h[i], h[i], sum[0]);
                sum[1] = __builtin_fmaf(dy[i] * w[i], h[i], sum[1]);
            }
            row_sums<2, kWave>(sum, part[parity]);
            const float r = 1.0f / __builtin_sqrtf(sum[0] * p.inv_n + p.eps), k = r * r * (sum[1] * p.inv_n);
#pragma unroll
            for (int i = 0; i < M; ++i) {
                dw[i] = __builtin_fmaf(dy[i], h[i] * r, dw[i]);
                dy[i] *= w[i];
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
                output(runs.first + c * runs.stride, h + c * E, dy + c * E, dh + c * E, r, k);
        } else {
            for (int i = runs.first; i < n; i += runs.stride) {
                float h[E], dy[E], wt[E];
                get<S, kVec>(ph, i, n, h);
                get<G, kVec>(pdy, i, n, dy);
                weights(i, wt);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sum[0] = __builtin_fmaf(h[e], h[e], sum[0]);
                    sum[1] = __builtin_fmaf(dy[e] * wt[e], h[e], sum[1]);
                }
            }
            row_sums<2, kWave>(sum, part[parity]);
            const float r = 1.0f / __builtin_sqrtf(sum[0] * p.inv_n + p.eps), k = r * r * (sum[1] * p.inv_n);
            for (int i = runs.first; i < n; i += runs.stride) {
                float h[E], dy[E], wt[E], dh[E], sums[E];
                get<S, kVec>(ph, i, n, h);
                get<G, kVec>(pdy, i, n, dy);
                weights(i, wt);
                stream_grad(i, dh);
                if (p.pw) {  // the thread's own channels of its own partial row
                    float *pw = p.pw + (long long)split * n;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int c = i + e * Runs<kVec>::kGap;
                        sums[e] = row != split && c < n ? pw[c] : 0.0f;
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int c = i + e * Runs<kVec>::kGap;
                        if (c < n) pw[c] = __builtin_fmaf(dy[e], h[e] * r, sums[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) dy[e] *= wt[e];
                output(i, h, dy, dh, r, k);
            }
        }
    }
    if constexpr (CH > 0)
        if (p.pw) {
            float *pw = p.pw + (long long)split * n;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = runs.first + c * runs.stride + e * Runs<kVec>::kGap;
                    if (i < n) pw[i] = dw[c * E + e];
                }
        }
}

// dw = the partial rows' sum, in a fixed order: 32 runs of rows a channel, four
// sums a run (their loads do not wait for one another), then the 32 runs.
__global__ __launch_bounds__(1024) void rms_sums_kernel(const float *pw, int splits, int n, float *dweight)
{
    __shared__ float part[32][32];
    const int lane = int(threadIdx.x) & 31, run = int(threadIdx.x) >> 5, c = int(blockIdx.x) * 32 + lane;
    float s[4] = {0, 0, 0, 0};
    if (c < n) {
        const float *src = pw + c;
        int i = run;
        for (; i + 96 < splits; i += 128)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += src[(long long)(i + 32 * j) * n];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 32 * j < splits) s[j] += src[(long long)(i + 32 * j) * n];
    }
    part[run][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (run == 0 && c < n) {
        float t = part[0][lane];
        for (int i = 1; i < 32; ++i) t += part[i][lane];
        dweight[c] = t;
    }
}

// ------------------------------------------------------------ launches
// How a row is held: CH runs by each of `threads` threads (0: read twice), or by
// a wave of a workgroup of four rows.  A wave takes rows of up to 512 channels;
// longer ones fare better with more waves, which have less to load each (bf16 x, fp32
// residual, 21 M elements, the wave's limit at 2048 against 512: 64 against 52 us
// forward and 84 against 75 back at 2048; rows at odd addresses, back, 1024 against 512: 105
// against 87 at 1024, and at 512 a workgroup takes 90 where a wave takes 70).  Rows at odd
// addresses are bound by their memory instructions, 8 (bf16) or 4 (fp32) for one that takes
// 16 bytes: 62 against 43 us forward and 88 against 59 back at 1024.  Rows read twice are those that registers do not hold: at 2560 channels held ones take 59 against 104.
struct Shape {
    int ch, threads;
    bool wave;
};
Shape rms_shape(int n, bool vec)
{
    const int run = vec ? 8 : 2, runs = (n + run - 1) / run;
    if (n <= 512) return {vec ? 1 : 4, 64, true};
    const int waves = vec ? (runs + 63) / 64 : (n + 127) / 128, most = vec ? 2 : 4;
    if (waves <= 16) return {1, 64 * waves, false};
    if (waves <= 16 * most) return {most, 64 * ((waves + most - 1) / most), false};
    return {0, kMaxThreads, false};
}

// Rows in work at once.  Forward: several times what the chip holds, since the next
// workgroups' loads then overlap the last one's stores (2560 channels: 59 us for 2^22 / n
// rows, 51 for twice and 50 for four times as many; short rows gain nothing).
// Gradients: few, so that dw's partial rows stay small beside the tensors, but every
// compute unit one (16-byte accesses, 2^20 / n against 2^21 / n: 80 against 86 us at 2560
// channels, 74 against 81 at 512; 8192: 104 for 128 rows, 77 for 256).  Narrow accesses
// leave more loads to a row: 2^21 / n.
unsigned rms_splits(long long rows, int n, bool bwd, bool vec)
{
    long long want;
    if (bwd) {
        const long long few = (rows + 1) / 2 < 256 ? (rows + 1) / 2 : 256;
        want = (vec ? 1ll << 20 : 1ll << 21) / n;
        if (want < few) want = few;
    } else {
        want = (1ll << 24) / n;
        if (want > 1 << 15) want = 1 << 15;
    }
    return unsigned(want < rows ? want : rows);
}

template <int CH> using Ch = std::integral_constant<int, CH>;
template <typename F> hipError_t by_shape(const Shape &s, bool vec, F &&f)
{
    const std::true_type yes;
    const std::false_type no;
    if (vec && s.wave) return f(yes, Ch<1>{}, yes);
    if (vec) return s.ch == 1 ? f(yes, Ch<1>{}, no) : s.ch == 2 ? f(yes, Ch<2>{}, no) : f(yes, Ch<0>{}, no);
    if (s.wave) return f(no, Ch<4>{}, yes);
    return s.ch == 1 ? f(no, Ch<1>{}, no) : s.ch == 4 ? f(no, Ch<4>{}, no) : f(no, Ch<0>{}, no);
}

template <typename T, typename S, typename TOut>
hipError_t launch_fwd(RmsParams p, bool vec, hipStream_t stream)
{
    const Shape s = rms_shape(p.n, vec);
    p.splits = rms_splits(p.rows, p.n, false, vec);
    return by_shape(s, vec, [&](auto v, auto ch, auto wave) {
        constexpr bool kVec = decltype(v)::value, kWave = decltype(wave)::value;
        constexpr int CH = decltype(ch)::value;
        const unsigned grid = kWave ? (p.splits + kWaveRows - 1) / kWaveRows : p.splits;
        const unsigned block = kWave ? 64 * kWaveRows : s.threads;
        p.splits = kWave ? grid * kWaveRows : grid;
        if (log_enabled())
            log_line("rms_norm: rms_fwd_kernel<in %s, stream %s, out %s, vec %d, runs %d, wave %d>, grid %u x %u threads",
                     type_tag<T>(), type_tag<S>(), kIs8<TOut> ? "e4m3" : sizeof(TOut) == 2 ? "bf16" : "f32", int(kVec), CH,
                     int(kWave), grid, block);
        rms_fwd_kernel<T, S, TOut, kVec, CH, kWave><<<dim3(grid), dim3(block), 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename S, typename G> hipError_t launch_bwd(RmsParams p, bool vec, hipStream_t stream)
{
    const Shape s = rms_shape(p.n, vec);
    p.splits = rms_splits(p.rows, p.n, true, vec);
    return by_shape(s, vec, [&](auto v, auto ch, auto wave) {
        constexpr bool kVec = decltype(v)::value, kWave = decltype(wave)::value;
        constexpr int CH = decltype(ch)::value;
        const unsigned grid = kWave ? (p.splits + kWaveRows - 1) / kWaveRows : p.splits;
        const unsigned block = kWave ? 64 * kWaveRows : s.threads;
        if (log_enabled())
            log_line("rms_norm: rms_bwd_kernel<stream %s, grad %s, vec %d, runs %d, wave %d>, grid %u x %u threads",
                     type_tag<S>(), type_tag<G>(), int(kVec), CH, int(kWave), grid, block);
        rms_bwd_kernel<S, G, kVec, CH, kWave><<<dim3(grid), dim3(block), 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T, typename S>
hipError_t fwd_out(const RmsParams &p, int out_t, bool vec, hipStream_t stream)
{
    if (out_t == SSM_E4M3) return launch_fwd<T, S, e4m3_t>(p, vec, stream);
    if (out_t == SSM_BF16) return launch_fwd<T, S, bf16_t>(p, vec, stream);
    return launch_fwd<T, S, float>(p, vec, stream);
}

using namespace check;

bool rms_sizes(int batch, int seqlen, int dim)
{
    return batch >= 1 && seqlen >= 1 && dim >= 1 && dim <= (1 << 24) && (long long)batch * seqlen < (1ll << 31);
}

size_t esize(int t) { return t == SSM_E4M3 ? 1 : dsize(t); }

// The tensors of a call: p.step and p.batch are filled in.
struct Tensor {
    const void *p;
    int type;
    size_t span;
};
// For the overlap check; a stride that leads nowhere is 0.
Steps rms_steps(const Tensor &t, const RmsParams &p, int i, int batch, int seqlen)
{
    const size_t es = esize(t.type);
    return one_step({t.p, t.span * es, p.n * es, (long long)(p.step[i] * es),
                     batch == 1 ? 0 : (long long)(p.batch[i] * es)}, seqlen);
}
// Exactly the same elements: an output in place of an input.
bool in_place(const Tensor *t, const RmsParams &p, int i, int j, int batch, int seqlen)
{
    return t[i].p == t[j].p && t[i].type == t[j].type && (seqlen == 1 || p.step[i] == p.step[j]) &&
           (batch == 1 || p.batch[i] == p.batch[j]);
}
// All tensors admit the accesses of a run of 8 channels.
bool rms_vec(const Tensor *t, int count, const RmsParams &p, int batch)
{
    if (p.n % 8 || misaligned(p.weight, 16)) return false;
    for (int i = 0; i < count; ++i) {
        if (!t[i].p) continue;
        const int es = int(esize(t[i].type)), bytes = es == 1 ? 8 : 16;
        if (misaligned(t[i].p, bytes) || (p.seqlen > 1 && p.step[i] * es % bytes) ||
            (batch > 1 && p.batch[i] * es % bytes))
            return false;
    }
    return true;
}

}  // namespace
}  // namespace ssm

extern "C" {

ssm_status_t ssm_rms_norm_fwd(int batch, int seqlen, int dim, ssm_dtype_t in_dtype, ssm_dtype_t stream_dtype,
                              const float *eps, const void *x, const void *residual, const float *weight,
                              void *residual_out, ssm_dtype_t out_dtype, void *y, float *scales,
                              const ssm_rms_layout_t *layout, void *stream)
{
    using namespace ssm;
    using namespace ssm::check;
    const int in_t = enum_bits(in_dtype), s_t = enum_bits(stream_dtype), out_t = enum_bits(out_dtype);
    if (!x || !y || (out_t == SSM_E4M3 && !scales)) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(s_t) || (!valid_dtype(out_t) && out_t != SSM_E4M3)) return SSM_ERR_BAD_DTYPE;
    if (!rms_sizes(batch, seqlen, dim)) return SSM_ERR_BAD_SHAPE;
    if (scales && out_t != SSM_E4M3) return SSM_ERR_UNSUPPORTED;
    const ssm_rms_layout_t dense{};
    const ssm_rms_layout_t &lay = layout ? *layout : dense;
    RmsParams p{};
    Tensor t[4] = {{x, in_t, 0}, {residual, s_t, 0}, {residual_out, s_t, 0}, {y, out_t, 0}};
    for (int i = 0; i < 4; ++i)
        if (!row_strides(lay.step[i], lay.batch[i], batch, seqlen, dim, p.step[i], p.batch[i], t[i].span))
            return SSM_ERR_BAD_SHAPE;
    const int blocks = (dim + SSM_RMS_BLOCK - 1) / SSM_RMS_BLOCK;
    size_t scale_span = 0;
    if (!delta_stride(lay.scale_step, lay.scale_block, lay.scale_batch, batch, seqlen, blocks, 1, p.ss, scale_span))
        return SSM_ERR_BAD_SHAPE;
    for (const Tensor &q : t)
        if (misaligned(q.p, esize(q.type))) return SSM_ERR_MISALIGNED;
    if (misaligned(weight, 4) || misaligned(scales, 4)) return SSM_ERR_MISALIGNED;
    p.n = dim;
    Steps st[4];
    for (int i = 0; i < 4; ++i) st[i] = rms_steps(t[i], p, i, batch, seqlen);
    const Steps wt = range_of(weight, 4 * size_t(dim)), sc = range_of(scales, 4 * scale_span);
    // in place: every element is read before it is written, by the same thread
    for (int o = 2; o < 4; ++o) {
        for (int i = 0; i < 2; ++i)
            if (!in_place(t, p, i, o, batch, seqlen) && overlaps(st[o], st[i])) return SSM_ERR_ALIAS;
        if (overlaps(st[o], wt)) return SSM_ERR_ALIAS;
    }
    if (overlaps(st[2], st[3])) return SSM_ERR_ALIAS;
    for (const Steps &q : {st[0], st[1], st[2], st[3], wt})
        if (overlaps(sc, q)) return SSM_ERR_ALIAS;
    p.seqlen = seqlen;
    p.rows = unsigned(batch) * unsigned(seqlen);
    p.eps = eps ? *eps : 1e-5f;
    p.inv_n = 1.0f / float(dim);
    p.in[0] = x;
    p.in[1] = residual;
    p.out[0] = residual_out;
    p.out[1] = y;
    p.weight = weight;
    p.scales = scales;
    const bool vec = rms_vec(t, 4, p, batch);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = in_t == SSM_BF16 ? (s_t == SSM_BF16 ? fwd_out<bf16_t, bf16_t>(p, out_t, vec, s)
                                                             : fwd_out<bf16_t, float>(p, out_t, vec, s))
                                          : (s_t == SSM_BF16 ? fwd_out<float, bf16_t>(p, out_t, vec, s)
                                                             : fwd_out<float, float>(p, out_t, vec, s));
    return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_rms_norm_bwd_workspace_bytes(int batch, int seqlen, int dim)
{
    if (!ssm::rms_sizes(batch, seqlen, dim)) return 0;
    return sizeof(float) * size_t(dim) * size_t(ssm::rms_splits((long long)batch * seqlen, dim, true, false));  // (the larger)
}

ssm_status_t ssm_rms_norm_bwd(int batch, int seqlen, int dim, ssm_dtype_t stream_dtype, ssm_dtype_t grad_dtype,
                              const float *eps, const void *h, const float *weight, const void *dy, const void *dh,
                              void *dx, void *dresidual, float *dweight, void *workspace, size_t workspace_bytes,
                              const ssm_rms_bwd_layout_t *layout, void *stream)
{
    using namespace ssm;
    using namespace ssm::check;
    const int s_t = enum_bits(stream_dtype), g_t = enum_bits(grad_dtype);
    if (!h || !dy || (!dx && !dresidual)) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(s_t) || !valid_dtype(g_t)) return SSM_ERR_BAD_DTYPE;
    if (!rms_sizes(batch, seqlen, dim)) return SSM_ERR_BAD_SHAPE;
    const ssm_rms_bwd_layout_t dense{};
    const ssm_rms_bwd_layout_t &lay = layout ? *layout : dense;
    RmsParams p{};
    Tensor t[5] = {{h, s_t, 0}, {dy, g_t, 0}, {dh, s_t, 0}, {dx, g_t, 0}, {dresidual, s_t, 0}};
    for (int i = 0; i < 5; ++i)
        if (!row_strides(lay.step[i], lay.batch[i], batch, seqlen, dim, p.step[i], p.batch[i], t[i].span))
            return SSM_ERR_BAD_SHAPE;
    for (const Tensor &q : t)
        if (misaligned(q.p, esize(q.type))) return SSM_ERR_MISALIGNED;
    if (misaligned(weight, 4) || misaligned(dweight, 4) || (dweight && misaligned(workspace, 16)))
        return SSM_ERR_MISALIGNED;
    const size_t need = ssm_rms_norm_bwd_workspace_bytes(batch, seqlen, dim), wb = 4 * size_t(dim);
    if (dweight && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
    p.n = dim;
    Steps st[5];
    for (int i = 0; i < 5; ++i) st[i] = rms_steps(t[i], p, i, batch, seqlen);
    const Steps in[] = {st[0], st[1], st[2], range_of(weight, wb)};
    const Steps out[] = {st[3], st[4], range_of(dweight, wb), range_of(dweight ? workspace : nullptr, need)};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 4; ++i) {
            const bool same = (o == 0 && i == 1 && in_place(t, p, 1, 3, batch, seqlen)) ||
                              (o == 1 && i == 2 && in_place(t, p, 2, 4, batch, seqlen));
            if (!same && overlaps(out[o], in[i])) return SSM_ERR_ALIAS;
        }
        for (int i = 0; i < 4; ++i)
            if (i != o && overlaps(out[o], out[i])) return SSM_ERR_ALIAS;
    }
    p.seqlen = seqlen;
    p.rows = unsigned(batch) * unsigned(seqlen);
    p.eps = eps ? *eps : 1e-5f;
    p.inv_n = 1.0f / float(dim);
    p.in[0] = h;
    p.in[1] = dy;
    p.in[2] = dh;
    p.out[0] = dx;
    p.out[1] = dresidual;
    p.weight = weight;
    p.pw = dweight ? static_cast<float *>(workspace) : nullptr;
    const bool vec = rms_vec(t, 5, p, batch);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = s_t == SSM_BF16 ? (g_t == SSM_BF16 ? launch_bwd<bf16_t, bf16_t>(p, vec, s)
                                                      : launch_bwd<bf16_t, float>(p, vec, s))
                                   : (g_t == SSM_BF16 ? launch_bwd<float, bf16_t>(p, vec, s)
                                                      : launch_bwd<float, float>(p, vec, s));
    if (e == hipSuccess && dweight) {
        rms_sums_kernel<<<dim3((dim + 31) / 32), dim3(1024), 0, s>>>(p.pw, int(rms_splits(p.rows, dim, true, vec)), dim,
                                                                     dweight);
        e = hipGetLastError();
    }
    return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
