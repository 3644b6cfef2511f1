// group_norm.hip -- grouped norm with an activation on (batch, L, dim)
// tensors and its gradients, for gfx950 (C ABI in include/ssm_norm.h).
//
// Per (batch, step, group) of n = dim / groups channels, with x replaced by
// x silu(z) for the gate-first form:
//     m = mean(x) or 0,  r = (mean((x - m)^2) + eps)^(-1/2),  h = (x - m) r
//     a = h w + b,       y = a | silu(a) | a silu(z)
// and for l = sum dy . y, with da = dy y'(a) and dh = da w:
//     dx = r (dh - mean(dh) - h mean(dh h))      (no mean(dh) for the RMS form)
//     dw = sum da h,  db = sum da over batch and steps
// Each input is read once and each output written once, so the calls are
// bound by HBM bandwidth.  A group is held by lpg = 1..64 neighbouring lanes
// with up to 4 runs of 8 elements each in registers (the mean is subtracted
// before squaring, no E[x^2] - E[x]^2), and a thread keeps the same channels
// from row to row: weight and bias stay in registers, and dw, db are summed
// there and written once per thread, then added in a fixed order by a second
// small kernel.  Groups too long for that (above 2048 channels, 1024 where
// 16-byte accesses do not fit) take one workgroup each and read x again per
// pass, from the L2.
//
// Measured, calls on tensors out of memory: 4 x 2048 steps of 5120 channels in 40
// groups, bf16 with a gate, 53 us for 252 MB (4.7 TB/s, a large copy's rate), the
// gradients with their second kernel 94 us for 419 MB (4.5 TB/s); a workgroup a row
// of several groups, so that small groups still make whole 16-byte lines.  Small
// calls are bound by the host's part of them (8 x 1536: 11 us).  The gradients'
// partial rows are one per workgroup and channel, added by the second kernel in 5 us
// (by the profiler); more or fewer of them made no difference.  The long groups are far
// from the floor: one group of 5120 bf16 channels, gated, 142 us where 52 are the bytes',
// the gradients 646 us against 86 (three passes over each row, and the sums of every
// row added to the partial rows in memory).
#include "ssm_norm.h"

#include "ssm_check.hpp"
#include "ssm_device.hpp"
#include "ssm_launch.hpp"

namespace ssm {
namespace {

constexpr int kLaneThreads = 256;
constexpr int kWgThreads = 512;
enum { kPlain = 0, kSilu = 1, kGate = 2, kGateFirst = 3 };

struct NormParams {
    int seqlen, groups, n, lpg;
    unsigned rows, row_splits;  // rows = batch * seqlen; row_splits rows are in work at once
    int act, rms;
    float eps, inv_n;
    const void *x, *z, *dy;
    const float *weight, *bias;
    void *out0, *out1;      // y | dx, dz
    float *pw, *pb;         // gradient partials [row_splits][dim], or NULL
    long long step[5], batch[5];  // x, z, dy, out0, out1
};

__device__ inline long long row_at(const NormParams &p, int i, unsigned b, unsigned t)
{
    return (long long)b * p.batch[i] + (long long)t * p.step[i];
}

// E consecutive elements (E = 8: 16-byte accesses; E = 1: one element)
template <typename T, int E>
__device__ inline void get(const T *p, float *v)
{
    if constexpr (E == 1) {
        v[0] = io<T>::load1(p);
    } else {
#pragma unroll
        for (int i = 0; i < E / io<T>::kVec; ++i)
            io<T>::unpack(reinterpret_cast<const u32x4 *>(p)[i], v + i * io<T>::kVec);
    }
}

template <typename T, int E>
__device__ inline void put(T *p, const float *v)
{
    if constexpr (sizeof(T) == 4) {
        if constexpr (E == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < E / 4; ++i)
                reinterpret_cast<f32x4 *>(p)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        }
    } else {
        if constexpr (E == 1) {
            p->bits = uint16_t(pack_bf16x2(v[0], v[0]));
        } else {
#pragma unroll
            for (int i = 0; i < E / 8; ++i)
                reinterpret_cast<u32x4 *>(p)[i] =
                    u32x4{pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                          pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7])};
        }
    }
}

// Sum over lpg neighbouring lanes, to all of them: DPP moves inside 16 lanes
// (each step adds a lane of the other half), shuffles across.
template <int kCtrl>
__device__ inline float dpp_add(float v)
{
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true));
}
__device__ inline float lanes_sum(float v, int lpg)
{
    if (lpg > 1) v = dpp_add<0xB1>(v);    // quad_perm 1,0,3,2
    if (lpg > 2) v = dpp_add<0x4E>(v);    // quad_perm 2,3,0,1
    if (lpg > 4) v = dpp_add<0x141>(v);   // row_half_mirror
    if (lpg > 8) v = dpp_add<0x140>(v);   // row_mirror
    if (lpg > 16) v += __shfl_xor(v, 16);
    if (lpg > 32) v += __shfl_xor(v, 32);
    return v;
}

__device__ inline float sigmoid(float z) { return rcp_hw(1.0f + exp2_hw(-z * kLog2e)); }
// d silu(z) / dz, given s = sigmoid(z); z s (1 - s) tends to 0 at both ends,
// where z may be infinite: 1 - s is 0 or s is 0 and the product is dropped.
__device__ inline float dsilu(float z, float s)
{
    const float t = s * (1.0f - s);
    return t == 0.0f ? s : __builtin_fmaf(z, t, s);
}

// ------------------------------------------------------------ groups in registers
template <typename T, int E, int CH, bool kBwd, typename TOut>
__global__ __launch_bounds__(kLaneThreads) void norm_lanes_kernel(const NormParams p)
{
    const int l = int(threadIdx.x) & (p.lpg - 1);
    const unsigned slot = blockIdx.x * unsigned(kLaneThreads / p.lpg) + threadIdx.x / unsigned(p.lpg);
    if (slot >= p.row_splits * unsigned(p.groups)) return;  // whole groups of lanes leave together
    const unsigned group = slot % unsigned(p.groups), split = slot / unsigned(p.groups);
    const int n = p.n, base = int(group) * n;
    constexpr int M = CH * E;
    float w[M], b[M], sw[M], sb[M];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = (l + c * p.lpg) * E + e;
            w[c * E + e] = (p.weight && i < n) ? p.weight[base + i] : 1.0f;
            b[c * E + e] = (p.bias && i < n) ? p.bias[base + i] : 0.0f;
            sw[c * E + e] = sb[c * E + e] = 0.0f;
        }
    const T *px = static_cast<const T *>(p.x) + base, *pz = static_cast<const T *>(p.z);
    const TOut *pdy = static_cast<const TOut *>(p.dy);
    const bool gated = p.act >= kGate;
    for (unsigned row = split; row < p.rows; row += p.row_splits) {
        const unsigned bi = row / unsigned(p.seqlen), t = row - bi * unsigned(p.seqlen);
        const long long ax = row_at(p, 0, bi, t);
        const long long az = gated ? row_at(p, 1, bi, t) + base : 0;
        const long long ady = kBwd ? row_at(p, 2, bi, t) + base : 0;
        float x[M], z[M], dy[M];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (l + c * p.lpg) * E;
            if (i < n) {
                get<T, E>(px + ax + i, x + c * E);
                if (gated) get<T, E>(pz + az + i, z + c * E);
                if constexpr (kBwd) get<TOut, E>(pdy + ady + i, dy + c * E);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) x[c * E + e] = z[c * E + e] = dy[c * E + e] = 0.0f;
            }
        }
        float h[M];
        if (p.act == kGateFirst) {
#pragma unroll
            for (int i = 0; i < M; ++i) h[i] = x[i] * silu(z[i]);
        } else {
#pragma unroll
            for (int i = 0; i < M; ++i) h[i] = x[i];
        }
        if (!p.rms) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < M; ++i) s += h[i];
            const float mean = lanes_sum(s, p.lpg) * p.inv_n;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if ((l + c * p.lpg) * E < n) {
#pragma unroll
                    for (int e = 0; e < E; ++e) h[c * E + e] -= mean;
                }
        }
        float s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < M; ++i) s2 = __builtin_fmaf(h[i], h[i], s2);
        const float r = 1.0f / __builtin_sqrtf(lanes_sum(s2, p.lpg) * p.inv_n + p.eps);
#pragma unroll
        for (int i = 0; i < M; ++i) h[i] *= r;

        if constexpr (!kBwd) {
            TOut *py = static_cast<TOut *>(p.out0) + row_at(p, 3, bi, t) + base;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = (l + c * p.lpg) * E;
                float y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float a = __builtin_fmaf(h[c * E + e], w[c * E + e], b[c * E + e]);
                    y[e] = p.act == kSilu ? silu(a) : p.act == kGate ? a * silu(z[c * E + e]) : a;
                }
                if (i < n) put<TOut, E>(py + i, y);
            }
        } else {
            float s1 = 0.0f, sh = 0.0f;
#pragma unroll
            for (int i = 0; i < M; ++i) {  // dy becomes dh; z becomes dz under the gate
                float da = dy[i];
                const float a = __builtin_fmaf(h[i], w[i], b[i]);
                if (p.act == kSilu) {
                    da *= dsilu(a, sigmoid(a));
                } else if (p.act == kGate) {
                    const float s = sigmoid(z[i]);
                    da *= z[i] * s;
                    z[i] = dy[i] * a * dsilu(z[i], s);
                }
                sw[i] = __builtin_fmaf(da, h[i], sw[i]);
                sb[i] += da;
                dy[i] = da * w[i];
                s1 += dy[i];
                sh = __builtin_fmaf(dy[i], h[i], sh);
            }
            s1 = p.rms ? 0.0f : lanes_sum(s1, p.lpg) * p.inv_n;
            sh = lanes_sum(sh, p.lpg) * p.inv_n;
#pragma unroll
            for (int i = 0; i < M; ++i) {
                float dx = r * (dy[i] - s1 - h[i] * sh);
                if (p.act == kGateFirst) {
                    const float s = sigmoid(z[i]);
                    const float dxg = dx * z[i] * s;
                    z[i] = dx * x[i] * dsilu(z[i], s);
                    dx = dxg;
                }
                x[i] = dx;
            }
            TOut *pdx = static_cast<TOut *>(p.out0) + row_at(p, 3, bi, t) + base;
            TOut *pdz = static_cast<TOut *>(p.out1) + (gated ? row_at(p, 4, bi, t) + base : 0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = (l + c * p.lpg) * E;
                if (i < n) {
                    put<TOut, E>(pdx + i, x + c * E);
                    if (gated) put<TOut, E>(pdz + i, z + c * E);
                }
            }
        }
    }
    if constexpr (kBwd) {
        const long long at = (long long)split * (p.groups * (long long)n) + base;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = (l + c * p.lpg) * E + e;
                if (i < n) {
                    if (p.pw) p.pw[at + i] = sw[c * E + e];
                    if (p.pb) p.pb[at + i] = sb[c * E + e];
                }
            }
    }
}

// ------------------------------------------------------------ one workgroup a group
// Sum over the workgroup, to every thread (part: one float per wave).
__device__ inline float wg_sum(float v, float *part)
{
    v = lanes_sum(v, 64);
    __syncthreads();  // the readers of the last sum are done
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWgThreads / 64; ++i) s += part[i];
    return s;
}

template <typename T, int E, bool kBwd, typename TOut>
__global__ __launch_bounds__(kWgThreads) void norm_wg_kernel(const NormParams p)
{
    __shared__ float part[kWgThreads / 64];
    const unsigned group = blockIdx.x % unsigned(p.groups), split = blockIdx.x / unsigned(p.groups);
    const int n = p.n, first = int(threadIdx.x) * E, stride = kWgThreads * E;
    const long long base = (long long)group * n;
    const bool gated = p.act >= kGate, gate_first = p.act == kGateFirst;
    const long long sums_at = (long long)split * ((long long)p.groups * n) + base;
    for (unsigned row = split; row < p.rows; row += p.row_splits) {
        const unsigned bi = row / unsigned(p.seqlen), t = row - bi * unsigned(p.seqlen);
        const T *px = static_cast<const T *>(p.x) + row_at(p, 0, bi, t) + base;
        const T *pz = gated ? static_cast<const T *>(p.z) + row_at(p, 1, bi, t) + base : nullptr;
        // the element(s) that are normalised
        auto input = [&](int i, float *h) {
            get<T, E>(px + i, h);
            if (gate_first) {
                float z[E];
                get<T, E>(pz + i, z);
#pragma unroll
                for (int e = 0; e < E; ++e) h[e] *= silu(z[e]);
            }
        };
        float mean = 0.0f, s = 0.0f;
        if (!p.rms) {
            for (int i = first; i < n; i += stride) {
                float h[E];
                input(i, h);
#pragma unroll
                for (int e = 0; e < E; ++e) s += h[e];
            }
            mean = wg_sum(s, part) * p.inv_n;
        }
        s = 0.0f;
        for (int i = first; i < n; i += stride) {
            float h[E];
            input(i, h);
#pragma unroll
            for (int e = 0; e < E; ++e) s = __builtin_fmaf(h[e] - mean, h[e] - mean, s);
        }
        const float r = 1.0f / __builtin_sqrtf(wg_sum(s, part) * p.inv_n + p.eps);
        if constexpr (!kBwd) {
            TOut *py = static_cast<TOut *>(p.out0) + row_at(p, 3, bi, t) + base;
            for (int i = first; i < n; i += stride) {
                float h[E], z[E];
                input(i, h);
                if (p.act == kGate) get<T, E>(pz + i, z);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float a = (h[e] - mean) * r;
                    if (p.weight) a *= p.weight[base + i + e];
                    if (p.bias) a += p.bias[base + i + e];
                    h[e] = p.act == kSilu ? silu(a) : p.act == kGate ? a * silu(z[e]) : a;
                }
                put<TOut, E>(py + i, h);
            }
        } else {
            const TOut *pdy = static_cast<const TOut *>(p.dy) + row_at(p, 2, bi, t) + base;
            TOut *pdx = static_cast<TOut *>(p.out0) + row_at(p, 3, bi, t) + base;
            TOut *pdz = gated ? static_cast<TOut *>(p.out1) + row_at(p, 4, bi, t) + base : nullptr;
            // h = the normalised element, da, and under the gate dz
            auto grads = [&](int i, float *h, float *da, float *dz) {
                input(i, h);
                get<TOut, E>(pdy + i, da);
                if (p.act == kGate) get<T, E>(pz + i, dz);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    h[e] = (h[e] - mean) * r;
                    const float a = h[e] * (p.weight ? p.weight[base + i + e] : 1.0f) +
                                    (p.bias ? p.bias[base + i + e] : 0.0f);
                    if (p.act == kSilu) {
                        da[e] *= dsilu(a, sigmoid(a));
                    } else if (p.act == kGate) {
                        const float sg = sigmoid(dz[e]), dy = da[e];
                        da[e] *= dz[e] * sg;
                        dz[e] = dy * a * dsilu(dz[e], sg);
                    }
                }
            };
            float s1 = 0.0f, sh = 0.0f;
            for (int i = first; i < n; i += stride) {
                float h[E], da[E], dz[E];
                grads(i, h, da, dz);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float dh = da[e] * (p.weight ? p.weight[base + i + e] : 1.0f);
                    s1 += dh;
                    sh = __builtin_fmaf(dh, h[e], sh);
                    // the thread's own channels of its own partial row
                    const bool begin = row == split;
                    if (p.pw) p.pw[sums_at + i + e] = (begin ? 0.0f : p.pw[sums_at + i + e]) + da[e] * h[e];
                    if (p.pb) p.pb[sums_at + i + e] = (begin ? 0.0f : p.pb[sums_at + i + e]) + da[e];
                }
            }
            s1 = p.rms ? 0.0f : wg_sum(s1, part) * p.inv_n;
            sh = wg_sum(sh, part) * p.inv_n;
            for (int i = first; i < n; i += stride) {
                float h[E], da[E], dz[E];
                grads(i, h, da, dz);
                float x[E], z[E];
                if (gate_first) {
                    get<T, E>(px + i, x);
                    get<T, E>(pz + i, z);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float dh = da[e] * (p.weight ? p.weight[base + i + e] : 1.0f);
                    float dx = r * (dh - s1 - h[e] * sh);
                    if (gate_first) {
                        const float sg = sigmoid(z[e]);
                        dz[e] = dx * x[e] * dsilu(z[e], sg);
                        dx *= z[e] * sg;
                    }
                    da[e] = dx;
                }
                put<TOut, E>(pdx + i, da);
                if (gated) put<TOut, E>(pdz + i, dz);
            }
        }
    }
}

// Sums of the partial rows, in a fixed order: 16 runs of rows per channel, four
// sums a run (their loads do not wait for one another), then the 64 sums.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float *pw, const float *pb, int splits,
                                                         int dim, float *dweight, float *dbias)
{
    __shared__ float part[16][64];
    const int c = blockIdx.x * 64 + int(threadIdx.x & 63), run = int(threadIdx.x >> 6);
    const float *src = (blockIdx.y ? pb : pw) + c;
    float *dst = blockIdx.y ? dbias : dweight;
    if (!dst) return;  // the whole workgroup
    float s[4] = {0, 0, 0, 0};
    if (c < dim) {
        int i = run;
        for (; i + 48 < splits; i += 64)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += src[(long long)(i + 16 * j) * dim];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 16 * j < splits) s[j] += src[(long long)(i + 16 * j) * dim];
    }
    part[run][threadIdx.x & 63] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (run == 0 && c < dim) {
        float t = part[0][threadIdx.x];
        for (int i = 1; i < 16; ++i) t += part[i][threadIdx.x];
        dst[c] = t;
    }
}

// Rows in work at once.  A thread keeps its channels for rows / splits rows:
// enough threads to fill the chip (256 compute units of 2048 threads, 8 channels a
// thread), few enough that the gradients' partial rows stay small beside the
// tensors.
int norm_splits(long long rows, int dim, bool bwd)
{
    const long long want = (bwd ? 1ll << 21 : 1ll << 22) / dim;
    return int(want < 1 ? 1 : want < rows ? want : rows);
}

template <typename T, typename TOut, bool kBwd>
hipError_t launch_norm(NormParams p, bool vec, long long rows, hipStream_t stream)
{
    const long long dim = (long long)p.groups * p.n;
    p.row_splits = unsigned(norm_splits(rows, int(dim), kBwd));
    const int most = vec ? 64 * 8 * 4 : 64 * 16;
    const long long slots = (long long)p.row_splits * p.groups;
    if (p.n > most) {
        if (log_enabled())
            log_line("group_norm: norm_wg_kernel<in %s, out %s, run %d, bwd %d>, grid %lld x %d threads",
                     type_tag<T>(), type_tag<TOut>(), vec ? 8 : 1, int(kBwd), slots, kWgThreads);
        const dim3 grid{unsigned(slots)}, block(kWgThreads);
        if (vec) norm_wg_kernel<T, 8, kBwd, TOut><<<grid, block, 0, stream>>>(p);
        else norm_wg_kernel<T, 1, kBwd, TOut><<<grid, block, 0, stream>>>(p);
        return hipGetLastError();
    }
    const int run = vec ? 8 : 1;
    const int runs = (p.n + run - 1) / run;
    int ch = vec ? 1 : 4;  // runs of a lane
    while (ch * 64 < runs) ch *= vec ? 2 : 4;
    p.lpg = 1;
    while (p.lpg * ch < runs) p.lpg *= 2;
    const int per_wg = kLaneThreads / p.lpg;
    const dim3 grid{unsigned((slots + per_wg - 1) / per_wg)}, block(kLaneThreads);
    if (log_enabled())
        log_line("group_norm: norm_lanes_kernel<in %s, out %s, run %d, runs %d, bwd %d>, %d lanes a group, "
                 "grid %u x %d threads", type_tag<T>(), type_tag<TOut>(), run, ch, int(kBwd), p.lpg, grid.x,
                 kLaneThreads);
    if (vec && ch == 1) norm_lanes_kernel<T, 8, 1, kBwd, TOut><<<grid, block, 0, stream>>>(p);
    else if (vec && ch == 2) norm_lanes_kernel<T, 8, 2, kBwd, TOut><<<grid, block, 0, stream>>>(p);
    else if (vec) norm_lanes_kernel<T, 8, 4, kBwd, TOut><<<grid, block, 0, stream>>>(p);
    else if (ch == 4) norm_lanes_kernel<T, 1, 4, kBwd, TOut><<<grid, block, 0, stream>>>(p);
    else norm_lanes_kernel<T, 1, 16, kBwd, TOut><<<grid, block, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool kBwd>
hipError_t dispatch_norm(const NormParams &p, bool in_bf16, bool out_bf16, bool vec, long long rows,
                         hipStream_t stream)
{
    if (in_bf16 && out_bf16) return launch_norm<bf16_t, bf16_t, kBwd>(p, vec, rows, stream);
    if (in_bf16) return launch_norm<bf16_t, float, kBwd>(p, vec, rows, stream);
    if (out_bf16) return launch_norm<float, bf16_t, kBwd>(p, vec, rows, stream);
    return launch_norm<float, float, kBwd>(p, vec, rows, stream);
}

using namespace check;

bool norm_sizes(int batch, int seqlen, int dim, int groups)
{
    return batch >= 1 && seqlen >= 1 && dim >= 1 && groups >= 1 && dim <= (1 << 24) && dim % groups == 0 &&
           (long long)batch * seqlen < (1ll << 31);
}

// Tensor i for the overlap check; the batch stride of one entry leads nowhere.
Steps norm_steps(const void *ptr, size_t span, size_t es, const NormParams &p, int i, int batch, int seqlen, int dim)
{
    return one_step({ptr, span * es, dim * es, (long long)(p.step[i] * es),
                     batch == 1 ? 0 : (long long)(p.batch[i] * es)}, seqlen);
}

// All of the call's tensors admit 16-byte accesses at every run of 8 channels.
bool norm_vec(const NormParams &p, const void *const *ptrs, const size_t *es, int count, int batch)
{
    if (p.n % 8) return false;
    for (int i = 0; i < count; ++i) {
        if (!ptrs[i]) continue;
        const long long per = 16 / (long long)es[i];
        if (misaligned(ptrs[i], 16) || (p.seqlen > 1 && p.step[i] % per) || (batch > 1 && p.batch[i] % per))
            return false;
    }
    return true;
}

int norm_act(unsigned flags, const void *z)
{
    return (flags & SSM_NORM_GATE_FIRST) ? kGateFirst : z ? kGate : (flags & SSM_NORM_SILU) ? kSilu : kPlain;
}

bool norm_flags_ok(unsigned flags, const void *z)
{
    if (flags & ~(SSM_NORM_RMS | SSM_NORM_SILU | SSM_NORM_GATE_FIRST)) return false;
    if ((flags & SSM_NORM_SILU) && (z || (flags & SSM_NORM_GATE_FIRST))) return false;
    return true;
}

}  // namespace
}  // namespace ssm

extern "C" {

ssm_status_t ssm_group_norm_fwd(int batch, int seqlen, int dim, int groups, ssm_dtype_t in_dtype,
                                unsigned flags, const float *eps, const void *x, const float *weight,
                                const float *bias, const void *z, ssm_dtype_t out_dtype, void *y,
                                const ssm_norm_layout_t *layout, void *stream)
{
    using namespace ssm;
    using namespace ssm::check;
    const int in_t = enum_bits(in_dtype), out_t = enum_bits(out_dtype);
    if (!x || !y || ((flags & SSM_NORM_GATE_FIRST) && !z)) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(out_t)) return SSM_ERR_BAD_DTYPE;
    if (!norm_sizes(batch, seqlen, dim, groups)) return SSM_ERR_BAD_SHAPE;
    if (!norm_flags_ok(flags, z)) return SSM_ERR_UNSUPPORTED;
    const ssm_norm_layout_t dense{};
    const ssm_norm_layout_t &lay = layout ? *layout : dense;
    NormParams p{};
    size_t sp[3];
    const int at[3] = {0, 1, 3};
    for (int i = 0; i < 3; ++i)
        if (!row_strides(lay.step[i], lay.batch[i], batch, seqlen, dim, p.step[at[i]], p.batch[at[i]], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), os = dsize(out_t);
    if (misaligned(x, es) || misaligned(z, es) || misaligned(y, os) || misaligned(weight, 4) ||
        misaligned(bias, 4))
        return SSM_ERR_MISALIGNED;
    const size_t ybytes = sp[2] * os;
    // y in place of x or z: every element is read before it is written, by the same thread
    for (int i = 0; i < 2; ++i) {
        const void *in = i ? z : x;
        const bool same = in == y && in_t == out_t && (seqlen == 1 || p.step[i] == p.step[3]) &&
                          (batch == 1 || p.batch[i] == p.batch[3]);
        if (!same && overlaps(norm_steps(in, sp[i], es, p, i, batch, seqlen, dim),
                              norm_steps(y, sp[2], os, p, 3, batch, seqlen, dim)))
            return SSM_ERR_ALIAS;
    }
    if (overlaps(y, ybytes, weight, 4 * size_t(dim)) || overlaps(y, ybytes, bias, 4 * size_t(dim)))
        return SSM_ERR_ALIAS;
    p.seqlen = seqlen;
    p.groups = groups;
    p.n = dim / groups;
    p.rows = unsigned(batch) * unsigned(seqlen);
    p.act = norm_act(flags, z);
    p.rms = (flags & SSM_NORM_RMS) != 0;
    p.eps = eps ? *eps : 1e-5f;
    p.inv_n = 1.0f / float(p.n);
    p.x = x;
    p.z = z;
    p.weight = weight;
    p.bias = bias;
    p.out0 = y;
    const void *ptrs[4] = {x, z, nullptr, y};
    const size_t sizes[4] = {es, es, 0, os};
    const bool vec = norm_vec(p, ptrs, sizes, 4, batch);
    const hipError_t e = dispatch_norm<false>(p, in_t == SSM_BF16, out_t == SSM_BF16, vec, p.rows,
                                              static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_group_norm_bwd_workspace_bytes(int batch, int seqlen, int dim, int groups)
{
    if (!ssm::norm_sizes(batch, seqlen, dim, groups)) return 0;
    return 2 * sizeof(float) * size_t(dim) * size_t(ssm::norm_splits((long long)batch * seqlen, dim, true));
}

ssm_status_t ssm_group_norm_bwd(int batch, int seqlen, int dim, int groups, ssm_dtype_t in_dtype,
                                unsigned flags, const float *eps, const void *x, const float *weight,
                                const float *bias, const void *z, ssm_dtype_t grad_dtype,
                                const void *dy, void *dx, void *dz, float *dweight, float *dbias,
                                void *workspace, size_t workspace_bytes,
                                const ssm_norm_bwd_layout_t *layout, void *stream)
{
    using namespace ssm;
    using namespace ssm::check;
    const int in_t = enum_bits(in_dtype), g_t = enum_bits(grad_dtype);
    if (!x || !dy || !dx || (z && !dz) || ((flags & SSM_NORM_GATE_FIRST) && !z)) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(g_t)) return SSM_ERR_BAD_DTYPE;
    if (!norm_sizes(batch, seqlen, dim, groups)) return SSM_ERR_BAD_SHAPE;
    if (!norm_flags_ok(flags, z) || (!z && dz)) return SSM_ERR_UNSUPPORTED;
    const ssm_norm_bwd_layout_t dense{};
    const ssm_norm_bwd_layout_t &lay = layout ? *layout : dense;
    NormParams p{};
    size_t sp[5];
    for (int i = 0; i < 5; ++i)
        if (!row_strides(lay.step[i], lay.batch[i], batch, seqlen, dim, p.step[i], p.batch[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), gs = dsize(g_t), wb = 4 * size_t(dim);
    const void *ptrs[5] = {x, z, dy, dx, dz};
    const size_t sizes[5] = {es, es, gs, gs, gs};
    for (int i = 0; i < 5; ++i)
        if (misaligned(ptrs[i], sizes[i])) return SSM_ERR_MISALIGNED;
    const bool sums = dweight || dbias;
    const size_t need = ssm_group_norm_bwd_workspace_bytes(batch, seqlen, dim, groups);
    if (misaligned(weight, 4) || misaligned(bias, 4) || misaligned(dweight, 4) || misaligned(dbias, 4) ||
        (sums && misaligned(workspace, 16)))
        return SSM_ERR_MISALIGNED;
    if (sums && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
    Steps t[5];
    for (int i = 0; i < 5; ++i)
        t[i] = norm_steps(ptrs[i], sp[i], sizes[i], p, i, batch, seqlen, dim);
    auto range = [](const void *ptr, size_t bytes) { return Steps{ptr, bytes, bytes, 0, 0}; };
    const Steps in[] = {t[0], t[1], t[2], range(weight, wb), range(bias, wb)};
    const Steps out[] = {t[3], t[4], range(dweight, wb), range(dbias, wb), range(sums ? workspace : nullptr, need)};
    for (const Steps &o : out) {
        for (const Steps &i : in)
            if (overlaps(o, i)) return SSM_ERR_ALIAS;
        for (const Steps &i : out)
            if (&i != &o && overlaps(o, i)) return SSM_ERR_ALIAS;
    }
    p.seqlen = seqlen;
    p.groups = groups;
    p.n = dim / groups;
    p.rows = unsigned(batch) * unsigned(seqlen);
    p.act = norm_act(flags, z);
    p.rms = (flags & SSM_NORM_RMS) != 0;
    p.eps = eps ? *eps : 1e-5f;
    p.inv_n = 1.0f / float(p.n);
    p.x = x;
    p.z = z;
    p.dy = dy;
    p.weight = weight;
    p.bias = bias;
    p.out0 = dx;
    p.out1 = dz;
    const int splits = norm_splits(p.rows, dim, true);
    float *ws = static_cast<float *>(workspace);
    p.pw = dweight ? ws : nullptr;
    p.pb = dbias ? ws + size_t(splits) * dim : nullptr;
    const bool vec = norm_vec(p, ptrs, sizes, 5, batch);
    hipError_t e = dispatch_norm<true>(p, in_t == SSM_BF16, g_t == SSM_BF16, vec, p.rows,
                                       static_cast<hipStream_t>(stream));
    if (e == hipSuccess && sums) {
        norm_sums_kernel<<<dim3((dim + 63) / 64, 2), dim3(1024), 0, static_cast<hipStream_t>(stream)>>>(
            p.pw, p.pb, splits, dim, dweight, dbias);
        e = hipGetLastError();
    }
    return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
