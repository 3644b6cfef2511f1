// heads_grad.hip -- gradients of the selective scan with one decay a head
// (gfx950; C ABI in include/ssm_heads.h).
//
// The forward recurrence leaves the state S0 entering every chunk, the reverse
// one (heads_scan.hip) dx and the gradient dS1 of the state leaving it.  What
// is left has no order in time: one workgroup a chunk, group and part of the
// group's heads.  With M_ij = C_i . B_j, made once for the heads, and per head
// f_ij = e^{G_i - G_j} (j <= i), t_j = e^{Gc - G_j}, dW_ij = dy_i . x_j:
//     Q    += dW f D_j                          (D_j: the step size)
//     dC_i += e^{G_i} S0 dy_i,  dB_j += D_j t_j dS1 x_j
// and at the end dC += Q B, dB += Q^T C.  For the step sizes, with
//     F_i = e^{G_i} C_i . S0 dy_i,  E_j = t_j B_j . dS1 x_j,
//     R_ij = dW f M,  dD_j = sum_i R_ij + E_j       (all without D_j)
//     dG_i = sum_{j<i} R_ij D_j + F_i - D_i (dD_i - R_ii)
//     da_t = sum_{i >= t} dG_i + sum_j D_j E_j + e^{Gc} <S0, dS1>
//     ddt  = (dD + A da) sigmoid(dt + dt_bias),  dA = sum D da
// and dDskip is the sum of dW's diagonal.  (R's diagonal does not depend on G:
// left in both sums of dG it would cancel up to roundings, which are all that is
// left of dA where the decays are strong.)
#include "heads_common.hpp"

namespace ssm {
namespace heads {
namespace {

struct GradParams {
    int seqlen, nseq, rep, groups, h, N, P, parts, each;
    int in_bf16, g_bf16;
    long long records;
    const int *cu;
    const void *x, *dt, *B, *C, *dy;
    const float *A, *bias;
    void *ddt, *dB, *dC;
    float *dA, *dD, *dbias;
    DeltaStride sx, sdt, sB, sC, sdy, sddt, sdB, sdC;
    HeadsWs ws;
};

// A head's decays: G as two floats, the step size, e^G, e^{Gc - G}.
struct HeadVec {
    float hi[64], lo[64], dt[64], up[64], tail[64];
};

// The sums of 16 lanes' 16 values, value i to lane i of the 16: every step
// halves the values a lane still holds (15 moves for 16 sums).
template <int N> __device__ inline void fold16(float *v, int r)
{
    if constexpr (N > 1) {
        const bool high = (r & (N / 2)) != 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float mine = high ? v[i + N / 2] : v[i], theirs = high ? v[i] : v[i + N / 2];
            v[i] = mine + __shfl_xor(theirs, N / 2);
        }
        fold16<N / 2>(v, r);
    }
}

template <typename T, int ND, bool kFast>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 && ND <= 128 ? 2 : 1)) void heads_grad_kernel(const GradParams p)
{
    constexpr int NCH = ND / 8, KB = ND / 32, kTile = 64 * ND, NT = ND / 64;
    constexpr int PB = sizeof(T) == 4 && ND == 256 ? 32 : 64, PCH = PB / 8;  // columns of P at a time
    // S0 and dS1 as operands: three terms, since the fp32 sums dA and ddt_bias
    // are differences of what they form; Q: two, under the rounding of dB and dC
    constexpr int NR = 3, NQ = 2;
    constexpr int kFrag = 512 * (sizeof(T) == 2 ? NQ : 1);
    __shared__ __align__(16) E<T> tB[kTile];
    __shared__ __align__(16) E<T> tC[kTile];
    __shared__ __align__(16) E<T> tXY[2 * 64 * PB];
    static_assert(2 * 64 * PB >= 8 * kFrag, "Q's fragments take the place of x and dy");
    __shared__ __align__(16) HeadVec vecs[2 * kWaves];
    __shared__ float rows_[2][kWaves][64], ends_[2][kWaves][64], cols_[2][64], diag_[2][64], diagR_[2][64],
        dots_[2][kWaves];

    const int l = int(threadIdx.x) & 63, wave = wave_of(), r = l & 15, g = l >> 4;
    const int record = int(blockIdx.x), group = int(blockIdx.y), part = int(blockIdx.z);
    const int h0 = group * p.rep + part * p.each, nh = min(p.rep - part * p.each, p.each);
    const int si = delta_seq_of(p.cu, p.nseq, p.seqlen, record);
    const DeltaSeq seq = delta_seq(p.cu, si, p.seqlen);
    const int c = record - seq.chunk0, left = seq.len - c * kDeltaChunk;
    auto sum_at = [&](int which, int head) { return (which * (long long)p.h + head) * p.records + record; };
    if (left <= 0) {  // no such chunk
        for (int k = int(threadIdx.x); k < nh; k += kThreads)
            for (int i = 0; i < 3; ++i) p.ws.sums[sum_at(i, h0 + k)] = 0.0f;
        return;
    }
    const int rows = min(left, kDeltaChunk);
    const long long t0 = seq.first + (long long)c * kDeltaChunk;
    const int ein = p.in_bf16 ? 2 : 4, eg = p.g_bf16 ? 2 : 4;
    auto in_at = [&](const void *q, const DeltaStride &s, int head, int es) {
        return static_cast<const char *>(q) + (seq.batch * s.b + t0 * s.t + head * s.h) * es;
    };

    {
        TileIn<T, NCH, kFast> inB, inC;
        inB.init(p.sB.t, p.N);
        inC.init(p.sC.t, p.N);
        inB.fetch(in_at(p.B, p.sB, group, ein), p.sB.t, rows);
        inC.fetch(in_at(p.C, p.sC, group, ein), p.sC.t, rows);
        inB.store(tB, in_at(p.B, p.sB, group, ein), p.sB.t, rows, p.N, p.in_bf16);
        inC.store(tC, in_at(p.C, p.sC, group, ein), p.sC.t, rows, p.N, p.in_bf16);
    }
    TileIn<T, PCH, kFast> inX, inY;
    const int blocks = (p.P + PB - 1) / PB;
    auto x_at = [&](int k, int pb) { return in_at(p.x, p.sx, h0 + k, ein) + (long long)pb * PB * ein; };
    auto y_at = [&](int k, int pb) { return in_at(p.dy, p.sdy, h0 + k, eg) + (long long)pb * PB * eg; };
    auto fetch = [&](int k, int pb) {
        inX.init(p.sx.t, p.P - pb * PB);
        inY.init(p.sdy.t, p.P - pb * PB);
        inX.fetch(x_at(k, pb), p.sx.t, rows);
        inY.fetch(y_at(k, pb), p.sdy.t, rows);
    };
    fetch(0, 0);
    __syncthreads();

    // M's column tile of this wave: rows 16 m + 4 g + e, column 16 wave + r
    f32x4 M[4], Q[4], dC[NT][4], dB[NT][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        M[m] = Q[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < NT; ++t) dC[t][m] = dB[t][m] = f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
        In<T> fc[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) fc[m] = tile_row<T, NCH>(tC, 16 * m + r, 4 * b + g);
        mma_left<4>(M, fc, tile_row<T, NCH>(tB, 16 * wave + r, 4 * b + g));
    }

    // Head k's step sizes, once its sums are there (one wave, lane = step).
    auto finish = [&](int k) {
        const int head = h0 + k, q = k & 1;
        const HeadVec &v = vecs[k & (2 * kWaves - 1)];
        float row = 0.0f, E0 = 0.0f, dot = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            row += rows_[q][w][l];
            E0 += ends_[q][w][l];
            dot += dots_[q][w];
        }
        const float dt = v.dt[l], later = cols_[q][l] + E0, dD = later + diagR_[q][l], A = p.A[head];
        const float end = v.up[63];
        // the sums run in double: neighbours cancel
        double da = double(row) - double(dt) * later, own = double(dt) * E0;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const double after = __shfl_down(da, o);
            if (l + o < 64) da += after;
            own += __shfl_xor(own, o);
        }
        da += own + double(end) * dot;
        const float u = load_step(in_at(p.dt, p.sdt, head, ein), min(l, rows - 1) * p.sdt.t, p.in_bf16) +
                        (p.bias ? p.bias[head] : 0.0f);
        const float ddt = l < rows ? (dD + A * float(da)) * (1.0f / (1.0f + exp2_hw(-u * kLog2e))) : 0.0f;
        if (l < rows) {
            const long long at = seq.batch * p.sddt.b + (t0 + l) * p.sddt.t + head * p.sddt.h;
            if (p.g_bf16) static_cast<bf16_t *>(p.ddt)[at].bits = uint16_t(pack_bf16x2(ddt, ddt));
            else static_cast<float *>(p.ddt)[at] = ddt;
        }
        double s[3] = {double(dt) * da, l < rows ? double(diag_[q][l]) : 0.0, double(ddt)};
#pragma unroll
        for (int o = 1; o < 64; o *= 2)
#pragma unroll
            for (int i = 0; i < 3; ++i) s[i] += __shfl_xor(s[i], o);
        if (l == 0)
            for (int i = 0; i < 3; ++i) p.ws.sums[sum_at(i, head)] = float(s[i]);
    };

    for (int k = 0; k < nh; ++k) {
        const int head = h0 + k;
        // four heads' decays at a time, a wave each
        if ((k & (kWaves - 1)) == 0 && k + wave < nh) {
            const int mine = head + wave;
            const float raw = load_step(in_at(p.dt, p.sdt, mine, ein), min(l, rows - 1) * p.sdt.t, p.in_bf16);
            const Decays d = decays(raw, p.bias ? p.bias[mine] : 0.0f, p.A[mine], rows);
            HeadVec &v = vecs[(k + wave) & (2 * kWaves - 1)];
            v.hi[l] = float(d.G);
            v.lo[l] = float(d.G - double(float(d.G)));
            v.dt[l] = d.dt;
            v.up[l] = exp2_of(d.G);
            v.tail[l] = exp2_of(d.end - d.G);
        }
        const HeadVec &v = vecs[k & (2 * kWaves - 1)];
        const long long rec = ((long long)record * p.h + head) * p.ws.state;
        const int bytes = int(p.ws.state) * 4;
        const auto bufS = buffer_of(p.ws.S0 + rec, bytes), bufD = buffer_of(p.ws.dS1 + rec, bytes);
        f32x4 dW[4];
        float row[16], end[16], dot = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) dW[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) row[i] = end[i] = 0.0f;
        for (int pb = 0; pb < blocks; ++pb) {
            __syncthreads();  // the last tiles' reads are done
            E<T> *const tX = tXY, *const tY = tXY + 64 * PB;
            inX.store(tX, x_at(k, pb), p.sx.t, rows, p.P - pb * PB, p.in_bf16);
            inY.store(tY, y_at(k, pb), p.sdy.t, rows, p.P - pb * PB, p.g_bf16);
            __syncthreads();
            if (pb + 1 < blocks) fetch(k, pb + 1);
            else if (k + 1 < nh) fetch(k + 1, 0);
            if (pb == 0 && k > 0 && wave == ((k - 1) & (kWaves - 1))) finish(k - 1);
            In<T> fx[PB / 32][4], fy[PB / 32][4];
#pragma unroll
            for (int b = 0; b < PB / 32; ++b) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    fx[b][m] = tile_row<T, PCH>(tX, 16 * m + r, 4 * b + g);
                    fy[b][m] = tile_row<T, PCH>(tY, 16 * m + r, 4 * b + g);
                }
                mma_left<4>(dW, fy[b], tile_row<T, PCH>(tX, 16 * wave + r, 4 * b + g));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int n = 16 * (NT * wave + t) + r;
                f32x4 Sy[4], Dx[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) Sy[m] = Dx[m] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < PB / 32; ++b) {
                    const int col = pb * PB + 32 * b + 8 * g;
                    // rows behind the record and columns behind Pp read as 0
                    const uint32_t off = col < p.ws.Pp ? uint32_t(n * p.ws.Pp + col) * 4u : kOutside;
                    f32x4 s[2], d[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        s[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(bufS, off + 16 * i, 0, 0));
                        d[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(bufD, off + 16 * i, 0, 0));
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(s[i][e], d[i][e], dot);
                    mma_left<4>(Sy, fy[b], to_sum<T, NR>(s[0], s[1]));
                    mma_left<4>(Dx, fx[b], to_sum<T, NR>(d[0], d[1]));
                }
                // rows 16 m + 4 g + e, column n
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const f32x4 up = *reinterpret_cast<const f32x4 *>(v.up + 16 * m + 4 * g);
                    const f32x4 tail = *reinterpret_cast<const f32x4 *>(v.tail + 16 * m + 4 * g);
                    const f32x4 dts = *reinterpret_cast<const f32x4 *>(v.dt + 16 * m + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 16 * m + 4 * g + e, at = chunk_at<NCH>(i, n >> 3) + (n & 7);
                        float Cn, Bn;
                        if constexpr (sizeof(T) == 4) {
                            Cn = tC[at];
                            Bn = tB[at];
                        } else {
                            Cn = __uint_as_float(uint32_t(tC[at]) << 16);
                            Bn = __uint_as_float(uint32_t(tB[at]) << 16);
                        }
                        const float a = up[e] * Sy[m][e], b = tail[e] * Dx[m][e];
                        dC[t][m][e] += a;
                        row[4 * m + e] = __builtin_fmaf(Cn, a, row[4 * m + e]);
                        dB[t][m][e] = __builtin_fmaf(dts[e], b, dB[t][m][e]);
                        end[4 * m + e] = __builtin_fmaf(Bn, b, end[4 * m + e]);
                    }
                }
            }
        }
        // dW: rows i = 16 m + 4 g + e, column j = 16 wave + r
        const int j = 16 * wave + r, q = k & 1;
        const float jhi = v.hi[j], jlo = v.lo[j], jdt = v.dt[j];
        float col = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(v.hi + 16 * m + 4 * g);
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(v.lo + 16 * m + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * m + 4 * g + e;
                const float f = exp2_hw((hi[e] - jhi) + (lo[e] - jlo));
                const float w = j <= i ? dW[m][e] * f : 0.0f;
                Q[m][e] = __builtin_fmaf(w, jdt, Q[m][e]);
                const float R = j < i ? w * M[m][e] : 0.0f;
                col += R;
                row[4 * m + e] = __builtin_fmaf(R, jdt, row[4 * m + e]);
                if (i == j) {
                    diag_[q][j] = dW[m][e];
                    diagR_[q][j] = w * M[m][e];
                }
            }
        }
        col += __shfl_xor(col, 16);
        col += __shfl_xor(col, 32);
        if (g == 0) cols_[q][j] = col;
        // over the 16 lanes of a row group: value 4 m + e to lane 4 m + e
        fold16<16>(row, r);
        fold16<16>(end, r);
        rows_[q][wave][16 * (r >> 2) + 4 * g + (r & 3)] = row[0];
        ends_[q][wave][16 * (r >> 2) + 4 * g + (r & 3)] = end[0];
#pragma unroll
        for (int o = 1; o < 64; o *= 2) dot += __shfl_xor(dot, o);
        if (l == 0) dots_[q][wave] = dot;
    }
    __syncthreads();
    if (wave == ((nh - 1) & (kWaves - 1))) finish(nh - 1);

    // dB += Q^T C, dC += Q B: Q's fragments through LDS, as rows j and as rows i
    auto read_frags = [&](int b, Sum<T, NQ> *f) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const E<T> *at = tXY + (2 * m + b) * kFrag;
            if constexpr (sizeof(T) == 4) {
                const f32x4 *s = reinterpret_cast<const f32x4 *>(at + l * 8);
                f[m] = F32x8{s[0], s[1]};
            } else {
#pragma unroll
                for (int i = 0; i < NQ; ++i) f[m].t[i] = *reinterpret_cast<const bf16x8 *>(at + (i * 64 + l) * 8);
            }
        }
    };
    auto product = [&](f32x4 (*to)[4], const E<T> *tile) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            Sum<T, NQ> f[4];
            read_frags(b, f);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                mma_left<4>(to[t], f, tile_cols<T, NCH>(tile, 32 * b + 4 * g, 32 * b + 16 + 4 * g,
                                                        [&](int s) { return 16 * (NT * wave + t) + 4 * s; }));
        }
    };
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const Sum<T, NQ> f = to_sum<T, NQ>(Q[2 * b], Q[2 * b + 1]);
        E<T> *at = tXY + (2 * wave + b) * kFrag;
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<f32x4 *>(at + l * 8)[0] = f.lo;
            reinterpret_cast<f32x4 *>(at + l * 8)[1] = f.hi;
        } else {
#pragma unroll
            for (int i = 0; i < NQ; ++i) *reinterpret_cast<bf16x8 *>(at + (i * 64 + l) * 8) = f.t[i];
        }
    }
    __syncthreads();
    product(dB, tC);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // row i = 16 m + 4 g + e, column j = 16 wave + r of the block wave / 2
            const int lane = (r >> 2) * 16 + 4 * g + e, at = 4 * (wave & 1) + (r & 3);
            E<T> *to = tXY + (2 * m + (wave >> 1)) * kFrag + lane * 8 + at;
            if constexpr (sizeof(T) == 4) {
                *to = Q[m][e];
            } else {
                float v = Q[m][e], none = 0.0f;
#pragma unroll
                for (int i = 0; i < NQ; ++i) to[i * 512] = uint16_t(split_pair(v, none));
            }
        }
    __syncthreads();
    product(dC, tB);

    if (p.parts > 1) {
        const long long at = (((long long)part * p.records + record) * p.groups + group) * 64 * p.ws.Nr;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int n = 16 * (NT * wave + t) + r;
            store_column<float, false>(p.ws.dBp + at, p.ws.Nr, rows, g, n, n < p.ws.Nr, dB[t]);
            store_column<float, false>(p.ws.dCp + at, p.ws.Nr, rows, g, n, n < p.ws.Nr, dC[t]);
        }
    } else {
        const long long bAt = seq.batch * p.sdB.b + t0 * p.sdB.t + group * p.sdB.h;
        const long long cAt = seq.batch * p.sdC.b + t0 * p.sdC.t + group * p.sdC.h;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int n = 16 * (NT * wave + t) + r;
            if (p.g_bf16) {
                store_column<bf16_t, false>(static_cast<bf16_t *>(p.dB) + bAt, p.sdB.t, rows, g, n, n < p.N, dB[t]);
                store_column<bf16_t, false>(static_cast<bf16_t *>(p.dC) + cAt, p.sdC.t, rows, g, n, n < p.N, dC[t]);
            } else {
                store_column<float, false>(static_cast<float *>(p.dB) + bAt, p.sdB.t, rows, g, n, n < p.N, dB[t]);
                store_column<float, false>(static_cast<float *>(p.dC) + cAt, p.sdC.t, rows, g, n, n < p.N, dC[t]);
            }
        }
    }
}

// dB (blockIdx.z 0) and dC: the parts' sums, in order.
__global__ __launch_bounds__(kThreads) void heads_parts_kernel(const GradParams p)
{
    const int record = int(blockIdx.x), group = int(blockIdx.y);
    const DeltaSeq seq = delta_seq(p.cu, delta_seq_of(p.cu, p.nseq, p.seqlen, record), p.seqlen);
    const int c = record - seq.chunk0, left = seq.len - c * kDeltaChunk;
    if (left <= 0) return;
    const bool isC = blockIdx.z != 0;
    const DeltaStride &s = isC ? p.sdC : p.sdB;
    const float *src = (isC ? p.ws.dCp : p.ws.dBp) + ((long long)record * p.groups + group) * 64 * p.ws.Nr;
    const long long part = p.records * p.groups * 64 * p.ws.Nr;
    const long long to = seq.batch * s.b + (seq.first + (long long)c * kDeltaChunk) * s.t + group * s.h;
    void *const dst = isC ? p.dC : p.dB;
    const int quads = p.ws.Nr / 4;
    for (int i = int(threadIdx.x); i < min(left, kDeltaChunk) * quads; i += kThreads) {
        const int row = i / quads, n = i % quads * 4;
        f32x4 v = *reinterpret_cast<const f32x4 *>(src + row * p.ws.Nr + n);
        for (int k = 1; k < p.parts; ++k) v += *reinterpret_cast<const f32x4 *>(src + k * part + row * p.ws.Nr + n);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < p.N) {
                const long long at = to + row * s.t + n + e;
                if (p.g_bf16) static_cast<bf16_t *>(dst)[at].bits = uint16_t(pack_bf16x2(v[e], v[e]));
                else static_cast<float *>(dst)[at] = v[e];
            }
    }
}

// dA, dDskip, ddt_bias of one head: the chunks' sums, in a fixed order.
__global__ __launch_bounds__(kThreads) void heads_sums_kernel(const GradParams p)
{
    __shared__ double part[kWaves];
    float *const to = blockIdx.y == 0 ? p.dA : blockIdx.y == 1 ? p.dD : p.dbias;
    if (!to) return;  // the whole workgroup
    const float *src = p.ws.sums + ((long long)blockIdx.y * p.h + blockIdx.x) * p.records;
    double s = 0.0;
    for (long long i = threadIdx.x; i < p.records; i += kThreads) s += src[i];
#pragma unroll
    for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) to[blockIdx.x] = float((part[0] + part[1]) + (part[2] + part[3]));
}

template <typename T, int ND, bool kFast> hipError_t grad_run(const GradParams &p, hipStream_t stream)
{
    const dim3 grid(unsigned(p.records), p.groups, p.parts), block(kThreads);
    if (log_enabled())
        log_line("head_scan_bwd: heads_grad_kernel<%s, N %d, fast %d>, grid (%u, %u, %u) x %u threads, %d heads a part",
                 type_tag<T>(), ND, int(kFast), grid.x, grid.y, grid.z, block.x, p.each);
    heads_grad_kernel<T, ND, kFast><<<grid, block, 0, stream>>>(p);
    if (p.parts > 1) heads_parts_kernel<<<dim3(grid.x, grid.y, 2), block, 0, stream>>>(p);
    heads_sums_kernel<<<dim3(p.h, 3), block, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t grad_typed(const GradParams &p, bool fast, hipStream_t stream)
{
    const int nd = heads_nd(p.N);
    if (nd == 64) return fast ? grad_run<T, 64, true>(p, stream) : grad_run<T, 64, false>(p, stream);
    if (nd == 128) return fast ? grad_run<T, 128, true>(p, stream) : grad_run<T, 128, false>(p, stream);
    return fast ? grad_run<T, 256, true>(p, stream) : grad_run<T, 256, false>(p, stream);
}

}  // namespace
}  // namespace heads

size_t heads_bwd_workspace_bytes(int batch, int seqlen, int groups, int h, int N, int P, int num_seqs)
{
    size_t bytes = 0;
    heads::heads_ws(nullptr, batch, seqlen, groups, h, N, P, num_seqs, true, &bytes);
    return bytes;
}

hipError_t launch_heads_bwd(const HeadsBwdArgs &b, hipStream_t stream)
{
    using namespace heads;
    const HeadsArgs &a = b.f;
    const HeadsWs ws = heads_ws(a, true);
    hipError_t e = hipSuccess;
    if (!b.ckpt_given) {  // the states alone
        HeadsScan p{a.seqlen, a.nseq, a.h / a.groups, a.h, a.N, a.P, a.in_bf16, a.in_bf16, 0, a.cu, a.C, a.B, a.x, a.dt,
                    a.A, a.dt_bias, nullptr, a.h0, nullptr, nullptr, ws.S0, a.sC, a.sB, a.sx, a.sdt, {}, ws};
        e = launch_heads_scan(a, p, false, stream);
        if (e != hipSuccess) return e;
    }
    HeadsScan r{a.seqlen, a.nseq, a.h / a.groups, a.h, a.N, a.P, a.in_bf16, b.grad_bf16, b.grad_bf16, a.cu, a.B, a.C,
                b.dy, a.dt, a.A, a.dt_bias, a.Dskip, b.dhL, b.dh0, b.dx, ws.dS1, a.sB, a.sC, b.sdy, a.sdt, b.sdx, ws};
    e = launch_heads_scan(a, r, true, stream);
    if (e != hipSuccess) return e;
    const int rep = a.h / a.groups;
    const long long records = delta_chunks(a.batch, a.seqlen, a.cu ? a.nseq : 0);
    const GradParams p{a.seqlen, a.nseq, rep, a.groups, a.h, a.N, a.P, ws.parts, (rep + ws.parts - 1) / ws.parts,
                       a.in_bf16, b.grad_bf16, records, a.cu, a.x, a.dt, a.B, a.C, b.dy, a.A, a.dt_bias, b.ddt, b.dB,
                       b.dC, b.dA, b.dDskip, b.ddt_bias, a.sx, a.sdt, a.sB, a.sC, b.sdy, b.sddt, b.sdB, b.sdC, ws};
    const int es = a.in_bf16 ? 2 : 4;
    const bool fast = a.in_bf16 == b.grad_bf16 && heads_fast(a.B, a.sB, a.N, es, a, a.groups) &&
                      heads_fast(a.C, a.sC, a.N, es, a, a.groups) && heads_fast(a.x, a.sx, a.P, es, a, a.h) &&
                      heads_fast(b.dy, b.sdy, a.P, es, a, a.h);
    return a.in_bf16 && b.grad_bf16 ? grad_typed<bf16_t>(p, fast, stream) : grad_typed<float>(p, fast, stream);
}

}  // namespace ssm
