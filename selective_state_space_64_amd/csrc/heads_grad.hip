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
//
// What bounds it (4 x 2048 steps, 80 heads of 128 x 64 with one group, bf16): the states.  They
// are 671 MB of the 860 MB read, 165 us at a large copy's rate; the kernel takes 284,
// one workgroup of eight waves on every compute unit (the registers hold no second one),
// and the two runs that write them 209 and 217 (all under the profiler) where a forward
// call without them takes 126.  The whole training step takes 673 us (parts and sums 14),
// where its inputs and outputs, 457 MB, take 88; with fp32 tensors 1.56 ms, with fp32
// gradients of bf16 inputs 2.07 ms, with 256 state rows (203 registers of bf16 kernels and
// 139 of fp32 ones spilled here) 2.37 ms in bf16 and 7.28 in fp32.
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

template <int kCtrl> __device__ inline float from_dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true));
}
// The sums of 16 lanes' 16 values, value i to lane i of the 16.  Every step halves
// the values that a lane still holds (15 moves for 16 sums) and trades the others with
// the lane whose number differs in the bit that tells them apart, and in those below
// it: the mirrors of 16, 8, 4 and 2 lanes.
template <int kCtrl, int N> __device__ inline void fold_step(float *v, bool high)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float mine = high ? v[i + N] : v[i], theirs = high ? v[i] : v[i + N];
        v[i] = mine + from_dpp<kCtrl>(theirs);
    }
}
__device__ inline float fold16(float *v, int r)
{
    fold_step<0x140, 8>(v, r & 8);  // row_mirror
    fold_step<0x141, 4>(v, r & 4);  // row_half_mirror
    fold_step<0x1B, 2>(v, r & 2);   // quad_perm 3,2,1,0
    fold_step<0xB1, 1>(v, r & 1);   // quad_perm 1,0,3,2
    return v[0];
}
// 1 - e^-x for x >= 0: sigmoid(u) of x = softplus(u), to an ulp or two
__device__ inline float one_minus_exp(float x)
{
    // the series to x^8 where the difference would lose bits (the next term is below 2^-25)
    float q = 1.0f / 40320.0f;
    q = __builtin_fmaf(-x, q, 1.0f / 5040.0f);
    q = __builtin_fmaf(-x, q, 1.0f / 720.0f);
    q = __builtin_fmaf(-x, q, 1.0f / 120.0f);
    q = __builtin_fmaf(-x, q, 1.0f / 24.0f);
    q = __builtin_fmaf(-x, q, 1.0f / 6.0f);
    q = __builtin_fmaf(-x, q, 0.5f);
    q = __builtin_fmaf(-x, q, 1.0f);
    return x > 0.5f ? 1.0f - exp2_hw(-x * kLog2e) : x * q;
}

// Eight waves: each forms the scores of a column tile j of 16 steps and two row
// tiles i, and the columns n of dB and dC that are its own.  S0 and dS1 are read
// once, straight from memory to the lanes that need them as operands (8
// neighbouring columns of P of one n), a block of 64 columns ahead.
constexpr int kGradThreads = kHeadsGradThreads, kGradWaves = kGradThreads / 64;
static_assert(kGradWaves == 8, "the column tiles and halves below");

template <typename T, int ND, bool kFast>
__global__ __launch_bounds__(kGradThreads) void heads_grad_kernel(const GradParams p)
{
    constexpr int NCH = ND / 8, KB = ND / 32, kTile = 64 * ND;
    constexpr int NT = ND == 256 ? 2 : 1, MT = ND == 64 ? 2 : 4;  // tiles of n and of rows for a wave's dB, dC
    constexpr int PB = sizeof(T) == 4 && ND == 256 ? 32 : 64, PCH = PB / 8, NB = PB / 32;  // columns of P at a time
    // S0 and dS1 as operands: three terms, since the fp32 sums dA and ddt_bias
    // are differences of what they form; Q: two, under the rounding of dB and dC
    constexpr int NR = 3, NQ = 2;
    constexpr int kFrag = 512 * (sizeof(T) == 2 ? NQ : 1);
    constexpr int kAhead = sizeof(T) == 4 && ND == 256 ? 1 : 4;  // heads whose decays are formed at a time
    __shared__ __align__(16) E<T> tB[kTile];
    __shared__ __align__(16) E<T> tC[kTile];
    __shared__ __align__(16) E<T> tXY[2 * 64 * PB];
    static_assert(2 * 64 * PB >= 8 * kFrag, "Q's fragments take the place of x and dy");
    __shared__ __align__(16) HeadVec vecs[2 * kAhead];
    __shared__ float rows_[2][kGradWaves][16 * MT], ends_[2][kGradWaves][16 * MT], rowsR_[2][kGradWaves][32], cols_[2][2][64],
        diag_[2][64], diagR_[2][64], dots_[2][kGradWaves], rates[2 * kAhead];  // rates: the heads' A

    const int l = int(threadIdx.x) & 63, wave = wave_of(), r = l & 15, g = l >> 4;
    const int jt = wave & 3, ih = wave >> 2;  // the wave's column tile, and half of the row tiles, of the scores
    const int n0 = 16 * (MT == 2 ? jt : NT * wave), m0 = MT == 2 ? 2 * ih : 0;  // of dB and dC
    const int record = int(blockIdx.x), group = int(blockIdx.y), part = int(blockIdx.z);
    const int h0 = group * p.rep + part * p.each, nh = min(p.rep - part * p.each, p.each);
    const int si = delta_seq_of(p.cu, p.nseq, p.seqlen, record);
    const DeltaSeq seq = delta_seq(p.cu, si, p.seqlen);
    const int c = record - seq.chunk0, left = seq.len - c * kDeltaChunk;
    auto sum_at = [&](int which, int head) { return (which * (long long)p.h + head) * p.records + record; };
    if (c < 0 || left <= 0) {  // no such chunk: records in front of the first sequence, or behind one's last
        for (int k = int(threadIdx.x); k < nh; k += kGradThreads)
            for (int i = 0; i < 3; ++i) p.ws.sums[sum_at(i, h0 + k)] = 0.0f;
        return;
    }
    const int rows = min(left, kDeltaChunk);
    const long long t0 = seq.first + (long long)c * kDeltaChunk;
    const int ein = p.in_bf16 ? 2 : 4, eg = p.g_bf16 ? 2 : 4;
    auto in_at = [&](const void *q, const DeltaStride &s, int head, int es) {
        return static_cast<const char *>(q) + (seq.batch * s.b + t0 * s.t + head * s.h) * es;
    };

    // the steps of the loop: head k, block pb of its columns
    const int blocks = (p.P + PB - 1) / PB;
    TileIn<T, PCH, kFast, kGradThreads> inX, inY;
    auto x_at = [&](int k, int pb) { return in_at(p.x, p.sx, h0 + k, ein) + (long long)pb * PB * ein; };
    auto y_at = [&](int k, int pb) { return in_at(p.dy, p.sdy, h0 + k, eg) + (long long)pb * PB * eg; };
    auto fetch = [&](int k, int pb) {
        inX.init(p.sx.t, p.P - pb * PB);
        inY.init(p.sdy.t, p.P - pb * PB);
        inX.fetch(x_at(k, pb), p.sx.t, rows);
        inY.fetch(y_at(k, pb), p.sdy.t, rows);
    };
    f32x4 s0[NT][NB][2], d1[NT][NB][2];
    auto fetch_state = [&](const float *from, f32x4 (*to)[NB][2], int k, int pb) {
        const auto buf = buffer_of(from + ((long long)record * p.h + h0 + k) * p.ws.state, p.ws.state * 4);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // rows behind the record and columns behind Pp read as 0
                const int col = pb * PB + 32 * b + 8 * g;
                const uint32_t off = col < p.ws.Pp ? uint32_t((n0 + 16 * t + r) * p.ws.Pp + col) * 4u : kOutside;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    to[t][b][i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off + 16 * i, 0, 0));
            }
    };
    {
        TileIn<T, NCH, kFast, kGradThreads> inB, inC;
        inB.init(p.sB.t, p.N);
        inC.init(p.sC.t, p.N);
        inB.fetch(in_at(p.B, p.sB, group, ein), p.sB.t, rows);
        inC.fetch(in_at(p.C, p.sC, group, ein), p.sC.t, rows);
        fetch(0, 0);
        fetch_state(p.ws.S0, s0, 0, 0);
        fetch_state(p.ws.dS1, d1, 0, 0);
        inB.store(tB, in_at(p.B, p.sB, group, ein), p.sB.t, rows, p.N, p.in_bf16);
        inC.store(tC, in_at(p.C, p.sC, group, ein), p.sC.t, rows, p.N, p.in_bf16);
    }
    __syncthreads();

    // M's tiles of this wave: rows 16 (2 ih + m) + 4 g + e, column 16 jt + r
    f32x4 M[2], Q[2], dC[NT][MT], dB[NT][MT];
#pragma unroll
    for (int m = 0; m < 2; ++m) M[m] = Q[m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) dC[t][m] = dB[t][m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < KB; ++b) {
        const In<T> fc[2] = {tile_row<T, NCH>(tC, 32 * ih + r, 4 * b + g), tile_row<T, NCH>(tC, 32 * ih + 16 + r, 4 * b + g)};
        mma_left<2>(M, fc, tile_row<T, NCH>(tB, 16 * jt + r, 4 * b + g));
    }
    // an element of B or C in the place of a sum (held in registers they cost spills)
    auto value = [&](const E<T> *tile, int r, int g, int t, int m, int e) {
        const int n = n0 + 16 * t + r, at = chunk_at<NCH>(16 * (m0 + m) + 4 * g + e, n >> 3) + (n & 7);
        if constexpr (sizeof(T) == 4) return tile[at];
        else return io<bf16_t>::lo(tile[at]);
    };

    // Head k's step sizes, once its sums are there (one wave, lane = step).
    auto finish = [&](int k) {
        uint32_t lane = l;  // (its masks and addresses are not kept from before the loop)
        opaque(lane);
        const int l = int(lane);
        const int head = h0 + k, q = k & 1;
        const HeadVec &v = vecs[k & (2 * kAhead - 1)];
        float row = 0.0f, E0 = 0.0f, dot = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWaves; ++w) {
            // (MT = 2: waves 0 .. 3 have the first half of the steps)
            const bool has = MT == 4 || (w >> 2) == (l >> 5);
            row += has ? rows_[q][w][l & (16 * MT - 1)] : 0.0f;
            E0 += has ? ends_[q][w][l & (16 * MT - 1)] : 0.0f;
            row += (w >> 2) == (l >> 5) ? rowsR_[q][w][l & 31] : 0.0f;
            if (MT == 4 || w < 4) dot += dots_[q][w];  // (MT = 2: the others hold the same states)
        }
        const float dt = v.dt[l], later = cols_[q][0][l] + cols_[q][1][l] + E0, dD = later + diagR_[q][l], A = rates[k & (2 * kAhead - 1)];
        const float end = v.up[63];
        // the sums run in double: neighbours cancel
        const double dG = double(row) - double(dt) * later;
        const double upto = wave_prefix(dG), own = from_lane(wave_prefix(double(dt) * E0), 63);
        const double da = from_lane(upto, 63) - upto + dG + own + double(end) * dot;
        // sigmoid(dt + dt_bias)
        const float ddt = l < rows ? (dD + A * float(da)) * one_minus_exp(dt) : 0.0f;
        if (l < rows) {
            const long long at = seq.batch * p.sddt.b + (t0 + l) * p.sddt.t + head * p.sddt.h;
            if (p.g_bf16) static_cast<bf16_t *>(p.ddt)[at].bits = uint16_t(pack_bf16x2(ddt, ddt));
            else static_cast<float *>(p.ddt)[at] = ddt;
        }
        const double s[3] = {wave_prefix(double(dt) * da), wave_prefix(l < rows ? double(diag_[q][l]) : 0.0),
                             wave_prefix(double(ddt))};
        if (l == 63)
            for (int i = 0; i < 3; ++i) p.ws.sums[sum_at(i, head)] = float(s[i]);
    };

    f32x4 dW[2];
    float dot = 0.0f;
    int k = 0, pb = 0;
    // the raw steps of one of the next four heads, its A and dt_bias (loaded at every step: a
    // load in a branch would be waited for where the branch ends)
    RawStep raw;
    float rate, bias;
    const float *const biases = p.bias ? p.bias : p.A;
    auto load_raw = [&](int k) {
        uint32_t lane = l;
        opaque(lane);
        const int l = int(lane);
        const int head = h0 + min(k + (wave & (kAhead - 1)), nh - 1);
        raw.load(in_at(p.dt, p.sdt, head, ein), min(l, rows - 1) * p.sdt.t, p.in_bf16);
        rate = p.A[head];
        bias = biases[head];
    };
    load_raw(0);
    const int steps = nh * blocks;
    for (int step = 0; step < steps; ++step) {
        __syncthreads();  // the last tiles' reads are done, and the finishing wave's of its head's decays
        if (pb == 0) {
            // four heads' decays at a time, a wave each (behind the barrier: with kAhead = 1 and one
            // block of columns a head they take the place of those that finish() read last)
            if ((k & (kAhead - 1)) == 0 && wave < kAhead && k + wave < nh) {
                const Decays d = decays(raw.value(p.in_bf16), p.bias ? bias : 0.0f, rate, rows);
                if (l == 0) rates[(k + wave) & (2 * kAhead - 1)] = rate;
                HeadVec &v = vecs[(k + wave) & (2 * kAhead - 1)];
                v.hi[l] = float(d.G);
                v.lo[l] = float(d.G - double(float(d.G)));
                v.dt[l] = d.dt;
                v.up[l] = exp2_of(d.G);
                v.tail[l] = exp2_of(d.end - d.G);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) dW[m] = f32x4{0, 0, 0, 0};
            dot = 0.0f;
        }
        const HeadVec &v = vecs[k & (2 * kAhead - 1)];
        E<T> *const tX = tXY, *const tY = tXY + 64 * PB;
        inX.store(tX, x_at(k, pb), p.sx.t, rows, p.P - pb * PB, p.in_bf16);
        inY.store(tY, y_at(k, pb), p.sdy.t, rows, p.P - pb * PB, p.g_bf16);
        __syncthreads();
        const bool done = pb + 1 == blocks;  // of the head
        const int nk = done ? k + 1 : k, npb = done ? 0 : pb + 1;
        // (behind the last step the same again: a branch here would wait for the loads)
        const int fk = step + 1 < steps ? nk : k, fpb = step + 1 < steps ? npb : pb;
        load_raw(k + 1);
        fetch(fk, fpb);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(s0[t][b][i][e], d1[t][b][i][e], dot);
        if (pb == 0 && k > 0 && wave == ((k - 1) & (kGradWaves - 1))) finish(k - 1);
        // rows 16 (m0 + m) + 4 g + e, columns n: e^G S0 dy to dC and to row, t dS1 x to dB and to end
        // (the state as an operand first, and the next one's on its way in its place)
        auto side = [&](const E<T> *tile, f32x4 (*state)[NB][2], const float *from, const float *scales, bool isC) {
            uint32_t lane = l;
            opaque(lane);
            const int r = int(lane) & 15, g = int(lane) >> 4;
            Sum<T, NR> f[NT][NB];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    f[t][b] = to_sum<T, NR>(state[t][b][0], state[t][b][1]);
                    pin(f[t][b]);
                }
            fence();
            fetch_state(from, state, fk, fpb);
            fence();
            f32x4 sums[NT][MT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m) sums[t][m] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                In<T> fa[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) fa[m] = tile_row<T, PCH>(tile, 16 * (m0 + m) + r, 4 * b + g);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_left<MT>(sums[t], fa, f[t][b]);
                fence();
            }
            float part[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) part[i] = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const f32x4 *const acc = sums[t];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const f32x4 scale = *reinterpret_cast<const f32x4 *>(scales + 16 * (m0 + m) + 4 * g);
                    const f32x4 dts = *reinterpret_cast<const f32x4 *>(v.dt + 16 * (m0 + m) + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = scale[e] * acc[m][e];
                        if (isC) {
                            dC[t][m][e] += a;
                            part[4 * m + e] = __builtin_fmaf(value(tC, r, g, t, m, e), a, part[4 * m + e]);
                        } else {
                            dB[t][m][e] = __builtin_fmaf(dts[e], a, dB[t][m][e]);
                            part[4 * m + e] = __builtin_fmaf(value(tB, r, g, t, m, e), a, part[4 * m + e]);
                        }
                    }
                }
            }
            // over the 16 lanes of a row group, value 4 m + e to lane 4 m + e: row 16 (m0 + m) + 4 g + e
            const float sum = fold16(part, r);
            float *const to = (isC ? rows_ : ends_)[k & 1][wave] + (16 * (r >> 2) + 4 * g + (r & 3));
            if (r < 4 * MT) *to = pb ? *to + sum : sum;
        };
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const In<T> fy[2] = {tile_row<T, PCH>(tY, 32 * ih + r, 4 * b + g), tile_row<T, PCH>(tY, 32 * ih + 16 + r, 4 * b + g)};
            mma_left<2>(dW, fy, tile_row<T, PCH>(tX, 16 * jt + r, 4 * b + g));
        }
        side(tY, s0, p.ws.S0, v.up, true);
        side(tX, d1, p.ws.dS1, v.tail, false);
        if (done) {
            // dW: rows i = 16 (2 ih + m) + 4 g + e, column j = 16 jt + r
            uint32_t lane = l;
            opaque(lane);
            const int r = int(lane) & 15, g = int(lane) >> 4, l = int(lane);
            const int j = 16 * jt + r, q = k & 1;
            const float jhi = v.hi[j], jlo = v.lo[j], jdt = v.dt[j];
            float sums[16], col = 0.0f;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const f32x4 hi = *reinterpret_cast<const f32x4 *>(v.hi + 32 * ih + 16 * m + 4 * g);
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(v.lo + 32 * ih + 16 * m + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 32 * ih + 16 * m + 4 * g + e;
                    // (no branch around the exponential)
                    const float d = j <= i ? (hi[e] - jhi) + (lo[e] - jlo) : -__builtin_inff();
                    const float w = dW[m][e] * exp2_hw(d);
                    Q[m][e] = __builtin_fmaf(w, jdt, Q[m][e]);
                    const float R = w * M[m][e], below = j < i ? R : 0.0f;
                    col += below;
                    sums[4 * m + e] = below * jdt;
                    if (i == j) {
                        diag_[q][j] = dW[m][e];
                        diagR_[q][j] = R;
                    }
                }
            }
            col += __shfl_xor(col, 16);
            col += __shfl_xor(col, 32);
            if (g == 0) cols_[q][ih][j] = col;
#pragma unroll
            for (int i = 8; i < 16; ++i) sums[i] = 0.0f;
            const float sum = fold16(sums, r);
            if (r < 8) rowsR_[q][wave][16 * (r >> 2) + 4 * g + (r & 3)] = sum;
            dot += from_dpp<0x140>(dot);  // all of 16 lanes by mirrors, then across
            dot += from_dpp<0x141>(dot);
            dot += from_dpp<0x1B>(dot);
            dot += from_dpp<0xB1>(dot);
            dot += __shfl_xor(dot, 16);
            dot += __shfl_xor(dot, 32);
            if (l == 0) dots_[q][wave] = dot;
        }
        k = nk;
        pb = npb;
    }
    __syncthreads();
    if (wave == ((nh - 1) & (kGradWaves - 1))) finish(nh - 1);

    // dB += Q^T C, dC += Q B: Q's fragments through LDS, as rows j and as rows i
    auto product = [&](f32x4 (*to)[MT], const E<T> *tile) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            Sum<T, NQ> f[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const E<T> *at = tXY + (2 * (m0 + m) + b) * kFrag;
                if constexpr (sizeof(T) == 4) {
                    const f32x4 *s = reinterpret_cast<const f32x4 *>(at + l * 8);
                    f[m] = F32x8{s[0], s[1]};
                } else {
#pragma unroll
                    for (int i = 0; i < NQ; ++i) f[m].t[i] = *reinterpret_cast<const bf16x8 *>(at + (i * 64 + l) * 8);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
                mma_left<MT>(to[t], f, tile_cols<T, NCH>(tile, 32 * b + 4 * g, 32 * b + 16 + 4 * g,
                                                         [&](int s) { return n0 + 16 * t + 4 * s; }));
        }
    };
    {
        const Sum<T, NQ> f = to_sum<T, NQ>(Q[0], Q[1]);  // rows j of tile jt, block ih of the i
        E<T> *at = tXY + (2 * jt + ih) * kFrag;
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
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // row i = 16 (2 ih + m) + 4 g + e, column j = 16 jt + r of the block jt / 2
            const int lane = (r >> 2) * 16 + 4 * g + e, at = 4 * (jt & 1) + (r & 3);
            E<T> *to = tXY + (2 * (2 * ih + m) + (jt >> 1)) * kFrag + lane * 8 + at;
            if constexpr (sizeof(T) == 4) {
                *to = Q[m][e];
            } else {
                float q = Q[m][e], none = 0.0f;
#pragma unroll
                for (int i = 0; i < NQ; ++i) to[i * 512] = uint16_t(split_pair(q, none));
            }
        }
    __syncthreads();
    product(dC, tB);

    // the parts' sums in the workspace, or dB and dC themselves
    const long long at = (((long long)part * p.records + record) * p.groups + group) * 64 * p.ws.Nr;
    const long long bAt = seq.batch * p.sdB.b + t0 * p.sdB.t + group * p.sdB.h;
    const long long cAt = seq.batch * p.sdC.b + t0 * p.sdC.t + group * p.sdC.h;
    auto put = [&](void *to, bool bf16, long long i, float x) {
        if (bf16) static_cast<bf16_t *>(to)[i].bits = uint16_t(pack_bf16x2(x, x));
        else static_cast<float *>(to)[i] = x;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * (m0 + m) + 4 * g + e, n = n0 + 16 * t + r;
                if (i >= rows) continue;
                if (p.parts > 1) {
                    if (n < p.ws.Nr) {
                        p.ws.dBp[at + i * p.ws.Nr + n] = dB[t][m][e];
                        p.ws.dCp[at + i * p.ws.Nr + n] = dC[t][m][e];
                    }
                } else if (n < p.N) {
                    put(p.dB, p.g_bf16, bAt + i * p.sdB.t + n, dB[t][m][e]);
                    put(p.dC, p.g_bf16, cAt + i * p.sdC.t + n, dC[t][m][e]);
                }
            }
}

// dB (blockIdx.z 0) and dC: the parts' sums, in order.
__global__ __launch_bounds__(kThreads) void heads_parts_kernel(const GradParams p)
{
    const int record = int(blockIdx.x), group = int(blockIdx.y);
    const DeltaSeq seq = delta_seq(p.cu, delta_seq_of(p.cu, p.nseq, p.seqlen, record), p.seqlen);
    const int c = record - seq.chunk0, left = seq.len - c * kDeltaChunk;
    if (c < 0 || left <= 0) return;
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
    const dim3 grid(unsigned(p.records), p.groups, p.parts), block(kThreads), wide(kGradThreads);
    if (log_enabled())
        log_line("head_scan_bwd: heads_grad_kernel<%s, N %d, fast %d>, grid (%u, %u, %u) x %u threads, %d heads a part",
                 type_tag<T>(), ND, int(kFast), grid.x, grid.y, grid.z, wide.x, p.each);
    heads_grad_kernel<T, ND, kFast><<<grid, wide, 0, stream>>>(p);
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
