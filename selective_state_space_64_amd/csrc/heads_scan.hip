// heads_scan.hip -- the selective scan with one decay a head over whole
// sequences, a chunk of 64 steps at a time on the matrix cores, and the same
// recurrence backwards (gfx950; C ABI in include/ssm_heads.h).
//
// With D_t = softplus(dt_t + dt_bias), G_i the sum of the chunk's decays D_t A
// up to step i and S0 (N x P) the state entering it:
//     W_ij = e^{G_i - G_j} D_j C_i . B_j  (j <= i)
//     y_i  = e^{G_i} S0^T C_i + sum_j W_ij x_j + Dskip x_i
//     S1   = e^{Gc} S0 + sum_j B_j (D_j e^{Gc - G_j} x_j)^T
// and for the gradients, from the last step to the first, with dS1 the
// gradient of the state leaving the chunk:
//     dx_j = D_j e^{Gc - G_j} dS1^T B_j + sum_i W_ij dy_i + Dskip dy_j
//     dS0  = e^{Gc} dS1 + sum_i C_i (e^{G_i} dy_i)^T
// which is the same recurrence with B and C exchanged, dy for x, the triangle
// transposed and the two row scales exchanged: one kernel runs both, on L, R,
// v and out.  The columns of the state are independent of one another, so a
// workgroup holds 64 columns of one head's state over the whole sequence, each
// of its four waves 16 of them in registers; a product's result is the next
// one's right operand in place.  W is made by the four waves together and goes
// through LDS.
//
// What bounds it (4 x 2048 steps, 80 heads of 128 x 64 with one group, bf16): the chain of
// products inside a chunk.  126 us, where the tensors' 184 MB take 35 us at a large copy's
// rate and the products, split terms and all, 56 us at a large matrix product's; of the
// busy compute units' cycles vector ALUs issue in 41 %, matrix pipes are busy in 31 %, LDS
// in 44 %.  320 workgroups leave 192 of the compute units with one, which takes 95 us by
// itself, and 64 with two: 512 workgroups take 153.  Not faster for the same layer (at 132
// us then): two waves of 32 columns with copies straight to LDS (164), four waves with such
// copies (139), a third barrier a chunk (150).  fp32 tensors take 564 us.  256 state rows
// do not fit the registers: 290 us with 104 bytes of scratch a lane in bf16, 2.55 ms with
// 1072 in fp32.
#include "heads_common.hpp"

namespace ssm {
namespace heads {
namespace {

// What a run leaves: out and the final state; beside them the state entering
// every chunk; only these; or a segment's end state and decay.
enum { kOutRun = 0, kOutKeepRun = 1, kKeepRun = 2, kEndRun = 3 };

// Rows 16 m + r, columns c .. c + 3 of y[m], `rows` and `cols` of them there.  kFast: the
// columns are stored together, into one buffer whose end stands for the mask of rows.
template <bool kFast>
__device__ inline void store_out(char *out, long long step, int bf16, int rows, int c, int cols, int r, const f32x4 *y)
{
    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
    if constexpr (kFast) {
        const int row = int(step) * (bf16 ? 2 : 4);
        const auto buf = buffer_of(out, rows * (long long)row);
        const uint32_t off = c < cols ? uint32_t(r * row + c * (bf16 ? 2 : 4)) : kOutside;
        if (bf16) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16x2(y[m][0], y[m][1]), pack_bf16x2(y[m][2], y[m][3])},
                                                      buf, off + uint32_t(16 * m * row), 0, 0);
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[m]), buf, off + uint32_t(16 * m * row), 0, 0);
        }
    } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const long long at = (long long)(16 * m + r) * step + c;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (16 * m + r < rows && c + e < cols) {
                    if (bf16) reinterpret_cast<bf16_t *>(out)[at + e].bits = uint16_t(pack_bf16x2(y[m][e], y[m][e]));
                    else reinterpret_cast<float *>(out)[at + e] = y[m][e];
                }
        }
    }
}

// NY: terms of W and of the state as the readout sees it (bf16 compute).
template <typename T, int ND, int kRun, bool kRev, bool kFast, int NY>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 && ND <= 128 ? 2 : 1)) void heads_scan_kernel(const HeadsScan p)
{
    constexpr bool kOut = kRun == kOutRun || kRun == kOutKeepRun, kKeep = kRun == kOutKeepRun || kRun == kKeepRun,
                   kEnd = kRun == kEndRun;
    constexpr int NCH = ND / 8, KB = ND / 32, kTile = 64 * ND, kVCH = kCols / 8;
    // Terms of bf16 compute.  W and the state as the readout sees it: two under a bf16 y (up to
    // 2^-17 of a value, 256 times under its rounding: its error is that of fp32 products to four
    // digits, and single elements next to a tie round the other way), three for an fp32 y (off by
    // 1e-7 of its size, as fp32 products are; with two by 2.4e-6).  The layer's forward takes
    // 151 us with an fp32 y, 134 with two terms.  Three under a bf16 y too were measured: 144 us
    // against 126, packed prompts 138 against 126, the training step 682 against 672.  What
    // enters the state: three (2^-25), since the fp32 states of a whole sequence are sums of it.
    constexpr int NW = NY, NR = NY, NX = 3;
    constexpr int kFrag = 512 * (sizeof(T) == 2 ? NW : 1);
    // Chunks whose decays are formed at a time, a wave each; the next ones' while these
    // are in work (fp32 tiles of 256 entries leave LDS for two).
    constexpr int kAhead = sizeof(T) == 4 && ND == 256 ? 1 : kWaves;
    __shared__ __align__(16) E<T> tileL[kOut ? kTile : 8];
    __shared__ __align__(16) E<T> tileR[kTile];
    __shared__ __align__(16) E<T> tileV[64 * kCols];
    __shared__ __align__(16) E<T> tri[kOut ? kTriFrags * kFrag : 8];
    __shared__ __align__(16) Vec vecs[2 * kAhead];

    const int head = int(blockIdx.y), group = head / p.rep, l = int(threadIdx.x) & 63, wave = wave_of();
    const int r = l & 15, g = l >> 4;
    const DeltaSegment seg = delta_segment(p.cu, p.nseq, p.seqlen, p.ws.seg_chunks, int(blockIdx.x));
    if (!seg.live) return;  // the whole workgroup
    // the segment's place in the order of the run
    const bool first = kRev ? seg.behind == 0 : seg.index == 0, last = kRev ? seg.index == 0 : seg.last;
    if (kEnd && last) return;  // nothing follows
    const DeltaSeq &seq = seg.s;
    const int c0 = seg.c0, n = seg.c1 - seg.c0;
    const int col0 = int(blockIdx.z) * kCols, wcol = 16 * wave, col = col0 + wcol + r;  // wcol: the wave's first of them
    const long long state_at = ((long long)seg.seq * p.h + head) * p.N * (long long)p.P + col;
    const long long slot = (long long)blockIdx.x * p.h + head;
    // this segment's place in ends, the one before it in the run's order, and the last one's
    float *const end_to = p.ws.ends + slot * p.ws.state;
    const float *const entry = p.ws.ends + (slot + (kRev ? p.h : -p.h)) * p.ws.state;
    float *const initial = p.ws.ends + (slot + (long long)p.h * (kRev ? -seg.index : seg.behind)) * p.ws.state;
    const bool split = p.ws.seg_chunks > 0 && !(first && last);
    const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.0f, D = p.D ? p.D[head] : 0.0f;

    // S: tiles 2 b and 2 b + 1 hold the rows 32 b + 8 g + {0..3} and + {4..7}
    f32x4 S[ND / 16];
    auto row_of = [&](int m, int e) { return 32 * (m / 2) + 8 * g + 4 * (m % 2) + e; };
    // a record's rows behind Nr lie behind its end: they read as 0 and are not stored
    auto record_off = [&]() {
        uint32_t off = col0 + wcol < p.ws.Pp ? uint32_t(8 * g * p.ws.Pp + col) * 4u : kOutside;
        opaque(off);
        return off;
    };
    auto record_row = [&](int m, int e) { return uint32_t((32 * (m / 2) + 4 * (m % 2) + e) * p.ws.Pp) * 4u; };
    auto keep_rows = [&](float *to, int b) {  // 32 b and the 31 behind
        const auto buf = buffer_of(to, p.ws.state * 4);
        const uint32_t off = record_off();
#pragma unroll
        for (int m = 2 * b; m < 2 * b + 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[m][e]), buf, off + record_row(m, e), 0, 0);
    };
    auto keep_state = [&](float *to) {
#pragma unroll
        for (int b = 0; b < KB; ++b) keep_rows(to, b);
    };
    auto load_state = [&](const float *from) {
        const auto buf = buffer_of(from, p.ws.state * 4);
        const uint32_t off = record_off();
#pragma unroll
        for (int m = 0; m < ND / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[m][e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, off + record_row(m, e), 0, 0));
    };
#pragma unroll
    for (int m = 0; m < ND / 16; ++m) S[m] = f32x4{0, 0, 0, 0};
    if (!first) {
        if (!kEnd) load_state(entry);
    } else if (p.s0 && split && !kEnd) {
        // a split sequence's initial state, kept by the ends' run: sL may be the same
        // memory, and the last segment may end before the first begins
        load_state(initial);
    } else if (p.s0) {
#pragma unroll
        for (int m = 0; m < ND / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col < p.P && row_of(m, e) < p.N) S[m][e] = p.s0[state_at + (long long)row_of(m, e) * p.P];
        if (kEnd) keep_state(initial);
    }

    // the chunks in the order of the run, and where each one's rows begin
    const int ein = p.in_bf16 ? 2 : 4, ev = p.v_bf16 ? 2 : 4, eo = p.out_bf16 ? 2 : 4;
    auto chunk_of = [&](int k) { return kRev ? seg.c1 - 1 - k : c0 + k; };
    const long long begin = seq.first + (long long)chunk_of(0) * kDeltaChunk;
    const int turn = kRev ? -kDeltaChunk : kDeltaChunk;
    const char *pL = static_cast<const char *>(p.L) + (seq.batch * p.sL_.b + begin * p.sL_.t + group * p.sL_.h) * ein;
    const char *pR = static_cast<const char *>(p.R) + (seq.batch * p.sR.b + begin * p.sR.t + group * p.sR.h) * ein;
    const char *pV = static_cast<const char *>(p.v) + (seq.batch * p.sv.b + begin * p.sv.t + head * p.sv.h + col0) * ev;
    char *pO = static_cast<char *>(p.out) + (seq.batch * p.sout.b + begin * p.sout.t + head * p.sout.h + col0) * eo;
    const long long dL = turn * p.sL_.t * ein, dR = turn * p.sR.t * ein, dV = turn * p.sv.t * ev, dO = turn * p.sout.t * eo;
    float *pK = p.keep + (((long long)seq.chunk0 + chunk_of(0)) * p.h + head) * p.ws.state;
    const long long dK = (kRev ? -p.h : p.h) * p.ws.state;
    const long long dt_at = seq.batch * p.sdt.b + seq.first * p.sdt.t + head * p.sdt.h;
    auto rows_of = [&](int k) { return min(seq.len - chunk_of(k) * kDeltaChunk, kDeltaChunk); };

    TileIn<T, NCH, kFast> inL, inR;
    TileIn<T, kVCH, kFast> inV;
    inL.init(p.sL_.t, p.N);
    inR.init(p.sR.t, p.N);
    inV.init(p.sv.t, p.P - col0);
    // the chunk's rows on their way, and from there to the tiles
    auto fetch = [&](int rows) {
        if constexpr (kOut) inL.fetch(pL, p.sL_.t, rows);
        inR.fetch(pR, p.sR.t, rows);
        inV.fetch(pV, p.sv.t, rows);
    };
    auto store = [&](int rows) {
        if constexpr (kOut) inL.store(tileL, pL, p.sL_.t, rows, p.N, p.in_bf16);
        inR.store(tileR, pR, p.sR.t, rows, p.N, p.in_bf16);
        inV.store(tileV, pV, p.sv.t, rows, p.P - col0, p.v_bf16);
    };
    // the raw steps of the wave's chunk of those from `base` on (or of the last one: a load
    // in a branch would be waited for where the branch ends)
    RawStep raw{};
    auto load_raw = [&](int base) {
        const int k = min(base + wave, n - 1);
        raw.load(p.dt, dt_at + ((long long)chunk_of(k) * kDeltaChunk + min(l, rows_of(k) - 1)) * p.sdt.t, p.in_bf16);
    };
    double passed = 0.0;  // the wave's part of the segment's decay
    auto prepare = [&](int base) {
        if (wave >= kAhead || base + wave >= n) return;
        const Decays d = decays(raw.value(p.in_bf16), bias, A, rows_of(base + wave));
        Vec &v = vecs[(base + wave) & (2 * kAhead - 1)];
        v.hi[l] = float(d.G);
        v.lo[l] = float(d.G - double(float(d.G)));
        v.dt[l] = d.dt;
        const float up = exp2_of(d.G), down = d.dt * exp2_of(d.end - d.G);
        v.out[l] = kRev ? down : up;
        v.in[l] = kRev ? up : down;
        if (l == 0) v.end[0] = exp2_of(d.end);
        passed += d.end;
    };

    if (n > 0) {
        load_raw(0);
        fetch(rows_of(0));
        if constexpr (kOut)  // the halves of fragments on the far side of the diagonal stay 0
            for (int i = int(threadIdx.x); i < kTriFrags * kFrag; i += kThreads) tri[i] = E<T>(0);
        prepare(0);
        load_raw(kAhead);
        store(rows_of(0));
        __syncthreads();
    }
    // What is still on its way is waited for here: a wait in the loop would be one for the
    // stores of the chunk before as well.
    raw.pin();
#pragma unroll
    for (int m = 0; m < ND / 16; ++m) asm volatile("" : "+v"(S[m]));

    // All chunks, as the wave that is the W-th.  Each phase's fragments are read while the
    // phase before it computes, and the vector work (terms, decays) takes turns with matrix
    // instructions that do not wait for it.
    auto run = [&](auto is) {
        constexpr int W = decltype(is)::value;
        for (int k = 0; k < n; ++k) {
            const Vec &vec = vecs[k & (2 * kAhead - 1)];
            if ((k & (kAhead - 1)) == 0) prepare(k + kAhead);
            load_raw(k + 1 + kAhead);  // for the next chunk's prepare()
            const bool more = k + 1 < n;  // (the last chunk is fetched again: a branch here would wait for the loads)
            const int next_rows = rows_of(more ? k + 1 : k);
            pL += more ? dL : 0;
            pR += more ? dR : 0;
            pV += more ? dV : 0;
            // the wave's columns of v: rows 32 b + 4 g + {0..3} and + 16
            In<T> fv[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                fv[b] = tile_cols<T, kVCH>(tileV, 32 * b + 4 * g, 32 * b + 16 + 4 * g, [&](int q) { return wcol + 4 * q; });
            const float end = vec.end[0];

            // S^T L (y[m]: row of L 16 m + r, columns 4 g + e of the tile), and W's column tile of
            // this wave (w[m]: the same row, rows of R 16 W + 4 g + e)
            f32x4 y[4], w[4];
            Sum<T, NX> fx[2];
            auto enter = [&](int b) {  // the scaled rows 32 b .. of v
                f32x4 x[2];
                to_floats(fv[b], x[0], x[1]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const f32x4 scale = *reinterpret_cast<const f32x4 *>(vec.in + 32 * b + 16 * m + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[m][e] *= scale[e];
                }
                fx[b] = to_sum<T, NX>(x[0], x[1]);
                pin(fx[b]);
            };
            if constexpr (kOut) {
                In<T> fl[2][4], fr[2];
                Sum<T, NR> fs[2];
                auto read = [&](int b) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) fl[b & 1][m] = tile_row<T, NCH>(tileL, 16 * m + r, 4 * b + g);
                    fr[b & 1] = tile_row<T, NCH>(tileR, 16 * W + r, 4 * b + g);
                };
                auto form = [&](int b) {
                    fs[b & 1] = to_sum<T, NR>(S[2 * b], S[2 * b + 1]);
                    pin(fs[b & 1]);
                };
#pragma unroll
                for (int m = 0; m < 4; ++m) y[m] = w[m] = f32x4{0, 0, 0, 0};
                read(0);
                form(0);
                fence();
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    if (b + 1 < KB) {
                        read(b + 1);
                        form(b + 1);
                    }
                    // (the tiles of the triangle: from the diagonal's on, or up to it)
                    constexpr int m0 = kRev ? 0 : W, kTiles = kRev ? W + 1 : 4 - W;
                    // Kept a part at a time, between the products: a compute unit's stores take about
                    // 16 bytes a cycle, and a wave that has 32 of them to give waits for that (the
                    // layer's training step 716 us with all of them in front of the state's update,
                    // 671 so; rows on their way ahead of them cost registers: 691).
                    if constexpr (kKeep) keep_rows(pK, b);
                    mma_right<kTiles>(w + m0, fr[b & 1], fl[b & 1] + m0);
                    mma_right<4>(y, fs[b & 1], fl[b & 1]);
                    // the last two have the time to form the operands of the next phase
                    if (b >= KB - 2) enter(b - (KB - 2));
                    interleave<sizeof(T) == 2 ? 5 : 10, sizeof(T) == 2 ? kTiles + 4 * NR : 64, sizeof(T) == 2 ? 5 : 0>();
                    fence();
                }
            } else {
                enter(0);
                enter(1);
            }
            fetch(next_rows);  // the next chunk's, on their way
            if constexpr (kKeep) {
                if constexpr (!kOut) keep_state(pK);
                pK += dK;
            }
            // S = e^{Gc} S + R^T (scaled v);  beside it W's decays
            In<T> fc[2][2];  // [parity of the time block][tile of the pair]
            auto read_cols_of = [&](int b, int t) {
#pragma unroll
                for (int o = 0; o < 2; ++o)
                    fc[t][o] = tile_cols<T, NCH>(tileR, 32 * t + 4 * g, 32 * t + 16 + 4 * g,
                                                 [&](int q) { return 32 * b + 8 * q + 4 * o; });
            };
            auto decay = [&](int b) {
#pragma unroll
                for (int m = 2 * b; m < 2 * b + 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[m][e] *= end;
            };
            // W's row tile m.  Off the diagonal a decay is a product
            // over the step between the tiles: one exponential a row and one a column.
            f32x4 far;
            auto weigh = [&](int m) {
                // the last step of the earlier tile
                const int ref = kRev ? (W ? 16 * W - 1 : 0) : 16 * W + 15;
                const int at = 16 * m + r;
                const float ihi = vec.hi[at], ilo = vec.lo[at], rhi = vec.hi[ref], rlo = vec.lo[ref];
                if (m == W) {
                    const f32x4 hi = *reinterpret_cast<const f32x4 *>(vec.hi + 16 * W + 4 * g);
                    const f32x4 lo = *reinterpret_cast<const f32x4 *>(vec.lo + 16 * W + 4 * g);
                    const f32x4 dts = *reinterpret_cast<const f32x4 *>(vec.dt + 16 * W + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float q = (rhi - hi[e]) + (rlo - lo[e]);
                        far[e] = kRev ? exp2_hw(-q) : exp2_hw(q) * dts[e];
                        const int j = 16 * W + 4 * g + e;
                        float d = (ihi - hi[e]) + (ilo - lo[e]);
                        if (kRev) d = -d;
                        d = (kRev ? j >= at : j <= at) ? d : -__builtin_inff();  // (no branch around the exponential)
                        // the skip is the diagonal's
                        w[m][e] = __builtin_fmaf(w[m][e], exp2_hw(d) * (kRev ? vec.dt[at] : dts[e]), at == j ? D : 0.0f);
                    }
                } else {
                    const float d = (ihi - rhi) + (ilo - rlo);
                    const float f = kRev ? exp2_hw(-d) * vec.dt[at] : exp2_hw(d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[m][e] *= f * far[e];
                }
                // the half of a fragment that these four are
                E<T> *to = tri + (kRev ? tri_upper(m, W / 2) : tri_lower(m, W / 2)) * kFrag + l * 8 + 4 * (W & 1);
                if constexpr (sizeof(T) == 4) {
                    *reinterpret_cast<f32x4 *>(to) = w[m];
                } else {
                    float v0 = w[m][0], v1 = w[m][1], v2 = w[m][2], v3 = w[m][3];
#pragma unroll
                    for (int q = 0; q < NW; ++q) {
                        typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
                        const uint32_t ab = split_pair(v0, v1), cd = split_pair(v2, v3);
                        *reinterpret_cast<u32x2 *>(to + q * 512) = u32x2{ab, cd};
                    }
                }
            };
            read_cols_of(0, 0);
            decay(0);
            fence();
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                read_cols_of(b, 1);
                if (b + 1 < KB) decay(b + 1);
                mma_left<2>(S + 2 * b, fc[0], fx[0]);
                if (b + 1 < KB) read_cols_of(b + 1, 0);
                mma_left<2>(S + 2 * b, fc[1], fx[1]);
                if constexpr (kOut) {
                    // from the diagonal's tile on to the corner of the triangle
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q * KB / 4 == b && (kRev ? W - q >= 0 : W + q < 4)) weigh(kRev ? W - q : W + q);
                }
                interleave<sizeof(T) == 2 ? 4 : 0, sizeof(T) == 2 ? 4 * NX : 32, sizeof(T) == 2 ? 4 : 0>();
                fence();
            }
            if constexpr (kOut) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float scale = vec.out[16 * m + r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[m][e] *= scale;
                }
            }
            __syncthreads();  // W is complete, the tiles have been read
            store(next_rows);
            if constexpr (kOut) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    // row tiles with a fragment in block b: all four, but two in one of the blocks
                    constexpr int kAll = kRev ? 1 : 0;
                    auto frag = [&](int m) {
                        const E<T> *at = tri + (kRev ? tri_upper(m, b) : tri_lower(m, b)) * kFrag;
                        if constexpr (sizeof(T) == 4) {
                            const f32x4 *q = reinterpret_cast<const f32x4 *>(at + l * 8);
                            return F32x8{q[0], q[1]};
                        } else {
                            Frag<NW> f;
#pragma unroll
                            for (int i = 0; i < NW; ++i) f.t[i] = *reinterpret_cast<const bf16x8 *>(at + (i * 64 + l) * 8);
                            return f;
                        }
                    };
                    if (b == kAll) {
                        const Sum<T, NW> a[4] = {frag(0), frag(1), frag(2), frag(3)};
                        mma_right<4>(y, fv[b], a);
                    } else {
                        constexpr int m0 = kRev ? 0 : 2;
                        const Sum<T, NW> a[2] = {frag(m0), frag(m0 + 1)};
                        mma_right<2>(y + m0, fv[b], a);
                    }
                }
                store_out<kFast>(pO, p.sout.t, p.out_bf16, rows_of(k), wcol + 4 * g, p.P - col0, r, y);
                pO += dO;
            }
            __syncthreads();
        }
        settle();
    };
    if constexpr (kOut) {
        if (wave == 0) run(std::integral_constant<int, 0>{});
        else if (wave == 1) run(std::integral_constant<int, 1>{});
        else if (wave == 2) run(std::integral_constant<int, 2>{});
        else run(std::integral_constant<int, 3>{});
    } else {
        run(std::integral_constant<int, 0>{});
    }

    if constexpr (kEnd) {
        keep_state(end_to);
        if (blockIdx.z == 0) {
            double *part = reinterpret_cast<double *>(vecs);
            __syncthreads();
            if (l == 0) part[wave] = passed;
            __syncthreads();
            if (threadIdx.x == 0) {
                double sum = 0.0;
                for (int i = 0; i < kWaves; ++i) sum += part[i];
                p.ws.decay[slot] = exp2_of(sum);
            }
        }
    } else if (p.sL && last) {
#pragma unroll
        for (int m = 0; m < ND / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col < p.P && row_of(m, e) < p.N) p.sL[state_at + (long long)row_of(m, e) * p.P] = S[m][e];
    }
}

// The states that a sequence's segments enter with, in place of the end states
// (element by element: a segment's decay is a number), in the order of the run.
__global__ __launch_bounds__(kThreads) void heads_compose_kernel(const HeadsScan p, bool reverse)
{
    const int head = int(blockIdx.y), L = p.ws.seg_chunks;
    const DeltaSeq seq = delta_seq(p.cu, int(blockIdx.x), p.seqlen);
    const int per = (p.seqlen + kDeltaChunk - 1) / kDeltaChunk;
    const int chunks = (seq.len + kDeltaChunk - 1) / kDeltaChunk, segs = (chunks + L - 1) / L;
    const long long z0 = p.cu ? seq.chunk0 / L + int(blockIdx.x) : (long long)blockIdx.x * ((per + L - 1) / L);
    const long long i = ((long long)blockIdx.z * kThreads + threadIdx.x) * 4;
    if (i >= p.ws.state) return;
    auto at = [&](int k) { return (z0 + (reverse ? segs - 1 - k : k)) * p.h + head; };
    auto place = [&](int k) { return reinterpret_cast<f32x4 *>(p.ws.ends + at(k) * p.ws.state + i); };
    if (segs < 3) return;
    f32x4 s = *place(0);
    constexpr int kDeep = 4;  // loads under way
    f32x4 ends[kDeep];
    float d[kDeep];
    auto load = [&](int k, int i) {
        k = min(k, segs - 2);
        ends[i] = *place(k);
        d[i] = p.ws.decay[at(k)];
    };
#pragma unroll
    for (int i = 0; i < kDeep; ++i) load(1 + i, i);
    for (int k = 1; k + 1 < segs; k += kDeep)
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            if (k + i + 1 < segs) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = __builtin_fmaf(d[i], s[e], ends[i][e]);
                load(k + i + kDeep, i);
                *place(k + i) = s;
            }
        }
}

template <typename T, int ND, bool kRev, bool kFast>
hipError_t scan_run(const HeadsArgs &a, const HeadsScan &p, hipStream_t stream)
{
    const HeadsSplit split = heads_split(a.batch, a.seqlen, a.h, a.P, a.cu ? a.nseq : 0);
    const dim3 grid(split.segs ? split.segs : a.nseq, a.h, (a.P + kCols - 1) / kCols), block(kThreads);
    if (log_enabled())
        log_line("head_scan: heads_scan_kernel<%s, N %d, reverse %d, fast %d>, out %d (%s), keep %d, grid (%u, %u, %u) x %u "
                 "threads, %d chunks a segment", type_tag<T>(), ND, int(kRev), int(kFast), int(p.out != nullptr),
                 p.out_bf16 ? "bf16" : "f32", int(p.keep != nullptr), grid.x, grid.y, grid.z, block.x, split.seg_chunks);
    if (split.segs) {
        heads_scan_kernel<T, ND, kEndRun, kRev, kFast, 2><<<grid, block, 0, stream>>>(p);
        const dim3 parts(a.nseq, a.h, (p.ws.state / 4 + kThreads - 1) / kThreads);
        heads_compose_kernel<<<parts, block, 0, stream>>>(p, kRev);
    }
    if constexpr (kRev) {
        // (bf16 compute has gradients of bf16)
        heads_scan_kernel<T, ND, kOutKeepRun, kRev, kFast, 2><<<grid, block, 0, stream>>>(p);
    } else {
        auto run = [&](auto terms) {
            constexpr int NY = decltype(terms)::value;
            if (p.keep) heads_scan_kernel<T, ND, kOutKeepRun, kRev, kFast, NY><<<grid, block, 0, stream>>>(p);
            else heads_scan_kernel<T, ND, kOutRun, kRev, kFast, NY><<<grid, block, 0, stream>>>(p);
        };
        if (!p.out) heads_scan_kernel<T, ND, kKeepRun, kRev, kFast, 2><<<grid, block, 0, stream>>>(p);
        else if (p.out_bf16) run(std::integral_constant<int, 2>{});
        else run(std::integral_constant<int, sizeof(T) == 4 ? 2 : 3>{});  // (fp32 compute has no terms)
    }
    return hipGetLastError();
}

template <typename T>
hipError_t scan_typed(const HeadsArgs &a, const HeadsScan &p, bool reverse, bool fast, hipStream_t stream)
{
    const int nd = heads_nd(a.N);
    auto sized = [&](auto n) {
        constexpr int ND = decltype(n)::value;
        if (reverse) return fast ? scan_run<T, ND, true, true>(a, p, stream) : scan_run<T, ND, true, false>(a, p, stream);
        return fast ? scan_run<T, ND, false, true>(a, p, stream) : scan_run<T, ND, false, false>(a, p, stream);
    };
    return nd == 64 ? sized(std::integral_constant<int, 64>{})
         : nd == 128 ? sized(std::integral_constant<int, 128>{})
                     : sized(std::integral_constant<int, 256>{});
}

}  // namespace

hipError_t launch_heads_scan(const HeadsArgs &a, const HeadsScan &p, bool reverse, hipStream_t stream)
{
    const bool bf16 = p.in_bf16 && p.v_bf16, same = p.in_bf16 == p.v_bf16;
    const int es = p.in_bf16 ? 2 : 4;
    const bool fast = same && heads_fast(p.L, p.sL_, a.N, es, a, a.groups) && heads_fast(p.R, p.sR, a.N, es, a, a.groups) &&
                      heads_fast(p.v, p.sv, a.P, es, a, a.h) &&
                      (!p.out || heads_fast(p.out, p.sout, a.P, p.out_bf16 ? 2 : 4, a, a.h));
    return bf16 ? scan_typed<bf16_t>(a, p, reverse, fast, stream) : scan_typed<float>(a, p, reverse, fast, stream);
}

}  // namespace heads

size_t heads_fwd_workspace_bytes(int batch, int seqlen, int groups, int h, int N, int P, int num_seqs)
{
    size_t bytes = 0;
    heads::heads_ws(nullptr, batch, seqlen, groups, h, N, P, num_seqs, false, &bytes);
    return bytes;
}

hipError_t launch_heads_fwd(const HeadsArgs &a, hipStream_t stream)
{
    heads::HeadsScan p{a.seqlen, a.nseq, a.h / a.groups, a.h, a.N, a.P, a.in_bf16, a.in_bf16, a.out_bf16, a.cu,
                       a.C, a.B, a.x, a.dt, a.A, a.dt_bias, a.Dskip, a.h0, a.hL, a.y, nullptr,
                       a.sC, a.sB, a.sx, a.sdt, a.sy, heads::heads_ws(a, a.checkpoints)};
    p.keep = p.ws.S0;
    return launch_heads_scan(a, p, false, stream);
}

}  // namespace ssm
