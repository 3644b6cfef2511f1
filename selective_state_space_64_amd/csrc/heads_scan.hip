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
#include "heads_common.hpp"

namespace ssm {
namespace heads {
namespace {

// What a run leaves: out and the final state; beside them the state entering
// every chunk; only these; or a segment's end state and decay.
enum { kOutRun = 0, kOutKeepRun = 1, kKeepRun = 2, kEndRun = 3 };

// A chunk's decays for the workgroup: G as two floats, D, the scales of rows
// that read the state (out) and of rows that enter it (in), e^{Gc}.
struct Vec {
    float hi[64], lo[64], dt[64], out[64], in[64], end[4];
};

template <typename T, int ND, int kRun, bool kRev, bool kFast>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 && ND <= 128 ? 2 : 1)) void heads_scan_kernel(const HeadsScan p)
{
    constexpr bool kOut = kRun == kOutRun || kRun == kOutKeepRun, kKeep = kRun == kOutKeepRun || kRun == kKeepRun,
                   kEnd = kRun == kEndRun;
    constexpr int NCH = ND / 8, KB = ND / 32, kTile = 64 * ND, kVCH = kCols / 8;
    // Terms of bf16 compute.  W and the state as the readout sees it: two (2^-17 of a
    // value, under the rounding of a bf16 y); what enters the state: three (2^-25),
    // since the fp32 states of a whole sequence are sums of it.
    constexpr int NW = 2, NR = 2, NX = 3;
    constexpr int kTri = kTriFrags * 512 * (sizeof(T) == 2 ? NW : 1);
    __shared__ __align__(16) E<T> tileL[kOut ? kTile : 8];
    __shared__ __align__(16) E<T> tileR[kTile];
    __shared__ __align__(16) E<T> tileV[64 * kCols];
    __shared__ __align__(16) E<T> tri[kOut ? kTri : 8];
    __shared__ __align__(16) Vec vecs[2];

    const int head = int(blockIdx.y), group = head / p.rep, l = int(threadIdx.x) & 63, wave = wave_of();
    const int r = l & 15, g = l >> 4;
    const DeltaSegment seg = delta_segment(p.cu, p.nseq, p.seqlen, p.ws.seg_chunks, int(blockIdx.x));
    if (!seg.live) return;  // the whole workgroup
    // the segment's place in the order of the run
    const bool first = kRev ? seg.behind == 0 : seg.index == 0, last = kRev ? seg.index == 0 : seg.last;
    if (kEnd && last) return;  // nothing follows
    const DeltaSeq &seq = seg.s;
    const int c0 = seg.c0, n = seg.c1 - seg.c0;
    const int col0 = int(blockIdx.z) * kCols, col = col0 + 16 * wave + r;
    const bool mine = col < p.P, kept = col0 + 16 * wave < p.ws.Pp;  // (of whole tiles)
    const long long state_at = ((long long)seg.seq * p.h + head) * p.N * (long long)p.P + col;
    const long long slot = (long long)blockIdx.x * p.h + head;
    // this segment's place in ends, the one before it in the run's order, and the last one's
    float *const end_to = p.ws.ends + slot * p.ws.state + col;
    const float *const entry = p.ws.ends + (slot + (kRev ? p.h : -p.h)) * p.ws.state + col;
    float *const initial = p.ws.ends + (slot + (long long)p.h * (kRev ? -seg.index : seg.behind)) * p.ws.state + col;
    const bool split = p.ws.seg_chunks > 0 && !(first && last);

    const char *const L0 = static_cast<const char *>(p.L), *const R0 = static_cast<const char *>(p.R);
    const int ein = p.in_bf16 ? 2 : 4, ev = p.v_bf16 ? 2 : 4;
    const long long l_at = seq.batch * p.sL_.b + seq.first * p.sL_.t + group * p.sL_.h;
    const long long r_at = seq.batch * p.sR.b + seq.first * p.sR.t + group * p.sR.h;
    const long long v_at = seq.batch * p.sv.b + seq.first * p.sv.t + head * p.sv.h + col0;
    const long long dt_at = seq.batch * p.sdt.b + seq.first * p.sdt.t + head * p.sdt.h;
    const long long out_at = seq.batch * p.sout.b + seq.first * p.sout.t + head * p.sout.h;
    const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.0f, D = p.D ? p.D[head] : 0.0f;

    // S: tiles 2 b and 2 b + 1 hold the rows 32 b + 8 g + {0..3} and + {4..7}
    f32x4 S[ND / 16];
#pragma unroll
    for (int m = 0; m < ND / 16; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
            float s = 0.0f;
            if (!first) {
                if (!kEnd && kept && row < p.ws.Nr) s = entry[(long long)row * p.ws.Pp];
            } else if (p.s0) {
                // a split sequence's initial state: kept by the ends' run, because sL may
                // be the same memory and the last segment may end before the first begins
                if (split && !kEnd) {
                    if (kept && row < p.ws.Nr) s = initial[(long long)row * p.ws.Pp];
                } else if (mine && row < p.N) {
                    s = p.s0[state_at + (long long)row * p.P];
                }
            }
            S[m][e] = s;
        }
    auto keep_state = [&](float *to) {
        if (kept) {
#pragma unroll
            for (int m = 0; m < ND / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
                    if (row < p.ws.Nr) to[(long long)row * p.ws.Pp] = S[m][e];
                }
        }
    };
    if (kEnd && first && p.s0) keep_state(initial);

    auto chunk_of = [&](int k) { return kRev ? seg.c1 - 1 - k : c0 + k; };
    TileIn<T, NCH, kFast> inL, inR;
    TileIn<T, kVCH, kFast> inV;
    inL.init(p.sL_.t, p.N);
    inR.init(p.sR.t, p.N);
    inV.init(p.sv.t, p.P - col0);
    float raw = 0.0f;
    auto fetch = [&](int c) {
        const long long t = (long long)c * kDeltaChunk;
        const int rows = min(seq.len - c * kDeltaChunk, kDeltaChunk);
        if constexpr (kOut) inL.fetch(L0 + (l_at + t * p.sL_.t) * ein, p.sL_.t, rows, p.N);
        inR.fetch(R0 + (r_at + t * p.sR.t) * ein, p.sR.t, rows, p.N);
        inV.fetch(static_cast<const char *>(p.v) + (v_at + t * p.sv.t) * ev, p.sv.t, rows, p.P - col0);
        if (wave == kWaves - 1) raw = load_step(p.dt, dt_at + (t + min(l, rows - 1)) * p.sdt.t, p.in_bf16);
    };
    double passed = 0.0;  // the segment's decay
    auto prepare = [&](int c, Vec &v) {
        if (wave != kWaves - 1) return;
        const Decays d = decays(raw, bias, A, min(seq.len - c * kDeltaChunk, kDeltaChunk));
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
        fetch(chunk_of(0));
        prepare(chunk_of(0), vecs[0]);
    }
    for (int k = 0; k < n; ++k) {
        const int c = chunk_of(k), rows = seq.len - c * kDeltaChunk;
        const long long t = (long long)c * kDeltaChunk;
        const Vec &vec = vecs[k & 1];
        __syncthreads();  // the last chunk's reads are done
        {
            const int have = min(rows, kDeltaChunk);
            if constexpr (kOut) inL.store(tileL, L0 + (l_at + t * p.sL_.t) * ein, p.sL_.t, have, p.N, p.in_bf16);
            inR.store(tileR, R0 + (r_at + t * p.sR.t) * ein, p.sR.t, have, p.N, p.in_bf16);
            inV.store(tileV, static_cast<const char *>(p.v) + (v_at + t * p.sv.t) * ev, p.sv.t, have, p.P - col0,
                      p.v_bf16);
        }
        __syncthreads();
        if (k + 1 < n) fetch(chunk_of(k + 1));
        if constexpr (kKeep) {
            const long long record = (long long)seq.chunk0 + c;
            keep_state(p.keep + (record * p.h + head) * p.ws.state + col);
        }
        // W's column tile of this wave (rows of R 16 wave ..), and S^T L
        f32x4 y[4];
        if constexpr (kOut) {
            f32x4 w[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) y[m] = w[m] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                In<T> fl[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) fl[m] = tile_row<T, NCH>(tileL, 16 * m + r, 4 * b + g);
                const In<T> fr = tile_row<T, NCH>(tileR, 16 * wave + r, 4 * b + g);
                mma_right<4>(w, fr, fl);
                mma_left<4>(y, fl, to_sum<T, NR>(S[2 * b], S[2 * b + 1]));
            }
            // w[m]: rows of R 16 wave + 4 g + e, row of L 16 m + r
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(vec.hi + 16 * wave + 4 * g);
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(vec.lo + 16 * wave + 4 * g);
            const f32x4 dts = *reinterpret_cast<const f32x4 *>(vec.dt + 16 * wave + 4 * g);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int i = 16 * m + r;
                const float ihi = vec.hi[i], ilo = vec.lo[i], idt = vec.dt[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * wave + 4 * g + e;
                    const float d = (ihi - hi[e]) + (ilo - lo[e]);
                    const float f = exp2_hw(kRev ? -d : d) * (kRev ? idt : dts[e]);
                    w[m][e] = (kRev ? j >= i : j <= i) ? w[m][e] * f : 0.0f;
                }
                // the half of a fragment that these four are, if the triangle has it
                const int block = wave >> 1;
                if (kRev ? m < 2 || block == 1 : m >= 2 || block == 0) {
                    E<T> *to = tri + (kRev ? tri_upper(m, block) : tri_lower(m, block)) * (kTri / kTriFrags);
                    if constexpr (sizeof(T) == 4) {
                        *reinterpret_cast<f32x4 *>(to + l * 8 + 4 * (wave & 1)) = w[m];
                    } else {
#pragma unroll
                        for (int i = 0; i < NW; ++i) {
                            typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
                            float a = w[m][0], b = w[m][1], c2 = w[m][2], d2 = w[m][3];
                            const u32x2 bits = {split_pair(a, b), split_pair(c2, d2)};
                            w[m] = f32x4{a, b, c2, d2};
                            *reinterpret_cast<u32x2 *>(to + (i * 64 + l) * 8 + 4 * (wave & 1)) = bits;
                        }
                    }
                }
            }
        }
        if (k + 1 < n) prepare(chunk_of(k + 1), vecs[(k + 1) & 1]);
        // the wave's columns of v: rows 32 b + 4 g + {0..3} and + 16
        In<T> fv[2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
            fv[b] = tile_cols<T, kVCH>(tileV, 32 * b + 4 * g, 32 * b + 16 + 4 * g, [&](int q) { return 16 * wave + 4 * q; });
        f32x4 x[4];
        to_floats(fv[0], x[0], x[1]);
        to_floats(fv[1], x[2], x[3]);
        if constexpr (kOut) {
            // e^G S^T L + D v, then W v
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4 scale = *reinterpret_cast<const f32x4 *>(vec.out + 16 * m + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[m][e] = __builtin_fmaf(D, x[m][e], scale[e] * y[m][e]);
            }
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // row tiles with a fragment in block b: all four, but two in one of the blocks
                constexpr int kAll = kRev ? 1 : 0;
                auto frag = [&](int m) {
                    const E<T> *at = tri + (kRev ? tri_upper(m, b) : tri_lower(m, b)) * (kTri / kTriFrags);
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
                    mma_left<4>(y, a, fv[b]);
                } else {
                    constexpr int m0 = kRev ? 0 : 2;
                    const Sum<T, NW> a[2] = {frag(m0), frag(m0 + 1)};
                    mma_left<2>(y + m0, a, fv[b]);
                }
            }
        }
        // S = e^{Gc} S + R^T (scaled v)
        const float end = vec.end[0];
        Sum<T, NX> fx[2];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 scale = *reinterpret_cast<const f32x4 *>(vec.in + 16 * m + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[m][e] *= scale[e];
        }
        fx[0] = to_sum<T, NX>(x[0], x[1]);
        fx[1] = to_sum<T, NX>(x[2], x[3]);
#pragma unroll
        for (int m = 0; m < ND / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[m][e] *= end;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
                In<T> fr[2];
#pragma unroll
                for (int o = 0; o < 2; ++o)
                    fr[o] = tile_cols<T, NCH>(tileR, 32 * t2 + 4 * g, 32 * t2 + 16 + 4 * g,
                                              [&](int q) { return 32 * b + 8 * q + 4 * o; });
                mma_left<2>(S + 2 * b, fr, fx[t2]);
            }
        if constexpr (kOut) {
            const long long at = out_at + t * p.sout.t;
            if (p.out_bf16)
                store_column<bf16_t, false>(static_cast<bf16_t *>(p.out) + at, p.sout.t, rows, g, col, mine, y);
            else
                store_column<float, false>(static_cast<float *>(p.out) + at, p.sout.t, rows, g, col, mine, y);
        }
    }
    if constexpr (kEnd) {
        keep_state(end_to);
        if (blockIdx.z == 0 && wave == kWaves - 1 && l == 0) p.ws.decay[slot] = exp2_of(passed);
    } else if (p.sL && mine && last) {
#pragma unroll
        for (int m = 0; m < ND / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
                if (row < p.N) p.sL[state_at + (long long)row * p.P] = S[m][e];
            }
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
    if (segs < 2) return;
    f32x4 s = *place(0);
    for (int k = 1; k + 1 < segs; ++k) {
        const f32x4 end = *place(k);
        const float d = p.ws.decay[at(k)];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = __builtin_fmaf(d, s[e], end[e]);
        *place(k) = s;
    }
}

template <typename T, int ND, bool kRev, bool kFast>
hipError_t scan_run(const HeadsArgs &a, const HeadsScan &p, hipStream_t stream)
{
    const HeadsSplit split = heads_split(a.batch, a.seqlen, a.h, a.P, a.cu ? a.nseq : 0);
    const dim3 grid(split.segs ? split.segs : a.nseq, a.h, (a.P + kCols - 1) / kCols), block(kThreads);
    if (log_enabled())
        log_line("head_scan: heads_scan_kernel<%s, N %d, reverse %d, fast %d>, out %d, keep %d, grid (%u, %u, %u) x %u "
                 "threads, %d chunks a segment", type_tag<T>(), ND, int(kRev), int(kFast), int(p.out != nullptr),
                 int(p.keep != nullptr), grid.x, grid.y, grid.z, block.x, split.seg_chunks);
    if (split.segs) {
        heads_scan_kernel<T, ND, kEndRun, kRev, kFast><<<grid, block, 0, stream>>>(p);
        const dim3 parts(a.nseq, a.h, (p.ws.state / 4 + kThreads - 1) / kThreads);
        heads_compose_kernel<<<parts, block, 0, stream>>>(p, kRev);
    }
    if constexpr (kRev) {
        heads_scan_kernel<T, ND, kOutKeepRun, kRev, kFast><<<grid, block, 0, stream>>>(p);
    } else {
        if (p.out && p.keep) heads_scan_kernel<T, ND, kOutKeepRun, kRev, kFast><<<grid, block, 0, stream>>>(p);
        else if (p.out) heads_scan_kernel<T, ND, kOutRun, kRev, kFast><<<grid, block, 0, stream>>>(p);
        else heads_scan_kernel<T, ND, kKeepRun, kRev, kFast><<<grid, block, 0, stream>>>(p);
    }
    return hipGetLastError();
}

template <typename T, int ND>
hipError_t scan_sized(const HeadsArgs &a, const HeadsScan &p, bool reverse, bool fast, hipStream_t stream)
{
    if (reverse) return fast ? scan_run<T, ND, true, true>(a, p, stream) : scan_run<T, ND, true, false>(a, p, stream);
    return fast ? scan_run<T, ND, false, true>(a, p, stream) : scan_run<T, ND, false, false>(a, p, stream);
}

template <typename T>
hipError_t scan_typed(const HeadsArgs &a, const HeadsScan &p, bool reverse, bool fast, hipStream_t stream)
{
    const int nd = heads_nd(a.N);
    return nd == 64 ? scan_sized<T, 64>(a, p, reverse, fast, stream)
         : nd == 128 ? scan_sized<T, 128>(a, p, reverse, fast, stream)
                     : scan_sized<T, 256>(a, p, reverse, fast, stream);
}

}  // namespace

hipError_t launch_heads_scan(const HeadsArgs &a, const HeadsScan &p, bool reverse, hipStream_t stream)
{
    const bool bf16 = p.in_bf16 && p.v_bf16, same = p.in_bf16 == p.v_bf16;
    const int es = p.in_bf16 ? 2 : 4;
    const bool fast = same && heads_fast(p.L, p.sL_, a.N, es, a, a.groups) && heads_fast(p.R, p.sR, a.N, es, a, a.groups) &&
                      heads_fast(p.v, p.sv, a.P, es, a, a.h);
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
