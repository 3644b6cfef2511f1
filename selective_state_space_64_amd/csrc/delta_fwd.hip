// delta_fwd.hip -- the gated delta rule over whole sequences, a chunk of 64
// steps at a time on the matrix cores (gfx950; C ABI in include/ssm_delta.h).
//
// With G_i the sum of the chunk's log decays up to step i, S0 the state
// entering it, and U the rows beta_t (v_t - e^{g_t} S_{t-1}^T k_t):
//     M_ij = beta_i e^{G_i - G_j} k_i . k_j  (i > j),    T = (1 + M)^-1
//     P_ij = scale e^{G_i - G_j} q_i . k_j   (i >= j)
//     X = beta (V - e^G K S0),   U = T X
//     Y = scale e^G Q S0 + P U
//     S1 = e^{Gc} S0 + K^T (e^{Gc - G} U)
// M, T and P do not depend on the state: one workgroup per (chunk, head)
// makes them (delta_prep_kernel) and leaves T - 1 and P in the workspace in
// the order in which the matrix instruction reads them.  The columns of S
// (the value channels) are independent of one another, so the recurrence
// (delta_scan_kernel) gives each wave 16 columns of one head's state, kept in
// registers over the whole sequence; every product's result is the next
// one's right operand in place, and the four or eight waves of a workgroup
// share only the chunk's K, Q, T, P (and V) in LDS, which bf16 rows reach by
// copies that pass no register, a chunk ahead.
//
// Measured with 4 x 40 heads of 128 x 128, 2048 steps, bf16: 221 us a call.  By
// the profiler, under which each kernel takes a few us longer than its part of a
// call, the chunks' matrices take 71 us (the longest is the triangular inverse,
// products of 16 x 16 blocks after one another) and the recurrence 162 us, where
// the call's reads and writes alone would take 70.  No one thing bounds it: the matrix pipe is
// busy for about 36 % of it, LDS for 50 %, the vector ALU (conversions to
// terms) for 40 %, and taking any one phase away gains at most 30 us; the chain of
// products of a chunk (K S0, T X, P U, K^T U) leaves each wave waiting for its
// own results.  Two column tiles a wave to fill those waits need more registers
// than two waves a SIMD have (212 to 232 us).
#include "delta_chunk.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------ a chunk's matrices
struct PrepParams {
    int seqlen, nseq, rep, h, K;
    float scale;
    const int *cu;
    const void *q, *k;
    const float *g, *beta;
    DeltaStride sq, sk, sg, sbeta;
    DeltaWs ws;
};

constexpr int kPitch = 68;  // floats a row of the 64 x 64 matrices in LDS

// (r, b) of fragment f
__device__ inline void tri_place(bool upper, int f, int &r, int &b)
{
    if (upper) {
        r = f < 4 ? f >> 1 : f - 2;
        b = f < 4 ? f & 1 : 1;
    } else {
        r = f < 2 ? f : f >> 1;
        b = f < 2 ? 0 : f & 1;
    }
    if (!upper && f >= 2) r = f < 4 ? 2 : 3;
}

// The fragments of a lower-triangular matrix m (or of its transpose); entries
// with j + diag <= i are kept (diag 1: the strict part).
template <int N, bool kUpper>
__device__ inline void write_tri(const float *m, int diag, uint16_t *out)
{
    for (int it = int(threadIdx.x); it < kTriFrags * 64; it += kThreads) {
        const int f = it >> 6, l = it & 63;
        int r, b;
        tri_place(kUpper, f, r, b);
        const int row = 16 * r + (l & 15), g = l >> 4;
        float v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int col = 32 * b + 4 * g + (s & 3) + (s >= 4 ? 16 : 0);
            const int i = kUpper ? col : row, j = kUpper ? row : col;
            v[s] = j + diag <= i ? m[i * kPitch + j] : 0.0f;
        }
        const Frag<N> x = split8<N>(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
#pragma unroll
        for (int n = 0; n < N; ++n)
            *reinterpret_cast<bf16x8 *>(out + ((f * N + n) * 64 + l) * 8) = x.t[n];
    }
}

// 4 x 40 heads, 32 chunks of 64 x 128 in bf16 (168 MB in): 71 us by the
// profiler, with the transposes for the backward pass 90 us; bound by the
// inverse's chain, so four workgroups share a compute unit.
template <typename T, int KD, bool kBoth, bool kFast>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 && kFast ? 4 : 1)) void delta_prep_kernel(const PrepParams p)
{
    constexpr int NI = Terms<T>::kIn, NS = Terms<T>::kSum;
    constexpr int KH = KD < 128 ? KD : 128, NCH = KH / 8, kTile = 64 * KH;
    constexpr int kTiles = 2 * NI * kTile * 2, kMats = 2 * 64 * kPitch * 4;
    __shared__ __align__(16) unsigned char lds[kTiles > kMats ? kTiles : kMats];
    __shared__ double G[64];
    __shared__ float beta[64];
    uint16_t *kt = reinterpret_cast<uint16_t *>(lds), *qt = kt + NI * kTile;
    float *M = reinterpret_cast<float *>(lds), *P = M + 64 * kPitch, *Tm = P;

    const int chunk = int(blockIdx.x), head = int(blockIdx.y);
    const int si = delta_seq_of(p.cu, p.nseq, p.seqlen, chunk);
    const DeltaSeq sq = delta_seq(p.cu, si, p.seqlen);
    const int at = (chunk - sq.chunk0) * kDeltaChunk;  // the chunk's first step in its sequence
    const int rows = min(kDeltaChunk, sq.len - at);
    if (at < 0 || rows <= 0) return;  // the whole workgroup: a record that no chunk uses
    uint16_t *out = p.ws.prep + ((long long)chunk * p.h + head) * p.ws.prep_stride;
    const long long t0 = sq.first + at;
    const int tid = int(threadIdx.x), wave = tid >> 6, l = tid & 63, r = l & 15, g = l >> 4;

    if (wave == 0) {
        float gi = 0.0f, bi = 0.0f;
        if (l < rows) {
            gi = p.g[sq.batch * p.sg.b + (t0 + l) * p.sg.t + head * p.sg.h];
            bi = p.beta[sq.batch * p.sbeta.b + (t0 + l) * p.sbeta.t + head * p.sbeta.h];
        }
        const double sum = decay_sums(gi);
        G[l] = sum;
        beta[l] = bi;
        const double last = __shfl(sum, 63);
        const float eg = exp2_hw(float(sum) * kLog2e);
        float *vec = reinterpret_cast<float *>(out + 2 * tri_size(NS));
        vec[l] = eg;
        vec[64 + l] = exp2_hw(float(last - sum) * kLog2e);
        vec[128 + l] = bi * eg;
        vec[192 + l] = bi;
    }

    // K K^T and Q K^T: wave w the tiles (w, 0..w)
    const T *kp = static_cast<const T *>(p.k) + sq.batch * p.sk.b + t0 * p.sk.t + (head / p.rep) * p.sk.h;
    const T *qp = static_cast<const T *>(p.q) + sq.batch * p.sq.b + t0 * p.sq.t + (head / p.rep) * p.sq.h;
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) kk[c] = qk[c] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int half = 0; half < KD / KH; ++half) {
        TileLoad<T, NCH, kThreads, kFast> lk, lq;
        lk.init(p.sk.t, p.K - half * KH);
        lq.init(p.sq.t, p.K - half * KH);
        lk.fetch(kp + half * KH, p.sk.t, rows, p.K - half * KH);
        lq.fetch(qp + half * KH, p.sq.t, rows, p.K - half * KH);
        if (half) __syncthreads();
        lk.template store<NI>(kt, rows, p.K - half * KH);
        lq.template store<NI>(qt, rows, p.K - half * KH);
        __syncthreads();
#pragma unroll
        for (int b = 0; b < KH / 32; ++b) {
            Frag<NI> ka, qa;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                ka.t[n] = read_row<NCH>(kt + n * kTile, 16 * wave + r, 4 * b + g);
                qa.t[n] = read_row<NCH>(qt + n * kTile, 16 * wave + r, 4 * b + g);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c <= wave) {
                    Frag<NI> kb;
#pragma unroll
                    for (int n = 0; n < NI; ++n)
                        kb.t[n] = read_row<NCH>(kt + n * kTile, 16 * c + r, 4 * b + g);
                    kk[c] = mma<NI, NI>(ka, kb, kk[c]);
                    qk[c] = mma<NI, NI>(qa, kb, qk[c]);
                    settle();
                }
        }
    }
    __syncthreads();  // K, Q are read: M, P, T take their place
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c <= wave) {
            const int j = 16 * c + r;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * wave + 4 * g + e;
                const float d = i >= j ? exp2_hw(float(G[i] - G[j]) * kLog2e) : 0.0f;
                M[i * kPitch + j] = i > j ? beta[i] * d * kk[c][e] : 0.0f;
                P[i * kPitch + j] = i >= j ? p.scale * d * qk[c][e] : 0.0f;
            }
        }
    __syncthreads();

    // P leaves, T takes its place.  T's diagonal blocks by forward substitution,
    // lane r one column (the four lane groups alike); every finished entry is
    // taken from those below it, which do not wait for one another.
    write_tri<NS, false>(P, 0, out + tri_size(NS));
    if constexpr (kBoth) write_tri<NS, true>(P, 0, out + 3 * tri_size(NS) + 512);
    {
        const float *m = M + (16 * wave) * kPitch + 16 * wave;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = i == r ? 1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < 15; ++j)
#pragma unroll
            for (int i = j + 1; i < 16; ++i) t[i] = __builtin_fmaf(-m[i * kPitch + j], t[j], t[i]);
        __syncthreads();  // P is read
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) Tm[(16 * wave + i) * kPitch + 16 * wave + r] = t[i];
        }
    }
    __syncthreads();
    // then the blocks below, T_ij = -T_ii sum_m M_im T_mj, in fp32 matrix
    // instructions: distance d = i - j at a time, wave i its row
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        if (wave >= d) {
            const int j = wave - d;
            f32x4 acc = {0, 0, 0, 0}, res = {0, 0, 0, 0};
#pragma unroll
            for (int n = 0; n < d; ++n) {
                const int m = j + n;
                const f32x4 a = *reinterpret_cast<const f32x4 *>(M + (16 * wave + r) * kPitch + 16 * m + 4 * g);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    acc = mfma16_f32(a[s], Tm[(16 * m + 4 * g + s) * kPitch + 16 * j + r], acc);
            }
            const f32x4 a = *reinterpret_cast<const f32x4 *>(Tm + (16 * wave + r) * kPitch + 16 * wave + 4 * g);
#pragma unroll
            for (int s = 0; s < 4; ++s) res = mfma16_f32(a[s], acc[s], res);
#pragma unroll
            for (int e = 0; e < 4; ++e) Tm[(16 * wave + 4 * g + e) * kPitch + 16 * j + r] = -res[e];
        }
        __syncthreads();
    }
    write_tri<NS, false>(Tm, 1, out);
    if constexpr (kBoth) write_tri<NS, true>(Tm, 1, out + 2 * tri_size(NS) + 512);
}

// ------------------------------------------------------------ the recurrence
struct ScanParams {
    int seqlen, nseq, rep, h, K, V, Vp;
    int out_bf16;
    float scale;
    const int *cu;
    const void *q, *k, *v;
    const float *h0;
    void *y;
    float *hL;
    DeltaStride sq, sk, sv, sy;
    DeltaWs ws;
};

// What a run of the recurrence leaves: y and hL; beside them S0 and U of every
// chunk; or only a segment's end state and transfer matrix.
enum { kPlainRun = 0, kKeepRun = 1, kEndRun = 2 };

template <typename T, int KD, int kWaves, int kRun, int kPath>
__global__ __launch_bounds__(64 * kWaves, (kWaves == 8 ? 2 : 1)) void delta_scan_kernel(const ScanParams p)
{
    constexpr bool kFast = kPath >= kByRun, kAsync = kPath == kByCopy, kKeep = kRun == kKeepRun, kEnd = kRun == kEndRun;
    using Stage = ChunkStage<T, KD, kWaves, kFast, kAsync, false, !kEnd>;
    constexpr int NI = Stage::NI, NS = Stage::NS, NCH = Stage::NCH, kTile = Stage::kTile, KB = KD / 32;
    constexpr int kKept = kKeep ? (KB + 2) * NS : 0;  // stores of a chunk beside y's 16
    __shared__ __align__(16) uint16_t lds[Stage::kBuffers * Stage::kBuffer];

    const int head = int(blockIdx.y), l = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6), r = l & 15, g = l >> 4;
    const DeltaSegment seg = delta_segment(p.cu, p.nseq, p.seqlen, p.ws.seg_chunks, int(blockIdx.z));
    const DeltaSeq &seq = seg.s;
    // kEnd: the workgroups behind the value columns run the unit columns
    const int value_wgs = (p.V + 16 * kWaves - 1) / (16 * kWaves);
    const bool unit = kEnd && int(blockIdx.x) >= value_wgs;
    if (!seg.live) return;                                       // the whole workgroup
    if (kEnd && (seg.last || (unit && seg.index == 0))) return;  // nothing follows, or nothing enters it
    const int col_tile = (int(blockIdx.x) - (unit ? value_wgs : 0)) * kWaves + wave, col = 16 * col_tile + r;
    const bool mine = !unit && col < p.V, kept = 16 * col_tile < p.Vp;  // the record has whole tiles up to Vp
    const int c0 = seg.c0, chunks = seg.c1;
    const long long state_at = ((long long)seg.seq * p.h + head) * p.K * (long long)p.V + col;
    const long long rec0 = (long long)seq.chunk0 * p.h + head;
    // this segment's place in N and M, and the state entering it: the composed one, h0
    // as the ends' run kept it, or h0 itself where this workgroup also writes hL
    const long long slot = (long long)blockIdx.z * p.h + head;
    float *const first_entry = p.ws.N + (slot + (long long)seg.behind * p.h) * p.ws.state + col;
    const float *entry = seg.index ? p.ws.N + (slot - p.h) * p.ws.state + col : nullptr;
    if (!kEnd && !seg.index && seg.behind && p.h0) entry = first_entry;

    Stage st;
    st.init(lds, static_cast<const T *>(p.k) + seq.batch * p.sk.b + seq.first * p.sk.t + (head / p.rep) * p.sk.h, p.sk.t,
            static_cast<const T *>(p.q) + seq.batch * p.sq.b + seq.first * p.sq.t + (head / p.rep) * p.sq.h, p.sq.t,
            p.ws.prep + rec0 * p.ws.prep_stride, p.h * p.ws.prep_stride, seq.len, p.K);
    const T *vp = static_cast<const T *>(p.v) + seq.batch * p.sv.b + seq.first * p.sv.t + head * p.sv.h;
    if constexpr (kAsync) {
        const int first = int(blockIdx.x) * 16 * kWaves;
        st.init_columns(vp + first, p.sv.t, unit ? 0 : p.V - first);
    }
    const long long y0 = seq.batch * p.sy.b + seq.first * p.sy.t + head * p.sy.h;

    // S: tiles 2 b and 2 b + 1 hold the rows 32 b + 8 g + {0..3} and + {4..7}
    f32x4 S[KD / 16];
#pragma unroll
    for (int m = 0; m < KD / 16; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
            float s = 0.0f;
            if (kEnd ? seg.index != 0 : false) s = unit && row == col ? 1.0f : 0.0f;
            else if (entry) s = kept ? entry[(long long)row * p.Vp] : 0.0f;
            else if (p.h0 && mine && row < p.K) s = p.h0[state_at + (long long)row * p.V];
            S[m][e] = s;
        }
    if (kEnd && !seg.index && p.h0 && kept) {
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                first_entry[(long long)(32 * (m / 2) + 8 * g + 4 * (m % 2) + e) * p.Vp] = S[m][e];
    }

    Column<T, kFast> lc;
    if (chunks > c0) {
        const long long t = (long long)c0 * kDeltaChunk;
        st.start(c0);
        if constexpr (!kAsync) lc.fetch(vp + t * p.sv.t, p.sv.t, seq.len - c0 * kDeltaChunk, g, col, mine);
    }
    for (int c = c0; c < chunks; ++c) {
        const int rows = seq.len - c * kDeltaChunk;
        const long long t = (long long)c * kDeltaChunk, rec = rec0 + (long long)c * p.h;
        if constexpr (kAsync) {  // all but the stores that the last chunk made behind the copies
            if (kEnd || c == c0 || (!kept && !p.y)) wait_loads<0>();
            else if (!kept) wait_loads<16>();
            else if (p.y) wait_loads<kKept + 16>();
            else wait_loads<kKept>();
        }
        st.store(c);
        f32x4 X[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (kAsync) X[m] = st.column(c, m);
            else X[m] = lc.tile(m, rows, g, mine);
        }
        constexpr bool kOther = Stage::kOneTile && !kEnd;  // K takes Q's place after Q S
        if (c + 1 < chunks) {
            if constexpr (!kOther) st.start(c + 1);
            if constexpr (!kAsync)
                lc.fetch(vp + (t + kDeltaChunk) * p.sv.t, p.sv.t, rows - kDeltaChunk, g, col, mine);
        }
        const uint16_t *kt = st.k_tile(c), *qt = st.q_tile(c), *tt = st.first(c), *pt = st.second(c);
        const float *vec = st.vec(c);

        // K S and Q S.  Each phase's fragments are read while the phase before
        // it computes (the fences keep the reads ahead of those products).
        f32x4 ks[4], qs[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) ks[m] = qs[m] = f32x4{0, 0, 0, 0};
        Frag<NI> ka[2][4], qa[2][4];
        Frag<NS> tf[kTriFrags], pf[kTriFrags];
        auto read_kq = [&](int b) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NI; ++n) {
                    ka[b & 1][m].t[n] = read_row<NCH>(kt + n * kTile, 16 * m + r, 4 * b + g);
                    if constexpr (!kEnd && !kOther)
                        qa[b & 1][m].t[n] = read_row<NCH>(qt + n * kTile, 16 * m + r, 4 * b + g);
                }
        };
        auto read_tri = [&](const uint16_t *from, Frag<NS> *to) {
#pragma unroll
            for (int i = 0; i < kTriFrags; ++i)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    to[i].t[n] = *reinterpret_cast<const bf16x8 *>(from + ((i * NS + n) * 64 + l) * 8);
        };
        if constexpr (kOther) {
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                read_kq(b);
                const Frag<NS> sb = split8<NS>(S[2 * b], S[2 * b + 1]);
#pragma unroll
                for (int m = 0; m < 4; ++m) qs[m] = mma<NI, NS>(ka[b & 1][m], sb, qs[m]);
            }
            st.store_other(c);
            if (c + 1 < chunks) st.start(c + 1);
        }
        read_kq(0);
        Frag<NS> sb[2];
        sb[0] = split8<NS>(S[0], S[1]);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            if (b + 1 < KB) {
                read_kq(b + 1);
                sb[(b + 1) & 1] = split8<NS>(S[2 * b + 2], S[2 * b + 3]);
            } else {
                read_tri(tt, tf);
            }
            if constexpr (kKeep)
                if (kept) record_store<NS, KB>(p.ws.S0 + rec * NS * p.ws.state, col_tile, b, sb[b & 1]);
            for_terms<NI, NS>([&](int i, int j) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    ks[m] = mfma16(ka[b & 1][m].t[i], sb[b & 1].t[j], ks[m]);
                    if constexpr (!kEnd && !kOther) qs[m] = mfma16(qa[b & 1][m].t[i], sb[b & 1].t[j], qs[m]);
                }
            });
            interleave<(kEnd || kOther ? 4 : 8) * NI, 8 * NS, 3>();
        }
        // X = beta V - beta e^G K S;  U = X + (T - 1) X
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 be = *reinterpret_cast<const f32x4 *>(vec + 128 + 16 * m + 4 * g);
            const f32x4 bt = *reinterpret_cast<const f32x4 *>(vec + 192 + 16 * m + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) X[m][e] = __builtin_fmaf(bt[e], X[m][e], -be[e] * ks[m][e]);
        }
        f32x4 U[4];
        const float ec = vec[63];
        {
            const Frag<NS> xb[2] = {split8<NS>(X[0], X[1]), split8<NS>(X[2], X[3])};
            fence();
            if constexpr (!kEnd) read_tri(pt, pf);
#pragma unroll
            for (int m = 0; m < 4; ++m) U[m] = X[m];
            for_terms<NS, NS>([&](int i, int j) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 2 * b; m < 4; ++m) U[m] = mfma16(tf[tri_lower(m, b)].t[i], xb[b].t[j], U[m]);
            });
            // beside them: Q S and S take their decays
            if constexpr (!kEnd) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const f32x4 eg = *reinterpret_cast<const f32x4 *>(vec + 16 * m + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) qs[m][e] *= p.scale * eg[e];
                }
            }
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][e] *= ec;
            interleave<(kEnd ? 0 : 6 * NS + 4), 18, 3>();
        }
        // Y = scale e^G Q S + P U;  beside it e^{Gc - G} U
        Frag<NI> kc[2][2][2];  // K^T: [step parity][tile of the pair][time block]
        auto read_kc = [&](int b) {
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NI; ++n)
                        kc[b & 1][o][i].t[n] = read_cols<NCH>(kt + n * kTile, 32 * i + 4 * g, 32 * i + 16 + 4 * g,
                                                              32 * b + 8 * (r & 3) + 4 * o);
        };
        Frag<NS> wb[2];
        auto tailed = [&]() {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4 tail = *reinterpret_cast<const f32x4 *>(vec + 64 + 16 * m + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) U[m][e] *= tail[e];
            }
            wb[0] = split8<NS>(U[0], U[1]);
            wb[1] = split8<NS>(U[2], U[3]);
        };
        if constexpr (!kEnd) {
            const Frag<NS> ub[2] = {split8<NS>(U[0], U[1]), split8<NS>(U[2], U[3])};
            if constexpr (kKeep)
                if (kept) {
                    record_store<NS, 2>(p.ws.U + rec * NS * p.ws.step, col_tile, 0, ub[0]);
                    record_store<NS, 2>(p.ws.U + rec * NS * p.ws.step, col_tile, 1, ub[1]);
                }
            fence();
            read_kc(0);
            for_terms<NS, NS>([&](int i, int j) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 2 * b; m < 4; ++m) qs[m] = mfma16(pf[tri_lower(m, b)].t[i], ub[b].t[j], qs[m]);
            });
            tailed();
            interleave<8 * NI + 4, 18, 4>();
            fence();
        } else {
            read_kc(0);
            tailed();
        }
        // S = e^{Gc} S + K^T (e^{Gc - G} U);  beside it the stores of Y
        if constexpr (!kEnd) {
            const long long at = y0 + t * p.sy.t;
            if (p.y && p.out_bf16)
                store_column<bf16_t, kFast>(static_cast<bf16_t *>(p.y) + at, p.sy.t, rows, g, col, mine, qs);
            else if (p.y)
                store_column<float, kFast>(static_cast<float *>(p.y) + at, p.sy.t, rows, g, col, mine, qs);
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            if (b + 1 < KB) read_kc(b + 1);
            for_terms<NI, NS>([&](int i, int j) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int o = 0; o < 2; ++o) S[2 * b + o] = mfma16(kc[b & 1][o][t].t[i], wb[t].t[j], S[2 * b + o]);
            });
            interleave<8 * NI, 4 * NS, 0>();
        }
    }
    if constexpr (kEnd) {
        if (unit) {  // row-major terms, as the composition reads them
            uint16_t *out = p.ws.M + slot * 3 * KD * KD + col;
            if (col < KD) {
#pragma unroll
                for (int m = 0; m < KD / 16; ++m)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
                        float x = S[m][e], y = S[m][e + 1];
#pragma unroll
                        for (int n = 0; n < NS; ++n) {
                            const uint32_t w = split_pair(x, y);
                            out[(n * KD + row) * KD] = uint16_t(w);
                            out[(n * KD + row + 1) * KD] = uint16_t(w >> 16);
                        }
                    }
            }
        } else if (kept) {
            float *out = p.ws.N + slot * p.ws.state + col;
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    out[(long long)(32 * (m / 2) + 8 * g + 4 * (m % 2) + e) * p.Vp] = S[m][e];
        }
    } else if (p.hL && mine && seg.last) {
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
                if (row < p.K) p.hL[state_at + (long long)row * p.V] = S[m][e];
            }
    }
}

// ------------------------------------------------------------ the split's composition
// entry_{s+1} = M_s entry_s + N_s over one sequence's segments, in place of
// N_s.  entry_1 is N_0.  A wave holds 16 columns, as in the recurrence; M's
// terms come to LDS for the workgroup's four waves, a segment ahead where two
// of them fit.  A chain of products, 3 to 4 us a segment (12 heads of 65521
// steps in 21 segments: 74 us of 850 to 890).
template <typename T, int KD>
__global__ __launch_bounds__(256) void delta_compose_kernel(const ScanParams p)
{
    constexpr int NS = Terms<T>::kSum, NCH = KD / 8, KB = KD / 32, kTile = KD * KD;
    constexpr int kPlanes = KD > 128 ? 1 : NS;  // of M in LDS at a time
    constexpr int kBuffers = 2 * kPlanes * kTile * 2 <= 160 * 1024 ? 2 : 1;
    __shared__ __align__(16) uint16_t lds[kBuffers * kPlanes * kTile];
    const int head = int(blockIdx.y), tid = int(threadIdx.x), l = tid & 63, r = l & 15, g = l >> 4;
    const int col = int(blockIdx.x) * 64 + 16 * (tid >> 6) + r;  // below Vp: a multiple of 64
    const DeltaSeq seq = delta_seq(p.cu, int(blockIdx.z), p.seqlen);
    const int per = (p.seqlen + kDeltaChunk - 1) / kDeltaChunk, L = p.ws.seg_chunks;
    const int chunks = (seq.len + kDeltaChunk - 1) / kDeltaChunk, segs = (chunks + L - 1) / L;
    const long long z0 = p.cu ? seq.chunk0 / L + int(blockIdx.z) : (long long)blockIdx.z * ((per + L - 1) / L);

    f32x4 S[KD / 16], N[KD / 16];
    auto load = [&](int s, f32x4 *to) {
        const float *n = p.ws.N + ((z0 + s) * p.h + head) * p.ws.state + col;
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                to[m][e] = n[(long long)(32 * (m / 2) + 8 * g + 4 * (m % 2) + e) * p.Vp];
    };
    // terms [first, first + kPlanes) of M_s, rows' chunks in the tiles' order
    constexpr int kRows = 256 / NCH;
    uint32_t off[2];  // of even and odd runs of rows: their order differs where a run has 8
#pragma unroll
    for (int i = 0; i < 2; ++i)
        off[i] = uint32_t(tid / NCH * NCH + (chunk_at<NCH>(tid / NCH + i * kRows, tid % NCH) / 8) % NCH) * 16;
    auto copy = [&](int s, int first) {
        const uint16_t *M = p.ws.M + ((z0 + s) * p.h + head) * 3 * kTile + first * kTile;
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds_offset(lds)) + wave_of() * 1024 +
                            (kBuffers == 2 ? (s & 1) * kPlanes * kTile * 2 : 0);
        const sgpr4 buf = copy_buffer(M, kPlanes * kTile * 2);
        for (int i = 0; i < kPlanes * KD / kRows; i += 2) {
            copy_to_lds(buf, off[0] + i * 4096, to + i * 4096);
            copy_to_lds(buf, off[1] + (i + 1) * 4096, to + (i + 1) * 4096);
        }
    };
    static_assert(2 * kRows % 16 == 0 && KD / kRows % 2 == 0, "the same order in every second run");
    if (segs > 1) load(0, S);
    if (kBuffers == 2 && segs > 2) copy(1, 0);
    for (int s = 1; s + 1 < segs; ++s) {
        load(s, N);
        const uint16_t *tile = lds + (kBuffers == 2 ? (s & 1) * kPlanes * kTile : 0);
        Frag<NS> sb[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) sb[b] = split8<NS>(S[2 * b], S[2 * b + 1]);
#pragma unroll
        for (int first = 0; first < NS; first += kPlanes) {
            if constexpr (kBuffers == 1) {
                __syncthreads();  // the last reads are done
                copy(s, first);
            }
            wait_loads<0>();
            __syncthreads();
            if (kBuffers == 2 && s + 2 < segs) copy(s + 1, 0);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m) {
                const int row = 32 * (m / 2) + 8 * (r >> 2) + 4 * (m % 2) + (r & 3);
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    if constexpr (kPlanes == NS) {
                        Frag<NS> a;
#pragma unroll
                        for (int n = 0; n < NS; ++n) a.t[n] = read_row<NCH>(tile + n * kTile, row, 4 * b + g);
                        N[m] = mma<NS, NS>(a, sb[b], N[m]);
                    } else {  // one term of M: the pairs that it stands in, as in for_terms
                        const bf16x8 a = read_row<NCH>(tile, row, 4 * b + g);
#pragma unroll
                        for (int n = 0; n < NS; ++n)
                            if (first + n <= kTermOrder<NS, NS>) N[m] = mfma16(a, sb[b].t[n], N[m]);
                    }
                }
            }
        }
        float *out = p.ws.N + ((z0 + s) * p.h + head) * p.ws.state + col;
#pragma unroll
        for (int m = 0; m < KD / 16; ++m) {
            S[m] = N[m];
#pragma unroll
            for (int e = 0; e < 4; ++e) out[(long long)(32 * (m / 2) + 8 * g + 4 * (m % 2) + e) * p.Vp] = S[m][e];
        }
    }
}

template <typename T, int KD>
hipError_t prep_kd(const DeltaArgs &a, const PrepParams &p, bool both, bool fast, hipStream_t stream)
{
    const dim3 grid(unsigned(delta_chunks(a.batch, a.seqlen, a.cu ? a.nseq : 0)), a.h);
    if (log_enabled())
        log_line("delta_prep: delta_prep_kernel<in %s, K %d, transposes %d, fast %d>, grid (%u, %u) x %d threads",
                 type_tag<T>(), KD, int(both), int(fast), grid.x, grid.y, kThreads);
    if (both && fast) delta_prep_kernel<T, KD, true, true><<<grid, dim3(kThreads), 0, stream>>>(p);
    else if (both) delta_prep_kernel<T, KD, true, false><<<grid, dim3(kThreads), 0, stream>>>(p);
    else if (fast) delta_prep_kernel<T, KD, false, true><<<grid, dim3(kThreads), 0, stream>>>(p);
    else delta_prep_kernel<T, KD, false, false><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, int KD, int kWaves, int kPath>
hipError_t scan_waves(const DeltaArgs &a, const ScanParams &p, hipStream_t stream)
{
    const DeltaSplit split = delta_split(a.batch, a.seqlen, a.h, a.V, a.cu ? a.nseq : 0);
    const int tiles = (a.V + 16 * kWaves - 1) / (16 * kWaves);
    const dim3 grid(tiles, a.h, split.segs ? split.segs : a.nseq), block(64 * kWaves);
    if (log_enabled())
        log_line("delta_fwd: delta_scan_kernel<in %s, K %d, waves %d, keep %d, path %d>, grid (%u, %u, %u) x %u threads, "
                 "%d chunks a segment", type_tag<T>(), KD, kWaves, int(p.ws.S0 != nullptr), kPath, grid.x, grid.y,
                 grid.z, block.x, split.seg_chunks);
    if (split.segs) {
        const dim3 ends(tiles + (KD + 16 * kWaves - 1) / (16 * kWaves), a.h, split.segs), compose(p.Vp / 64, a.h, a.nseq);
        delta_scan_kernel<T, KD, kWaves, kEndRun, kPath><<<ends, block, 0, stream>>>(p);
        delta_compose_kernel<T, KD><<<compose, dim3(256), 0, stream>>>(p);
    }
    if (p.ws.S0) delta_scan_kernel<T, KD, kWaves, kKeepRun, kPath><<<grid, block, 0, stream>>>(p);
    else delta_scan_kernel<T, KD, kWaves, kPlainRun, kPath><<<grid, block, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, int KD>
hipError_t scan_kd(const DeltaArgs &a, const ScanParams &p, int path, hipStream_t stream)
{
    if (path == kByElement) return scan_waves<T, KD, 4, kByElement>(a, p, stream);
    if constexpr (kDeltaAsync<T, KD>) {
        if (path == kByCopy && delta_wide(a, p.ws.seg_chunks)) return scan_waves<T, KD, 8, kByCopy>(a, p, stream);
        if (path == kByCopy) return scan_waves<T, KD, 4, kByCopy>(a, p, stream);
    }
    return scan_waves<T, KD, 4, kByRun>(a, p, stream);
}

}  // namespace

hipError_t launch_delta_prep(const DeltaArgs &a, const DeltaWs &ws, bool both, hipStream_t stream)
{
    const int es = a.in_bf16 ? 2 : 4;
    const PrepParams p{a.seqlen, a.nseq, a.h / a.hk, a.h, a.K, a.scale, a.cu, a.q, a.k, a.g, a.beta,
                       a.sq, a.sk, a.sg, a.sbeta, ws};
    const bool fast = delta_fast(a.q, a.sq, a.K, es, a, a.hk) && delta_fast(a.k, a.sk, a.K, es, a, a.hk);
    return delta_dispatch(a.in_bf16, true, a.K, [&](auto t, auto, auto kd) {
        return prep_kd<decltype(t), decltype(kd)::value>(a, p, both, fast, stream);
    });
}

hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaWs &ws, hipStream_t stream)
{
    const int es = a.in_bf16 ? 2 : 4;
    const ScanParams p{a.seqlen, a.nseq, a.h / a.hk, a.h, a.K, a.V, delta_vp(a.V), a.out_bf16, a.scale, a.cu, a.q, a.k,
                       a.v, a.h0, a.y, a.hL, a.sq, a.sk, a.sv, a.sy, ws};
    // the columns of v and y need no 16-byte accesses, only 64 steps in one buffer
    constexpr long long most = (1ll << 31) / 64 / 4;
    const bool fast = delta_fast(a.q, a.sq, a.K, es, a, a.hk) && delta_fast(a.k, a.sk, a.K, es, a, a.hk) &&
                      a.sv.t < most && a.sy.t < most;
    const int path = !fast ? kByElement : delta_fast(a.v, a.sv, a.V, es, a, a.h) ? kByCopy : kByRun;
    return delta_dispatch(a.in_bf16, true, a.K, [&](auto t, auto, auto kd) {
        return scan_kd<decltype(t), decltype(kd)::value>(a, p, path, stream);
    });
}

size_t delta_fwd_workspace_bytes(int batch, int seqlen, int hk, int h, int K, int V, int num_seqs)
{
    size_t bytes = 0;
    delta_ws(nullptr, batch, seqlen, h, K, V, num_seqs, false, &bytes);
    return bytes;
}

hipError_t launch_delta_fwd(const DeltaArgs &a, hipStream_t stream)
{
    const DeltaWs ws = delta_ws(a, a.checkpoints);
    const hipError_t e = launch_delta_prep(a, ws, a.checkpoints, stream);
    return e == hipSuccess ? launch_delta_scan(a, ws, stream) : e;
}

}  // namespace ssm
