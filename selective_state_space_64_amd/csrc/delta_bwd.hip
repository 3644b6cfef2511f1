// delta_bwd.hip -- gradients of the gated delta rule (gfx950; C ABI in
// include/ssm_delta.h).
//
// In the chunk form of delta_fwd.hip, with dS1 the gradient of the state
// leaving the chunk (tail = e^{Gc - G}):
//     dU = P^T dY + tail (K dS1),   dX = T^T dU,   dV = beta dX
//     dS0 = e^{Gc} dS1 + Q^T (scale e^G dY) - K^T (beta e^G dX)
// is a recurrence over the chunks from last to first whose columns are
// independent, as the forward's: delta_scan_bwd_kernel runs it with the state's
// gradient in registers and leaves dS1 and dX of every chunk in the
// workspace, beside the forward's S0 and U.  What sums over the value
// channels is then done for all chunks at once (delta_grad_kernel):
//     dP = scale Gam (dY U^T) (i >= j),   dM = -Gam (dX U^T) (i > j),
//     dQ = scale e^G (dY S0^T) + dP K
//     dK = tail (U dS1^T) - beta e^G (dX S0^T) + dP^T Q + (N + N^T) K,
//          N = beta dM
//     dbeta = dX . V - e^G k . (dX S0^T) + rowsum(dM (K K^T))
// with Gam_ij = e^{G_i - G_j}.  A log decay g_m stands in every exponential
// that spans step m, so its gradient is the sum over those terms only (no
// difference of running sums):
//     dg_m = sum_{i >= m > j} W_ij + sum_{i >= m} (scale e^{G_i} q_i.(dY S0^T)_i
//            - beta_i e^{G_i} k_i.(dX S0^T)_i) + sum_{j < m} tail_j k_j.(U dS1^T)_j
//            + e^{Gc} <S0, dS1>,      W = dP (Q K^T) + N (K K^T)
//
// Measured with 4 x 40 heads of 128 x 128, 2048 steps, bf16: 986 us a training
// step.  By the profiler (a few us longer for each kernel) the forward's part takes
// 90 + 255 us, the reverse recurrence 286 us and the gradients 399 us.
// Both are bound by the records between them: S0 and dS1 of
// two terms are 64 KB each a chunk and head, 330 MB each here, and U and dX
// another 170 MB each, written once and read once (410 us of the 986 at the
// rate of a large copy); recomputing S0 from fewer kept chunks would trade them
// for another forward recurrence of 160 us.  No atomics: a chunk and key head
// is one workgroup, so results do not change from run to run.
#include "delta_chunk.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

// bf16 terms of dY
template <typename T, typename TG>
constexpr int kGradTerms = sizeof(TG) == 2 ? 1 : Terms<T>::kSum;

template <typename TG> __device__ inline void store_grad(TG *p, float v)
{
    if constexpr (sizeof(TG) == 2) p->bits = uint16_t(pack_bf16x2(v, v));
    else *p = v;
}

// ------------------------------------------------------------ the recurrence
struct ScanBwdParams {
    int seqlen, rep, h, K, V, Vp;
    float scale;
    const int *cu;
    const void *q, *k, *dy;
    const float *dhL;
    void *dv;
    float *dh0;
    DeltaStride sq, sk, sdy, sdv;
    DeltaWs ws;
};

template <typename T, typename TG, int KD, int kWaves, int kPath>
__global__ __launch_bounds__(64 * kWaves, (kWaves == 8 ? 2 : 1)) void delta_scan_bwd_kernel(const ScanBwdParams p)
{
    constexpr bool kFast = kPath >= kByRun, kAsync = kPath == kByCopy;
    using Stage = ChunkStage<T, KD, kWaves, kFast, kAsync, true, true>;
    constexpr int NI = Stage::NI, NS = Stage::NS, NG = kGradTerms<T, TG>;
    constexpr int NCH = Stage::NCH, kTile = Stage::kTile, KB = KD / 32;
    constexpr int kKept = (KB + 2) * NS;  // stores of a chunk beside dv's 16
    __shared__ __align__(16) uint16_t lds[Stage::kBuffers * Stage::kBuffer];

    const int head = int(blockIdx.y), l = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6), r = l & 15, g = l >> 4;
    const int col_tile = int(blockIdx.x) * kWaves + wave, col = 16 * col_tile + r;
    const bool mine = col < p.V, kept = 16 * col_tile < p.Vp;  // the record has whole tiles up to Vp
    const DeltaSeq seq = delta_seq(p.cu, int(blockIdx.z), p.seqlen);
    const int chunks = (seq.len + kDeltaChunk - 1) / kDeltaChunk;
    const long long state_at = ((long long)blockIdx.z * p.h + head) * p.K * (long long)p.V + col;
    const long long rec0 = (long long)seq.chunk0 * p.h + head;

    Stage st;
    st.init(lds, static_cast<const T *>(p.k) + seq.batch * p.sk.b + seq.first * p.sk.t + (head / p.rep) * p.sk.h, p.sk.t,
            static_cast<const T *>(p.q) + seq.batch * p.sq.b + seq.first * p.sq.t + (head / p.rep) * p.sq.h, p.sq.t,
            p.ws.prep + rec0 * p.ws.prep_stride, p.h * p.ws.prep_stride, seq.len, p.K);
    const TG *yp = static_cast<const TG *>(p.dy) + seq.batch * p.sdy.b + seq.first * p.sdy.t + head * p.sdy.h;
    if constexpr (kAsync) {
        const int first = int(blockIdx.x) * 16 * kWaves;
        st.init_columns(yp + first, p.sdy.t, p.V - first);
    }
    TG *vp = static_cast<TG *>(p.dv) + seq.batch * p.sdv.b + seq.first * p.sdv.t + head * p.sdv.h;

    // dS, laid out as S in the forward
    f32x4 S[KD / 16];
#pragma unroll
    for (int m = 0; m < KD / 16; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
            S[m][e] = p.dhL && mine && row < p.K ? p.dhL[state_at + (long long)row * p.V] : 0.0f;
        }

    Column<TG, kFast> lc;
    constexpr bool kOther = Stage::kOneTile;  // Q takes K's place at the end of a chunk
    auto fetch = [&](int c) {
        if (!kOther || c == chunks - 1) st.start(c);
        const long long t = (long long)c * kDeltaChunk;
        if constexpr (!kAsync) lc.fetch(yp + t * p.sdy.t, p.sdy.t, seq.len - c * kDeltaChunk, g, col, mine);
    };
    if (chunks > 0) fetch(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
        const int rows = seq.len - c * kDeltaChunk;
        const long long t = (long long)c * kDeltaChunk, rec = rec0 + (long long)c * p.h;
        if constexpr (kAsync) {  // all but the stores that the last chunk made behind the copies
            if (c == chunks - 1) wait_loads<0>();
            else if (!kept) wait_loads<16>();
            else wait_loads<kKept + 16>();
        }
        st.store(c);
        f32x4 Y[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (kAsync) Y[m] = st.column(c, m);
            else Y[m] = lc.tile(m, rows, g, mine);
        }
        if (c > 0) fetch(c - 1);
        const uint16_t *kt = st.k_tile(c), *qt = st.q_tile(c), *tt = st.first(c), *pt = st.second(c);
        const float *vec = st.vec(c);

        // dU = P^T dY + tail (K dS); fragments are read a phase ahead, as in the forward
        f32x4 U[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) U[m] = f32x4{0, 0, 0, 0};
        Frag<NI> ka[2][4];
        Frag<NS> tf[kTriFrags], pf[kTriFrags];
        auto read_k = [&](int b) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NI; ++n)
                    ka[b & 1][m].t[n] = read_row<NCH>(kt + n * kTile, 16 * m + r, 4 * b + g);
        };
        auto read_tri = [&](const uint16_t *from, Frag<NS> *to) {
#pragma unroll
            for (int i = 0; i < kTriFrags; ++i)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    to[i].t[n] = *reinterpret_cast<const bf16x8 *>(from + ((i * NS + n) * 64 + l) * 8);
        };
        read_k(0);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            if (b + 1 < KB) read_k(b + 1);
            else read_tri(pt, pf);
            const Frag<NS> sb = split8<NS>(S[2 * b], S[2 * b + 1]);
            if (kept) record_store<NS, KB>(p.ws.dS1 + rec * NS * p.ws.state, col_tile, b, sb);
            fence();
            for_terms<NI, NS>([&](int i, int j) {
#pragma unroll
                for (int m = 0; m < 4; ++m) U[m] = mfma16(ka[b & 1][m].t[i], sb.t[j], U[m]);
            });
            fence();
        }
        read_tri(tt, tf);
        {
            const Frag<NG> yb[2] = {split8<NG>(Y[0], Y[1]), split8<NG>(Y[2], Y[3])};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4 tail = *reinterpret_cast<const f32x4 *>(vec + 64 + 16 * m + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) U[m][e] *= tail[e];
            }
            fence();
            for_terms<NS, NG>([&](int i, int j) {
#pragma unroll
                for (int b = 1; b >= 0; --b)
#pragma unroll
                    for (int m = 0; m < 2 + 2 * b; ++m) U[m] = mfma16(pf[tri_upper(m, b)].t[i], yb[b].t[j], U[m]);
            });
            fence();
        }
        // dX = dU + (T - 1)^T dU
        Frag<NI> qc[2][2][2], kc[2][2][2];  // Q^T, K^T: [step parity][tile of the pair][time block]
        auto read_qk = [&](int b) {
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NI; ++n) {
                        const int col4 = 32 * b + 8 * (r & 3) + 4 * o;
                        if constexpr (!kOther)
                            qc[b & 1][o][i].t[n] = read_cols<NCH>(qt + n * kTile, 32 * i + 4 * g, 32 * i + 16 + 4 * g, col4);
                        kc[b & 1][o][i].t[n] = read_cols<NCH>(kt + n * kTile, 32 * i + 4 * g, 32 * i + 16 + 4 * g, col4);
                    }
        };
        read_qk(0);
        f32x4 X[4];
        {
            const Frag<NS> ub[2] = {split8<NS>(U[0], U[1]), split8<NS>(U[2], U[3])};
            fence();
#pragma unroll
            for (int m = 0; m < 4; ++m) X[m] = U[m];
            for_terms<NS, NS>([&](int i, int j) {
#pragma unroll
                for (int b = 1; b >= 0; --b)
#pragma unroll
                    for (int m = 0; m < 2 + 2 * b; ++m) X[m] = mfma16(tf[tri_upper(m, b)].t[i], ub[b].t[j], X[m]);
            });
            fence();
        }
        {
            if (kept) {
                record_store<NS, 2>(p.ws.dX + rec * NS * p.ws.step, col_tile, 0, split8<NS>(X[0], X[1]));
                record_store<NS, 2>(p.ws.dX + rec * NS * p.ws.step, col_tile, 1, split8<NS>(X[2], X[3]));
            }
            f32x4 dv[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4 bt = *reinterpret_cast<const f32x4 *>(vec + 192 + 16 * m + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) dv[m][e] = bt[e] * X[m][e];
            }
            store_column<TG, kFast>(vp + t * p.sdv.t, p.sdv.t, rows, g, col, mine, dv);
        }
        // dS = e^{Gc} dS + Q^T (scale e^G dY) - K^T (beta e^G dX)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 eg = *reinterpret_cast<const f32x4 *>(vec + 16 * m + 4 * g);
            const f32x4 be = *reinterpret_cast<const f32x4 *>(vec + 128 + 16 * m + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                Y[m][e] *= p.scale * eg[e];
                X[m][e] *= -be[e];
            }
        }
        {
            const Frag<NS> yb[2] = {split8<NS>(Y[0], Y[1]), split8<NS>(Y[2], Y[3])};
            const Frag<NS> xb[2] = {split8<NS>(X[0], X[1]), split8<NS>(X[2], X[3])};
            const float ec = vec[63];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                if (b + 1 < KB) read_qk(b + 1);
                fence();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[2 * b][e] *= ec;
                    S[2 * b + 1][e] *= ec;
                }
                for_terms<NI, NS>([&](int i, int j) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            f32x4 &d = S[2 * b + o];
                            if constexpr (!kOther) d = mfma16(qc[b & 1][o][t].t[i], yb[t].t[j], d);
                            d = mfma16(kc[b & 1][o][t].t[i], xb[t].t[j], d);
                        }
                });
            }
            if constexpr (kOther) {
                st.store_other(c);
                if (c > 0) st.start(c - 1);
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    read_qk(b);
#pragma unroll
                    for (int o = 0; o < 2; ++o)
#pragma unroll
                        for (int i = 0; i < 2; ++i) S[2 * b + o] = mma<NI, NS>(kc[b & 1][o][i], yb[i], S[2 * b + o]);
                }
            }
        }
    }
    if (p.dh0 && mine) {
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * (m / 2) + 8 * g + 4 * (m % 2) + e;
                if (row < p.K) p.dh0[state_at + (long long)row * p.V] = S[m][e];
            }
    }
}

// ------------------------------------------------------------ sums over the value channels
struct GradParams {
    int seqlen, nseq, rep, h, K, V, Vp;
    float scale;
    const int *cu;
    const void *q, *k, *v, *dy;
    const float *gate, *beta;
    void *dq, *dk;
    float *dg, *dbeta;
    DeltaStride sq, sk, sv, sg, sbeta, sdy, sdq, sdk;
    DeltaWs ws;
};

// Sum over 16 neighbouring lanes, to all of them.
template <int kCtrl> __device__ inline float row_move(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true));
}
__device__ inline float row_sum(float v)
{
    v += row_move<0xB1>(v);   // quad_perm 1,0,3,2
    v += row_move<0x4E>(v);   // quad_perm 2,3,0,1
    v += row_move<0x141>(v);  // row_half_mirror
    v += row_move<0x140>(v);  // row_mirror
    return v;
}

template <int N> __device__ inline float tile_value(const uint16_t *tile, int plane, int at)
{
    float v = 0.0f;
#pragma unroll
    for (int n = N - 1; n >= 0; --n) v += __uint_as_float(uint32_t(tile[n * plane + at]) << 16);
    return v;
}

// Sum of a . b over the lane's 8 elements, both in N terms.
template <int N> __device__ inline float dot8(const Frag<N> &a, const Frag<N> &b, float s)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j + i < N; ++j)
#pragma unroll
            for (int e = 0; e < 8; e += 2)
                s = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{a.t[i][e], a.t[i][e + 1]}, bf16x2{b.t[j][e], b.t[j][e + 1]}, s,
                                                    false);
    return s;
}

// kShared: a key head has several value heads, whose sums meet here.
template <typename T, typename TG, int KD, bool kShared, bool kFast>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 && KD <= 128 && !kShared ? 2 : 1))
void delta_grad_kernel(const GradParams p)
{
    constexpr int NI = Terms<T>::kIn, NS = Terms<T>::kSum, NG = kGradTerms<T, TG>;
    constexpr int KH = KD < 128 ? KD : 128, NCH = KH / 8, kTile = 64 * KH;  // K and Q are staged KH columns at a time
    constexpr int kHalves = KD / KH, NT = KH / 64, NTT = KD / 64, KB = KD / 32;  // NTT column tiles a wave
    // LDS: 32 value columns of S0, dS1, U, dX, dY and V, then K, Q and the 64 x 64 matrices
    constexpr int kStates = 2 * KB * NS * 512, kSteps = 2 * 2 * NS * 512, kCols = 64 * 32, kZ = 64 * 64;
    constexpr int kStage = 2 * kStates + 2 * kSteps + (NG + NI) * kCols;
    constexpr int kMats = 2 * NS * kZ > 64 * 68 * 2 ? 2 * NS * kZ : 64 * 68 * 2;
    constexpr int kLds = kStage > 2 * NI * kTile + kMats ? kStage : 2 * NI * kTile + kMats;
    __shared__ __align__(16) uint16_t lds[kLds];
    __shared__ double G[64];
    __shared__ __align__(16) float vec[256];
    __shared__ float rowd[4][3][64], rect[4][64], row_v[64], row_m[64], dots[4];
    uint16_t *ts = lds, *td = ts + kStates, *tu = td + kStates, *tx = tu + kSteps, *ty = tx + kSteps, *tv = ty + NG * kCols;
    uint16_t *kt = lds, *qt = kt + NI * kTile, *zp = qt + NI * kTile, *zn = zp + NS * kZ;
    float *W = reinterpret_cast<float *>(zp);

    const int chunk = int(blockIdx.x), qk_head = int(blockIdx.y);
    const int si = delta_seq_of(p.cu, p.nseq, p.seqlen, chunk);
    const DeltaSeq seq = delta_seq(p.cu, si, p.seqlen);
    const int at0 = (chunk - seq.chunk0) * kDeltaChunk;
    const int rows = min(kDeltaChunk, seq.len - at0);
    if (at0 < 0 || rows <= 0) return;  // the whole workgroup
    const long long t0 = seq.first + at0;
    const int tid = int(threadIdx.x), l = tid & 63, r = l & 15, g = l >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const T *kp = static_cast<const T *>(p.k) + seq.batch * p.sk.b + t0 * p.sk.t + qk_head * p.sk.h;
    const T *qp = static_cast<const T *>(p.q) + seq.batch * p.sq.b + t0 * p.sq.t + qk_head * p.sq.h;
    auto stage_qk = [&](int half) {
        TileLoad<T, NCH, kThreads, kFast> lk, lq;
        lk.init(p.sk.t, p.K - half * KH);
        lq.init(p.sq.t, p.K - half * KH);
        lk.fetch(kp + half * KH, p.sk.t, rows, p.K - half * KH);
        lq.fetch(qp + half * KH, p.sq.t, rows, p.K - half * KH);
        lk.template store<NI>(kt, rows, p.K - half * KH);
        lq.template store<NI>(qt, rows, p.K - half * KH);
    };

    // column tile n of a wave: keys' entries key(n) + lane's r
    auto key = [&](int n) { return (n / NT) * KH + wave * (KH / 4) + 16 * (n % NT); };
    f32x4 dq[kShared ? NTT : 1][4], dk[kShared ? NTT : 1][4];
    if constexpr (kShared) {
#pragma unroll
        for (int n = 0; n < NTT; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m) dq[n][m] = dk[n][m] = f32x4{0, 0, 0, 0};
    }

    auto store = [&](const f32x4 (*q)[4], const f32x4 (*k)[4]) {
        TG *dqp = static_cast<TG *>(p.dq) + seq.batch * p.sdq.b + t0 * p.sdq.t + qk_head * p.sdq.h;
        TG *dkp = static_cast<TG *>(p.dk) + seq.batch * p.sdk.b + t0 * p.sdk.t + qk_head * p.sdk.h;
#pragma unroll
        for (int n = 0; n < NTT; ++n) {
            const int c = key(n) + r;
            store_column<TG, kFast>(dqp, p.sdq.t, rows, g, c, c < p.K, q[n]);
            store_column<TG, kFast>(dkp, p.sdk.t, rows, g, c, c < p.K, k[n]);
        }
    };

    for (int hi = 0; hi < (kShared ? p.rep : 1); ++hi) {
        const int head = qk_head * p.rep + hi;
        const long long rec = (long long)chunk * p.h + head;
        __syncthreads();  // the last head's LDS is read
        vec[tid] = reinterpret_cast<const float *>(p.ws.prep + rec * p.ws.prep_stride + 2 * tri_size(NS))[tid];
        if (wave == 0) {
            float gi = 0.0f;
            if (l < rows) gi = p.gate[seq.batch * p.sg.b + (t0 + l) * p.sg.t + head * p.sg.h];
            G[l] = decay_sums(gi);
        }
        const T *vp = static_cast<const T *>(p.v) + seq.batch * p.sv.b + t0 * p.sv.t + head * p.sv.h;
        const TG *yp = static_cast<const TG *>(p.dy) + seq.batch * p.sdy.b + t0 * p.sdy.t + head * p.sdy.h;
        const uint16_t *U = p.ws.U + rec * NS * p.ws.step, *dX = p.ws.dX + rec * NS * p.ws.step;
        const uint16_t *S0 = p.ws.S0 + rec * NS * p.ws.state, *dS1 = p.ws.dS1 + rec * NS * p.ws.state;

        f32x4 ys[NTT][4], xs[NTT][4], us[NTT][4], dP[4], dM[4], xv = {0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int n = 0; n < NTT; ++n) ys[n][m] = xs[n][m] = us[n][m] = f32x4{0, 0, 0, 0};
            dP[m] = dM[m] = f32x4{0, 0, 0, 0};
        }
        float dot = 0.0f;
        for (int v0 = 0; v0 < p.V; v0 += 32) {
            if (v0) __syncthreads();  // the last columns' reads are done
            const long long tile = v0 / 16;
            const uint32_t to = __builtin_amdgcn_readfirstlane(lds_offset(lds));
            copy_linear<kStates * 2, 4>(S0 + tile * (kStates / 2), to, wave);
            copy_linear<kStates * 2, 4>(dS1 + tile * (kStates / 2), to + 2 * kStates, wave);
            copy_linear<kSteps * 2, 4>(U + tile * (kSteps / 2), to + 4 * kStates, wave);
            copy_linear<kSteps * 2, 4>(dX + tile * (kSteps / 2), to + 4 * kStates + 2 * kSteps, wave);
            TileLoad<TG, 4, kThreads, kFast> ly;
            TileLoad<T, 4, kThreads, kFast> lv;
            ly.init(p.sdy.t, p.V - v0);
            lv.init(p.sv.t, p.V - v0);
            ly.fetch(yp + v0, p.sdy.t, rows, p.V - v0);
            lv.fetch(vp + v0, p.sv.t, rows, p.V - v0);
            ly.template store<NG>(ty, rows, p.V - v0);
            lv.template store<NI>(tv, rows, p.V - v0);
            wait_loads<0>();
            __syncthreads();

            // S0 and dS1 as right operands: 32 columns by the wave's key entries
            Frag<NS> sb[NTT], db[NTT];
#pragma unroll
            for (int n = 0; n < NTT; ++n) {
                const int k4 = key(n) + 4 * (r & 3);
                sb[n] = record_cols<NS, KB>(ts, key(n) >> 5, (k4 >> 3) & 3, (k4 >> 2) & 1);
                db[n] = record_cols<NS, KB>(td, key(n) >> 5, (k4 >> 3) & 3, (k4 >> 2) & 1);
            }
            Frag<NG> yw;
            Frag<NI> vw;
            const Frag<NS> xw = record_cols<NS, 2>(tx, wave >> 1, r & 3, wave & 1);
#pragma unroll
            for (int n = 0; n < NG; ++n) yw.t[n] = read_row<4>(ty + n * kCols, 16 * wave + r, g);
#pragma unroll
            for (int n = 0; n < NI; ++n) vw.t[n] = read_row<4>(tv + n * kCols, 16 * wave + r, g);
            Frag<NG> ay[2];
            Frag<NS> ax[2], au[2];
            auto read_a = [&](int m) {
#pragma unroll
                for (int n = 0; n < NG; ++n) ay[m & 1].t[n] = read_row<4>(ty + n * kCols, 16 * m + r, g);
                ax[m & 1] = record_cols<NS, 2>(tx, m >> 1, r & 3, m & 1);
                au[m & 1] = record_cols<NS, 2>(tu, m >> 1, r & 3, m & 1);
            };
            read_a(0);
#pragma unroll
            for (int n = 0; n < NTT; ++n) dot = dot8<NS>(sb[n], db[n], dot);
            xv = mma<NS, NI>(xw, vw, xv);  // its diagonal: dX . V
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (m + 1 < 4) read_a(m + 1);
                fence();
                if (m <= wave) {  // row tile `wave` of dY U^T and dX U^T
                    dP[m] = mma<NG, NS>(yw, au[m & 1], dP[m]);
                    dM[m] = mma<NS, NS>(xw, au[m & 1], dM[m]);
                    settle();
                }
                for_terms<NS, NS>([&](int i, int j) {
#pragma unroll
                    for (int n = 0; n < NTT; ++n) {
                        if (i < NG)
                            ys[n][m] = mfma16(ay[m & 1].t[i], sb[n].t[j], ys[n][m]);
                        xs[n][m] = mfma16(ax[m & 1].t[i], sb[n].t[j], xs[n][m]);
                        us[n][m] = mfma16(au[m & 1].t[i], db[n].t[j], us[n][m]);
                    }
                });
                fence();
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (r == 4 * g + e) row_v[16 * wave + r] = xv[e];
#pragma unroll
        for (int o = 1; o < 64; o *= 2) dot += __shfl_xor(dot, o);
        if (l == 0) dots[wave] = dot;

        // Q K^T, K K^T again, and the row sums that dg and dbeta need
        f32x4 kk[4], qk[4], rq[4], rr[4], ru[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) kk[m] = qk[m] = rq[m] = rr[m] = ru[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
            __syncthreads();
            stage_qk(half);
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
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int c = wave * (KH / 4) + 16 * n + r;
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = chunk_at<NCH>(16 * m + 4 * g + e, c >> 3) + (c & 7);
                        const float kv = tile_value<NI>(kt, kTile, at), qv = tile_value<NI>(qt, kTile, at);
                        rq[m][e] = __builtin_fmaf(qv, ys[half * NT + n][m][e], rq[m][e]);
                        rr[m][e] = __builtin_fmaf(kv, xs[half * NT + n][m][e], rr[m][e]);
                        ru[m][e] = __builtin_fmaf(kv, us[half * NT + n][m][e], ru[m][e]);
                    }
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = row_sum(rq[m][e]), b = row_sum(rr[m][e]), c = row_sum(ru[m][e]);
                if (r == 0) {
                    const int i = 16 * m + 4 * g + e;
                    rowd[wave][0][i] = a;
                    rowd[wave][1][i] = b;
                    rowd[wave][2][i] = c;
                }
            }
        // ys and us become the products with S0 and dS1 in dQ and dK
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 eg = *reinterpret_cast<const f32x4 *>(vec + 16 * m + 4 * g);
            const f32x4 tail = *reinterpret_cast<const f32x4 *>(vec + 64 + 16 * m + 4 * g);
            const f32x4 be = *reinterpret_cast<const f32x4 *>(vec + 128 + 16 * m + 4 * g);
#pragma unroll
            for (int n = 0; n < NTT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ys[n][m][e] *= p.scale * eg[e];
                    us[n][m][e] = tail[e] * us[n][m][e] - be[e] * xs[n][m][e];
                }
        }
        // dP, N = beta dM, W
        f32x4 sums = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = 16 * c + r;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * wave + 4 * g + e;
                float w = 0.0f;
                if (c <= wave) {
                    const float d = i >= j ? exp2_hw(float(G[i] - G[j]) * kLog2e) : 0.0f;
                    dP[c][e] *= p.scale * d;
                    const float mm = i > j ? -d * dM[c][e] : 0.0f;
                    sums[e] = __builtin_fmaf(mm, kk[c][e], sums[e]);
                    dM[c][e] = vec[192 + i] * mm;
                    if (i > j) w = dP[c][e] * qk[c][e] + dM[c][e] * kk[c][e];
                }
                W[i * 68 + j] = w;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float s = row_sum(sums[e]);
            if (r == 0) row_m[16 * wave + 4 * g + e] = s;
        }
        __syncthreads();
        {   // W_ij <- sum of W_i before j: four threads a row
            float *w = W + (tid >> 2) * 68 + (tid & 3) * 16;
            f32x4 x[4];
            float run = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = reinterpret_cast<f32x4 *>(w)[i];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = x[i / 4][i % 4];
                x[i / 4][i % 4] = run;
                run += v;
            }
            const float a = __shfl_up(run, 1), b = __shfl_up(run, 2), c = __shfl_up(run, 3);
            const int quarter = tid & 3;
            const float before = (quarter > 0 ? a : 0.0f) + (quarter > 1 ? b : 0.0f) + (quarter > 2 ? c : 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] += before;
                reinterpret_cast<f32x4 *>(w)[i] = x[i];
            }
        }
        __syncthreads();
        {   // sum over i >= m of those, a quarter of the rows a wave
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * wave + i >= l) s += W[(16 * wave + i) * 68 + l];
            rect[wave][l] = s;
        }
        __syncthreads();
        if (wave == 0) {
            const float eg = vec[l], tail = vec[64 + l], be = vec[128 + l];
            float a[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) a[i] = rowd[0][i][l] + rowd[1][i][l] + rowd[2][i][l] + rowd[3][i][l];
            const float here = p.scale * eg * a[0] - be * a[1], wr = tail * a[2];
            float after = here, before = wr;  // sums over i >= l and over j <= l
#pragma unroll
            for (int o = 1; o < 64; o *= 2) {
                const float x = __shfl_down(after, o), y = __shfl_up(before, o);
                if (l + o < 64) after += x;
                if (l >= o) before += y;
            }
            before = __shfl_up(before, 1);
            if (l == 0) before = 0.0f;
            const float inner = rect[0][l] + rect[1][l] + rect[2][l] + rect[3][l];
            const float state = vec[63] * (dots[0] + dots[1] + dots[2] + dots[3]);
            if (l < rows) {
                const long long at = ((long long)seq.batch * p.seqlen + t0 + l) * p.h + head;
                p.dg[at] = inner + after + before + state;
                p.dbeta[at] = row_v[l] - eg * a[1] + row_m[l];
            }
        }
        // dP and N transposed into LDS: row j, columns i
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c <= wave || (c == wave + 1 && wave % 2 == 0)) {
                const int at = chunk_at<8>(16 * c + r, 2 * wave + (g >> 1)) + 4 * (g & 1);
                float a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] = c <= wave ? dP[c][e] : 0.0f;
                    b[e] = c <= wave ? dM[c][e] : 0.0f;
                }
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
                    const u32x2 x = {split_pair(a[0], a[1]), split_pair(a[2], a[3])};
                    const u32x2 y = {split_pair(b[0], b[1]), split_pair(b[2], b[3])};
                    *reinterpret_cast<u32x2 *>(zp + n * kZ + at) = x;
                    *reinterpret_cast<u32x2 *>(zn + n * kZ + at) = y;
                }
            }
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
            if (kHalves > 1) {
                if (half) __syncthreads();
                stage_qk(half);
            }
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                Frag<NI> kb[NT], qb[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int col4 = wave * (KH / 4) + 16 * n + 4 * (r & 3);
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        kb[n].t[i] = read_cols<NCH>(kt + i * kTile, 32 * b + 8 * g, 32 * b + 8 * g + 4, col4);
                        qb[n].t[i] = read_cols<NCH>(qt + i * kTile, 32 * b + 8 * g, 32 * b + 8 * g + 4, col4);
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    Frag<NS> a, z;
                    if (b <= m / 2) {  // rows i: dP K and N K
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            a.t[i] = read_cols<8>(zp + i * kZ, 32 * b + 8 * g, 32 * b + 8 * g + 4, 16 * m + 4 * (r & 3));
                            z.t[i] = read_cols<8>(zn + i * kZ, 32 * b + 8 * g, 32 * b + 8 * g + 4, 16 * m + 4 * (r & 3));
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            ys[half * NT + n][m] = mma<NS, NI>(a, kb[n], ys[half * NT + n][m]);
                            us[half * NT + n][m] = mma<NS, NI>(z, kb[n], us[half * NT + n][m]);
                        }
                    }
                    if (b >= m / 2) {  // rows j: dP^T Q and N^T K
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            a.t[i] = read_row<8>(zp + i * kZ, 16 * m + r, 4 * b + g);
                            z.t[i] = read_row<8>(zn + i * kZ, 16 * m + r, 4 * b + g);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            us[half * NT + n][m] = mma<NS, NI>(a, qb[n], us[half * NT + n][m]);
                            us[half * NT + n][m] = mma<NS, NI>(z, kb[n], us[half * NT + n][m]);
                        }
                    }
                }
            }
        }
        if constexpr (kShared) {
#pragma unroll
            for (int n = 0; n < NTT; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    dq[n][m] += ys[n][m];
                    dk[n][m] += us[n][m];
                }
        } else {
            store(ys, us);
        }
    }
    if constexpr (kShared) store(dq, dk);
}

template <typename T, typename TG, int KD>
hipError_t launch_typed(const DeltaBwdArgs &b, const DeltaWs &ws, hipStream_t stream)
{
    const DeltaArgs &a = b.f;
    const int es = sizeof(T), gs = sizeof(TG), rep = a.h / a.hk, Vp = delta_vp(a.V);
    const bool qk = delta_fast(a.q, a.sq, a.K, es, a, a.hk) && delta_fast(a.k, a.sk, a.K, es, a, a.hk);
    constexpr long long most = (1ll << 31) / 64 / 4;
    const bool sfast = qk && b.sdy.t < most && b.sdv.t < most;
    const bool gfast = qk && delta_fast(a.v, a.sv, a.V, es, a, a.h) && delta_fast(b.dy, b.sdy, a.V, gs, a, a.h) &&
                       b.sdq.t < most && b.sdk.t < most;
    const ScanBwdParams sp{a.seqlen, rep, a.h, a.K, a.V, Vp, a.scale, a.cu, a.q, a.k, b.dy, b.dhL, b.dv,
                           b.dh0, a.sq, a.sk, b.sdy, b.sdv, ws};
    const GradParams gp{a.seqlen, a.nseq, rep, a.h, a.K, a.V, Vp, a.scale, a.cu, a.q, a.k, a.v, b.dy, a.g, a.beta,
                        b.dq, b.dk, b.dg, b.dbeta, a.sq, a.sk, a.sv, a.sg, a.sbeta, b.sdy, b.sdq, b.sdk, ws};
    constexpr bool kCan = kDeltaAsync<T, KD> && sizeof(TG) == 2;
    const int path = !sfast ? kByElement : kCan && delta_fast(b.dy, b.sdy, a.V, gs, a, a.h) ? kByCopy : kByRun;
    const int waves = path == kByCopy && delta_wide(a, false) ? 8 : 4;
    const dim3 sgrid((a.V + 16 * waves - 1) / (16 * waves), a.h, a.nseq), sblock(64 * waves);
    const dim3 ggrid(unsigned(delta_chunks(a.batch, a.seqlen, a.cu ? a.nseq : 0)), a.hk), gblock(kThreads);
    if (log_enabled())
        log_line("delta_bwd: delta_scan_bwd_kernel, delta_grad_kernel<in %s, grad %s, K %d>, paths %d, %d, "
                 "grids (%u, %u, %u) x %u, (%u, %u) x %u threads", type_tag<T>(), type_tag<TG>(), KD, path,
                 int(gfast), sgrid.x, sgrid.y, sgrid.z, sblock.x, ggrid.x, ggrid.y, gblock.x);
    if (path == kByElement) {
        delta_scan_bwd_kernel<T, TG, KD, 4, kByElement><<<sgrid, sblock, 0, stream>>>(sp);
    } else if (path == kByRun) {
        delta_scan_bwd_kernel<T, TG, KD, 4, kByRun><<<sgrid, sblock, 0, stream>>>(sp);
    } else {
        if constexpr (kCan) {
            if (waves == 8) delta_scan_bwd_kernel<T, TG, KD, 8, kByCopy><<<sgrid, sblock, 0, stream>>>(sp);
            else delta_scan_bwd_kernel<T, TG, KD, 4, kByCopy><<<sgrid, sblock, 0, stream>>>(sp);
        }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (rep > 1 && gfast) delta_grad_kernel<T, TG, KD, true, true><<<ggrid, gblock, 0, stream>>>(gp);
    else if (rep > 1) delta_grad_kernel<T, TG, KD, true, false><<<ggrid, gblock, 0, stream>>>(gp);
    else if (gfast) delta_grad_kernel<T, TG, KD, false, true><<<ggrid, gblock, 0, stream>>>(gp);
    else delta_grad_kernel<T, TG, KD, false, false><<<ggrid, gblock, 0, stream>>>(gp);
    return hipGetLastError();
}

}  // namespace

size_t delta_bwd_workspace_bytes(int batch, int seqlen, int hk, int h, int K, int V, int num_seqs)
{
    size_t bytes = 0;
    delta_ws(nullptr, batch, seqlen, h, K, V, num_seqs, true, &bytes);
    return bytes;
}

hipError_t launch_delta_bwd(const DeltaBwdArgs &b, hipStream_t stream)
{
    const DeltaArgs &a = b.f;
    const DeltaWs ws = delta_ws(a, true);
    if (!b.ckpt_given) {  // the forward, for its records only
        hipError_t e = launch_delta_prep(a, ws, true, stream);
        if (e == hipSuccess) e = launch_delta_scan(a, ws, stream);
        if (e != hipSuccess) return e;
    }
    return delta_dispatch(a.in_bf16, b.grad_bf16, a.K, [&](auto t, auto tg, auto kd) {
        return launch_typed<decltype(t), decltype(tg), decltype(kd)::value>(b, ws, stream);
    });
}

}  // namespace ssm
