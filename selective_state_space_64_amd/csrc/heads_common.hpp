// heads_common.hpp -- what the kernels of the head-wise selective scan share:
// fragments of either compute type, tiles in LDS, a chunk's decays, and the
// workspace (gfx950).
//
// A chunk is 64 steps.  Two compute types: bf16 inputs are operands of
// v_mfma_f32_16x16x32_bf16 as they are, and what the kernels form (states,
// decayed products) is split into bf16 terms (delta_mfma.hpp); everything
// else, fp32 or mixed types, runs on v_mfma_f32_16x16x4_f32, whose operands
// are fp32.  Both see the same fragments: a lane's 8 elements of a contraction
// over 32.
#pragma once

#include "delta_chunk.hpp"
#include "heads_launch.hpp"

namespace ssm {
namespace heads {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 64;  // columns of P that a workgroup of the recurrence holds

struct F32x8 {
    f32x4 lo, hi;
};
// An operand as it was given, and one that the kernels formed, with NS terms.
template <typename T> struct InOf {
    typedef bf16x8 type;
};
template <> struct InOf<float> {
    typedef F32x8 type;
};
template <typename T> using In = typename InOf<T>::type;
template <typename T, int NS> struct SumOf {
    typedef Frag<NS> type;
};
template <int NS> struct SumOf<float, NS> {
    typedef F32x8 type;
};
template <typename T, int NS> using Sum = typename SumOf<T, NS>::type;

template <typename T, int NS> __device__ inline Sum<T, NS> to_sum(f32x4 a, f32x4 b)
{
    if constexpr (sizeof(T) == 4) return F32x8{a, b};
    else return split8<NS>(a, b);
}

// acc[m] += a[m] b, and acc[m] += a b[m]: M products whose instructions take
// turns, so that none waits for the one before it.
__device__ inline bf16x8 term(const bf16x8 &f, int) { return f; }
template <int N> __device__ inline bf16x8 term(const Frag<N> &f, int i) { return f.t[i]; }
template <typename F> struct TermsIn {
    static constexpr int n = 1;
};
template <int N> struct TermsIn<Frag<N>> {
    static constexpr int n = N;
};
__device__ inline float element(const F32x8 &f, int e) { return e < 4 ? f.lo[e & 3] : f.hi[e & 3]; }

template <int M, typename FA, typename FB>
__device__ inline void mma_left(f32x4 *acc, const FA *a, const FB &b)
{
    if constexpr (std::is_same_v<FA, F32x8>) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m] = mfma16_f32(element(a[m], e), element(b, e), acc[m]);
    } else {
        for_terms<TermsIn<FA>::n, TermsIn<FB>::n>([&](int i, int j) {
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m] = mfma16(term(a[m], i), term(b, j), acc[m]);
        });
    }
}
template <int M, typename FA, typename FB>
__device__ inline void mma_right(f32x4 *acc, const FA &a, const FB *b)
{
    if constexpr (std::is_same_v<FA, F32x8>) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m] = mfma16_f32(element(a, e), element(b[m], e), acc[m]);
    } else {
        for_terms<TermsIn<FA>::n, TermsIn<FB>::n>([&](int i, int j) {
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m] = mfma16(term(a, i), term(b[m], j), acc[m]);
        });
    }
}

// ---------------------------------------------------------------- tiles
// Rows of NCH chunks of 8 elements, permuted as chunk_at says.
template <typename T> struct Elem {
    typedef uint16_t type;
};
template <> struct Elem<float> {
    typedef float type;
};
template <typename T> using E = typename Elem<T>::type;

template <typename T, int NCH> __device__ inline In<T> tile_row(const E<T> *tile, int t, int c)
{
    if constexpr (sizeof(T) == 2) {
        return read_row<NCH>(tile, t, c);
    } else {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(tile + chunk_at<NCH>(t, c));
        return F32x8{p[0], p[1]};
    }
}
// Rows ta .. ta + 3 and tb .. tb + 3 of the lane's column; `quarter`: the first
// column of the four that lanes 4 b .. 4 b + 3 of 16 take, as a function of b
// (neighbouring lanes' columns are neighbours in fours).
template <typename T, int NCH, typename F>
__device__ inline In<T> tile_cols(const E<T> *tile, int ta, int tb, F &&quarter)
{
    const int r = int(threadIdx.x) & 15;
    if constexpr (sizeof(T) == 2) {
        return read_cols<NCH>(tile, ta, tb, quarter(r & 3));
    } else {
        const int col = quarter(r >> 2) + (r & 3);
        F32x8 f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f.lo[e] = tile[chunk_at<NCH>(ta + e, col >> 3) + (col & 7)];
            f.hi[e] = tile[chunk_at<NCH>(tb + e, col >> 3) + (col & 7)];
        }
        return f;
    }
}
__device__ inline void to_floats(const bf16x8 &v, f32x4 &lo, f32x4 &hi)
{
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    lo = f32x4{io<bf16_t>::lo(w[0]), io<bf16_t>::hi(w[0]), io<bf16_t>::lo(w[1]), io<bf16_t>::hi(w[1])};
    hi = f32x4{io<bf16_t>::lo(w[2]), io<bf16_t>::hi(w[2]), io<bf16_t>::lo(w[3]), io<bf16_t>::hi(w[3])};
}
__device__ inline void to_floats(const F32x8 &v, f32x4 &lo, f32x4 &hi)
{
    lo = v.lo;
    hi = v.hi;
}

// Hides where a value comes from, so that what is computed of it in a loop is
// not kept in registers from before the loop.
__device__ inline void opaque(uint32_t &v) { asm volatile("" : "+v"(v)); }

// An operand is formed here and not later: the compiler moves what has no side
// effects to where it is used, out of the shadow of the matrix instructions that
// stand beside it in the source.
template <int N> __device__ inline void pin(Frag<N> &f)
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f.t[i]));
}
__device__ inline void pin(F32x8 &) {}

// 64 rows on their way from memory to a tile.  kFast: in registers from
// fetch() to store(), 16-byte loads from one buffer whose end stands for the
// masks of rows; otherwise store() loads them element by element, of the type
// that `bf16` says (fp32 compute takes either).
template <typename T, int NCH, bool kFast, int kThreads = 256> struct TileIn {
    static constexpr int kPer = (64 * NCH + kThreads - 1) / kThreads, kWords = int(sizeof(T) / 2);
    static constexpr bool kSpare = 64 * NCH < kThreads;  // threads without a chunk
    u32x4 raw[kFast ? kPer : 1][kWords];
    uint32_t off, run;  // of the thread's first chunk; from one of its rows to the next
    // rows `step` elements apart, columns [0, n) exist
    __device__ inline void init(long long step, int n)
    {
        if constexpr (kFast) {
            const int t = int(threadIdx.x) / NCH, c = int(threadIdx.x) % NCH;
            run = uint32_t(kThreads / NCH) * uint32_t(step) * uint32_t(sizeof(T));
            off = c * 8 < n ? uint32_t(t * int(step) + c * 8) * uint32_t(sizeof(T)) : kOutside;
        }
    }
    // rows >= 1 from p on
    __device__ inline void fetch(const void *p, long long step, int rows)
    {
        if constexpr (kFast) {
            const auto buf = buffer_of(p, (long long)(rows * int(step)) * int(sizeof(T)));
            uint32_t off = this->off;
            opaque(off);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
#pragma unroll
                for (int w = 0; w < kWords; ++w)
                    raw[i][w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off + i * run + 16 * w, 0, 0));
        }
    }
    __device__ inline void store(E<T> *tile, const void *p, long long step, int rows, int n, int bf16) const
    {
        if constexpr (kFast) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) put(tile, i, raw[i]);
        } else {
            for (int i = 0; i < kPer; ++i) {
                const int at = int(threadIdx.x) + i * kThreads, t = at / NCH, c = at % NCH;
                if (kSpare && t >= 64) return;
                const long long row = (long long)min(t, rows - 1) * step;
                const int count = t < rows ? n - c * 8 : 0;
                if (sizeof(T) == 2 || !bf16) {
                    put(tile, i, (n < 1 ? Raw8<T>{} : keep8(load8(static_cast<const T *>(p) + row, c, n), count)).w);
                } else {
                    const Raw8<bf16_t> v =
                        n < 1 ? Raw8<bf16_t>{} : keep8(load8(static_cast<const bf16_t *>(p) + row, c, n), count);
                    f32x4 lo, hi;
                    to_floats(__builtin_bit_cast(bf16x8, v.w[0]), lo, hi);
                    const u32x4 w[2] = {__builtin_bit_cast(u32x4, lo), __builtin_bit_cast(u32x4, hi)};
                    put(tile, i, w);
                }
            }
        }
    }
    __device__ static inline void put(E<T> *tile, int i, const u32x4 *w)
    {
        const int at = int(threadIdx.x) + i * kThreads;
        if (kSpare && at >= 64 * NCH) return;
        u32x4 *to = reinterpret_cast<u32x4 *>(tile + chunk_at<NCH>(at / NCH, at % NCH));
#pragma unroll
        for (int k = 0; k < kWords; ++k) to[k] = w[k];
    }
};

// ---------------------------------------------------------------- a chunk's decays
// Sums over the lanes up to each one, in double: inside 16 lanes by shifts, then
// the last lane of a row to the row behind it and of the first half to the second.
template <int kCtrl, int kRows> __device__ inline double dpp_add(double v)
{
    const unsigned long long bits = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = unsigned(__builtin_amdgcn_update_dpp(0, int(unsigned(bits)), kCtrl, kRows, 0xf, false));
    const unsigned hi = unsigned(__builtin_amdgcn_update_dpp(0, int(unsigned(bits >> 32)), kCtrl, kRows, 0xf, false));
    return v + __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ inline double wave_prefix(double v)
{
    v = dpp_add<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8 (lanes without a source add 0)
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);         // row_bcast 15, to rows 1 and 3
    return dpp_add<0x143, 0xc>(v);      // row_bcast 31, to rows 2 and 3
}
__device__ inline double from_lane(double v, int lane)
{
    const unsigned long long bits = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = unsigned(__builtin_amdgcn_readlane(int(unsigned(bits)), lane));
    const unsigned hi = unsigned(__builtin_amdgcn_readlane(int(unsigned(bits >> 32)), lane));
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}

// Lane t of a wave has step t; G in units of log2.
struct Decays {
    float dt;    // softplus(dt + bias), 0 behind the last row
    double G;    // sum of the decays up to the step
    double end;  // of all 64
};
__device__ inline Decays decays(float raw, float bias, float A, int rows)
{
    Decays d;
    const bool live = int(threadIdx.x & 63) < rows;
    d.dt = live ? softplus(raw + bias) : 0.0f;
    // a decay of e^-110 is 0 in fp32; clamped, it does not cost later steps'
    // differences their low bits (a NaN stays one)
    const double a = double(d.dt) * double(A);
    d.G = wave_prefix(live ? (a < -110.0 ? -110.0 : a) * 1.4426950408889634 : 0.0);
    d.end = from_lane(d.G, 63);
    return d;
}
// 2^v for v of any size, to about an ulp: the fraction that float(v) loses is put back.
__device__ inline float exp2_of(double v)
{
    const float hi = float(v);
    const float lo = float(v - double(hi));
    return exp2_hw(hi) * __builtin_fmaf(lo, kLn2, 1.0f);
}
// A chunk's decays for a workgroup: G as two floats, the step size, the scales
// of rows that read the state and of rows that enter it, e^{Gc}.
struct Vec {
    float hi[64], lo[64], dt[64], out[64], in[64], end[4];
};

// An element of a [steps] column of either type, as it was loaded: what would convert
// it here would wait for it here, and so would the end of a branch by type.
struct RawStep {
    uint16_t lo, hi;
    __device__ inline void load(const void *p, long long at, int bf16)
    {
        const char *const q = static_cast<const char *>(p) + at * (bf16 ? 2 : 4);
        lo = *reinterpret_cast<const uint16_t *>(q);
        hi = *reinterpret_cast<const uint16_t *>(q + (bf16 ? 0 : 2));
    }
    __device__ inline void pin() { asm volatile("" : "+v"(lo), "+v"(hi)); }  // waits for it
    __device__ inline float value(int bf16) const
    {
        return __uint_as_float(bf16 ? uint32_t(lo) << 16 : uint32_t(hi) << 16 | lo);
    }
};

// ---------------------------------------------------------------- workspace
inline int heads_nd(int N) { return N <= 64 ? 64 : N <= 128 ? 128 : 256; }

// Sequence split: where heads x sequences x column tiles leave compute units without
// work, a sequence is cut into segments.  All but a sequence's last (in the direction of
// the run) first yield their end state from zero, by the recurrence without its
// outputs; composed with the segments' decays, which are numbers here, these give the
// states that the segments enter with, and all segments run at once.
//
// Segments fill the card twice (512 workgroups), which is as many as it holds where the
// rule was measured: bf16 operands with N <= 128 (and fp32 ones with N <= 64).  Of the
// other kernels a compute unit holds one workgroup, and 512 run in two rounds: not
// measured apart.  A sequence is cut into three at least: two halves cost as much as they
// gain.  Measured, N = 128, P = 64, bf16, cut against whole: 24 heads of 65521 steps 329
// against 2426 us (400 for 256 workgroups, 352 for 1024), 4 sequences of 24 heads of 2048
// 59 against 84, 80 heads of 4096 81 against 160, 24 of 768 28 against 36; below the rule,
// 8 sequences of 24 heads of 2048 105 cut in two against 84, 2 of 80 heads of 1024 52
// against 45.  Two chunks a segment at least: 12 heads x 2 of 777 steps in fp32 31 us,
// with four 42.
// A packed batch is judged as if one sequence were all of it, since the host does not know
// the lengths.  That suits a long one among short ones; equal ones lose by it: 8 packed
// sequences of 24 heads of 2048 are cut in two and take 116 us (as batch rows, whole, 81);
// of 16 of 1024 none is cut, and the run for the ends and the composition find nothing to
// do (74 against 66).
struct HeadsSplit {
    int seg_chunks, segs;  // segs: an upper bound over all sequences
};
constexpr long long kFill = 512, kSegments = 3, kMinSeg = 2;
inline HeadsSplit heads_split(int batch, int seqlen, int h, int P, int num_seqs)
{
    const long long chunks = delta_chunks(batch, seqlen, num_seqs), nseq = num_seqs ? num_seqs : batch;
    const long long wgs = (long long)h * ((P + kCols - 1) / kCols);
    const long long per = num_seqs ? chunks : chunks / batch;  // of the longest sequence
    if (kSegments * (num_seqs ? 1 : nseq) * wgs > kFill) return {0, 0};
    // segments in all; of packed sequences the last ones are short (by half of one each, and some
    // more: the factor was not varied)
    long long want = kFill / wgs - num_seqs * 5 / 8;
    if (want < kSegments) want = kSegments;
    long long seg = (chunks + want - 1) / want;
    if (seg < kMinSeg) seg = kMinSeg;
    if (per < kSegments * seg) return {0, 0};
    const long long segs = num_seqs ? chunks / seg + num_seqs : batch * ((per + seg - 1) / seg);
    return {int(seg), int(segs)};
}

struct HeadsWs {
    // per (chunk, head): the state entering it and the gradient of the one
    // leaving it, [Nr][Pp] fp32
    float *S0, *dS1;
    int Nr, Pp;  // N and P padded to 32
    long long state;
    // sequence split, per segment and head: end states [Nr][Pp], then the states
    // entering the next segment (the last segment's place holds the sequence's
    // initial state), and the segment's decay
    float *ends, *decay;
    int seg_chunks;  // 0: not split
    // gradients' partial sums: dA, dDskip, ddt_bias per (chunk, head); dB and dC
    // per (part of a group's heads, chunk, group), [64][Nr]
    float *sums, *dBp, *dCp;
    int parts;
};

// Parts that a group's heads are cut into for the gradients' workgroups: each
// sums its heads' dB and dC, so few parts keep the partial sums small, and enough of
// them fill the card.
inline int heads_parts(int batch, int seqlen, int groups, int h, int num_seqs)
{
    const long long wgs = delta_chunks(batch, seqlen, num_seqs) * groups, rep = h / groups;
    long long parts = (256 + wgs - 1) / wgs;
    if (parts > rep) parts = rep;
    // parts of the same number of heads, none of them empty
    const long long each = (rep + parts - 1) / parts;
    return int((rep + each - 1) / each);
}

inline HeadsWs heads_ws(void *workspace, int batch, int seqlen, int groups, int h, int N, int P, int num_seqs, bool bwd,
                        size_t *bytes)
{
    const size_t records = size_t(delta_chunks(batch, seqlen, num_seqs));
    HeadsWs w{};
    w.Nr = (N + 31) / 32 * 32;
    w.Pp = (P + 31) / 32 * 32;
    w.state = (long long)w.Nr * w.Pp;
    char *p = static_cast<char *>(workspace);
    size_t at = 0;
    auto take = [&](size_t floats) {
        float *r = p ? reinterpret_cast<float *>(p + at) : nullptr;
        at += (floats * sizeof(float) + 15) / 16 * 16;
        return r;
    };
    if (bwd) {
        w.S0 = take(records * h * w.state);
        w.dS1 = take(records * h * w.state);
        w.sums = take(records * h * 3);
        w.parts = heads_parts(batch, seqlen, groups, h, num_seqs);
        if (w.parts > 1) {
            w.dBp = take(w.parts * records * groups * 64 * w.Nr);
            w.dCp = take(w.parts * records * groups * 64 * w.Nr);
        }
    }
    const HeadsSplit split = heads_split(batch, seqlen, h, P, num_seqs);
    w.seg_chunks = split.seg_chunks;
    if (split.segs) {
        w.ends = take(size_t(split.segs) * h * w.state);
        w.decay = take(size_t(split.segs) * h);
    }
    if (bytes) *bytes = at;
    return w;
}
inline HeadsWs heads_ws(const HeadsArgs &a, bool bwd)
{
    return heads_ws(a.workspace, a.batch, a.seqlen, a.groups, a.h, a.N, a.P, a.cu ? a.nseq : 0, bwd, nullptr);
}

// 16-byte loads fit every row of a tensor with n elements a row, and 64 steps of it
// are one buffer of less than 2^31 bytes (see TileLoad).
inline bool heads_fast(const void *p, const DeltaStride &s, int n, int esize, const HeadsArgs &a, int heads)
{
    const long long per = 16 / esize;
    return n % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.seqlen == 1 || s.t % per == 0) &&
           (heads == 1 || s.h % per == 0) && (a.batch == 1 || s.b % per == 0) && s.t < (1ll << 31) / 64 / esize;
}

// A run of the recurrence.  Forward: L = C, R = B, v = x, out = y; reverse, over
// the steps from the last to the first: L = B, R = C, v = dy, out = dx.
struct HeadsScan {
    int seqlen, nseq, rep, h, N, P;
    int in_bf16, v_bf16, out_bf16;
    const int *cu;
    const void *L, *R, *v, *dt;
    const float *A, *bias, *D;
    const float *s0;  // [sequence][h][N][P] states that the run begins with, or NULL
    float *sL;        // and ends with, or NULL
    void *out;        // or NULL
    float *keep;      // the state entering every chunk, or NULL
    DeltaStride sL_, sR, sv, sdt, sout;
    HeadsWs ws;
};
hipError_t launch_heads_scan(const HeadsArgs &a, const HeadsScan &p, bool reverse, hipStream_t stream);

}  // namespace heads
}  // namespace ssm
