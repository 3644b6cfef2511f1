// delta_chunk.hpp -- what the chunked delta rule's kernels agree on: the
// workspace, the number of bf16 terms, and the launch parameters.
#pragma once

#include <type_traits>

#include "delta_mfma.hpp"
#include "ssm_launch.hpp"

namespace ssm {

// Padded key size of the kernels' tiles.
inline int delta_kd(int K) { return K <= 64 ? 64 : K <= 128 ? 128 : 256; }
inline int delta_vp(int V) { return (V + 63) / 64 * 64; }

// bf16 terms of the inputs (kIn) and of what the kernels form from them
// (kSum: states, U, T, P, ... as operands and as records; the running states and
// sums themselves are fp32).  fp32 inputs take three (2^-25 of a value's size).
// bf16 inputs take two (2^-17), 200 times under the rounding of a bf16 output:
// their fp32 outputs (hL, dh0, dg, dbeta) have errors of 1.5e-6 to 4.3e-6 where
// fp32 arithmetic has 1e-7 to 4e-7.  A caller who wants these passes the same
// values as fp32 (an exact conversion; the outputs may still be bf16): errors of 1.1e-7
// to 3.4e-7 for the layer of 4 x 40 heads, at 976 us against 220 forward and 2.99 ms
// against 0.99 for a training step.  Three terms for bf16 inputs were measured too: in
// the update of the state alone hL 1.1e-6 and dh0 0.9e-6 with a forward 3.7 % slower, in
// T X as well hL 3.2e-7 with a forward 11 to 15 % slower (5 % a training step), dg and
// dbeta as before in both; in all products two buffers do not fit 160 KB of LDS with
// eight waves.
template <typename T> struct Terms {
    static constexpr int kIn = sizeof(T) == 2 ? 1 : 3;
    static constexpr int kSum = sizeof(T) == 2 ? 2 : 3;
};

struct DeltaWs {
    uint16_t *prep;     // prep_stride elements a record
    long long prep_stride;
    uint16_t *S0, *U, *dS1, *dX;
    // elements a record for one term (the space is for three)
    long long state, step;
    // sequence split (delta_split), per segment and head: end states [KD][Vp],
    // then the states entering the next segment, and in the last segment's place, which
    // has neither, the sequence's h0; transfer matrices' terms [KD][KD]
    float *N;
    uint16_t *M;
    int seg_chunks;  // 0: not split
};

// Sequence split: where heads x sequences x 128-column tiles leave most of
// the 256 compute units without a workgroup, a sequence is cut into segments
// of seg_chunks chunks.  The recurrence is affine in the state, so each
// segment but a sequence's last first yields its end state from zero (or h0)
// and its K x K transfer matrix (the same recurrence on the unit columns, no
// values), these are composed in order, and then all segments run at once.
// That last run reads h0 from the workspace, where the first has copied it: hL
// may be the same memory, and a last segment may end before a first one begins.
// Sizes only, so that the workspace is known before the call.
//
// seg_chunks fills the card once (256 workgroups of 128 columns), but is at
// least sqrt(chunks): s segments are composed one after another (s x 3.5 us),
// while a segment's two runs take about 4.2 us a chunk each (16 heads of 4096
// steps: segments of 4 chunks 136 us, of 8 118; 8 heads of 2048: 78, 91).
// Only sequences of more than four segments are split, the others lose more
// to the second run and the two launches than they gain.  Measured, K = V =
// 128, bf16, split against whole: 40 heads of 16384 steps 684 against 1025 us,
// 8 heads of 4096 106 against 209, of 2048 78 against 112, 48 of 2048 134
// against 133; below the rule 48 of 1024 90 against 73, 64 of 2048 152
// against 137.  A packed batch is judged as if one sequence were all of it: the
// sequences shorter than a segment cost no second run.
struct DeltaSplit {
    int seg_chunks, segs;  // segs: an upper bound over all sequences
};
inline DeltaSplit delta_split(int batch, int seqlen, int h, int V, int num_seqs)
{
    const long long chunks = delta_chunks(batch, seqlen, num_seqs), nseq = num_seqs ? num_seqs : batch;
    const long long wgs = (long long)h * ((V + 127) / 128);
    if (nseq * wgs > 256) return {0, 0};
    const long long per = num_seqs ? chunks : chunks / batch;  // of the longest sequence
    const long long want = 256 / wgs;                          // segments in all
    long long seg = (chunks + want - 1) / want;
    if (seg < 4) seg = 4;
    while ((seg + 1) * (seg + 1) <= per) ++seg;
    if (per <= 4 * seg) return {0, 0};
    const long long segs = num_seqs ? chunks / seg + num_seqs : batch * ((per + seg - 1) / seg);
    return {int(seg), int(segs)};
}

inline DeltaWs delta_ws(void *workspace, int batch, int seqlen, int h, int K, int V, int num_seqs, bool bwd,
                        size_t *bytes)
{
    size_t n = size_t(delta_chunks(batch, seqlen, num_seqs)) * h;
    DeltaWs w{};
    w.state = (long long)delta_kd(K) * delta_vp(V);
    w.step = 64ll * delta_vp(V);
    w.prep_stride = prep_size(3, bwd);  // three terms at most
    char *p = static_cast<char *>(workspace);
    size_t at = 0;
    auto take = [&](long long each) {
        uint16_t *r = p ? reinterpret_cast<uint16_t *>(p + at) : nullptr;
        at += n * size_t(each) * sizeof(uint16_t);
        return r;
    };
    w.prep = take(w.prep_stride);
    if (bwd) {
        w.S0 = take(3 * w.state);
        w.U = take(3 * w.step);
        w.dS1 = take(3 * w.state);
        w.dX = take(3 * w.step);
    }
    const DeltaSplit split = delta_split(batch, seqlen, h, V, num_seqs);
    w.seg_chunks = split.seg_chunks;
    if (split.segs) {
        n = size_t(split.segs) * h;
        w.N = reinterpret_cast<float *>(take(2 * w.state));
        w.M = take(3ll * delta_kd(K) * delta_kd(K));
    }
    if (bytes) *bytes = at;
    return w;
}

inline DeltaWs delta_ws(const DeltaArgs &a, bool bwd)
{
    return delta_ws(a.workspace, a.batch, a.seqlen, a.h, a.K, a.V, a.cu ? a.nseq : 0, bwd, nullptr);
}

// 16-byte accesses fit every row of a tensor with n elements a row.
inline bool delta_vec(const void *p, const DeltaStride &s, int n, int esize, const DeltaArgs &a, int heads)
{
    const long long per = 16 / esize;
    return n % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.seqlen == 1 || s.t % per == 0) &&
           (heads == 1 || s.h % per == 0) && (a.batch == 1 || s.b % per == 0);
}

// Sum of the first l + 1 log decays of a chunk, for lane l of one wave; in
// double: a step that clears the state (-110) must not cost the later steps'
// differences their low bits.
__device__ inline double decay_sums(float g)
{
    double sum = g < -110.0f ? -110.0f : g;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const double v = __shfl_up(sum, o);
        if (int(threadIdx.x & 63) >= o) sum += v;
    }
    return sum;
}

// 64 steps of a tensor are one buffer of less than 2^31 bytes, and 16-byte
// accesses fit its rows (see TileLoad).
inline bool delta_fast(const void *p, const DeltaStride &s, int n, int esize, const DeltaArgs &a, int heads)
{
    return delta_vec(p, s, n, esize, a, heads) && s.t < (1ll << 31) / 64 / esize;
}

// What one workgroup runs through: chunks [c0, c1) of a sequence.
struct DeltaSegment {
    int seq, index, c0, c1;
    int behind;  // segments of its sequence after it
    bool live;   // there is such a segment (an empty sequence has one)
    bool last;  // of its sequence
    DeltaSeq s;
};
// Segment z: a whole sequence, or with seg_chunks > 0 a part; packed sequence
// i's segments are numbered from chunk0 / seg_chunks + i on, as its chunks are
// (delta_seq).
__device__ inline DeltaSegment delta_segment(const int *cu, int nseq, int seqlen, int seg_chunks, int z)
{
    DeltaSegment d{};
    const int per = (seqlen + kDeltaChunk - 1) / kDeltaChunk;
    if (!seg_chunks) {
        d.seq = z;
    } else if (!cu) {
        const int n = (per + seg_chunks - 1) / seg_chunks;
        d.seq = z / n;
        d.index = z % n;
    } else {
        int lo = 0, hi = nseq - 1;  // the last i whose first segment is at or before z
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (delta_seq(cu, mid, seqlen).chunk0 / seg_chunks + mid <= z) lo = mid;
            else hi = mid - 1;
        }
        d.seq = lo;
        d.index = z - (delta_seq(cu, lo, seqlen).chunk0 / seg_chunks + lo);
    }
    d.s = delta_seq(cu, d.seq, seqlen);
    const int chunks = (d.s.len + kDeltaChunk - 1) / kDeltaChunk;
    d.c0 = seg_chunks ? d.index * seg_chunks : 0;
    d.c1 = seg_chunks ? min(d.c0 + seg_chunks, chunks) : chunks;
    d.live = d.index == 0 || (d.index > 0 && d.c0 < chunks);
    d.last = d.c1 == chunks;
    d.behind = seg_chunks ? max((chunks + seg_chunks - 1) / seg_chunks - 1 - d.index, 0) : 0;
    return d;
}

// f(T{}, TG{}, padded K) for the call's types.
template <typename F>
hipError_t delta_dispatch(bool in_bf16, bool g_bf16, int K, F &&f)
{
    const int kd = delta_kd(K);
    auto sized = [&](auto t, auto tg) {
        return kd == 64 ? f(t, tg, std::integral_constant<int, 64>{})
             : kd == 128 ? f(t, tg, std::integral_constant<int, 128>{})
                         : f(t, tg, std::integral_constant<int, 256>{});
    };
    if (in_bf16) return g_bf16 ? sized(bf16_t{}, bf16_t{}) : sized(bf16_t{}, 0.0f);
    return g_bf16 ? sized(0.0f, bf16_t{}) : sized(0.0f, 0.0f);
}

// One chunk's K, Q, two triangular matrices and decays for the kWaves waves of
// a workgroup.  kAsync (bf16 rows that fit 16-byte accesses): copied straight to
// LDS into the buffer that the chunk before does not use, so that a whole
// chunk's work hides the copy.  Otherwise they wait in registers meanwhile (fp32
// is split into its terms on the way) and there is one buffer.
// kUpper: the record's second half (vec, Tt, Pt); !kNeedQ: without Q.
template <typename T, int KD, int kWaves, bool kFast, bool kAsync, bool kUpper, bool kNeedQ> struct ChunkStage {
    static constexpr int NI = Terms<T>::kIn, NS = Terms<T>::kSum, NCH = KD / 8, kTile = 64 * KD;
    static constexpr int kThreads = 64 * kWaves, kTri = tri_size(NS), kPart = 2 * kTri + 512;
    // fp32 keys of over 128 entries leave LDS for one of K and Q at a time: store()
    // then brings Q (kUpper: K), store_other() the other in its place
    static constexpr bool kOneTile = NI * KD > 512;
    static constexpr int kTiles = kOneTile ? 1 : 2;
    // kAsync: the workgroup's columns of V (or dY) too, 64 steps of kCols
    static constexpr int kCols = 16 * kWaves, kColChunks = kCols / 8, kColTile = kAsync ? 64 * kCols : 0;
    static constexpr int kColRows = kThreads / kColChunks;
    static constexpr int kBuffers = kAsync ? 2 : 1, kBuffer = kTiles * NI * kTile + kPart + kColTile;  // u16 elements
    static constexpr int kPartLoads = (kPart / 8 + kThreads - 1) / kThreads;
    static constexpr int kRows = kThreads / NCH;  // rows of one copy of all threads
    static_assert(!kAsync || (NI == 1 && kFast && kRows % 16 == 0),
                  "rows as they are; the same chunk order in each copy");

    uint16_t *lds;
    const T *kp, *qp;
    const uint16_t *prep;  // the record's half
    long long k_step, q_step, prep_step;
    int len, K;
    TileLoad<T, NCH, kThreads, kFast> lk, lq;
    u32x4 lt[kAsync ? 1 : kPartLoads];
    uint32_t k_off, q_off, c_off, lds0;  // lds0: the wave's place in the first buffer
    const uint16_t *cp;
    long long c_step;
    int wave;

    // The columns from c0 on, n of them there (bf16; kAsync).
    __device__ inline void init_columns(const void *c0, long long cst, int n)
    {
        const int t = int(threadIdx.x) / kColChunks;
        const int c = (chunk_at<kColChunks>(t, int(threadIdx.x) % kColChunks) / 8) % kColChunks;
        cp = static_cast<const uint16_t *>(c0);
        c_step = cst;
        c_off = c * 8 < n ? uint32_t(t * int(cst) + c * 8) * 2u : kOutside;
    }
    // The wave's 16 columns of them as D tile m: a lane's column, steps 16 m + 4 g + {0..3}
    __device__ inline f32x4 column(int c, int m) const
    {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int l = int(threadIdx.x) & 63, r = l & 15, g = l >> 4;
        const int col4 = 16 * (int(threadIdx.x) >> 6) + 4 * (r & 3);
        const uint16_t *tile = buffer(c) + kTiles * NI * kTile + kPart;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(tile + chunk_at<kColChunks>(16 * m + 4 * g + (r >> 2), col4 >> 3) + (col4 & 4)));
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(uint32_t(uint16_t(x[e])) << 16);
        return v;
    }

    // k0, q0: the sequence's first step; rec0: the record of its first chunk,
    // records of a head rec_step elements apart
    __device__ inline void init(uint16_t *buffers, const T *k0, long long kst, const T *q0, long long qst,
                                const uint16_t *rec0, long long rec_step, int length, int n)
    {
        lds = buffers;
        kp = k0;
        qp = q0;
        k_step = kst;
        q_step = qst;
        prep = rec0 + (kUpper ? 2 * kTri : 0);
        prep_step = rec_step;
        len = length;
        K = n;
        wave = wave_of();
        if constexpr (kAsync) {
            lds0 = __builtin_amdgcn_readfirstlane(lds_offset(buffers)) + wave * 1024;
            const int t = int(threadIdx.x) / NCH, c = (chunk_at<NCH>(t, int(threadIdx.x) % NCH) / 8) % NCH;
            k_off = c * 8 < n ? uint32_t(t * int(kst) + c * 8) * 2u : kOutside;
            q_off = c * 8 < n ? uint32_t(t * int(qst) + c * 8) * 2u : kOutside;
        } else {
            lk.init(kst, n);
            lq.init(qst, n);
        }
    }
    __device__ inline uint16_t *buffer(int c) const { return lds + (kAsync ? (c & 1) * kBuffer : 0); }
    __device__ inline const uint16_t *k_tile(int c) const { return buffer(c); }
    __device__ inline const uint16_t *q_tile(int c) const { return buffer(c) + (kTiles - 1) * NI * kTile; }
    __device__ inline const uint16_t *first(int c) const { return buffer(c) + kTiles * NI * kTile + (kUpper ? 512 : 0); }
    __device__ inline const uint16_t *second(int c) const { return first(c) + kTri; }
    __device__ inline const float *vec(int c) const
    {
        return reinterpret_cast<const float *>(buffer(c) + kTiles * NI * kTile + (kUpper ? 0 : 2 * kTri));
    }

    // Starts chunk c's way here.
    __device__ inline void start(int c)
    {
        const int rows = min(len - c * kDeltaChunk, kDeltaChunk);
        const T *k = kp + (long long)c * (kDeltaChunk * k_step), *q = qp + (long long)c * (kDeltaChunk * q_step);
        const uint16_t *part = prep + c * prep_step;
        if constexpr (kAsync) {
            // one buffer a tensor: 64 steps span less than 2^31 bytes
            const uint32_t to = lds0 + (c & 1) * (kBuffer * 2);
            const uint32_t kb = uint32_t(k_step) * 2, qb = uint32_t(q_step) * 2, cb = uint32_t(c_step) * 2;
            const sgpr4 k_buf = copy_buffer(k, rows * kb), q_buf = copy_buffer(q, rows * qb);
            const sgpr4 c_buf = copy_buffer(cp + (long long)c * (kDeltaChunk * c_step), rows * cb);
#pragma unroll
            for (int i = 0; i < 64 / kRows; ++i) {
                copy_to_lds(k_buf, k_off + i * kRows * kb, to + i * kThreads * 16);
                if constexpr (kNeedQ) copy_to_lds(q_buf, q_off + i * kRows * qb, to + kTile * 2 + i * kThreads * 16);
            }
            copy_linear<kPart * 2, kWaves>(part, to - wave * 1024 + 4 * kTile, wave);
#pragma unroll
            for (int i = 0; i < 64 / kColRows; ++i)
                copy_to_lds(c_buf, c_off + i * kColRows * cb, to + 4 * kTile + 2 * kPart + i * kThreads * 16);
        } else {
            lk.fetch(k, k_step, rows, K);
            if constexpr (kNeedQ) lq.fetch(q, q_step, rows, K);
#pragma unroll
            for (int i = 0; i < kPartLoads; ++i) {
                const int at = int(threadIdx.x) + i * kThreads;
                if (at < kPart / 8) lt[i] = reinterpret_cast<const u32x4 *>(part)[at];
            }
        }
    }
    // Chunk c is in its buffer for every wave after this.
    __device__ inline void store(int c)
    {
        if constexpr (!kAsync) {
            const int rows = len - c * kDeltaChunk;
            __syncthreads();  // the last chunk's reads are done
            if constexpr (!kOneTile || kUpper || !kNeedQ) lk.template store<NI>(buffer(c), rows, K);
            if constexpr (kNeedQ && !(kOneTile && kUpper))
                lq.template store<NI>(buffer(c) + (kTiles - 1) * NI * kTile, rows, K);
#pragma unroll
            for (int i = 0; i < kPartLoads; ++i) {
                const int at = int(threadIdx.x) + i * kThreads;
                if (at < kPart / 8) reinterpret_cast<u32x4 *>(buffer(c) + kTiles * NI * kTile)[at] = lt[i];
            }
        }
        __syncthreads();
    }
    __device__ inline void store_other(int c)
    {
        static_assert(!kAsync && kOneTile && kNeedQ, "both tiles are there");
        const int rows = len - c * kDeltaChunk;
        __syncthreads();  // the first tile's reads are done
        if constexpr (kUpper) lq.template store<NI>(buffer(c), rows, K);
        else lk.template store<NI>(buffer(c), rows, K);
        __syncthreads();
    }
};

// How a call's recurrence reads its rows: element by element, in 16-byte runs
// through registers, or copied straight to LDS (bf16, two buffers: K <= 128),
// and then with eight waves a workgroup (128 columns) or four.
enum { kByElement = 0, kByRun = 1, kByCopy = 2 };
template <typename T, int KD> constexpr bool kDeltaAsync = sizeof(T) == 2 && KD <= 128;
// Eight waves share a chunk's copies to LDS, which is what counts once every
// compute unit has a workgroup (160 heads of 2048 steps: 217 us against 300);
// four leave each wave more of a compute unit where twice the workgroups still
// fit the card at one each (96 heads: 154 us against 181, 128: 179 against 200).
inline bool delta_wide(const DeltaArgs &a, bool split)
{
    return a.V > 64 && (split || (long long)a.nseq * a.h * ((a.V + 127) / 128) > 128);
}

// Matrices of every chunk (delta_fwd.hip); both: the transposes too.
hipError_t launch_delta_prep(const DeltaArgs &a, const DeltaWs &ws, bool both, hipStream_t stream);
// The recurrence over the chunks; with ws.S0 the states entering them and U
// are kept.
hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaWs &ws, hipStream_t stream);

}  // namespace ssm
