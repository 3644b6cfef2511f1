// delta_mfma.hpp -- matrix-core building blocks of the chunked delta rule
// (gfx950).
//
// Products run as v_mfma_f32_16x16x32_bf16 (fp32 sums).  An operand that is
// not exact in bf16 is a sum of N bf16 terms, each the rounding of what the
// earlier ones leave (N = 2: 16 bits of significand, 3: 24), and a product
// of split operands keeps the pairs of terms up to order max(NA, NB) - 1, and
// of order 3 for 3 x 3 terms (where a sum cancels, the pairs of 2^-24 each
// that this adds cost 3 times the error of fp32 products if left out).
// Two terms cost at most 3 matrix instructions where an fp32 one costs 16.
//
// Lane l = 16 g + r of a wave holds
//   A (16 x 32):  row r, columns 8 g .. 8 g + 7
//   B (32 x 16):  column r, rows 8 g .. 8 g + 7
//   D (16 x 16):  column r, rows 4 g .. 4 g + 3
// The contraction index may be numbered freely as long as A and B agree, so a
// product's result D is the next product's B without leaving the lane: two D
// tiles give the 8 rows of B, and A is read from memory in that numbering.
#pragma once

#include "delta_launch.hpp"
#include "ssm_device.hpp"

namespace ssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ inline f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x4 mfma16_f32(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <int N> struct Frag {
    bf16x8 t[N];
};

// f(i, j) for the pairs of terms that a product keeps, the largest first: where
// it cancels what the sum holds (U = X + (T - 1) X under keys that point the
// same way), the small ones are then added to what is left and not rounded at
// the size of the sum.  Several products' pairs are issued in turn, so that no
// matrix instruction waits for the one before it.
template <int NA, int NB> constexpr int kTermOrder = NA == 3 && NB == 3 ? 3 : (NA > NB ? NA : NB) - 1;
template <int NA, int NB, typename F> __device__ inline void for_terms(F &&f)
{
    constexpr int kOrder = kTermOrder<NA, NB>;
#pragma unroll
    for (int o = 0; o <= kOrder; ++o)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (o - i >= 0 && o - i < NB) f(i, o - i);
}
template <int NA, int NB>
__device__ inline f32x4 mma(const Frag<NA> &a, const Frag<NB> &b, f32x4 c)
{
    for_terms<NA, NB>([&](int i, int j) { c = mfma16(a.t[i], b.t[j], c); });
    return c;
}

// Two values to bf16, leaving what is lost in them.
__device__ inline uint32_t split_pair(float &x, float &y)
{
    const uint32_t w = pack_bf16x2(x, y);
    x -= io<bf16_t>::lo(w);
    y -= io<bf16_t>::hi(w);
    return w;
}
template <int N>
__device__ inline Frag<N> split8(float v0, float v1, float v2, float v3, float v4, float v5, float v6, float v7)
{
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u32x4 w;
        if (i + 1 < N) {
            w = u32x4{split_pair(v0, v1), split_pair(v2, v3), split_pair(v4, v5), split_pair(v6, v7)};
        } else {
            w = u32x4{pack_bf16x2(v0, v1), pack_bf16x2(v2, v3), pack_bf16x2(v4, v5), pack_bf16x2(v6, v7)};
        }
        f.t[i] = __builtin_bit_cast(bf16x8, w);
    }
    return f;
}
template <int N> __device__ inline Frag<N> split8(f32x4 a, f32x4 b)
{
    return split8<N>(a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]);
}

// Keeps the instructions before it before those after it.
__device__ inline void fence() { __builtin_amdgcn_sched_barrier(0); }

// Ends a block of matrix instructions that some waves skip: ten wait states, after
// which any result may be read.  The hardware does not wait by itself; the compiler
// counts the states between a product and its use along the paths through the code,
// but has missed the short one where such a block is joined (three states of eight
// in the gradients with shared fp32 keys of more than 128 entries).
__device__ inline void settle()
{
    fence();
    asm volatile("s_nop 7\n\ts_nop 1");
    fence();
}

// Orders what stands before it since the last fence: kReads LDS reads (of the
// next phase) first, then kMatrix matrix instructions with kValu others behind
// each.
template <int kReads, int kMatrix, int kValu> __device__ inline void interleave()
{
    if constexpr (kReads > 0) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
#pragma unroll
    for (int i = 0; i < kMatrix; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if constexpr (kValu > 0) __builtin_amdgcn_sched_group_barrier(0x2, kValu, 0);
    }
}

// ---------------------------------------------------------------- LDS tiles
// A tile of rows of NCH 16-byte chunks (8 bf16 each); a row's chunks are
// permuted so that 16 rows' same chunk lie in different banks.
template <int NCH> __device__ inline int chunk_at(int t, int c)
{
    const int s = NCH >= 16 ? (t & 15) : NCH == 8 ? ((t >> 1) & 7) : ((t >> 2) & 3);
    return (t * NCH + (c ^ s)) * 8;
}
// 8 neighbouring elements of row t
template <int NCH> __device__ inline bf16x8 read_row(const uint16_t *tile, int t, int c)
{
    return *reinterpret_cast<const bf16x8 *>(tile + chunk_at<NCH>(t, c));
}
// Columns of the tile as a lane's 8 elements: element j of a lane with
// r = lane % 16 is tile[ta + j][col(r)] (j < 4), tile[tb + j - 4][col(r)];
// `col` is the column that this lane's r / 4-th quarter hands in: the
// hardware's transposing read takes, from lane 4 a + b of 16, the 4 elements
// at row ta + a and column col4, and gives lane r column r % 4 of quarter
// r / 4.  So lane 4 a + b passes col4 = the first column of quarter b.
template <int NCH> __device__ inline bf16x8 read_cols(const uint16_t *tile, int ta, int tb, int col4)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int a = (int(threadIdx.x) & 15) >> 2;
    const int h = col4 & 4, c = col4 >> 3;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4 *)(tile + chunk_at<NCH>(ta + a, c) + h));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4 *)(tile + chunk_at<NCH>(tb + a, c) + h));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 v = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// ---------------------------------------------------------------- staging
// 8 elements of one row as loaded.  Loads in flight must not meet a use or a
// branch of their own, so places outside the tensor are loaded from a place
// inside it and cleared when the tile is stored.
template <typename T> struct Raw8 {
    u32x4 w[sizeof(T) / 2];
};
// columns [8 c, 8 c + 8) of the n that exist (n >= 1), element by element
template <typename T> __device__ inline Raw8<T> load8(const T *row, int c, int n)
{
    Raw8<T> r;
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const T *p = row + min(c * 8 + e, n - 1);
        if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(*p);
        else v[e] = p->bits;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 4) r.w[e / 4][e % 4] = v[e];
        else if (e % 2) r.w[0][e / 2] |= v[e] << 16;
        else r.w[0][e / 2] = v[e];
    }
    return r;
}
// Zeros from element `count` on.
template <typename T> __device__ inline Raw8<T> keep8(Raw8<T> r, int count)
{
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * 2); ++i) {
        uint32_t &w = reinterpret_cast<uint32_t *>(r.w)[i];
        if constexpr (sizeof(T) == 4) {
            w = i < count ? w : 0u;
        } else {
            w = 2 * i + 1 < count ? w : 2 * i < count ? w & 0xffffu : 0u;
        }
    }
    return r;
}
// The same as N bf16 terms.
template <typename T, int N> __device__ inline Frag<N> terms8(const Raw8<T> &r)
{
    if constexpr (sizeof(T) == 2) {
        static_assert(N == 1, "bf16 is exact in one term");
        Frag<N> f;
        f.t[0] = __builtin_bit_cast(bf16x8, r.w[0]);
        return f;
    } else {
        float v[8];
        io<float>::unpack(r.w[0], v);
        io<float>::unpack(r.w[1], v + 4);
        return split8<N>(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
    }
}

// Buffer descriptor of `bytes` bytes from p on (p the same in every lane):
// loads outside give 0, stores outside are dropped; a negative size is empty.
__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void *p, long long bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, max(int(bytes), 0), 0x00020000);
}
constexpr uint32_t kOutside = 0x80000000u;  // past every buffer, also with 2^31 added

// Tensor rows as the kernels walk them.  kFast: 16-byte loads fit every row
// and 64 steps span less than 2^31 bytes, so that a chunk is one buffer whose
// bounds stand for the masks of steps and columns, and a lane's offsets are
// the same in every chunk; otherwise element loads with 64-bit addresses.

// A tile of 64 rows x 8 NCH columns held by kThreads threads on its way from
// memory to N planes in LDS.
template <typename T, int NCH, int kThreads, bool kFast> struct TileLoad {
    static constexpr int kPer = 64 * NCH / kThreads, kRows = kThreads / NCH;  // rows of one load of all threads
    Raw8<T> raw[kPer];
    uint32_t off;
    // rows of `step` elements, columns [0, n) exist (n < 1: none)
    __device__ inline void init(long long step, int n)
    {
        if constexpr (kFast) {
            const int t = int(threadIdx.x) / NCH, c = int(threadIdx.x) % NCH;
            off = c * 8 < n ? uint32_t(t * int(step) + c * 8) * uint32_t(sizeof(T)) : kOutside;
        }
    }
    // from p on; rows >= 1
    __device__ inline void fetch(const T *p, long long step, int rows, int n)
    {
        if constexpr (kFast) {
            // a buffer for each run of rows: the offset in it is the same
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int left = min(rows - i * kRows, kRows);
                // rows that are not there (left < 1): a negative size
                const auto buf = buffer_of(p + (long long)(i * kRows) * step, n < 1 ? 0 : left * step * (long long)sizeof(T));
#pragma unroll
                for (int w = 0; w < int(sizeof(T) / 2); ++w)
                    raw[i].w[w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off + 16 * w, 0, 0));
            }
        } else {
            if (n < 1) return;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int at = int(threadIdx.x) + i * kThreads, t = at / NCH, c = at % NCH;
                raw[i] = load8(p + (long long)min(t, rows - 1) * step, c, n);
            }
        }
    }
    // with the same rows and n
    __device__ inline Raw8<T> at(int i, int rows, int n) const
    {
        if constexpr (kFast) return raw[i];
        const int a = int(threadIdx.x) + i * kThreads;
        return keep8(raw[i], a / NCH < rows ? n - a % NCH * 8 : 0);
    }
    template <int N> __device__ inline void store(uint16_t *tile, int rows, int n) const
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int a = int(threadIdx.x) + i * kThreads, t = a / NCH, c = a % NCH;
            const Frag<N> f = terms8<T, N>(at(i, rows, n));
#pragma unroll
            for (int j = 0; j < N; ++j)
                *reinterpret_cast<bf16x8 *>(tile + j * (64 * NCH * 8) + chunk_at<NCH>(t, c)) = f.t[j];
        }
    }
};

// One column's 16 elements of a 64-step chunk in the order of four D tiles:
// steps 16 m + 4 g + e.  A buffer for each tile, its bound the last step.
template <typename T, bool kFast> struct Column {
    T raw[16];
    // p: column 0
    __device__ inline void fetch(const T *p, long long step, int rows, int g, int col, bool live)
    {
        if constexpr (kFast) {
            const uint32_t off = live ? uint32_t(4 * g * int(step) + col) * uint32_t(sizeof(T)) : kOutside;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const auto buf = buffer_of(p + (long long)(16 * m) * step, (long long)min(rows - 16 * m, 16) * step * sizeof(T));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t o = off + uint32_t(e * int(step)) * uint32_t(sizeof(T));
                    if constexpr (sizeof(T) == 4)
                        raw[4 * m + e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, o, 0, 0));
                    else
                        raw[4 * m + e].bits = __builtin_amdgcn_raw_buffer_load_b16(buf, o, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                raw[i] = p[(long long)min(16 * (i / 4) + 4 * g + i % 4, rows - 1) * step + (live ? col : 0)];
        }
    }
    __device__ inline f32x4 tile(int m, int rows, int g, bool live) const
    {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = io<T>::load1(&raw[4 * m + e]);
            if (!kFast) v[e] = live && 16 * m + 4 * g + e < rows ? v[e] : 0.0f;
        }
        return v;
    }
};

// Stores one column's steps in the same order.
template <typename T, bool kFast>
__device__ inline void store_column(T *p, long long step, int rows, int g, int col, bool live, const f32x4 *v)
{
    const uint32_t off = live ? uint32_t(4 * g * int(step) + col) * uint32_t(sizeof(T)) : kOutside;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const auto buf = buffer_of(p + (long long)(16 * m) * step, (long long)min(rows - 16 * m, 16) * step * sizeof(T));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t o = off + uint32_t(e * int(step)) * uint32_t(sizeof(T));
            if constexpr (!kFast) {
                const int i = 16 * m + 4 * g + e;
                if (live && i < rows) {
                    if constexpr (sizeof(T) == 4) p[(long long)i * step + col] = v[m][e];
                    else p[(long long)i * step + col].bits = uint16_t(pack_bf16x2(v[m][e], v[m][e]));
                }
            } else if constexpr (sizeof(T) == 4) {
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[m][e]), buf, o, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b16(uint16_t(pack_bf16x2(v[m][e], v[m][e])), buf, o, 0, 0);
            }
        }
    }
}

// ---------------------------------------------------------------- copies to LDS
// 64 lanes x 16 bytes from a buffer straight into LDS at byte offset `lds`
// (+ 16 a lane); places outside the buffer give 0.  The data are there for the
// wave after wait_loads(), for the workgroup after a barrier behind that.  In
// asm because the compiler would put a wait for the copy before every later
// LDS read that it cannot tell apart from the copy's place.
typedef unsigned int sgpr4 __attribute__((ext_vector_type(4)));
__device__ inline sgpr4 copy_buffer(const void *p, long long bytes)
{
    const unsigned long long a = reinterpret_cast<unsigned long long>(p);
    return sgpr4{unsigned(a), unsigned(a >> 32) & 0xffffu, unsigned(max(int(bytes), 0)), 0x00020000u};
}
__device__ inline uint32_t lds_offset(const void *p)
{
    return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}
// (lds: the same in every lane)
// The copy wants one wait state behind the write of m0, and five behind a vector
// instruction that wrote an SGPR of `buf` (readfirstlane, a spill's return): the
// compiler keeps neither inside an asm block, so the s_nop is there for both.  m0 is
// a reserved register, which the compiler sets anew wherever it needs it: it does not
// belong on the clobber list.
__device__ inline void copy_to_lds(sgpr4 buf, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(buf)
                 : "memory");
}
// Until at most N of the wave's vector-memory operations are under way (they
// end in order).
template <int N> __device__ inline void wait_loads()
{
    static_assert(N < 64, "the counter has 6 bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ inline int wave_of() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6); }
// kBytes (a multiple of 1 KB) of memory to LDS, spread over kWaves waves
template <int kBytes, int kWaves> __device__ inline void copy_linear(const void *p, uint32_t lds, int wave)
{
    const sgpr4 buf = copy_buffer(p, kBytes);
#pragma unroll
    for (int i = 0; i < kBytes / 1024; i += kWaves) {
        const int at = (i + wave) * 1024;
        if (i + kWaves <= kBytes / 1024 || at < kBytes)
            copy_to_lds(buf, uint32_t(i * 1024) + threadIdx.x * 16, lds + at);
    }
}

// ---------------------------------------------------------------- records
// S0, dS1 (K x V), U, dX (64 x V) of a chunk are kept as the B fragments that
// the recurrences form of them: [16 columns][block of 32 rows][term][lane][8].
// A lane's place is its own but for one bit, so that reading a fragment across
// (record_cols) meets every LDS bank once.
__device__ inline int record_lane(int g, int r) { return g * 16 + (r ^ ((g & 1) << 2)); }
template <int N, int NB>
__device__ inline void record_store(uint16_t *rec, int col_tile, int b, const Frag<N> &f)
{
    const int l = int(threadIdx.x) & 63;
#pragma unroll
    for (int n = 0; n < N; ++n)
        *reinterpret_cast<bf16x8 *>(rec + (long long)((col_tile * NB + b) * N + n) * 512 +
                                    record_lane(l >> 4, l & 15) * 8) = f.t[n];
}
// From a record's 32 columns in LDS: the lane's columns 8 g + {0..7} of one row.
// As in read_cols, each quarter b of 16 lanes hands in the place of four rows,
// and lane r gets row r % 4 of quarter r / 4's: (block, lane group, half of the
// lane's 8) name the four rows that this lane's l % 4-th quarter means.
template <int N, int NB>
__device__ inline Frag<N> record_cols(const uint16_t *rec, int b, int lg, int half)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const int l = int(threadIdx.x) & 63, g = l >> 4, a = (l & 15) >> 2;
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint16_t *t = rec + (((g >> 1) * NB + b) * N + n) * 512 + half * 4;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(t + record_lane(lg, 8 * (g & 1) + a) * 8));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(t + record_lane(lg, 8 * (g & 1) + 4 + a) * 8));
        f.t[n] = __builtin_bit_cast(bf16x8, s16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    }
    return f;
}

// ---------------------------------------------------------------- chunks
// The steps of one sequence: `first` in batch row `batch`, `len` of them; its
// chunks' records in the workspace start at `chunk0`.
struct DeltaSeq {
    long long first;
    int batch, len, chunk0;
};
// Packed sequence i starts its records at first / 64 + i: that leaves room
// for every chunk of every sequence (a sequence's chunks are at most one more
// than the multiples of 64 it spans) without a sum over the sequences.
__device__ inline DeltaSeq delta_seq(const int *cu, int i, int seqlen)
{
    if (!cu) return {0, i, seqlen, i * ((seqlen + kDeltaChunk - 1) / kDeltaChunk)};
    const int lo = min(max(cu[i], 0), seqlen);
    const int hi = min(max(cu[i + 1], lo), seqlen);
    return {lo, 0, hi - lo, lo / kDeltaChunk + i};
}
// The sequence that record `chunk` belongs to.
__device__ inline int delta_seq_of(const int *cu, int nseq, int seqlen, int chunk)
{
    if (!cu) return chunk / ((seqlen + kDeltaChunk - 1) / kDeltaChunk);
    int lo = 0, hi = nseq - 1;  // the last i with first_i / 64 + i <= chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (min(max(cu[mid], 0), seqlen) / kDeltaChunk + mid <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------- a chunk's matrices
// Per (chunk record, head), in this order:
//   T, P    the chunk's lower-triangular matrices T - 1 and P as A fragments
//   vec     4 x 64 fp32: e^{G_i}, e^{Gc - G_i}, beta_i e^{G_i}, beta_i
//   Tt, Pt  their transposes', for the backward pass
// A triangular 64 x 64 matrix is 6 fragments of 16 x 32: row tile r, column
// block b; the columns of a fragment are numbered as two D tiles hold them:
// lane group g's 8 are 32 b + 4 g + {0..3} and 32 b + 16 + 4 g + {0..3}.
constexpr int kTriFrags = 6;
// lower: tiles (0,0) (1,0) (2,0) (2,1) (3,0) (3,1); their transposes' (upper):
// (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
__host__ __device__ constexpr int tri_lower(int r, int b) { return r < 2 ? r : r == 2 ? 2 + b : 4 + b; }
__host__ __device__ constexpr int tri_upper(int r, int b) { return r < 2 ? 2 * r + b : 2 + r; }
// u16 elements of one, and of the record up to vec and in all, for N terms
constexpr int tri_size(int n) { return kTriFrags * n * 512; }
constexpr int prep_size(int n, bool both) { return (both ? 4 : 2) * tri_size(n) + 512; }

}  // namespace ssm
