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

// The largest product first: where it cancels what c holds (U = X + (T - 1) X
// under keys that point the same way), the small ones are then added to what
// is left and not rounded at the size of c.
template <int NA, int NB>
__device__ inline f32x4 mma(const Frag<NA> &a, const Frag<NB> &b, f32x4 c)
{
    constexpr int kOrder = NA == 3 && NB == 3 ? 3 : (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int o = 0; o <= kOrder; ++o)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (o - i >= 0 && o - i < NB) c = mfma16(a.t[i], b.t[o - i], c);
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
// 8 elements of one row as loaded; zeros outside the tensor.
template <typename T> struct Raw8 {
    u32x4 w[sizeof(T) / 2];
};
template <typename T>
__device__ inline Raw8<T> load8(const T *row, int c, int n, bool live, bool vec)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) r.w[i] = u32x4{0, 0, 0, 0};
    if (!live || c * 8 >= n) return r;
    if (vec) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i)
            r.w[i] = reinterpret_cast<const u32x4 *>(row + c * 8)[i];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c * 8 + e < n) {
                if constexpr (sizeof(T) == 4) {
                    r.w[e / 4][e % 4] = __float_as_uint(row[c * 8 + e]);
                } else {
                    r.w[0][e / 2] |= uint32_t(row[c * 8 + e].bits) << (16 * (e % 2));
                }
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

// A tile of 64 rows x 8 NCH columns held by kThreads threads on its way from
// memory to N planes in LDS.
template <typename T, int NCH, int kThreads> struct TileLoad {
    static constexpr int kPer = 64 * NCH / kThreads;
    Raw8<T> raw[kPer];
    // rows of `step` elements from p on, `rows` of them and columns [0, n) exist
    __device__ inline void fetch(const T *p, long long step, int rows, int n, bool vec)
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = int(threadIdx.x) + i * kThreads, t = at / NCH, c = at % NCH;
            raw[i] = load8(p + (long long)t * step, c, n, t < rows, vec);
        }
    }
    template <int N> __device__ inline void store(uint16_t *tile) const
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = int(threadIdx.x) + i * kThreads, t = at / NCH, c = at % NCH;
            const Frag<N> f = terms8<T, N>(raw[i]);
#pragma unroll
            for (int j = 0; j < N; ++j)
                *reinterpret_cast<bf16x8 *>(tile + j * (64 * NCH * 8) + chunk_at<NCH>(t, c)) = f.t[j];
        }
    }
};

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

// ---------------------------------------------------------------- workspace
// Per (chunk record, head), in this order:
//   vec   4 x 64 fp32: e^{G_i}, e^{Gc - G_i}, beta_i e^{G_i}, beta_i
//   T, P  the chunk's lower-triangular matrices T - 1 and P as A fragments
//   Tt, Pt, S0, U, dS1, dX  for the backward pass
// A triangular 64 x 64 matrix is 6 fragments of 16 x 32: row tile r, column
// block b; the columns of a fragment are numbered as two D tiles hold them:
// lane group g's 8 are 32 b + 4 g + {0..3} and 32 b + 16 + 4 g + {0..3}.
constexpr int kTriFrags = 6;
// lower: tiles (0,0) (1,0) (2,0) (2,1) (3,0) (3,1); their transposes' (upper):
// (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
__host__ __device__ constexpr int tri_lower(int r, int b) { return r < 2 ? r : r == 2 ? 2 + b : 4 + b; }
__host__ __device__ constexpr int tri_upper(int r, int b) { return r < 2 ? 2 * r + b : 2 + r; }

}  // namespace ssm
