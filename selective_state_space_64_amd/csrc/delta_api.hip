// delta_api.hip -- the C ABI declared in include/ssm_delta.h: argument
// validation and dispatch.  Every argument error is detected here, before
// anything is enqueued.
#include "ssm_delta.h"

#include <math.h>

#include "delta_launch.hpp"
#include "ssm_check.hpp"
#include "ssm_launch.hpp"

using namespace ssm::check;

namespace {

constexpr int kMaxHeads = 65535;

bool delta_sizes(int batch, int seqlen, int hk, int h, int K, int V, int num_seqs)
{
    return batch >= 1 && batch <= ssm::kMaxBatch && seqlen >= 1 && seqlen <= ssm::kMaxSeqlen && hk >= 1 &&
           h >= hk && h <= kMaxHeads && h % hk == 0 && K >= 1 && K <= ssm::kDeltaMaxK && V >= 1 &&
           V <= ssm::kDeltaMaxV && num_seqs >= 0 && num_seqs <= ssm::kMaxBatch &&
           (num_seqs == 0 || batch == 1) && mul3(batch, seqlen, (long long)h * (V > K ? V : K)) != 0 &&
           // the chunks' states (64 bits of address space to spare)
           mul3(ssm::delta_chunks(batch, seqlen, num_seqs), h, (long long)K * V) != 0 &&
           (unsigned __int128)ssm::delta_chunks(batch, seqlen, num_seqs) * unsigned(h) *
                   (unsigned long long)(K * (long long)V) < ((unsigned __int128)1 << 48);
}

// Strides with defaults filled in and the span in elements of a tensor of
// batch x steps x heads x row elements: false when a stride is negative, two
// elements share a place, or the span reaches 2^56.
bool delta_stride(long long given_t, long long given_h, long long given_b, int batch, int steps, int heads,
                  int row, ssm::DeltaStride &s, size_t &sp)
{
    if (given_t < 0 || given_h < 0 || given_b < 0) return false;
    constexpr __int128 most = (__int128)1 << 56;
    const __int128 dh = given_h ? given_h : row;
    const __int128 dt = given_t ? (__int128)given_t : heads * dh;
    const __int128 db = given_b ? (__int128)given_b : steps * dt;
    if (dh >= most || dt >= most || db >= most) return false;
    struct Dim {
        __int128 stride;
        int n;
    } d[3] = {{dh, heads}, {dt, steps}, {db, batch}};
    for (int i = 0; i < 2; ++i)  // smallest stride first; dimensions of one entry do not count
        for (int j = 0; j < 2 - i; ++j)
            if (d[j].n == 1 ? d[j + 1].n != 1 : (d[j + 1].n != 1 && d[j].stride > d[j + 1].stride)) {
                const Dim t = d[j];
                d[j] = d[j + 1];
                d[j + 1] = t;
            }
    __int128 span = row;  // of everything inside the dimension
    for (const Dim &x : d) {
        if (x.n == 1) continue;
        if (x.stride < span) return false;
        span += x.stride * (x.n - 1);
        if (span >= most) return false;
    }
    // the kernels bound a buffer of rows by rows x step: one step's is a row, whatever the
    // stride that leads to no second one
    s = {steps == 1 ? row : (long long)dt, (long long)dh, (long long)db};
    sp = size_t(span);
    return true;
}

float scale_or_default(const float *scale, int K) { return scale ? *scale : 1.0f / sqrtf(float(K)); }

// A tensor for the overlap check, element strides given: runs of one step's
// heads, and the strides from run to run, the smaller first (the batch's in
// time-major tensors; one that leads nowhere is 0).  Where the heads do not lie
// inside a run, the range alone counts.
Steps steps_of(const void *p, size_t span, size_t es, const ssm::DeltaStride &s, int heads, int row, int seqlen,
               int batch)
{
    const long long run = (heads - 1) * s.h + row, t = seqlen > 1 ? s.t : 0, b = batch > 1 ? s.b : 0;
    const bool time_major = !t || (b && b < t);
    const long long inner = time_major ? b : t, outer = time_major ? t : b;
    if (run > inner) return {p, span * es, span * es, 0, 0};
    return {p, span * es, size_t(run) * es, (long long)(inner * es), (long long)(outer * es)};
}
Steps range_of(const void *p, size_t bytes) { return {p, bytes, bytes, 0, 0}; }

}  // namespace

extern "C" {

size_t ssm_delta_fwd_workspace_bytes(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                                     int num_seqs)
{
    if (!delta_sizes(batch, seqlen, qk_heads, heads, K, V, num_seqs)) return 0;
    return ssm::delta_fwd_workspace_bytes(batch, seqlen, qk_heads, heads, K, V, num_seqs);
}

size_t ssm_delta_bwd_workspace_bytes(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                                     int num_seqs)
{
    if (!delta_sizes(batch, seqlen, qk_heads, heads, K, V, num_seqs)) return 0;
    return ssm::delta_bwd_workspace_bytes(batch, seqlen, qk_heads, heads, K, V, num_seqs);
}

ssm_status_t ssm_delta_fwd(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                           ssm_dtype_t in_dtype, unsigned flags, const float *scale_p, const void *q,
                           const void *k, const void *v, const float *g, const float *beta,
                           const float *h0, const int *cu_seqlens, int num_seqs,
                           ssm_dtype_t out_dtype, void *y, float *hL, void *workspace,
                           size_t workspace_bytes, const ssm_delta_layout_t *layout, void *stream)
{
    const int in_t = enum_bits(in_dtype), out_t = enum_bits(out_dtype);
    const bool ckpt = (flags & SSM_FLAG_CHECKPOINTS) != 0;
    if (!q || !k || !v || !g || !beta || !y || (ckpt && !workspace)) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(out_t)) return SSM_ERR_BAD_DTYPE;
    if (!delta_sizes(batch, seqlen, qk_heads, heads, K, V, num_seqs) || (cu_seqlens && num_seqs < 1) ||
        (!cu_seqlens && num_seqs != 0))
        return SSM_ERR_BAD_SHAPE;
    if (flags & ~SSM_FLAG_CHECKPOINTS) return SSM_ERR_UNSUPPORTED;
    const ssm_delta_layout_t dense{};
    const ssm_delta_layout_t &lay = layout ? *layout : dense;
    ssm::DeltaStride s[6];
    size_t sp[6];
    const int nh[6] = {qk_heads, qk_heads, heads, heads, heads, heads}, row[6] = {K, K, V, V, 1, 1};
    for (int i = 0; i < 6; ++i)
        if (!delta_stride(lay.step[i], lay.head[i], lay.batch[i], batch, seqlen, nh[i], row[i], s[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), os = dsize(out_t);
    const int nseq = cu_seqlens ? num_seqs : batch;
    const size_t ws_bytes = ckpt ? ssm::delta_bwd_workspace_bytes(batch, seqlen, qk_heads, heads, K, V, num_seqs)
                                 : ssm::delta_fwd_workspace_bytes(batch, seqlen, qk_heads, heads, K, V, num_seqs);
    if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(y, os) || misaligned(g, 4) ||
        misaligned(beta, 4) || misaligned(h0, 4) || misaligned(hL, 4) || misaligned(cu_seqlens, 4) ||
        (ws_bytes && misaligned(workspace, 16)))
        return SSM_ERR_MISALIGNED;
    if (ws_bytes && (!workspace || workspace_bytes < ws_bytes)) return SSM_ERR_WORKSPACE;
    const size_t hbytes = 4 * size_t(nseq) * heads * K * V;
    const void *const ptr[6] = {q, k, v, y, g, beta};
    const size_t size[6] = {es, es, es, os, 4, 4};
    Steps t[6];
    for (int i = 0; i < 6; ++i) t[i] = steps_of(ptr[i], sp[i], size[i], s[i], nh[i], row[i], seqlen, batch);
    const Steps in[] = {t[0], t[1], t[2], t[4], t[5], range_of(h0, hbytes),
                        range_of(cu_seqlens, 4 * (size_t(nseq) + 1))};
    const Steps yb = t[3], wb = range_of(ws_bytes ? workspace : nullptr, ws_bytes), hb = range_of(hL, hbytes);
    for (const Steps &i : in) {
        if (overlaps(yb, i) || overlaps(wb, i)) return SSM_ERR_ALIAS;
        if (!(i.p == h0 && hL == h0) && overlaps(hb, i)) return SSM_ERR_ALIAS;
    }
    if (overlaps(yb, hb) || overlaps(wb, yb) || overlaps(wb, hb)) return SSM_ERR_ALIAS;
    const float scale = scale_or_default(scale_p, K);
    const ssm::DeltaArgs a{batch, seqlen, qk_heads, heads, K, V, in_t == SSM_BF16, out_t == SSM_BF16, nseq,
                           cu_seqlens, scale, q, k, v, g, beta, h0, y, hL, s[0], s[1], s[2], s[3], s[4], s[5],
                           workspace, ckpt};
    return ssm::launch_delta_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_delta_bwd(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                           ssm_dtype_t in_dtype, unsigned flags, const float *scale_p, const void *q,
                           const void *k, const void *v, const float *g, const float *beta,
                           const float *h0, const int *cu_seqlens, int num_seqs,
                           ssm_dtype_t grad_dtype, const void *dy, const float *dhL, void *dq,
                           void *dk, void *dv, float *dg, float *dbeta, float *dh0,
                           void *workspace, size_t workspace_bytes,
                           const ssm_delta_bwd_layout_t *layout, void *stream)
{
    const int in_t = enum_bits(in_dtype), g_t = enum_bits(grad_dtype);
    if (!q || !k || !v || !g || !beta || !dy || !dq || !dk || !dv || !dg || !dbeta || !workspace)
        return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(g_t)) return SSM_ERR_BAD_DTYPE;
    if (!delta_sizes(batch, seqlen, qk_heads, heads, K, V, num_seqs) || (cu_seqlens && num_seqs < 1) ||
        (!cu_seqlens && num_seqs != 0))
        return SSM_ERR_BAD_SHAPE;
    if (flags & ~SSM_FLAG_CHECKPOINTS) return SSM_ERR_UNSUPPORTED;
    const ssm_delta_bwd_layout_t dense{};
    const ssm_delta_bwd_layout_t &lay = layout ? *layout : dense;
    ssm::DeltaStride s[9];
    size_t sp[9];
    // q, k, v, g, beta, dy, dq, dk, dv
    const int nh[9] = {qk_heads, qk_heads, heads, heads, heads, heads, qk_heads, qk_heads, heads};
    const int row[9] = {K, K, V, 1, 1, V, K, K, V};
    for (int i = 0; i < 9; ++i)
        if (!delta_stride(lay.step[i], lay.head[i], lay.batch[i], batch, seqlen, nh[i], row[i], s[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), gs = dsize(g_t);
    const int nseq = cu_seqlens ? num_seqs : batch;
    const size_t ws_bytes = ssm::delta_bwd_workspace_bytes(batch, seqlen, qk_heads, heads, K, V, num_seqs);
    for (const void *p : {q, k, v})
        if (misaligned(p, es)) return SSM_ERR_MISALIGNED;
    for (const void *p : {dy, (const void *)dq, (const void *)dk, (const void *)dv})
        if (misaligned(p, gs)) return SSM_ERR_MISALIGNED;
    for (const void *p : {(const void *)g, (const void *)beta, (const void *)h0, (const void *)dhL,
                          (const void *)dg, (const void *)dbeta, (const void *)dh0, (const void *)cu_seqlens})
        if (misaligned(p, 4)) return SSM_ERR_MISALIGNED;
    if (misaligned(workspace, 16)) return SSM_ERR_MISALIGNED;
    if (workspace_bytes < ws_bytes) return SSM_ERR_WORKSPACE;
    const size_t hbytes = 4 * size_t(nseq) * heads * K * V, gbytes = 4 * size_t(batch) * seqlen * heads;
    const void *const ptr[9] = {q, k, v, g, beta, dy, dq, dk, dv};
    const size_t size[9] = {es, es, es, 4, 4, gs, gs, gs, gs};
    Steps t[9];
    for (int i = 0; i < 9; ++i) t[i] = steps_of(ptr[i], sp[i], size[i], s[i], nh[i], row[i], seqlen, batch);
    const Steps in[] = {t[0], t[1], t[2], t[3], t[4], t[5], range_of(h0, hbytes), range_of(dhL, hbytes),
                        range_of(cu_seqlens, 4 * (size_t(nseq) + 1))};
    const Steps out[] = {t[6], t[7], t[8], range_of(dg, gbytes), range_of(dbeta, gbytes), range_of(dh0, hbytes),
                         range_of(workspace, ws_bytes)};
    for (const Steps &o : out) {
        for (const Steps &i : in)
            if (!(o.p == dh0 && i.p == dhL && dh0 == dhL) && overlaps(o, i)) return SSM_ERR_ALIAS;
        for (const Steps &i : out)
            if (&i != &o && overlaps(o, i)) return SSM_ERR_ALIAS;
    }
    const float scale = scale_or_default(scale_p, K);
    ssm::DeltaBwdArgs a{};
    a.f = ssm::DeltaArgs{batch, seqlen, qk_heads, heads, K, V, in_t == SSM_BF16, 0, nseq, cu_seqlens, scale,
                         q, k, v, g, beta, h0, nullptr, nullptr, s[0], s[1], s[2], {}, s[3], s[4], workspace, 1};
    a.grad_bf16 = g_t == SSM_BF16;
    a.ckpt_given = (flags & SSM_FLAG_CHECKPOINTS) != 0;
    a.dy = dy;
    a.dhL = dhL;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    a.dh0 = dh0;
    a.sdy = s[5];
    a.sdq = s[6];
    a.sdk = s[7];
    a.sdv = s[8];
    return ssm::launch_delta_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_delta_update(int batch, int qk_heads, int heads, int K, int V,
                              ssm_dtype_t in_dtype, const float *scale_p, float *state, int num_slots,
                              const int *slots, const void *q, const void *k, const void *v,
                              const float *g, const float *beta, ssm_dtype_t out_dtype, void *y,
                              const ssm_delta_layout_t *layout, void *stream)
{
    const int in_t = enum_bits(in_dtype), out_t = enum_bits(out_dtype);
    if (!state || !q || !k || !v || !g || !beta || !y) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(out_t)) return SSM_ERR_BAD_DTYPE;
    if (!delta_sizes(batch, 1, qk_heads, heads, K, V, 0) || num_slots < 1 || (!slots && num_slots != batch) ||
        !mul3(num_slots, heads, (long long)K * V))
        return SSM_ERR_BAD_SHAPE;
    const ssm_delta_layout_t dense{};
    const ssm_delta_layout_t &lay = layout ? *layout : dense;
    ssm::DeltaStride s[6];
    size_t sp[6];
    const int nh[6] = {qk_heads, qk_heads, heads, heads, heads, heads}, row[6] = {K, K, V, V, 1, 1};
    for (int i = 0; i < 6; ++i)
        if (!delta_stride(0, lay.head[i], lay.batch[i], batch, 1, nh[i], row[i], s[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), os = dsize(out_t);
    if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(y, os) || misaligned(g, 4) ||
        misaligned(beta, 4) || misaligned(slots, 4) || misaligned(state, 16))
        return SSM_ERR_MISALIGNED;
    const void *const ptr[6] = {q, k, v, y, g, beta};
    const size_t size[6] = {es, es, es, os, 4, 4};
    const size_t sbytes = 4 * size_t(num_slots) * heads * K * V;
    Steps t[6];
    for (int i = 0; i < 6; ++i) t[i] = steps_of(ptr[i], sp[i], size[i], s[i], nh[i], row[i], 1, batch);
    const Steps st = range_of(state, sbytes), sl = range_of(slots, 4 * size_t(batch));
    for (int i = 0; i < 6; ++i)
        if ((i != 3 && overlaps(t[3], t[i])) || overlaps(st, t[i])) return SSM_ERR_ALIAS;
    if (overlaps(t[3], sl) || overlaps(st, sl)) return SSM_ERR_ALIAS;
    const float scale = scale_or_default(scale_p, K);
    ssm::DeltaUpdateArgs a{};
    a.f = ssm::DeltaArgs{batch, 1, qk_heads, heads, K, V, in_t == SSM_BF16, out_t == SSM_BF16, batch, nullptr,
                         scale, q, k, v, g, beta, nullptr, y, nullptr, s[0], s[1], s[2], s[3], s[4], s[5],
                         nullptr, 0};
    a.state = state;
    a.slots = slots;
    a.num_slots = num_slots;
    return ssm::launch_delta_update(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
