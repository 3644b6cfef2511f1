// heads_api.hip -- the C ABI declared in include/ssm_heads.h: argument
// validation and dispatch.  Every argument error is detected here, before
// anything is enqueued.
#include "ssm_heads.h"

#include "heads_launch.hpp"
#include "ssm_launch.hpp"
#include "ssm_stride.hpp"

using namespace ssm::check;

namespace {

constexpr int kMaxHeads = 65535;

bool heads_sizes(int batch, int seqlen, int groups, int h, int N, int P, int num_seqs)
{
    return batch >= 1 && batch <= ssm::kMaxBatch && seqlen >= 1 && seqlen <= ssm::kMaxSeqlen && groups >= 1 &&
           h >= groups && h <= kMaxHeads && h % groups == 0 && N >= 1 && N <= ssm::kHeadsMaxN && P >= 1 &&
           P <= ssm::kHeadsMaxP && num_seqs >= 0 && num_seqs <= ssm::kMaxBatch && (num_seqs == 0 || batch == 1) &&
           mul3(batch, seqlen, (long long)h * (P > N ? P : N)) != 0 &&
           // the chunks' states, padded (64 bits of address space to spare)
           (unsigned __int128)ssm::delta_chunks(batch, seqlen, num_seqs) * unsigned(h) *
                   (unsigned long long)((N + 31ll) * (P + 31ll)) < ((unsigned __int128)1 << 48);
}

// The gradients' grid has a workgroup a chunk, and a grid's index less than 2^32
// work-items: sizes whose states may be kept.
bool heads_kept_sizes(int batch, int seqlen, int num_seqs)
{
    return ssm::delta_chunks(batch, seqlen, num_seqs) < (1ll << 32) / ssm::kHeadsGradThreads;
}

}  // namespace

extern "C" {

size_t ssm_head_scan_fwd_workspace_bytes(int batch, int seqlen, int groups, int heads, int N, int P, int num_seqs)
{
    if (!heads_sizes(batch, seqlen, groups, heads, N, P, num_seqs)) return 0;
    return ssm::heads_fwd_workspace_bytes(batch, seqlen, groups, heads, N, P, num_seqs);
}

size_t ssm_head_scan_bwd_workspace_bytes(int batch, int seqlen, int groups, int heads, int N, int P, int num_seqs)
{
    if (!heads_sizes(batch, seqlen, groups, heads, N, P, num_seqs) || !heads_kept_sizes(batch, seqlen, num_seqs)) return 0;
    return ssm::heads_bwd_workspace_bytes(batch, seqlen, groups, heads, N, P, num_seqs);
}

ssm_status_t ssm_head_scan_fwd(int batch, int seqlen, int groups, int heads, int N, int P, ssm_dtype_t in_dtype,
                               unsigned flags, const void *x, const void *dt, const float *dt_bias, const float *A,
                               const void *Bm, const void *Cm, const float *Dskip, const float *h0,
                               const int *cu_seqlens, int num_seqs, ssm_dtype_t out_dtype, void *y, float *hL,
                               void *workspace, size_t workspace_bytes, const ssm_head_scan_layout_t *layout,
                               void *stream)
{
    const int in_t = enum_bits(in_dtype), out_t = enum_bits(out_dtype);
    const bool ckpt = (flags & SSM_FLAG_CHECKPOINTS) != 0;
    if (!x || !dt || !A || !Bm || !Cm || !y || (ckpt && !workspace)) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(out_t)) return SSM_ERR_BAD_DTYPE;
    if (!heads_sizes(batch, seqlen, groups, heads, N, P, num_seqs) || (cu_seqlens && num_seqs < 1) ||
        (!cu_seqlens && num_seqs != 0) || (ckpt && !heads_kept_sizes(batch, seqlen, num_seqs)))
        return SSM_ERR_BAD_SHAPE;
    if (flags & ~SSM_FLAG_CHECKPOINTS) return SSM_ERR_UNSUPPORTED;
    const ssm_head_scan_layout_t dense{};
    const ssm_head_scan_layout_t &lay = layout ? *layout : dense;
    ssm::DeltaStride s[5];
    size_t sp[5];
    // x, dt, B, C, y
    const int nh[5] = {heads, heads, groups, groups, heads}, row[5] = {P, 1, N, N, P};
    for (int i = 0; i < 5; ++i)
        if (!delta_stride(lay.step[i], lay.head[i], lay.batch[i], batch, seqlen, nh[i], row[i], s[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), os = dsize(out_t);
    const int nseq = cu_seqlens ? num_seqs : batch;
    const size_t ws_bytes = ckpt ? ssm::heads_bwd_workspace_bytes(batch, seqlen, groups, heads, N, P, num_seqs)
                                 : ssm::heads_fwd_workspace_bytes(batch, seqlen, groups, heads, N, P, num_seqs);
    if (misaligned(x, es) || misaligned(dt, es) || misaligned(Bm, es) || misaligned(Cm, es) || misaligned(y, os) ||
        misaligned(A, 4) || misaligned(dt_bias, 4) || misaligned(Dskip, 4) || misaligned(h0, 4) || misaligned(hL, 4) ||
        misaligned(cu_seqlens, 4) || (ws_bytes && misaligned(workspace, 16)))
        return SSM_ERR_MISALIGNED;
    if (ws_bytes && (!workspace || workspace_bytes < ws_bytes)) return SSM_ERR_WORKSPACE;
    const size_t hbytes = 4 * size_t(nseq) * heads * N * P, vbytes = 4 * size_t(heads);
    const void *const ptr[5] = {x, dt, Bm, Cm, y};
    const size_t size[5] = {es, es, es, es, os};
    Steps t[5];
    for (int i = 0; i < 5; ++i) t[i] = steps_of(ptr[i], sp[i], size[i], s[i], nh[i], row[i], seqlen, batch);
    const Steps in[] = {t[0], t[1], t[2], t[3], range_of(A, vbytes), range_of(dt_bias, vbytes),
                        range_of(Dskip, vbytes), range_of(h0, hbytes),
                        range_of(cu_seqlens, 4 * (size_t(nseq) + 1))};
    const Steps yb = t[4], wb = range_of(ws_bytes ? workspace : nullptr, ws_bytes), hb = range_of(hL, hbytes);
    for (const Steps &i : in) {
        if (overlaps(yb, i) || overlaps(wb, i)) return SSM_ERR_ALIAS;
        if (!(i.p == h0 && hL == h0) && overlaps(hb, i)) return SSM_ERR_ALIAS;
    }
    if (overlaps(yb, hb) || overlaps(wb, yb) || overlaps(wb, hb)) return SSM_ERR_ALIAS;
    const ssm::HeadsArgs a{batch, seqlen, groups, heads, N, P, in_t == SSM_BF16, out_t == SSM_BF16, nseq, cu_seqlens,
                           x, dt, Bm, Cm, A, Dskip, dt_bias, h0, y, hL, s[0], s[1], s[2], s[3], s[4], workspace, ckpt};
    return ssm::launch_heads_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_head_scan_bwd(int batch, int seqlen, int groups, int heads, int N, int P, ssm_dtype_t in_dtype,
                               unsigned flags, const void *x, const void *dt, const float *dt_bias, const float *A,
                               const void *Bm, const void *Cm, const float *Dskip, const float *h0,
                               const int *cu_seqlens, int num_seqs, ssm_dtype_t grad_dtype, const void *dy,
                               const float *dhL, void *dx, void *ddt, float *ddt_bias, float *dA, void *dBm, void *dCm,
                               float *dDskip, float *dh0, void *workspace, size_t workspace_bytes,
                               const ssm_head_scan_bwd_layout_t *layout, void *stream)
{
    const int in_t = enum_bits(in_dtype), g_t = enum_bits(grad_dtype);
    if (!x || !dt || !A || !Bm || !Cm || !dy || !dx || !ddt || !dA || !dBm || !dCm || !workspace)
        return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(g_t)) return SSM_ERR_BAD_DTYPE;
    if (!heads_sizes(batch, seqlen, groups, heads, N, P, num_seqs) || (cu_seqlens && num_seqs < 1) ||
        (!cu_seqlens && num_seqs != 0) || !heads_kept_sizes(batch, seqlen, num_seqs))
        return SSM_ERR_BAD_SHAPE;
    if (flags & ~SSM_FLAG_CHECKPOINTS) return SSM_ERR_UNSUPPORTED;
    const ssm_head_scan_bwd_layout_t dense{};
    const ssm_head_scan_bwd_layout_t &lay = layout ? *layout : dense;
    ssm::DeltaStride s[9];
    size_t sp[9];
    // x, dt, B, C, dy, dx, ddt, dB, dC
    const int nh[9] = {heads, heads, groups, groups, heads, heads, heads, groups, groups};
    const int row[9] = {P, 1, N, N, P, P, 1, N, N};
    for (int i = 0; i < 9; ++i)
        if (!delta_stride(lay.step[i], lay.head[i], lay.batch[i], batch, seqlen, nh[i], row[i], s[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), gs = dsize(g_t);
    const int nseq = cu_seqlens ? num_seqs : batch;
    const size_t ws_bytes = ssm::heads_bwd_workspace_bytes(batch, seqlen, groups, heads, N, P, num_seqs);
    const void *const ptr[9] = {x, dt, Bm, Cm, dy, dx, ddt, dBm, dCm};
    const size_t size[9] = {es, es, es, es, gs, gs, gs, gs, gs};
    for (int i = 0; i < 9; ++i)
        if (misaligned(ptr[i], size[i])) return SSM_ERR_MISALIGNED;
    const void *const f32[] = {A, dt_bias, Dskip, h0, dhL, cu_seqlens, ddt_bias, dA, dDskip, dh0};
    for (const void *q : f32)
        if (misaligned(q, 4)) return SSM_ERR_MISALIGNED;
    if (misaligned(workspace, 16)) return SSM_ERR_MISALIGNED;
    if (workspace_bytes < ws_bytes) return SSM_ERR_WORKSPACE;
    const size_t hbytes = 4 * size_t(nseq) * heads * N * P, vbytes = 4 * size_t(heads);
    Steps t[9];
    for (int i = 0; i < 9; ++i) t[i] = steps_of(ptr[i], sp[i], size[i], s[i], nh[i], row[i], seqlen, batch);
    const Steps in[] = {t[0], t[1], t[2], t[3], t[4], range_of(A, vbytes), range_of(dt_bias, vbytes),
                        range_of(Dskip, vbytes), range_of(h0, hbytes), range_of(dhL, hbytes),
                        range_of(cu_seqlens, 4 * (size_t(nseq) + 1))};
    const Steps out[] = {t[5], t[6], t[7], t[8], range_of(ddt_bias, vbytes), range_of(dA, vbytes),
                         range_of(dDskip, vbytes), range_of(dh0, hbytes), range_of(workspace, ws_bytes)};
    for (const Steps &o : out) {
        for (const Steps &i : in)
            if (!(o.p == dh0 && i.p == dhL && dh0 == dhL) && overlaps(o, i)) return SSM_ERR_ALIAS;
        for (const Steps &i : out)
            if (&i != &o && overlaps(o, i)) return SSM_ERR_ALIAS;
    }
    ssm::HeadsBwdArgs a{};
    a.f = ssm::HeadsArgs{batch, seqlen, groups, heads, N, P, in_t == SSM_BF16, 0, nseq, cu_seqlens,
                         x, dt, Bm, Cm, A, Dskip, dt_bias, h0, nullptr, nullptr, s[0], s[1], s[2], s[3], {}, workspace,
                         1};
    a.grad_bf16 = g_t == SSM_BF16;
    a.ckpt_given = (flags & SSM_FLAG_CHECKPOINTS) != 0;
    a.dy = dy;
    a.dhL = dhL;
    a.dx = dx;
    a.ddt = ddt;
    a.dB = dBm;
    a.dC = dCm;
    a.dA = dA;
    a.dDskip = dDskip;
    a.ddt_bias = ddt_bias;
    a.dh0 = dh0;
    a.sdy = s[4];
    a.sdx = s[5];
    a.sddt = s[6];
    a.sdB = s[7];
    a.sdC = s[8];
    return ssm::launch_heads_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_head_scan_update(int batch, int groups, int heads, int N, int P, ssm_dtype_t in_dtype, float *state,
                                  int num_slots, const int *slots, const void *x, const void *dt,
                                  const float *dt_bias, const float *A, const void *Bm, const void *Cm,
                                  const float *Dskip, ssm_dtype_t out_dtype, void *y,
                                  const ssm_head_scan_layout_t *layout, void *stream)
{
    const int in_t = enum_bits(in_dtype), out_t = enum_bits(out_dtype);
    if (!state || !x || !dt || !A || !Bm || !Cm || !y) return SSM_ERR_NULL_ARG;
    if (!valid_dtype(in_t) || !valid_dtype(out_t)) return SSM_ERR_BAD_DTYPE;
    if (!heads_sizes(batch, 1, groups, heads, N, P, 0) || num_slots < 1 || (!slots && num_slots != batch) ||
        !mul3(num_slots, heads, (long long)N * P))
        return SSM_ERR_BAD_SHAPE;
    const ssm_head_scan_layout_t dense{};
    const ssm_head_scan_layout_t &lay = layout ? *layout : dense;
    ssm::DeltaStride s[5];
    size_t sp[5];
    const int nh[5] = {heads, heads, groups, groups, heads}, row[5] = {P, 1, N, N, P};
    for (int i = 0; i < 5; ++i)
        if (!delta_stride(0, lay.head[i], lay.batch[i], batch, 1, nh[i], row[i], s[i], sp[i]))
            return SSM_ERR_BAD_SHAPE;
    const size_t es = dsize(in_t), os = dsize(out_t);
    if (misaligned(x, es) || misaligned(dt, es) || misaligned(Bm, es) || misaligned(Cm, es) || misaligned(y, os) ||
        misaligned(A, 4) || misaligned(dt_bias, 4) || misaligned(Dskip, 4) || misaligned(slots, 4) ||
        misaligned(state, 16))
        return SSM_ERR_MISALIGNED;
    const void *const ptr[5] = {x, dt, Bm, Cm, y};
    const size_t size[5] = {es, es, es, es, os};
    const size_t sbytes = 4 * size_t(num_slots) * heads * N * P, vbytes = 4 * size_t(heads);
    Steps t[5];
    for (int i = 0; i < 5; ++i) t[i] = steps_of(ptr[i], sp[i], size[i], s[i], nh[i], row[i], 1, batch);
    const Steps st = range_of(state, sbytes);
    const Steps in[] = {t[0], t[1], t[2], t[3], range_of(A, vbytes), range_of(dt_bias, vbytes),
                        range_of(Dskip, vbytes), range_of(slots, 4 * size_t(batch))};
    for (const Steps &i : in)
        if (overlaps(t[4], i) || overlaps(st, i)) return SSM_ERR_ALIAS;
    if (overlaps(st, t[4])) return SSM_ERR_ALIAS;
    ssm::HeadsUpdateArgs a{};
    a.f = ssm::HeadsArgs{batch, 1, groups, heads, N, P, in_t == SSM_BF16, out_t == SSM_BF16, batch, nullptr,
                         x, dt, Bm, Cm, A, Dskip, dt_bias, nullptr, y, nullptr, s[0], s[1], s[2], s[3], s[4], nullptr,
                         0};
    a.state = state;
    a.slots = slots;
    a.num_slots = num_slots;
    return ssm::launch_heads_update(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
