// delta_launch.hpp -- internal interface of the gated delta rule between the
// C-ABI layer and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace ssm {

// Element strides of one tensor: (b, t, h, i) at b * b_ + t * t_ + h * h_ + i.
struct DeltaStride {
    long long t, h, b;
};

// Sizes and inputs that every delta kernel takes; arguments are validated.
struct DeltaArgs {
    int batch, seqlen, hk, h, K, V;
    int in_bf16, out_bf16;
    int nseq;        // sequences: batch, or the packed ones
    const int *cu;   // packed sequences' bounds, or NULL
    float scale;
    const void *q, *k, *v;
    const float *g, *beta, *h0;
    void *y;
    float *hL;
    DeltaStride sq, sk, sv, sy, sg, sbeta;
    void *workspace;
    int checkpoints;  // leave in the workspace what the backward pass reads
};

struct DeltaBwdArgs {
    DeltaArgs f;  // inputs as in the forward (y, hL unused)
    int grad_bf16, ckpt_given;
    const void *dy;
    const float *dhL;
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dh0;
    DeltaStride sdy, sdq, sdk, sdv;
};

// The decode step: states [slots][h][K][V], row b's state is slots[b] (or b).
struct DeltaUpdateArgs {
    DeltaArgs f;  // seqlen 1; h0, hL, cu unused
    float *state;
    const int *slots;
    int num_slots;
};

constexpr int kDeltaChunk = 64;
constexpr int kDeltaMaxK = 256, kDeltaMaxV = 65536;

// Chunks of all sequences together: an upper bound for packed sequences,
// whose lengths only the device knows (each may end inside a chunk).
inline long long delta_chunks(int batch, int seqlen, int num_seqs)
{
    const long long per = (seqlen + kDeltaChunk - 1) / kDeltaChunk;
    return num_seqs ? per + num_seqs : per * batch;
}

size_t delta_fwd_workspace_bytes(int batch, int seqlen, int hk, int h, int K, int V, int num_seqs);
size_t delta_bwd_workspace_bytes(int batch, int seqlen, int hk, int h, int K, int V, int num_seqs);
hipError_t launch_delta_fwd(const DeltaArgs &a, hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaBwdArgs &a, hipStream_t stream);
hipError_t launch_delta_update(const DeltaUpdateArgs &a, hipStream_t stream);

}  // namespace ssm
