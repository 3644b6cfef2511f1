// heads_launch.hpp -- internal interface of the head-wise selective scan
// between the C-ABI layer and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "delta_launch.hpp"

namespace ssm {

// Sizes and inputs that every kernel takes; arguments are validated.
struct HeadsArgs {
    int batch, seqlen, groups, h, N, P;
    int in_bf16, out_bf16;
    int nseq;       // sequences: batch, or the packed ones
    const int *cu;  // packed sequences' bounds, or NULL
    const void *x, *dt, *B, *C;
    const float *A, *Dskip, *dt_bias, *h0;
    void *y;
    float *hL;
    DeltaStride sx, sdt, sB, sC, sy;
    void *workspace;
    int checkpoints;  // leave in the workspace what the backward pass reads
};

struct HeadsBwdArgs {
    HeadsArgs f;  // inputs as in the forward (y, hL unused)
    int grad_bf16, ckpt_given;
    const void *dy;
    const float *dhL;
    void *dx, *ddt, *dB, *dC;
    float *dA, *dDskip, *ddt_bias, *dh0;
    DeltaStride sdy, sdx, sddt, sdB, sdC;
};

// The decode step: states [slots][h][N][P], row b's state is slots[b] (or b).
struct HeadsUpdateArgs {
    HeadsArgs f;  // seqlen 1; h0, hL, cu unused
    float *state;
    const int *slots;
    int num_slots;
};

constexpr int kHeadsMaxN = 256, kHeadsMaxP = 65536;
constexpr int kHeadsGradThreads = 512;  // of a workgroup of the gradients

size_t heads_fwd_workspace_bytes(int batch, int seqlen, int groups, int h, int N, int P, int num_seqs);
size_t heads_bwd_workspace_bytes(int batch, int seqlen, int groups, int h, int N, int P, int num_seqs);
hipError_t launch_heads_fwd(const HeadsArgs &a, hipStream_t stream);
hipError_t launch_heads_bwd(const HeadsBwdArgs &a, hipStream_t stream);
hipError_t launch_heads_update(const HeadsUpdateArgs &a, hipStream_t stream);

}  // namespace ssm
