// kda_layers_internal.h -- launch descriptors of the operators of kda_layers.h.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// An address in elements: with the row strides, what a vector access has to divide.
inline long long elements(const void *p, bool bf16) { return (long long)((uintptr_t)p / (bf16 ? 2 : 4)); }

// Records opts->events[i] ahead of launch i (if given) and counts the launches.
struct LaunchMarks {
    cudaEvent_t *events;
    int n, i;
    void mark(cudaStream_t st) {
        if (events && i < n) cudaEventRecord(events[i], st);
        ++i;
    }
    void end(cudaStream_t st) {
        if (events && i < n) cudaEventRecord(events[i], st);
    }
};

struct ConvArgs {
    const void *x, *w, *bias, *state0;   // bias, state0 nullable
    void *y, *state_T;                   // state_T nullable
    const void *dy;                      // backward
    const float *dstate_T;               // nullable
    void *dx;
    float *dw, *dbias, *dstate0;         // dbias, dstate0 nullable
    const int *cu;
    int S, D, K, silu;
    long long T, rows;                   // rows a sequence (dense) or in all (packed); rows in all
    long long ld_x, ld_y, ld_dx;
    bool bf16;
    void *workspace;
    LaunchMarks *marks;
};
size_t short_conv_bwd_workspace_bytes(long long rows, int D, int K);
cudaError_t launch_short_conv_fwd(const ConvArgs &a, cudaStream_t st);
cudaError_t launch_short_conv_bwd(const ConvArgs &a, cudaStream_t st);
// x, y [S, D], state0 -> state_T (may be the same)
cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t st);

// Rows a span of the selective scan has at least, but the last of a sequence (the backward's; the
// forward's have 64): what bounds their number, and with it the sizes that a call may have.
constexpr int kShortestSpan = 16;

struct SsmArgs {
    const void *u, *dt, *Bm, *Cm, *z;    // z nullable
    const float *A, *Dskip, *dt_bias;    // Dskip, dt_bias nullable
    const float *h0;                     // nullable
    void *out;
    float *h_T;                          // nullable
    const void *dout;                    // backward
    const float *dh_T;                   // nullable
    void *du, *ddt, *dB, *dC, *dz;
    float *dA, *dDskip, *ddt_bias, *dh0; // the last three nullable
    const int *cu;
    int S, D, N, G, softplus;
    long long T, rows;
    long long ld_u, ld_dt, ld_z, ld_B, ld_C, ld_out;
    bool bf16;
    void *workspace;
    LaunchMarks *marks;
};
size_t ssm_scan_fwd_workspace_bytes(const SsmArgs &a);
size_t ssm_scan_bwd_workspace_bytes(const SsmArgs &a);
cudaError_t launch_ssm_scan_fwd(const SsmArgs &a, cudaStream_t st);
cudaError_t launch_ssm_scan_bwd(const SsmArgs &a, cudaStream_t st);
// one token a sequence, h0 -> h_T (may be the same)
cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t st);

struct NormArgs {
    const void *residual, *block, *gate;      // backward: residual is the forward's res_out
    const float *scale, *w_post, *w_pre;
    void *res_out, *x;
    const void *dres, *dx;
    void *dresidual, *dblock, *dgate;
    float *dscale, *dw_post, *dw_pre;
    int rows, D;
    float eps;
    long long ld_res, ld_block, ld_gate;
    bool bf16;
    void *workspace;
    LaunchMarks *marks;
};
size_t block_norm_bwd_workspace_bytes(int rows, int D);
cudaError_t launch_block_norm_fwd(const NormArgs &a, cudaStream_t st);
cudaError_t launch_block_norm_bwd(const NormArgs &a, cudaStream_t st);

// Zeroes the rows of a packed call that belong to no sequence: before cu[0], from cu[S] on.
// Up to five outputs of `bytes[i]` a row, rows `pitch[i]` bytes apart.
struct ZeroRest {
    void *p[5];
    long long bytes[5], pitch[5];
    int count;
};
cudaError_t launch_zero_rest(const ZeroRest &z, const int *cu, int S, long long T, cudaStream_t st);

}  // namespace kda
