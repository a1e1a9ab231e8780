// Launchers of the operators around the attention call.
#pragma once

#include "../common.cuh"

namespace la {

// SMs of the current device; 0 where it cannot be asked.
inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

// Gated linear recurrence (gated.cu), forward (reverse = 0) and its adjoint (reverse = 1).
struct GatedParams {
    const void* a;             // [T][C] gates
    const void* x;             // [T][C] b (forward) or dh (adjoint)
    const void* h;             // adjoint: [T][C] forward output
    void* y;                   // [T][C] h (forward) or db (adjoint)
    void* da;                  // adjoint: [T][C]
    const float* state_in;     // [nseq][C] or NULL: state before each first token
    const float* edge_in;      // [nseq][C] or NULL: what enters each sequence: state_in / dstate_out
    float* edge_out;           // [nseq][C] or NULL: what leaves it: state_out / dstate_in
    const int32_t* cu_seqlens;
    int nseq;
    int64_t T;
    int C;                     // H d
    // workspace
    WsHeader* hdr;
    int* ticket;
    int* tile_seq;             // [tiles]: 4 x the sequence of its first token, and what boundaries it holds
    float2* run;               // [tiles][Cpad]: product of the gates and state from 0; tiles in scan order
    float2* joint;             // [tiles / 8][Cpad]: the same of each group of 8 tiles
    float* state;              // [tiles / 64][Cpad]: state that leaves each block of 64 tiles
    int Cpad;                  // C rounded up to whole slices
};
size_t gated_workspace_bytes(int64_t T, int C);
cudaError_t gated_force_wait_timeout(int enable);   // test hook behind la_test_force_wait_timeout
cudaError_t gated_scan(GatedParams p, int a_dtype, int dtype, int reverse, void* workspace, cudaStream_t s);
cudaError_t gated_step(const void* a, const void* b, int a_dtype, int dtype, int64_t n, const float* state_in,
                       float* state_out, void* h, cudaStream_t s);

// Layer norm (layer_norm.cu).
cudaError_t layer_norm(const void* x, const float* weight, const float* bias, int dtype, int64_t rows, int groups,
                       int d, float eps, void* y, float* mean, float* rstd, cudaStream_t s);
size_t layer_norm_backward_workspace_bytes(int dtype, int64_t rows, int groups, int d);   // 0: no device
cudaError_t layer_norm_backward(const void* x, const void* dy, const float* weight, const float* mean,
                                const float* rstd, int dtype, int64_t rows, int groups, int d, void* dx,
                                float* dweight, float* dbias, void* workspace, cudaStream_t s);

// Rotary positions (rotary.cu).
struct RotaryParams {
    const void* q;
    const void* k;             // may be NULL
    void* q_out;
    void* k_out;
    const float* freq;         // [P]
    const int32_t* positions;  // [T][naxes]
    int64_t T;
    int H, d, P, naxes;
    int first[LA_MAX_AXES + 1];   // first pair of each axis, and P
    int interleaved, inverse;
};
cudaError_t rotary(const RotaryParams& p, int dtype, cudaStream_t s);

}  // namespace la
