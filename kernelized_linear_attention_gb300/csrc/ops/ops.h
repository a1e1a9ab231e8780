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

// What pairs turn by: pair p of token t by positions[t][axis(p)] freq[p].
struct Turns {
    const float* freq;         // [P]
    const int32_t* positions;  // [T][naxes]
    int P, naxes;
    int first[LA_MAX_AXES + 1];   // first pair of each axis, and P
    int interleaved, inverse;
};

// Rotary positions (rotary.cu).
struct RotaryParams : Turns {
    const void* q;
    const void* k;             // may be NULL
    void* q_out;
    void* k_out;
    int64_t T;
    int H, d;
};
cudaError_t rotary(const RotaryParams& p, int dtype, cudaStream_t s);

// Norm of queries and keys with their rotation (qk_norm_rotary.cu); [0] are the queries, [1] the keys or NULL.
struct QkNormParams : Turns {
    const void* x[2];          // [T][stride]: a token's rows [H][d] next to one another
    const void* dy[2];         // backward: [T][H][d]
    void* y[2];                // [T][H][d] outputs (forward) or dx (backward)
    const float* w[2];         // [d], or [H][d] per head, or NULL
    float* rstd[2];            // [T][H]: written if not NULL (forward), read (backward)
    float* dw[2];              // backward: as w, or NULL
    float* partial;            // backward: [blocks along tokens][H of both][d], or, where heads share a weight,
                               // [blocks][2][d] (of q, of k); NULL: no gradients of weights
    int64_t stride[2];         // of x's tokens, in elements
    int64_t T;
    int H[2];
    int d, per_head;
    float eps;
};
cudaError_t qk_norm_rotary(const QkNormParams& p, int dtype, cudaStream_t s);
size_t qk_norm_rotary_backward_workspace_bytes(int64_t T, int H, int d);   // H of both; 0: no device
cudaError_t qk_norm_rotary_backward(const QkNormParams& p, int dtype, cudaStream_t s);

}  // namespace la
