// Linear attention with a decay for each head: parameters, work table and launchers.
#pragma once

#include "chain.cuh"
#include "ops.h"

namespace la {

// A segment of one packed sequence: tokens [start, end).  `place` is the segment's slot times 4, plus 1 for a
// sequence's first segment and 2 for its last.  Segment c of a sequence has the slot (slots of earlier sequences) + c;
// a sequence of m segments owns m - 1 slots, one for each boundary between two of them: slot c is what segment c
// leaves to segment c + 1 (forward), or segment c + 1 to segment c (reverse).
struct DecaySegment {
    int seq, start, end, place;
};
__host__ __device__ inline bool decay_first(const DecaySegment& g) { return g.place & 1; }
__host__ __device__ inline bool decay_last(const DecaySegment& g) { return g.place & 2; }
__host__ __device__ inline int decay_slot(const DecaySegment& g) { return g.place >> 2; }

__host__ __device__ inline int decay_segments(int tokens, int L) { return tokens / L + (tokens % L != 0); }

struct DecayCall {
    const float* log_decay;      // [H]
    const int32_t* cu_seqlens;   // or NULL
    int nseq;
    int64_t T;
    int H, dk, dv;
    float scale;
    // workspace
    WsHeader* hdr;
    int* slot_first;             // [nseq + 1]: slots of earlier sequences      (cu_seqlens only)
    int* segment_first;          // [nseq + 1]: segments of earlier sequences   (cu_seqlens only)
    DecaySegment* table;         // [segments]                                  (cu_seqlens only)
    float* states[2];            // [slots][H][dk][dv]: forward, reverse
    int L;                       // tokens of a segment
    int segments;                // an upper bound on them (exact without cu_seqlens)
    int64_t slots;               // likewise
};

// One product pass.  Forward: out_i = sum_(j <= i) g^(i-j) (x_i . y_j) z_j + g^(i - first + 1) x_i^T S, with S what enters
// the segment; reverse: out_i = sum_(j >= i) g^(j-i) (x_i . y_j) z_j + g^(last - i) x_i^T E.  The products are scaled by
// `scale`, and x^T S too (E holds it already).
//   outputs        x = q,   y = k,   z = v, forward
//   gradient of q  x = dout, y = v,   z = k, forward, S transposed
//   gradient of k  x = v,   y = dout, z = q, reverse, E transposed
//   gradient of v  x = k,   y = q,   z = dout, reverse
struct DecayPass {
    const void* x;               // [T][H][ds]
    const void* y;               // [T][H][ds]
    const void* z;               // [T][H][dz]
    void* out;                   // [T][H][dz]
    int ds, dz;
    int reverse, transposed;     // states are [dk][dv]: [ds][dz], or transposed [dz][ds]
    const float* edge;           // [nseq][H][dk][dv] or NULL: what enters each sequence
};

// One state pass: sum over a segment's tokens of w_j y_j z_j^T, with w_j = g^(last - j) (forward; y = k, z = v) or
// scale g^(j - first + 1) (reverse; y = q, z = dout).
struct DecayStates {
    const void* y;               // [T][H][dk]
    const void* z;               // [T][H][dv]
    int reverse;
    const float* edge_in;        // [nseq][H][dk][dv] or NULL: what enters each sequence
    float* edge_out;             // [nseq][H][dk][dv] or NULL: what leaves it
};

// Which segments a state pass sums.  Inner: those that another one follows.  All: the ones at the sequences' ends too,
// whose sums wait in edge_out for the join to add what enters them.  Ends: these alone, with what enters them (where
// edge_out is edge_in, which the products still need, the ends come behind them).
enum DecayWhich { kInner, kAll, kEnds };

size_t decay_layout(DecayCall& c, int dtype, bool backward, void* workspace);   // bytes; sets the workspace members
cudaError_t decay_forward(const DecayCall& c, const void* q, const void* k, const void* v, int dtype,
                          const float* state_in, float* state_out, void* out, cudaStream_t s);
cudaError_t decay_backward(const DecayCall& c, const void* q, const void* k, const void* v, const void* dout, int dtype,
                           const float* state_in, const float* dstate_out, void* dq, void* dk, void* dv,
                           float* dstate_in, cudaStream_t s);
cudaError_t decay_step(const void* q, const void* k, const void* v, const float* log_decay, int dtype, int B, int H,
                       int dk, int dv, float scale, const float* state_in, float* state_out, void* out,
                       cudaStream_t s);

// Tensor cores: bf16 of up to 128 channels, a multiple of 8, in arrays that start on 16 bytes, sequences of more than a
// quarter of a chunk on average (decay_tc.cu).
bool decay_tc_fits(const DecayCall& c, int dtype);
cudaError_t decay_tc_states(const DecayCall& c, const DecayStates& p, DecayWhich which, Chain& chain);
cudaError_t decay_tc_pass(const DecayCall& c, const DecayPass& p, Chain& chain);
cudaError_t decay_force_wait_timeout(int enable);   // test hook behind la_test_force_wait_timeout

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------
// decay^n = 2^(n l), l = log2(e) log_decay as two floats: the rounding of n l is carried along, so that a power of
// many steps is as exact as one of few.  log_decay = -inf forgets everything: decay^0 = 1, all else 0.
struct DecayBase {
    float hi, lo;
};
__device__ __forceinline__ DecayBase decay_base(float log_decay) {
    constexpr float kHi = 1.44269502e+00f, kLo = 1.92596303e-08f;   // log2(e)
    const float x = log_decay < -1e30f ? -1e30f : log_decay > 1e30f ? 1e30f : log_decay;
    const float hi = x * kHi;
    return {hi, fmaf(x, kHi, -hi) + x * kLo};
}
__device__ __forceinline__ float decay_power(const DecayBase& b, int n) {
    if (n == 0) return 1.f;
    const float m = (float)n, p = m * b.hi;
    if (p < -200.f) return 0.f;
    if (p > 200.f) return __int_as_float(0x7f800000);
    const float e = fmaf(m, b.hi, -p) + m * b.lo, g = exp2f(p);
    return fmaf(g, e * 0.693147182f, g);
}

// Whether cu_seqlens broke the packing rules: nothing is computed then.  (Another error that a block of this call has
// recorded changes nothing for the others.)
__device__ __forceinline__ bool decay_malformed(const DecayCall& c) {
    return c.cu_seqlens && c.hdr->error == LA_DEVERR_CU_SEQLENS;
}

// The segment of block index i: from the table, or of an equal-length batch.
__device__ __forceinline__ bool decay_segment(const DecayCall& c, int i, DecaySegment& g) {
    if (c.cu_seqlens) {
        if (decay_malformed(c) || i >= c.hdr->n_units) return false;
        g = c.table[i];
        return true;
    }
    const int n = (int)(c.T / c.nseq), m = decay_segments(n, c.L);
    if (m == 0) return false;
    const int s = i / m, k = i - s * m;
    g.seq = s;
    g.start = s * n + k * c.L;
    g.end = (int)min64((int64_t)g.start + c.L, (int64_t)(s + 1) * n);
    g.place = (s * (m - 1) + k) * 4 + (k == 0) + 2 * (k == m - 1);
    return true;
}
// The first (reverse) or last (forward) segment of sequence s; false for an empty one.  *slots: of earlier sequences.
__device__ __forceinline__ bool decay_edge_segment(const DecayCall& c, int s, bool first, DecaySegment& g) {
    int lo, hi, slots;
    if (c.cu_seqlens) {
        lo = c.cu_seqlens[s];
        hi = c.cu_seqlens[s + 1];
        slots = c.slot_first[s];
    } else {
        const int n = (int)(c.T / c.nseq), m = decay_segments(n, c.L);
        lo = s * n;
        hi = lo + n;
        slots = s * (m > 0 ? m - 1 : 0);
    }
    g.seq = s;
    g.start = lo;
    g.end = hi;
    g.place = 0;
    if (hi == lo) return false;
    const int m = decay_segments(hi - lo, c.L), k = first ? 0 : m - 1;
    g.start = lo + k * c.L;
    g.end = (int)min64((int64_t)g.start + c.L, hi);
    g.place = (slots + k) * 4 + (k == 0) + 2 * (k == m - 1);
    return true;
}
// What enters a segment: [dk][dv] of one head, or NULL for nothing.
__device__ __forceinline__ const float* decay_entering(const DecayCall& c, const DecaySegment& g, int h, int reverse,
                                                       const float* edge) {
    const int64_t n = (int64_t)c.dk * c.dv;
    if (reverse ? decay_last(g) : decay_first(g)) return edge ? edge + ((int64_t)g.seq * c.H + h) * n : nullptr;
    return c.states[reverse] + ((int64_t)(decay_slot(g) - (reverse ? 0 : 1)) * c.H + h) * n;
}

}  // namespace la
