// Linear attention with a decay for each head, S_t = g S_(t-1) + k_t v_t^T, out_t = scale q_t^T S_t: the work table,
// the join of segment states, the one-token step, and the products on CUDA cores (any type and size).
//
// A sequence is cut into segments of L tokens that run at once.  State passes sum each segment's own k v^T; the join
// walks the segments of a sequence and leaves what enters each; the product passes walk a segment in chunks with the
// state on chip.  Decays are powers of g between two tokens, at most one, so no product of a large and a small
// factor is formed.  The gradients are the same three products with other operands, two of them from the end.
#include <initializer_list>

#include "ops/decay.h"
#include "ops/vec.cuh"

namespace la {

namespace {

// State passes and product passes of one call that start together.
struct StatesList {
    DecayStates p[2];
    bool ends[2];                // of the join: something leaves the sequences, and was summed with the segments
};
struct PassList {
    DecayPass p[3];
    int first[3];                // of its blocks in z
};

// ---------------------------------------------------------------------------
// Work table of packed sequences
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) decay_plan_kernel(const __grid_constant__ DecayCall c) {
    __shared__ int2 sums[32];
    __shared__ int bad;
    chain_go();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        bad = c.cu_seqlens[0] != 0 || c.cu_seqlens[c.nseq] != c.T;
        c.hdr->range = 0;
    }
    __syncthreads();
    const int per = (c.nseq + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(c.nseq, (int)threadIdx.x * per), s1 = min(c.nseq, s0 + per);
    int2 n = make_int2(0, 0);            // segments and slots of this thread's sequences
    bool wrong = false;
    for (int s = s0; s < s1; ++s) {
        const int lo = c.cu_seqlens[s], hi = c.cu_seqlens[s + 1];
        // (a decrease makes another sequence's sum wrong, so every sequence has to be right)
        if (lo < 0 || hi < lo || hi > c.T) {
            wrong = true;
            continue;
        }
        const int m = decay_segments(hi - lo, c.L);
        n.x += m;
        n.y += m > 0 ? m - 1 : 0;
    }
    if (wrong) bad = 1;
    int2 before = n;
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, before.x, o), y = __shfl_up_sync(0xffffffffu, before.y, o);
        if (lane >= o) {
            before.x += x;
            before.y += y;
        }
    }
    if (lane == 31) sums[warp] = before;
    before.x -= n.x;
    before.y -= n.y;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        before.x += sums[w].x;
        before.y += sums[w].y;
    }
    int total = 0;
    for (int w = 0; w < 32; ++w) total += sums[w].x;
    if (bad) {
        if (threadIdx.x == 0) {
            c.hdr->error = LA_DEVERR_CU_SEQLENS;
            c.hdr->n_units = 0;
        }
        return;
    }
    for (int s = s0; s < s1; ++s) {
        c.segment_first[s] = before.x;
        c.slot_first[s] = before.y;
        const int m = decay_segments(c.cu_seqlens[s + 1] - c.cu_seqlens[s], c.L);
        before.x += m;
        before.y += m > 0 ? m - 1 : 0;
    }
    if (threadIdx.x == 0) {
        c.segment_first[c.nseq] = total;
        c.hdr->error = LA_DEVERR_NONE;
        c.hdr->n_units = total;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += kPlanThreads) {
        // the last sequence that begins at or before segment i: the one that has it (empty ones begin where the next does)
        int lo = 0, hi = c.nseq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (c.segment_first[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int k = i - c.segment_first[lo], end = c.cu_seqlens[lo + 1];
        DecaySegment g;
        g.seq = lo;
        g.start = c.cu_seqlens[lo] + k * c.L;
        g.end = (int)min64((int64_t)g.start + c.L, end);
        g.place = (c.slot_first[lo] + k) * 4 + (k == 0) + 2 * (g.end == end);
        c.table[i] = g;
    }
}

// ---------------------------------------------------------------------------
// Join: what enters each segment, from the segments' own sums
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
// Segments whose loads are on their way together: fewer registers, for more threads at once, are better than more loads of
// each (64 sequences of 8 x 64 x 64 in 95 segments: 13 us; with eight 15, with sixteen 31; 7 of 4 in 135: 22, 19 and 16).
constexpr int kJoinAhead = 4;

template <int N>
__global__ void __launch_bounds__(kJoinThreads) decay_join_kernel(const __grid_constant__ DecayCall c,
                                                                  const __grid_constant__ StatesList list, int blocks) {
    using V = Vec<float, N>;
    chain_wait();
    chain_go();
    if (decay_malformed(c)) return;
    const int s = blockIdx.x, h = blockIdx.y, n = c.dk * c.dv, which = blockIdx.z / blocks;
    const DecayStates& p = list.p[which];
    const bool ends = list.ends[which];
    const int e = ((blockIdx.z - which * blocks) * kJoinThreads + threadIdx.x) * N;
    if (e >= n) return;
    const int64_t edge = ((int64_t)s * c.H + h) * n + e;
    V acc;
#pragma unroll
    for (int k = 0; k < N; ++k) acc.v[k] = 0.f;
    if (p.edge_in) acc = *reinterpret_cast<const V*>(p.edge_in + edge);
    DecaySegment last, first;
    if (!decay_edge_segment(c, s, false, last)) {
        // an empty sequence: what enters it leaves it
        if (ends) *reinterpret_cast<V*>(p.edge_out + edge) = acc;
        return;
    }
    if (decay_first(last) && !ends) return;                                       // no boundary inside
    decay_edge_segment(c, s, true, first);
    const int m = decay_slot(last) - decay_slot(first);                           // boundaries
    const DecayBase base = decay_base(c.log_decay[h]);
    const float whole = decay_power(base, c.L);
    float factor = p.reverse ? decay_power(base, last.end - last.start) : whole;
    const int64_t step = (int64_t)c.H * n;
    float* const own = c.states[p.reverse] + ((int64_t)decay_slot(first) * c.H + h) * n + e;
    for (int i0 = 0; i0 < m; i0 += kJoinAhead) {
        V part[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k)
            if (i0 + k < m) part[k] = *reinterpret_cast<const V*>(own + (p.reverse ? m - 1 - i0 - k : i0 + k) * step);
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            if (i0 + k >= m) break;
#pragma unroll
            for (int j = 0; j < N; ++j) acc.v[j] = fmaf(factor, acc.v[j], part[k].v[j]);
            *reinterpret_cast<V*>(own + (p.reverse ? m - 1 - i0 - k : i0 + k) * step) = acc;
            factor = whole;
        }
    }
    if (!ends) return;
    // the segment at the other end: its own sum, and what enters it where something does
    const DecaySegment& end = p.reverse ? first : last;
    const float keep = decay_power(base, end.end - end.start);
    V own_sum = *reinterpret_cast<const V*>(p.edge_out + edge);
    if (m > 0 || p.edge_in) {
#pragma unroll
        for (int k = 0; k < N; ++k) own_sum.v[k] = fmaf(keep, acc.v[k], own_sum.v[k]);
    }
    *reinterpret_cast<V*>(p.edge_out + edge) = own_sum;
}

// ---------------------------------------------------------------------------
// CUDA-core products: chunks of 32 tokens, 64 columns of z a block
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 256;
constexpr int kRows = 32;          // tokens of a chunk
constexpr int kCols = 64;          // columns of a block

__device__ __forceinline__ void copy4(float* to, const float* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
}

// Eight neighbouring values of a row, nothing from `valid` on; `vec`: the eight start on 16 bytes.
template <typename T>
__device__ __forceinline__ void load8(float (&f)[8], const T* p, int valid, bool vec) {
    if (vec && valid >= 8) {
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int k = 0; k < 8; k += N) {
            float g[N];
            unpack(g, *reinterpret_cast<const Vec<T, N>*>(p + k));
#pragma unroll
            for (int j = 0; j < N; ++j) f[k + j] = g[j];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = k < valid ? (float)p[k] : 0.f;
    }
}
__device__ __forceinline__ void store8(float* to, const float (&f)[8]) {
    reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Sums of one segment (or, final, what leaves each sequence): blocks of 64 x 64 of [dk][dv], 4 x 4 a thread.
template <typename T>
__global__ void __launch_bounds__(kSimtThreads) decay_states_kernel(const __grid_constant__ DecayCall c,
                                                                    const __grid_constant__ StatesList list,
                                                                    DecayWhich of_all, int blocks, bool vec) {
    __shared__ __align__(16) float ys[kRows][kCols], zs[kRows][kCols];
    chain_wait();
    chain_go();
    const int h = blockIdx.y, nb = (c.dv + kCols - 1) / kCols, item = blockIdx.z / blocks, block = blockIdx.z - item * blocks;
    const int a0 = block / nb * kCols, b0 = block % nb * kCols;
    const DecayStates& p = list.p[item];
    const DecayWhich which = of_all == kEnds ? kEnds : list.ends[item] ? kAll : kInner;
    DecaySegment g;
    bool any = true;
    if (decay_malformed(c)) return;
    if (which == kEnds) any = decay_edge_segment(c, blockIdx.x, p.reverse, g);
    else if (!decay_segment(c, blockIdx.x, g)) return;
    const bool end = which == kEnds || (p.reverse ? decay_first(g) : decay_last(g));
    if (end && which == kInner) return;
    const DecayBase base = decay_base(c.log_decay[h]);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, row = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    float fy[8], fz[8];
    auto load = [&](int t0) {
        const int t = t0 + row, out = t < g.end ? 0 : 1 << 20;
        const int64_t r = ((int64_t)(out ? g.start : t) * c.H + h);
        load8(fy, static_cast<const T*>(p.y) + r * c.dk + a0 + col, c.dk - a0 - col - out, vec);
        load8(fz, static_cast<const T*>(p.z) + r * c.dv + b0 + col, c.dv - b0 - col - out, vec);
        if (out) return;
        const float w = p.reverse ? c.scale * decay_power(base, t - g.start + 1) : decay_power(base, g.end - 1 - t);
#pragma unroll
        for (int k = 0; k < 8; ++k) fy[k] *= w;
    };
    if (any) load(g.start);
    for (int t0 = g.start; any && t0 < g.end; t0 += kRows) {
        store8(&ys[row][col], fy);
        store8(&zs[row][col], fz);
        __syncthreads();
        const int n = min(kRows, g.end - t0);
        if (t0 + kRows < g.end) load(t0 + kRows);
        for (int t = 0; t < n; ++t) {
            const float4 y = *reinterpret_cast<const float4*>(&ys[t][ty * 4]);
            const float4 z = *reinterpret_cast<const float4*>(&zs[t][tx * 4]);
            const float yv[4] = {y.x, y.y, y.z, y.w}, zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(yv[i], zv[j], acc[i][j]);
        }
        __syncthreads();
    }
    const int64_t n = (int64_t)c.dk * c.dv;
    const float* enter = nullptr;
    float* to;
    if (which == kEnds) enter = any ? decay_entering(c, g, h, p.reverse, p.edge_in)
                                    : p.edge_in ? p.edge_in + ((int64_t)blockIdx.x * c.H + h) * n : nullptr;
    if (end) to = p.edge_out + ((int64_t)(which == kEnds ? (int)blockIdx.x : g.seq) * c.H + h) * n;
    else to = c.states[p.reverse] + ((int64_t)(decay_slot(g) - (p.reverse ? 1 : 0)) * c.H + h) * n;
    const float keep = any ? decay_power(base, g.end - g.start) : 1.f;
    const bool whole = c.dv % 4 == 0 && reinterpret_cast<uintptr_t>(to) % 16 == 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = a0 + ty * 4 + i, b = b0 + tx * 4;
        if (a >= c.dk || b >= c.dv) continue;
        const int64_t at = (int64_t)a * c.dv + b;
        if (enter) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b + j < c.dv) acc[i][j] = fmaf(keep, enter[at + j], acc[i][j]);
        }
        if (whole) {
            *reinterpret_cast<float4*>(to + at) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b + j < c.dv) to[at + j] = acc[i][j];
        }
    }
}

constexpr int kStateRow = kCols + 4;         // a row of the state: eight rows of a column in as many groups of banks
__host__ __device__ inline int simt_stride(int ds) { return (ds + 31) / 32 * 32 + 4; }   // of rows: no bank twice
__host__ __device__ inline size_t simt_smem(int ds) {
    return sizeof(float) * ((size_t)(ds + 3) / 4 * 4 * kStateRow + 2 * (size_t)kRows * simt_stride(ds) + kRows * kCols +
                            kRows * (kRows + 4) + kRows + 1);
}

// One segment of a product pass.  A thread has two rows, 16 apart, and four columns (of the products with z and the
// state) or two (of the scores).  Passes of one call run in one launch: the gradients of 4099 x 4 x 64 in fp32, three
// passes of 540 blocks, take 58 us (three launches 30 each), of which 33 are instructions at the full rate; the rest are
// shared memory (three wavefronts for four FMA of a thread) and barriers.
template <typename T>
__global__ void __launch_bounds__(kSimtThreads) decay_pass_kernel(const __grid_constant__ DecayCall c,
                                                                  const __grid_constant__ PassList list, bool vec) {
    extern __shared__ __align__(16) float smem[];
    chain_wait();
    chain_go();
    const int item = ((int)blockIdx.z >= list.first[1]) + ((int)blockIdx.z >= list.first[2]);
    const DecayPass& p = list.p[item];
    const int ds = p.ds, ds4 = (ds + 3) / 4 * 4, ld = simt_stride(ds), h = blockIdx.y;
    const int c0 = ((int)blockIdx.z - list.first[item]) * kCols;
    float* S = smem;                          // [ds4][68]
    float* xs = S + ds4 * kStateRow;          // [32][ld]
    float* ys = xs + kRows * ld;              // [32][ld]
    float* zs = ys + kRows * ld;              // [32][64]
    float* P = zs + kRows * kCols;            // [32][36]
    float* pw = P + kRows * (kRows + 4);      // [33]: powers of the decay
    DecaySegment g;
    if (!decay_segment(c, blockIdx.x, g)) return;
    const DecayBase base = decay_base(c.log_decay[h]);
    if (threadIdx.x <= kRows) pw[threadIdx.x] = decay_power(base, threadIdx.x);
    const float* enter = decay_entering(c, g, h, p.reverse, p.edge);
    // The state, on its way while the first scores are made.  A warp of a transposed one has four columns of eight rows:
    // whole sectors of memory, and a bank for each lane.
    for (int i = threadIdx.x; i < (ds4 + 7) / 8 * 8 * kCols; i += kSimtThreads) {
        const int tile = i / 32, lane = i % 32;
        const int a = p.transposed ? tile / 16 * 8 + lane % 8 : i / kCols;
        const int b = p.transposed ? tile % 16 * 4 + lane / 8 : i % kCols;
        if (a >= ds4) continue;
        const bool in = enter && a < ds && c0 + b < p.dz;
        const float* from = p.transposed ? enter + (int64_t)(c0 + b) * ds + a : enter + (int64_t)a * p.dz + c0 + b;
        if (in) copy4(S + a * kStateRow + b, from);
        else S[a * kStateRow + b] = 0.f;
    }
    copies_done();
    const int r0 = threadIdx.x / 16, q0 = threadIdx.x % 16, row = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
    const int chunks = (g.end - g.start + kRows - 1) / kRows;
    for (int k = 0; k < chunks; ++k) {
        const int t0 = g.start + (p.reverse ? chunks - 1 - k : k) * kRows, n = min(kRows, g.end - t0);
        {   // the chunk's rows, nothing behind its end
            const int out = row < n ? 0 : 1 << 20;
            const int64_t r = (int64_t)(out ? t0 : t0 + row) * c.H + h;
            for (int a = col; a < ds4; a += 64) {
                float f[8];
                load8(f, static_cast<const T*>(p.x) + r * ds + a, ds - a - out, vec);
                store8(xs + row * ld + a, f);
                load8(f, static_cast<const T*>(p.y) + r * ds + a, ds - a - out, vec);
                store8(ys + row * ld + a, f);
            }
            float f[8];
            load8(f, static_cast<const T*>(p.z) + r * p.dz + c0 + col, p.dz - c0 - col - out, vec);
            store8(zs + row * kCols + col, f);
        }
        __syncthreads();
        {   // scores, decayed; only those of tokens that a row sees are read below
            float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
            for (int a = 0; a < ds4; a += 4) {
                float4 x[2], y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    x[i] = *reinterpret_cast<const float4*>(xs + (r0 + 16 * i) * ld + a);
                    y[i] = *reinterpret_cast<const float4*>(ys + (q0 + 16 * i) * ld + a);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w,
                                                                                                    acc[i][j]))));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int ri = r0 + 16 * i, rj = q0 + 16 * j, apart = p.reverse ? rj - ri : ri - rj;
                    P[ri * (kRows + 4) + rj] = apart >= 0 ? c.scale * pw[apart] * acc[i][j] : 0.f;
                }
        }
        wait_copies<0>();
        __syncthreads();
        {
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            for (int a = 0; a < ds4; a += 4) {
                float4 x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const float4*>(xs + (r0 + 16 * i) * ld + a);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 s = *reinterpret_cast<const float4*>(S + (a + u) * kStateRow + q0 * 4);
                    const float sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float xv = u == 0 ? x[i].x : u == 1 ? x[i].y : u == 2 ? x[i].z : x[i].w;
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv, sv[j], acc[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ri = r0 + 16 * i;
                const float f = p.reverse ? pw[max(0, n - 1 - ri)] : c.scale * pw[ri + 1];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = enter || k ? f * acc[i][j] : 0.f;
            }
            for (int t = 0; t < n; ++t) {
                const float4 z = *reinterpret_cast<const float4*>(zs + t * kCols + q0 * 4);
                const float zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // a token that the row does not see adds nothing, NaN neither
                    const int ri = r0 + 16 * i;
                    if (p.reverse ? t < ri : t > ri) continue;
                    const float s = P[ri * (kRows + 4) + t];
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s, zv[j], acc[i][j]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ri = r0 + 16 * i;
                if (ri >= n) continue;
                T* out = static_cast<T*>(p.out) + ((int64_t)(t0 + ri) * c.H + h) * p.dz + c0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + q0 * 4 + j < p.dz) store_elem(out, q0 * 4 + j, acc[i][j]);
            }
        }
        __syncthreads();
        if (k + 1 == chunks) break;
        const float keep = pw[n];
        for (int a = r0 * 4; a < ds4; a += 64) {
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 s = *reinterpret_cast<const float4*>(S + (a + i) * kStateRow + q0 * 4);
                acc[i][0] = keep * s.x;
                acc[i][1] = keep * s.y;
                acc[i][2] = keep * s.z;
                acc[i][3] = keep * s.w;
            }
            for (int t = 0; t < n; ++t) {
                const float w = p.reverse ? c.scale * pw[t + 1] : pw[n - 1 - t];
                const float4 y = *reinterpret_cast<const float4*>(ys + t * ld + a);
                const float4 z = *reinterpret_cast<const float4*>(zs + t * kCols + q0 * 4);
                const float yv[4] = {w * y.x, w * y.y, w * y.z, w * y.w}, zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(yv[i], zv[j], acc[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(S + (a + i) * kStateRow + q0 * 4) =
                    make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// One token for each of B sequences
// ---------------------------------------------------------------------------
// Threads of a block, and rows of the state that a thread has on their way together (a vector's lanes are LA_MAX_DV / N
// at most, so that a block always has a whole group of them).
template <int N>
constexpr int kStepThreads = N == 4 ? 128 : 256;
template <int N>
constexpr int kStepRows = N == 4 ? 8 : 4;

// A block has one (sequence, head); lanes along dv in vectors of N, thread groups along dk.  Bound by memory, each state
// read and written once: 256 x 16 x 64 x 64 in 25 us, 20 at the copy rate; 27 from cold caches, where 256 threads with four
// rows each took 31, 64 with sixteen 29, and streaming loads and stores nothing more or less.
template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads<N>) decay_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                                  const T* __restrict__ v,
                                                                  const float* __restrict__ log_decay, int H, int dk,
                                                                  int dv, int lanes, float scale, const float* state_in,
                                                                  float* state_out, T* __restrict__ out) {
    using V = Vec<float, N>;
    static_assert(LA_MAX_DV / N <= kStepThreads<N>, "a group of lanes for a row of the state");
    __shared__ float qs[LA_MAX_DK], ks[LA_MAX_DK];
    __shared__ float part[kStepThreads<N> * N];
    const int64_t pair = blockIdx.x;
    const int h = (int)(pair % H), cols = dv / N, groups = kStepThreads<N> / lanes;
    const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const bool on = lane < cols;
    const int64_t at = pair * dk * dv + lane * N, step = (int64_t)groups * dv;
    V held[kStepRows<N>];
#pragma unroll
    for (int r = 0; r < kStepRows<N>; ++r)
        if (on && group + r * groups < dk) held[r] = *reinterpret_cast<const V*>(state_in + at + group * dv + r * step);
    const float g = decay_power(decay_base(log_decay[h]), 1);
    for (int a = threadIdx.x; a < dk; a += kStepThreads<N>) {
        qs[a] = (float)q[pair * dk + a];
        ks[a] = (float)k[pair * dk + a];
    }
    float fv[N], sum[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        fv[j] = on ? (float)v[pair * dv + lane * N + j] : 0.f;
        sum[j] = 0.f;
    }
    __syncthreads();
    for (int a0 = group; a0 < dk; a0 += kStepRows<N> * groups) {
        if (a0 != group) {
#pragma unroll
            for (int r = 0; r < kStepRows<N>; ++r)
                if (on && a0 + r * groups < dk) held[r] = *reinterpret_cast<const V*>(state_in + at + (int64_t)a0 * dv + r * step);
        }
#pragma unroll
        for (int r = 0; r < kStepRows<N>; ++r) {
            const int a = a0 + r * groups;
            if (!on || a >= dk) continue;
            const float kv = ks[a], qv = qs[a];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float s = fmaf(g, held[r].v[j], __fmul_rn(kv, fv[j]));
                held[r].v[j] = s;
                sum[j] = fmaf(qv, s, sum[j]);
            }
            *reinterpret_cast<V*>(state_out + at + (int64_t)a0 * dv + r * step) = held[r];
        }
    }
    if (on) {
#pragma unroll
        for (int j = 0; j < N; ++j) part[(group * cols + lane) * N + j] = sum[j];
    }
    __syncthreads();
    for (int b = threadIdx.x; b < dv; b += kStepThreads<N>) {
        float o = 0.f;
        for (int i = 0; i < groups; ++i) o += part[i * dv + b];
        store_elem(out, pair * dv + b, scale * o);
    }
}

template <typename T>
cudaError_t step(const void* q, const void* k, const void* v, const float* log_decay, int B, int H, int dk, int dv,
                 float scale, const float* state_in, float* state_out, void* out, cudaStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(state_in) | reinterpret_cast<uintptr_t>(state_out);
    const bool vec = dv % 4 == 0 && at % 16 == 0;
    const int cols = vec ? dv / 4 : dv;
    int lanes = 1;
    while (lanes < cols) lanes *= 2;
    const unsigned grid = (unsigned)B * H;
    if (vec)
        decay_step_kernel<T, 4><<<grid, kStepThreads<4>, 0, s>>>(
            static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), log_decay, H, dk, dv, lanes,
            scale, state_in, state_out, static_cast<T*>(out));
    else
        decay_step_kernel<T, 1><<<grid, kStepThreads<1>, 0, s>>>(
            static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), log_decay, H, dk, dv, lanes,
            scale, state_in, state_out, static_cast<T*>(out));
    return cudaGetLastError();
}

bool on_16_bytes(std::initializer_list<const void*> arrays) {
    uintptr_t at = 0;
    for (const void* a : arrays) at |= reinterpret_cast<uintptr_t>(a);
    return at % 16 == 0;
}
bool vector_rows(const DecayCall& c, int dtype, std::initializer_list<const void*> arrays) {
    const int n = dtype == LA_F32 ? 4 : 8;
    return on_16_bytes(arrays) && c.dk % n == 0 && c.dv % n == 0;
}

// Tokens of a segment: exact in fp32.  The tensor cores cut off what they add to the state that the products keep: of 16
// tokens' terms all below 2^-25, of their sum with the state all below 2^-23 of the largest one's power of two (seen with
// terms of one bit each).  That is 5 2^-23 of the state at most, eight times a chunk: 2^-11 of it after 64 chunks, mostly
// toward zero, and half as much where terms are spread evenly, beside outputs rounded by 2^-8.  (256 chunks lose four times
// that; 65536 x 152 x 64 take 1180 us so and 1418 with 64, which sum seven eighths of the tokens a second time instead of
// half, 262144 x 16 x 64 635 and 668, 65536 x 40 x 128 960 both.)
constexpr int64_t kLongest = 1 << 20, kMostChunks = 64;

// Tokens of a segment.  Tensor cores: whole chunks of 128, one block per SM.  Equal sequences are cut so that the waves
// of blocks times a segment's chunks, and two for a block's beginning and end, are fewest.  Packed ones, whose lengths
// are not known here, are cut into one and a half blocks' worth per SM (40009 x 8 x 64 of 64 sequences 129 us, of one 96,
// 120000 of 64 245; three blocks' worth 135, 120 and 235; one 139, 102 and 247).  CUDA cores:
// four blocks per SM, of chunks of 32, so that what is short has one chunk to a block and nothing waits for a chunk ahead.
int64_t segment_length(const DecayCall& c, bool tensor, int sms) {
    // (packed: longer than T where one segment would do, so that no boundary inside a sequence has to be reckoned with)
    const int64_t n = c.cu_seqlens ? c.T + 1 : c.T / c.nseq;
    if (c.T < 1) return 128;
    if (!tensor) {
        const int64_t L = ceil_div(ceil_div(c.T * c.H * ceil_div(c.dv, kCols), 4 * sms), kRows) * kRows;
        return min64(min64(L, ceil_div(n, kRows) * kRows), kLongest);
    }
    const int64_t chunks = ceil_div(n, 128);
    int64_t best = 1, least = INT64_MAX;
    if (c.cu_seqlens) {
        best = ceil_div(c.T, 128) * c.H * 2 / (3 * sms);
        best = min64(min64(best < 1 ? 1 : best, chunks), kMostChunks);
    } else {
        // (more segments than a few per SM, or than chunks, never pay)
        const int64_t pairs = (int64_t)c.nseq * c.H, fewest = ceil_div(chunks, kMostChunks);
        const int64_t most = min64(chunks, ceil_div(8 * sms, pairs));
        for (int64_t per = fewest; per == fewest || per <= most; ++per) {
            const int64_t k = ceil_div(chunks, per);
            const int64_t cost = ceil_div(ceil_div(chunks, k) * pairs, sms) * (k + 2);
            if (cost < least) {
                least = cost;
                best = k;
            }
        }
    }
    return best * 128;
}

cudaError_t plan(const DecayCall& c, Chain& chain) {
    if (!c.cu_seqlens) return cudaMemsetAsync(c.hdr, 0, sizeof(WsHeader), chain.stream);
    return launch_in(chain, decay_plan_kernel, 1, kPlanThreads, 0, c);
}

// Whether what leaves the sequences is summed with the segments: unless it takes the place of what enters them.
bool with_segments(const DecayStates& p) { return p.edge_out && p.edge_out != p.edge_in; }

// States of sequences of up to 64 tokens on average are summed on CUDA cores, whose many small blocks begin and end beside
// one another: 256 of 64 x 8 x 64, carried, take 185 us and 240 with the sums on the tensor cores; 256 of 256 tokens 307
// and 283; 8 of 128 tokens 30 and 25.
constexpr int64_t kShortSums = 64;

cudaError_t states(const DecayCall& c, std::initializer_list<DecayStates> passes, int dtype, bool ends_alone,
                   Chain& chain) {
    StatesList simt{};
    int n = 0;
    bool vec = true;
    for (const DecayStates& p : passes) {
        if (!ends_alone && c.slots == 0 && !with_segments(p)) continue;
        if (decay_tc_fits(c, dtype) && on_16_bytes({p.y, p.z}) && c.T > kShortSums * c.nseq) {
            const cudaError_t e = decay_tc_states(c, p, ends_alone ? kEnds : with_segments(p) ? kAll : kInner, chain);
            if (e != cudaSuccess) return e;
            continue;
        }
        vec = vec && vector_rows(c, dtype, {p.y, p.z});
        simt.p[n] = p;
        simt.ends[n++] = with_segments(p);
    }
    if (n == 0) return cudaSuccess;
    const int blocks = (int)(ceil_div(c.dk, kCols) * ceil_div(c.dv, kCols));
    const dim3 grid(ends_alone ? c.nseq : c.segments, c.H, (unsigned)(n * blocks));
    const DecayWhich which = ends_alone ? kEnds : kAll;
    return launch_in(chain, dtype == LA_F32 ? decay_states_kernel<float> : decay_states_kernel<__nv_bfloat16>, grid,
                     kSimtThreads, 0, c, simt, which, blocks, vec);
}

cudaError_t join(const DecayCall& c, std::initializer_list<DecayStates> passes, Chain& chain) {
    const int n = c.dk * c.dv;
    StatesList list{};
    int items = 0;
    bool vec = n % 4 == 0;
    for (const DecayStates& p : passes) {
        list.p[items] = p;
        list.ends[items++] = with_segments(p);
        vec = vec && on_16_bytes({p.edge_in, with_segments(p) ? p.edge_out : nullptr});
    }
    const int blocks = (int)ceil_div(n, kJoinThreads * (vec ? 4 : 1));
    const dim3 grid(c.nseq, c.H, (unsigned)(items * blocks));
    return launch_in(chain, vec ? decay_join_kernel<4> : decay_join_kernel<1>, grid, kJoinThreads, 0, c, list, blocks);
}

// What enters every segment, and what leaves every sequence unless that overwrites what enters it (nothing to do where
// every sequence is one segment and nothing is to leave).
cudaError_t enter(const DecayCall& c, std::initializer_list<DecayStates> passes, int dtype, Chain& chain) {
    bool ends = false;
    for (const DecayStates& p : passes) ends = ends || with_segments(p);
    if (c.slots == 0 && !ends) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    if (c.T > 0) e = states(c, passes, dtype, false, chain);
    return e != cudaSuccess ? e : join(c, passes, chain);
}
// What leaves every sequence, where that takes the place of what enters it: once nothing reads it any more.
cudaError_t leave(const DecayCall& c, const DecayStates& p, int dtype, Chain& chain) {
    return p.edge_out && p.edge_out == p.edge_in ? states(c, {p}, dtype, true, chain) : cudaSuccess;
}

cudaError_t products(const DecayCall& c, std::initializer_list<DecayPass> passes, int dtype, Chain& chain) {
    if (c.T == 0) return cudaSuccess;
    PassList simt{};
    int n = 0, blocks = 0, widest = 0;
    bool vec = true;
    for (const DecayPass& p : passes) {
        if (decay_tc_fits(c, dtype) && on_16_bytes({p.x, p.y, p.z, p.out})) {
            const cudaError_t e = decay_tc_pass(c, p, chain);
            if (e != cudaSuccess) return e;
            continue;
        }
        vec = vec && vector_rows(c, dtype, {p.x, p.y, p.z});
        simt.p[n] = p;
        simt.first[n++] = blocks;
        blocks += (int)ceil_div(p.dz, kCols);
        widest = p.ds > widest ? p.ds : widest;
    }
    if (n == 0) return cudaSuccess;
    for (; n < 3; ++n) simt.first[n] = blocks;
    const dim3 grid(c.segments, c.H, (unsigned)blocks);
    const size_t smem = simt_smem(widest);
    auto kernel = dtype == LA_F32 ? decay_pass_kernel<float> : decay_pass_kernel<__nv_bfloat16>;
    const cudaError_t e = allow_all_shared(kernel);
    if (e != cudaSuccess) return e;
    return launch_in(chain, kernel, grid, kSimtThreads, smem, c, simt, vec);
}

}  // namespace

size_t decay_layout(DecayCall& c, int dtype, bool backward, void* workspace) {
    int sms = sm_count();
    if (sms <= 0) sms = 152;
    c.L = (int)segment_length(c, decay_tc_fits(c, dtype), sms);
    const int64_t n = c.cu_seqlens ? c.T : c.T / c.nseq, L = c.L;
    const int64_t per = n > 0 ? ceil_div(n, L) : 0;
    const int64_t segments = c.cu_seqlens ? c.T / L + c.nseq : per * c.nseq;
    c.segments = (int)segments;
    c.slots = c.cu_seqlens ? c.T / L : (per > 0 ? per - 1 : 0) * c.nseq;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        unsigned char* at = w ? w + o : nullptr;
        o = align_up(o + bytes, kAlign);
        return at;
    };
    c.hdr = reinterpret_cast<WsHeader*>(take(sizeof(WsHeader)));
    if (c.cu_seqlens) {
        c.slot_first = reinterpret_cast<int*>(take(sizeof(int) * ((size_t)c.nseq + 1)));
        c.segment_first = reinterpret_cast<int*>(take(sizeof(int) * ((size_t)c.nseq + 1)));
        c.table = reinterpret_cast<DecaySegment*>(take(sizeof(DecaySegment) * (size_t)segments));
    }
    for (int i = 0; i < (backward ? 2 : 1); ++i)
        c.states[i] = reinterpret_cast<float*>(take(sizeof(float) * (size_t)c.slots * c.H * c.dk * c.dv));
    return o;
}

cudaError_t decay_forward(const DecayCall& c, const void* q, const void* k, const void* v, int dtype,
                          const float* state_in, float* state_out, void* out, cudaStream_t s) {
    const DecayStates sums{k, v, 0, state_in, state_out};
    const DecayPass p{q, k, v, out, c.dk, c.dv, 0, 0, state_in};
    Chain chain{s};
    cudaError_t e = plan(c, chain);
    if (e == cudaSuccess) e = enter(c, {sums}, dtype, chain);
    if (e == cudaSuccess) e = products(c, {p}, dtype, chain);
    if (e == cudaSuccess) e = leave(c, sums, dtype, chain);
    return e;
}

cudaError_t decay_backward(const DecayCall& c, const void* q, const void* k, const void* v, const void* dout, int dtype,
                           const float* state_in, const float* dstate_out, void* dq, void* dk, void* dv,
                           float* dstate_in, cudaStream_t s) {
    const DecayStates sums{k, v, 0, state_in, nullptr}, back{q, dout, 1, dstate_out, dstate_in};
    const DecayPass pq{dout, v, k, dq, c.dv, c.dk, 0, 1, state_in}, pk{v, dout, q, dk, c.dv, c.dk, 1, 1, dstate_out},
        pv{k, q, dout, dv, c.dk, c.dv, 1, 0, dstate_out};
    Chain chain{s};
    cudaError_t e = plan(c, chain);
    if (e == cudaSuccess) e = enter(c, {sums, back}, dtype, chain);
    if (e == cudaSuccess) e = products(c, {pq, pk, pv}, dtype, chain);
    if (e == cudaSuccess) e = leave(c, back, dtype, chain);
    return e;
}

cudaError_t decay_step(const void* q, const void* k, const void* v, const float* log_decay, int dtype, int B, int H,
                       int dk, int dv, float scale, const float* state_in, float* state_out, void* out,
                       cudaStream_t s) {
    return dtype == LA_F32 ? step<float>(q, k, v, log_decay, B, H, dk, dv, scale, state_in, state_out, out, s)
                           : step<__nv_bfloat16>(q, k, v, log_decay, B, H, dk, dv, scale, state_in, state_out, out, s);
}

}  // namespace la
