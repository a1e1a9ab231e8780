// Layer norm over rows of d values and its gradients.
//
// Bound by memory: the forward reads x and writes y once, the backward reads x
// and dy and writes dx once.  A row stays in the registers of the L lanes that
// share it (E vectors of N values each) between the sums over it and its
// output; the variance comes from the deviations in registers, not from sums of
// squares (and a row whose mean is large against them is done once more, with a
// corrected mean).  Rows of up to 64 vectors share a warp, longer ones take a block.
// A group works on U rows at once so that their sums overlap, and each lane copies
// its vectors of the next turns to shared memory ahead (asynchronous copies that
// it alone waits for): what is in flight does not cost registers.  Where a row
// takes a block, its warps meet at one barrier a turn: in the forward they
// exchange their own sums and squared deviations from their own means, which
// join exactly, in the backward their two sums.
//
// A group of lanes keeps one weight row: it walks over rows a multiple of
// `groups` apart.  Its weights are read once, and in the backward its columns'
// weight gradients add up in registers over all its rows.  Blocks leave their
// sums in the workspace as rows of a [M][groups * d] matrix that a second
// kernel adds up by column with compensated sums, in a fixed order.
//
// Measured (GB300, 6.76 TB/s copies): bf16 rows with their statistics, 1048576 x 64 with weights per head 46 us,
// 6.0 TB/s; 8192 x 4096 28 us, 4.8 TB/s; 16384 x 1001 25 us, 2.7 TB/s; fp32 16384 x 768 23 us, 4.4 TB/s.  Gradients
// in bf16: 262144 x 64 per head 31 us, 3.3 TB/s; 8192 x 4096 46 us, 4.4 TB/s; 32768 x 1024 48 us, 4.2 TB/s;
// 229376 x 128 with 7 heads 43 us, 4.1 TB/s.  What bounds the backward is latency: for 8192 x 4096 it takes half of
// the issue slots (22 M instructions, 18 us of them) and 56 percent of DRAM with a quarter of the warps, one block of
// 512 threads per SM that meets at a barrier every turn, with one turn of rows on their way; the second kernel's
// launch and its read of the blocks' sums come on top.  More warps with fewer registers are slower (two blocks of 64
// registers a thread for 8192 x 4096: 62 us).
#include <float.h>

#include "ops/ops.h"
#include "ops/vec.cuh"

namespace la {

namespace {

constexpr int kHeldValues = 16;         // forward: weights and biases of so many columns a lane stay in registers
constexpr int kCopyBytes = 64 * 1024;   // of rows copied ahead, per SM
constexpr int kShiftRegisters = 16;      // for where in its vectors a row starts and ends
constexpr int kJoinCols = 8, kJoinRows = 32;

// Shift: rows that do not start on 16 bytes (in arrays that do) are taken as the vectors that hold them.  A row
// group's rows are a whole number of vectors apart, so its offset in the first vector, and with it the columns of
// each lane, stay the same on every turn.
template <int L_, int E_, int N_, bool Shift_ = false>
struct Shape {
    static constexpr int L = L_, E = E_, N = N_;
    static constexpr bool kShift = Shift_;
    static constexpr int kThreads = L > 32 ? L : 256;
    static constexpr int kRows = kThreads / L;              // row groups of a block
    static constexpr int kValues = E * N;                   // values a lane holds of a row
    using P = typename Pairs<N>::P;                         // in pairs, n of them to a vector
    static constexpr int n = Pairs<N>::n, kPairs = E * n;
};

constexpr int blocks_per_sm(int threads, int registers) {
    const int n = 65536 / (threads * registers);
    return n < 1 ? 1 : n * threads > 2048 ? 2048 / threads : n;
}
template <typename T, typename S>
constexpr int row_registers() { return S::kValues * (int)sizeof(T) / 4 > 0 ? S::kValues * (int)sizeof(T) / 4 : 1; }

// How far ahead rows are copied: `depth` turns of U rows (of x, or of x and dy) in a block's share of
// kCopyBytes, two turns where they are longer, one where two do not fit.  (96 KB per SM and more are no faster in the
// forward: 51 us instead of 48 for 1048576 rows of 64; the backward was not measured with more.)  Rows of single elements are loaded when they are needed
// (a copy has at least four bytes).
template <typename T, typename S, int U, int Arrays, int Blocks>
struct Ahead {
    static constexpr bool on = S::N > 1;
    static constexpr int turn_bytes = U * Arrays * S::E * S::kThreads * 16;
    static constexpr int most = kCopyBytes / Blocks / turn_bytes;
    static constexpr int depth = most > 8 ? 8 : most >= 2 ? most : 2 * turn_bytes <= 200 * 1024 ? 2 : 1;
    static constexpr size_t bytes = on ? (size_t)depth * turn_bytes : 0;   // a multiple of 16
};
// The registers to compile for, and the blocks of an SM that this and the copies' memory allow.  Some kernels want a few
// more and spill them: fp32 gradients of up to 256 columns 4 to 96 bytes a thread, those of rows beyond 8192 columns
// (beyond 4096 in arrays off 16 bytes) 470 to 800, a few forward ones 4 to 40.
template <typename T, typename S>
struct ForwardPlan {
    static constexpr int U = S::E == 1 ? 2 : 1;
    // (two vectors of bf16: with 16 registers for the shift as elsewhere 32768 x 1001 take 46 us instead of 41)
    static constexpr int registers = U * row_registers<T, S>() +
                                     (S::kShift ? (S::N == 8 ? 2 : 1) * kShiftRegisters : 0) +
                                     (S::kValues <= kHeldValues ? 2 * S::kValues + 38 : 52);
    static constexpr int by_registers = blocks_per_sm(S::kThreads, registers);
    using A = Ahead<T, S, U, 1, by_registers>;
    static constexpr size_t parameters = 2 * sizeof(float) * S::kValues * S::kThreads;
    static constexpr bool staged = S::kShift && S::kValues > kHeldValues && A::bytes + parameters <= 200 * 1024;
    static constexpr size_t bytes = A::bytes + (staged ? parameters : 0);
    static constexpr int by_memory = 227 * 1024 / ((int)bytes + 2048);
    static constexpr int per_sm = by_registers < by_memory ? by_registers : by_memory;
    static_assert(per_sm >= 1, "a block's shared memory");
};
template <typename T, typename S>
struct BackwardPlan {
    static constexpr bool held = S::kValues <= 8;           // xh and w dy of U rows stay in registers
    static constexpr int U = held ? 2 : 1, kForShift = S::kShift ? kShiftRegisters : 0;
    // (bf16: unpacked values want another 30; with 96 registers and five blocks instead of four 32768 x 1024
    // take 62 us instead of 48)
    static constexpr int registers = held ? (2 * U + 3) * S::kValues + (S::N == 8 ? 70 : 40 + kForShift)
                                          : 2 * row_registers<T, S>() + 3 * S::kValues + 44 + kForShift;
    static constexpr int by_registers = blocks_per_sm(S::kThreads, registers);
    using A = Ahead<T, S, U, 2, by_registers>;
    static constexpr bool staged = S::kShift && !held;
    static constexpr size_t bytes = A::bytes + (staged ? sizeof(float) * S::kValues * S::kThreads : 0);
    static constexpr int by_memory = 227 * 1024 / ((int)bytes + 2048);
    static constexpr int per_sm = by_registers < by_memory ? by_registers : by_memory;
    static_assert(per_sm >= 1, "a block's shared memory");
};

template <int Width>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
    for (int o = Width / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
constexpr int power_of_two(int n) { return n <= 1 ? 1 : 2 * power_of_two((n + 1) / 2); }
// The sums over a row group's L lanes of M values (two or four); every lane gets them.  Where a group is a block, a
// step across lanes halves what each lane still sums as long as there are several values (M = 4: six exchanges
// instead of 20), and the warps' sums are taken up the same way.  `scratch` holds two turns and `turn` chooses: one
// barrier keeps a turn's writers off the readers of the turn before last.
template <typename S, int M>
__device__ __forceinline__ void row_sums(float (&x)[M], float* scratch, int turn) {
    static_assert(M == 2 || M == 4, "halved once or twice");
    if constexpr (S::L <= 32) {
#pragma unroll
        for (int i = 0; i < M; ++i) x[i] = lane_sum<S::L>(x[i]);
    } else {
        constexpr int kWarps = S::L / 32, kLanes = 32 / M;         // lanes that end up with the same value
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = lane % kLanes, value = lane / kLanes;
        float* half = scratch + (turn & 1) * M * kWarps;
        const bool upper = lane & 16;
        float part[M / 2];
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
            const float keep = upper ? x[i + M / 2] : x[i], send = upper ? x[i] : x[i + M / 2];
            part[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
        }
        float t = part[0];
        if constexpr (M == 4) {
            const float send = lane & 8 ? part[0] : part[1];
            t = (lane & 8 ? part[1] : part[0]) + __shfl_xor_sync(0xffffffffu, send, 8);
        }
        t = lane_sum<kLanes>(t);
        if (mine == 0) half[value * kWarps + warp] = t;
        __syncthreads();
        t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; w += kLanes)
            if (w + mine < kWarps) t += half[value * kWarps + w + mine];
        t = lane_sum<kLanes>(t);
#pragma unroll
        for (int i = 0; i < M; ++i) x[i] = __shfl_sync(0xffffffffu, t, i * kLanes);
    }
}
// Of the d columns of a row, those that warp w of a block holds; the row starts at element `shift` of its
// first vector.
template <typename S>
__device__ __forceinline__ int warp_columns(int w, int d, int shift) {
    int n = 0;
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        const int start = (e * S::L + w * 32) * S::N - shift, end = start + 32 * S::N;
        const int a = S::kShift && start < 0 ? 0 : start, b = end < d ? end : d;
        n += b > a ? b - a : 0;
    }
    return n;
}

// What of a lane's vectors lies in its rows: column `col` of a row is the lane's first (below zero where the
// vector starts before the row), `left` columns of the row are there from it on.  Masks of the vectors' words (of an
// fp32, or of two bf16) stay in registers where they are few.
template <typename S, typename T>
struct Edges {
    static constexpr int kWords = S::N * (int)sizeof(T) >= 4 ? S::N * (int)sizeof(T) / 4 : 1, kEach = S::N / kWords;
    static constexpr bool kKept = S::kShift && S::E <= 2;
    int left, before;
    uint32_t masks[kKept ? S::E : 1][kWords];

    __device__ __forceinline__ Edges(int col, int d) : left(d - col), before(-col) {
        if (kKept)
#pragma unroll
            for (int e = 0; e < S::E; ++e)
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    masks[e][i] = made(e, i);
                    asm volatile("" : "+r"(masks[e][i]));      // made once
                }
    }
    __device__ __forceinline__ bool in(int e, int k) const {
        return k >= (e == 0 ? before : 0) && k < left - e * S::L * S::N;
    }
    __device__ __forceinline__ bool partial(int e) const {
        return S::kShift && ((e == 0 && before > 0) || left - e * S::L * S::N < S::N);
    }
    __device__ __forceinline__ uint32_t made(int e, int i) const {
        if (kEach == 1) return in(e, i) ? 0xffffffffu : 0u;
        return (in(e, 2 * i) ? 0xffffu : 0u) | (in(e, 2 * i + 1) ? 0xffff0000u : 0u);
    }
    __device__ __forceinline__ uint32_t mask(int e, int i) const { return kKept ? masks[e][i] : made(e, i); }
    // all ones or zero, for element k
    __device__ __forceinline__ uint32_t whole(int e, int k) const {
        if (kEach == 1) return mask(e, k);
        return __byte_perm(mask(e, k / 2), 0, k % 2 ? 0x3232 : 0x1010);
    }
};

// The lane's E vectors of a row, which `row` points into at the lane's first column; vector e lies e L N
// columns on and is there when that is below `left`, the columns from the lane's first on.  In shared
// memory vector e of a row has the place of this thread in a run of kThreads.
// `end`: of the array; its last vector may be there in part.
template <typename S, typename T>
__device__ __forceinline__ void copy_row(uint4* place, const T* row, int left, const T* end) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        constexpr int kStep = S::L * S::N;
        if (e * kStep >= left) continue;
        if (!S::kShift || row + e * kStep + S::N <= end) {
            copy_16(place + e * S::kThreads, row + e * kStep);
        } else {
#pragma unroll 1
            for (int k = 0; k < S::N; ++k)
                reinterpret_cast<T*>(place + e * S::kThreads)[k] =
                    row + e * kStep + k < end ? row[e * kStep + k] : T(0.f);
        }
    }
}
// Elements of a vector outside the row count as zeros.
template <typename S, typename T>
__device__ __forceinline__ void load_row(Vec<T, S::N> (&x)[S::E], const uint4* place, const T* row, int left,
                                         const Edges<S, T>& edges) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        constexpr int kStep = S::L * S::N;
        if (e * kStep < left) {
            x[e] = place ? *reinterpret_cast<const Vec<T, S::N>*>(place + e * S::kThreads)
                         : *reinterpret_cast<const Vec<T, S::N>*>(row + e * kStep);
        } else {
            const float zero[S::N] = {};
            pack(x[e], zero);
        }
    }
    if constexpr (S::kShift) {
#pragma unroll
        for (int e = 0; e < S::E; ++e)
            if (Edges<S, T>::kKept || edges.partial(e)) {
#pragma unroll
                for (int i = 0; i < Edges<S, T>::kWords; ++i) {
                    uint32_t* word = reinterpret_cast<uint32_t*>(&x[e].v[i]);
                    *word &= edges.mask(e, i);
                }
            }
    }
}

// A vector of weights or biases; `missing` where there are none.  Vectors of columns come with 16-byte
// aligned parameters.
template <typename S>
__device__ __forceinline__ void load_params(typename S::P* w, const float* p, float missing) {
    Vec<float, S::N> v;
    if (p) {
        if constexpr (S::N >= 4) {
#pragma unroll
            for (int k = 0; k < S::N; k += 4) {
                const float4 q = *reinterpret_cast<const float4*>(p + k);
                v.v[k] = q.x; v.v[k + 1] = q.y; v.v[k + 2] = q.z; v.v[k + 3] = q.w;
            }
        } else {
            v.v[0] = p[0];
        }
    } else {
#pragma unroll
        for (int k = 0; k < S::N; ++k) v.v[k] = missing;
    }
    typename S::P f[S::n];
    unpack_pairs<S::N>(f, v);
#pragma unroll
    for (int k = 0; k < S::n; ++k) w[k] = f[k];
}
// The same one by one, of columns in [before, left) of the vector; zero in the others.
template <typename S>
__device__ __forceinline__ void load_params_within(typename S::P* w, const float* p, float missing, int before,
                                                   int left) {
    Vec<float, S::N> v;
#pragma unroll
    for (int k = 0; k < S::N; ++k) v.v[k] = k >= before && k < left ? (p ? p[k] : missing) : 0.f;
    typename S::P f[S::n];
    unpack_pairs<S::N>(f, v);
#pragma unroll
    for (int k = 0; k < S::n; ++k) w[k] = f[k];
}
// Vector e of the lane's parameters, `p` at the lane's first column of the row.
template <typename S>
__device__ __forceinline__ void load_vector_params(typename S::P* w, const float* p, int e, int left, int before,
                                                   float missing) {
    const int at = e * S::L * S::N;
    if constexpr (S::kShift) load_params_within<S>(w, p ? p + at : nullptr, missing, e == 0 ? before : 0, left - at);
    else load_params<S>(w, p && at < left ? p + at : nullptr, missing);
}
// The lane's parameters of a whole row.
template <typename S>
__device__ __forceinline__ void load_row_params(typename S::P (&w)[S::kPairs], const float* p, int left, int before,
                                                float missing) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) load_vector_params<S>(w + e * S::n, p, e, left, before, missing);
}
// f + minus for vector e of a row; outside the row zeros stay zeros.
template <typename S, typename T>
__device__ __forceinline__ void deviations(typename S::P (&f)[S::n], typename S::P minus, int e,
                                           const Edges<S, T>& edges) {
#pragma unroll
    for (int k = 0; k < S::n; ++k) f[k] = padd(f[k], minus);
    if constexpr (S::kShift) {
        if (edges.partial(e))
#pragma unroll
            for (int k = 0; k < S::n; ++k)
                f[k] = tc::f32x2_of(__float_as_uint(tc::f32x2_lo(f[k])) & edges.whole(e, 2 * k),
                                    __float_as_uint(tc::f32x2_hi(f[k])) & edges.whole(e, 2 * k + 1));
    }
}
// Stores vector e of a row at `to`; of one that lies in the row in part, the elements that do.
template <typename S, typename T>
__device__ __forceinline__ void store_vector(T* to, const Vec<T, S::N>& v, int e, const Edges<S, T>& edges) {
    if (!edges.partial(e)) {
        *reinterpret_cast<Vec<T, S::N>*>(to) = v;
    } else {
#pragma unroll
        for (int k = 0; k < S::N; ++k)
            if (edges.whole(e, k)) to[k] = element(v, k);
    }
}
// A lane's parameters in shared memory, for rows whose columns its registers cannot hold and whose vectors are
// not the parameters': [kPairs][kThreads], each read by the thread that wrote it.
template <typename S>
__device__ __forceinline__ void staged_params(typename S::P* w, const typename S::P* place, int e) {
#pragma unroll
    for (int k = 0; k < S::n; ++k) w[k] = place[(e * S::n + k) * S::kThreads];
}
template <typename F>
__device__ __forceinline__ F* row_of(F* p, int64_t at) { return p ? p + at : nullptr; }
// The first element of row `row` within its 16 bytes.
template <typename S>
__device__ __forceinline__ int shift_of(int64_t row, int d) {
    return S::kShift ? (int)((uint64_t)row * (uint64_t)d % S::N) : 0;
}

// 1 / sqrt(v), within one step: the approximate root and one step of Newton's method (0 and infinity
// keep the root's answer).
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    return v > 0.f && v < INFINITY ? fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r) : r;
}
// A mean more than 16 times as large as the spread (or a variance that is not finite): the rounding of the row's sum,
// which is relative to the mean, shows in what is taken about it.
__device__ __forceinline__ bool far_mean(float mean, float var) {
    const float part = mean * 0.0625f, rest = fmaf(-part, part, var);
    return !(rest >= 0.f && rest <= FLT_MAX);
}
// The sums over a row group's L lanes of two values; every lane gets them.  Its barriers keep what other lanes wrote
// before and after apart.
template <int L>
__device__ __forceinline__ float2 group_sums(float a, float b, float2* scratch) {
    a = lane_sum<(L < 32 ? L : 32)>(a);
    b = lane_sum<(L < 32 ? L : 32)>(b);
    if constexpr (L > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
        for (int w = 0; w < L / 32; ++w) {
            a += scratch[w].x;
            b += scratch[w].y;
        }
    } else {
        __syncwarp();
    }
    return make_float2(a, b);
}
// Such a row once more (not `mine`: of another row group), its y, mean and rstd written anew: the first mean corrected
// by that of the deviations from it (its error is then its own rounding, and equal values have their value as mean), and
// the squares of the deviations from that.  A row without a finite mean keeps the first.  The lane's vectors come from
// where load_row found them; loops that are not unrolled, as this is rare and must not crowd what is not.
template <typename S, typename T>
__device__ __forceinline__ void far_row(bool mine, const uint4* place, const T* x, const float* weight,
                                        const float* bias, const Edges<S, T>& edges, float over_d, float eps, float mu,
                                        float2* scratch, T* y, float* mean, float* rstd) {
    constexpr int kStep = S::L * S::N;
    const int left = mine ? edges.left : 0;
    // each of the row's vectors that this lane holds: its number and its values
    const auto vectors = [&](auto f) {
#pragma unroll 1
        for (int e = 0; e * kStep < left; ++e) {
            Vec<T, S::N> v;
            if constexpr (S::N > 1) v = *reinterpret_cast<const Vec<T, S::N>*>(place + e * S::kThreads);
            else v = *reinterpret_cast<const Vec<T, S::N>*>(x + e * kStep);
            float q[S::N];
            unpack(q, v);
            f(e, q);
        }
    };
    float t = 0.f, t2 = 0.f;
    vectors([&](int e, float (&q)[S::N]) {
#pragma unroll
        for (int k = 0; k < S::N; ++k)
            if (!S::kShift || edges.in(e, k)) t += q[k] - mu;
    });
    const float off = group_sums<S::L>(t, 0.f, scratch).x * over_d;
    if (fabsf(off) <= FLT_MAX) mu += off;
    t = 0.f;
    vectors([&](int e, float (&q)[S::N]) {
#pragma unroll
        for (int k = 0; k < S::N; ++k)
            if (!S::kShift || edges.in(e, k)) {
                const float c = q[k] - mu;
                t += c;
                t2 = fmaf(c, c, t2);
            }
    });
    const float2 sums = group_sums<S::L>(t, t2, scratch);
    // about the unrounded mean
    const float squares = sums.y <= FLT_MAX ? fmaxf(fmaf(-sums.x, sums.x * over_d, sums.y), 0.f) : sums.y;
    const float rs = inverse_root(fmaf(squares, over_d, eps));
    vectors([&](int e, float (&q)[S::N]) {
        const int at = e * kStep;
        typename S::P we[S::n], be[S::n], c[S::n];
        load_vector_params<S>(we, weight, e, left, edges.before, 1.f);
        load_vector_params<S>(be, bias, e, left, edges.before, 0.f);
        Vec<float, S::N> f;
#pragma unroll
        for (int k = 0; k < S::N; ++k) f.v[k] = !S::kShift || edges.in(e, k) ? (q[k] - mu) * rs : 0.f;
        unpack_pairs<S::N>(c, f);
#pragma unroll
        for (int k = 0; k < S::n; ++k) c[k] = pfma(c[k], we[k], be[k]);
        Vec<T, S::N> o;
        pack_pairs<S::N>(o, c);
        if (!edges.partial(e)) {
            *reinterpret_cast<Vec<T, S::N>*>(y + at) = o;
        } else {
#pragma unroll
            for (int k = 0; k < S::N; ++k)
                if (edges.in(e, k)) y[at + k] = element(o, k);
        }
    });
    if (mine && threadIdx.x % S::L == 0) {
        if (mean) *mean = mu;
        if (rstd) *rstd = rs;
    }
}

// The rows of a row group: first, first + stride, ..; and the most that a group of the block has.
struct Rows {
    int mine, most;
};
__device__ __forceinline__ Rows rows_of(int64_t rows, int64_t stride, int64_t first, int64_t block) {
    return {first < rows ? (int)((rows - 1 - first) / stride) + 1 : 0,
            block < rows ? (int)((rows - 1 - block) / stride) + 1 : 0};
}

// stride is a multiple of groups: every row of a row group has the same weight row.
template <typename T, typename S>
__global__ void __launch_bounds__(S::kThreads, ForwardPlan<T, S>::by_registers)
layer_norm_kernel(const T* x, const float* weight, const float* bias, int64_t rows, int groups, int d, float eps, T* y,
                  float* mean, float* rstd, int64_t stride) {
    constexpr int U = ForwardPlan<T, S>::U;
    using A = typename ForwardPlan<T, S>::A;
    constexpr bool kBlock = S::L > 32;                       // a row takes the block
    constexpr int kWarps = S::L / 32;
    __shared__ float2 scratch[kBlock ? (2 * U + 1) * kWarps : 1];
    extern __shared__ uint4 ahead[];                         // [depth][U][E][kThreads]
    const int64_t first = (int64_t)blockIdx.x * S::kRows + threadIdx.x / S::L, step = stride * d;
    const int shift = shift_of<S>(first, d);
    const int lane = threadIdx.x % S::L, col = lane * S::N - shift;
    const Edges<S, T> edges(col, d);
    const int left = edges.left, before = edges.before;
    const float over_d = 1.f / (float)d;
    // of a row's columns, those of this warp, and those of the warp that this lane takes up
    constexpr int kWidth = power_of_two(kWarps);
    const int takes = (threadIdx.x & 31) % kWidth;
    const float over_columns = kBlock ? 1.f / fmaxf((float)warp_columns<S>(threadIdx.x >> 5, d, shift), 1.f) : over_d;
    const float n = kBlock && takes < kWarps ? (float)warp_columns<S>(takes, d, shift) : 0.f;
    const float over_n = 1.f / fmaxf(n, 1.f);
    // the group's weights stay where the registers allow it
    constexpr bool kHeld = S::kValues <= kHeldValues;
    using P = typename S::P;
    P w[S::kPairs], b[S::kPairs];
    const int64_t at = first % groups * d + col;
    constexpr bool kStaged = ForwardPlan<T, S>::staged;
    P* staged = reinterpret_cast<P*>(reinterpret_cast<char*>(ahead) + A::bytes) + threadIdx.x;
    if (kHeld) {
        load_row_params<S>(w, row_of(weight, at), left, before, 1.f);
        load_row_params<S>(b, row_of(bias, at), left, before, 0.f);
    } else if (kStaged) {
#pragma unroll 1
        for (int e = 0; e < S::E; ++e) {
            P we[S::n], be[S::n];
            load_vector_params<S>(we, row_of(weight, at), e, left, before, 1.f);
            load_vector_params<S>(be, row_of(bias, at), e, left, before, 0.f);
#pragma unroll
            for (int k = 0; k < S::n; ++k) {
                staged[(e * S::n + k) * S::kThreads] = we[k];
                staged[(S::kPairs + e * S::n + k) * S::kThreads] = be[k];
            }
        }
    }
    uint4* mine = ahead + threadIdx.x;
    const Rows have = rows_of(rows, stride, first, (int64_t)blockIdx.x * S::kRows);
    const T* next_x = x + first * d + col;                   // of the turn to copy, or to load
    T* next_y = y + first * d + col;
    int64_t row = first;
    auto copy_turn = [&](int turn) {
        if (A::on) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (turn * U + u < have.mine)
                    copy_row<S, T>(mine + ((turn % A::depth) * U + u) * S::E * S::kThreads, next_x + u * step, left,
                                   x + rows * d);
            copies_done();
            next_x += U * step;
        }
    };
    if (A::on)
        for (int t = 0; t < A::depth - 1; ++t) copy_turn(t);
    for (int turn = 0; turn * U < have.most; ++turn) {
        copy_turn(turn + A::depth - 1);
        if (A::on) wait_copies<A::depth - 1>();
        Vec<T, S::N> v[U][S::E];
        float s[U], q[U];
        bool far = false;
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_row<S, T>(v[u], A::on ? mine + ((turn % A::depth) * U + u) * S::E * S::kThreads : nullptr,
                           next_x + u * step, turn * U + u < have.mine ? left : 0, edges);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            P t = psplat<P>(0.f);
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                P f[S::n];
                unpack_pairs<S::N>(f, v[u][e]);
#pragma unroll
                for (int k = 0; k < S::n; ++k) t = padd(t, f[k]);
            }
            s[u] = lane_sum<kBlock ? 32 : S::L>(psum(t));
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < S::E; ++e) keep_packed(v[u][e]);
        // deviations from the mean, of the warp's own columns where a row takes several warps
        float mean_here[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean_here[u] = s[u] * over_columns;
            const P minus = psplat<P>(-mean_here[u]);
            P t = psplat<P>(0.f);
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                if (e * S::L * S::N < left) {
                    P f[S::n];
                    unpack_pairs<S::N>(f, v[u][e]);
                    deviations(f, minus, e, edges);
#pragma unroll
                    for (int k = 0; k < S::n; ++k) t = pfma(f[k], f[k], t);
                }
            q[u] = lane_sum<kBlock ? 32 : S::L>(psum(t));
        }
        if constexpr (kBlock) {
            // sum over the warps of q_w + n_w (mean_w - mean)^2
            const int wl = threadIdx.x & 31;
            float2* half = scratch + (turn & 1) * U * kWarps;
            if (wl == 0)
#pragma unroll
                for (int u = 0; u < U; ++u) half[u * kWarps + (threadIdx.x >> 5)] = make_float2(s[u], q[u]);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float2 of = takes < kWarps ? half[u * kWarps + takes] : make_float2(0.f, 0.f);
                mean_here[u] = lane_sum<kWidth>(of.x) * over_d;
                const float off = fmaf(of.x, over_n, -mean_here[u]);
                q[u] = lane_sum<kWidth>(fmaf(n * off, off, of.y));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < S::E; ++e) keep_packed(v[u][e]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (turn * U + u >= have.mine) continue;
            const float mu = mean_here[u], var = q[u] * over_d, rs = inverse_root(var + eps);
            far |= far_mean(mu, var);
            const P minus = psplat<P>(-mu), times = psplat<P>(rs);
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                constexpr int kStep = S::L * S::N;
                if (e * kStep >= left) continue;
                // parameters one vector at a time: loaded ahead they would push the row out of the registers
                if (!kHeld) asm volatile("" ::: "memory");
                P f[S::n], we[S::n], be[S::n];
                unpack_pairs<S::N>(f, v[u][e]);
                if (kStaged) {
                    staged_params<S>(we, staged, e);
                    staged_params<S>(be, staged + S::kPairs * S::kThreads, e);
                } else if (!kHeld) {
                    load_vector_params<S>(we, row_of(weight, at), e, left, before, 1.f);
                    load_vector_params<S>(be, row_of(bias, at), e, left, before, 0.f);
                }
#pragma unroll
                for (int k = 0; k < S::n; ++k)
                    f[k] = pfma(pmul(padd(f[k], minus), times), kHeld ? w[e * S::n + k] : we[k],
                                kHeld ? b[e * S::n + k] : be[k]);
                Vec<T, S::N> o;
                pack_pairs<S::N>(o, f);
                store_vector<S>(next_y + u * step + e * kStep, o, e, edges);
            }
            if (lane == 0) {
                if (mean) mean[row + u * stride] = mu;
                if (rstd) rstd[row + u * stride] = rs;
            }
        }
        // (after the turn: in its middle the branch cost 8 percent more; rows of a block: the same in all of it)
        if (__any_sync(0xffffffffu, far)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool mine_far = turn * U + u < have.mine && far_mean(mean_here[u], q[u] * over_d);
                far_row<S, T>(mine_far, mine + ((turn % A::depth) * U + u) * S::E * S::kThreads, next_x + u * step,
                              row_of(weight, at), row_of(bias, at), edges, over_d, eps, mean_here[u],
                              scratch + (kBlock ? 2 * U * kWarps : 0), next_y + u * step,
                              row_of(mean, row + u * stride), row_of(rstd, row + u * stride));
            }
        }
        if (!A::on) next_x += U * step;
        next_y += U * step;
        row += U * stride;
    }
}

// part[slot][d]: the weight and bias gradients of one weight row over some rows, slot i of weight row
// i mod groups.  A block has `weights` weight rows, and its row groups add up their sums of each first.  weights
// is kRows (nothing to add up), groups, or 1: then the block's rows lie `groups` apart.
template <typename T, typename S>
__global__ void __launch_bounds__(S::kThreads, BackwardPlan<T, S>::by_registers)
layer_norm_backward_kernel(const T* x, const T* dy, const float* weight, const float* mean, const float* rstd,
                           int64_t rows, int groups, int d, T* dx, float2* part, int64_t stride, int weights) {
    constexpr int U = BackwardPlan<T, S>::U;
    using A = typename BackwardPlan<T, S>::A;
    __shared__ float scratch[S::L > 32 ? 4 * U * S::L / 32 : 1];
    extern __shared__ uint4 ahead[];                        // [depth][U][x, dy][E][kThreads]
    float2* sums = reinterpret_cast<float2*>(ahead);        // afterwards [kRows][d], L <= 32
    uint4* mine = ahead + threadIdx.x;
    const int group = threadIdx.x / S::L, lane = threadIdx.x % S::L;
    const bool apart = S::kRows > 1 && weights == 1;         // (and for one weight row either is the same)
    const int64_t block = apart ? (int64_t)(blockIdx.x / groups) * groups * S::kRows + blockIdx.x % groups
                                : (int64_t)blockIdx.x * S::kRows;
    const int64_t first = block + (apart ? (int64_t)group * groups : group), step = stride * d;
    const int shift = shift_of<S>(first, d), col = lane * S::N - shift;
    const Edges<S, T> edges(col, d);
    const int left = edges.left, before = edges.before;
    const float over_d = 1.f / d;
    constexpr bool kHeld = S::kValues <= 8;
    const int64_t at = first % groups * d + col;            // stride is a multiple of groups
    using P = typename S::P;
    P w[S::kPairs], dw[S::kPairs], db[S::kPairs];
    constexpr bool kStaged = BackwardPlan<T, S>::staged;
    P* staged = reinterpret_cast<P*>(reinterpret_cast<char*>(ahead) + A::bytes) + threadIdx.x;
    if (kHeld || kStaged) load_row_params<S>(w, row_of(weight, at), left, before, 1.f);
    if (kStaged)
#pragma unroll
        for (int k = 0; k < S::kPairs; ++k) staged[k * S::kThreads] = w[k];
#pragma unroll
    for (int k = 0; k < S::kPairs; ++k) dw[k] = db[k] = psplat<P>(0.f);
    const Rows have = rows_of(rows, stride, first, block);
    auto place = [&](int turn, int u, int array) {
        return mine + (((turn % A::depth) * U + u) * 2 + array) * S::E * S::kThreads;
    };
    const T *next_x = x + first * d + col, *next_dy = dy + first * d + col;   // of the turn to copy, or to load
    T* next_dx = dx + first * d + col;
    const float *next_mean = mean + first, *next_rstd = rstd + first;
    auto copy_turn = [&](int turn) {
        if (A::on) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (turn * U + u < have.mine) {
                    copy_row<S, T>(place(turn, u, 0), next_x + u * step, left, x + rows * d);
                    copy_row<S, T>(place(turn, u, 1), next_dy + u * step, left, dy + rows * d);
                }
            copies_done();
            next_x += U * step;
            next_dy += U * step;
        }
    };
    float ahead_mu[U], ahead_rs[U];
    auto load_stats = [&](int turn) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ahead_mu[u] = turn * U + u < have.mine ? next_mean[u * stride] : 0.f;
            ahead_rs[u] = turn * U + u < have.mine ? next_rstd[u * stride] : 0.f;
        }
        next_mean += U * stride;
        next_rstd += U * stride;
    };
    if (A::on)
        for (int t = 0; t < A::depth - 1; ++t) copy_turn(t);
    load_stats(0);
    for (int turn = 0; turn * U < have.most; ++turn) {
        copy_turn(turn + A::depth - 1);
        if (A::on) wait_copies<A::depth - 1>();
        Vec<T, S::N> v[U][S::E], g[U][S::E];
        P xhs[U][kHeld ? S::kPairs : 1], ts[U][kHeld ? S::kPairs : 1];   // xh and w dy, kept where there is room
        float mu[U], rs[U], sums_of[2 * U];                 // of w dy, and of w dy xh
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int there = turn * U + u < have.mine ? left : 0;
            load_row<S, T>(v[u], A::on ? place(turn, u, 0) : nullptr, next_x + u * step, there, edges);
            load_row<S, T>(g[u], A::on ? place(turn, u, 1) : nullptr, next_dy + u * step, there, edges);
            mu[u] = ahead_mu[u];
            rs[u] = ahead_rs[u];
        }
        load_stats(turn + 1);
        if (kStaged) {
#pragma unroll
            for (int e = 0; e < S::E; ++e) staged_params<S>(w + e * S::n, staged, e);
        } else if (!kHeld) {
            load_row_params<S>(w, row_of(weight, at), left, before, 1.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const P minus = psplat<P>(-mu[u]), times = psplat<P>(rs[u]);
            P s1 = psplat<P>(0.f), s2 = s1;
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                if (turn * U + u < have.mine && e * S::L * S::N < left) {
                    P fx[S::n], fg[S::n];
                    unpack_pairs<S::N>(fx, v[u][e]);
                    unpack_pairs<S::N>(fg, g[u][e]);
                    // what lies outside the row is zero in dy: its xh matters where it is not finite
                    if (!S::kShift || fabsf(mu[u] * rs[u]) <= FLT_MAX) {
#pragma unroll
                        for (int k = 0; k < S::n; ++k) fx[k] = padd(fx[k], minus);
                    } else {
                        deviations(fx, minus, e, edges);
                    }
#pragma unroll
                    for (int k = 0; k < S::n; ++k) {
                        const int i = e * S::n + k;
                        const P xh = pmul(fx[k], times), t = pmul(fg[k], w[i]);
                        s1 = padd(s1, t);
                        s2 = pfma(t, xh, s2);
                        dw[i] = pfma(fg[k], xh, dw[i]);
                        db[i] = padd(db[i], fg[k]);
                        if (kHeld) {
                            xhs[u][i] = xh;
                            ts[u][i] = t;
                        }
                    }
                }
            sums_of[u] = psum(s1);
            sums_of[U + u] = psum(s2);
        }
        row_sums<S, 2 * U>(sums_of, scratch, turn);
        if (!kHeld)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < S::E; ++e) {
                    keep_packed(v[u][e]);
                    keep_packed(g[u][e]);
                }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (turn * U + u >= have.mine) continue;
            const P m1 = psplat<P>(-sums_of[u] * over_d), m2 = psplat<P>(-sums_of[U + u] * over_d);
            const P minus = psplat<P>(-mu[u]), times = psplat<P>(rs[u]);
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                constexpr int kStep = S::L * S::N;
                if (e * kStep >= left) continue;
                P o[S::n], fg[S::n];
                if (!kHeld) {
                    unpack_pairs<S::N>(o, v[u][e]);
                    unpack_pairs<S::N>(fg, g[u][e]);
                }
#pragma unroll
                for (int k = 0; k < S::n; ++k) {
                    const int i = e * S::n + k;
                    const P xh = kHeld ? xhs[u][i] : pmul(padd(o[k], minus), times);
                    const P t = kHeld ? ts[u][i] : pmul(fg[k], w[i]);
                    o[k] = pmul(times, pfma(xh, m2, padd(t, m1)));
                }
                Vec<T, S::N> out;
                pack_pairs<S::N>(out, o);
                store_vector<S>(next_dx + u * step + e * kStep, out, e, edges);
            }
        }
        if (!A::on) {
            next_x += U * step;
            next_dy += U * step;
        }
        next_dx += U * step;
    }
    asm volatile("griddepcontrol.launch_dependents;");
    if (!part) return;
    float wv[S::kValues], bv[S::kValues];
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        Vec<float, S::N> q;
        P f[S::n];
#pragma unroll
        for (int k = 0; k < S::n; ++k) f[k] = dw[e * S::n + k];
        pack_pairs<S::N>(q, f);
#pragma unroll
        for (int k = 0; k < S::N; ++k) wv[e * S::N + k] = q.v[k];
#pragma unroll
        for (int k = 0; k < S::n; ++k) f[k] = db[e * S::n + k];
        pack_pairs<S::N>(q, f);
#pragma unroll
        for (int k = 0; k < S::N; ++k) bv[e * S::N + k] = q.v[k];
    }
    if (weights < S::kRows) {
        __syncthreads();                                    // the copies' places are free
#pragma unroll
        for (int e = 0; e < S::E; ++e)
#pragma unroll
            for (int k = 0; k < S::N; ++k) {
                const int c = e * S::L * S::N + col + k;
                if ((!S::kShift || c >= 0) && c < d)
                    sums[group * d + c] = make_float2(wv[e * S::N + k], bv[e * S::N + k]);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < weights * d; i += S::kThreads) {
            float2 t = sums[i];
            for (int r = weights; r < S::kRows; r += weights) {
                const float2 q = sums[r * d + i];
                t.x += q.x;
                t.y += q.y;
            }
            part[(int64_t)blockIdx.x * weights * d + i] = t;
        }
    } else {
#pragma unroll
        for (int e = 0; e < S::E; ++e)
#pragma unroll
            for (int k = 0; k < S::N; ++k) {
                const int c = e * S::L * S::N + col + k;
                if ((!S::kShift || c >= 0) && c < d)
                    part[first * d + c] = make_float2(wv[e * S::N + k], bv[e * S::N + k]);
            }
    }
}

// A sum and what its additions have rounded away (the exact error of each, by two-sum): as good as fp64,
// whose two additions a clock per SM made the join take 40 us.
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x, b = t - s;
        c += (s - (t - b)) + (x - b);
        s = t;
    }
    __device__ __forceinline__ void join(float s2, float c2) {
        add(s2);
        c += c2;
    }
    __device__ __forceinline__ float value() const {
        const float t = s + c;
        return isfinite(s) ? t : s;     // infinities leave no error term
    }
};

// Column sums of part[M][n]: 8 columns a block, 32 threads a column (few columns per block, so that a few
// hundred columns still spread over the SMs: 32 a block took 9 us for 512 columns).
__global__ void __launch_bounds__(kJoinCols * kJoinRows) layer_norm_join_kernel(const float2* part, int64_t M,
                                                                                int64_t n, float* dweight,
                                                                                float* dbias) {
    constexpr int kWarps = kJoinCols * kJoinRows / 32;
    __shared__ float4 sums[kWarps][kJoinCols];
    const int col = threadIdx.x % kJoinCols, r = threadIdx.x / kJoinCols, warp = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * kJoinCols + col;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Sum dw, db;
    if (j < n)
#pragma unroll 4
        for (int64_t m = r; m < M; m += kJoinRows) {
            const float2 v = part[m * n + j];
            dw.add(v.x);
            db.add(v.y);
        }
#pragma unroll
    for (int o = 16; o >= kJoinCols; o >>= 1) {
        dw.join(__shfl_down_sync(0xffffffffu, dw.s, o), __shfl_down_sync(0xffffffffu, dw.c, o));
        db.join(__shfl_down_sync(0xffffffffu, db.s, o), __shfl_down_sync(0xffffffffu, db.c, o));
    }
    if ((threadIdx.x & 31) < kJoinCols) sums[warp][col] = make_float4(dw.s, dw.c, db.s, db.c);
    __syncthreads();
    if (threadIdx.x >= kJoinCols || j >= n) return;
    for (int w = 1; w < kWarps; ++w) {
        const float4 q = sums[w][col];
        dw.join(q.x, q.y);
        db.join(q.z, q.w);
    }
    if (dweight) dweight[j] = dw.value();
    if (dbias) dbias[j] = db.value();
}

struct Args {
    const void *x, *dy;
    const float *weight, *bias, *mean_in, *rstd_in;
    int64_t rows;
    int groups, d, sms;
    float eps;
    void* out;
    float *mean, *rstd;
    float2* part;
    cudaStream_t stream;
};

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// As many blocks as there are rows for, at most those that run at once (a few more would take as long again), a
// multiple of `unit`.
template <typename Plan, typename S>
int64_t blocks_for(int64_t rows, int64_t unit, int sms) {
    const int64_t most = (int64_t)sms * Plan::per_sm, wanted = rows > S::kRows ? ceil_div(rows, S::kRows) : 1;
    const int64_t blocks = ceil_div(wanted, unit) * unit;
    return blocks <= most ? blocks : most >= unit ? most / unit * unit : unit;
}
int64_t lcm(int64_t a, int b) { return a / gcd((int)(a % b), b) * b; }
// A block's row groups meet the same weight rows on every turn, and rows with the same shift.
template <typename S>
int64_t whole_turns(int groups, int d) {
    const int64_t unit = groups / gcd(groups, S::kRows);
    return S::kShift ? lcm(unit, S::N / gcd(S::N, S::kRows * (d % S::N))) : unit;
}
// Weight rows of a block of the backward (see the kernel).
template <typename Plan, typename S>
int weights_of_block(int groups, int sms) {
    if (S::kRows % groups == 0) return groups;
    return groups <= sms * Plan::per_sm ? 1 : S::kRows;
}
template <typename Plan, typename S>
int64_t backward_blocks(int64_t rows, int groups, int d, int sms) {
    const int64_t unit = whole_turns<S>(groups, d);
    return blocks_for<Plan, S>(rows, weights_of_block<Plan, S>(groups, sms) == 1 ? lcm(unit, groups) : unit, sms);
}
// Rows of the matrix of partial sums.
template <typename Plan, typename S>
int64_t slots(int64_t rows, int groups, int d, int sms) {
    if (rows <= 0) return 0;
    return backward_blocks<Plan, S>(rows, groups, d, sms) * weights_of_block<Plan, S>(groups, sms) / groups;
}

template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes) {
    if (bytes <= 40 * 1024) return cudaSuccess;      // 48 KB with the static part need no permission
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

struct Forward {
    static constexpr bool kForward = true;
    template <typename T, typename S>
    static int64_t run(const Args& a) {
        using Plan = ForwardPlan<T, S>;
        const int64_t blocks = blocks_for<Plan, S>(a.rows, whole_turns<S>(a.groups, a.d), a.sms);
        const cudaError_t e = allow_shared(layer_norm_kernel<T, S>, Plan::bytes);
        if (e != cudaSuccess) return (int64_t)e;
        layer_norm_kernel<T, S><<<(unsigned)blocks, S::kThreads, Plan::bytes, a.stream>>>(
            static_cast<const T*>(a.x), a.weight, a.bias, a.rows, a.groups, a.d, a.eps, static_cast<T*>(a.out), a.mean,
            a.rstd, blocks * S::kRows);
        return (int64_t)cudaGetLastError();
    }
};
struct Backward {
    static constexpr bool kForward = false;
    template <typename T, typename S>
    static int64_t run(const Args& a) {
        using Plan = BackwardPlan<T, S>;
        const int64_t blocks = backward_blocks<Plan, S>(a.rows, a.groups, a.d, a.sms);
        const int weights = weights_of_block<Plan, S>(a.groups, a.sms);
        const size_t join = a.part && weights < S::kRows ? sizeof(float2) * S::kRows * (size_t)a.d : 0;
        const size_t smem = join > Plan::bytes ? join : Plan::bytes;
        const cudaError_t e = allow_shared(layer_norm_backward_kernel<T, S>, smem);
        if (e != cudaSuccess) return (int64_t)e;
        layer_norm_backward_kernel<T, S><<<(unsigned)blocks, S::kThreads, smem, a.stream>>>(
            static_cast<const T*>(a.x), static_cast<const T*>(a.dy), a.weight, a.mean_in, a.rstd_in, a.rows, a.groups,
            a.d, static_cast<T*>(a.out), a.part, blocks * S::kRows, weights);
        return (int64_t)cudaGetLastError();
    }
};
struct Slots {
    static constexpr bool kForward = false;
    template <typename T, typename S>
    static int64_t run(const Args& a) { return slots<BackwardPlan<T, S>, S>(a.rows, a.groups, a.d, a.sms); }
};

// The lanes and vectors of a row.  One vector a lane, or two where the forward has bf16 rows (half the
// lanes: the sums across lanes are most of its instructions; 27 us instead of 31 for 8192 x 4096.  The
// backward's sums per column leave no room for two: 59 us instead of 48).  Up to 64 vectors share a
// warp, two a lane from 32 on, longer rows take a block of up to 512 lanes.
// Rows that are not whole vectors: by the vectors that hold them (16384 x 1001 in bf16: 25 us, element by
// element 33 us; 4096 x 5001 35 and 82 us, its gradients 59 and 171 us).  Element by element where an array does not
// start on 16 bytes, and for the gradients of rows of a few warps (65536 x 300 in bf16: 64 us, as vectors 68 us;
// 16384 x 1001 fp32 46 and 55 us; 4096 x 1023 bf16 17 and 19 us): the sums per column of lanes that hold
// vectors fill the registers, and blocks as small as that leave more of them to join.
enum RowLayout { kElements, kShifted, kVectors };

template <typename Op, typename T, bool Shift>
int64_t by_vectors(const Args& a, int n) {
    constexpr int N = 16 / sizeof(T), E = Op::kForward && N == 8 ? 2 : 1;
    if (n <= 4) return Op::template run<T, Shape<4, 1, N, Shift>>(a);
    if (n <= 8) return Op::template run<T, Shape<8 / E, E, N, Shift>>(a);
    if (n <= 16) return Op::template run<T, Shape<16 / E, E, N, Shift>>(a);
    if (n <= 32) return Op::template run<T, Shape<32 / E, E, N, Shift>>(a);
    // (shifted gradients in bf16: two vectors a lane leave no room to hold the weights)
    if (n <= 64) {
        if constexpr (Shift && !Op::kForward && N == 8) return Op::template run<T, Shape<64, 1, N, Shift>>(a);
        else return Op::template run<T, Shape<32, 2, N, Shift>>(a);
    }
    if (n <= 128) return Op::template run<T, Shape<128 / E, E, N, Shift>>(a);
    if (n <= 192) return Op::template run<T, Shape<192 / E, E, N, Shift>>(a);
    if (n <= 256) return Op::template run<T, Shape<256 / E, E, N, Shift>>(a);
    if constexpr (Shift)
        if (n <= 320) return Op::template run<T, Shape<320 / E, E, N, Shift>>(a);      // rows of a power of two of them
    if (n <= 384) return Op::template run<T, Shape<384 / E, E, N, Shift>>(a);
    if (n <= 512) return Op::template run<T, Shape<512 / E, E, N, Shift>>(a);
    if (n <= 1024) return Op::template run<T, Shape<512, 2, N, Shift>>(a);
    if (n <= 2048) return Op::template run<T, Shape<512, 4, N, Shift>>(a);
    if constexpr (N == 4) return Op::template run<T, Shape<512, 8, N, Shift>>(a);
    return (int64_t)cudaErrorInvalidValue;      // d <= LA_MAX_NORM_D: not reached
}
template <typename Op, typename T>
int64_t by_shape(const Args& a, RowLayout layout) {
    constexpr int N = 16 / sizeof(T);
    const int d = a.d, shifted = (d + 2 * N - 2) / N;      // vectors that hold a row, wherever it starts
    if (layout == kVectors && d % N == 0) return by_vectors<Op, T, false>(a, d / N);
    const bool few_warps = !Op::kForward && d > 256 && d <= 1024;
    if (layout != kElements && !few_warps && shifted <= LA_MAX_NORM_D / N) return by_vectors<Op, T, true>(a, shifted);
    if (d <= 32) return Op::template run<T, Shape<32, 1, 1>>(a);
    if (d <= 128) return Op::template run<T, Shape<32, 4, 1>>(a);
    if (d <= 512) return Op::template run<T, Shape<128, 4, 1>>(a);
    if (d <= 1024) return Op::template run<T, Shape<256, 4, 1>>(a);
    if (d <= 4096) return Op::template run<T, Shape<512, 8, 1>>(a);
    return Op::template run<T, Shape<512, 32, 1>>(a);
}
template <typename Op>
int64_t by_type(const Args& a, int dtype, RowLayout layout) {
    return dtype == LA_F32 ? by_shape<Op, float>(a, layout) : by_shape<Op, __nv_bfloat16>(a, layout);
}

bool on_16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int64_t slots_for(int dtype, int64_t rows, int groups, int d, int sms, RowLayout layout) {
    Args a{};
    a.rows = rows;
    a.groups = groups;
    a.d = d;
    a.sms = sms;
    return by_type<Slots>(a, dtype, layout);
}
// rows: the arrays of rows start on 16 bytes; weights: the arrays of weights too.
RowLayout layout_of(bool rows, bool weights) { return !rows ? kElements : weights ? kVectors : kShifted; }

}  // namespace

cudaError_t layer_norm(const void* x, const float* weight, const float* bias, int dtype, int64_t rows, int groups,
                       int d, float eps, void* y, float* mean, float* rstd, cudaStream_t s) {
    Args a{};
    a.x = x; a.weight = weight; a.bias = bias;
    a.rows = rows; a.groups = groups; a.d = d; a.sms = sm_count(); a.eps = eps;
    if (a.sms <= 0) return cudaErrorInvalidDevice;
    a.out = y; a.mean = mean; a.rstd = rstd; a.stream = s;
    return (cudaError_t)by_type<Forward>(a, dtype, layout_of(on_16(x) && on_16(y), on_16(weight) && on_16(bias)));
}

// Covers every layout of the rows: the choice between them goes by the call's pointers.
size_t layer_norm_backward_workspace_bytes(int dtype, int64_t rows, int groups, int d) {
    const int sms = sm_count();
    if (sms <= 0) return 0;
    int64_t most = 0;
    for (RowLayout l : {kElements, kShifted, kVectors}) {
        const int64_t n = slots_for(dtype, rows, groups, d, sms, l);
        if (n > most) most = n;
    }
    return align_up(sizeof(float2) * (size_t)most * groups * d, kAlign) + kAlign;
}

cudaError_t layer_norm_backward(const void* x, const void* dy, const float* weight, const float* mean,
                                const float* rstd, int dtype, int64_t rows, int groups, int d, void* dx,
                                float* dweight, float* dbias, void* workspace, cudaStream_t s) {
    const RowLayout layout = layout_of(on_16(x) && on_16(dy) && on_16(dx), on_16(weight));
    Args a{};
    a.x = x; a.dy = dy; a.weight = weight; a.mean_in = mean; a.rstd_in = rstd;
    a.rows = rows; a.groups = groups; a.d = d; a.sms = sm_count();
    if (a.sms <= 0) return cudaErrorInvalidDevice;
    a.out = dx; a.stream = s;
    a.part = dweight || dbias ? static_cast<float2*>(workspace) : nullptr;
    if (rows > 0) {
        const cudaError_t e = (cudaError_t)by_type<Backward>(a, dtype, layout);
        if (e != cudaSuccess) return e;
    }
    if (!a.part) return cudaSuccess;
    const int64_t n = (int64_t)groups * d, M = rows > 0 ? slots_for(dtype, rows, groups, d, a.sms, layout) : 0;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)ceil_div(n, kJoinCols));
    cfg.blockDim = dim3(kJoinCols * kJoinRows);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, layer_norm_join_kernel, static_cast<const float2*>(a.part), M, n, dweight, dbias);
}

}  // namespace la
