// Rotary positions: pair p of every head of token t turns by
// positions[t][axis(p)] * freq[p].
//
// Angles.  A position is an integer, so freq / 2 pi as a 64-bit fixed-point
// fraction of a turn times the position, modulo 2^64, is the angle modulo one
// turn with an error of |position| 2^-54 or less turns, at any distance.  Read as
// a signed number it is an angle in [-pi, pi), whose cos and sin are taken in fp32.
//
// Bound by memory: each channel is read and written once.  A block turns a few
// tokens: its threads first issue the loads of their channels, then compute the
// tokens' cos and sin into shared memory (once for all heads of q and k), then
// turn and store.  A thread's unit of work is N neighbouring channels and, where
// pairs are halves, their N partners; N channels are 16 bytes where every row
// allows it, else one pair is the unit.
#include "internal.h"
#include "vec.cuh"

namespace la {

namespace {

constexpr int kRotaryThreads = 256;
constexpr int kUnits = 4;               // units whose loads a thread issues before the first is used

// freq / 2 pi modulo 1 in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_fraction(float freq) {
    const double turns = (double)freq * 0.15915494309189533577;   // 1 / (2 pi)
    const double frac = turns - floor(turns);                     // [0, 1]
    return (unsigned long long)(long long)((frac < 0.5 ? frac : frac - 1.0) * 18446744073709551616.0);
}

// Units of a block: token x (q's heads, then k's) x unit within the head.  Units 0 .. pair_units - 1
// turn pairs, the rest copy channels that are not rotated.
struct RotaryPlan {
    int tokens;          // tokens per block
    int heads;           // heads of q and k together
    int pair_units, units;   // per head
};

template <typename T, int N, bool Interleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p,
                                                               const __grid_constant__ RotaryPlan plan) {
    extern __shared__ float2 cs[];       // [tokens][P]
    using V = Vec<T, N>;
    const int64_t t0 = (int64_t)blockIdx.x * plan.tokens;
    const int tokens = (int)min64(plan.tokens, p.T - t0);
    const int per_token = plan.heads * plan.units, total = tokens * per_token;

    auto turn_units = [&](int first, bool table) {
        V a[kUnits], b[kUnits];
        T* out[kUnits];
        int pair[kUnits];                // token * P + first pair, or -1: copied; -2: nothing
        constexpr bool kOne = Interleaved && N > 1;   // whole pairs in one vector
        constexpr int kPairs = kOne ? N / 2 : N;
        const int second = Interleaved ? 1 : p.P;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int i = first + u * kRotaryThreads;
            pair[u] = -2;
            if (i >= total) continue;
            const int t = i / per_token, r = i - t * per_token, h = r / plan.units, e = r - h * plan.units;
            const bool is_k = h >= p.H;
            const int64_t row = ((t0 + t) * p.H + (is_k ? h - p.H : h)) * p.d;
            const bool turned = e < plan.pair_units;
            const int c = turned ? (Interleaved ? 2 : 1) * e * kPairs : 2 * p.P + (e - plan.pair_units) * N;
            const T* x = static_cast<const T*>(is_k ? p.k : p.q) + row + c;
            out[u] = static_cast<T*>(is_k ? p.k_out : p.q_out) + row + c;
            a[u] = *reinterpret_cast<const V*>(x);
            if (turned && !kOne) b[u] = *reinterpret_cast<const V*>(x + second);
            pair[u] = turned ? t * p.P + e * kPairs : -1;
        }
        if (table) {
            for (int i = threadIdx.x; i < tokens * p.P; i += kRotaryThreads) {
                const int t = i / p.P, j = i - t * p.P;
                int axis = 0;
                while (axis + 1 < p.naxes && j >= p.first[axis + 1]) ++axis;
                const float f = p.freq[j];
                const unsigned long long turn =
                    turn_fraction(f) * (unsigned long long)(long long)p.positions[(t0 + t) * p.naxes + axis];
                float s, c;
                sincospif((float)(long long)turn * 0x1p-63f, &s, &c);
                if (!isfinite(f)) s = c = __int_as_float(0x7fc00000);
                cs[i] = make_float2(c, p.inverse ? -s : s);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (pair[u] == -2) continue;
            if (pair[u] >= 0) {
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const float2 w = cs[pair[u] + k];
                    T& x0 = a[u].v[kOne ? 2 * k : k];
                    T& x1 = kOne ? a[u].v[kOne ? 2 * k + 1 : 0] : b[u].v[k];
                    const float f0 = up(x0), f1 = up(x1);
                    x0 = down<T>(f0 * w.x - f1 * w.y);
                    x1 = down<T>(f1 * w.x + f0 * w.y);
                }
                if (!kOne) *reinterpret_cast<V*>(out[u] + second) = b[u];
            }
            *reinterpret_cast<V*>(out[u]) = a[u];
        }
    };
    turn_units(threadIdx.x, true);
    for (int first = threadIdx.x + kUnits * kRotaryThreads; first < total; first += kUnits * kRotaryThreads)
        turn_units(first, false);
}

template <typename T, int N>
cudaError_t run(const RotaryParams& p, cudaStream_t s) {
    RotaryPlan plan{};
    plan.heads = p.k ? 2 * p.H : p.H;
    plan.pair_units = p.interleaved && N > 1 ? 2 * p.P / N : p.P / N;
    plan.units = plan.pair_units + (p.d - 2 * p.P) / N;
    // enough tokens that every thread has kUnits units, as far as the table fits 32 KB
    const int64_t per_token = (int64_t)plan.heads * plan.units;
    int64_t tokens = ceil_div((int64_t)kUnits * kRotaryThreads, per_token);
    tokens = min64(tokens, 32 * 1024 / ((int64_t)sizeof(float2) * p.P));
    tokens = min64(tokens > 0 ? tokens : 1, p.T);
    plan.tokens = (int)tokens;
    const size_t smem = sizeof(float2) * (size_t)tokens * p.P;
    const unsigned blocks = (unsigned)ceil_div(p.T, tokens);
    if (p.interleaved) rotary_kernel<T, N, true><<<blocks, kRotaryThreads, smem, s>>>(p, plan);
    else rotary_kernel<T, N, false><<<blocks, kRotaryThreads, smem, s>>>(p, plan);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const RotaryParams& p, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    // every unit starts on 16 bytes: the pointers, the rows, and where the second half and the tail begin
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                         reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_out);
    if (at % 16 == 0 && p.d % N == 0 && (p.interleaved ? 2 : 1) * p.P % N == 0) return run<T, N>(p, s);
    return run<T, 1>(p, s);
}

}  // namespace

cudaError_t rotary(const RotaryParams& p, int dtype, cudaStream_t s) {
    return dtype == LA_F32 ? dispatch<float>(p, s) : dispatch<__nv_bfloat16>(p, s);
}

}  // namespace la
