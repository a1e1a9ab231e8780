// Rotary positions: pair p of every head of token t turns by
// positions[t][axis(p)] * freq[p].
//
// Angles.  A position is an integer, so freq / 2 pi as a 64-bit fixed-point
// fraction of a turn times the position, modulo 2^64, is the angle modulo one
// turn.  The fraction is off by 2^-63 + 2^-106 |freq| turns at most, and the angle
// by |position| times that.  What is left of it beside whole quarters of a turn, pi / 4
// at most, is rounded to 2^-32 turns and to fp32, by pi 2^-27 in all, and goes through
// fp32 cos and sin.
//
// Bound by memory: each channel is read and written once.  A block turns a few
// tokens: its threads first issue the loads of their channels, then compute the
// tokens' cos and sin into shared memory (once for all heads of q and k), then
// turn and store.  A thread's unit of work is N neighbouring channels and, where
// pairs are halves, their N partners; N channels are 16 bytes where every row
// allows it.  Other rows are turned in shared memory, or pair by pair where
// the arrays do not start on 16 bytes or a few tokens' rows do not fit there.
//
// Measured (GB300, 6.76 TB/s copies): q and k of 65536 x 16 x 64 in bf16 81 us, 6.6 TB/s (32768 x 16 x 64 in
// fp32 80 us); 32768 x 7 x 83 in fp32 53 us, 5.7 TB/s; 32768 x 9 x 77
// in bf16, bound by instructions per pair, 43 us, 4.2 TB/s.
#include "ops/ops.h"
#include "ops/vec.cuh"

namespace la {

namespace {

constexpr int kRotaryThreads = 256;
constexpr int kUnits = 4;               // units whose loads a thread issues before the first is used

// freq / 2 pi modulo 1 in units of 2^-64, within two of them, or 2^-106 |freq|.  Below 4 a fixed-point product of the
// mantissa and 2^66 / (2 pi) (fp64 is slow here: with it for all, 65536 x 1 x 128 in bf16 took 25 us instead of 23);
// from there on two doubles, what a product rounds away and what the constant does, less their whole turns.
__device__ __forceinline__ unsigned long long turn_fraction(float freq) {
    const uint32_t bits = __float_as_uint(fabsf(freq)), exponent = bits >> 23;
    unsigned long long r;
    if (exponent <= 128) {
        // (numbers below the normal range, which have no leading one, are less than a unit like others above them)
        constexpr unsigned long long kTurn = 0xa2f9836e4e44152aull;
        const unsigned long long mantissa = (bits << 8) | 0x80000000u;
        const unsigned long long product = mantissa * (kTurn >> 32) + (mantissa * (kTurn & 0xffffffffu) >> 32);
        const uint32_t down = 128 - exponent;
        r = down < 64 ? product >> down : 0;
    } else {
        constexpr double kTurn = 0x1.45f306dc9c883p+61, kRest = -0x1.6b01ec5417056p+7;      // 2^64 / (2 pi)
        const double f = fabsf(freq);
        double turns = f * kTurn, rest = fma(f, kRest, fma(f, kTurn, -turns));
        turns = fma(rint(turns * 0x1p-64), -0x1p64, turns);
        rest = fma(rint(rest * 0x1p-64), -0x1p64, rest);
        r = (unsigned long long)__double2ll_rn(turns) + (unsigned long long)__double2ll_rn(rest);
    }
    return freq < 0.f ? 0 - r : r;
}

// What pair j turns by per position: the fraction is the same for all tokens (when all of it was fp64 work, which is slow
// here, 30000 x 3 x 201 with 100 pairs took 60 us with a fraction for every token; 42 now).
struct Turn {
    unsigned long long fraction;
    int axis;
    bool finite;
};
__device__ __forceinline__ Turn turn_of(const RotaryParams& p, int j) {
    int axis = 0;
    while (axis + 1 < p.naxes && j >= p.first[axis + 1]) ++axis;
    const float f = p.freq[j];
    return {turn_fraction(f), axis, (bool)isfinite(f)};
}
// (cos, sin) at token t; sin negated for the inverse.
__device__ __forceinline__ float2 cos_sin(const RotaryParams& p, const Turn& turn, int64_t t) {
    const long long position = p.positions[t * p.naxes + turn.axis];
    const unsigned long long angle = turn.fraction * (unsigned long long)position;
    // the nearest quarter of a turn apart, so that fp32 rounds what is left: an eighth at most, in units of 2^-32
    const uint32_t turns = (uint32_t)(angle >> 32), quarter = (turns + (1u << 29)) >> 30;
    float s0, c0;
    sincospif((float)(int)(turns - (quarter << 30)) * 0x1p-31f, &s0, &c0);
    float s = __uint_as_float(__float_as_uint(quarter & 1 ? c0 : s0) ^ (quarter & 2) << 30);
    float c = __uint_as_float(__float_as_uint(quarter & 1 ? s0 : c0) ^ (quarter + 1 & 2) << 30);
    if (!turn.finite) s = c = __int_as_float(0x7fc00000);
    return make_float2(c, p.inverse ? -s : s);
}

// A block's units: token x head (of q's heads, then k's, the block's share of them) x unit of the head.
// Units 0 .. pair_units - 1 of a head turn pairs, the rest copy channels that are not rotated.
struct RotaryPlan {
    int tokens;              // tokens per block
    int heads, share;        // heads of q and k together; per block
    int pair_units, units;   // per head
    int groups;              // of threads that fill the table: a thread has one pair and every groups-th token
    uint32_t over_units, over_share;   // 2^32 / units and 2^32 / (share units), rounded up
};
constexpr int kMostUnits = 8192;     // of a block: products of a unit and a divisor stay below 2^32

// i / n for i, n <= kMostUnits, from m = 2^32 / n rounded up (0 for n = 1).
__device__ __forceinline__ int over(int i, uint32_t m) { return m ? (int)__umulhi((uint32_t)i, m) : i; }

template <typename T, int N, bool Interleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p,
                                                                const __grid_constant__ RotaryPlan plan) {
    // [tokens][P]; where pairs are halves [tokens][N][P / N]: the k-th pairs of all units lie together, so
    // that neighbouring lanes, which turn neighbouring units, read neighbouring words (82 us instead of 86
    // for q and k of 65536 x 16 x 64 in bf16; interleaved pairs, half as many a unit, lose 5 us that way)
    extern __shared__ float2 cs[];
    using V = Vec<T, N>;
    constexpr bool kOne = Interleaved && N > 1;   // whole pairs in one vector
    constexpr int kPairs = kOne ? N / 2 : N;
    const int64_t t0 = (int64_t)blockIdx.x * plan.tokens;
    const int h0 = blockIdx.y * plan.share;
    const int tokens = (int)min64(plan.tokens, p.T - t0), per_token = plan.share * plan.units;
    const int total = tokens * per_token, second = Interleaved ? 1 : p.P, apart = kOne ? 1 : p.P / kPairs;

    for (int first = threadIdx.x; first - (int)threadIdx.x < total; first += kUnits * kRotaryThreads) {
        V a[kUnits], b[kUnits];
        T* out[kUnits];
        int pair[kUnits];                // the unit's first place in the table, or -1: copied; -2: nothing
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int i = first + u * kRotaryThreads;
            pair[u] = -2;
            if (i >= total) continue;
            const int t = over(i, plan.over_share), r = i - t * per_token, hh = over(r, plan.over_units);
            const int e = r - hh * plan.units, h = h0 + hh;
            if (h >= plan.heads) continue;
            const bool is_k = h >= p.H, turned = e < plan.pair_units;
            const int64_t at = ((t0 + t) * p.H + (is_k ? h - p.H : h)) * p.d +
                               (turned ? (Interleaved ? 2 : 1) * e * kPairs : 2 * p.P + (e - plan.pair_units) * N);
            const T* x = static_cast<const T*>(is_k ? p.k : p.q) + at;
            out[u] = static_cast<T*>(is_k ? p.k_out : p.q_out) + at;
            a[u] = *reinterpret_cast<const V*>(x);
            if (turned && !kOne) b[u] = *reinterpret_cast<const V*>(x + second);
            pair[u] = turned ? t * p.P + e * (kOne ? kPairs : 1) : -1;
        }
        if (first == (int)threadIdx.x) {
            // the tokens' cos and sin, while the first loads are on their way
            for (int i = threadIdx.x; i < plan.groups * p.P; i += kRotaryThreads) {
                const int g = i / p.P, j = i - g * p.P, at = kOne ? j : j % kPairs * apart + j / kPairs;
                const Turn turn = turn_of(p, j);
                for (int t = g; t < tokens; t += plan.groups) cs[t * p.P + at] = cos_sin(p, turn, t0 + t);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (pair[u] == -2) continue;
            if (pair[u] >= 0) {
                float fa[N], fb[N];
                unpack(fa, a[u]);
                if (!kOne) unpack(fb, b[u]);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const float2 w = cs[pair[u] + k * apart];
                    float& x0 = fa[kOne ? 2 * k : k];
                    float& x1 = kOne ? fa[kOne ? 2 * k + 1 : 0] : fb[k];
                    const float f0 = x0, f1 = x1;
                    // written out, so that every layout rounds alike
                    x0 = fmaf(f0, w.x, -__fmul_rn(f1, w.y));
                    x1 = fmaf(f1, w.x, __fmul_rn(f0, w.y));
                }
                pack(a[u], fa);
                if (!kOne) {
                    pack(b[u], fb);
                    *reinterpret_cast<V*>(out[u] + second) = b[u];
                }
            }
            *reinterpret_cast<V*>(out[u]) = a[u];
        }
    }
}

// Rows that units do not divide: a block copies its tokens' rows of q and k, which lie together and start on 16
// bytes, to shared memory, turns the pairs there, wherever they lie, and writes the rows back as they came.
struct StagedPlan {
    int tokens;                        // per block: a whole number of vectors
    int groups;                        // as in RotaryPlan
    uint32_t over_pairs, over_heads;   // 2^32 / P and 2^32 / H, rounded up
};
constexpr int kStagedBytes = 24 * 1024;   // of rows of q and k that a block aims at
constexpr int kMostStaged = 40 * 1024;    // with the table

template <typename T, bool Interleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotary_staged_kernel(const __grid_constant__ RotaryParams p,
                                                                       const __grid_constant__ StagedPlan plan) {
    extern __shared__ uint4 rows[];             // [q, k][tokens H d], then cos and sin [tokens][P]
    constexpr int N = 16 / sizeof(T);
    const int64_t t0 = (int64_t)blockIdx.x * plan.tokens, at = t0 * p.H * p.d;
    const int tokens = (int)min64(plan.tokens, p.T - t0), row = p.H * p.d;
    const int arrays = p.k ? 2 : 1, n = tokens * row, place = plan.tokens * row;
    T* held = reinterpret_cast<T*>(rows);
    float2* cs = reinterpret_cast<float2*>(held + arrays * place);
    for (int a = 0; a < arrays; ++a) {
        const T* x = static_cast<const T*>(a ? p.k : p.q) + at;
        for (int i = threadIdx.x * N; i < n; i += kRotaryThreads * N) {
            if (i + N <= n) {
                copy_16(held + a * place + i, x + i);
            } else {
                for (int j = i; j < n; ++j) held[a * place + j] = x[j];
            }
        }
    }
    copies_done();
    for (int i = threadIdx.x; i < plan.groups * p.P; i += kRotaryThreads) {
        const int g = over(i, plan.over_pairs), j = i - g * p.P;
        const Turn turn = turn_of(p, j);
        for (int t = g; t < tokens; t += plan.groups) cs[t * p.P + j] = cos_sin(p, turn, t0 + t);
    }
    wait_copies<0>();
    __syncthreads();
    const int heads = tokens * p.H;
    for (int a = 0; a < arrays; ++a)
        for (int i = threadIdx.x; i < heads * p.P; i += kRotaryThreads) {
            const int r = over(i, plan.over_pairs), j = i - r * p.P;
            T* x = held + a * place + r * p.d + (Interleaved ? 2 * j : j);
            T* y = x + (Interleaved ? 1 : p.P);
            const float2 w = cs[over(r, plan.over_heads) * p.P + j];
            const float f0 = (float)*x, f1 = (float)*y;
            *x = T(fmaf(f0, w.x, -__fmul_rn(f1, w.y)));
            *y = T(fmaf(f1, w.x, __fmul_rn(f0, w.y)));
        }
    __syncthreads();
    for (int a = 0; a < arrays; ++a) {
        T* x = static_cast<T*>(a ? p.k_out : p.q_out) + at;
        for (int i = threadIdx.x * N; i < n; i += kRotaryThreads * N) {
            if (i + N <= n) {
                *reinterpret_cast<uint4*>(x + i) = *reinterpret_cast<const uint4*>(held + a * place + i);
            } else {
                for (int j = i; j < n; ++j) x[j] = held[a * place + j];
            }
        }
    }
}

int groups_of(int pairs) { return pairs < kRotaryThreads ? kRotaryThreads / pairs : 1; }
uint32_t reciprocal(int n) { return n > 1 ? (uint32_t)(0xffffffffu / (uint32_t)n) + 1 : 0; }

template <typename T, int N>
cudaError_t run(const RotaryParams& p, int sms, cudaStream_t s) {
    RotaryPlan plan{};
    plan.heads = p.k ? 2 * p.H : p.H;
    plan.pair_units = p.interleaved && N > 1 ? 2 * p.P / N : p.P / N;
    plan.units = plan.pair_units + (p.d - 2 * p.P) / N;
    plan.share = (int)min64(plan.heads, kMostUnits / 2 / plan.units);
    plan.share = (int)ceil_div(plan.heads, ceil_div(plan.heads, plan.share));
    // enough tokens that every thread has kUnits units, but no fewer blocks than SMs for it, and no more
    // than a table of 32 KB holds
    const int64_t per_token = (int64_t)plan.share * plan.units, rest = ceil_div(plan.heads, plan.share);
    int64_t tokens = ceil_div((int64_t)kUnits * kRotaryThreads, per_token);
    tokens = min64(tokens, 32 * 1024 / ((int64_t)sizeof(float2) * p.P));
    tokens = min64(tokens, p.T * rest / sms);
    if (tokens < 1) tokens = 1;
    plan.tokens = (int)tokens;
    plan.groups = groups_of(p.P);
    plan.over_units = reciprocal(plan.units);
    plan.over_share = reciprocal((int)per_token);
    const size_t smem = sizeof(float2) * (size_t)tokens * p.P;
    const dim3 blocks((unsigned)ceil_div(p.T, tokens), (unsigned)rest);
    if (p.interleaved) rotary_kernel<T, N, true><<<blocks, kRotaryThreads, smem, s>>>(p, plan);
    else rotary_kernel<T, N, false><<<blocks, kRotaryThreads, smem, s>>>(p, plan);
    return cudaGetLastError();
}

// Tokens per block of the staged form: as many as kStagedBytes hold, but no fewer blocks than SMs for it; 0 where
// not even the fewest whose rows are whole vectors fit.
template <typename T>
int64_t staged_tokens(const RotaryParams& p, int sms) {
    constexpr int N = 16 / sizeof(T);
    const int64_t row = (int64_t)p.H * p.d, arrays = p.k ? 2 : 1;
    int64_t step = 1;
    while (step * row % N) step *= 2;
    const int64_t bytes = arrays * row * (int64_t)sizeof(T), table = (int64_t)sizeof(float2) * p.P;
    if (step * (bytes + table) > kMostStaged) return 0;
    int64_t tokens = min64(min64(kStagedBytes / bytes, kMostStaged / (bytes + table)), p.T / sms);
    tokens = tokens / step * step;
    return tokens > step ? tokens : step;
}
template <typename T>
cudaError_t run_staged(const RotaryParams& p, int64_t tokens, cudaStream_t s) {
    const StagedPlan plan{(int)tokens, groups_of(p.P), reciprocal(p.P), reciprocal(p.H)};
    const size_t smem = (size_t)tokens * ((p.k ? 2 : 1) * sizeof(T) * p.H * p.d + sizeof(float2) * p.P);
    const unsigned blocks = (unsigned)ceil_div(p.T, tokens);
    if (p.interleaved) rotary_staged_kernel<T, true><<<blocks, kRotaryThreads, smem, s>>>(p, plan);
    else rotary_staged_kernel<T, false><<<blocks, kRotaryThreads, smem, s>>>(p, plan);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const RotaryParams& p, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // every unit starts on 16 bytes: the pointers, the rows, and where the second half and the tail begin
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                         reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_out);
    if (at % 16 == 0 && p.d % N == 0 && (p.interleaved ? 2 : 1) * p.P % N == 0) return run<T, N>(p, sms, s);
    // (32768 x 9 x 77 in bf16: 43 us, pair by pair 92; 32768 x 8 x 128 with 43 pairs 51 and 168; 4099 x 7 x 83 in
    // fp32 12.5 and 14.6)
    const int64_t tokens = at % 16 == 0 ? staged_tokens<T>(p, sms) : 0;
    return tokens > 0 ? run_staged<T>(p, tokens, s) : run<T, 1>(p, sms, s);
}

}  // namespace

cudaError_t rotary(const RotaryParams& p, int dtype, cudaStream_t s) {
    return dtype == LA_F32 ? dispatch<float>(p, s) : dispatch<__nv_bfloat16>(p, s);
}

}  // namespace la
