// Norm of queries and keys with their rotation in one pass, and its gradients.  A row x of d channels (one head of
// one token) becomes
//
//     u = x rstd w,  rstd = 1 / sqrt(mean(x^2) + eps),  y = u with its pairs turned (rotary.cu),
//
// and, with du the rows of dy turned back and g = du w,
//
//     dx = rstd (g - xh mean(g xh)),  dw = sum over rows of du xh,  xh = x rstd.
//
// Bound by memory: a row is read and written once.  A row belongs to a group of 1 to 32 lanes, whose units of work
// are those of rotary.cu: N neighbouring channels and, where pairs are halves, their N partners, 16 bytes each where
// every row allows it, so that a pair is turned inside a lane.  A group keeps one head and walks tokens: its weights,
// and in the backward pass its sums for their gradients, stay in registers.  A block has some heads of some tokens, and
// their cos and sin once for all heads.
#include "ops/ops.h"
#include "ops/turn.cuh"
#include "ops/vec.cuh"

namespace la {

namespace {

constexpr int kQkThreads = 256;       // the most a block has
constexpr int kJoinColumns = 32, kJoinRows = 16;

struct QkPlan {
    int G;                   // lanes of a row
    int heads, share;        // heads of q and k together; of a block
    int tokens;              // token places of a block: groups of its heads that run side by side
    int tile;                // tokens whose cos and sin are held together
    int64_t span;            // tokens of a block
    int pair_units, units;   // of a head
};

template <typename T, int N, bool Interleaved, int KU, bool Backward>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rotary_kernel(const __grid_constant__ QkNormParams p,
                                                             const __grid_constant__ QkPlan plan) {
    extern __shared__ float2 cs[];    // as in rotary.cu: [tile][P], where pairs are halves [tile][N][P / N]
    using V = Vec<T, N>;
    constexpr bool kOne = Interleaved && N > 1;   // whole pairs in one vector
    constexpr int kPairs = kOne ? N / 2 : N, kSides = kOne ? 1 : 2;
    // rows whose loads are on their way together: up to 64 bytes a lane and array
    constexpr int kAhead = KU * kSides * (int)sizeof(V) >= 64 ? 1 : 64 / (KU * kSides * (int)sizeof(V)) > 4 ? 4 : 64 / (KU * kSides * (int)sizeof(V));
    const int apart = kOne ? 1 : p.P / kPairs, second = Interleaved ? 1 : p.P;
    const int lane = threadIdx.x % plan.G, group = threadIdx.x / plan.G;
    const int hh = group % plan.share, place = group / plan.share, h0 = blockIdx.y * plan.share;
    const bool mine = place < plan.tokens && h0 + hh < plan.heads;
    const int k = mine && h0 + hh >= p.H[0], h = h0 + hh - (k ? p.H[0] : 0);
    int at[KU];                       // a unit's first channel, or -1
    bool turned[KU];
    float w[KU][kSides][N];
    float sum[Backward ? KU : 1][kSides][N];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
        const int e = lane + u * plan.G;
        turned[u] = e < plan.pair_units;
        at[u] = !mine || e >= plan.units ? -1
                : turned[u]              ? (Interleaved ? 2 : 1) * e * kPairs
                                         : 2 * p.P + (e - plan.pair_units) * N;
#pragma unroll
        for (int i = 0; i < kSides; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool on = at[u] >= 0 && (i == 0 || turned[u]);
                w[u][i][j] = on && p.w[k] ? p.w[k][(p.per_head ? (int64_t)h * p.d : 0) + at[u] + i * second + j] : 1.f;
                if (Backward) sum[u][i][j] = 0.f;
            }
    }
    const int64_t first = blockIdx.x * plan.span, end = min64(first + plan.span, p.T);
    for (int64_t t0 = first; t0 < end; t0 += plan.tile) {
        const int n = (int)min64(plan.tile, end - t0);
        for (int b = 0; b < n; b += kAhead * plan.tokens) {
            V x[kAhead][KU][kSides], dy[Backward ? kAhead : 1][KU][kSides];
            bool on[kAhead];
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int i = b + r * plan.tokens + place;
                on[r] = mine && i < n;
                const int64_t row = (t0 + (on[r] ? i : 0)) * p.H[k] + h;
                const T* px = static_cast<const T*>(p.x[k]) + (t0 + (on[r] ? i : 0)) * p.stride[k] + (int64_t)h * p.d;
                const T* pd = static_cast<const T*>(p.dy[k]) + row * p.d;
#pragma unroll
                for (int u = 0; u < KU; ++u)
#pragma unroll
                    for (int s = 0; s < kSides; ++s) {
                        const bool in = on[r] && at[u] >= 0 && (s == 0 || turned[u]);
                        x[r][u][s] = in ? *reinterpret_cast<const V*>(px + at[u] + s * second) : V{};
                        if (Backward) dy[r][u][s] = in ? *reinterpret_cast<const V*>(pd + at[u] + s * second) : V{};
                    }
            }
            if (b == 0) {
                // the tile's cos and sin, while the first loads are on their way
                if (t0 != first) __syncthreads();
                const int groups = max(1, (int)blockDim.x / p.P);
                for (int i = threadIdx.x; i < groups * p.P; i += blockDim.x) {
                    const int g = i / p.P, j = i - g * p.P, to = kOne ? j : j % kPairs * apart + j / kPairs;
                    const Turn turn = turn_of(p, j);
                    for (int t = g; t < n; t += groups) cs[t * p.P + to] = cos_sin(p, turn, t0 + t);
                }
                __syncthreads();
            }
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int i = b + r * plan.tokens + place;
                const int64_t row = (t0 + (on[r] ? i : 0)) * p.H[k] + h;
                T* py = static_cast<T*>(p.y[k]) + row * p.d;
                float rstd, f[KU][kSides][N], v[Backward ? KU : 1][kSides][N];
                float square = 0.f;
#pragma unroll
                for (int u = 0; u < KU; ++u)
#pragma unroll
                    for (int s = 0; s < kSides; ++s) {
                        unpack(f[u][s], x[r][u][s]);
                        if (Backward) unpack(v[u][s], dy[r][u][s]);
                        if (!Backward) {
#pragma unroll
                            for (int j = 0; j < N; ++j) square = fmaf(f[u][s][j], f[u][s][j], square);
                        }
                    }
                if (!Backward) {
                    for (int o = plan.G / 2; o > 0; o /= 2) square += __shfl_xor_sync(0xffffffffu, square, o);
                    rstd = rsqrtf(square / (float)p.d + p.eps);
                    if (on[r] && lane == 0 && p.rstd[k]) p.rstd[k][row] = rstd;
                } else {
                    rstd = on[r] ? p.rstd[k][row] : 0.f;
                }
                // forward: x becomes u and is turned; backward: dy is turned back
                float dot = 0.f;
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    auto& a = Backward ? v[Backward ? u : 0] : f[u];
#pragma unroll
                    for (int s = 0; s < kSides; ++s)
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            f[u][s][j] *= rstd;
                            if (!Backward) f[u][s][j] *= w[u][s][j];
                        }
                    if (turned[u] && on[r] && at[u] >= 0) {
                        const float2* c = cs + i * p.P + (lane + u * plan.G) * (kOne ? kPairs : 1);
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) {
                            const float2 cw = c[j * apart];
                            float& x0 = a[0][kOne ? 2 * j : j];
                            float& x1 = kOne ? a[0][kOne ? 2 * j + 1 : 0] : a[kSides - 1][j];
                            const float f0 = x0, f1 = x1;
                            x0 = fmaf(f0, cw.x, -__fmul_rn(f1, cw.y));
                            x1 = fmaf(f1, cw.x, __fmul_rn(f0, cw.y));
                        }
                    }
                    if (Backward) {
#pragma unroll
                        for (int s = 0; s < kSides; ++s)
#pragma unroll
                            for (int j = 0; j < N; ++j) {
                                sum[Backward ? u : 0][s][j] = fmaf(a[s][j], f[u][s][j], sum[Backward ? u : 0][s][j]);
                                a[s][j] *= w[u][s][j];
                                dot = fmaf(a[s][j], f[u][s][j], dot);
                            }
                    }
                }
                if (Backward) {
                    for (int o = plan.G / 2; o > 0; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    dot /= (float)p.d;
                }
#pragma unroll
                for (int u = 0; u < KU; ++u)
#pragma unroll
                    for (int s = 0; s < kSides; ++s) {
                        if (!on[r] || at[u] < 0 || (s > 0 && !turned[u])) continue;
                        if (Backward) {
#pragma unroll
                            for (int j = 0; j < N; ++j)
                                f[u][s][j] = rstd * fmaf(-f[u][s][j], dot, v[Backward ? u : 0][s][j]);
                        }
                        V o;
                        pack(o, f[u][s]);
                        *reinterpret_cast<V*>(py + at[u] + s * second) = o;
                    }
            }
        }
    }
    if (!Backward || !p.partial) return;
    // the block's sums for the weights' gradients: over its token places, in order
    __syncthreads();
    float* red = reinterpret_cast<float*>(cs);       // [place][head][d]
#pragma unroll
    for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int s = 0; s < kSides; ++s) {
            if (at[u] < 0 || (s > 0 && !turned[u])) continue;
#pragma unroll
            for (int j = 0; j < N; ++j)
                red[(place * plan.share + hh) * p.d + at[u] + s * second + j] = sum[Backward ? u : 0][s][j];
        }
    __syncthreads();
    const int heads = min(plan.share, plan.heads - h0);
    for (int i = threadIdx.x; i < heads * p.d; i += blockDim.x) {
        float v = 0.f;
        for (int t = 0; t < plan.tokens; ++t) v += red[t * plan.share * p.d + i];
        p.partial[((int64_t)blockIdx.x * plan.heads + h0) * p.d + i] = v;
    }
}

// dw [rows][d] of q or k from the blocks' sums: of one head (per_head) or of all.
__global__ void __launch_bounds__(kJoinColumns * kJoinRows) qk_join_kernel(const __grid_constant__ QkNormParams p,
                                                                           int blocks) {
    __shared__ float part[kJoinRows][kJoinColumns];
    const int heads = p.H[0] + p.H[1], c = blockIdx.x * kJoinColumns + threadIdx.x;
    int k, h0, n;                     // heads h0 .. h0 + n - 1 of q and k together
    if (p.per_head) {
        h0 = blockIdx.y;
        n = 1;
        k = h0 >= p.H[0];
    } else {
        k = blockIdx.y;
        h0 = k ? p.H[0] : 0;
        n = p.H[k];
    }
    float* const out = p.dw[k];
    // compensated: a thread's sum is as good as its terms
    float sum = 0.f, rest = 0.f;
    if (c < p.d) {
        for (int64_t i = threadIdx.y; i < (int64_t)blocks * n; i += kJoinRows) {
            const int64_t b = i / n, h = h0 + i % n;
            const float y = __fsub_rn(p.partial[(b * heads + h) * p.d + c], rest), t = __fadd_rn(sum, y);
            rest = __fsub_rn(__fsub_rn(t, sum), y);
            sum = t;
        }
    }
    part[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    for (int o = kJoinRows / 2; o > 0; o /= 2) {
        if ((int)threadIdx.y < o) part[threadIdx.y][threadIdx.x] += part[threadIdx.y + o][threadIdx.x];
        __syncthreads();
    }
    if (threadIdx.y == 0 && c < p.d && out)
        out[(p.per_head ? (int64_t)(h0 - (k ? p.H[0] : 0)) * p.d : 0) + c] = part[0][threadIdx.x];
}

constexpr int kTable = 16 * 1024;     // bytes of cos and sin that a block aims at

// Vectors of 16 bytes: the arrays, the rows of every token and where second halves and tails begin.
bool whole_vectors(const QkNormParams& p, int N, bool backward) {
    uintptr_t at = 0;
    int64_t strides = 0;
    for (int k = 0; k < 2; ++k) {
        if (!p.x[k]) continue;
        at |= reinterpret_cast<uintptr_t>(p.x[k]) | reinterpret_cast<uintptr_t>(p.y[k]);
        if (backward) at |= reinterpret_cast<uintptr_t>(p.dy[k]);
        strides |= p.stride[k];
    }
    return at % 16 == 0 && strides % N == 0 && p.d % N == 0 && (p.interleaved ? 2 : 1) * p.P % N == 0;
}

// Blocks along the tokens of the backward pass: what they sum is joined, so no more than run at once.
int64_t backward_blocks(int64_t T, int sms) { return min64(T, 4 * (int64_t)sms); }

QkPlan plan_of(const QkNormParams& p, int N, int sms, bool backward) {
    QkPlan plan{};
    plan.heads = p.H[0] + p.H[1];
    plan.pair_units = p.interleaved && N > 1 ? 2 * p.P / N : p.P / N;
    plan.units = plan.pair_units + (p.d - 2 * p.P) / N;
    plan.G = 1;
    while (plan.G < plan.units && plan.G < 32) plan.G *= 2;
    // as few blocks for a token's heads as there can be, with the heads spread evenly over them
    const int64_t most = kQkThreads / plan.G, parts = ceil_div(plan.heads, most);
    plan.share = (int)ceil_div(plan.heads, parts);
    plan.tokens = (int)(most / plan.share);
    const int64_t table = kTable / ((int64_t)sizeof(float2) * p.P);
    int64_t tile = min64(table, 8 * plan.tokens) / plan.tokens * plan.tokens;
    if (tile < plan.tokens) tile = plan.tokens;
    if (backward) {
        plan.span = ceil_div(p.T, backward_blocks(p.T, sms));
    } else {
        // but no fewer blocks than SMs
        plan.span = min64(tile, ceil_div(p.T * ceil_div(plan.heads, plan.share), 2 * sms));
        if (plan.span < 1) plan.span = 1;
    }
    plan.tile = (int)min64(tile, plan.span);
    return plan;
}

template <typename T, int N, bool Interleaved, int KU, bool Backward>
cudaError_t launch(const QkNormParams& p, const QkPlan& plan, cudaStream_t s) {
    size_t smem = sizeof(float2) * (size_t)plan.tile * p.P;
    if (Backward) {
        const size_t red = sizeof(float) * (size_t)plan.tokens * plan.share * p.d;
        if (red > smem) smem = red;
    }
    auto kernel = qk_norm_rotary_kernel<T, N, Interleaved, KU, Backward>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)ceil_div(p.T, plan.span), (unsigned)ceil_div(plan.heads, plan.share));
    const int threads = (plan.G * plan.share * plan.tokens + 31) / 32 * 32;
    kernel<<<grid, threads, smem, s>>>(p, plan);
    return cudaGetLastError();
}

template <typename T, int N, bool Interleaved, bool Backward>
cudaError_t units(const QkNormParams& p, int sms, cudaStream_t s) {
    const QkPlan plan = plan_of(p, N, sms, Backward);
    const int64_t per = ceil_div(plan.units, plan.G);
    // up to 32 / N units a lane: rows of LA_MAX_ROTARY_D that turn few pairs
    static_assert(LA_MAX_ROTARY_D == 32 * 32, "a lane's units");
    constexpr int kSome = N == 1 ? 4 : 2;
    if (per <= 1) return launch<T, N, Interleaved, 1, Backward>(p, plan, s);
    if (per <= kSome) return launch<T, N, Interleaved, kSome, Backward>(p, plan, s);
    return launch<T, N, Interleaved, 32 / N, Backward>(p, plan, s);
}

template <typename T, bool Backward>
cudaError_t dispatch(const QkNormParams& p, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (whole_vectors(p, N, Backward))
        return p.interleaved ? units<T, N, true, Backward>(p, sms, s) : units<T, N, false, Backward>(p, sms, s);
    return p.interleaved ? units<T, 1, true, Backward>(p, sms, s) : units<T, 1, false, Backward>(p, sms, s);
}

}  // namespace

cudaError_t qk_norm_rotary(const QkNormParams& p, int dtype, cudaStream_t s) {
    return dtype == LA_F32 ? dispatch<float, false>(p, s) : dispatch<__nv_bfloat16, false>(p, s);
}

size_t qk_norm_rotary_backward_workspace_bytes(int64_t T, int H, int d) {
    const int sms = sm_count();
    if (sms <= 0) return 0;
    return align_up(sizeof(float) * (size_t)(backward_blocks(T < 1 ? 1 : T, sms)) * H * d, kAlign);
}

cudaError_t qk_norm_rotary_backward(const QkNormParams& p, int dtype, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    cudaError_t e = cudaSuccess;
    int64_t blocks = 0;
    if (p.T > 0) {
        e = dtype == LA_F32 ? dispatch<float, true>(p, s) : dispatch<__nv_bfloat16, true>(p, s);
        blocks = ceil_div(p.T, ceil_div(p.T, backward_blocks(p.T, sms)));
    }
    if (e != cudaSuccess || !p.partial) return e;
    const dim3 grid((unsigned)ceil_div(p.d, kJoinColumns), p.per_head ? p.H[0] + p.H[1] : p.H[1] ? 2 : 1);
    qk_join_kernel<<<grid, dim3(kJoinColumns, kJoinRows), 0, s>>>(p, (int)blocks);
    return cudaGetLastError();
}

}  // namespace la
