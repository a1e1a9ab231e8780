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
#include "ops/chain.cuh"
#include "ops/ops.h"
#include "ops/turn.cuh"
#include "ops/vec.cuh"

namespace la {

namespace {

constexpr int kQkThreads = 256;       // the most a block has
constexpr int kJoinColumns = 32, kJoinRows = 32;

struct QkPlan {
    int log_G;               // lanes of a row
    int heads, share;        // heads of q and k together; of a block
    int tokens;              // token places of a block: groups of its heads that run side by side
    int tile;                // tokens whose cos and sin are held together
    int blocks;              // along the tokens
    int pair_units, units;   // of a head
};

// Forward, rows that a lane's vectors of 16 bytes hold are copied to shared memory ahead of their use, by the lane that
// uses them: two blocks of 256 threads per SM, with 100 registers a thread (65536 x 32 x 64 in bf16 98 us; four of 64, which
// take a quarter more instructions, 106).  The backward pass has twice the rows on their way and more registers to keep,
// and is faster with three blocks and loads to registers (32768 x 16 x 64: 48 us and 65).
constexpr int kRing = 4;              // rows on their way, a power of two
// Positions that a thread of the table's has on their way together: 16384 x 20 x 128 in bf16 take 36 us with four (45 with
// one, and each token's table made by two blocks); the backward pass has no registers for them (32768 x 16 x 64: 55 us with
// one, 60 with four).
template <bool Backward>
constexpr int kPositionsAhead = Backward ? 1 : 4;
template <typename T, int N, int KU, bool Backward>
constexpr bool copied = !Backward && N > 1 && KU == 1 && sizeof(T) * N == 16;

// Where pair j's cos lies in a token's part of the table, in floats, and how far behind it its sin.  Halves in vectors:
// [N / 2][P / N] of (cos, cos, sin, sin) of two neighbouring pairs, so that neighbouring lanes, which have neighbouring
// units, read neighbouring 16 bytes, two pairs in each half of a register pair; otherwise [P] of (cos, sin).
template <int N, bool Interleaved>
__device__ __forceinline__ int table_place(int j, int apart) {
    if constexpr (N > 1 && !Interleaved) return ((j % N / 2) * apart + j / N) * 4 + (j & 1);
    else return 2 * j;
}
template <int N, bool Interleaved>
constexpr int kSinBehind = N > 1 && !Interleaved ? 2 : 1;

// Turns a unit's pairs, two to an instruction: a[0] and a[1] hold the first and second channels of N pairs, or, whole
// pairs in one vector, a[0] N / 2 pairs.  `cs`: the unit's first place in its token's table.
template <int N, bool Interleaved, int Sides>
__device__ __forceinline__ void turn_unit(typename Pairs<N>::P (&a)[Sides][Pairs<N>::n], const float* cs, int apart) {
    if constexpr (N == 1) {
        const float c = cs[0], s = cs[1], f0 = a[0][0], f1 = a[1][0];
        a[0][0] = fmaf(f0, c, -__fmul_rn(f1, s));
        a[1][0] = fmaf(f1, c, __fmul_rn(f0, s));
    } else if constexpr (Interleaved) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const float2 w = *reinterpret_cast<const float2*>(cs + 2 * k);
            const float f0 = tc::f32x2_lo(a[0][k]), f1 = tc::f32x2_hi(a[0][k]);
            a[0][k] = tc::f32x2_of(__float_as_uint(fmaf(f0, w.x, -__fmul_rn(f1, w.y))),
                                   __float_as_uint(fmaf(f1, w.x, __fmul_rn(f0, w.y))));
        }
    } else {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(cs + 4 * k * apart);
            const uint64_t f0 = a[0][k], f1 = a[1][k];
            a[0][k] = pfma(f0, (uint64_t)w.x, pmul(pmul(f1, psplat<uint64_t>(-1.f)), (uint64_t)w.y));
            a[1][k] = pfma(f1, (uint64_t)w.x, pmul(f0, (uint64_t)w.y));
        }
    }
}

// Full: every lane of a group has KU units, and all turn.
template <typename T, int N, bool Interleaved, int KU, bool Backward, bool Full>
__global__ void __launch_bounds__(kQkThreads, KU > 1 && KU * N > 4 ? 1 : Backward ? 3 : 2)
    qk_norm_rotary_kernel(const __grid_constant__ QkNormParams p, const __grid_constant__ QkPlan plan) {
    // two tables [tile][2 P], a tile's and the next one's; behind them the rows on their way, 16 bytes of each vector a lane
    extern __shared__ __align__(16) float table[];
    if (Backward) chain_go();
    using V = Vec<T, N>;
    using R = Pairs<N>;
    using P = typename R::P;
    constexpr bool kOne = Interleaved && N > 1;   // whole pairs in one vector
    constexpr int kPairs = kOne ? N / 2 : N, kSides = kOne ? 1 : 2;
    constexpr bool kCopied = copied<T, N, KU, Backward>;
    const int apart = kOne ? 1 : p.P / kPairs, second = Interleaved ? 1 : p.P;
    const int G = 1 << plan.log_G, lane = threadIdx.x & (G - 1), group = threadIdx.x >> plan.log_G;
    const int hh = group % plan.share, place = group / plan.share, h0 = blockIdx.y * plan.share;
    const bool mine = place < plan.tokens && h0 + hh < plan.heads;
    const int k = mine && h0 + hh >= p.H[0], h = h0 + hh - (k ? p.H[0] : 0);
    const float over_d = 1.f / (float)p.d;
    int at[KU];                       // a unit's first channel, or -1
    bool turned[KU];
    P w[KU][kSides][R::n];
    P sum[Backward ? KU : 1][kSides][R::n];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
        const int e = lane + u * G;
        turned[u] = Full || e < plan.pair_units;
        at[u] = !Full && e >= plan.units ? -1
                : turned[u]              ? (Interleaved ? 2 : 1) * e * kPairs
                                         : 2 * p.P + (e - plan.pair_units) * N;
#pragma unroll
        for (int s = 0; s < kSides; ++s) {
            Vec<float, N> v;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool on = mine && (Full || (at[u] >= 0 && (s == 0 || turned[u])));
                v.v[j] = on && p.w[k] ? p.w[k][(p.per_head ? (int64_t)h * p.d : 0) + at[u] + s * second + j] : 1.f;
            }
            unpack_pairs<N>(w[u][s], v);
#pragma unroll
            for (int j = 0; j < R::n; ++j)
                if (Backward) sum[u][s][j] = psplat<P>(0.f);
        }
    }
    const T* const x0 = static_cast<const T*>(p.x[k]) + (int64_t)h * p.d;
    const T* const d0 = static_cast<const T*>(p.dy[k]) + (int64_t)h * p.d;
    T* const y0 = static_cast<T*>(p.y[k]) + (int64_t)h * p.d;
    const int64_t row = (int64_t)p.H[k] * p.d, stride = p.stride[k];
    float* const rstds = p.rstd[k];
    const int heads_of = p.H[k];
    uint4* const ring = reinterpret_cast<uint4*>(table + 4 * (int64_t)plan.tile * p.P) + threadIdx.x;
    constexpr int kVectors = KU * kSides;      // of a row and lane
    // the block's tiles are gridDim.x apart, so that all blocks together work on neighbouring tokens; a row of this group
    // is token `place` of each `tokens` of them
    const int64_t apart_tiles = (int64_t)gridDim.x * plan.tile;
    struct Row {
        int64_t t0;                   // of its tile
        int in;                       // its first place in the tile
    };
    auto advance = [&](Row& r) {
        r.in += plan.tokens;
        if (r.in >= plan.tile) {
            r.in = 0;
            r.t0 += apart_tiles;
        }
    };
    // a lane copies what it will use itself, kRing - 1 rows ahead
    Row ahead{(int64_t)blockIdx.x * plan.tile, 0};
    int slot = 0;
    auto fetch = [&]() {
        const int64_t t = ahead.t0 + ahead.in + place;
        if (mine && t < p.T) {
            uint4* const to = ring + slot * kVectors * blockDim.x;
#pragma unroll
            for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int s = 0; s < kSides; ++s) {
                    if (!Full && (at[u] < 0 || (s > 0 && !turned[u]))) continue;
                    copy_16(to + (u * kSides + s) * blockDim.x, x0 + t * stride + at[u] + s * second);
                }
        }
        copies_done();
        advance(ahead);
        slot = (slot + 1) & (kRing - 1);
    };
    if (kCopied) {
        for (int q = 0; q < kRing - 1; ++q) fetch();
    }
    Row now{(int64_t)blockIdx.x * plan.tile, 0};
    float next = 0.f;                 // backward: rstd of the next row
    if (Backward && mine && now.t0 + place < p.T) next = rstds[(now.t0 + place) * heads_of + h];
    int which = 1;                    // of the tables
    for (; now.t0 < p.T; advance(now)) {
        const int64_t t = now.t0 + now.in + place;
        const bool on = mine && t < p.T;
        V x[KU][kSides], dy[Backward ? KU : 1][kSides];
        const float held = next;
        if (kCopied) {
            fetch();
        } else {
#pragma unroll
            for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int s = 0; s < kSides; ++s) {
                    const bool in = Full ? on : on && at[u] >= 0 && (s == 0 || turned[u]);
                    x[u][s] = in ? *reinterpret_cast<const V*>(x0 + t * stride + at[u] + s * second) : V{};
                    if (Backward) dy[u][s] = in ? *reinterpret_cast<const V*>(d0 + t * row + at[u] + s * second) : V{};
                }
        }
        if (Backward) {
            Row after = now;
            advance(after);
            const int64_t ta = after.t0 + after.in + place;
            next = mine && ta < p.T ? rstds[ta * heads_of + h] : 0.f;
        }
        if (now.in == 0) {
            // the next tile's cos and sin (whoever still works on the one before has the other table)
            which ^= 1;
            const int n = (int)min64(plan.tile, p.T - now.t0), groups = max(1, (int)blockDim.x / p.P);
            float* const fill = table + which * 2 * plan.tile * p.P;
            for (int i = threadIdx.x; i < groups * p.P; i += blockDim.x) {
                const int g = i / p.P, j = i - g * p.P, to = table_place<N, Interleaved>(j, apart);
                const Turn turn = turn_of(p, j);
                constexpr int kAhead = kPositionsAhead<Backward>;
                for (int e0 = g; e0 < n; e0 += kAhead * groups) {
                    int position[kAhead];
#pragma unroll
                    for (int q = 0; q < kAhead; ++q)
                        position[q] = e0 + q * groups < n ? position_of(p, turn, now.t0 + e0 + q * groups) : 0;
#pragma unroll
                    for (int q = 0; q < kAhead; ++q) {
                        const int e = e0 + q * groups;
                        if (e >= n) break;
                        const float2 cw = cos_sin_at(p, turn, position[q]);
                        fill[2 * e * p.P + to] = cw.x;
                        fill[2 * e * p.P + to + kSinBehind<N, Interleaved>] = cw.y;
                    }
                }
            }
            __syncthreads();
        }
        if (kCopied) {
            wait_copies<kRing - 1>();
            const uint4* const from = ring + slot * kVectors * blockDim.x;      // (the slot after the newest is the oldest)
#pragma unroll
            for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int s = 0; s < kSides; ++s) {
                    const bool in = Full ? on : on && at[u] >= 0 && (s == 0 || turned[u]);
                    x[u][s] = in ? *reinterpret_cast<const V*>(from + (u * kSides + s) * blockDim.x) : V{};
                }
        }
        const float* const cs = table + 2 * (which * plan.tile + now.in + place) * p.P;
        P f[KU][kSides][R::n], v[Backward ? KU : 1][kSides][R::n];
        float rstd;
        P part = psplat<P>(0.f);
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
            for (int s = 0; s < kSides; ++s) {
                unpack_pairs<N>(f[u][s], x[u][s]);
                if (Backward) unpack_pairs<N>(v[Backward ? u : 0][s], dy[Backward ? u : 0][s]);
                if (!Backward) {
#pragma unroll
                    for (int j = 0; j < R::n; ++j) part = pfma(f[u][s][j], f[u][s][j], part);
                }
            }
        if (!Backward) {
            float square = psum(part);
            for (int o = G >> 1; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
            rstd = rsqrtf(fmaf(square, over_d, p.eps));
            if (on && lane == 0 && rstds) rstds[t * heads_of + h] = rstd;
        } else {
            rstd = held;
        }
        const P scale = psplat<P>(rstd);
        // forward: x becomes u and is turned; backward: dy is turned back
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            auto& a = Backward ? v[Backward ? u : 0] : f[u];
#pragma unroll
            for (int s = 0; s < kSides; ++s)
#pragma unroll
                for (int j = 0; j < R::n; ++j) {
                    // (the weight last: x w may leave fp32 where x rstd w does not, as in a row whose rstd is 0)
                    f[u][s][j] = pmul(f[u][s][j], scale);
                    if (!Backward) f[u][s][j] = pmul(f[u][s][j], w[u][s][j]);
                }
            if (Full ? on : turned[u] && on && at[u] >= 0) {
                const int e = lane + u * G;
                turn_unit<N, Interleaved>(a, cs + (N > 1 && !Interleaved ? 4 * e : 2 * e * kPairs), apart);
            }
            if (Backward) {
#pragma unroll
                for (int s = 0; s < kSides; ++s)
#pragma unroll
                    for (int j = 0; j < R::n; ++j) {
                        sum[Backward ? u : 0][s][j] = pfma(a[s][j], f[u][s][j], sum[Backward ? u : 0][s][j]);
                        a[s][j] = pmul(a[s][j], w[u][s][j]);
                        part = pfma(a[s][j], f[u][s][j], part);
                    }
            }
        }
        P less = psplat<P>(0.f);
        if (Backward) {
            float dot = psum(part);
            for (int o = G >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            less = psplat<P>(-dot * over_d);
        }
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
            for (int s = 0; s < kSides; ++s) {
                if (Full ? !on : !on || at[u] < 0 || (s > 0 && !turned[u])) continue;
                if (Backward) {
#pragma unroll
                    for (int j = 0; j < R::n; ++j)
                        f[u][s][j] = pmul(scale, pfma(f[u][s][j], less, v[Backward ? u : 0][s][j]));
                }
                V o;
                pack_pairs<N>(o, f[u][s]);
                *reinterpret_cast<V*>(y0 + t * row + at[u] + s * second) = o;
            }
    }
    if (!Backward || !p.partial) return;
    // the block's sums for the weights' gradients: over its token places, and heads that share a weight, in order
    __syncthreads();
    float* const red = table;                        // [place][head][d]
#pragma unroll
    for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int s = 0; s < kSides; ++s) {
            if (!mine || (!Full && (at[u] < 0 || (s > 0 && !turned[u])))) continue;
            Vec<float, N> v;
            pack_pairs<N>(v, sum[Backward ? u : 0][s]);
#pragma unroll
            for (int j = 0; j < N; ++j) red[(place * plan.share + hh) * p.d + at[u] + s * second + j] = v.v[j];
        }
    __syncthreads();
    const int heads = min(plan.share, plan.heads - h0);
    if (p.per_head) {
        for (int i = threadIdx.x; i < heads * p.d; i += blockDim.x) {
            float v = 0.f;
            for (int t = 0; t < plan.tokens; ++t) v += red[t * plan.share * p.d + i];
            p.partial[((int64_t)blockIdx.x * plan.heads + h0) * p.d + i] = v;
        }
    } else {
        const int mid = min(max(p.H[0] - h0, 0), heads);      // heads of q in this block
        for (int i = threadIdx.x; i < 2 * p.d; i += blockDim.x) {
            const int key = i >= p.d, c = i - key * p.d;
            float v = 0.f;
            for (int t = 0; t < plan.tokens; ++t)
                for (int e = key ? mid : 0; e < (key ? heads : mid); ++e) v += red[(t * plan.share + e) * p.d + c];
            p.partial[((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * 2 * p.d + i] = v;
        }
    }
}

// dw [rows][d] of q or k from the blocks' sums: of one head (per_head) or of all that share one.
__global__ void __launch_bounds__(kJoinColumns * kJoinRows) qk_join_kernel(const __grid_constant__ QkNormParams p,
                                                                           int sums) {
    __shared__ float part[kJoinRows][kJoinColumns];
    chain_wait();
    // (the blocks in one dimension: there may be more weight rows than a grid has in y)
    const int rows = p.per_head ? p.H[0] + p.H[1] : 2, across = (p.d + kJoinColumns - 1) / kJoinColumns;
    const int r = blockIdx.x / across, c = (blockIdx.x - r * across) * kJoinColumns + threadIdx.x;
    const int k = p.per_head ? r >= p.H[0] : r;
    float* const out = p.dw[k];
    // compensated: a thread's sum is as good as its terms
    float sum = 0.f, rest = 0.f;
    if (c < p.d) {
#pragma unroll 8
        for (int i = threadIdx.y; i < sums; i += kJoinRows) {
            const float y = __fsub_rn(p.partial[((int64_t)i * rows + r) * p.d + c], rest), t = __fadd_rn(sum, y);
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
        out[(p.per_head ? (int64_t)(r - (k ? p.H[0] : 0)) * p.d : 0) + c] = part[0][threadIdx.x];
}

constexpr int kTable = 8 * 1024;      // bytes of a tile's cos and sin that a block aims at

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

// Blocks along the tokens: no more than run at once (more where they are smaller, in the forward pass); what those of the
// backward pass sum is joined.
constexpr int kForwardBlocks = 2, kBackwardBlocks = 3;      // of kQkThreads threads, per SM
int64_t backward_blocks(int64_t T, int sms) { return min64(T, kBackwardBlocks * (int64_t)sms); }

QkPlan plan_of(const QkNormParams& p, int N, int sms, bool backward) {
    QkPlan plan{};
    plan.heads = p.H[0] + p.H[1];
    plan.pair_units = p.interleaved && N > 1 ? 2 * p.P / N : p.P / N;
    plan.units = plan.pair_units + (p.d - 2 * p.P) / N;
    while ((1 << plan.log_G) < plan.units && plan.log_G < 5) ++plan.log_G;
    // a token's heads over as many blocks as fill them best (each makes the table once), evenly
    const int64_t most = kQkThreads >> plan.log_G, fewest = ceil_div(plan.heads, most);
    const int64_t of_sm = backward ? most : kForwardBlocks * most;
    int64_t best = -1;
    for (int64_t parts = fewest; parts <= fewest + 3 && parts <= plan.heads; ++parts) {
        const int64_t share = ceil_div(plan.heads, parts), groups = most / share * share;
        const int64_t used = of_sm / groups * (most / share) * plan.heads * 100 / (parts * of_sm);
        if (used > best + 10) {
            best = used;
            plan.share = (int)share;
        }
    }
    plan.tokens = (int)(most / plan.share);
    const int64_t table = kTable / ((int64_t)sizeof(float2) * p.P);
    int64_t tile = min64(table, (int64_t)8 * plan.tokens) / plan.tokens * plan.tokens;
    if (tile < plan.tokens) tile = plan.tokens;
    // no more blocks than run at once, and no fewer than that for long tiles
    const int64_t most_blocks = backward ? backward_blocks(p.T, sms) : of_sm / (plan.tokens * plan.share) * (int64_t)sms;
    tile = min64(tile, ceil_div(ceil_div(p.T, most_blocks), plan.tokens) * plan.tokens);
    plan.blocks = (int)min64(most_blocks, ceil_div(p.T, tile));
    plan.tile = (int)tile;
    return plan;
}

template <typename T, int N, bool Interleaved, int KU, bool Backward, bool Full>
cudaError_t launch(const QkNormParams& p, const QkPlan& plan, Chain& chain, int64_t* sums) {
    const int threads = ((plan.share * plan.tokens << plan.log_G) + 31) / 32 * 32;
    size_t smem = 2 * sizeof(float2) * (size_t)plan.tile * p.P;
    if (copied<T, N, KU, Backward>) smem += (size_t)kRing * 16 * threads * KU * (Interleaved && N > 1 ? 1 : 2);
    if (Backward) {
        const size_t red = sizeof(float) * (size_t)plan.tokens * plan.share * p.d;
        if (red > smem) smem = red;
    }
    auto kernel = qk_norm_rotary_kernel<T, N, Interleaved, KU, Backward, Full>;
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_all_shared(kernel);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)plan.blocks, (unsigned)ceil_div(plan.heads, plan.share));
    if (sums) *sums = (int64_t)grid.x * (p.per_head ? 1 : grid.y);
    return launch_in(chain, kernel, grid, threads, smem, p, plan);
}

template <typename T, int N, bool Interleaved, bool Backward>
cudaError_t units(const QkNormParams& p, int sms, Chain& chain, int64_t* sums) {
    const QkPlan plan = plan_of(p, N, sms, Backward);
    const int64_t per = ceil_div(plan.units, 1 << plan.log_G);
    // up to 32 / N units a lane: rows of LA_MAX_ROTARY_D that turn few pairs
    static_assert(LA_MAX_ROTARY_D == 32 * 32, "a lane's units");
    constexpr int kSome = N == 1 ? 4 : 2;
    if (N == 1 && per == 2) return launch<T, N, Interleaved, N == 1 ? 2 : kSome, Backward, false>(p, plan, chain, sums);
    if (N > 1 && per <= 1 && plan.pair_units == 1 << plan.log_G && plan.units == plan.pair_units)
        return launch<T, N, Interleaved, 1, Backward, (N > 1)>(p, plan, chain, sums);
    if (per <= 1) return launch<T, N, Interleaved, 1, Backward, false>(p, plan, chain, sums);
    if (per <= kSome) return launch<T, N, Interleaved, kSome, Backward, false>(p, plan, chain, sums);
    return launch<T, N, Interleaved, 32 / N, Backward, false>(p, plan, chain, sums);
}

template <typename T, bool Backward>
cudaError_t dispatch(const QkNormParams& p, Chain& chain, int64_t* sums = nullptr) {   // sums: of the blocks, for each weight
    constexpr int N = 16 / sizeof(T);
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (whole_vectors(p, N, Backward))
        return p.interleaved ? units<T, N, true, Backward>(p, sms, chain, sums) : units<T, N, false, Backward>(p, sms, chain, sums);
    return p.interleaved ? units<T, 1, true, Backward>(p, sms, chain, sums) : units<T, 1, false, Backward>(p, sms, chain, sums);
}

}  // namespace

cudaError_t qk_norm_rotary(const QkNormParams& p, int dtype, cudaStream_t s) {
    Chain chain{s};
    return dtype == LA_F32 ? dispatch<float, false>(p, chain) : dispatch<__nv_bfloat16, false>(p, chain);
}

size_t qk_norm_rotary_backward_workspace_bytes(int64_t T, int H, int d) {
    const int sms = sm_count();
    if (sms <= 0) return 0;
    // (shared weights: two rows for each block, and no more blocks for a token than heads)
    return align_up(sizeof(float) * (size_t)(backward_blocks(T < 1 ? 1 : T, sms)) * 2 * H * d, kAlign);
}

cudaError_t qk_norm_rotary_backward(const QkNormParams& p, int dtype, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    cudaError_t e = cudaSuccess;
    int64_t sums = 0;
    Chain chain{s};
    if (p.T > 0) e = dtype == LA_F32 ? dispatch<float, true>(p, chain, &sums) : dispatch<__nv_bfloat16, true>(p, chain, &sums);
    if (e != cudaSuccess || !p.partial) return e;
    const int rows = p.per_head ? p.H[0] + p.H[1] : p.H[1] ? 2 : 1;
    return launch_in(chain, qk_join_kernel, (unsigned)(ceil_div(p.d, kJoinColumns) * rows), dim3(kJoinColumns, kJoinRows), 0, p,
                     (int)sums);
}

}  // namespace la
