// Layer norm over rows of d values and its gradients.
//
// Bound by memory: the forward reads x and writes y once, the backward reads x
// and dy and writes dx once.  A row stays in the registers of the L lanes that
// share it (E vectors of N values each) between the sums over it and its
// output; the variance comes from the deviations in registers, not from sums of
// squares.  A group holds U rows at once so that their loads and sums overlap.
// In the forward a row shares a warp as far as its lanes can hold it (16 vectors
// each: sums without a barrier); in the backward, whose lanes also keep two fp32
// sums per column, rows of more than a kilobyte take a block.
//
// A group of lanes keeps one weight row: it walks over rows a multiple of
// `groups` apart.  Its weights are read once, and in the backward its columns'
// weight gradients add up in registers over all its rows.  Blocks leave their
// sums in the workspace as rows of a [M][groups * d] matrix that a second
// kernel adds up by column with compensated sums, in a fixed order.
#include "internal.h"
#include "vec.cuh"

namespace la {

namespace {

constexpr int kMaxBlocks = 608;     // backward: four blocks of 256 threads on each of 152 SMs
constexpr int kJoinCols = 32, kJoinRows = 32;

template <int L_, int E_, int N_>
struct Shape {
    static constexpr int L = L_, E = E_, N = N_;
    static constexpr int kThreads = L > 32 ? L : 256;
    static constexpr int kRows = kThreads / L;              // row groups of a block
    static constexpr int kValues = E * N;                   // values a lane holds of a row
};

// Sum over the L lanes of a row group, for each of U rows; every lane gets it.
template <typename S, int U>
__device__ __forceinline__ void row_sums(float (&x)[U], float* scratch) {
#pragma unroll
    for (int o = (S::L < 32 ? S::L : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], o);
    if constexpr (S::L > 32) {
        constexpr int kWarps = S::L / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();                                    // the scratch of the sums before is read
        if (lane == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) scratch[u * kWarps + warp] = x[u];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = lane < kWarps ? scratch[u * kWarps + lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x[u] += __shfl_xor_sync(0xffffffffu, x[u], o);
        }
    }
}

// The lane's E vectors of a row, which `row` points into at the lane's first column; vector e lies e L N
// columns on and is there when that is below `left`, the columns from the lane's first on.
template <typename S, typename T>
__device__ __forceinline__ void load_row(Vec<T, S::N> (&x)[S::E], const T* row, int left) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        constexpr int kStep = S::L * S::N;
        if (e * kStep < left) {
            x[e] = *reinterpret_cast<const Vec<T, S::N>*>(row + e * kStep);
        } else {
            const float zero[S::N] = {};
            pack(x[e], zero);
        }
    }
}

// N weights or biases from column c < d on; `missing` where there are none.  Vectors of columns come with
// 16-byte aligned parameters.
template <int N>
__device__ __forceinline__ void load_params(float* w, const float* p, int64_t at, float missing) {
    if (!p) {
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = missing;
    } else if constexpr (N >= 4) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + at + k);
            w[k] = v.x; w[k + 1] = v.y; w[k + 2] = v.z; w[k + 3] = v.w;
        }
    } else {
        w[0] = p[at];
    }
}
// The lane's parameters of a whole row, `p` at its first column.
template <typename S>
__device__ __forceinline__ void load_row_params(float (&w)[S::kValues], const float* p, int left, float missing) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        constexpr int kStep = S::L * S::N;
        load_params<S::N>(w + e * S::N, e * kStep < left ? p : nullptr, e * kStep, missing);
    }
}
__device__ __forceinline__ const float* row_of(const float* p, int64_t at) { return p ? p + at : nullptr; }

template <int V>
struct Count {
    static constexpr int value = V;
};

// 1 / sqrt(v), within one step: the approximate root and one step of Newton's method (0 and infinity
// keep the root's answer).
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    return v > 0.f && v < INFINITY ? fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r) : r;
}
// s / d: the product with 1 / d and what it leaves (equal values have their value as mean).
__device__ __forceinline__ float mean_of(float s, float d, float over_d) {
    const float m = s * over_d;
    return fmaf(fmaf(-m, d, s), over_d, m);
}

// The turns of a row group: rows first, first + stride, ..  `whole` turns of U rows that every group of
// the block has; the rest one row at a time, which some groups may not have.
struct Turns {
    int whole, rest, mine;       // turns of U; further turns of one; the group's rows
};
template <typename S, int U>
__device__ __forceinline__ Turns turns_of(int64_t rows, int64_t stride, int64_t first) {
    const int64_t block = (int64_t)blockIdx.x * S::kRows, last = block + S::kRows - 1;
    Turns t;
    t.mine = first < rows ? (int)((rows - 1 - first) / stride) + 1 : 0;
    const int most = block < rows ? (int)((rows - 1 - block) / stride) + 1 : 0;
    t.whole = last < rows ? ((int)((rows - 1 - last) / stride) + 1) / U : 0;
    t.rest = most - t.whole * U;
    return t;
}

// stride is a multiple of groups: every row of a row group has the same weight row.
template <typename T, typename S, int U>
__global__ void __launch_bounds__(S::kThreads, S::E == 1 && S::L <= 32 ? 4 : 1)
layer_norm_kernel(const T* x, const float* weight, const float* bias, int64_t rows, int groups, int d, float eps, T* y,
                  float* mean, float* rstd, int64_t stride) {
    __shared__ float scratch[S::L > 32 ? U * S::L / 32 : 1];
    const int lane = threadIdx.x % S::L, col = lane * S::N, left = d - col;
    const int64_t first = (int64_t)blockIdx.x * S::kRows + threadIdx.x / S::L, step = stride * d;
    const float fd = (float)d, over_d = 1.f / fd;
    // the group's weights stay where the registers allow it
    constexpr bool kHeld = S::kValues <= 8;
    float w[S::kValues], b[S::kValues];
    const int64_t at = first % groups * d + col;
    if (kHeld) {
        load_row_params<S>(w, row_of(weight, at), left, 1.f);
        load_row_params<S>(b, row_of(bias, at), left, 0.f);
    }
    const Turns turns = turns_of<S, U>(rows, stride, first);

    // V rows from `row` on, stride apart; `live`: there are any
    auto some_rows = [&](auto count, int64_t row, bool live) {
        constexpr int V = decltype(count)::value;
        Vec<T, S::N> v[V][S::E];
        float s[V], q[V];
        const T* at_x = x + row * d + col;
        T* at_y = y + row * d + col;
#pragma unroll
        for (int u = 0; u < V; ++u) load_row<S, T>(v[u], at_x + u * step, live ? left : 0);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                float f[S::N];
                unpack(f, v[u][e]);
#pragma unroll
                for (int k = 0; k < S::N; ++k) s[u] += f[k];
            }
        }
        row_sums<S, V>(s, scratch);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            s[u] = mean_of(s[u], fd, over_d);
            q[u] = 0.f;
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                if (e * S::L * S::N < left) {
                    float f[S::N];
                    unpack(f, v[u][e]);
#pragma unroll
                    for (int k = 0; k < S::N; ++k) q[u] = fmaf(f[k] - s[u], f[k] - s[u], q[u]);
                }
        }
        row_sums<S, V>(q, scratch);
        if (!live) return;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const float mu = s[u], rs = inverse_root(fmaf(q[u], over_d, eps));
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                constexpr int kStep = S::L * S::N;
                if (e * kStep >= left) continue;
                float f[S::N], we[S::N], be[S::N];
                unpack(f, v[u][e]);
                if (!kHeld) {
                    load_params<S::N>(we, weight, at + e * kStep, 1.f);
                    load_params<S::N>(be, bias, at + e * kStep, 0.f);
                }
#pragma unroll
                for (int k = 0; k < S::N; ++k)
                    f[k] = kHeld ? fmaf((f[k] - mu) * rs, w[e * S::N + k], b[e * S::N + k])
                                 : fmaf((f[k] - mu) * rs, we[k], be[k]);
                Vec<T, S::N> o;
                pack(o, f);
                *reinterpret_cast<Vec<T, S::N>*>(at_y + u * step + e * kStep) = o;
            }
            if (lane == 0) {
                if (mean) mean[row + u * stride] = mu;
                if (rstd) rstd[row + u * stride] = rs;
            }
        }
    };
    int64_t row = first;
    for (int turn = 0; turn < turns.whole; ++turn, row += U * stride) some_rows(Count<U>{}, row, true);
    for (int turn = 0; turn < turns.rest; ++turn, row += stride)
        some_rows(Count<1>{}, row, turns.whole * U + turn < turns.mine);
}

// part[slot][d]: the weight and bias gradients of one weight row over some rows, slot i of weight row
// i mod groups.  Row groups of a block that share a weight row are added up first where every one of
// its weight rows has equally many (kRows a multiple of groups).
template <typename T, typename S, int U>
__global__ void __launch_bounds__(S::kThreads) layer_norm_backward_kernel(const T* x, const T* dy, const float* weight,
                                                                          const float* mean, const float* rstd,
                                                                          int64_t rows, int groups, int d, T* dx,
                                                                          float2* part, int64_t stride) {
    __shared__ float scratch[S::L > 32 ? 2 * U * S::L / 32 : 1];
    extern __shared__ float2 sums[];                        // [kRows][d], L <= 32
    const int lane = threadIdx.x % S::L, group = threadIdx.x / S::L, col = lane * S::N, left = d - col;
    const int64_t first = (int64_t)blockIdx.x * S::kRows + group, step = stride * d;
    const float over_d = 1.f / d;
    constexpr bool kHeld = S::kValues <= 8;
    const int64_t at = first % groups * d + col;            // stride is a multiple of groups
    float w[S::kValues], dw[S::kValues], db[S::kValues];
    if (kHeld) load_row_params<S>(w, row_of(weight, at), left, 1.f);
#pragma unroll
    for (int k = 0; k < S::kValues; ++k) dw[k] = db[k] = 0.f;
    const Turns turns = turns_of<S, U>(rows, stride, first);

    auto some_rows = [&](auto count, int64_t row, bool live) {
        constexpr int V = decltype(count)::value;
        Vec<T, S::N> v[V][S::E], g[V][S::E];
        float mu[V], rs[V], sums_of[2 * V];                 // of w dy, and of w dy xh
        const int64_t at_row = row * d + col;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            load_row<S, T>(v[u], x + at_row + u * step, live ? left : 0);
            load_row<S, T>(g[u], dy + at_row + u * step, live ? left : 0);
            mu[u] = live ? mean[row + u * stride] : 0.f;
            rs[u] = live ? rstd[row + u * stride] : 0.f;
        }
        if (!kHeld) load_row_params<S>(w, row_of(weight, at), left, 1.f);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                if (live && e * S::L * S::N < left) {
                    float fx[S::N], fg[S::N];
                    unpack(fx, v[u][e]);
                    unpack(fg, g[u][e]);
#pragma unroll
                    for (int k = 0; k < S::N; ++k) {
                        const int i = e * S::N + k;
                        const float xh = (fx[k] - mu[u]) * rs[u], t = fg[k] * w[i];
                        s1 += t;
                        s2 = fmaf(t, xh, s2);
                        dw[i] = fmaf(fg[k], xh, dw[i]);
                        db[i] += fg[k];
                    }
                }
            sums_of[u] = s1;
            sums_of[V + u] = s2;
        }
        row_sums<S, 2 * V>(sums_of, scratch);
        if (!live) return;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const float m1 = sums_of[u] * over_d, m2 = sums_of[V + u] * over_d;
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                constexpr int kStep = S::L * S::N;
                if (e * kStep >= left) continue;
                float fx[S::N], fg[S::N];
                unpack(fx, v[u][e]);
                unpack(fg, g[u][e]);
#pragma unroll
                for (int k = 0; k < S::N; ++k) {
                    const float xh = (fx[k] - mu[u]) * rs[u];
                    fx[k] = rs[u] * (fmaf(fg[k], w[e * S::N + k], -m1) - xh * m2);
                }
                Vec<T, S::N> o;
                pack(o, fx);
                *reinterpret_cast<Vec<T, S::N>*>(dx + at_row + u * step + e * kStep) = o;
            }
        }
    };
    int64_t row = first;
    for (int turn = 0; turn < turns.whole; ++turn, row += U * stride) some_rows(Count<U>{}, row, true);
    for (int turn = 0; turn < turns.rest; ++turn, row += stride)
        some_rows(Count<1>{}, row, turns.whole * U + turn < turns.mine);
    asm volatile("griddepcontrol.launch_dependents;");
    if (!part) return;
    if (S::kRows > 1 && S::kRows % groups == 0) {
#pragma unroll
        for (int e = 0; e < S::E; ++e)
#pragma unroll
            for (int k = 0; k < S::N; ++k) {
                const int c = (e * S::L + lane) * S::N + k;
                if (c < d) sums[group * d + c] = make_float2(dw[e * S::N + k], db[e * S::N + k]);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < groups * d; i += S::kThreads) {
            float2 t = sums[i];
            for (int r = groups; r < S::kRows; r += groups) {
                const float2 q = sums[r * d + i];
                t.x += q.x;
                t.y += q.y;
            }
            part[(int64_t)blockIdx.x * groups * d + i] = t;
        }
    } else {
#pragma unroll
        for (int e = 0; e < S::E; ++e)
#pragma unroll
            for (int k = 0; k < S::N; ++k) {
                const int c = (e * S::L + lane) * S::N + k;
                if (c < d) part[first * d + c] = make_float2(dw[e * S::N + k], db[e * S::N + k]);
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
    __device__ __forceinline__ float value() const {
        const float t = s + c;
        return isfinite(s) ? t : s;     // infinities leave no error term
    }
};

// Column sums of part[M][n]: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(kJoinCols * kJoinRows) layer_norm_join_kernel(const float2* part, int64_t M, int64_t n,
                                                                                float* dweight, float* dbias) {
    __shared__ float4 sums[kJoinRows][kJoinCols];
    const int col = threadIdx.x % kJoinCols, r = threadIdx.x / kJoinCols;
    const int64_t j = (int64_t)blockIdx.x * kJoinCols + col;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Sum dw, db;
    if (j < n)
#pragma unroll 8
        for (int64_t m = r; m < M; m += kJoinRows) {
            const float2 v = part[m * n + j];
            dw.add(v.x);
            db.add(v.y);
        }
    for (int o = kJoinRows / 2; o > 0; o >>= 1) {
        if (r < 2 * o) sums[r][col] = make_float4(dw.s, dw.c, db.s, db.c);
        __syncthreads();
        if (r < o) {
            const float4 q = sums[r + o][col];
            dw.add(q.x);
            dw.c += q.y;
            db.add(q.z);
            db.c += q.w;
        }
        __syncthreads();
    }
    if (r == 0 && j < n) {
        if (dweight) dweight[j] = dw.value();
        if (dbias) dbias[j] = db.value();
    }
}

struct Args {
    const void *x, *dy;
    const float *weight, *bias, *mean_in, *rstd_in;
    int64_t rows;
    int groups, d;
    float eps;
    void* out;
    float *mean, *rstd;
    float2* part;
    cudaStream_t stream;
};

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Blocks of the backward: as many as there are rows for, at most kMaxBlocks (half as many of 512
// threads), rounded up so that a block's row groups meet the same weight rows on every turn.
template <typename S>
int64_t backward_blocks(int64_t rows, int groups) {
    const int64_t unit = groups / gcd(groups, S::kRows);
    int64_t blocks = min64(ceil_div(rows, S::kRows), S::kThreads > 256 ? kMaxBlocks / 2 : kMaxBlocks);
    return ceil_div(blocks > 0 ? blocks : 1, unit) * unit;
}
// Rows of the matrix of partial sums.
template <typename S>
int64_t backward_slots(int64_t rows, int groups) {
    const int64_t per_block = S::kRows > 1 && S::kRows % groups == 0 ? groups : S::kRows;
    return rows > 0 ? backward_blocks<S>(rows, groups) * per_block / groups : 0;
}

struct Forward {
    static constexpr bool kWide = true;      // rows of up to 16 vectors a lane share a warp
    template <typename T, typename S>
    static int64_t run(const Args& a) {
        constexpr int U = S::E == 1 && S::L <= 32 ? 4 : S::E <= 2 ? 2 : 1;
        // as many blocks as fill the SMs several times, more only where the grid limit asks for it
        int64_t blocks = ceil_div(a.rows, (int64_t)S::kRows * U);
        const int64_t most = 152 * 16 * 256 / S::kThreads, unit = a.groups / gcd(a.groups, S::kRows);
        if (blocks > most) blocks = most;
        blocks = ceil_div(blocks, unit) * unit;
        layer_norm_kernel<T, S, U><<<(unsigned)blocks, S::kThreads, 0, a.stream>>>(
            static_cast<const T*>(a.x), a.weight, a.bias, a.rows, a.groups, a.d, a.eps, static_cast<T*>(a.out), a.mean,
            a.rstd, blocks * S::kRows);
        return (int64_t)cudaGetLastError();
    }
};
struct Backward {
    static constexpr bool kWide = false;
    template <typename T, typename S>
    static int64_t run(const Args& a) {
        constexpr int U = S::kValues <= 8 ? 4 : S::kValues <= 16 && S::L <= 32 ? 2 : 1;
        const int64_t blocks = backward_blocks<S>(a.rows, a.groups);
        const bool reduce = a.part && S::kRows > 1 && S::kRows % a.groups == 0;
        const size_t smem = reduce ? sizeof(float2) * S::kRows * (size_t)a.d : 0;
        layer_norm_backward_kernel<T, S, U><<<(unsigned)blocks, S::kThreads, smem, a.stream>>>(
            static_cast<const T*>(a.x), static_cast<const T*>(a.dy), a.weight, a.mean_in, a.rstd_in, a.rows, a.groups,
            a.d, static_cast<T*>(a.out), a.part, blocks * S::kRows);
        return (int64_t)cudaGetLastError();
    }
};
struct Slots {
    static constexpr bool kWide = false;
    template <typename T, typename S>
    static int64_t run(const Args& a) { return backward_slots<S>(a.rows, a.groups); }
};

// The lanes and vectors of a row: the fewest lanes that hold it in one vector each up to a warp, then
// more vectors a lane or a block of 128 to 512 lanes.
template <typename Op, typename T>
int64_t by_shape(const Args& a, bool aligned) {
    constexpr int N = 16 / sizeof(T);
    const int d = a.d;
    if (aligned && d % N == 0) {
        const int n = d / N;
        if (n <= 4) return Op::template run<T, Shape<4, 1, N>>(a);
        if (n <= 8) return Op::template run<T, Shape<8, 1, N>>(a);
        if (n <= 16) return Op::template run<T, Shape<16, 1, N>>(a);
        if (n <= 32) return Op::template run<T, Shape<32, 1, N>>(a);
        if (n <= 64) return Op::template run<T, Shape<32, 2, N>>(a);
        if constexpr (Op::kWide) {
            if (n <= 128) return Op::template run<T, Shape<32, 4, N>>(a);
            if (n <= 192) return Op::template run<T, Shape<32, 6, N>>(a);
            if (n <= 256) return Op::template run<T, Shape<32, 8, N>>(a);
            if (n <= 512) return Op::template run<T, Shape<32, 16, N>>(a);
        }
        if (n <= 128) return Op::template run<T, Shape<128, 1, N>>(a);
        if (n <= 256) return Op::template run<T, Shape<256, 1, N>>(a);
        if (n <= 512) return Op::template run<T, Shape<512, 1, N>>(a);
        if (n <= 1024) return Op::template run<T, Shape<512, 2, N>>(a);
        if (n <= 2048) return Op::template run<T, Shape<512, 4, N>>(a);
        if constexpr (N == 4) return Op::template run<T, Shape<512, 8, N>>(a);
        return (int64_t)cudaErrorInvalidValue;      // d <= LA_MAX_NORM_D: not reached
    }
    if (d <= 32) return Op::template run<T, Shape<32, 1, 1>>(a);
    if (d <= 128) return Op::template run<T, Shape<32, 4, 1>>(a);
    if constexpr (Op::kWide) {
        if (d <= 512) return Op::template run<T, Shape<32, 16, 1>>(a);
        if (d <= 1024) return Op::template run<T, Shape<32, 32, 1>>(a);
    }
    if (d <= 512) return Op::template run<T, Shape<128, 4, 1>>(a);
    if (d <= 1024) return Op::template run<T, Shape<256, 4, 1>>(a);
    if (d <= 4096) return Op::template run<T, Shape<512, 8, 1>>(a);
    return Op::template run<T, Shape<512, 32, 1>>(a);
}
template <typename Op>
int64_t by_type(const Args& a, int dtype, bool aligned) {
    return dtype == LA_F32 ? by_shape<Op, float>(a, aligned) : by_shape<Op, __nv_bfloat16>(a, aligned);
}

bool on_16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int64_t slots_for(int dtype, int64_t rows, int groups, int d, bool aligned) {
    Args a{};
    a.rows = rows;
    a.groups = groups;
    a.d = d;
    return by_type<Slots>(a, dtype, aligned);
}

}  // namespace

cudaError_t layer_norm(const void* x, const float* weight, const float* bias, int dtype, int64_t rows, int groups,
                       int d, float eps, void* y, float* mean, float* rstd, cudaStream_t s) {
    Args a{};
    a.x = x; a.weight = weight; a.bias = bias;
    a.rows = rows; a.groups = groups; a.d = d; a.eps = eps;
    a.out = y; a.mean = mean; a.rstd = rstd; a.stream = s;
    return (cudaError_t)by_type<Forward>(a, dtype, on_16(x) && on_16(y) && on_16(weight) && on_16(bias));
}

// Covers both layouts of the rows: the choice between them goes by the call's pointers.
size_t layer_norm_backward_workspace_bytes(int dtype, int64_t rows, int groups, int d) {
    const int64_t v = slots_for(dtype, rows, groups, d, true), e = slots_for(dtype, rows, groups, d, false);
    return align_up(sizeof(float2) * (size_t)(v > e ? v : e) * groups * d, kAlign) + kAlign;
}

cudaError_t layer_norm_backward(const void* x, const void* dy, const float* weight, const float* mean,
                                const float* rstd, int dtype, int64_t rows, int groups, int d, void* dx,
                                float* dweight, float* dbias, void* workspace, cudaStream_t s) {
    const bool aligned = on_16(x) && on_16(dy) && on_16(dx) && on_16(weight);
    Args a{};
    a.x = x; a.dy = dy; a.weight = weight; a.mean_in = mean; a.rstd_in = rstd;
    a.rows = rows; a.groups = groups; a.d = d;
    a.out = dx; a.stream = s;
    a.part = dweight || dbias ? static_cast<float2*>(workspace) : nullptr;
    if (rows > 0) {
        const cudaError_t e = (cudaError_t)by_type<Backward>(a, dtype, aligned);
        if (e != cudaSuccess) return e;
    }
    if (!a.part) return cudaSuccess;
    const int64_t n = (int64_t)groups * d, M = rows > 0 ? slots_for(dtype, rows, groups, d, aligned) : 0;
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
