// Layer norm over rows of d values and its gradients.
//
// Bound by memory: the forward reads x and writes y once, the backward reads x
// and dy and writes dx once.  A row stays in the registers of the L lanes that
// share it (E vectors of N values each) between the sums over it and its
// output; the variance comes from the deviations in registers, not from sums of
// squares.  Rows of up to 64 vectors share a warp, which then holds U rows at
// once so that their loads and sums overlap; longer rows take a block.
//
// A group of lanes keeps one weight row: it walks over rows a multiple of
// `groups` apart.  Its weights are read once, and in the backward its columns'
// weight gradients add up in registers over all its rows.  Blocks leave their
// sums in the workspace as rows of a [M][groups * d] matrix that a second
// kernel adds up by column in fp64, in a fixed order.
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

// The lane's E vectors of a row: vector e starts at column (e L + lane) N.
template <typename S, typename T>
__device__ __forceinline__ void load_row(Vec<T, S::N> (&x)[S::E], const T* row, int d, int lane, bool live) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        const int c = (e * S::L + lane) * S::N;
        if (live && c < d) x[e] = *reinterpret_cast<const Vec<T, S::N>*>(row + c);
        else
#pragma unroll
            for (int k = 0; k < S::N; ++k) x[e].v[k] = down<T>(0.f);
    }
}
template <typename S>
__device__ __forceinline__ void load_params(float (&w)[S::kValues], const float* p, int64_t at, int d, int lane, float missing) {
#pragma unroll
    for (int e = 0; e < S::E; ++e)
#pragma unroll
        for (int k = 0; k < S::N; ++k) {
            const int c = (e * S::L + lane) * S::N + k;
            w[e * S::N + k] = p && c < d ? p[at + c] : missing;
        }
}

template <typename T, typename S, int U>
__global__ void __launch_bounds__(S::kThreads) layer_norm_kernel(const T* x, const float* weight, const float* bias,
                                                                 int64_t rows, int groups, int d, float eps, T* y,
                                                                 float* mean, float* rstd, int64_t stride) {
    __shared__ float scratch[S::L > 32 ? U * S::L / 32 : 1];
    const int lane = threadIdx.x % S::L;
    const int64_t first = (int64_t)blockIdx.x * S::kRows + threadIdx.x / S::L;
    const float fd = (float)d;
    // one weight row for all rows of the group, held where the registers allow it
    constexpr bool kHeld = S::kValues <= 8;
    const bool one = stride % groups == 0;
    float w[S::kValues], b[S::kValues];
    if (kHeld && one) {
        const int64_t at = first % groups * d;
        load_params<S>(w, weight, at, d, lane, 1.f);
        load_params<S>(b, bias, at, d, lane, 0.f);
    }
    // a row group that starts behind the last row still takes part in the block's sums
    const int64_t turns = (rows - (int64_t)blockIdx.x * S::kRows + stride * U - 1) / (stride * U);
    for (int64_t turn = 0; turn < turns; ++turn) {
        Vec<T, S::N> v[U][S::E];
        float s[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + (turn * U + u) * stride;
            load_row<S, T>(v[u], x + row * d, d, lane, row < rows);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < S::E; ++e)
#pragma unroll
                for (int k = 0; k < S::N; ++k) s[u] += up(v[u][e].v[k]);
        }
        row_sums<S, U>(s, scratch);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] /= fd;         // (a product with 1 / d would miss the mean of equal values)
            q[u] = 0.f;
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                if ((e * S::L + lane) * S::N < d)
#pragma unroll
                    for (int k = 0; k < S::N; ++k) {
                        const float c = up(v[u][e].v[k]) - s[u];
                        q[u] = fmaf(c, c, q[u]);
                    }
        }
        row_sums<S, U>(q, scratch);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + (turn * U + u) * stride;
            if (row >= rows) continue;
            const float mu = s[u], rs = 1.f / sqrtf(q[u] / fd + eps);
            const int64_t at = kHeld && one ? 0 : row % groups * d;
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                const int c = (e * S::L + lane) * S::N;
                if (c >= d) continue;
                Vec<T, S::N> o;
#pragma unroll
                for (int k = 0; k < S::N; ++k) {
                    const float xh = (up(v[u][e].v[k]) - mu) * rs;
                    float we, be;
                    if (kHeld && one) {
                        we = w[e * S::N + k];
                        be = b[e * S::N + k];
                    } else {
                        we = weight ? weight[at + c + k] : 1.f;
                        be = bias ? bias[at + c + k] : 0.f;
                    }
                    o.v[k] = down<T>(fmaf(xh, we, be));
                }
                *reinterpret_cast<Vec<T, S::N>*>(y + row * d + c) = o;
            }
            if (lane == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
        }
    }
}

// part[slot][d]: the weight and bias gradients of one weight row over some rows, slot i of weight row
// i mod groups.  Row groups of a block that share a weight row are added up first where every one of
// its weight rows has equally many (kRows a multiple of groups).
template <typename T, typename S, int U>
__global__ void __launch_bounds__(S::kThreads) layer_norm_backward_kernel(const T* x, const T* dy, const float* weight,
                                                                          const float* mean, const float* rstd,
                                                                          int64_t rows, int groups, int d, T* dx,
                                                                          float2* part, int64_t stride) {
    __shared__ float scratch[S::L > 32 ? U * S::L / 32 : 1];
    extern __shared__ float2 sums[];                        // [kRows][d], L <= 32
    const int lane = threadIdx.x % S::L, group = threadIdx.x / S::L;
    const int64_t first = (int64_t)blockIdx.x * S::kRows + group;
    const float over_d = 1.f / d;
    constexpr bool kHeld = S::kValues <= 8;
    const int64_t at = first % groups * d;                  // stride is a multiple of groups
    float w[S::kValues], dw[S::kValues], db[S::kValues];
    if (kHeld) load_params<S>(w, weight, at, d, lane, 1.f);
#pragma unroll
    for (int k = 0; k < S::kValues; ++k) dw[k] = db[k] = 0.f;
    const int64_t turns = (rows - (int64_t)blockIdx.x * S::kRows + stride * U - 1) / (stride * U);
    for (int64_t turn = 0; turn < turns; ++turn) {
        Vec<T, S::N> v[U][S::E], g[U][S::E];
        float mu[U], rs[U], s1[U], s2[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + (turn * U + u) * stride;
            load_row<S, T>(v[u], x + row * d, d, lane, row < rows);
            load_row<S, T>(g[u], dy + row * d, d, lane, row < rows);
            mu[u] = row < rows ? mean[row] : 0.f;
            rs[u] = row < rows ? rstd[row] : 0.f;
        }
        if (!kHeld) load_params<S>(w, weight, at, d, lane, 1.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s1[u] = s2[u] = 0.f;
            const bool live = first + (turn * U + u) * stride < rows;
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                if (live && (e * S::L + lane) * S::N < d)
#pragma unroll
                    for (int k = 0; k < S::N; ++k) {
                        const int i = e * S::N + k;
                        const float gy = up(g[u][e].v[k]), xh = (up(v[u][e].v[k]) - mu[u]) * rs[u], t = gy * w[i];
                        s1[u] += t;
                        s2[u] = fmaf(t, xh, s2[u]);
                        dw[i] = fmaf(gy, xh, dw[i]);
                        db[i] += gy;
                    }
        }
        row_sums<S, U>(s1, scratch);
        row_sums<S, U>(s2, scratch);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + (turn * U + u) * stride;
            if (row >= rows) continue;
            const float m1 = s1[u] * over_d, m2 = s2[u] * over_d;
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                const int c = (e * S::L + lane) * S::N;
                if (c >= d) continue;
                Vec<T, S::N> o;
#pragma unroll
                for (int k = 0; k < S::N; ++k) {
                    const float t = up(g[u][e].v[k]) * w[e * S::N + k], xh = (up(v[u][e].v[k]) - mu[u]) * rs[u];
                    o.v[k] = down<T>(rs[u] * (t - m1 - xh * m2));
                }
                *reinterpret_cast<Vec<T, S::N>*>(dx + row * d + c) = o;
            }
        }
    }
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

// Column sums of part[M][n]: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(kJoinCols * kJoinRows) layer_norm_join_kernel(const float2* part, int64_t M, int64_t n,
                                                                                float* dweight, float* dbias) {
    __shared__ double sw[kJoinRows][kJoinCols], sb[kJoinRows][kJoinCols];
    const int col = threadIdx.x % kJoinCols, r = threadIdx.x / kJoinCols;
    const int64_t j = (int64_t)blockIdx.x * kJoinCols + col;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    double dw = 0., db = 0.;
    if (j < n)
#pragma unroll 4
        for (int64_t m = r; m < M; m += kJoinRows) {
            const float2 v = part[m * n + j];
            dw += v.x;
            db += v.y;
        }
    sw[r][col] = dw;
    sb[r][col] = db;
    for (int o = kJoinRows / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (r < o) {
            sw[r][col] += sw[r + o][col];
            sb[r][col] += sb[r + o][col];
        }
    }
    if (r == 0 && j < n) {
        if (dweight) dweight[j] = (float)sw[0][col];
        if (dbias) dbias[j] = (float)sb[0][col];
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
    template <typename T, typename S>
    static int64_t run(const Args& a) {
        constexpr int U = S::kValues <= 8 && S::L <= 32 ? 4 : S::kValues <= 16 ? 2 : 1;
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
    template <typename T, typename S>
    static int64_t run(const Args& a) {
        constexpr int U = S::kValues <= 8 && S::L <= 32 ? 2 : 1;
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
    template <typename T, typename S>
    static int64_t run(const Args& a) { return backward_slots<S>(a.rows, a.groups); }
};

// The lanes and vectors of a row: the fewest lanes that hold it in one vector each up to a warp, two
// vectors a lane up to 64, then a block of 128 to 512 lanes.
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
    return (cudaError_t)by_type<Forward>(a, dtype, on_16(x) && on_16(y));
}

// Covers both layouts of the rows: the choice between them goes by the call's pointers.
size_t layer_norm_backward_workspace_bytes(int dtype, int64_t rows, int groups, int d) {
    const int64_t v = slots_for(dtype, rows, groups, d, true), e = slots_for(dtype, rows, groups, d, false);
    return align_up(sizeof(float2) * (size_t)(v > e ? v : e) * groups * d, kAlign) + kAlign;
}

cudaError_t layer_norm_backward(const void* x, const void* dy, const float* weight, const float* mean,
                                const float* rstd, int dtype, int64_t rows, int groups, int d, void* dx,
                                float* dweight, float* dbias, void* workspace, cudaStream_t s) {
    const bool aligned = on_16(x) && on_16(dy) && on_16(dx);
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
