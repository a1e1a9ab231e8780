// Layer norm over rows of d values and its gradients.
#include "internal.h"

namespace la {

namespace {

constexpr int kNormWarps = 4;
constexpr int kDwThreads = 128;
constexpr int kMaxStripes = 256;   // row stripes whose weight gradients are summed apart

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(kNormWarps * 32) layer_norm_kernel(const T* x, const float* weight,
                                                                     const float* bias, int64_t rows, int groups,
                                                                     int d, float eps, T* y, float* mean,
                                                                     float* rstd) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t wb = (row % groups) * (int64_t)d;
    float sum = 0.f;
    for (int i = lane; i < d; i += 32) sum += load_elem(x, row * d + i);
    const float mu = warp_sum(sum) / d;
    float sq = 0.f;
    for (int i = lane; i < d; i += 32) {
        const float c = load_elem(x, row * d + i) - mu;
        sq = fmaf(c, c, sq);
    }
    const float rs = 1.f / sqrtf(warp_sum(sq) / d + eps);
    for (int i = lane; i < d; i += 32) {
        const float xh = (load_elem(x, row * d + i) - mu) * rs;
        store_elem(y, row * d + i, fmaf(xh, weight ? weight[wb + i] : 1.f, bias ? bias[wb + i] : 0.f));
    }
    if (lane == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
}

template <typename T>
__global__ void __launch_bounds__(kNormWarps * 32) layer_norm_dx_kernel(const T* x, const T* dy, const float* weight,
                                                                        const float* mean, const float* rstd,
                                                                        int64_t rows, int groups, int d, T* dx) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t wb = (row % groups) * (int64_t)d;
    const float mu = mean[row], rs = rstd[row];
    float su = 0.f, sux = 0.f;
    for (int i = lane; i < d; i += 32) {
        const float u = load_elem(dy, row * d + i) * (weight ? weight[wb + i] : 1.f);
        su += u;
        sux = fmaf(u, (load_elem(x, row * d + i) - mu) * rs, sux);
    }
    su = warp_sum(su) / d;
    sux = warp_sum(sux) / d;
    for (int i = lane; i < d; i += 32) {
        const float u = load_elem(dy, row * d + i) * (weight ? weight[wb + i] : 1.f);
        const float xh = (load_elem(x, row * d + i) - mu) * rs;
        store_elem(dx, row * d + i, rs * (u - su - xh * sux));
    }
}

// Column j of the groups * d weights: the rows of group j / d in stripe blockIdx.y.
template <typename T>
__global__ void __launch_bounds__(kDwThreads) layer_norm_dw_kernel(const T* x, const T* dy, const float* mean,
                                                                   const float* rstd, int64_t rows, int groups, int d,
                                                                   float2* part) {
    const int j = blockIdx.x * kDwThreads + threadIdx.x;
    if (j >= groups * d) return;
    const int g = j / d, i = j - g * d;
    float dw = 0.f, db = 0.f;
    for (int64_t row = (int64_t)blockIdx.y * groups + g; row < rows; row += (int64_t)gridDim.y * groups) {
        const float gy = load_elem(dy, row * d + i);
        dw = fmaf(gy, (load_elem(x, row * d + i) - mean[row]) * rstd[row], dw);
        db += gy;
    }
    part[(int64_t)blockIdx.y * groups * d + j] = make_float2(dw, db);
}

__global__ void __launch_bounds__(kDwThreads) layer_norm_join_kernel(const float2* part, int stripes, int n,
                                                                     float* dweight, float* dbias) {
    const int j = blockIdx.x * kDwThreads + threadIdx.x;
    if (j >= n) return;
    double dw = 0., db = 0.;
    for (int s = 0; s < stripes; ++s) {
        const float2 v = part[(int64_t)s * n + j];
        dw += v.x;
        db += v.y;
    }
    if (dweight) dweight[j] = (float)dw;
    if (dbias) dbias[j] = (float)db;
}

int stripes_for(int64_t rows, int groups) { return (int)min64(rows / groups, kMaxStripes); }

template <typename T>
cudaError_t backward(const void* x, const void* dy, const float* weight, const float* mean, const float* rstd,
                     int64_t rows, int groups, int d, void* dx, float* dweight, float* dbias, float2* part,
                     cudaStream_t s) {
    const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy);
    if (rows > 0)
        layer_norm_dx_kernel<T><<<(unsigned)ceil_div(rows, kNormWarps), kNormWarps * 32, 0, s>>>(
            xt, dyt, weight, mean, rstd, rows, groups, d, static_cast<T*>(dx));
    if (dweight || dbias) {
        const int n = groups * d, stripes = stripes_for(rows, groups);
        const unsigned cols = (unsigned)ceil_div(n, kDwThreads);
        if (stripes > 0)
            layer_norm_dw_kernel<T><<<dim3(cols, stripes), kDwThreads, 0, s>>>(xt, dyt, mean, rstd, rows, groups, d,
                                                                              part);
        layer_norm_join_kernel<<<cols, kDwThreads, 0, s>>>(part, stripes, n, dweight, dbias);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t layer_norm(const void* x, const float* weight, const float* bias, int dtype, int64_t rows, int groups,
                       int d, float eps, void* y, float* mean, float* rstd, cudaStream_t s) {
    const unsigned blocks = (unsigned)ceil_div(rows, kNormWarps);
    if (dtype == LA_F32)
        layer_norm_kernel<float><<<blocks, kNormWarps * 32, 0, s>>>(static_cast<const float*>(x), weight, bias, rows,
                                                                    groups, d, eps, static_cast<float*>(y), mean, rstd);
    else
        layer_norm_kernel<__nv_bfloat16><<<blocks, kNormWarps * 32, 0, s>>>(
            static_cast<const __nv_bfloat16*>(x), weight, bias, rows, groups, d, eps, static_cast<__nv_bfloat16*>(y),
            mean, rstd);
    return cudaGetLastError();
}

size_t layer_norm_backward_workspace_bytes(int dtype, int64_t rows, int groups, int d) {
    (void)dtype;
    return align_up(sizeof(float2) * (size_t)stripes_for(rows, groups) * groups * d, kAlign) + kAlign;
}

cudaError_t layer_norm_backward(const void* x, const void* dy, const float* weight, const float* mean,
                                const float* rstd, int dtype, int64_t rows, int groups, int d, void* dx,
                                float* dweight, float* dbias, void* workspace, cudaStream_t s) {
    float2* part = static_cast<float2*>(workspace);
    if (dtype == LA_F32)
        return backward<float>(x, dy, weight, mean, rstd, rows, groups, d, dx, dweight, dbias, part, s);
    return backward<__nv_bfloat16>(x, dy, weight, mean, rstd, rows, groups, d, dx, dweight, dbias, part, s);
}

}  // namespace la
