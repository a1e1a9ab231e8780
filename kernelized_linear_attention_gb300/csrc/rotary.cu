// Rotary positions: pair p of every head of token t turns by
// positions[t][axis(p)] * freq[p].
//
// Angles.  A position is an integer, so freq / 2 pi as a 64-bit fixed-point
// fraction of a turn times the position, modulo 2^64, is the angle modulo one
// turn with an error of |position| 2^-54 or less turns, at any distance.  Read as
// a signed number it is an angle in [-pi, pi), whose cos and sin are taken in fp32.
#include "internal.h"

namespace la {

namespace {

constexpr int kRotaryThreads = 256;

// freq / 2 pi modulo 1 in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_fraction(float freq) {
    const double turns = (double)freq * 0.15915494309189533577;   // 1 / (2 pi)
    const double frac = turns - floor(turns);                     // [0, 1]
    return (unsigned long long)(long long)((frac < 0.5 ? frac : frac - 1.0) * 18446744073709551616.0);
}

template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(RotaryParams p) {
    extern __shared__ float2 cs[];
    const int64_t t = blockIdx.x;
    for (int i = threadIdx.x; i < p.P; i += kRotaryThreads) {
        int axis = 0;
        while (axis + 1 < p.naxes && i >= p.first[axis + 1]) ++axis;
        const float f = p.freq[i];
        const unsigned long long turn =
            turn_fraction(f) * (unsigned long long)(long long)p.positions[t * p.naxes + axis];
        float s, c;
        sincospif((float)(long long)turn * 0x1p-63f, &s, &c);
        if (!isfinite(f)) s = c = __int_as_float(0x7fc00000);
        cs[i] = make_float2(c, p.inverse ? -s : s);
    }
    __syncthreads();
    const int64_t base = t * p.H * p.d;
    for (int which = 0; which < (p.k ? 2 : 1); ++which) {
        const T* x = static_cast<const T*>(which ? p.k : p.q) + base;
        T* y = static_cast<T*>(which ? p.k_out : p.q_out) + base;
        for (int j = threadIdx.x; j < p.H * p.P; j += kRotaryThreads) {
            const int head = j / p.P, i = j - head * p.P;
            const int64_t i0 = (int64_t)head * p.d + (p.interleaved ? 2 * i : i);
            const int64_t i1 = i0 + (p.interleaved ? 1 : p.P);
            const float x0 = load_elem(x, i0), x1 = load_elem(x, i1);
            store_elem(y, i0, x0 * cs[i].x - x1 * cs[i].y);
            store_elem(y, i1, x1 * cs[i].x + x0 * cs[i].y);
        }
        const int rest = p.d - 2 * p.P;
        if (x != y)
            for (int j = threadIdx.x; j < p.H * rest; j += kRotaryThreads) {
                const int64_t i = (int64_t)(j / rest) * p.d + 2 * p.P + j % rest;
                y[i] = x[i];
            }
    }
}

}  // namespace

cudaError_t rotary(const RotaryParams& p, int dtype, cudaStream_t s) {
    const size_t smem = sizeof(float2) * (size_t)p.P;
    if (dtype == LA_F32) rotary_kernel<float><<<(unsigned)p.T, kRotaryThreads, smem, s>>>(p);
    else rotary_kernel<__nv_bfloat16><<<(unsigned)p.T, kRotaryThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace la
