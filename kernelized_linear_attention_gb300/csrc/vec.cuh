// Short vectors of storage elements for 16-byte loads and stores, and their
// conversion to and from fp32 (bf16 two at a time).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace la {

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};
template <int N>
struct alignas(2 * N) Vec<__nv_bfloat16, N> {
    uint32_t v[N / 2];
};
template <>
struct Vec<__nv_bfloat16, 1> {
    __nv_bfloat16 v[1];
};

template <int N>
__device__ __forceinline__ void unpack(float (&f)[N], const Vec<float, N>& x) {
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = x.v[k];
}
template <int N>
__device__ __forceinline__ void unpack(float (&f)[N], const Vec<__nv_bfloat16, N>& x) {
    if constexpr (N == 1) {
        f[0] = __bfloat162float(x.v[0]);
    } else {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {   // a bf16 is the upper half of its fp32
            f[2 * k] = __uint_as_float(x.v[k] << 16);
            f[2 * k + 1] = __uint_as_float(x.v[k] & 0xffff0000u);
        }
    }
}
template <int N>
__device__ __forceinline__ void pack(Vec<float, N>& x, const float (&f)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) x.v[k] = f[k];
}
template <int N>
__device__ __forceinline__ void pack(Vec<__nv_bfloat16, N>& x, const float (&f)[N]) {
    if constexpr (N == 1) {
        x.v[0] = __float2bfloat16_rn(f[0]);
    } else {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            x.v[k] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
}

}  // namespace la
