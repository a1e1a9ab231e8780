// Short vectors of storage elements for 16-byte loads and stores, and their
// conversion to and from fp32 (bf16 two at a time).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../tc_ptx.cuh"

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

// Element k of a vector.
template <typename T, int N>
__device__ __forceinline__ T element(const Vec<T, N>& x, int k) {
    if constexpr (sizeof(T) == 2 && N > 1) return __ushort_as_bfloat16((unsigned short)(x.v[k / 2] >> (k % 2 * 16)));
    else return x.v[k];
}

// Makes the compiler unpack a bf16 vector anew after this point, instead of keeping the twice as many
// registers of its fp32 values.
template <typename T, int N>
__device__ __forceinline__ void keep_packed(Vec<T, N>& x) {
    if constexpr (sizeof(T) == 2 && N > 1) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) asm volatile("" : "+r"(x.v[k]));
    }
}

// A vector's values two to a register pair (f32x2 arithmetic: one instruction for both); a single value
// alone.
template <int N>
struct Pairs {
    using P = uint64_t;
    static constexpr int n = N / 2;
};
template <>
struct Pairs<1> {
    using P = float;
    static constexpr int n = 1;
};
__device__ __forceinline__ float padd(float a, float b) { return a + b; }
__device__ __forceinline__ float pmul(float a, float b) { return a * b; }
__device__ __forceinline__ float pfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float psum(float a) { return a; }
__device__ __forceinline__ uint64_t padd(uint64_t a, uint64_t b) { return tc::f32x2_add(a, b); }
__device__ __forceinline__ uint64_t pmul(uint64_t a, uint64_t b) { return tc::f32x2_mul(a, b); }
__device__ __forceinline__ uint64_t pfma(uint64_t a, uint64_t b, uint64_t c) { return tc::f32x2_fma(a, b, c); }
__device__ __forceinline__ float psum(uint64_t a) { return tc::f32x2_lo(a) + tc::f32x2_hi(a); }
template <typename P> __device__ __forceinline__ P psplat(float x);
template <> __device__ __forceinline__ float psplat<float>(float x) { return x; }
template <> __device__ __forceinline__ uint64_t psplat<uint64_t>(float x) { return tc::f32x2_splat(x); }

template <int N, typename T>
__device__ __forceinline__ void unpack_pairs(typename Pairs<N>::P (&f)[Pairs<N>::n], const Vec<T, N>& x) {
    if constexpr (N == 1) {
        float v[1];
        unpack(v, x);
        f[0] = v[0];
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) f[k] = tc::f32x2_of(x.v[k] << 16, x.v[k] & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) f[k] = tc::f32x2_of(__float_as_uint(x.v[2 * k]), __float_as_uint(x.v[2 * k + 1]));
    }
}
template <int N, typename T>
__device__ __forceinline__ void pack_pairs(Vec<T, N>& x, const typename Pairs<N>::P (&f)[Pairs<N>::n]) {
    float v[N];
    if constexpr (N == 1) {
        v[0] = f[0];
    } else {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            v[2 * k] = tc::f32x2_lo(f[k]);
            v[2 * k + 1] = tc::f32x2_hi(f[k]);
        }
    }
    pack(x, v);
}

// Asynchronous copies of 16 bytes to shared memory; a group of them ends with copies_done(), and wait_copies<N>
// waits until at most N groups of this thread are on their way.
__device__ __forceinline__ void copy_16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace la
