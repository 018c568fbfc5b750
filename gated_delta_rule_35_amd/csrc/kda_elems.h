// Eight neighbouring elements of a row as a lane holds them: 16 bytes of bf16 or fp16, 32 of
// fp32, widened to fp32 and rounded back once (to nearest, ties to even).
#pragma once
#include "kda_gdr_device.h"

namespace kda {

template <int XT>
struct Elems;
template <>
struct Elems<0> {   // bf16
    typedef uint16_t T;
    typedef u32x4 Raw;   // eight channels as they lie in memory
    static __device__ __forceinline__ Raw load(const void* p, int64_t at) {
        return *reinterpret_cast<const Raw*>(static_cast<const T*>(p) + at);
    }
    static __device__ __forceinline__ void widen(const Raw& v, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf_lo(v[i]);
            x[2 * i + 1] = bf_hi(v[i]);
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[8]) {
        *reinterpret_cast<u32x4*>(static_cast<T*>(p) + at) =
            u32x4{pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7])};
    }
};
template <>
struct Elems<1> {   // fp16
    typedef uint16_t T;
    typedef half8 Raw;
    static __device__ __forceinline__ Raw load(const void* p, int64_t at) {
        return *reinterpret_cast<const Raw*>(static_cast<const T*>(p) + at);
    }
    static __device__ __forceinline__ void widen(const Raw& v, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[8]) {
        *reinterpret_cast<u32x4*>(static_cast<T*>(p) + at) =
            u32x4{pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]), pack_h2(x[6], x[7])};
    }
};
template <>
struct Elems<2> {   // fp32
    typedef float T;
    struct Raw {
        f32x4 a, b;
    };
    static __device__ __forceinline__ Raw load(const void* p, int64_t at) {
        const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const T*>(p) + at);
        return {s[0], s[1]};
    }
    static __device__ __forceinline__ void widen(const Raw& v, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = v.a[i];
            x[4 + i] = v.b[i];
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[8]) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<T*>(p) + at);
        d[0] = f32x4{x[0], x[1], x[2], x[3]};
        d[1] = f32x4{x[4], x[5], x[6], x[7]};
    }
};

// e^x for finite and infinite x to about one unit in the last place: the product with log2 e is
// kept with what its rounding leaves.  Below -200 the result is 0 either way; NaN stays.
__device__ __forceinline__ float exp_of(float x) {
    x = x < -200.f ? -200.f : (x > 200.f ? 200.f : x);
    const float h = x * LOG2E, l = fmaf(x, LOG2E, -h) + x * 1.92596299e-8f;
    return fexp2(h) * fmaf(l, LN2, 1.f);
}
// x, formed where this stands: the compiler would put what a select drops behind a branch, which
// parts matrix instructions (and a row's elements) from what could run beside them.
__device__ __forceinline__ float formed(float x) {
    asm volatile("" : "+v"(x));
    return x;
}

// 1 / (1 + e^-z).  FULL: to fp32's accuracy; else, for values of 16 bits, e^-z as 2^{-z log2 e}, off by up to |z| 2^-24 of
// itself: what a convolution's sum z is rounded by, and far below the half step of a 16-bit result.  Weights'
// gradients in fp32 are as near to 64 bits either way (2.0 10^-7 of their norm, convolution 2 x 4096 x 4352 in bf16, gated
// 3001 x 4096 1.4 10^-7); the full one took 66 us there and not 61, 33 and not 31.
template <bool FULL>
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + (FULL ? exp_of(-z) : fexp2(-LOG2E * z)));
}

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_SIGMOID = 2 };
// act(z) and its derivative from s = sigmoid(z): z s and s (1 + z (1 - s)), or s and s (1 - s).
__device__ __forceinline__ float activation(int act, float z, float s) {
    return act == ACT_NONE ? z : (act == ACT_SILU ? z : 1.f) * s;
}
__device__ __forceinline__ float slope(int act, float z, float s) {
    return act == ACT_NONE ? 1.f : s * fmaf(act == ACT_SILU ? z : 1.f, 1.f - s, act == ACT_SILU ? 1.f : 0.f);
}

}  // namespace kda
