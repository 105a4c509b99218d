// gdn_vec.cuh -- eight consecutive elements of fp32 or bf16 at a time, in 16-byte accesses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_common.cuh"

namespace gdn {

// 2^x, a relative error of 2^-22, two units in the last place, which is what the library's functions of this kind promise as well;
// results under 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// sigmoid(x) = 1 / (1 + 2^t), t = -x log2 e, with the approximate 2^x and reciprocal, a fifth of the instructions of expf and a
// division (norms of 8192 rows of 5120, fp32 stream: 116 us with those, 98 with this, 96 without kFine).
// kFine: a relative error of 2^-21 (2^-22 of the power, 2^-23 of the reciprocal, 2^-24 of the sum).  t's rounding error, |x| 2^-24
// of the result, goes into 2^t as the factor 1 + lo ln 2, lo = -x log2 e - t with log2 e in two parts.  (Where t is infinite
// lo is infinite or not a number; 1 will do, 2^t is 0 or infinite then.)  Otherwise |x| 2^-24 more: nothing beside a bf16
// result's 2^-9, and bf16 norms are bound by these instructions (77.6 us without the factor, 80 with it).
template <bool kFine = true>
__device__ __forceinline__ float gate_of(float x) {
    const float t = -x * 1.4426950408889634f;
    float e = ex2(t), y;
    if constexpr (kFine) {
        const float lo = fmaf(-x, static_cast<float>(1.4426950408889634 - static_cast<double>(1.4426950408889634f)), fmaf(-x, 1.4426950408889634f, -t));
        e = fmaf(e, fmaf(fminf(fmaxf(lo, -1.0f), 1.0f), 0.6931471805599453f, 1.0f), 1.0f);
    } else {
        e += 1.0f;
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(e));
    return y;
}

// Hint: bring the 128-byte line of p into L2.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Two fp32 operations in one instruction (each rounds as the single one does).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + i);
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint4 x;
    x.x = StateIO<__nv_bfloat16>::pack(v[0], v[1]);
    x.y = StateIO<__nv_bfloat16>::pack(v[2], v[3]);
    x.z = StateIO<__nv_bfloat16>::pack(v[4], v[5]);
    x.w = StateIO<__nv_bfloat16>::pack(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = x;
}

// Eight elements as they lie in memory, for loads that are issued ahead of their use.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];

    __device__ __forceinline__ void load(const T* p) {   // read once: not kept in L1
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w) : "l"(reinterpret_cast<const uint4*>(p) + i));
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    // The elements of lane `from`.
    __device__ __forceinline__ Raw8 shuffled(int from) const {
        Raw8 r;
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
            r.w[i].x = __shfl_sync(0xffffffffu, w[i].x, from);
            r.w[i].y = __shfl_sync(0xffffffffu, w[i].y, from);
            r.w[i].z = __shfl_sync(0xffffffffu, w[i].z, from);
            r.w[i].w = __shfl_sync(0xffffffffu, w[i].w, from);
        }
        return r;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(w[i].x);
                v[4 * i + 1] = __uint_as_float(w[i].y);
                v[4 * i + 2] = __uint_as_float(w[i].z);
                v[4 * i + 3] = __uint_as_float(w[i].w);
            }
        } else {
            const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(x[i] << 16);
                v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
            }
        }
    }
};

}  // namespace gdn
