// vectors.hpp — eight neighbouring elements of fp32, bf16 or fp16 at a time, and
// sums over a workgroup in double (gfx950).
#pragma once

#include "common.hpp"

namespace a2av {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// An element type: `vec` holds eight of them as they lie in memory.
struct ElemF32 {
    typedef float scalar;
    struct vec {
        f32x4 lo, hi;
    };
    static __device__ __forceinline__ float to_float(scalar v) { return v; }
    static __device__ __forceinline__ scalar from_float(float f) { return f; }
    static __device__ __forceinline__ vec load(const scalar *p) { return {*(const f32x4 *)p, *(const f32x4 *)(p + 4)}; }
    static __device__ __forceinline__ void store(scalar *p, vec v) {
        *(f32x4 *)p = v.lo;
        *(f32x4 *)(p + 4) = v.hi;
    }
    static __device__ __forceinline__ float get(const vec &v, int i) { return i < 4 ? v.lo[i & 3] : v.hi[i & 3]; }
    static __device__ __forceinline__ void set(vec &v, int i, float f) {
        if (i < 4) v.lo[i & 3] = f;
        else v.hi[i & 3] = f;
    }
};

struct ElemBf16 {
    typedef uint16_t scalar;
    typedef u16x8 vec;
    static __device__ __forceinline__ float to_float(scalar v) { return bf16_lo(v); }
    static __device__ __forceinline__ scalar from_float(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
    static __device__ __forceinline__ vec load(const scalar *p) { return *(const vec *)p; }
    static __device__ __forceinline__ void store(scalar *p, vec v) { *(vec *)p = v; }
    static __device__ __forceinline__ float get(const vec &v, int i) { return to_float(v[i]); }
    static __device__ __forceinline__ void set(vec &v, int i, float f) { v[i] = from_float(f); }
};

struct ElemF16 {
    typedef uint16_t scalar;
    typedef u16x8 vec;
    static __device__ __forceinline__ float to_float(scalar v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ scalar from_float(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
    static __device__ __forceinline__ vec load(const scalar *p) { return *(const vec *)p; }
    static __device__ __forceinline__ void store(scalar *p, vec v) { *(vec *)p = v; }
    static __device__ __forceinline__ float get(const vec &v, int i) { return to_float(v[i]); }
    static __device__ __forceinline__ void set(vec &v, int i, float f) { v[i] = from_float(f); }
};

// The wave's sum, the same in every lane and every run; every lane is active.
__device__ __forceinline__ double wave_sum(double x) {
    const auto add = [&](uint64_t t) { x += __longlong_as_double((int64_t)t); };
    add(dpp_row_shr<1>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_shr<2>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_shr<4>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_shr<8>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_bcast<0x142, 0xa>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_bcast<0x143, 0xc>((uint64_t)__double_as_longlong(x)));
    return __longlong_as_double((int64_t)readlane_u64((uint64_t)__double_as_longlong(x), kWave - 1));
}

// N sums over the workgroup of BLOCK threads at once, in a fixed order; `part`
// is LDS that the workgroup does not touch before its next barrier.
template <int BLOCK, int N>
__device__ __forceinline__ void block_sums(double (&x)[N], double (*part)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) x[i] = wave_sum(x[i]);
    if constexpr (BLOCK > kWave) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int i = 0; i < N; i++) part[wave][i] = x[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) x[i] = part[0][i];
#pragma unroll
        for (int w = 1; w < BLOCK / kWave; w++)
#pragma unroll
            for (int i = 0; i < N; i++) x[i] += part[w][i];
    }
}

}  // namespace a2av
