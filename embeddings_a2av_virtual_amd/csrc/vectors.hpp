// vectors.hpp — eight neighbouring elements of fp32, bf16 or fp16 at a time, and
// sums over a workgroup in double (gfx950).
#pragma once

#include "common.hpp"

namespace a2av {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The same at any address of an element: global accesses of 16 bytes need no
// alignment here.
typedef uint16_t u16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// An element type: `vec` holds eight of them as they lie in memory. What is loaded
// and stored is not used again soon, but for the lines of `cached` loads, which come in
// two halves or are shared with a neighbour.
struct ElemF32 {
    // The product of two is exact in fp32 where it is inside its range: of fp16 always, of
    // bf16 from 2^-126 to 2^128.
    static constexpr bool kExact = false;
    typedef float scalar;
    struct vec {
        f32x4 lo, hi;
    };
    static __device__ __forceinline__ vec load(const scalar *p) {
        return {__builtin_nontemporal_load((const f32x4_any *)p), __builtin_nontemporal_load((const f32x4_any *)p + 1)};
    }
    static __device__ __forceinline__ vec cached(const scalar *p) {
        return {*(const f32x4_any *)p, *((const f32x4_any *)p + 1)};
    }
    static __device__ __forceinline__ void store(scalar *p, vec v) {
        __builtin_nontemporal_store(v.lo, (f32x4_any *)p);
        __builtin_nontemporal_store(v.hi, (f32x4_any *)p + 1);
    }
    static __device__ __forceinline__ float get(const vec &v, int i) { return i < 4 ? v.lo[i & 3] : v.hi[i & 3]; }
    static __device__ __forceinline__ void put(vec &v, int i, scalar x) {
        if (i < 4) v.lo[i & 3] = x;
        else v.hi[i & 3] = x;
    }
    static __device__ __forceinline__ void set(vec &v, int i, float f) { put(v, i, f); }
    static __device__ __forceinline__ scalar raw(const vec &v, int i) { return get(v, i); }
};

struct Elem16 {
    static constexpr bool kExact = true;
    typedef uint16_t scalar;
    typedef u16x8 vec;
    static __device__ __forceinline__ vec load(const scalar *p) { return __builtin_nontemporal_load((const u16x8_any *)p); }
    static __device__ __forceinline__ vec cached(const scalar *p) { return *(const u16x8_any *)p; }
    static __device__ __forceinline__ void store(scalar *p, vec v) { __builtin_nontemporal_store(v, (u16x8_any *)p); }
    static __device__ __forceinline__ void put(vec &v, int i, scalar x) { v[i] = x; }
    static __device__ __forceinline__ scalar raw(const vec &v, int i) { return v[i]; }
};

struct ElemBf16 : Elem16 {
    static __device__ __forceinline__ float get(const vec &v, int i) { return bf16_lo(v[i]); }
    static __device__ __forceinline__ void set(vec &v, int i, float f) { v[i] = __builtin_bit_cast(uint16_t, (__bf16)f); }
};

struct ElemF16 : Elem16 {
    static __device__ __forceinline__ float get(const vec &v, int i) {
        const scalar u = v[i];  // (a bit cast of the element itself takes the vector's first)
        return (float)__builtin_bit_cast(_Float16, u);
    }
    static __device__ __forceinline__ void set(vec &v, int i, float f) { v[i] = __builtin_bit_cast(uint16_t, (_Float16)f); }
};

// Eight elements at c .. c + 7 of a row of H from p: those behind its end are 0, or
// not stored.
template <typename E>
__device__ __forceinline__ typename E::vec load_row(const typename E::scalar *p, int64_t c, int64_t H) {
    if (c + 8 <= H) return E::cached(p + c);
    typename E::vec v = {};
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (c + i < H) E::put(v, i, p[c + i]);
    return v;
}
template <typename E>
__device__ __forceinline__ void store_row(typename E::scalar *p, int64_t c, int64_t H, const typename E::vec &v) {
    if (c + 8 <= H) {
        E::store(p + c, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (c + i < H) p[c + i] = E::raw(v, i);
}

// The sum of 16 lanes, the first of the wave's rows of them, in every lane.
__device__ __forceinline__ double row_sum(double x) {
    const auto add = [&](uint64_t t) { x += __longlong_as_double((int64_t)t); };
    add(dpp_row_shr<1>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_shr<2>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_shr<4>((uint64_t)__double_as_longlong(x)));
    add(dpp_row_shr<8>((uint64_t)__double_as_longlong(x)));
    return __longlong_as_double((int64_t)readlane_u64((uint64_t)__double_as_longlong(x), 15));
}

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

// N sums over the workgroup at once, in a fixed order: `part` has a place for each of
// 16 waves, cleared by clear_parts before the kernel's first sums, and is not touched
// again before the barrier after the next.
template <int N>
__device__ __forceinline__ void clear_parts(double (&part)[2][16][N]) {
    if (threadIdx.x < 32 * N) (&part[0][0][0])[threadIdx.x] = 0.0;
    __syncthreads();
}
template <int N>
__device__ __forceinline__ void block_sums(double (&x)[N], double (*part)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) x[i] = wave_sum(x[i]);
    if (threadIdx.x % kWave == 0)
#pragma unroll
        for (int i = 0; i < N; i++) part[threadIdx.x / kWave][i] = x[i];
    __syncthreads();
    double y[N];
#pragma unroll
    for (int i = 0; i < N; i++) y[i] = part[threadIdx.x % 16][i];
#pragma unroll
    for (int i = 0; i < N; i++) x[i] = row_sum(y[i]);
}

}  // namespace a2av
