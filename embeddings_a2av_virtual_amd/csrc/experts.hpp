// experts.hpp — what the experts' products in 16 bits and on microscaled rows
// share (gfx950): element types, activations, buffers and the plan of row tiles.
#pragma once

#include "common.hpp"

namespace a2av {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------ element types
struct Bf16 {
    typedef bf16x8 frag;
    static __device__ __forceinline__ float to_float(uint16_t v) { return bf16_lo(v); }
    // to nearest even by the conversion instruction (NaN stays some NaN): ten
    // instructions an element less than by integers
    static __device__ __forceinline__ uint16_t from_float(float f) {
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    }
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma(frag a, frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

struct Fp16 {
    typedef f16x8 frag;
    static __device__ __forceinline__ float to_float(uint16_t v) {
        return (float)__builtin_bit_cast(_Float16, v);
    }
    static __device__ __forceinline__ uint16_t from_float(float f) {
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    }
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma(frag a, frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// ------------------------------------------------------------------ activations
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// The normal distribution function Phi(h), with e = exp(-h^2 / 2): for x = |h|
// / sqrt(2), erfc(x) exp(x^2) / t is a polynomial in t = 1 / (1 + 0.3 x) to
// 2e-8 of its value on 0 <= x <= 10 (weighted least squares on a grid dense
// at 0, reweighted towards equal errors); in fp32 that leaves 5e-7.
__device__ __forceinline__ float normal_cdf(float h, float e) {
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.21213203f * fabsf(h));
    float p = -0.129522592f;
    p = __builtin_fmaf(p, t, 0.485561503f);
    p = __builtin_fmaf(p, t, -0.512274073f);
    p = __builtin_fmaf(p, t, 0.547714727f);
    p = __builtin_fmaf(p, t, -0.0946464393f);
    p = __builtin_fmaf(p, t, 0.214923891f);
    p = __builtin_fmaf(p, t, 0.148339838f);
    p = __builtin_fmaf(p, t, 0.170715113f);
    p = __builtin_fmaf(p, t, 0.169188013f);
    const float q = 0.5f * p * t * e;
    return h > 0.0f ? 1.0f - q : q;
}

// act(h) for one product; NaN stays NaN.
__device__ __forceinline__ float act_of(int act, float h) {
    switch (act) {
    case A2AV_ACT_RELU: return h < 0.0f ? 0.0f : h;
    case A2AV_ACT_GELU: return h * normal_cdf(h, __expf(-0.5f * h * h));
    case A2AV_ACT_SILU: return h * sigmoid(h);
    default: return h;
    }
}

// The weight row behind column c of the product: with SwiGLU, blocks of 16
// gate columns and the 16 up columns of the same outputs alternate, so that
// one lane ends with both.
__device__ __forceinline__ int64_t weight_row(int64_t c, int64_t N, bool glu) {
    if (!glu) return c;
    return ((c >> 4) & 1) * N + ((c >> 5) << 4) + (c & 15);
}

// ------------------------------------------------------------------ buffers
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;

constexpr uint32_t kGroup = 4;                // columns that an expert's row tiles go through together
constexpr uint32_t kOutside = 0x80000000u;    // a byte offset past every buffer

__device__ __forceinline__ rsrc_t buffer(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)bytes, 0x00020000);
}

// s_waitcnt with these many loads still in flight and, with lds, no LDS access.
template <int LOADS, bool LDS>
__device__ __forceinline__ void wait_for() {
    static_assert(LOADS < 64, "");
    __builtin_amdgcn_s_waitcnt((LOADS & 15) | ((LOADS >> 4) << 14) | 0x70 | (LDS ? 0 : 0xf00));
}

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

// Eight neighbouring elements: added to y, and y rounded into them.
template <typename T>
__device__ __forceinline__ void add8(float (&y)[8], const uint16_t *p) {
    const u16x8 v = *(const u16x8 *)p;
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] += T::to_float(v[i]);
}
template <typename T, bool NT = false>
__device__ __forceinline__ void put8(uint16_t *p, const float (&y)[8]) {
    u16x8 v;
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = T::from_float(y[i]);
    st<NT>((u16x8 *)p, v);
}

// ------------------------------------------------------------------ host
constexpr int kFewRows = 16;              // rows of the smallest tiles
constexpr int64_t kMostGroups = 1 << 22;  // workgroups of a launch, times 512 threads inside 32 bits

struct Layout {
    int64_t tiles;      // most tiles, of the smallest size
    size_t first, part; // byte offsets
    size_t total;
};

inline size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }
inline bool aligned16(const void *p) { return (uintptr_t)p % 16 == 0; }
inline bool fits(int64_t rows, int64_t width) {
    return (uint64_t)rows <= (uint64_t)INT64_MAX / 4 / (uint64_t)width;
}

// In experts.hip: the most row tiles of tile_rows, -1 for sizes that are not
// valid; the workspace's parts; the plan; the most tiles of `rows` rows.
int64_t tile_bound(int W, int P, int64_t K, int64_t N, int act, const int64_t *x_rows, int tile_rows);
bool plan_layout(int W, int P, int64_t K, int64_t N, int act, const int64_t *x_rows, bool with_part, Layout *l);
void launch_plan(int W, int P, const int64_t *x_rows, const int64_t *offsets, int tile_rows, unsigned char *ws,
                 const Layout &l, int32_t *status, hipStream_t stream);
int64_t most_tiles(const int64_t *x_rows, int W, int P, int rows);

}  // namespace a2av
