// mx.hpp — microscaled rows (gfx950): their layout, and blocks of 32 values to
// and from elements of 8 or 4 bits with one scale.
//
// A row of width H: H elements, padded with zeros to a multiple of 256 (e4m3: a
// byte each; e2m1: two a byte, the even one in the low half), a scale byte b =
// 2^(b - 127) for every 32 of them, and unused bytes up to a multiple of 128.
// So every row starts on a cache line, a contraction of 128 bytes of elements
// never ends inside a row, and the rows travel with their scales.
#pragma once

#include "common.hpp"

namespace a2av {

constexpr int kMxBlock = 32;    // elements of a scale
constexpr int kMxPad = 256;     // elements that a row is padded to
constexpr int kMxNan = 255;     // the scale byte of a block that stands for NaN

__host__ __device__ inline int64_t mx_padded(int64_t width) { return (width + kMxPad - 1) / kMxPad * kMxPad; }
__host__ __device__ inline int64_t mx_element_bytes(int format, int64_t width) {
    return mx_padded(width) >> (format == A2AV_MX_FP4);
}
__host__ __device__ inline int64_t mx_stride(int format, int64_t width) {
    return (mx_element_bytes(format, width) + mx_padded(width) / kMxBlock + 127) / 128 * 128;
}

// Elements of a format: the largest is 1.75 * 2^8 or 1.5 * 2^2, so the scale that
// puts a block's largest magnitude m there is 2^(floor(log2 m) - 8) or - 2.
template <int FORMAT>
struct Mx;

template <>
struct Mx<A2AV_MX_FP8> {
    static constexpr int kTop = 8;
    typedef u32x2 packed;  // eight elements
    // to nearest even; past 448 (the instruction gives NaN) 448
    static __device__ __forceinline__ float stop(float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); }
    static __device__ __forceinline__ packed pack(const float (&v)[8]) {
        packed p;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(stop(v[i * 4]), stop(v[i * 4 + 1]), 0, false);
            p[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(stop(v[i * 4 + 2]), stop(v[i * 4 + 3]), w, true);
        }
        return p;
    }
    static __device__ __forceinline__ void unpack(packed p, float scale, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], true);
            v[i * 4] = lo[0] * scale;
            v[i * 4 + 1] = lo[1] * scale;
            v[i * 4 + 2] = hi[0] * scale;
            v[i * 4 + 3] = hi[1] * scale;
        }
    }
};

template <>
struct Mx<A2AV_MX_FP4> {
    static constexpr int kTop = 2;
    typedef uint32_t packed;
    // to nearest even; past 6 the instruction gives 6
    static __device__ __forceinline__ packed pack(const float (&v)[8]) {
        packed p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
        p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[2], v[3], 1.0f, 1);
        p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[4], v[5], 1.0f, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[6], v[7], 1.0f, 3);
    }
    static __device__ __forceinline__ void unpack(packed p, float scale, float (&v)[8]) {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 0);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 1);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 2);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 3);
        const float e[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = e[i] * scale;
    }
};

// The largest m of the lane's quad: four lanes with 8 values each hold a block.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, true);  // lanes 1 0 3 2
    m = a > m ? a : m;
    const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, true);  // lanes 2 3 0 1
    return b > m ? b : m;
}

// The bits of the largest magnitude of a quad's values, NaN above all.
__device__ __forceinline__ uint32_t quad_top(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = u > m ? u : m;
    }
    return quad_max(m);
}

// The same by the maximum that gives NaN if an operand is: half the instructions.
__device__ __forceinline__ uint32_t quad_largest(const float (&v)[8]) {
    float m;
    asm("v_maximum3_f32 %0, |%1|, |%2|, 0" : "=v"(m) : "v"(v[0]), "v"(v[1]));
#pragma unroll
    for (int i = 2; i < 8; i += 2) asm("v_maximum3_f32 %0, |%1|, |%2|, %0" : "+v"(m) : "v"(v[i]), "v"(v[i + 1]));
    return quad_max(__float_as_uint(m) & 0x7FFFFFFFu);
}

// The scale byte of a block whose largest magnitude has these bits, and the
// elements of a lane's eight values; every lane of the quad is active. A block
// with an infinity or NaN is NaN: its scale says so and its elements are 0.
template <int FORMAT>
__device__ __forceinline__ typename Mx<FORMAT>::packed mx_block(const float (&v)[8], int &scale) {
    const int e = (int)(quad_top(v) >> 23);
    const bool bad = e == 255;
    scale = bad ? kMxNan : e > Mx<FORMAT>::kTop ? e - Mx<FORMAT>::kTop : 0;
    // 2^(127 - scale): the product is exact, or far below the smallest element
    const float inv = bad ? 0.0f : __uint_as_float((uint32_t)(254 - scale) << 23);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) s[i] = v[i] * inv;
    return bad ? typename Mx<FORMAT>::packed{} : Mx<FORMAT>::pack(s);
}

// The scale byte for a largest magnitude in double, and the factor 2^(127 - it);
// NaN or an infinity gives the byte of NaN.
template <int FORMAT>
__device__ __forceinline__ int mx_scale_of(uint32_t upper, double &inv) {
    const int e = (int)((upper & 0x7FFFFFFFu) >> 20), want = e - 1023 + 127 - Mx<FORMAT>::kTop;
    const int scale = want < 0 ? 0 : want > 254 ? 254 : want;
    inv = __longlong_as_double((int64_t)(1023 + 127 - scale) << 52);
    return e == 2047 ? kMxNan : scale;
}
__device__ __forceinline__ uint32_t upper_word(double v) { return (uint32_t)((uint64_t)__double_as_longlong(v) >> 32); }

// A double for the rounding to an element: its upper word (20 bits of the mantissa)
// with the last bit set if any bits follow is on the same side of every middle of
// two elements as the double, and exact in fp32. A rounding to fp32 could put it on
// a middle.
__device__ __forceinline__ float jam(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t rest = (uint32_t)u < 1u ? (uint32_t)u : 1u;
    return (float)__longlong_as_double((int64_t)((uint64_t)((uint32_t)(u >> 32) | rest) << 32));
}

// The same for values in double, from whose last places the elements of a norm are
// decided.
template <int FORMAT>
__device__ __forceinline__ typename Mx<FORMAT>::packed mx_block(const double (&v)[8], int &scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t u = upper_word(v[i]) & 0x7FFFFFFFu;
        m = u > m ? u : m;
    }
    double inv;
    scale = mx_scale_of<FORMAT>(quad_max(m), inv);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) s[i] = jam(v[i] * inv);
    return scale == kMxNan ? typename Mx<FORMAT>::packed{} : Mx<FORMAT>::pack(s);
}

// The same for the products v[i] * r, r in double, of a quad whose largest v has the
// magnitude m: one product in double each.
template <int FORMAT>
__device__ __forceinline__ typename Mx<FORMAT>::packed mx_block(const float (&v)[8], uint32_t m, double r, int &scale) {
    double inv;
    scale = mx_scale_of<FORMAT>(upper_word((double)__uint_as_float(m) * r), inv);
    inv *= r;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) s[i] = jam((double)v[i] * inv);
    return scale == kMxNan ? typename Mx<FORMAT>::packed{} : Mx<FORMAT>::pack(s);
}

// 2^(b - 127) as a factor: 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

}  // namespace a2av
