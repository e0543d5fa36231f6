// norm.hip — the root-mean-square norm in front of the router, with the
// residual's addition and its rows in 16 or 32 bits or microscaled for the
// dispatch, and its gradient (gfx950).
//
//   h = x + residual (rounded to the type)      r = 1 / sqrt(mean(h^2) + eps)
//   y = h * r * weight
//   d_x = r * (d_y * weight - h * r^2 * mean(d_y * weight * h)) + d_h
//   d_weight = sum over rows of d_y * h * r
//
//   k_norm_row        rows of up to 16384, held in a wave's or a workgroup's registers
//   k_norm_any        wider rows, read twice
//   k_norm_grad_row   the gradient of the first, weight sums of a workgroup's rows
//   k_norm_grad_any   the gradient of the second
//   k_norm_weight     the workgroups' weight sums, in order
#include <hip/hip_runtime.h>

#include <cstring>

#include "mx.hpp"
#include "vectors.hpp"

namespace a2av {

struct NormArgs {
    const void *x[A2AV_MAX_W];
    const void *residual[A2AV_MAX_W];
    void *sum[A2AV_MAX_W];
    void *out[A2AV_MAX_W];
    unsigned char *rows[A2AV_MAX_W];
    const void *weight;
    const int32_t *status;
    int64_t T, H;
    double eps, per;  // per: 1 / H
    int has_residual, has_sum, has_out;
};

// 1 / sqrt(m) to the last place of double or next to it: the instruction's 2^-28 and
// a step of third order. (Division and root as written take 60 instructions a thread
// and row, a third of what a row of two vectors a thread takes.) 0 and infinity give
// infinity and 0.
__device__ __forceinline__ double inverse_root(double m) {
    const double r = __builtin_amdgcn_rsq(m), e = __builtin_fma(-m * r, r, 1.0);
    const double better = __builtin_fma(r * e, __builtin_fma(e, 0.375, 0.5), r);
    return m > 0.0 && m < (double)INFINITY ? better : r;
}

// What a row is multiplied by, r = 1 / sqrt(mean(h^2) + eps), in two steps: a power
// of two and the rest in double, from 1 to 2 (to 128 for the smallest rows of bf16). In
// types of 16 bits h * power * w is then exact in fp32 and not past its range where y is
// not, so that an element of a block takes one product in double; but for a y below
// 2^-132 and elements 2^-140 below their row's magnitude. (A branch for the power 1 cost
// what it saved: 91.3 us without a residual with it, 90.4 without.)
struct RowScale {
    double r, rest;
    float power;
    __device__ __forceinline__ explicit RowScale(double mean) {  // of h^2, and eps
        r = inverse_root(mean);
        int k = (int)(upper_word(r) >> 20) - 1023;  // NaN, infinity and 0 at the ends
        k = min(max(k, -128), 127);
        power = __builtin_ldexpf(1.0f, k);  // may be subnormal
        rest = r * __longlong_as_double((int64_t)(1023 - k) << 52);
    }
};

// A lane's eight weights.
struct Weights {
    float v[8];
    template <typename E>
    __device__ __forceinline__ void set(const typename E::vec &w) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = E::get(w, i);
    }
};

// Outputs of a lane's eight elements h and weights w at column c of row t; every lane
// of a quad comes here together. FORMAT 0: no microscaled rows.
template <typename E, int FORMAT>
__device__ __forceinline__ void put_norm(const NormArgs &a, int rank, int64_t t, int64_t c, const typename E::vec &h,
                                         const Weights &w, const RowScale &s) {
    if constexpr (E::kExact) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = E::get(h, i) * s.power * w.v[i];
        if (a.has_out) {  // one rounding to fp32 of the factor and one of the product before that to 16 bits
            const float rest = (float)s.rest;
            typename E::vec o;
#pragma unroll
            for (int i = 0; i < 8; i++) E::set(o, i, y[i] * rest);
            store_row<E>((typename E::scalar *)a.out[rank] + t * a.H, c, a.H, o);
        }
        if constexpr (FORMAT != 0) {
            int scale;
            // a block behind the row is 0, also where the row has no finite factor
            const auto p = mx_block<FORMAT>(y, quad_largest(y), (c & ~(int64_t)31) < a.H ? s.rest : 0.0, scale);
            unsigned char *row = a.rows[rank] + t * mx_stride(FORMAT, a.H);
            __builtin_nontemporal_store(p, (typename Mx<FORMAT>::packed *)(row + c / 8 * (int64_t)sizeof(p)));
            if (threadIdx.x % 4 == 0) row[mx_element_bytes(FORMAT, a.H) + c / kMxBlock] = (unsigned char)scale;
        }
    } else {
        double y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = (double)E::get(h, i) * s.r * (double)w.v[i];
        if (a.has_out) {
            typename E::vec o;
#pragma unroll
            for (int i = 0; i < 8; i++) E::set(o, i, (float)y[i]);
            store_row<E>((typename E::scalar *)a.out[rank] + t * a.H, c, a.H, o);
        }
        if constexpr (FORMAT != 0) {
            int scale;
            if (c + 8 > a.H)
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (c + i >= a.H) y[i] = 0.0;
            const auto p = mx_block<FORMAT>(y, scale);
            unsigned char *row = a.rows[rank] + t * mx_stride(FORMAT, a.H);
            __builtin_nontemporal_store(p, (typename Mx<FORMAT>::packed *)(row + c / 8 * (int64_t)sizeof(p)));
            if (threadIdx.x % 4 == 0) row[mx_element_bytes(FORMAT, a.H) + c / kMxBlock] = (unsigned char)scale;
        }
    }
}

// The rows of a workgroup, one after the other: a wave each (MOST 64), or the whole
// workgroup of up to MOST threads together. A lane has VPT vectors of 8 elements of
// the row in registers; the next row's are loaded before this one's sum is waited for,
// and the weight's once. The mean and the values are in double: an element of 8 or 4
// bits then comes out the same however the sum is ordered, and double costs what fp32
// does beside the row's bytes. WHOLE: rows are whole vectors.
// Bound by the bytes: 8 x 2048 rows of 7168 in bf16 with a residual, the sum and 8-bit
// rows 142 us, 5.8 TB/s (a copy reaches 6.5; 150 with stores of the rows that stay in
// the caches, 162 with a workgroup for every row and no load ahead); 8 x 8192 of 2048
// 157, 6.0; odd ones 8 x 2048 x 1003 in fp16 25 (39 read twice). One row of 7168 takes
// 4 us. Without a residual the arithmetic shows: 90 us, 3.9 TB/s.
template <typename E, int FORMAT, int VPT, int MOST, bool WHOLE>
__global__ __launch_bounds__(MOST == kWave ? 256 : MOST) void k_norm_row(const NormArgs a) {
    __shared__ double part[2][1024 / kWave][1];
    if (status_at_entry(a.status)) return;
    clear_parts(part);
    typedef typename E::scalar scalar;
    typedef typename E::vec vec;
    constexpr bool WAVE = MOST == kWave, kNext = MOST < 1024;  // registers for the next row
    const int rank = blockIdx.y, lanes = WAVE ? kWave : blockDim.x;
    const int lane = WAVE ? threadIdx.x % kWave : threadIdx.x;
    const int vecs = (int)((FORMAT ? mx_padded(a.H) : a.H + 7) / 8);
    const int64_t step = WAVE ? gridDim.x * 4 : gridDim.x;
    const scalar *x = (const scalar *)a.x[rank], *residual = (const scalar *)a.residual[rank];
    vec h[VPT], r[VPT], h1[VPT], r1[VPT];
    Weights w[VPT];
    // a lane behind the row loads its last vector again, and counts 0, of weight +0
    const int own = (int)((a.H + 7) / 8);
    const auto load = [&](vec(&to)[VPT], const scalar *p) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int c = min(i * lanes + lane, own - 1) * 8;
            // (8 x 1024 rows of 7168 in fp32: 141 us, 159 with loads past the caches; in 16 bits
            // those are the better ones, 142 and 146)
            if constexpr (WHOLE && E::kExact) to[i] = E::load(p + c);
            else if constexpr (WHOLE) to[i] = E::cached(p + c);
            else to[i] = load_row<E>(p, c, a.H);
        }
    };
    load(h, (const scalar *)a.weight);
#pragma unroll
    for (int i = 0; i < VPT; i++) w[i].template set<E>(i * lanes + lane < own ? h[i] : vec{});
    int64_t t = WAVE ? (int64_t)blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
    if (kNext && t < a.T) {
        load(h1, x + t * a.H);
        if (a.has_residual) load(r1, residual + t * a.H);
    }
    for (int turn = 0; t < a.T; t += step, turn ^= 1) {
        if constexpr (kNext) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                h[i] = h1[i];
                r[i] = r1[i];
            }
            if (t + step < a.T) {
                load(h1, x + (t + step) * a.H);
                if (a.has_residual) load(r1, residual + (t + step) * a.H);
            }
        } else {
            load(h, x + t * a.H);
            if (a.has_residual) load(r, residual + t * a.H);
        }
        double s[1] = {0.0};
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * lanes + lane;
            if (a.has_residual)
#pragma unroll
                for (int c = 0; c < 8; c++) E::set(h[i], c, E::get(h[i], c) + E::get(r[i], c));
            if (v >= own) h[i] = vec{};
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const double d = E::get(h[i], c);
                s[0] = __builtin_fma(d, d, s[0]);
            }
            if (a.has_sum && v < own) {
                scalar *sum = (scalar *)a.sum[rank] + t * a.H;
                if constexpr (WHOLE) E::store(sum + v * 8, h[i]);
                else store_row<E>(sum, v * 8, a.H, h[i]);
            }
        }
        if constexpr (WAVE) s[0] = wave_sum(s[0]);
        else block_sums<1>(s, part[turn]);
        const RowScale scale(__builtin_fma(s[0], a.per, a.eps));
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * lanes + lane;
            if (v >= vecs) continue;
            put_norm<E, FORMAT>(a, rank, t, (int64_t)v * 8, h[i], w[i], scale);
        }
    }
}

// Rows wider than the registers, eight elements at a time: the second pass reads what the first has read
// or, of an addition, written (each thread its own elements, so that sum and out may
// be x or the residual).
template <typename E, int FORMAT>
__global__ __launch_bounds__(1024) void k_norm_any(const NormArgs a) {
    __shared__ double part[2][1024 / kWave][1];
    if (status_at_entry(a.status)) return;
    clear_parts(part);
    typedef typename E::scalar scalar;
    typedef typename E::vec vec;
    const int rank = blockIdx.y;
    const int64_t end = FORMAT ? mx_padded(a.H) : a.H;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const scalar *x = (const scalar *)a.x[rank] + t * a.H;
        const scalar *residual = (const scalar *)a.residual[rank] + t * a.H;
        scalar *sum = (scalar *)a.sum[rank] + t * a.H;
        const auto added = [&](int64_t c) {
            vec h = load_row<E>(x, c, a.H);
            if (a.has_residual) {
                const vec r = load_row<E>(residual, c, a.H);
#pragma unroll
                for (int i = 0; i < 8; i++) E::set(h, i, E::get(h, i) + E::get(r, i));
            }
            return h;
        };
        double s[1] = {0.0};
        for (int64_t c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
            const vec h = added(c);
            if (a.has_sum) store_row<E>(sum, c, a.H, h);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const double d = E::get(h, i);
                s[0] = __builtin_fma(d, d, s[0]);
            }
        }
        block_sums<1>(s, part[turn]);
        const RowScale scale(__builtin_fma(s[0], a.per, a.eps));
        // whole quads of lanes: `end` is a multiple of 32 where blocks are made
        for (int64_t c = threadIdx.x * 8; c < end; c += blockDim.x * 8) {
            const vec h = a.has_sum ? load_row<E>(sum, c, a.H) : added(c);
            Weights w;
            w.template set<E>(load_row<E>((const scalar *)a.weight, c, a.H));
            put_norm<E, FORMAT>(a, rank, t, c, h, w, scale);
        }
    }
}

// ------------------------------------------------------------------ gradient
struct NormGradArgs {
    const void *x[A2AV_MAX_W];
    const void *d_out[A2AV_MAX_W];
    const void *d_sum[A2AV_MAX_W];
    void *d_x[A2AV_MAX_W];
    const void *weight;
    float *part;      // [groups][H]
    float *d_weight;  // [H]
    const int32_t *status;
    int64_t T, H, rows;  // rows: of all ranks
    double eps, per;  // per: 1 / H
    int groups;
    int has_d_sum, has_d_weight;
};

// A workgroup takes rows g, g + groups, ... (MOST 64: each of its waves those of its
// own); each is read once, the next before this one's sums are waited for, and its
// products with d_out are added to the weight's sums in registers. Bound by the bytes:
// 8 x 2048 rows of 7168 in bf16 with d_sum 162 us with the sums' kernel, 5.8 TB/s (176
// without the loads ahead), 8 x 8192 of 2048 182, 5.9.
template <typename E, int VPT, int MOST, bool WHOLE>
__global__ __launch_bounds__(MOST == kWave ? 256 : MOST) void k_norm_grad_row(const NormGradArgs a) {
    constexpr bool WAVE = MOST == kWave, kNext = MOST < 1024 && VPT <= 2;  // registers for the next row
    __shared__ double part[2][1024 / kWave][2];
    __shared__ float waves[WAVE ? 3 : 1][WAVE ? VPT * 512 : 1];
    if (status_at_entry(a.status)) return;
    clear_parts(part);
    typedef typename E::scalar scalar;
    typedef typename E::vec vec;
    const int lanes = WAVE ? kWave : blockDim.x, lane = WAVE ? threadIdx.x % kWave : threadIdx.x;
    const int wave = threadIdx.x / kWave;
    const int64_t step = WAVE ? gridDim.x * 4 : gridDim.x;
    const int own = (int)((a.H + 7) / 8);  // a lane behind the row loads its last vector again, and counts 0
    float dw[VPT][8] = {};
    vec w[VPT], h[VPT], g[VPT], d[VPT], h1[VPT], g1[VPT], d1[VPT];
    const auto load = [&](vec(&to)[VPT], const scalar *p) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int c = min(i * lanes + lane, own - 1) * 8;
            if constexpr (WHOLE) to[i] = E::load(p + c);
            else to[i] = load_row<E>(p, c, a.H);
        }
    };
    const auto load_all = [&](vec(&x)[VPT], vec(&y)[VPT], vec(&z)[VPT], int64_t row) __attribute__((always_inline)) {
        const int64_t rank = row / a.T, at = (row - rank * a.T) * a.H;
        load(x, (const scalar *)a.x[rank] + at);
        load(y, (const scalar *)a.d_out[rank] + at);
        if (a.has_d_sum) load(z, (const scalar *)a.d_sum[rank] + at);
    };
    load(w, (const scalar *)a.weight);
    int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (kNext && row < a.rows) load_all(h1, g1, d1, row);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        if constexpr (kNext) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                h[i] = h1[i];
                g[i] = g1[i];
                d[i] = d1[i];
            }
            if (row + step < a.rows) load_all(h1, g1, d1, row + step);
        } else {
            load_all(h, g, d, row);
        }
        double s[2] = {0.0, 0.0};
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            if (i * lanes + lane >= own) h[i] = g[i] = vec{};  // (an infinite g times 0 is NaN)
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const double hc = E::get(h[i], c);
                s[0] = __builtin_fma(hc, hc, s[0]);
                // In 16 bits the product is exact in fp32, inside the range that the elements' fp32
                // below needs too (in double 8 x 2048 rows of 7168 in bf16 take 172 us, 162 so).
                const double gw = E::kExact ? (double)(E::get(g[i], c) * E::get(w[i], c))
                                            : (double)E::get(g[i], c) * (double)E::get(w[i], c);
                s[1] = __builtin_fma(gw, hc, s[1]);
            }
        }
        if constexpr (WAVE) {
            s[0] = wave_sum(s[0]);
            s[1] = wave_sum(s[1]);
        } else {
            block_sums<2>(s, part[turn]);
        }
        const double rd = inverse_root(__builtin_fma(s[0], a.per, a.eps));
        const float r = (float)rd, m = (float)(rd * rd * (s[1] * a.per));
        const int64_t rank = row / a.T, t = row - rank * a.T;
        scalar *d_x = (scalar *)a.d_x[rank] + t * a.H;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * lanes + lane;
            if (v >= own) continue;
            vec o;
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const float hc = E::get(h[i], c), gc = E::get(g[i], c);
                dw[i][c] += gc * (hc * r);
                float y = r * (gc * E::get(w[i], c) - hc * m);
                if (a.has_d_sum) y += E::get(d[i], c);
                E::set(o, c, y);
            }
            if constexpr (WHOLE) E::store(d_x + v * 8, o);
            else store_row<E>(d_x, v * 8, a.H, o);
        }
    }
    if (!a.has_d_weight) return;
    if constexpr (WAVE) {
        // the four waves' sums, in order
        if (wave > 0)
#pragma unroll
            for (int i = 0; i < VPT; i++)
#pragma unroll
                for (int c = 0; c < 8; c++) waves[wave - 1][(i * 8 + c) * kWave + lane] = dw[i][c];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int k = 0; k < 3; k++)
#pragma unroll
            for (int i = 0; i < VPT; i++)
#pragma unroll
                for (int c = 0; c < 8; c++) dw[i][c] += waves[k][(i * 8 + c) * kWave + lane];
    }
    float *p = a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int v = i * lanes + lane;
        if (v >= own) continue;
        const ElemF32::vec o = {{dw[i][0], dw[i][1], dw[i][2], dw[i][3]}, {dw[i][4], dw[i][5], dw[i][6], dw[i][7]}};
        store_row<ElemF32>(p, v * 8, a.H, o);
    }
}

// Rows wider than the registers: the weight's sums of a workgroup stay in its part
// of the workspace, each thread adding to its own columns.
template <typename E>
__global__ __launch_bounds__(1024) void k_norm_grad_any(const NormGradArgs a) {
    __shared__ double part[2][1024 / kWave][2];
    if (status_at_entry(a.status)) return;
    clear_parts(part);
    typedef typename E::scalar scalar;
    typedef typename E::vec vec;
    const scalar *weight = (const scalar *)a.weight;
    float *p = a.part + (int64_t)blockIdx.x * a.H;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const int64_t rank = row / a.T, t = row - rank * a.T;
        const scalar *x = (const scalar *)a.x[rank] + t * a.H, *d_out = (const scalar *)a.d_out[rank] + t * a.H;
        const scalar *d_sum = (const scalar *)a.d_sum[rank] + t * a.H;
        scalar *d_x = (scalar *)a.d_x[rank] + t * a.H;
        double s[2] = {0.0, 0.0};
        for (int64_t c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
            const vec h = load_row<E>(x, c, a.H), g = load_row<E>(d_out, c, a.H), w = load_row<E>(weight, c, a.H);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const double hc = E::get(h, i);
                s[0] = __builtin_fma(hc, hc, s[0]);
                s[1] = __builtin_fma((double)E::get(g, i) * (double)E::get(w, i), hc, s[1]);
            }
        }
        block_sums<2>(s, part[turn]);
        const double rd = inverse_root(__builtin_fma(s[0], a.per, a.eps));
        const float r = (float)rd, m = (float)(rd * rd * (s[1] * a.per));
        for (int64_t c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
            const vec h = load_row<E>(x, c, a.H), g = load_row<E>(d_out, c, a.H), w = load_row<E>(weight, c, a.H);
            vec o = {}, d = {};
            if (a.has_d_sum) d = load_row<E>(d_sum, c, a.H);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float hc = E::get(h, i), gc = E::get(g, i);
                float y = r * (gc * E::get(w, i) - hc * m);
                if (a.has_d_sum) y += E::get(d, i);
                E::set(o, i, y);
                if (a.has_d_weight && c + i < a.H) p[c + i] = (row == blockIdx.x ? 0.0f : p[c + i]) + gc * (hc * r);
            }
            store_row<E>(d_x, c, a.H, o);
        }
    }
}

// 32 columns by 32 runs of the workgroups' sums, then the runs in order.
__global__ __launch_bounds__(1024) void k_norm_weight(const NormGradArgs a) {
    __shared__ float run[32][33];
    if (status_at_entry(a.status)) return;
    const int col = threadIdx.x % 32, k = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    float s = 0.0f;
    if (c < a.H) {
        const int per = (a.groups + 31) / 32, from = k * per, to = min(from + per, a.groups);
#pragma unroll 16
        for (int g = from; g < to; g++) s += a.part[(int64_t)g * a.H + c];
    }
    run[k][col] = s;
    __syncthreads();
    if (k != 0 || c >= a.H) return;
#pragma unroll
    for (int i = 1; i < 32; i++) s += run[i][col];
    a.d_weight[c] = s;
}

// ------------------------------------------------------------------ host
static bool norm_sizes(int W, int64_t T, int64_t H, int type) {
    return W >= 1 && W <= A2AV_MAX_W && T >= 0 && T <= (int64_t)1 << 30 && H >= 1 && H <= A2AV_MAX_WIDTH &&
           type >= A2AV_DT_F32 && type <= A2AV_DT_F16;
}
static bool at16(const void *p) { return (uintptr_t)p % 16 == 0; }

// Rows of the register kernels: up to 1024 threads of two vectors.
static bool in_registers(int64_t H) { return H <= 1024 * 2 * 8; }
static int64_t up_to(int64_t x, int64_t most) { return x < most ? x : most; }
// Waves of the gradient, whose workgroups have sums of their own (2048, 4096 and 8192: 16384
// rows of 2048 in bf16 52, 56 and 66 us, of 7168 155, 162 and 172, of 512 25, 21 and 25, of
// 16384 495, 365 and 367).
constexpr int kGradWaves = 4096;

// A launch of a kernel that goes through `rows` rows (of each of W ranks): a few times
// the workgroups that the compute units hold at once (8 x 2048 rows of 7168 in bf16,
// residual and 8-bit rows: 162 us with as many, 154 with twice, 149 with four times, 162
// with one for every row; 8 x 8192 rows of 2048, two waves each: 203, 200, 194, 172).
template <typename K, typename A>
static void launch_rows(K kernel, const A &a, int64_t rows, int W, int threads, hipStream_t stream) {
    int held = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&held, kernel, threads, 0) != hipSuccess || held < 1) held = 1;
    const int64_t fill = up_to(max_grid(), (int64_t)held * device_cu_count(stream) * (threads >= 256 ? 4 : 16)) / W;
    hipLaunchKernelGGL(kernel, dim3((unsigned)up_to(rows, fill > 0 ? fill : 1), W), dim3(threads), 0, stream, a);
}

// How a row is spread: a wave each up to 1024 elements, else a workgroup of just
// enough waves; two vectors a thread leave registers for the next row's, but few rows
// of whole vectors are sooner done with one (one or two, in bf16 with residual and 8-bit
// rows: 1 row of 4096 2.8 or 3.4 us, 1024 6.6 or 7.1, 4096 22.0 or 22.4, 16384 83.3 or
// 82.2; of 7168 3.7 or 3.9, 13.6 or 12.5, 44 or 41, 159 or 145).
template <typename E, int FORMAT, bool WHOLE>
static void launch_norm(const NormArgs &a, int W, hipStream_t stream) {
    const int64_t vecs = (FORMAT ? mx_padded(a.H) : a.H + 7) / 8;
    const bool wave = vecs <= 128;
    const int per = !WHOLE ? 2 : wave ? (vecs <= 64 ? 1 : 2) : vecs <= 1024 && W * a.T < 2048 ? 1 : 2;
    const int threads = wave ? 256 : (int)((vecs + per * kWave - 1) / (per * kWave) * kWave);
    if constexpr (WHOLE) {
        if (wave && per == 1) {
            launch_rows(k_norm_row<E, FORMAT, 1, kWave, true>, a, (a.T + 3) / 4, W, threads, stream);
            return;
        }
        if (per == 1) {
            launch_rows(k_norm_row<E, FORMAT, 1, 1024, true>, a, a.T, W, threads, stream);
            return;
        }
    }
    if (wave) launch_rows(k_norm_row<E, FORMAT, 2, kWave, WHOLE>, a, (a.T + 3) / 4, W, threads, stream);
    else if (threads <= 512) launch_rows(k_norm_row<E, FORMAT, 2, 512, WHOLE>, a, a.T, W, threads, stream);
    else launch_rows(k_norm_row<E, FORMAT, 2, 1024, WHOLE>, a, a.T, W, threads, stream);
}
template <typename E, int FORMAT>
static void launch_norm(const NormArgs &a, int W, hipStream_t stream) {
    if (!in_registers(a.H)) launch_rows(k_norm_any<E, FORMAT>, a, a.T, W, 1024, stream);
    else if (a.H % 8 == 0) launch_norm<E, FORMAT, true>(a, W, stream);
    else launch_norm<E, FORMAT, false>(a, W, stream);
}
template <typename E>
static void launch_norm(const NormArgs &a, int W, int format, hipStream_t stream) {
    if (format == A2AV_MX_FP8) launch_norm<E, A2AV_MX_FP8>(a, W, stream);
    else if (format == A2AV_MX_FP4) launch_norm<E, A2AV_MX_FP4>(a, W, stream);
    else launch_norm<E, 0>(a, W, stream);
}

// The gradient's: a wave each up to 1024 elements, and of many rows up to 2048 (fewer
// workgroups, whose weight sums have to be read again; a wave or a workgroup a row: 64
// rows of 1536 in bf16 6.7 or 5.9 us, 512 8.6 or 8.5, 2048 12 or 20, 16384 47 or 55; 64 of
// 1111 11.9 or 9.4, 1021 15 or 19, 16384 99 or 134; in fp32 64 of 2048 7.2 or 6.1, 2048 23
// or 31, 16384 119 or 123), else a workgroup with two vectors a thread, which leaves
// registers for the next row's, and one where there are few rows of whole vectors (one or
// two, in bf16: 1 row of 7168 6.3 or 6.3 us, 1024 20.9 or 21.4, 4096 53 or 51, 16384 177
// or 163; of 4096 5.6 or 5.8, 14 or 20, 31 or 37, 97 or 112).
struct GradShape {
    bool wave;
    int per, threads;
    int64_t groups, most;
};
static GradShape grad_shape(int W, int64_t T, int64_t H) {
    const int64_t vecs = (H + 7) / 8, rows = (int64_t)W * T;
    const bool whole = H % 8 == 0;
    GradShape s = {};
    s.wave = vecs <= 128 || (vecs <= 256 && rows > 512);
    s.per = !whole ? (s.wave && vecs > 128 ? 4 : 2) : s.wave ? (int)((vecs + kWave - 1) / kWave) : vecs <= 1024 && rows < 2048 ? 1 : 2;
    if (!in_registers(H)) s.threads = 1024;
    else s.threads = s.wave ? 256 : (int)((vecs + s.per * kWave - 1) / (s.per * kWave) * kWave);
    s.most = up_to(rows, kGradWaves / (s.threads / kWave) / 256 * 256);
    s.groups = up_to(s.wave ? (rows + 3) / 4 : rows, s.most);
    return s;
}

template <typename E>
static void launch_grad(const NormGradArgs &a, int W, hipStream_t stream) {
    const GradShape s = grad_shape(W, a.T, a.H);
    const dim3 g((unsigned)a.groups), b((unsigned)s.threads);
    if (!in_registers(a.H)) hipLaunchKernelGGL(k_norm_grad_any<E>, g, b, 0, stream, a);
    else if (a.H % 8 != 0 && s.wave && s.per == 2)
        hipLaunchKernelGGL((k_norm_grad_row<E, 2, kWave, false>), g, b, 0, stream, a);
    else if (a.H % 8 != 0 && s.wave) hipLaunchKernelGGL((k_norm_grad_row<E, 4, kWave, false>), g, b, 0, stream, a);
    else if (a.H % 8 != 0 && b.x <= 512) hipLaunchKernelGGL((k_norm_grad_row<E, 2, 512, false>), g, b, 0, stream, a);
    else if (a.H % 8 != 0) hipLaunchKernelGGL((k_norm_grad_row<E, 2, 1024, false>), g, b, 0, stream, a);
    else if (s.wave && s.per == 1) hipLaunchKernelGGL((k_norm_grad_row<E, 1, kWave, true>), g, b, 0, stream, a);
    else if (s.wave && s.per == 2) hipLaunchKernelGGL((k_norm_grad_row<E, 2, kWave, true>), g, b, 0, stream, a);
    else if (s.wave) hipLaunchKernelGGL((k_norm_grad_row<E, 4, kWave, true>), g, b, 0, stream, a);
    else if (s.per == 1) hipLaunchKernelGGL((k_norm_grad_row<E, 1, 1024, true>), g, b, 0, stream, a);
    else if (b.x <= 512) hipLaunchKernelGGL((k_norm_grad_row<E, 2, 512, true>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((k_norm_grad_row<E, 2, 1024, true>), g, b, 0, stream, a);
}

}  // namespace a2av

using namespace a2av;

A2AV_API int moe_rms_norm(int W, int64_t T, int64_t H, int type, double eps, const void *const *x,
                          const void *const *residual, const void *weight, void *const *sum,
                          void *const *out, void *const *rows, int format, int32_t *status,
                          hipStream_t stream) {
    if (!norm_sizes(W, T, H, type) || !(eps >= 0.0) || !x || !weight || !status) return A2AV_EARG;
    if ((!out && !rows) || (sum && !residual)) return A2AV_EARG;
    if (format != A2AV_MX_FP8 && format != A2AV_MX_FP4) return A2AV_EARG;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int d = 0; d < W && T > 0; d++) {
        if (!x[d] || (residual && !residual[d]) || (sum && !sum[d]) || (out && !out[d]) || (rows && !rows[d]))
            return A2AV_EARG;
        if (rows && (!at16(rows[d]) || rows[d] == x[d] || (residual && rows[d] == residual[d]) ||
                     (sum && rows[d] == sum[d]) || (out && rows[d] == out[d])))
            return A2AV_EARG;
        if (sum && out && sum[d] == out[d]) return A2AV_EARG;
        a.x[d] = x[d];
        a.residual[d] = residual ? residual[d] : nullptr;
        a.sum[d] = sum ? sum[d] : nullptr;
        a.out[d] = out ? out[d] : nullptr;
        a.rows[d] = rows ? (unsigned char *)rows[d] : nullptr;
    }
    if (T == 0) return A2AV_OK;
    a.weight = weight;
    a.status = status;
    a.T = T;
    a.H = H;
    a.eps = eps;
    a.per = 1.0 / (double)H;
    a.has_residual = residual != nullptr;
    a.has_sum = sum != nullptr;
    a.has_out = out != nullptr;
    if (!rows) format = 0;
    if (type == A2AV_DT_F32) launch_norm<ElemF32>(a, W, format, stream);
    else if (type == A2AV_DT_BF16) launch_norm<ElemBf16>(a, W, format, stream);
    else launch_norm<ElemF16>(a, W, format, stream);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}

A2AV_API size_t moe_rms_norm_backward_workspace_bytes(int W, int64_t T, int64_t H) {
    if (!norm_sizes(W, T, H, A2AV_DT_F32)) return 0;
    return ((size_t)grad_shape(W, T, H).most * (size_t)H * 4 + 255) / 256 * 256 + 256;
}

A2AV_API int moe_rms_norm_backward(int W, int64_t T, int64_t H, int type, double eps,
                                   const void *const *x, const void *weight,
                                   const void *const *d_out, const void *const *d_sum,
                                   void *const *d_x, float *d_weight, void *workspace,
                                   size_t workspace_bytes, int32_t *status, hipStream_t stream) {
    if (!norm_sizes(W, T, H, type) || !(eps >= 0.0) || !x || !weight || !d_out || !d_x || !status) return A2AV_EARG;
    if (!workspace || !at16(workspace) || workspace_bytes < moe_rms_norm_backward_workspace_bytes(W, T, H))
        return A2AV_EARG;
    NormGradArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int d = 0; d < W && T > 0; d++) {
        if (!x[d] || !d_out[d] || !d_x[d] || (d_sum && !d_sum[d])) return A2AV_EARG;
        a.x[d] = x[d];
        a.d_out[d] = d_out[d];
        a.d_sum[d] = d_sum ? d_sum[d] : nullptr;
        a.d_x[d] = d_x[d];
    }
    if (T == 0 && !d_weight) return A2AV_OK;
    a.weight = weight;
    a.part = (float *)workspace;
    a.d_weight = d_weight;
    a.status = status;
    a.T = T;
    a.H = H;
    a.rows = (int64_t)W * T;
    a.eps = eps;
    a.per = 1.0 / (double)H;
    a.groups = (int)up_to(grad_shape(W, T, H).groups, max_grid());
    a.has_d_sum = d_sum != nullptr;
    a.has_d_weight = d_weight != nullptr;
    if (T > 0) {
        if (type == A2AV_DT_F32) launch_grad<ElemF32>(a, W, stream);
        else if (type == A2AV_DT_BF16) launch_grad<ElemBf16>(a, W, stream);
        else launch_grad<ElemF16>(a, W, stream);
    }
    if (d_weight)
        hipLaunchKernelGGL(k_norm_weight, dim3((unsigned)((H + 31) / 32)), dim3(1024), 0, stream, a);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
