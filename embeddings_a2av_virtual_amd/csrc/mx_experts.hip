// mx_experts.hip — the experts' products on microscaled rows with 4-bit weights
// (gfx950).
//
// out = act(x . W_e^T + b_e) on expert-major rows, x in e4m3 or e2m1 blocks and
// W_e in e2m1 blocks of 32 with a scale each: the block-scaled matrix
// instructions take both operands as they lie and multiply by the scales, with
// fp32 sums.
//
//   k_mx_plain   one 64 x 128 tile, operands straight from memory
#include <hip/hip_runtime.h>

#include <cstring>

#include "experts.hpp"
#include "mx.hpp"

namespace a2av {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// out's element type
enum { kOutBf16, kOutF16, kOutMx };

struct MxExpertArgs {
    const unsigned char *x[A2AV_MAX_W];
    const unsigned char *weight[A2AV_MAX_W];
    const float *bias[A2AV_MAX_W];
    void *out[A2AV_MAX_W];
    const int64_t *offsets;
    const int32_t *tiles;
    const int32_t *first;
    const int32_t *status;
    int64_t K, N, NW;
    int64_t x_stride, w_stride, out_stride;  // bytes of a row; of out if microscaled
    int W, P;
    int act, out_type, has_bias;
    int wide;  // out and bias by 16-byte vectors
    int cols;  // column tiles
};

// The first operand's rows are the weight's (e2m1), the second's x's; a lane has
// the fp32 sums of x row lane % 32 (or 16).
template <int FORMAT>
__device__ __forceinline__ f32x16 mfma32(i32x4 w, i32x8 x, f32x16 c, int sw, int sx) {
    const i32x8 w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, x, c, 4, FORMAT == A2AV_MX_FP8 ? 0 : 4, 0, sw, 0, sx);
}

// ------------------------------------------------------------------ epilogue
// The sums of a wave leave through its part of LDS, so that one lane gets 8
// neighbouring columns of a row and a quad of lanes a block of 32: ROWS rows of
// COLS fp32 sums, the 16-byte chunks of a row permuted by the row.
template <int COLS>
__device__ __forceinline__ int chunk(int r, int at) {
    return r * (COLS / 4) + (at ^ (r & 15 & (COLS / 4 - 1)));
}

// Into LDS: one 32 x 32 block, u-th by rows and v-th by columns.
template <int COLS>
__device__ __forceinline__ void put_sums(f32x4 *sums, int u, int v, const f32x16 &acc, int lane) {
#pragma unroll
    for (int g = 0; g < 4; g++)
        sums[chunk<COLS>(u * 32 + (lane & 31), v * 8 + g * 2 + (lane >> 5))] =
            f32x4{acc[g * 4], acc[g * 4 + 1], acc[g * 4 + 2], acc[g * 4 + 3]};
}

// Eight outputs y of row `row`, columns n .. n + 7; every lane of a quad comes
// here together with the same row and its own eight columns of a block of 32.
__device__ __forceinline__ void put_out(const MxExpertArgs &a, int d, int64_t row, int64_t n, float (&y)[8]) {
    if (a.out_type == kOutMx) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (n + i >= a.N) y[i] = 0.0f;
        int scale;
        const auto e = mx_block<A2AV_MX_FP8>(y, scale);
        unsigned char *out = (unsigned char *)a.out[d] + row * a.out_stride;
        *(u32x2 *)(out + n) = e;
        if (n % kMxBlock == 0) out[mx_padded(a.N) + n / kMxBlock] = (unsigned char)scale;
        return;
    }
    uint16_t *out = (uint16_t *)a.out[d] + row * a.N + n;
    if (a.wide) {
        if (a.out_type == kOutBf16) put8<Bf16>(out, y);
        else put8<Fp16>(out, y);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (n + i < a.N) out[i] = a.out_type == kOutBf16 ? Bf16::from_float(y[i]) : Fp16::from_float(y[i]);
}

__device__ __forceinline__ void add_bias(const MxExpertArgs &a, const float *bias, int64_t n, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (a.wide || n + i < a.N) y[i] += bias[n + i];
}

// The rows of a pass; `row_of(r)` is the expert's row behind LDS row r, c0 the
// first product column of the wave.
template <int ROWS, int COLS, typename RowOf>
__device__ __forceinline__ void emit(const MxExpertArgs &a, const f32x4 *sums, int d, int j, int64_t row0, int64_t M,
                                     int64_t c0, int lane, RowOf row_of) {
    const bool glu = a.act == A2AV_ACT_SWIGLU;
    const int per = glu ? COLS / 16 : COLS / 8;  // lanes a row
    const int64_t end = a.out_type == kOutMx ? mx_padded(a.N) : a.N;
    const float *bias = a.bias[d] + (int64_t)j * a.NW;
    const auto take = [&](int r, int at, float(&y)[8]) {
        const f32x4 lo = sums[chunk<COLS>(r, at)], hi = sums[chunk<COLS>(r, at + 1)];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            y[i] = lo[i];
            y[i + 4] = hi[i];
        }
    };
    for (int r = lane / per; r < ROWS; r += kWave / per) {
        const int64_t m = row_of(r);
        if (m >= M) continue;
        const int q = lane % per;
        const int64_t n = (glu ? c0 / 2 : c0) + q * 8;
        if (n >= end) continue;
        float y[8];
        // gated: blocks of 16 gate and 16 up columns alternate
        take(r, glu ? (q >> 1) * 8 + (q & 1) * 2 : q * 2, y);
        if (a.has_bias) add_bias(a, bias, n, y);
        if (glu) {
            float up[8];
            take(r, (q >> 1) * 8 + (q & 1) * 2 + 4, up);
            if (a.has_bias) add_bias(a, bias + a.N, n, up);
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = y[i] * sigmoid(y[i]) * up[i];
        } else if (a.act != A2AV_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = act_of(a.act, y[i]);
        }
        put_out(a, d, row0 + m, n, y);
    }
}

// ------------------------------------------------------------------ products
// One 64 x 128 tile by four waves of 32 x 64; every lane loads its own 16 bytes
// of each operand and the four scales of its row's 128 elements.
template <int FORMAT>
__global__ __launch_bounds__(256) void k_mx_plain(const MxExpertArgs a) {
    __shared__ f32x4 sums[4][32 * 16];
    if (status_at_entry(a.status)) return;
    const int t = blockIdx.y + gridDim.y * blockIdx.z;
    if (t >= a.tiles[0]) return;
    const int e = a.tiles[2 + 2 * t], mt = a.tiles[3 + 2 * t];
    const int d = e / a.P, j = e - d * a.P;
    const int64_t row0 = a.offsets[(int64_t)d * (a.P + 1) + j];
    const int64_t M = a.offsets[(int64_t)d * (a.P + 1) + j + 1] - row0;
    const bool glu = a.act == A2AV_ACT_SWIGLU;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, half = lane >> 5;
    const int64_t m0 = (int64_t)mt * 64 + (wave >> 1) * 32, c0 = (int64_t)blockIdx.x * 128 + (wave & 1) * 64;
    const int64_t m = m0 + (lane & 31);
    const bool in_m = m < M;
    const unsigned char *x = a.x[d] + (row0 + (in_m ? m : 0)) * a.x_stride;
    const unsigned char *w[2];
    bool in_c[2];
#pragma unroll
    for (int v = 0; v < 2; v++) {
        const int64_t c = c0 + v * 32 + (lane & 31), n = weight_row(c, a.N, glu);
        in_c[v] = glu ? n - ((c >> 4) & 1) * a.N < a.N : n < a.N;
        w[v] = a.weight[d] + ((int64_t)j * a.NW + (in_c[v] ? n : 0)) * a.w_stride;
    }
    const int64_t steps = mx_padded(a.K) / 128, x_scales = mx_element_bytes(FORMAT, a.K), w_scales = mx_padded(a.K) / 2;
    constexpr int kBytes = FORMAT == A2AV_MX_FP8 ? 128 : 64;  // of 128 elements
    f32x16 acc[2] = {};
    for (int64_t s = 0; s < steps; s++) {
        const uint32_t sx = *(const uint32_t *)(x + x_scales + s * 4) >> (half * 8);
#pragma unroll
        for (int q = 0; q < 2; q++) {
            i32x8 fx = {};
            if constexpr (FORMAT == A2AV_MX_FP8) {
                // a half wave has elements 16 h .. + 15 and 32 + 16 h .. + 15 of the 64
                const i32x4 lo = *(const i32x4 *)(x + s * kBytes + q * 64 + half * 16);
                const i32x4 hi = *(const i32x4 *)(x + s * kBytes + q * 64 + 32 + half * 16);
                fx = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
                const i32x4 lo = *(const i32x4 *)(x + s * kBytes + q * 32 + half * 16);
                fx = __builtin_shufflevector(lo, lo, 0, 1, 2, 3, 0, 1, 2, 3);
            }
            if (!in_m) fx = i32x8{};
#pragma unroll
            for (int v = 0; v < 2; v++) {
                i32x4 fw = *(const i32x4 *)(w[v] + s * 64 + q * 32 + half * 16);
                const uint32_t sw = *(const uint32_t *)(w[v] + w_scales + s * 4) >> (half * 8);
                if (!in_c[v]) fw = i32x4{};
                acc[v] = mfma32<FORMAT>(fw, fx, acc[v], in_c[v] ? (int)(sw >> q * 16) & 255 : 0,
                                        in_m ? (int)(sx >> q * 16) & 255 : 0);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < 2; v++) put_sums<64>(sums[wave], 0, v, acc[v], lane);
    asm volatile("" ::: "memory");
    emit<32, 64>(a, sums[wave], d, j, row0, M, c0, lane, [&](int r) { return m0 + r; });
}

// ------------------------------------------------------------------ host
// Product columns that have outputs: with microscaled rows their padding too.
static int64_t product_columns(const MxExpertArgs &a) {
    const int64_t n = a.out_type == kOutMx ? mx_padded(a.N) : a.N;
    return a.act == A2AV_ACT_SWIGLU ? (n + 15) / 16 * 32 : n;
}

}  // namespace a2av

using namespace a2av;

A2AV_API size_t moe_expert_linear_mx_workspace_bytes(int W, int P, int64_t K, int64_t N, int act,
                                                     const int64_t *x_rows) {
    Layout l;
    return plan_layout(W, P, K, N, act, x_rows, false, &l) ? l.total : 0;
}

A2AV_API int moe_expert_linear_mx(int W, int P, int64_t K, int64_t N, int x_format, int act,
                                  const void *const *x, const int64_t *x_rows,
                                  const int64_t *expert_offsets, const void *const *weight,
                                  const float *const *bias, void *const *out, int out_type,
                                  void *workspace, size_t workspace_bytes, int32_t *status,
                                  hipStream_t stream) {
    Layout l;
    if (!plan_layout(W, P, K, N, act, x_rows, false, &l)) return A2AV_EARG;
    if ((x_format != A2AV_MX_FP8 && x_format != A2AV_MX_FP4) || !x || !expert_offsets || !weight || !out || !status)
        return A2AV_EARG;
    if (out_type != A2AV_DT_BF16 && out_type != A2AV_DT_F16 && out_type != A2AV_MX_FP8) return A2AV_EARG;
    if (!workspace || (uintptr_t)workspace % 8 != 0 || workspace_bytes < l.total) return A2AV_EARG;
    MxExpertArgs a;
    std::memset(&a, 0, sizeof(a));
    a.K = K;
    a.N = N;
    a.NW = act == A2AV_ACT_SWIGLU ? 2 * N : N;
    a.x_stride = mx_stride(x_format, K);
    a.w_stride = mx_stride(A2AV_MX_FP4, K);
    a.out_stride = mx_stride(A2AV_MX_FP8, N);
    a.act = act;
    a.out_type = out_type == A2AV_DT_BF16 ? kOutBf16 : out_type == A2AV_DT_F16 ? kOutF16 : kOutMx;
    a.has_bias = bias != nullptr;
    a.wide = N % 8 == 0;
    for (int d = 0; d < W; d++) {
        if (!fits(x_rows[d], a.x_stride) || !fits(x_rows[d], a.out_stride)) return A2AV_EARG;
        if (!weight[d] || !aligned16(weight[d]) || (bias && !bias[d])) return A2AV_EARG;
        if (x_rows[d] > 0 && (!x[d] || !out[d] || out[d] == x[d] || !aligned16(x[d]))) return A2AV_EARG;
        if (x_rows[d] > 0 && a.out_type == kOutMx && !aligned16(out[d])) return A2AV_EARG;
        a.x[d] = (const unsigned char *)x[d];
        a.weight[d] = (const unsigned char *)weight[d];
        a.bias[d] = bias ? bias[d] : nullptr;
        a.out[d] = out[d];
        a.wide = a.wide && aligned16(a.bias[d]) && aligned16(out[d]);
    }
    a.offsets = expert_offsets;
    a.tiles = (const int32_t *)workspace;
    a.first = (const int32_t *)((unsigned char *)workspace + l.first);
    a.status = status;
    a.W = W;
    a.P = P;
    launch_plan(W, P, x_rows, expert_offsets, 64, (unsigned char *)workspace, l, status, stream);
    const int64_t tiles = most_tiles(x_rows, W, P, 64), y = tiles < 32768 ? tiles : 32768;
    a.cols = (int)((product_columns(a) + 127) / 128);
    const dim3 g((unsigned)a.cols, (unsigned)y, (unsigned)((tiles + y - 1) / y));
    if (x_format == A2AV_MX_FP8) hipLaunchKernelGGL(k_mx_plain<A2AV_MX_FP8>, g, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(k_mx_plain<A2AV_MX_FP4>, g, dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
