// norm.hip — the root-mean-square norm in front of the router, with the
// residual's addition and its rows in 16 or 32 bits or microscaled for the
// dispatch, and its gradient (gfx950).
//
//   h = x + residual (rounded to the type)      r = 1 / sqrt(mean(h^2) + eps)
//   y = h * r * weight
//   d_x = r * (d_y * weight - h * r^2 * mean(d_y * weight * h)) + d_h
//   d_weight = sum over rows of d_y * h * r
//
//   k_norm_row        rows of 16-byte vectors, each held in a workgroup's registers
//   k_norm_any        rows of any width and alignment, read twice
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
    double eps;
    int format;
    int has_residual, has_sum, has_out, has_rows;
};

// A lane's eight values as elements of vector `vec` of a microscaled row.
template <int FORMAT>
__device__ __forceinline__ void put_block(unsigned char *row, int64_t vec, int64_t element_bytes, const double (&y)[8]) {
    int scale;
    const auto p = mx_block<FORMAT>(y, scale);
    *(typename Mx<FORMAT>::packed *)(row + vec * (int64_t)sizeof(p)) = p;
    if (threadIdx.x % 4 == 0) row[element_bytes + vec / 4] = (unsigned char)scale;
}
__device__ __forceinline__ void put_block(int format, unsigned char *row, int64_t vec, int64_t element_bytes,
                                          const double (&y)[8]) {
    if (format == A2AV_MX_FP8) put_block<A2AV_MX_FP8>(row, vec, element_bytes, y);
    else put_block<A2AV_MX_FP4>(row, vec, element_bytes, y);
}

// One workgroup per row, every thread VPT vectors of 8 elements; the row is read
// once. The mean and the values are in double: an element of 8 or 4 bits then
// comes out the same however the sum is ordered, and double costs what fp32
// does beside the row's bytes.
template <typename E, int BLOCK, int VPT>
__global__ __launch_bounds__(BLOCK) void k_norm_row(const NormArgs a) {
    __shared__ double part[BLOCK / kWave][1];
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const int rank = blockIdx.y;
    const int vecs = (int)(a.H / 8), padded = (int)(mx_padded(a.H) / 8);
    const int64_t stride = mx_stride(a.format, a.H), element_bytes = mx_element_bytes(a.format, a.H);
    const scalar *weight = (const scalar *)a.weight;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const scalar *x = (const scalar *)a.x[rank] + t * a.H;
        const scalar *residual = (const scalar *)a.residual[rank] + t * a.H;
        typename E::vec h[VPT], w[VPT];
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * BLOCK + threadIdx.x;
            if (v < vecs) {
                h[i] = E::load(x + v * 8);
                w[i] = E::load(weight + v * 8);
            }
        }
        if (a.has_residual) {
            typename E::vec r[VPT];
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int v = i * BLOCK + threadIdx.x;
                if (v < vecs) r[i] = E::load(residual + v * 8);
            }
#pragma unroll
            for (int i = 0; i < VPT; i++)
#pragma unroll
                for (int c = 0; c < 8; c++) E::set(h[i], c, E::get(h[i], c) + E::get(r[i], c));
        }
        double s[1] = {0.0};
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * BLOCK + threadIdx.x;
            if (v >= vecs) continue;
            if (a.has_sum) E::store((scalar *)a.sum[rank] + t * a.H + v * 8, h[i]);
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const double d = E::get(h[i], c);
                s[0] = __builtin_fma(d, d, s[0]);
            }
        }
        block_sums<BLOCK, 1>(s, part);
        const double r = 1.0 / sqrt(s[0] / (double)a.H + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * BLOCK + threadIdx.x;
            if (v >= padded) continue;
            double y[8];
#pragma unroll
            for (int c = 0; c < 8; c++)
                y[c] = v < vecs ? (double)E::get(h[i], c) * r * (double)E::get(w[i], c) : 0.0;
            if (a.has_out && v < vecs) {
                typename E::vec o;
#pragma unroll
                for (int c = 0; c < 8; c++) E::set(o, c, (float)y[c]);
                E::store((scalar *)a.out[rank] + t * a.H + v * 8, o);
            }
            if (a.has_rows) put_block(a.format, a.rows[rank] + t * stride, v, element_bytes, y);
        }
        if (BLOCK > kWave) __syncthreads();  // part is the next row's
    }
}

// Any width, element by element: the second pass reads what the first has read
// or, of an addition, written (each thread its own elements, so that sum and
// out may be x or the residual).
template <typename E>
__global__ __launch_bounds__(256) void k_norm_any(const NormArgs a) {
    __shared__ double part[4][1];
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const int rank = blockIdx.y;
    const int64_t stride = mx_stride(a.format, a.H), element_bytes = mx_element_bytes(a.format, a.H);
    const int64_t end = a.has_rows ? mx_padded(a.H) : a.H;
    const scalar *weight = (const scalar *)a.weight;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const scalar *x = (const scalar *)a.x[rank] + t * a.H;
        const scalar *residual = (const scalar *)a.residual[rank] + t * a.H;
        scalar *sum = (scalar *)a.sum[rank] + t * a.H, *out = (scalar *)a.out[rank] + t * a.H;
        const auto added = [&](int64_t i) {
            return a.has_residual ? E::from_float(E::to_float(x[i]) + E::to_float(residual[i])) : x[i];
        };
        double s[1] = {0.0};
        for (int64_t v = threadIdx.x; v * 8 < a.H; v += 256)
            for (int64_t i = v * 8; i < v * 8 + 8 && i < a.H; i++) {
                const scalar h = added(i);
                if (a.has_sum) sum[i] = h;
                const double d = E::to_float(h);
                s[0] = __builtin_fma(d, d, s[0]);
            }
        block_sums<256, 1>(s, part);
        const double r = 1.0 / sqrt(s[0] / (double)a.H + a.eps);
        // whole quads of lanes: `end` is a multiple of 32 where blocks are made
        for (int64_t v = threadIdx.x; v * 8 < end; v += 256) {
            double y[8];
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const int64_t i = v * 8 + c;
                y[c] = 0.0;
                if (i < a.H) {
                    y[c] = (double)E::to_float(a.has_sum ? sum[i] : added(i)) * r * (double)E::to_float(weight[i]);
                    if (a.has_out) out[i] = E::from_float((float)y[c]);
                }
            }
            if (a.has_rows) put_block(a.format, a.rows[rank] + t * stride, v, element_bytes, y);
        }
        __syncthreads();
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
    double eps;
    int groups;
    int has_d_sum, has_d_weight;
};

// A workgroup takes rows g, g + groups, ...; each is read once, and its
// products with d_out are added to the weight's sums in registers.
template <typename E, int BLOCK, int VPT>
__global__ __launch_bounds__(BLOCK) void k_norm_grad_row(const NormGradArgs a) {
    __shared__ double part[BLOCK / kWave][2];
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const int vecs = (int)(a.H / 8);
    const scalar *weight = (const scalar *)a.weight;
    float dw[VPT][8] = {};
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t rank = row / a.T, t = row - rank * a.T;
        const scalar *x = (const scalar *)a.x[rank] + t * a.H, *d_out = (const scalar *)a.d_out[rank] + t * a.H;
        const scalar *d_sum = (const scalar *)a.d_sum[rank] + t * a.H;
        typename E::vec h[VPT], g[VPT], w[VPT], d[VPT];
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * BLOCK + threadIdx.x;
            if (v < vecs) {
                h[i] = E::load(x + v * 8);
                g[i] = E::load(d_out + v * 8);
                w[i] = E::load(weight + v * 8);
                if (a.has_d_sum) d[i] = E::load(d_sum + v * 8);
            }
        }
        double s[2] = {0.0, 0.0};
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            if (i * BLOCK + (int)threadIdx.x >= vecs) continue;
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const double hc = E::get(h[i], c);
                s[0] = __builtin_fma(hc, hc, s[0]);
                s[1] = __builtin_fma((double)E::get(g[i], c) * (double)E::get(w[i], c), hc, s[1]);
            }
        }
        block_sums<BLOCK, 2>(s, part);
        const double rd = 1.0 / sqrt(s[0] / (double)a.H + a.eps);
        const float r = (float)rd, m = (float)(rd * rd * (s[1] / (double)a.H));
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * BLOCK + threadIdx.x;
            if (v >= vecs) continue;
            typename E::vec o;
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const float hc = E::get(h[i], c), gc = E::get(g[i], c);
                dw[i][c] += gc * (hc * r);
                float y = r * (gc * E::get(w[i], c) - hc * m);
                if (a.has_d_sum) y += E::get(d[i], c);
                E::set(o, c, y);
            }
            E::store((scalar *)a.d_x[rank] + t * a.H + v * 8, o);
        }
        if (BLOCK > kWave) __syncthreads();
    }
    if (!a.has_d_weight) return;
    float *p = a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int v = i * BLOCK + threadIdx.x;
        if (v >= vecs) continue;
        *(f32x4 *)(p + v * 8) = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        *(f32x4 *)(p + v * 8 + 4) = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
}

// Any width: the weight's sums of a workgroup stay in its part of the workspace,
// each thread adding to its own columns.
template <typename E>
__global__ __launch_bounds__(256) void k_norm_grad_any(const NormGradArgs a) {
    __shared__ double part[4][2];
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const scalar *weight = (const scalar *)a.weight;
    float *p = a.part + (int64_t)blockIdx.x * a.H;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t rank = row / a.T, t = row - rank * a.T;
        const scalar *x = (const scalar *)a.x[rank] + t * a.H, *d_out = (const scalar *)a.d_out[rank] + t * a.H;
        const scalar *d_sum = (const scalar *)a.d_sum[rank] + t * a.H;
        scalar *d_x = (scalar *)a.d_x[rank] + t * a.H;
        double s[2] = {0.0, 0.0};
        for (int64_t i = threadIdx.x; i < a.H; i += 256) {
            const double h = E::to_float(x[i]);
            s[0] = __builtin_fma(h, h, s[0]);
            s[1] = __builtin_fma((double)E::to_float(d_out[i]) * (double)E::to_float(weight[i]), h, s[1]);
        }
        block_sums<256, 2>(s, part);
        const double rd = 1.0 / sqrt(s[0] / (double)a.H + a.eps);
        const float r = (float)rd, m = (float)(rd * rd * (s[1] / (double)a.H));
        for (int64_t i = threadIdx.x; i < a.H; i += 256) {
            const float h = E::to_float(x[i]), g = E::to_float(d_out[i]);
            float y = r * (g * E::to_float(weight[i]) - h * m);
            if (a.has_d_sum) y += E::to_float(d_sum[i]);
            if (a.has_d_weight) p[i] = (row == blockIdx.x ? 0.0f : p[i]) + g * (h * r);
            d_x[i] = E::from_float(y);
        }
        __syncthreads();
    }
}

// 64 columns by 16 runs of the workgroups' sums, then the runs in order.
__global__ __launch_bounds__(1024) void k_norm_weight(const NormGradArgs a) {
    __shared__ float run[16][64];
    if (status_at_entry(a.status)) return;
    const int col = threadIdx.x % 64, k = threadIdx.x / 64;
    const int64_t c = (int64_t)blockIdx.x * 64 + col;
    float s = 0.0f;
    if (c < a.H) {
        const int per = (a.groups + 15) / 16, from = k * per, to = min(from + per, a.groups);
#pragma unroll 8
        for (int g = from; g < to; g++) s += a.part[(int64_t)g * a.H + c];
    }
    run[k][col] = s;
    __syncthreads();
    if (k != 0 || c >= a.H) return;
#pragma unroll
    for (int i = 1; i < 16; i++) s += run[i][col];
    a.d_weight[c] = s;
}

// ------------------------------------------------------------------ host
static bool norm_sizes(int W, int64_t T, int64_t H, int type) {
    return W >= 1 && W <= A2AV_MAX_W && T >= 0 && T <= (int64_t)1 << 30 && H >= 1 && H <= A2AV_MAX_WIDTH &&
           type >= A2AV_DT_F32 && type <= A2AV_DT_F16;
}
static bool at16(const void *p) { return (uintptr_t)p % 16 == 0; }

// Widest row of the register kernels: 1024 threads of four vectors.
constexpr int64_t kWidest = 1024 * 4 * 8;
constexpr unsigned kMostRows = 1u << 20;  // workgroups of a launch, times 1024 threads inside 32 bits
constexpr int kGradGroups = 512;          // workgroups of the gradient

template <typename E>
static void launch_norm(const NormArgs &a, bool fast, int W, hipStream_t stream) {
    unsigned most = max_grid() < kMostRows ? max_grid() : kMostRows;
    most = most / (unsigned)W ? most / (unsigned)W : 1;
    const dim3 g((unsigned)(a.T < (int64_t)most ? a.T : (int64_t)most), (unsigned)W);
    if (!fast) {
        hipLaunchKernelGGL(k_norm_any<E>, g, dim3(256), 0, stream, a);
        return;
    }
    const int64_t vecs = mx_padded(a.H) / 8;
    if (vecs <= 256) hipLaunchKernelGGL((k_norm_row<E, 256, 1>), g, dim3(256), 0, stream, a);
    else if (vecs <= 1024 && (int64_t)W * a.T < 512) hipLaunchKernelGGL((k_norm_row<E, 1024, 1>), g, dim3(1024), 0, stream, a);
    else if (vecs <= 512) hipLaunchKernelGGL((k_norm_row<E, 256, 2>), g, dim3(256), 0, stream, a);
    else if (vecs <= 1024) hipLaunchKernelGGL((k_norm_row<E, 256, 4>), g, dim3(256), 0, stream, a);
    else if (vecs <= 2048) hipLaunchKernelGGL((k_norm_row<E, 1024, 2>), g, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((k_norm_row<E, 1024, 4>), g, dim3(1024), 0, stream, a);
}

template <typename E>
static void launch_grad(const NormGradArgs &a, bool fast, hipStream_t stream) {
    const dim3 g((unsigned)a.groups);
    const int64_t vecs = a.H / 8;
    if (!fast) hipLaunchKernelGGL(k_norm_grad_any<E>, g, dim3(256), 0, stream, a);
    else if (vecs <= 256) hipLaunchKernelGGL((k_norm_grad_row<E, 256, 1>), g, dim3(256), 0, stream, a);
    else if (vecs <= 512) hipLaunchKernelGGL((k_norm_grad_row<E, 256, 2>), g, dim3(256), 0, stream, a);
    else if (vecs <= 1024) hipLaunchKernelGGL((k_norm_grad_row<E, 256, 4>), g, dim3(256), 0, stream, a);
    else if (vecs <= 2048) hipLaunchKernelGGL((k_norm_grad_row<E, 1024, 2>), g, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((k_norm_grad_row<E, 1024, 4>), g, dim3(1024), 0, stream, a);
}

static int grad_groups(int W, int64_t T) {
    const int64_t n = (int64_t)W * T;
    return (int)(n < kGradGroups ? n : kGradGroups);
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
    bool fast = H % 8 == 0 && H <= kWidest && at16(weight);
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
        fast = fast && at16(x[d]) && at16(a.residual[d]) && at16(a.sum[d]) && at16(a.out[d]);
    }
    if (T == 0) return A2AV_OK;
    a.weight = weight;
    a.status = status;
    a.T = T;
    a.H = H;
    a.eps = eps;
    a.format = format;
    a.has_residual = residual != nullptr;
    a.has_sum = sum != nullptr;
    a.has_out = out != nullptr;
    a.has_rows = rows != nullptr;
    if (type == A2AV_DT_F32) launch_norm<ElemF32>(a, fast, W, stream);
    else if (type == A2AV_DT_BF16) launch_norm<ElemBf16>(a, fast, W, stream);
    else launch_norm<ElemF16>(a, fast, W, stream);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}

A2AV_API size_t moe_rms_norm_backward_workspace_bytes(int W, int64_t T, int64_t H) {
    if (!norm_sizes(W, T, H, A2AV_DT_F32)) return 0;
    return ((size_t)grad_groups(W, T) * (size_t)H * 4 + 255) / 256 * 256 + 256;
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
    bool fast = H % 8 == 0 && H <= kWidest && at16(weight);
    for (int d = 0; d < W && T > 0; d++) {
        if (!x[d] || !d_out[d] || !d_x[d] || (d_sum && !d_sum[d])) return A2AV_EARG;
        a.x[d] = x[d];
        a.d_out[d] = d_out[d];
        a.d_sum[d] = d_sum ? d_sum[d] : nullptr;
        a.d_x[d] = d_x[d];
        fast = fast && at16(x[d]) && at16(d_out[d]) && at16(a.d_sum[d]) && at16(d_x[d]);
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
    a.groups = grad_groups(W, T);
    a.has_d_sum = d_sum != nullptr;
    a.has_d_weight = d_weight != nullptr;
    if (T > 0) {
        if (type == A2AV_DT_F32) launch_grad<ElemF32>(a, fast, stream);
        else if (type == A2AV_DT_BF16) launch_grad<ElemBf16>(a, fast, stream);
        else launch_grad<ElemF16>(a, fast, stream);
    }
    if (d_weight)
        hipLaunchKernelGGL(k_norm_weight, dim3((unsigned)((H + 63) / 64)), dim3(1024), 0, stream, a);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
