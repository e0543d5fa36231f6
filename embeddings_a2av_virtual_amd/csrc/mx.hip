// mx.hip — values to microscaled rows of 8- or 4-bit elements and back (gfx950).
//
//   k_mx_quantize     one thread per 8 elements, four of them a block
//   k_mx_dequantize   the same, the other way
#include <hip/hip_runtime.h>

#include <cstring>

#include "mx.hpp"
#include "vectors.hpp"

namespace a2av {

// n / d for n < 2^31 by a product with a number worked out on the host.
struct Divider {
    uint32_t d, magic, shift;
    explicit Divider(uint32_t by = 1) : d(by), magic(0), shift(0) {
        while (shift < 31 && (1u << shift) < by) shift++;
        magic = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - by)) / by + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(magic, n) + n) >> shift; }
};

struct MxArgs {
    const void *in[A2AV_MAX_W];
    void *out[A2AV_MAX_W];
    int64_t rows[A2AV_MAX_W];
    const int32_t *status;
    int64_t H;
    Divider pieces;  // of 256 elements in a row
    int vec;         // arrays of 16-byte vectors
};

// A half wave per piece of 256 elements of a row, eight to a lane.
template <typename E, int FORMAT>
__global__ __launch_bounds__(256) void k_mx_quantize(const MxArgs a) {
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const int rank = blockIdx.y, lane = threadIdx.x % 32;
    const uint32_t total = (uint32_t)a.rows[rank] * a.pieces.d;
    const int64_t stride = mx_stride(FORMAT, a.H), element_bytes = mx_element_bytes(FORMAT, a.H);
    for (uint32_t p = blockIdx.x * 8 + threadIdx.x / 32; p < total; p += gridDim.x * 8) {
        const uint32_t row = a.pieces(p), at = p - row * a.pieces.d;
        const int64_t c = (int64_t)at * kMxPad + lane * 8;
        const scalar *x = (const scalar *)a.in[rank] + (int64_t)row * a.H + c;
        float v[8];
        if (a.vec) {
            typename E::vec u = {};
            if (c < a.H) u = E::load(x);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = E::get(u, i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = c + i < a.H ? E::to_float(x[i]) : 0.0f;
        }
        int scale;
        const auto e = mx_block<FORMAT>(v, scale);
        unsigned char *out = (unsigned char *)a.out[rank] + (int64_t)row * stride;
        *(typename Mx<FORMAT>::packed *)(out + c / 8 * (int64_t)sizeof(e)) = e;
        if (lane % 4 == 0) out[element_bytes + c / kMxBlock] = (unsigned char)scale;
    }
}

template <typename E, int FORMAT>
__global__ __launch_bounds__(256) void k_mx_dequantize(const MxArgs a) {
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const int rank = blockIdx.y, lane = threadIdx.x % 32;
    const uint32_t total = (uint32_t)a.rows[rank] * a.pieces.d;
    const int64_t stride = mx_stride(FORMAT, a.H), element_bytes = mx_element_bytes(FORMAT, a.H);
    for (uint32_t p = blockIdx.x * 8 + threadIdx.x / 32; p < total; p += gridDim.x * 8) {
        const uint32_t row = a.pieces(p), at = p - row * a.pieces.d;
        const int64_t c = (int64_t)at * kMxPad + lane * 8;
        if (c >= a.H) continue;
        const unsigned char *in = (const unsigned char *)a.in[rank] + (int64_t)row * stride;
        typedef typename Mx<FORMAT>::packed packed;
        float v[8];
        Mx<FORMAT>::unpack(*(const packed *)(in + c / 8 * (int64_t)sizeof(packed)), mx_scale(in[element_bytes + c / kMxBlock]), v);
        scalar *out = (scalar *)a.out[rank] + (int64_t)row * a.H + c;
        if (a.vec) {
            typename E::vec o;
#pragma unroll
            for (int i = 0; i < 8; i++) E::set(o, i, v[i]);
            E::store(out, o);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < a.H) out[i] = E::from_float(v[i]);
        }
    }
}

// ------------------------------------------------------------------ host
// Checks and arguments of both directions: `mx` has the microscaled rows.
static int fill(MxArgs &a, int W, int64_t H, int type, int format, const void *const *in, void *const *out,
                const int64_t *n_rows, const int32_t *status, bool to_mx, uint32_t *groups) {
    if (W < 1 || W > A2AV_MAX_W || H < 1 || H > A2AV_MAX_WIDTH || type < A2AV_DT_F32 || type > A2AV_DT_F16)
        return A2AV_EARG;
    if ((format != A2AV_MX_FP8 && format != A2AV_MX_FP4) || !in || !out || !n_rows || !status) return A2AV_EARG;
    std::memset((void *)&a, 0, sizeof(a));
    a.status = status;
    a.H = H;
    const int64_t pieces = mx_padded(H) / kMxPad;
    a.pieces = Divider((uint32_t)pieces);
    a.vec = H % 8 == 0;
    int64_t most = 0;
    for (int d = 0; d < W; d++) {
        if (n_rows[d] < 0 || n_rows[d] > (((int64_t)1 << 31) - 1) / pieces) return A2AV_EARG;
        if (n_rows[d] == 0) continue;
        if (!in[d] || !out[d] || in[d] == out[d] || (uintptr_t)(to_mx ? out[d] : in[d]) % 16 != 0) return A2AV_EARG;
        a.in[d] = in[d];
        a.out[d] = out[d];
        a.rows[d] = n_rows[d];
        if ((uintptr_t)(to_mx ? in[d] : out[d]) % 16 != 0) a.vec = 0;
        most = n_rows[d] * pieces > most ? n_rows[d] * pieces : most;
    }
    const int64_t want = (most + 7) / 8;
    const int64_t cap = (int64_t)max_grid() / W > 0 ? (int64_t)max_grid() / W : 1;
    *groups = (uint32_t)(want < cap ? want : cap);
    return A2AV_OK;
}

}  // namespace a2av

using namespace a2av;

A2AV_API size_t moe_mx_row_bytes(int format, int64_t H) {
    if ((format != A2AV_MX_FP8 && format != A2AV_MX_FP4) || H < 1 || H > A2AV_MAX_WIDTH) return 0;
    return (size_t)mx_stride(format, H);
}

#define A2AV_MX_LAUNCH(KERNEL)                                                                                 \
    do {                                                                                                       \
        const dim3 g(groups, (unsigned)W);                                                                     \
        if (format == A2AV_MX_FP8) {                                                                           \
            if (type == A2AV_DT_F32) hipLaunchKernelGGL((KERNEL<ElemF32, A2AV_MX_FP8>), g, dim3(256), 0, stream, a);        \
            else if (type == A2AV_DT_BF16) hipLaunchKernelGGL((KERNEL<ElemBf16, A2AV_MX_FP8>), g, dim3(256), 0, stream, a); \
            else hipLaunchKernelGGL((KERNEL<ElemF16, A2AV_MX_FP8>), g, dim3(256), 0, stream, a);               \
        } else {                                                                                               \
            if (type == A2AV_DT_F32) hipLaunchKernelGGL((KERNEL<ElemF32, A2AV_MX_FP4>), g, dim3(256), 0, stream, a);        \
            else if (type == A2AV_DT_BF16) hipLaunchKernelGGL((KERNEL<ElemBf16, A2AV_MX_FP4>), g, dim3(256), 0, stream, a); \
            else hipLaunchKernelGGL((KERNEL<ElemF16, A2AV_MX_FP4>), g, dim3(256), 0, stream, a);               \
        }                                                                                                      \
    } while (0)

A2AV_API int moe_mx_quantize(int W, int64_t H, int type, int format, const void *const *x,
                             const int64_t *n_rows, void *const *rows, int32_t *status,
                             hipStream_t stream) {
    MxArgs a;
    uint32_t groups;
    if (fill(a, W, H, type, format, x, rows, n_rows, status, true, &groups) != A2AV_OK) return A2AV_EARG;
    if (!groups) return A2AV_OK;
    A2AV_MX_LAUNCH(k_mx_quantize);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}

A2AV_API int moe_mx_dequantize(int W, int64_t H, int type, int format, const void *const *rows,
                               const int64_t *n_rows, void *const *out, int32_t *status,
                               hipStream_t stream) {
    MxArgs a;
    uint32_t groups;
    if (fill(a, W, H, type, format, rows, out, n_rows, status, false, &groups) != A2AV_OK) return A2AV_EARG;
    if (!groups) return A2AV_OK;
    A2AV_MX_LAUNCH(k_mx_dequantize);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
