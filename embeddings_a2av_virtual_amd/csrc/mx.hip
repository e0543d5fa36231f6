// mx.hip — values to microscaled rows of 8- or 4-bit elements and back (gfx950).
//
//   k_mx_quantize     one thread per 8 elements, four of them a block
//   k_mx_dequantize   the same, the other way
#include <hip/hip_runtime.h>

#include <cstring>

#include "mx.hpp"
#include "vectors.hpp"

namespace a2av {

// n / d for n < 2^31 by a product with a number worked out on the host (division by an
// invariant integer after Granlund and Montgomery).
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
};

// A half wave per piece of 256 elements of a row, eight to a lane, kPieces pieces in
// flight. Bound by the bytes: 8 x 2048 rows of 7168 in bf16 to 8 bits 57.5 us (6.19
// TB/s, a copy reaches 6.52; 66.0 with one piece, 56.8 with four), 32768 rows to 4
// bits 95 (109, 95) and back 96 (105, 100).
constexpr int kPieces = 2;

template <typename E, int FORMAT, bool WHOLE>
__global__ __launch_bounds__(256) void k_mx_quantize(const MxArgs a) {
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    const int rank = blockIdx.y, lane = threadIdx.x % 32;
    const uint32_t total = (uint32_t)a.rows[rank] * a.pieces.d;
    const int64_t stride = mx_stride(FORMAT, a.H), element_bytes = mx_element_bytes(FORMAT, a.H);
    for (uint32_t p0 = blockIdx.x * 8 * kPieces + threadIdx.x / 32; p0 < total; p0 += gridDim.x * 8 * kPieces) {
        typename E::vec u[kPieces] = {};
        uint32_t row[kPieces];
        int64_t c[kPieces];
#pragma unroll
        for (int k = 0; k < kPieces; k++) {
            const uint32_t p = min(p0 + k * 8, total - 1);  // past the end: the last again, not stored
            row[k] = a.pieces(p);
            c[k] = (int64_t)(p - row[k] * a.pieces.d) * kMxPad + lane * 8;
            const scalar *x = (const scalar *)a.in[rank] + (int64_t)row[k] * a.H;
            if constexpr (WHOLE) {
                if (c[k] < a.H) u[k] = E::load(x + c[k]);
            } else {
                u[k] = load_row<E>(x, c[k], a.H);
            }
        }
#pragma unroll
        for (int k = 0; k < kPieces; k++) {
            if (p0 + k * 8 >= total) break;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = E::get(u[k], i);
            int scale;
            const auto e = mx_block<FORMAT>(v, scale);
            unsigned char *out = (unsigned char *)a.out[rank] + (int64_t)row[k] * stride;
            __builtin_nontemporal_store(e, (typename Mx<FORMAT>::packed *)(out + c[k] / 8 * (int64_t)sizeof(e)));
            if (lane % 4 == 0) out[element_bytes + c[k] / kMxBlock] = (unsigned char)scale;
        }
    }
}

template <typename E, int FORMAT, bool WHOLE>
__global__ __launch_bounds__(256) void k_mx_dequantize(const MxArgs a) {
    if (status_at_entry(a.status)) return;
    typedef typename E::scalar scalar;
    typedef typename Mx<FORMAT>::packed packed;
    const int rank = blockIdx.y, lane = threadIdx.x % 32;
    const uint32_t total = (uint32_t)a.rows[rank] * a.pieces.d;
    const int64_t stride = mx_stride(FORMAT, a.H), element_bytes = mx_element_bytes(FORMAT, a.H);
    for (uint32_t p0 = blockIdx.x * 8 * kPieces + threadIdx.x / 32; p0 < total; p0 += gridDim.x * 8 * kPieces) {
        packed e[kPieces];
        uint32_t row[kPieces], scale[kPieces];
        int64_t c[kPieces];
#pragma unroll
        for (int k = 0; k < kPieces; k++) {
            const uint32_t p = min(p0 + k * 8, total - 1);
            row[k] = a.pieces(p);
            c[k] = (int64_t)(p - row[k] * a.pieces.d) * kMxPad + lane * 8;
            const unsigned char *in = (const unsigned char *)a.in[rank] + (int64_t)row[k] * stride;
            e[k] = __builtin_nontemporal_load((const packed *)(in + c[k] / 8 * (int64_t)sizeof(packed)));
            scale[k] = in[element_bytes + c[k] / kMxBlock];
        }
#pragma unroll
        for (int k = 0; k < kPieces; k++) {
            if (p0 + k * 8 >= total) break;
            if (c[k] >= a.H) continue;
            float v[8];
            Mx<FORMAT>::unpack(e[k], mx_scale(scale[k]), v);
            typename E::vec o;
#pragma unroll
            for (int i = 0; i < 8; i++) E::set(o, i, v[i]);
            scalar *out = (scalar *)a.out[rank] + (int64_t)row[k] * a.H;
            if constexpr (WHOLE) E::store(out + c[k], o);
            else store_row<E>(out, c[k], a.H, o);
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
    int64_t most = 0;
    for (int d = 0; d < W; d++) {
        if (n_rows[d] < 0 || n_rows[d] > (((int64_t)1 << 31) - 1) / pieces) return A2AV_EARG;
        if (n_rows[d] == 0) continue;
        if (!in[d] || !out[d] || in[d] == out[d] || (uintptr_t)(to_mx ? out[d] : in[d]) % 16 != 0) return A2AV_EARG;
        a.in[d] = in[d];
        a.out[d] = out[d];
        a.rows[d] = n_rows[d];
        most = n_rows[d] * pieces > most ? n_rows[d] * pieces : most;
    }
    const int64_t want = (most + 8 * kPieces - 1) / (8 * kPieces);
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

// WHOLE: rows of whole vectors
#define A2AV_MX_LAUNCH2(KERNEL, E, F)                                                                        \
    do {                                                                                                     \
        if (H % 8 == 0) hipLaunchKernelGGL((KERNEL<E, F, true>), dim3(groups, W), dim3(256), 0, stream, a);   \
        else hipLaunchKernelGGL((KERNEL<E, F, false>), dim3(groups, W), dim3(256), 0, stream, a);             \
    } while (0)
#define A2AV_MX_LAUNCH(KERNEL)                                                        \
    do {                                                                              \
        if (format == A2AV_MX_FP8) {                                                  \
            if (type == A2AV_DT_F32) A2AV_MX_LAUNCH2(KERNEL, ElemF32, A2AV_MX_FP8);    \
            else if (type == A2AV_DT_BF16) A2AV_MX_LAUNCH2(KERNEL, ElemBf16, A2AV_MX_FP8); \
            else A2AV_MX_LAUNCH2(KERNEL, ElemF16, A2AV_MX_FP8);                       \
        } else {                                                                      \
            if (type == A2AV_DT_F32) A2AV_MX_LAUNCH2(KERNEL, ElemF32, A2AV_MX_FP4);    \
            else if (type == A2AV_DT_BF16) A2AV_MX_LAUNCH2(KERNEL, ElemBf16, A2AV_MX_FP4); \
            else A2AV_MX_LAUNCH2(KERNEL, ElemF16, A2AV_MX_FP4);                       \
        }                                                                             \
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
