// mx_experts.hip — the experts' products on microscaled rows with 4-bit weights
// (gfx950).
//
// out = act(x . W_e^T + b_e) on expert-major rows, x in e4m3 or e2m1 blocks and
// W_e in e2m1 blocks of 32 with a scale each: the block-scaled matrix
// instructions take both operands as they lie and multiply by the scales, with
// fp32 sums.
//
//   k_mx_tile   one tile, operands through LDS
//   k_mx_few    32 columns of up to 16 rows, which read their weights once
//
// Outputs of 8 bits (MX) come out as in 64 bits wherever fp32 can hold the sums.
#include <hip/hip_runtime.h>

#include <cstring>
#include <type_traits>
#include <utility>

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
    int32_t *status_out;             // the same word
    int64_t x_rows[A2AV_MAX_W];
    int64_t K, N, NW;
    int64_t x_stride, w_stride, out_stride;  // bytes of a row; of out if microscaled
    int W, P;
    int act, out_type, has_bias;
    int wide;  // out by 16-byte vectors
    int cols;  // column tiles
};

// The matrix instruction sums eight products at a time (k = 8i .. 8i + 7): with 2^e the
// largest product of their powers of two, each is cut towards 0 at 2^(e - 13); sums of
// eight are added in fp32 (measured). Of e2m1 rows that cuts nothing. Of e4m3 ones it
// takes less than 7 * 2^-13 of the largest product from a sum of eight, 5e-6 of random
// sums: for results of 16 bits that is left so (32 experts of 512 rows 378 us to bf16,
// split and to 8 bits 769), but where the result becomes an element of 8 bits it decides
// three in ten thousand of them otherwise than fp32 sums. There, and where few rows leave
// the matrix cores idle, an e4m3 operand is split by its exponent's top bit into elements
// of 2 and above and those below; neither part's products with e2m1 are cut, so both sums
// of eight are exact, and with a sum in fp32 for either part, both of few bits, so are
// most of these (added in double at the end).
struct Split {
    i32x8 hi, lo;
};
__device__ __forceinline__ Split split(i32x8 v) {
    Split s;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        // a byte permutation gives 0xFF for a selector above 12 and 0 for 12
        const uint32_t top = ((uint32_t)v[i] & 0x40404040u) | 0x0C0C0C0Cu;
        s.hi[i] = (int)((uint32_t)v[i] & __builtin_amdgcn_perm(0u, 0u, top));
        s.lo[i] = v[i] ^ s.hi[i];
    }
    return s;
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

// Activations where the output becomes an element of 8 bits, in double to 1e-10: the
// fp32 ones are a few steps off, which decides an element near a border otherwise than
// the formula (K 7168, SwiGLU: 59 of 33 million elements with one fp32 sum and these
// in fp32, 42 with these in double, 1 with the two sums of the split as well; 8 experts
// of 512 rows).
__device__ __forceinline__ double exp_wide(double x) {
    const double t = __builtin_fmin(__builtin_fmax(x * 1.4426950408889634, -1000.0), 1000.0), n = __builtin_rint(t);
    const double f = (t - n) * 0.69314718055994531;  // at most 0.35: the series to f^9 leaves 1e-11
    double p = 1.0 / 362880;
    p = __builtin_fma(p, f, 1.0 / 40320);
    p = __builtin_fma(p, f, 1.0 / 5040);
    p = __builtin_fma(p, f, 1.0 / 720);
    p = __builtin_fma(p, f, 1.0 / 120);
    p = __builtin_fma(p, f, 1.0 / 24);
    p = __builtin_fma(p, f, 1.0 / 6);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    return p * __longlong_as_double((int64_t)((int)n + 1023) << 52);
}
__device__ __forceinline__ double inverse(double d) {  // of 1 .. 2^1001
    const double r = __builtin_amdgcn_rcp(d), e = __builtin_fma(-d, r, 1.0);
    return __builtin_fma(r, __builtin_fma(e, e, e), r);
}
__device__ __forceinline__ double silu_wide(double h) { return h * inverse(1.0 + exp_wide(-h)); }

// As normal_cdf, a polynomial in t - 0.6 to 5e-11 for |h| <= 19.
__device__ __forceinline__ double gelu_wide(double h) {
    const double x = __builtin_fabs(h) * 0.70710678118654752, t = inverse(1.0 + 0.3 * x), u = t - 0.6;
    double p = -0.021166241996014044;
    p = __builtin_fma(p, u, 0.0105805190538479);
    p = __builtin_fma(p, u, 0.063256953723092021);
    p = __builtin_fma(p, u, -0.0021860954671192008);
    p = __builtin_fma(p, u, -0.15132855689646429);
    p = __builtin_fma(p, u, -0.1364120761610744);
    p = __builtin_fma(p, u, 0.22425531289121886);
    p = __builtin_fma(p, u, 0.80774900059842292);
    p = __builtin_fma(p, u, 1.2778910601161468);
    p = __builtin_fma(p, u, 1.3850097074199901);
    p = __builtin_fma(p, u, 1.1416704294489632);
    p = __builtin_fma(p, u, 0.74455288756601934);
    p = __builtin_fma(p, u, 0.38928356801009617);
    const double q = 0.5 * p * t * exp_wide(-0.5 * h * h);
    return h * (h > 0.0 ? 1.0 - q : q);
}
__device__ __forceinline__ double act_wide(int act, double h) {
    switch (act) {
    case A2AV_ACT_RELU: return h < 0.0 ? 0.0 : h;
    case A2AV_ACT_GELU: return gelu_wide(h);
    case A2AV_ACT_SILU: return silu_wide(h);
    default: return h;
    }
}

// Eight outputs y of row `row`, columns n .. n + 7; every lane of a quad comes
// here together with the same row and its own eight columns of a block of 32.
__device__ __forceinline__ void put_mx(const MxExpertArgs &a, int d, int64_t row, int64_t n, double (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (n + i >= a.N) y[i] = 0.0;
    int scale;
    const auto e = mx_block<A2AV_MX_FP8>(y, scale);
    unsigned char *out = (unsigned char *)a.out[d] + row * a.out_stride;
    *(u32x2 *)(out + n) = e;
    if (n % kMxBlock == 0) out[mx_padded(a.N) + n / kMxBlock] = (unsigned char)scale;
}

__device__ __forceinline__ void put_out(const MxExpertArgs &a, int d, int64_t row, int64_t n, const float (&y)[8]) {
    uint16_t *out = (uint16_t *)a.out[d] + row * a.N + n;
    if (a.wide) {
        if (a.out_type == kOutBf16) put8<Bf16, true>(out, y);
        else put8<Fp16, true>(out, y);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (n + i < a.N) out[i] = a.out_type == kOutBf16 ? Bf16::from_float(y[i]) : Fp16::from_float(y[i]);
}

// (the columns of a row's padding have no bias)
template <typename T>
__device__ __forceinline__ void add_bias(const MxExpertArgs &a, const float *bias, int64_t n, T (&y)[8]) {
    const bool whole = n + 8 <= a.N;
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (whole || n + i < a.N) y[i] += bias[n + i];
}

// The rows of a pass; `row_of(r)` is the expert's row behind LDS row r, c0 the
// first product column of the wave. Several rows' LDS reads are in flight at once.
// MX: the outputs are microscaled; TWO: the sums are sums + low.
template <int ROWS, int COLS, bool GLU, bool MX, bool TWO, typename RowOf>
__device__ __forceinline__ void emit_rows(const MxExpertArgs &a, const f32x4 *sums, const f32x4 *low, int d, int j,
                                          int64_t row0, int64_t M, int64_t c0, int lane, RowOf row_of) {
    constexpr int kPer = GLU ? COLS / 16 : COLS / 8, kStep = kWave / kPer;  // lanes a row, rows at once
    constexpr int kTimes = (ROWS + kStep - 1) / kStep, kMost = GLU || MX ? 2 : 4, kBatch = kTimes < kMost ? kTimes : kMost;
    static_assert(kTimes % kBatch == 0, "");
    constexpr int kUnroll = MX ? 1 : kTimes;  // activations in double are a thousand instructions
    typedef typename std::conditional<MX, double, float>::type value;
    const int64_t end = MX ? mx_padded(a.N) : a.N;
    const int q = lane % kPer;
    const int64_t n = (GLU ? c0 / 2 : c0) + q * 8;
    if (n >= end) return;
    const float *bias = a.bias[d] + (int64_t)j * a.NW;
    const auto take = [&](int r, int at, value(&y)[8]) {
        const f32x4 v[2] = {sums[chunk<COLS>(r, at)], sums[chunk<COLS>(r, at + 1)]};
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i / 4][i % 4];
        if constexpr (TWO) {
            const f32x4 l[2] = {low[chunk<COLS>(r, at)], low[chunk<COLS>(r, at + 1)]};
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] += l[i / 4][i % 4];
        }
    };
    // gated: blocks of 16 gate and 16 up columns alternate
    const int at = GLU ? (q >> 1) * 8 + (q & 1) * 2 : q * 2;
#pragma unroll kUnroll
    for (int r0 = 0; r0 < kTimes * kStep; r0 += kBatch * kStep) {
        value y[kBatch][8], up[GLU ? kBatch : 1][8];
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            take(r0 + b * kStep + lane / kPer, at, y[b]);
            if constexpr (GLU) take(r0 + b * kStep + lane / kPer, at + 4, up[b]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            const int64_t m = row_of(r0 + b * kStep + lane / kPer);
            if (m >= M) continue;
            if (a.has_bias) add_bias(a, bias, n, y[b]);
            if constexpr (GLU) {
                if (a.has_bias) add_bias(a, bias + a.N, n, up[b]);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if constexpr (MX) y[b][i] = silu_wide(y[b][i]) * up[b][i];
                    else y[b][i] = y[b][i] * sigmoid(y[b][i]) * up[b][i];
            } else if (a.act != A2AV_ACT_NONE) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if constexpr (MX) y[b][i] = act_wide(a.act, y[b][i]);
                    else y[b][i] = act_of(a.act, y[b][i]);
            }
            if constexpr (MX) put_mx(a, d, row0 + m, n, y[b]);
            else put_out(a, d, row0 + m, n, y[b]);
        }
    }
}
template <int ROWS, int COLS, bool MX, bool TWO, typename RowOf>
__device__ __forceinline__ void emit(const MxExpertArgs &a, const f32x4 *sums, const f32x4 *low, int d, int j, int64_t row0,
                                     int64_t M, int64_t c0, int lane, RowOf row_of) {
    if (a.act == A2AV_ACT_SWIGLU) emit_rows<ROWS, COLS, true, MX, TWO>(a, sums, low, d, j, row0, M, c0, lane, row_of);
    else emit_rows<ROWS, COLS, false, MX, TWO>(a, sums, low, d, j, row0, M, c0, lane, row_of);
}

// ------------------------------------------------------------------ the tiles
// Bound by the matrix cores, their operands' LDS reads and the clock under their power:
// 32 experts of 512 rows, K 7168, 4096 columns: 4-bit rows 271 us (3.5 PFLOP/s), 291 with
// 8-bit outputs, 8-bit ones 380 (2.5), with 8-bit outputs, two products an element, 769; K 2048, 7168
// columns 187 and 243. Without the loads the first would take 180, with all of them
// in the L2 240; spreading them over a step, or two steps further ahead, changes nothing.
// Tiles of BM rows and BC columns. LDS rows are 128 bytes of an operand's row: 256
// elements of e2m1 or 128 of e4m3, so that a step is 256 elements of 4-bit rows or
// 128 of 8-bit ones, and every second step of those takes new weights. Buffer
// loads fill two stages of either operand; the eight 16-byte chunks of LDS row r
// are permuted by r / 2, which puts the 16 lanes of rows r .. r + 15 in different
// banks. Rows and elements outside are loaded out of the buffer's range, which
// writes zeros.
template <int ROWS, int WAVES>
struct MxOperand {
    static constexpr int kLoads = ROWS / 8 / WAVES;  // 16-byte loads a thread and stage
    const unsigned char *base;
    uint32_t span;         // bytes of the buffer: the tile's rows
    uint32_t off[kLoads];  // of a thread's loads in the first stage
    int at, end;           // byte of the next stage, and behind the last

    // `rows` rows of `stride` bytes from p; a gated product takes blocks of 16 rows
    // from p and p2 in turn (a wave's loads are all of the one or of the other).
    __device__ __forceinline__ void init(const unsigned char *p, const unsigned char *p2, int64_t stride, int64_t rows,
                                         int64_t bytes, int wave, int lane) {
        static_assert(WAVES % 4 == 0, "");
        const int64_t most = p2 ? ROWS / 2 : ROWS;
        base = p2 && ((wave >> 1) & 1) ? p2 : p;
        span = (uint32_t)((rows < 0 ? 0 : rows < most ? rows : most) * stride);
        at = 0;
        end = (int)bytes;
        const int k = ((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4))) * 16;
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int r = (i * WAVES + wave) * 8;
            off[i] = (uint32_t)((p2 ? (r >> 5) * 16 + (r & 8) : r) + (lane >> 3)) * (uint32_t)stride + k;
        }
    }
    // Loads FROM .. TO of the next stage.
    template <int FROM, int TO>
    __device__ __forceinline__ void load(unsigned char *lds, int wave) const {
        const rsrc_t b = buffer(base, at < end ? span : 0);
#pragma unroll
        for (int i = FROM; i < TO; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void *)(lds + (i * WAVES + wave) * 1024), 16, (int)off[i],
                                                     at, 0, 0);
    }
    __device__ __forceinline__ void next() { at += 128; }
};

template <int FORMAT, int BM, int BC, int WM, int WC>
struct MxShape {
    static constexpr int kWaves = WM * WC, kThreads = kWaves * kWave;
    static constexpr int kBlocksM = BM / WM / 32, kBlocksC = BC / WC / 32;
    static constexpr int kQuarters = FORMAT == A2AV_MX_FP8 ? 2 : 4;  // of 64 elements in a step
    static constexpr int kScaleRows = BM + BC;
    static_assert(BM <= kThreads / 2 && BC <= kThreads / 2 && kBlocksC == 2, "");
    typedef MxOperand<BM, kWaves> A;
    typedef MxOperand<BC, kWaves> B;
};

// The scales of a tile's rows, 1024 elements (32 bytes a row) at a time: half of a
// row's, of x and of the weight, per thread, through registers to the two LDS
// buffers. In LDS the halves of 16 bytes lie apart, row after row.
constexpr int kScaleMacros = 4;  // steps of 256 elements in a buffer

template <int BM, int BC>
struct MxScales {
    const unsigned char *x, *w;  // the thread's rows' scales
    int last_x, last_w;          // offset of the last 16 bytes inside the rows
    u32x4 v[2];
    __device__ __forceinline__ void load(int chunk) {
        const int at = chunk * 32 + (threadIdx.x & 1) * 16;
        v[0] = *(const u32x4 *)(x + min(at, last_x));
        v[1] = *(const u32x4 *)(w + min(at, last_w));
    }
    __device__ __forceinline__ void store(u32x4 *lds, int chunk) const {
        const int row = threadIdx.x / 2;
        lds += ((chunk & 1) * 2 + (threadIdx.x & 1)) * (BM + BC) + row;
        if (row < BM) lds[0] = v[0];
        if (row < BC) lds[BM] = v[1];
    }
};

// One position: a block of 32 rows times the wave's 64 columns, 64 elements.
template <int FORMAT>
struct MxFrag {
    typedef i32x8 type;
};
template <>
struct MxFrag<A2AV_MX_FP4> {
    typedef i32x4 type;
};

template <int FORMAT, int BYTE>
__device__ __forceinline__ f32x16 mfma_at(i32x4 w, i32x8 x, f32x16 c, uint32_t sw, uint32_t sx) {
    const i32x8 w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, x, c, 4, FORMAT == A2AV_MX_FP8 ? 0 : 4, BYTE, (int)sw, BYTE,
                                                           (int)sx);
}
template <int FORMAT, int BYTE>
__device__ __forceinline__ f32x16 mfma_at(i32x4 w, i32x4 x, f32x16 c, uint32_t sw, uint32_t sx) {
    return mfma_at<FORMAT, BYTE>(w, __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1), c, sw, sx);
}

// f of 0, 1, ... as constants.
template <typename F, int... I>
__device__ __forceinline__ void each(const F &f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

// The contraction of one tile with NB row blocks a wave (the blocks of the waves
// alternate, so that a tile with few rows keeps all of them busy). The step's
// positions follow each other quarter by quarter; the rows' fragments are read
// kAhead positions ahead. kAhead positions before a step's end everything of its
// stages has been read: one barrier there frees them for the loads of the step
// after the next, and publishes the next one's.
template <int FORMAT, bool SPLIT, int BM, int BC, int WM, int WC, int NB>
__device__ __forceinline__ void mx_contract(typename MxShape<FORMAT, BM, BC, WM, WC>::A &oa,
                                            typename MxShape<FORMAT, BM, BC, WM, WC>::B &ob,
                                            MxScales<BM, BC> &os, unsigned char *const (&sa)[2],
                                            unsigned char *const (&sb)[2], u32x4 *ss, int macros,
                                            f32x16 (&acc)[1 + SPLIT][MxShape<FORMAT, BM, BC, WM, WC>::kBlocksM][2]) {
    typedef MxShape<FORMAT, BM, BC, WM, WC> S;
    typedef typename MxFrag<FORMAT>::type frag;
    constexpr bool k8 = FORMAT == A2AV_MX_FP8;
    // where rows are split, that is done a position ahead, beside the matrix
    // instructions of the one before
    constexpr bool kPipe = SPLIT && NB >= 2;
    constexpr int Q = S::kQuarters, P = Q * NB, kRing = NB >= 4 && !kPipe ? 4 : 2, kAhead = kPipe ? 2 : kRing - 1;
    constexpr int kLoadsA = (NB * WM * 32 + S::kWaves * 8 - 1) / (S::kWaves * 8) < S::A::kLoads
                                ? (NB * WM * 32 + S::kWaves * 8 - 1) / (S::kWaves * 8) : S::A::kLoads;
    constexpr int kLoadsB = S::B::kLoads;
    constexpr int kWords = k8 ? 1 : 2;  // of scales of a row and step
    static_assert(P % kRing == 0 && kAhead <= NB, "");
    const int lane = threadIdx.x & (kWave - 1), half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WC, wc = wave % WC;
    int spot = (lane & 31) * 128 + ((half ^ ((lane >> 1) & 7)) << 4);  // of a row's first chunk
    const auto read_a = [&](const unsigned char *s, int m, int q) __attribute__((always_inline)) -> frag {
        const unsigned char *p = s + (m * WM + wm) * 32 * 128;
        if constexpr (k8) {
            const i32x4 lo = *(const i32x4 *)(p + (spot ^ q * 64)), hi = *(const i32x4 *)(p + (spot ^ (q * 64 + 32)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return *(const i32x4 *)(p + (spot ^ q * 32));
        }
    };
    const auto read_b = [&](i32x4(&f)[2], const unsigned char *s, int q) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < 2; c++) f[c] = *(const i32x4 *)(s + (wc * 2 + c) * 32 * 128 + (spot ^ q * 32));
    };
    uint32_t wa[2][NB][kWords], wb[2][2][kWords];
    const int scale_row = lane & 31, shift = half * 8;
    // the scales of step `of` of macro step `macro`
    const auto read_scales = [&](auto set, int macro, int of) __attribute__((always_inline)) {
        constexpr int kSet = decltype(set)::value;
        const uint32_t *p = (const uint32_t *)(ss + ((macro >> 1) & 3) * S::kScaleRows + scale_row) + (macro & 1) * 2 + of;
        const auto get = [&](uint32_t(&w)[kWords], int row) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kWords; i++) w[i] = p[row * 4 + i];
        };
#pragma unroll
        for (int m = 0; m < NB; m++) get(wa[kSet][m], (m * WM + wm) * 32);
#pragma unroll
        for (int c = 0; c < 2; c++) get(wb[kSet][c], BM + (wc * 2 + c) * 32);
    };
    const auto shift_scales = [&](auto set) __attribute__((always_inline)) {
        constexpr int kSet = decltype(set)::value;
#pragma unroll
        for (int i = 0; i < kWords; i++) {
#pragma unroll
            for (int m = 0; m < NB; m++) wa[kSet][m][i] >>= shift;
#pragma unroll
            for (int c = 0; c < 2; c++) wb[kSet][c][i] >>= shift;
        }
    };
    typedef std::integral_constant<int, 0> zero;
    frag fa[kRing];
    i32x4 fb[2][2];
    os.load(0);
    oa.template load<0, kLoadsA>(sa[0], wave);
    ob.template load<0, kLoadsB>(sb[0], wave);
    oa.next();
    ob.next();
    oa.template load<0, kLoadsA>(sa[1], wave);
    ob.template load<0, kLoadsB>(sb[1], wave);
    oa.next();
    ob.next();
    os.store(ss, 0);
    wait_for<0, true>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_scales(zero{}, 0, 0);
    read_b(fb[0], sb[0], 0);
#pragma unroll
    for (int p = 0; p < kAhead; p++) fa[p] = read_a(sa[0], p % NB, p / NB);
    Split parts[2];
    if constexpr (kPipe) parts[0] = split(fa[0]);
    // step `i` of the unrolled ones (its stages by its number), in macro step `macro`
    const auto step = [&](auto number, int macro) __attribute__((always_inline)) {
        constexpr int i = decltype(number)::value;
        constexpr int kStageA = i % 2, kStageB = k8 ? i / 2 % 2 : i % 2, kPart = k8 ? i % 2 : 0;
        constexpr bool kFreesB = !k8 || i % 2 == 1;
        constexpr int kNextB = kFreesB ? 1 - kStageB : kStageB, kFirstB = k8 && !kFreesB ? 2 : 0;
        constexpr int kSet = i % 2;
        shift_scales(std::integral_constant<int, kSet>{});
        if constexpr (kPart == 0) {
            if ((macro & (kScaleMacros - 1)) == 0) os.load(macro / kScaleMacros + 1);
            if ((macro & (kScaleMacros - 1)) == 2) os.store(ss, macro / kScaleMacros + 1);
        }
        const auto position = [&](auto place) __attribute__((always_inline)) {
            constexpr int p = decltype(place)::value, q = p / NB, m = p % NB, next = p + kAhead;
            if constexpr (p == P - kAhead) {
                // the weights behind the rows of the step before have one more to arrive
                wait_for<k8 && !kFreesB ? kLoadsB : 0, true>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (next < P) fa[next % kRing] = read_a(sa[kStageA], next % NB, next / NB);
            else fa[next % kRing] = read_a(sa[1 - kStageA], (next - P) % NB, (next - P) / NB);
            if constexpr (m == 0 && q + 1 < Q) read_b(fb[(q + 1) & 1], sb[kStageB], kPart * 2 + q + 1);
            if constexpr (p == P - kAhead) read_b(fb[0], sb[kNextB], kFirstB);
            if constexpr (p == 0)
                read_scales(std::integral_constant<int, 1 - kSet>{}, kFreesB ? macro + 1 : macro, k8 && !kFreesB ? 1 : 0);
            if constexpr (p >= P - kAhead) {
                // all loads of the rows, then those of the weights
                constexpr int k = p - (P - kAhead);
                constexpr int kAll = kLoadsA + (kFreesB ? kLoadsB : 0), kFrom = kAll * k / kAhead, kTo = kAll * (k + 1) / kAhead;
                oa.template load<(kFrom < kLoadsA ? kFrom : kLoadsA), (kTo < kLoadsA ? kTo : kLoadsA)>(sa[kStageA], wave);
                if constexpr (kTo > kLoadsA)
                    ob.template load<(kFrom > kLoadsA ? kFrom - kLoadsA : 0), kTo - kLoadsA>(sb[kStageB], wave);
                if constexpr (p == P - 1) {
                    oa.next();
                    if constexpr (kFreesB) ob.next();
                }
            }
            constexpr int kWord = k8 ? 0 : q / 2, kByte = (q & 1) * 2;
            if constexpr (SPLIT) {
                if constexpr (!kPipe) parts[p & 1] = split(fa[p % kRing]);
                const Split &x = parts[p & 1];
#pragma unroll
                for (int c = 0; c < 2; c++)
                    acc[0][m][c] = mfma_at<FORMAT, kByte>(fb[q & 1][c], x.hi, acc[0][m][c], wb[kSet][c][kWord],
                                                          wa[kSet][m][kWord]);
#pragma unroll
                for (int c = 0; c < 2; c++)
                    acc[1][m][c] = mfma_at<FORMAT, kByte>(fb[q & 1][c], x.lo, acc[1][m][c], wb[kSet][c][kWord],
                                                          wa[kSet][m][kWord]);
            } else {
#pragma unroll
                for (int c = 0; c < 2; c++)
                    acc[0][m][c] = mfma_at<FORMAT, kByte>(fb[q & 1][c], fa[p % kRing], acc[0][m][c], wb[kSet][c][kWord],
                                                          wa[kSet][m][kWord]);
            }
            if constexpr (kPipe) {
                parts[(p + 1) & 1] = split(fa[(p + 1) % kRing]);
                // a quarter of the splitting behind each matrix instruction
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        each(position, std::make_integer_sequence<int, P>{});
    };
    typedef std::integral_constant<int, 1> one;
    typedef std::integral_constant<int, 2> two;
    typedef std::integral_constant<int, 3> three;
    int macro = 0;
    for (; macro + 2 <= macros; macro += 2) {
        step(zero{}, macro);
        if constexpr (k8) {
            step(one{}, macro);
            step(two{}, macro + 1);
            step(three{}, macro + 1);
        } else {
            step(one{}, macro + 1);
        }
    }
    if (macro < macros) {
        step(zero{}, macro);
        if constexpr (k8) step(one{}, macro);
    }
    wait_for<0, true>();
}

template <int FORMAT, bool MX, int BM, int BC, int WM, int WC>
__global__ __launch_bounds__(WM *WC *kWave, 2) void k_mx_tile(const MxExpertArgs a) {
    typedef MxShape<FORMAT, BM, BC, WM, WC> S;
    constexpr bool SPLIT = MX && FORMAT == A2AV_MX_FP8;
    __shared__ __align__(16) unsigned char a0[BM * 128], a1[BM * 128], b0[BC * 128], b1[BC * 128];
    __shared__ u32x4 ss[4 * S::kScaleRows];
    unsigned char *const sa[2] = {a0, a1}, *const sb[2] = {b0, b1};
    if (status_at_entry(a.status)) return;
    // Workgroups go round the eight XCDs; each XCD takes a run of tiles of its own,
    // kGroup columns through an expert's row tiles.
    const uint32_t cols = (uint32_t)a.cols, tiles = (uint32_t)a.tiles[0];
    const uint32_t run = (tiles * cols + 7) / 8, at = (blockIdx.x & 7) * run + blockIdx.x / 8;
    if (blockIdx.x / 8 >= run || at >= tiles * cols) return;
    const int e = a.tiles[2 + 2 * (at / cols)];
    const uint32_t f = (uint32_t)a.first[e], n = (uint32_t)a.first[e + 1] - f;
    uint32_t i = at - f * cols;
    const uint32_t group = i / (n * kGroup), wide = min(cols - group * kGroup, kGroup);
    i -= group * n * kGroup;
    const int mt = (int)(i / wide), ct = (int)(group * kGroup + i % wide);
    const int d = e / a.P, j = e - d * a.P;
    const int64_t row0 = a.offsets[(int64_t)d * (a.P + 1) + j];
    const int64_t M = a.offsets[(int64_t)d * (a.P + 1) + j + 1] - row0;
    const bool glu = a.act == A2AV_ACT_SWIGLU;
    const int64_t m0 = (int64_t)mt * BM, c0 = (int64_t)ct * BC, left = M - m0;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WC, wc = wave % WC;
    const int64_t padded = mx_padded(a.K), x_bytes = mx_element_bytes(FORMAT, a.K), n0 = glu ? c0 / 2 : c0;
    const unsigned char *x = a.x[d] + (row0 + m0) * a.x_stride, *w = a.weight[d] + (int64_t)j * a.NW * a.w_stride;
    typename S::A oa;
    typename S::B ob;
    oa.init(x, nullptr, a.x_stride, left, x_bytes, wave, lane);
    ob.init(w + n0 * a.w_stride, glu ? w + (a.N + n0) * a.w_stride : nullptr, a.w_stride, a.N - n0, padded / 2, wave, lane);
    MxScales<BM, BC> os;
    {
        // a row outside has elements 0: any scale that is not NaN will do, and what a
        // NaN would make of it is not written
        const int r = threadIdx.x / 2;
        const int64_t c = weight_row(c0 + (r < BC ? r : 0), a.N, glu);
        os.x = x + (r < BM && r < left ? r : 0) * a.x_stride + x_bytes;
        os.w = w + (c < a.NW ? c : 0) * a.w_stride + padded / 2;
        os.last_x = (int)(a.x_stride - x_bytes) - 16;
        os.last_w = (int)(a.w_stride - padded / 2) - 16;
    }
    f32x16 acc[1 + SPLIT][S::kBlocksM][2] = {};
    const int macros = (int)(padded / kMxPad);
    if (S::kBlocksM >= 4 && left <= WM * 32)
        mx_contract<FORMAT, SPLIT, BM, BC, WM, WC, 1>(oa, ob, os, sa, sb, ss, macros, acc);
    else if (S::kBlocksM >= 2 && left <= WM * 32 * (S::kBlocksM / 2))
        mx_contract<FORMAT, SPLIT, BM, BC, WM, WC, (S::kBlocksM >= 2 ? S::kBlocksM / 2 : 1)>(oa, ob, os, sa, sb, ss, macros, acc);
    else
        mx_contract<FORMAT, SPLIT, BM, BC, WM, WC, S::kBlocksM>(oa, ob, os, sa, sb, ss, macros, acc);
    __syncthreads();
    // in passes of kPass row blocks, each wave in its own part of the stages
    constexpr int kPass = SPLIT || S::kBlocksM < 2 ? 1 : 2, kPlane = kPass * 32 * 64 * 4, kParts = S::kWaves / 4;
    constexpr bool kSpare = SPLIT && kPlane == BM * 128;  // the second sums of the last wave have no room in them
    static_assert(kParts * kPlane <= BM * 128 && (SPLIT ? 2 : 1) * kParts * kPlane <= BC * 128, "");
    static_assert(!SPLIT || (kParts == 1 && (kSpare || 2 * kPlane <= BM * 128)), "");
    __shared__ __align__(16) unsigned char spare[kSpare ? 2 * kPlane : 16];
    const int in = wave / kParts;
    f32x4 *sums, *low;
    if constexpr (kSpare) {
        sums = (f32x4 *)(in == 0 ? a0 : in == 1 ? b0 : in == 2 ? b1 : spare);
        low = (f32x4 *)(in == 0 ? a1 : (in == 1 ? b0 : in == 2 ? b1 : spare) + kPlane);
    } else {
        sums = (f32x4 *)((in == 0 ? a0 : in == 1 ? a1 : in == 2 ? b0 : b1) + wave % kParts * kPlane);
        low = sums + kPlane / 16;
    }
    const auto pass = [&](auto number) __attribute__((always_inline)) {
        constexpr int p = decltype(number)::value;
        if (p * kPass * WM * 32 >= left) return;
#pragma unroll
        for (int u = 0; u < kPass; u++)
#pragma unroll
            for (int v = 0; v < 2; v++) {
                put_sums<64>(sums, u, v, acc[0][p * kPass + u][v], lane);
                if constexpr (SPLIT) put_sums<64>(low, u, v, acc[1][p * kPass + u][v], lane);
            }
        asm volatile("" ::: "memory");
        emit<kPass * 32, 64, MX, SPLIT>(a, sums, low, d, j, row0, M, c0 + wc * 64, lane,
                                        [&](int r) { return m0 + ((p * kPass + (r >> 5)) * WM + wm) * 32 + (r & 31); });
        asm volatile("" ::: "memory");
    };
    each(pass, std::make_integer_sequence<int, S::kBlocksM / kPass>{});
}

// ------------------------------------------------------------------ few rows
// Experts with a few rows each (decoded tokens): what has to move is the weights,
// once, so they go from memory to the matrix cores' operands without LDS. A
// workgroup has 32 output columns (gated: the gate rows and the up rows behind
// them) of one tile of up to 16 rows; its waves take steps of 256 elements in turn,
// and their sums meet in LDS in wave order. Every workgroup checks the offsets and
// finds its tile in them by itself, which saves the launch of the plan (one row for each of
// 32 experts, K 1024, 512 columns: 12.4 us where the rank has 32 or 512 experts, 18.3 of
// 4096). One token's 8 experts, K 7168 and 4096 columns: 25 us, 4.9 TB/s of weights; 32
// experts of one row 89, 5.6; of 8 and 16 rows 107 and 118 where tiles take 140 and 136
// (K 2048, 7168 columns 60 and 72, tiles 62 and 62).
constexpr int kFewWaves = 4, kFewCols = 32;
constexpr int kFewMacros = 32;                       // steps of 256 elements whose scales LDS holds
constexpr int kFewScaleRow = kFewMacros * 8 + 16;    // LDS bytes of a row of them: rows in different banks

template <int FORMAT>
__device__ __forceinline__ f32x4 mfma_few(i32x4 w, i32x8 x, f32x4 c, uint32_t sw, uint32_t sx) {
    const i32x8 w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x, c, 4, FORMAT == A2AV_MX_FP8 ? 0 : 4, 0, (int)sw, 0,
                                                            (int)sx);
}

__device__ __forceinline__ i32x4 load16(rsrc_t b, uint32_t off) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}

// What the plan finds, for row tile t of kFewRows rows: false if the offsets are
// wrong (the first workgroup says so), or there are no more tiles. Every thread of
// every workgroup comes to the same verdict.
struct FewTile {
    int expert, tile;
    int64_t row0, rows;
};
template <int THREADS>
__device__ __forceinline__ bool find_tile(const MxExpertArgs &a, uint32_t t, FewTile &f) {
    __shared__ uint32_t part[THREADS / kWave];
    __shared__ FewTile found;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, n = a.W * a.P;
    const int per = (n + THREADS - 1) / THREADS, from = tid * per, to = min(from + per, n);
    int bad = 0;
    uint32_t sum = 0;
    for (int i = from; i < to; i++) {
        const int d = i / a.P, j = i - d * a.P;
        const int64_t *off = a.offsets + (int64_t)d * (a.P + 1) + j;
        const int64_t r0 = off[0], r1 = off[1];
        if ((j == 0 && r0 != 0) || r0 < 0 || r1 < r0) bad |= A2AV_ST_BAD_OFFSETS;
        else if (r1 > a.x_rows[d]) bad |= A2AV_ST_SEND_OVERRUN;
        else sum += (uint32_t)((r1 - r0 + kFewRows - 1) / kFewRows);
    }
    const uint32_t inc = wave_incl_scan_u32(sum);
    if (lane == kWave - 1) part[wave] = inc;
    if (tid == 0) found.expert = -1;
    const int off_bad = __syncthreads_or(bad & A2AV_ST_BAD_OFFSETS);
    const int run_bad = __syncthreads_or(bad & A2AV_ST_SEND_OVERRUN);
    if (off_bad | run_bad) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(a.status_out, off_bad ? A2AV_ST_BAD_OFFSETS : A2AV_ST_SEND_OVERRUN);
        return false;
    }
    uint32_t at = inc - sum;
    for (int w = 0; w < wave; w++) at += part[w];
    if (t >= at && t < at + sum) {
        for (int i = from; i < to; i++) {
            const int d = i / a.P, j = i - d * a.P;
            const int64_t *off = a.offsets + (int64_t)d * (a.P + 1) + j;
            const int64_t r0 = off[0], rows = off[1] - r0;
            const uint32_t mine = (uint32_t)((rows + kFewRows - 1) / kFewRows);
            if (t >= at && t < at + mine) found = {i, (int)(t - at), r0, rows};
            at += mine;
        }
    }
    __syncthreads();
    f.expert = __builtin_amdgcn_readfirstlane(found.expert);
    f.tile = __builtin_amdgcn_readfirstlane(found.tile);
    f.row0 = (int64_t)readlane_u64((uint64_t)found.row0, 0);
    f.rows = (int64_t)readlane_u64((uint64_t)found.rows, 0);
    return f.expert >= 0;
}

template <int FORMAT, bool GLU, bool MX>
__global__ __launch_bounds__(kFewWaves *kWave, 2) void k_mx_few(const MxExpertArgs a) {
    constexpr int kFrags = GLU ? 4 : 2, kCols = kFrags * 16, kChunks = kFewRows * kCols / 4;
    constexpr bool k8 = FORMAT == A2AV_MX_FP8;
    constexpr int kThreads = kFewWaves * kWave, kScaleRows = kCols + kFewRows;
    constexpr int kScaleLoads = (kScaleRows * kFewMacros / 2 + kThreads - 1) / kThreads;  // of 16 bytes a thread
    constexpr bool kTwo = MX && k8;
    // the scales, and then the waves' sums
    constexpr int kSums = (1 + kTwo) * kFewWaves * kChunks * 16, kScales = kScaleRows * kFewScaleRow;
    __shared__ __align__(16) unsigned char scales[kSums > kScales ? kSums : kScales];
    f32x4 *const sums = (f32x4 *)scales;  // [waves][1 or 2][kChunks]
    if (status_at_entry(a.status)) return;
    const uint32_t t = blockIdx.x / (uint32_t)a.cols, ct = blockIdx.x - t * a.cols;
    FewTile tile;
    if (!find_tile<kThreads>(a, t, tile)) return;
    const int d = tile.expert / a.P, j = tile.expert - d * a.P;
    const int64_t row0 = tile.row0 + (int64_t)tile.tile * kFewRows, n0 = (int64_t)ct * kFewCols;
    const int rows = (int)min(tile.rows - (int64_t)tile.tile * kFewRows, (int64_t)kFewRows);
    const int cols = (int)max(min(a.N - n0, (int64_t)kFewCols), (int64_t)0);
    const int lane = threadIdx.x & (kWave - 1), quarter = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t ws = (uint32_t)a.w_stride, xs = (uint32_t)a.x_stride;
    const unsigned char *w = a.weight[d] + ((int64_t)j * a.NW + n0) * a.w_stride;
    const rsrc_t bx = buffer(a.x[d] + row0 * a.x_stride, (uint32_t)rows * xs);
    const rsrc_t bw[2] = {buffer(w, (uint32_t)cols * ws), buffer(w + (GLU ? a.N * a.w_stride : 0), (uint32_t)cols * ws)};
    const uint32_t padded = (uint32_t)mx_padded(a.K), w_scales = padded / 2, x_scales = k8 ? padded : padded / 2;
    const int macros = (int)(padded / kMxPad);
    f32x4 acc[1 + kTwo][kFrags] = {};
    for (int from = 0; from < macros; from += kFewMacros) {
        const int to = min(from + kFewMacros, macros);
        // the scales of all rows for these steps, sixteen bytes a load, rows along the threads
        i32x4 sv[kScaleLoads];
#pragma unroll
        for (int i = 0; i < kScaleLoads; i++) {
            const int k = i * kThreads + threadIdx.x, row = k / (kFewMacros / 2), at = k % (kFewMacros / 2);
            const uint32_t byte = (uint32_t)(from * 8 + at * 16);
            // gated: gate and up blocks of 16 alternate
            const int wrow = GLU ? (row >> 5) * 16 + (row & 15) : row;
            const bool in = from + at * 2 < macros;
            if (row < kCols)
                sv[i] = load16(GLU && (row & 16) ? bw[1] : bw[0], in ? (uint32_t)wrow * ws + w_scales + byte : kOutside);
            else
                sv[i] = load16(bx, in ? (uint32_t)(row - kCols) * xs + x_scales + byte : kOutside);
        }
        bool stored = false;
        for (int macro = from + wave; macro < to || !stored; macro += kFewWaves) {
            i32x4 fw[kFrags][2], fx[2][2];
            const uint32_t out = macro < to ? 0 : kOutside;
#pragma unroll
            for (int f = 0; f < kFrags; f++) {
                const uint32_t row = (uint32_t)((GLU ? f >> 1 : f) * 16 + (lane & 15)) * ws;
                const rsrc_t b = bw[GLU ? f & 1 : 0];
#pragma unroll
                for (int s = 0; s < 2; s++) fw[f][s] = load16(b, (row + macro * 128 + quarter * 32 + s * 16) | out);
            }
            const uint32_t row = (uint32_t)(lane & 15) * xs;
#pragma unroll
            for (int s = 0; s < 2; s++) {
                if constexpr (k8) {
                    const uint32_t at = row + macro * 256 + (quarter >> 1) * 64 + s * 32 + (quarter & 1) * 16;
                    fx[s][0] = load16(bx, at | out);
                    fx[s][1] = load16(bx, (at + 128) | out);
                } else {
                    fx[s][0] = fx[s][1] = load16(bx, (row + macro * 128 + quarter * 32 + s * 16) | out);
                }
            }
            if (!stored) {
                if (from > 0) __syncthreads();  // the last steps' scales have been read
#pragma unroll
                for (int i = 0; i < kScaleLoads; i++) {
                    const int k = i * kThreads + threadIdx.x, r = k / (kFewMacros / 2), at = k % (kFewMacros / 2);
                    if (r < kScaleRows) *(i32x4 *)(scales + r * kFewScaleRow + at * 16) = sv[i];
                }
                __syncthreads();
                stored = true;
            }
            __builtin_amdgcn_sched_barrier(0);
            if (macro >= to) break;  // a wave without a step only stored scales
            const unsigned char *ps = scales + (lane & 15) * kFewScaleRow + (macro & (kFewMacros - 1)) * 8;
            u32x2 sw[kFrags], sx = *(const u32x2 *)(ps + kCols * kFewScaleRow);
#pragma unroll
            for (int f = 0; f < kFrags; f++) sw[f] = *(const u32x2 *)(ps + f * 16 * kFewScaleRow);
            // a lane's elements of product s are block 2 quarter + s of the eight
            const int shift = (quarter & 1) * 16;
            const auto word = [&](u32x2 v) { return (quarter & 2 ? v.y : v.x) >> shift; };
#pragma unroll
            for (int f = 0; f < kFrags; f++) sw[f].x = word(sw[f]);
            sx.x = word(sx);
#pragma unroll
            for (int s = 0; s < 2; s++) {
                const i32x8 x8 = __builtin_shufflevector(fx[s][0], fx[s][1], 0, 1, 2, 3, 4, 5, 6, 7);
                if constexpr (k8) {  // the matrix cores have time for both parts
                    const Split x = split(x8);
#pragma unroll
                    for (int f = 0; f < kFrags; f++) {
                        acc[0][f] = mfma_few<FORMAT>(fw[f][s], x.hi, acc[0][f], sw[f].x >> (s * 8), sx.x >> (s * 8));
                        acc[kTwo][f] = mfma_few<FORMAT>(fw[f][s], x.lo, acc[kTwo][f], sw[f].x >> (s * 8), sx.x >> (s * 8));
                    }
                } else {
#pragma unroll
                    for (int f = 0; f < kFrags; f++)
                        acc[0][f] = mfma_few<FORMAT>(fw[f][s], x8, acc[0][f], sw[f].x >> (s * 8), sx.x >> (s * 8));
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p <= kTwo; p++)
#pragma unroll
        for (int f = 0; f < kFrags; f++)
            sums[(wave * (1 + kTwo) + p) * kChunks + chunk<kCols>(lane & 15, f * 4 + quarter)] = acc[p][f];
    __syncthreads();
    // with two sums in double, which leave as two numbers again
    for (int k = threadIdx.x; k < kChunks; k += kThreads) {
        if constexpr (kTwo) {
            f32x4 y, rest;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                double t = 0.0;
#pragma unroll
                for (int i = 0; i < 2 * kFewWaves; i++) t += (double)sums[i * kChunks + k][c];
                y[c] = (float)t;
                rest[c] = __builtin_isinf(y[c]) ? 0.0f : (float)(t - y[c]);
            }
            sums[k] = y;
            sums[kChunks + k] = rest;
        } else {
            f32x4 y = sums[k];
#pragma unroll
            for (int i = 1; i < kFewWaves; i++) y += sums[i * kChunks + k];
            sums[k] = y;
        }
    }
    __syncthreads();
    if (wave != 0) return;
    emit_rows<kFewRows, kCols, GLU, MX, kTwo>(a, sums, sums + kChunks, d, j, row0, rows, (int64_t)ct * kCols, lane,
                                              [](int r) { return (int64_t)r; });
}

// ------------------------------------------------------------------ host
// Product columns that have outputs: with microscaled rows their padding too.
static int64_t product_columns(const MxExpertArgs &a) {
    const int64_t n = a.out_type == kOutMx ? mx_padded(a.N) : a.N;
    return a.act == A2AV_ACT_SWIGLU ? (n + 15) / 16 * 32 : n;
}

// Tile shapes, largest first.
enum { kBig, kMid, kSmall, kFew };
constexpr int kRows[] = {256, 128, 64, kFewRows}, kCols[] = {256, 128, 128};

// Of 8-bit rows with outputs of 8 bits there are no tiles of 256: their two sums would
// take all registers (16384 ragged rows on 32 experts, K 7168, 4096 columns: 757 us in
// tiles of 128; with one sum in tiles of 256 745; equal experts 769 and 705).
// The largest tile of which the product has enough to fill the compute units, R
// rows over n experts, C product columns, and which the mean expert more than half
// fills (32 experts of 64, 128 and 192 rows, 4-bit rows, K 7168, 4096 columns: 106,
// 164 and 210 us in tiles of 64, 107, 125 and 175 of 128, 114, 127 and 146 of 256; of
// 8-bit rows with K 2048 and 7168 columns 69, 103, 141; 69, 87, 124; 78, 93, 132).
static int shape_of(int64_t R, int64_t n, int64_t C, bool two) {
    for (int s = R <= 64 * n ? kSmall : R <= 128 * n || two ? kMid : kBig; s < kSmall; s++) {
        const int64_t t = kRows[s], cols = (C + kCols[s] - 1) / kCols[s];
        const int64_t tiles = R / t + (R % (n * t) ? n / 2 : 0);
        if (tiles * cols >= 200) return s;
    }
    return kSmall;
}

template <int FORMAT, bool MX>
static void launch_few(const MxExpertArgs &a, int64_t tiles, hipStream_t stream) {
    const dim3 g((unsigned)(tiles ? tiles * a.cols : 1)), b(kFewWaves * kWave);  // without rows the offsets are still checked
    if (a.act == A2AV_ACT_SWIGLU) hipLaunchKernelGGL((k_mx_few<FORMAT, true, MX>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((k_mx_few<FORMAT, false, MX>), g, b, 0, stream, a);
}

template <int FORMAT, bool MX>
static void launch_tile(const MxExpertArgs &a, int shape, int64_t tiles, hipStream_t stream) {
    const dim3 g((unsigned)((tiles * a.cols + 7) / 8 * 8));
    if constexpr (FORMAT == A2AV_MX_FP4 || !MX)
        if (shape == kBig) {
            hipLaunchKernelGGL((k_mx_tile<FORMAT, MX, 256, 256, 2, 4>), g, dim3(512), 0, stream, a);
            return;
        }
    if (shape == kMid) hipLaunchKernelGGL((k_mx_tile<FORMAT, MX, 128, 128, 2, 2>), g, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_mx_tile<FORMAT, MX, 64, 128, 2, 2>), g, dim3(256), 0, stream, a);
}

template <int FORMAT, bool MX>
static void launch(const MxExpertArgs &a, int shape, int64_t tiles, hipStream_t stream) {
    if (shape == kFew) launch_few<FORMAT, MX>(a, tiles, stream);
    else launch_tile<FORMAT, MX>(a, shape, tiles, stream);
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
        a.wide = a.wide && aligned16(out[d]);
    }
    a.offsets = expert_offsets;
    a.tiles = (const int32_t *)workspace;
    a.first = (const int32_t *)((unsigned char *)workspace + l.first);
    a.status = a.status_out = status;
    a.W = W;
    a.P = P;
    int64_t R = 0;
    for (int d = 0; d < W; d++) R += a.x_rows[d] = x_rows[d];
    const bool mx = a.out_type == kOutMx, two = mx && x_format == A2AV_MX_FP8;
    // few rows: the two meet between 12 and 16 rows an expert
    int shape = R <= 12 * (int64_t)W * P ? kFew : shape_of(R, (int64_t)W * P, product_columns(a), two);
    const auto tiles_of = [&](int s) {
        const int64_t t = most_tiles(x_rows, W, P, kRows[s]);
        return R < t ? R : t;
    };
    const auto cols_of = [&](int s) {
        const int64_t n = a.out_type == kOutMx ? mx_padded(N) : N;
        return s == kFew ? (n + kFewCols - 1) / kFewCols : (product_columns(a) + kCols[s] - 1) / kCols[s];
    };
    while (shape > (two ? kMid : kBig) && tiles_of(shape) * cols_of(shape) > kMostGroups) shape--;
    const int64_t tiles = tiles_of(shape);
    a.cols = (int)cols_of(shape);
    if (tiles * a.cols > kMostGroups) return A2AV_EARG;
    if (shape != kFew)
        launch_plan(W, P, x_rows, expert_offsets, kRows[shape], (unsigned char *)workspace, l, status, stream);
    if (x_format == A2AV_MX_FP4 && mx) launch<A2AV_MX_FP4, true>(a, shape, tiles, stream);
    else if (x_format == A2AV_MX_FP4) launch<A2AV_MX_FP4, false>(a, shape, tiles, stream);
    else if (mx) launch<A2AV_MX_FP8, true>(a, shape, tiles, stream);
    else launch<A2AV_MX_FP8, false>(a, shape, tiles, stream);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
