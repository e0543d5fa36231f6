// experts.hip — the experts' products on expert-major rows, and their gradient
// (gfx950).
//
// Rank d's rows lie expert by expert (expert_offsets[d]), so every product is
// a batch of matrix products whose row counts only the device knows:
//   forward    out = act(x . W_e^T + b_e) + residual   contraction over K
//   d_x        d_pre . W_e                             contraction over NW
//   d_weight   d_pre^T . x                             contraction over rows
//
//   k_expert_plan   checks the offsets, lists the row tiles of all experts
//   k_expert_tile   one tile of one product, 16-byte rows
//   k_expert_few    16 columns of up to 16 rows, which read their weights once
//   k_expert_any    one 64 x 64 tile of one product, any size and alignment
//   k_expert_dpre   d_pre = d_out * act'(pre), with the bias sums of row blocks
//   k_expert_dbias  the bias sums of an expert's row blocks, in order
#include <hip/hip_runtime.h>

#include <cstring>

#include "common.hpp"

namespace a2av {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

enum { kForward, kDx, kDweight };

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

// act'(h).
__device__ __forceinline__ float act_slope(int act, float h) {
    switch (act) {
    case A2AV_ACT_RELU: return h <= 0.0f ? 0.0f : 1.0f;
    case A2AV_ACT_GELU: {
        const float e = __expf(-0.5f * h * h);
        return normal_cdf(h, e) + h * 0.39894228f * e;
    }
    case A2AV_ACT_SILU: {
        const float s = sigmoid(h);
        return s * (1.0f + h * (1.0f - s));
    }
    default: return 1.0f;
    }
}

// ------------------------------------------------------------------ plan
struct PlanArgs {
    int64_t x_rows[A2AV_MAX_W];
    const int64_t *offsets;  // [W][P + 1]
    int32_t *tiles;          // [0] tile count, then (expert, tile of the expert) pairs
    int32_t *first;          // [W * P + 1] first tile of each expert
    int32_t *status;
    int W, P;
    int tile_rows;
};

// One workgroup. Thread t owns up to kPlanPer consecutive experts of the
// W * P; a scan of their tile counts gives every expert its first tile, and
// the threads then fill the list tile by tile (a search in the scan), so that
// one expert with most of the rows does not leave the list to one thread.
__global__ __launch_bounds__(kPlanThreads) void k_expert_plan(const PlanArgs a) {
    __shared__ int32_t first[A2AV_MAX_EXPERTS + 1];
    __shared__ int32_t part[kPlanThreads / kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int n = a.W * a.P;
    int bad = 0;
    uint32_t mine[kPlanPer], sum = 0;
#pragma unroll
    for (int u = 0; u < kPlanPer; u++) {
        const int i = tid * kPlanPer + u;
        mine[u] = 0;
        if (i < n) {
            const int d = i / a.P, j = i - d * a.P;
            const int64_t *off = a.offsets + (int64_t)d * (a.P + 1) + j;
            const int64_t r0 = off[0], r1 = off[1];
            if ((j == 0 && r0 != 0) || r0 < 0 || r1 < r0) bad |= A2AV_ST_BAD_OFFSETS;
            else if (r1 > a.x_rows[d]) bad |= A2AV_ST_SEND_OVERRUN;
            else mine[u] = (uint32_t)((r1 - r0 + a.tile_rows - 1) / a.tile_rows);
        }
        sum += mine[u];
    }
    const int off_bad = __syncthreads_or(bad & A2AV_ST_BAD_OFFSETS);
    const int run_bad = __syncthreads_or(bad & A2AV_ST_SEND_OVERRUN);
    const int poisoned = __syncthreads_or(tid == 0 ? status_poisoned(a.status) : 0);
    if (poisoned) return;
    if (off_bad | run_bad) {
        // descending offsets alone: what lies past x_rows then says nothing
        if (tid == 0) atomicOr(a.status, off_bad ? A2AV_ST_BAD_OFFSETS : A2AV_ST_SEND_OVERRUN);
        return;
    }
    const uint32_t inc = wave_incl_scan_u32(sum);
    if (lane == kWave - 1) part[wave] = (int32_t)inc;
    __syncthreads();
    uint32_t at = inc - sum, total = 0;
    for (int w = 0; w < kPlanThreads / kWave; w++) {
        if (w < wave) at += (uint32_t)part[w];
        total += (uint32_t)part[w];
    }
#pragma unroll
    for (int u = 0; u < kPlanPer; u++) {
        const int i = tid * kPlanPer + u;
        if (i < n) first[i] = a.first[i] = (int32_t)at;
        at += mine[u];
    }
    if (tid == 0) {
        first[n] = a.first[n] = (int32_t)total;
        a.tiles[0] = (int32_t)total;
    }
    __syncthreads();
    for (uint32_t t = tid; t < total; t += kPlanThreads) {
        int lo = 0, hi = n;  // the last expert whose first tile is at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if ((uint32_t)first[mid] <= t) lo = mid;
            else hi = mid;
        }
        a.tiles[2 + 2 * t] = lo;
        a.tiles[3 + 2 * t] = (int32_t)t - first[lo];
    }
}

// ------------------------------------------------------------------ products
struct ExpertArgs {
    const void *a[A2AV_MAX_W];         // x (forward), d_pre (gradients)
    const void *b[A2AV_MAX_W];         // weight (forward, d_x), x (d_weight)
    const void *bias[A2AV_MAX_W];      // forward
    const void *residual[A2AV_MAX_W];  // forward
    void *out[A2AV_MAX_W];             // out, d_x, d_weight
    void *pre[A2AV_MAX_W];             // forward
    const int64_t *offsets;
    const int32_t *tiles;
    const int32_t *first;
    const int32_t *status;
    int64_t K, N, NW;
    int W, P;
    int act;
    int has_bias, has_residual, has_pre;
    int cols;       // column tiles of the fast product
    int row_tiles;  // of d_weight
};

// The weight row behind column c of the product: with SwiGLU, blocks of 16
// gate columns and the 16 up columns of the same outputs alternate, so that
// one lane ends with both.
__device__ __forceinline__ int64_t weight_row(int64_t c, int64_t N, bool glu) {
    if (!glu) return c;
    return ((c >> 4) & 1) * N + ((c >> 5) << 4) + (c & 15);
}

constexpr int kAny = 64;       // tile rows and columns
constexpr int kAnyK = 32;      // contraction step
constexpr int kAnyPad = 40;    // LDS row, in elements

// One 64 x 64 tile by four waves of 32 x 32, elements loaded one by one with
// their bounds checked; what lies outside is 0 in both operands, so it adds
// nothing even where the other holds infinities or NaN.
// Bound by those loads: 16384 rows, K 7168, NW 4096 at a base that is no 16-byte
// multiple 13.0 / 17.3 / 15.4 ms (forward / d_x / d_weight; 1.0 / 1.0 / 1.2 ms by
// 16-byte rows).
template <int KIND, typename T>
__global__ __launch_bounds__(256) void k_expert_any(const ExpertArgs a) {
    __shared__ __align__(16) uint16_t sa[kAny * kAnyPad], sb[kAny * kAnyPad];
    if (status_at_entry(a.status)) return;
    int e, mt;
    if constexpr (KIND == kDweight) {
        e = blockIdx.z;
        mt = blockIdx.y;
    } else {
        const int t = blockIdx.y + gridDim.y * blockIdx.z;
        if (t >= a.tiles[0]) return;
        e = a.tiles[2 + 2 * t];
        mt = a.tiles[3 + 2 * t];
    }
    const int d = e / a.P, j = e - d * a.P;
    const int64_t row0 = a.offsets[(int64_t)d * (a.P + 1) + j];
    const int64_t rows = a.offsets[(int64_t)d * (a.P + 1) + j + 1] - row0;
    const bool glu = KIND == kForward && a.act == A2AV_ACT_SWIGLU;
    const int64_t M = KIND == kDweight ? a.NW : rows;
    const int64_t C = KIND == kForward ? (glu ? (a.N + 15) / 16 * 32 : a.N) : a.K;
    const int64_t L = KIND == kForward ? a.K : KIND == kDx ? a.NW : rows;
    const int64_t m0 = (int64_t)mt * kAny, c0 = (int64_t)blockIdx.x * kAny;
    const uint16_t *pa = (const uint16_t *)a.a[d], *pb = (const uint16_t *)a.b[d];
    if constexpr (KIND == kForward) pa += row0 * a.K;
    else pa += row0 * a.NW;
    if constexpr (KIND == kDweight) pb += row0 * a.K;
    else pb += (int64_t)j * a.NW * a.K;
    const auto at_a = [&](int64_t m, int64_t k) -> uint16_t {
        if (m >= M || k >= L) return 0;
        if constexpr (KIND == kDweight) return pa[k * a.NW + m];
        return pa[m * L + k];
    };
    const auto at_b = [&](int64_t c, int64_t k) -> uint16_t {
        if (c >= C || k >= L) return 0;
        if constexpr (KIND == kForward) {
            const int64_t w = weight_row(c, a.N, glu);
            if (glu && w - ((c >> 4) & 1) * a.N >= a.N) return 0;
            return pb[w * a.K + k];
        }
        return pb[k * a.K + c];
    };
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int wm = (wave >> 1) * 32, wc = (wave & 1) * 32;
    f32x4 acc[2][2] = {};
    for (int64_t k0 = 0; k0 < L; k0 += kAnyK) {
#pragma unroll
        for (int u = 0; u < kAny * kAnyK / 256; u++) {
            const int i = tid + u * 256;
            // neighbouring threads along what is contiguous in memory
            const int ar = KIND == kDweight ? i % kAny : i / kAnyK, ak = KIND == kDweight ? i / kAny : i % kAnyK;
            const int br = KIND == kForward ? i / kAnyK : i % kAny, bk = KIND == kForward ? i % kAnyK : i / kAny;
            sa[ar * kAnyPad + ak] = at_a(m0 + ar, k0 + ak);
            sb[br * kAnyPad + bk] = at_b(c0 + br, k0 + bk);
        }
        __syncthreads();
        typename T::frag fa[2], fb[2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            fa[u] = *(const typename T::frag *)&sa[(wm + u * 16 + (lane & 15)) * kAnyPad + (lane >> 4) * 8];
            fb[u] = *(const typename T::frag *)&sb[(wc + u * 16 + (lane & 15)) * kAnyPad + (lane >> 4) * 8];
        }
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int v = 0; v < 2; v++) acc[u][v] = T::mfma(fa[u], fb[v], acc[u][v]);
        __syncthreads();
    }
    // lane l holds column l % 16 and rows (l / 16) * 4 .. + 3 of each 16 x 16
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t m = m0 + wm + u * 16 + (lane >> 4) * 4 + i;
            if (m >= M) continue;
            if constexpr (KIND == kForward) {
                const int64_t row = row0 + m;
                const uint16_t *bias = (const uint16_t *)a.bias[d] + (int64_t)j * a.NW;
                float y[2];
                int64_t n[2];
                int outs = 2;
                if (glu) {
                    n[0] = ((c0 + wc) >> 1) + (lane & 15);
                    if (n[0] >= a.N) continue;
                    float h0 = acc[u][0][i], h1 = acc[u][1][i];
                    if (a.has_bias) {
                        h0 += T::to_float(bias[n[0]]);
                        h1 += T::to_float(bias[a.N + n[0]]);
                    }
                    if (a.has_pre) {
                        uint16_t *pre = (uint16_t *)a.pre[d] + row * a.NW;
                        pre[n[0]] = T::from_float(h0);
                        pre[a.N + n[0]] = T::from_float(h1);
                    }
                    y[0] = h0 * sigmoid(h0) * h1;
                    outs = 1;
                } else {
                    for (int v = 0; v < 2; v++) {
                        n[v] = c0 + wc + v * 16 + (lane & 15);
                        float h = acc[u][v][i];
                        if (n[v] < a.N) {
                            if (a.has_bias) h += T::to_float(bias[n[v]]);
                            if (a.has_pre) ((uint16_t *)a.pre[d])[row * a.NW + n[v]] = T::from_float(h);
                        }
                        y[v] = act_of(a.act, h);
                    }
                }
                for (int v = 0; v < outs; v++) {
                    if (n[v] >= a.N) continue;
                    if (a.has_residual) y[v] += T::to_float(((const uint16_t *)a.residual[d])[row * a.N + n[v]]);
                    ((uint16_t *)a.out[d])[row * a.N + n[v]] = T::from_float(y[v]);
                }
            } else {
                uint16_t *out = (uint16_t *)a.out[d] + (KIND == kDx ? (row0 + m) * a.K : ((int64_t)j * a.NW + m) * a.K);
#pragma unroll
                for (int v = 0; v < 2; v++) {
                    const int64_t c = c0 + wc + v * 16 + (lane & 15);
                    if (c < C) out[c] = T::from_float(acc[u][v][i]);
                }
            }
        }
}

// ------------------------------------------------------------------ the fast products
// Tiles of BM rows and BC columns, a contraction step of 64 (whole 128-byte
// lines), both operands through LDS stages that buffer loads fill directly
// (three of the rows' operand, two of the other). An operand comes in one of
// two forms, by what its memory holds contiguously:
//   along the contraction (x and weight forward, d_pre for d_x): LDS rows of
//     64 elements, the eight 16-byte chunks of row r permuted by r % 8, read
//     as 16-byte fragments;
//   along the tile's rows or columns (the others): LDS rows are contraction
//     steps of BM or BC elements, 32-byte units permuted by the row, read with
//     the transposing LDS load (4 contraction steps x 16 columns a group).
// The second permutation puts the lanes of one LDS access in different banks;
// with the first, conflicts are counted for half of the forward product's LDS
// cycles and a third of d_x's.
// Rows, columns and contraction steps outside are loaded out of the buffer's
// range, which writes zeros to LDS; so the last steps can go on loading what
// nobody reads, and every step waits for the same number of loads.
//
// What bounds it, K 7168 and 4096 columns in bf16 (one library product of 16384
// rows: 615-650 us). 32 equal experts of 512 rows: 806-820 us, 1.2 PFLOP/s, the
// matrix cores' power (the clock falls to 1.5 GHz). Ragged ones (lognormal):
// 990-1020 us, and 585-640 against 490-580 at 256 rows an expert: a last row
// tile of a few rows still loads all of its columns' weights, step by step, and
// so takes most of a full tile's time; with 256 workgroups at once the calls
// take as many rounds as the fullest compute unit has tiles. There the matrix
// cores are busy 60 % of the cycles, and 3.6 GB are read, weights once 1.9 GB.
// d_x of 256 rows an expert: 3.5 rounds of tiles run as 4, 50 % busy; d_weight
// on the middle tiles 33 % (eight steps of sums, then 64 KiB of them through
// LDS and 1.9 GB of stores).
//
// Other shapes at 16384 rows, same box, all three products (forward / d_x /
// d_weight, us through): eight waves and two stages of 64 with one barrier a
// step 848 / 849 / spills; two groups of waves in turn at reading and
// multiplying 928 / 778 / 852; four stages of 32, whose 64-byte requests double
// the L2's work, 920 / 834 / 755; four waves of 128 x 128, half the LDS reads
// but no second wave to issue beside a stalled one, 889 / 818 / 825; this one
// 875 / 811 / 808.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

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

// The 32-byte unit of LDS row r that holds unit 0 of a contraction-major
// operand with COLS columns is the one at this number; the others by xor. Of
// an access's eight rows (0 .. 3 and 8 .. 11 of 16) and two units, as many as
// the row's length allows are in different banks.
template <int COLS>
__device__ __forceinline__ int unit_shift(int r) {
    if constexpr (COLS == 256) return (r & 3) << 1 | ((r >> 3) & 1) << 3;
    else if constexpr (COLS == 128) return (r & 3) << 1;
    else return ((r >> 1) & 1) << 1;
}

// One operand of a tile: where its elements are and how they reach LDS, step
// after step. ROWS: tile rows (or columns); MAJOR: contiguous along the
// contraction. The byte offsets of a thread's loads are kept in registers and
// one buffer serves all loads of a step: beside a wave's matrix instructions
// there is little room to issue anything else.
template <int ROWS, int THREADS, bool MAJOR, int STEP>
struct Operand {
    static_assert(!MAJOR || STEP == 64, "");
    static constexpr int kLoads = ROWS * STEP / 8 / THREADS;  // 16-byte loads a thread and step
    static constexpr int kWaves = THREADS / kWave;
    static constexpr int kPer = ROWS / 8;                      // not MAJOR: lanes a memory row
    // loads that the first `most` rows take
    static constexpr int loads(int most) {
        return !MAJOR || most >= ROWS ? kLoads : (most + kWaves * 8 - 1) / (kWaves * 8);
    }
    const unsigned char *base;   // MAJOR: row 0 of the tile; else the next step's row 0, column 0
    uint32_t stride;             // bytes of a memory row
    uint32_t span;               // bytes of the buffer: MAJOR the tile's rows, else a step's
    uint32_t off[kLoads];
    int left;                    // contraction elements from the next step on
    int at;                      // MAJOR: byte offset of the next step
    int k;                       // MAJOR: this lane's element of a step

    // MAJOR: `rows` rows from p, ld elements wide, all of them contraction.
    // A gated product takes blocks of 16 rows from p and p2 in turn; a wave's
    // loads are all of the one or of the other.
    __device__ __forceinline__ void along(const uint16_t *p, const uint16_t *p2, int64_t ld, int64_t rows, int wave,
                                          int lane) {
        static_assert(kWaves % 4 == 0, "");
        const int64_t most = p2 ? ROWS / 2 : ROWS;
        base = (const unsigned char *)(p2 && ((wave >> 1) & 1) ? p2 : p);
        stride = (uint32_t)ld * 2;
        left = (int)ld;
        at = 0;
        span = (uint32_t)(rows < most ? rows : most) * stride;
        k = ((lane & 7) ^ (lane >> 3)) * 8;
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int r = (i * kWaves + wave) * 8;
            off[i] = (uint32_t)((p2 ? (r >> 5) * 16 + (r & 8) : r) + (lane >> 3)) * stride + k * 2;
        }
    }
    // The memory row of a step that load i of a wave begins with: the row bits
    // that unit_shift goes by (0, 1 and 3) come from the wave and the lane.
    static __device__ __forceinline__ int first(int i, int wave) {
        static_assert(kWaves == (kPer == 32 ? 8 : 4), "");
        if constexpr (kPer == 32) return (wave & 1) << 1 | (wave >> 1) << 3 | (i & 1) << 2 | (i >> 1) << 5;
        else if constexpr (kPer == 16) return wave << 3 | (i & 1) << 2 | (i >> 1) << 5;
        else return wave << 3 | i << 5;
    }
    // Not MAJOR: `steps` memory rows of ld elements from p, columns c0 .. of cols.
    __device__ __forceinline__ void across(const uint16_t *p, int64_t ld, int64_t steps, int64_t c0, int64_t cols,
                                           int wave, int lane) {
        base = (const unsigned char *)(p + c0);
        stride = (uint32_t)ld * 2;
        left = (int)steps;
        const int row = lane / kPer, in = lane % kPer;
        const int c = ((((in >> 1) ^ unit_shift<ROWS>(row | first(0, wave))) << 1) | (in & 1)) * 8;
#pragma unroll
        for (int i = 0; i < kLoads; i++)
            off[i] = c0 + c < cols ? (uint32_t)(first(i, wave) + row) * stride + c * 2 : kOutside;
        span = (uint32_t)min(left, STEP) * stride;
    }
    // The next step's loads into an LDS stage; rows at or past MOST of a MAJOR
    // operand are not needed.
    template <int MOST>
    __device__ __forceinline__ void load(uint16_t *lds, int wave) {
        part<MOST, 0, 1>(lds, wave);
    }
    // Part P of N of them, in order.
    template <int MOST, int P, int N>
    __device__ __forceinline__ void part(uint16_t *lds, int wave) {
        constexpr int kAll = loads(MOST), kFrom = kAll * P / N, kTo = kAll * (P + 1) / N;
        const rsrc_t b = buffer(base, span);
        if constexpr (MAJOR) {
            const uint32_t out = k < left ? 0 : kOutside;
#pragma unroll
            for (int i = kFrom; i < kTo; i++)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void *)(lds + (i * kWaves + wave) * 8 * STEP), 16,
                                                         (int)(off[i] | out), at, 0, 0);
            if constexpr (P + 1 == N) at += STEP * 2;
        } else {
#pragma unroll
            for (int i = kFrom; i < kTo; i++)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void *)(lds + first(i, wave) * ROWS), 16, (int)off[i],
                                                         0, 0, 0);
        }
        if constexpr (P + 1 == N) {
            left -= STEP;
            if constexpr (!MAJOR) {
                base += (uint64_t)STEP * stride;
                span = (uint32_t)min(max(left, 0), STEP) * stride;
            }
        }
    }
};

// Where a lane's part of a 32 x 16 fragment is in an LDS stage: row lane % 32,
// contraction elements (lane / 32) * 8 .. + 7. The values are made opaque for
// every read: the addresses are cheap beside the matrix instructions, and
// keeping them all in registers makes the kernel spill.
template <typename T, int ROWS, bool MAJOR>
struct Reader {
    int base, shift;
    __device__ __forceinline__ explicit Reader(int lane) {
        if constexpr (MAJOR) {
            base = (lane & 31) * 64 + (((lane >> 5) ^ (lane & 7)) << 3);
            shift = 0;
        } else {
            // groups of 16 lanes take 4 contraction steps of 16 columns
            const int r = (lane >> 5) * 8 + ((lane >> 2) & 3);
            base = r * ROWS + (lane & 3) * 4;
            shift = unit_shift<ROWS>(r) ^ ((lane >> 4) & 1);
        }
    }
    __device__ __forceinline__ void refresh() { asm volatile("" : "+v"(base), "+v"(shift)); }
    // tile row `row` (a multiple of 32), quarter q of a step
    __device__ __forceinline__ typename T::frag operator()(const uint16_t *lds, int row, int q) const {
        if constexpr (MAJOR) {
            return *(const typename T::frag *)(lds + (base ^ q * 16) + row * 64);
        } else {
            const uint16_t *p = lds + base + (((row >> 4) ^ shift) << 4) + q * 16 * ROWS;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * ROWS));
            return __builtin_bit_cast(typename T::frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

template <int KIND, int BM, int BC, int WM, int WC, int STEP>
struct Shape {
    static constexpr int kThreads = WM * WC * kWave;
    static constexpr bool kMajorA = KIND != kDweight, kMajorB = KIND == kForward;
    static constexpr int kBlocksM = BM / WM / 32, kBlocksC = BC / WC / 32;
    typedef Operand<BM, kThreads, kMajorA, STEP> A;
    typedef Operand<BC, kThreads, kMajorB, STEP> B;
};

// The contraction of one tile with NB row blocks a wave: the blocks of the
// waves alternate, so that a tile with few rows keeps all of them busy. Each
// quarter step's fragments are read while the quarter before is multiplied.
// Before the last quarter every wave has read all of the step's stages: one
// barrier there frees them for later loads, and publishes the next step's. A
// has three stages and B two, which is what 160 KiB hold of the largest
// tiles: B's loads then have one step to arrive in and A's two.
template <int KIND, typename T, int BM, int BC, int WM, int WC, int STEP, int NB>
__device__ __forceinline__ void contract(typename Shape<KIND, BM, BC, WM, WC, STEP>::A &oa,
                                         typename Shape<KIND, BM, BC, WM, WC, STEP>::B &ob, uint16_t *const (&sa)[3],
                                         uint16_t *const (&sb)[2],
                                         f32x16 (&acc)[Shape<KIND, BM, BC, WM, WC, STEP>::kBlocksM]
                                                      [Shape<KIND, BM, BC, WM, WC, STEP>::kBlocksC]) {
    typedef Shape<KIND, BM, BC, WM, WC, STEP> S;
    typedef typename T::frag frag;
    constexpr int kMost = NB * WM * 32, kLoadsA = S::A::loads(kMost), kLoadsB = S::B::kLoads;
    constexpr int kReads = NB * (S::kMajorA ? 1 : 2) + S::kBlocksC * (S::kMajorB ? 1 : 2);  // of a quarter step
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WC, wc = wave % WC;
    const int steps = (oa.left + STEP - 1) / STEP;
    constexpr int kQuarters = STEP / 16;
    if (steps == 0) return;  // an expert without rows: its d_weight is 0
    Reader<T, BM, S::kMajorA> ra(lane);
    Reader<T, BC, S::kMajorB> rb(lane);
    const auto read = [&](frag(&fa)[NB], frag(&fb)[S::kBlocksC], const uint16_t *a, const uint16_t *b, int q)
                          __attribute__((always_inline)) {
        ra.refresh();
        rb.refresh();
#pragma unroll
        for (int c = 0; c < S::kBlocksC; c++) fb[c] = rb(b, (wc * S::kBlocksC + c) * 32, q);
#pragma unroll
        for (int m = 0; m < NB; m++) fa[m] = ra(a, (m * WM + wm) * 32, q);
    };
    const auto multiply = [&](const frag(&fa)[NB], const frag(&fb)[S::kBlocksC]) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < NB; m++)
#pragma unroll
            for (int c = 0; c < S::kBlocksC; c++) acc[m][c] = T::mfma(fb[c], fa[m], acc[m][c]);
    };
    // reads, loads and products in turn, the reads in front
    const auto mix = [](auto loads) __attribute__((always_inline)) {
        constexpr int kProducts = NB * S::kBlocksC, kL = decltype(loads)::value;
        constexpr int kEachRead = (kReads + kProducts - 1) / kProducts, kEachLoad = (kL + kProducts - 1) / kProducts;
#pragma unroll
        for (int i = 0; i < kProducts; i++) {
            __builtin_amdgcn_sched_group_barrier(0x100, kEachRead, 0);
            if constexpr (kL > 0) __builtin_amdgcn_sched_group_barrier(0x020, kEachLoad, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
    };
    frag fa[2][NB], fb[2][S::kBlocksC];
    oa.template load<kMost>(sa[0], wave);
    ob.template load<BC>(sb[0], wave);
    oa.template load<kMost>(sa[1], wave);
    ob.template load<BC>(sb[1], wave);
    wait_for<kLoadsA + kLoadsB, false>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(fa[0], fb[0], sa[0], sb[0], 0);
    // Quarter q of step i's sequence (a step of 32 has two); the loads that
    // barrier i frees the stages for are spread over it and the quarters
    // after: B's, which are needed first, then A's.
    const auto quarter = [&](int i, auto q) __attribute__((always_inline)) {
        constexpr int kQ = decltype(q)::value, kParts = kQuarters - 1;
        if constexpr (kQ < kParts) read(fa[(kQ + 1) & 1], fb[(kQ + 1) & 1], sa[i % 3], sb[i % 2], kQ + 1);
        else read(fa[0], fb[0], sa[(i + 1) % 3], sb[(i + 1) % 2], 0);
        if constexpr (kQ == kParts) ob.template load<BC>(sb[i % 2], wave);
        else oa.template part<kMost, kQ, kParts>(sa[(i + 2) % 3], wave);
        multiply(fa[kQ & 1], fb[kQ & 1]);
        constexpr int kL = kQ == kParts ? kLoadsB : kLoadsA * (kQ + 1) / kParts - kLoadsA * kQ / kParts;
        mix(std::integral_constant<int, kL>{});
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto step = [&](int i) __attribute__((always_inline)) {
        quarter(i, std::integral_constant<int, 0>{});
        if constexpr (kQuarters == 4) {
            quarter(i, std::integral_constant<int, 1>{});
            quarter(i, std::integral_constant<int, 2>{});
        }
        wait_for<kLoadsA, true>();  // all but A's loads of the step after the next
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        quarter(i, std::integral_constant<int, kQuarters - 1>{});
    };
    int s = 0;
    for (; s + 6 <= steps; s += 6) {
#pragma unroll
        for (int i = 0; i < 6; i++) step(i);
    }
    if (s < steps) step(0);
    if (s + 1 < steps) step(1);
    if (s + 2 < steps) step(2);
    if (s + 3 < steps) step(3);
    if (s + 4 < steps) step(4);
    wait_for<0, true>();
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

template <int KIND, typename T, int BM, int BC, int WM, int WC, int STEP>
__global__ __launch_bounds__(WM *WC *kWave, STEP == 32 ? 4 : 2) void k_expert_tile(const ExpertArgs a) {
    typedef Shape<KIND, BM, BC, WM, WC, STEP> S;
    __shared__ __align__(16) uint16_t a0[BM * STEP], a1[BM * STEP], a2[BM * STEP], b0[BC * STEP], b1[BC * STEP];
    uint16_t *const sa[3] = {a0, a1, a2}, *const sb[2] = {b0, b1};
    if (status_at_entry(a.status)) return;
    // Workgroups go round the eight XCDs. Of the products that sum over K or
    // NW each XCD takes a run of its own, kGroup columns through an expert's
    // row tiles, so that what its compute units work on together shares row
    // and weight tiles in its L2. d_weight writes most of what it moves and
    // sums over few rows: there the XCDs write neighbouring tiles.
    const uint32_t cols = (uint32_t)a.cols;
    const uint32_t tiles = KIND == kDweight ? (uint32_t)(a.W * a.P) * a.row_tiles : (uint32_t)a.tiles[0];
    const uint32_t run = (tiles * cols + 7) / 8;
    const uint32_t at = KIND == kDweight ? blockIdx.x : (blockIdx.x & 7) * run + blockIdx.x / 8;
    if ((KIND != kDweight && blockIdx.x / 8 >= run) || at >= tiles * cols) return;
    int e;
    uint32_t n, i;  // the expert's row tiles, and this one of its n * cols tiles
    if constexpr (KIND == kDweight) {
        n = a.row_tiles;
        e = (int)(at / (n * cols));
        i = at - (uint32_t)e * n * cols;
    } else {
        e = a.tiles[2 + 2 * (at / cols)];
        const uint32_t f = (uint32_t)a.first[e];
        n = (uint32_t)a.first[e + 1] - f;
        i = at - f * cols;
    }
    int mt, ct;
    if constexpr (KIND == kDweight) {
        mt = (int)(i / cols);
        ct = (int)(i % cols);
    } else {
        const uint32_t group = i / (n * kGroup), wide = min(cols - group * kGroup, kGroup);
        i -= group * n * kGroup;
        mt = (int)(i / wide);
        ct = (int)(group * kGroup + i % wide);
    }
    const int d = e / a.P, j = e - d * a.P;
    const int64_t row0 = a.offsets[(int64_t)d * (a.P + 1) + j];
    const int64_t rows = a.offsets[(int64_t)d * (a.P + 1) + j + 1] - row0;
    const bool glu = KIND == kForward && a.act == A2AV_ACT_SWIGLU;
    const int64_t M = KIND == kDweight ? a.NW : rows;
    const int64_t C = KIND == kForward ? (glu ? (a.N + 15) / 16 * 32 : a.N) : a.K;
    const int64_t m0 = (int64_t)mt * BM, c0 = (int64_t)ct * BC;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WC, wc = wave % WC;
    typename S::A oa;
    typename S::B ob;
    const uint16_t *pa = (const uint16_t *)a.a[d], *pb = (const uint16_t *)a.b[d];
    if constexpr (KIND == kForward) {
        oa.along(pa + (row0 + m0) * a.K, nullptr, a.K, M - m0, wave, lane);
        const uint16_t *w = pb + (int64_t)j * a.NW * a.K;
        const int64_t n0 = glu ? c0 / 2 : c0;
        ob.along(w + n0 * a.K, glu ? w + (a.N + n0) * a.K : nullptr, a.K, a.N - n0, wave, lane);
    } else if constexpr (KIND == kDx) {
        oa.along(pa + (row0 + m0) * a.NW, nullptr, a.NW, M - m0, wave, lane);
        ob.across(pb + (int64_t)j * a.NW * a.K, a.K, a.NW, c0, C, wave, lane);
    } else {
        oa.across(pa + row0 * a.NW, a.NW, rows, m0, M, wave, lane);
        ob.across(pb + row0 * a.K, a.K, rows, c0, C, wave, lane);
    }
    f32x16 acc[S::kBlocksM][S::kBlocksC] = {};
    const int64_t left = M - m0;
    if (S::kBlocksM >= 4 && left <= WM * 32)
        contract<KIND, T, BM, BC, WM, WC, STEP, 1>(oa, ob, sa, sb, acc);
    else if (S::kBlocksM >= 2 && left <= WM * 32 * (S::kBlocksM / 2))
        contract<KIND, T, BM, BC, WM, WC, STEP, (S::kBlocksM >= 2 ? S::kBlocksM / 2 : 1)>(oa, ob, sa, sb, acc);
    else
        contract<KIND, T, BM, BC, WM, WC, STEP, S::kBlocksM>(oa, ob, sa, sb, acc);
    // The sums leave through LDS, so that one lane gets 8 neighbouring columns
    // of a row (16-byte stores, whole rows of the wave's columns at a time)
    // and the epilogue's code exists once: in passes of kPass row blocks, each
    // wave in its own part of the stages. A lane holds columns g * 8 + (lane /
    // 32) * 4 .. + 3, g = 0 .. 3, of row lane % 32 of each 32 x 32; the 16-byte
    // chunks of a row are permuted by the row, which keeps both sides off each
    // other's banks.
    constexpr int kPass = S::kBlocksM < 2 || STEP == 32 ? 1 : 2, kCols = S::kBlocksC * 32;
    __syncthreads();
    constexpr int kPart = kPass * 32 * kCols * 4;                               // bytes of a wave's part
    constexpr int kParts = STEP == 32 ? BM * STEP * 2 / kPart : WM * WC / 4;       // parts in one stage
    static_assert( (STEP == 64 || WM * WC <= 4 * kParts), "");
    const int in = wave / kParts;
    f32x4 *sums = (f32x4 *)(in == 0 ? a0 : in == 1 ? a1 : in == 2 ? a2 : b0) + wave % kParts * (kPart / 16);
    uint16_t *const out0 = (uint16_t *)a.out[d], *const pre0 = (uint16_t *)a.pre[d];
    const uint16_t *const bias0 = (const uint16_t *)a.bias[d], *const residual0 = (const uint16_t *)a.residual[d];
#pragma unroll
    for (int p = 0; p < S::kBlocksM / kPass; p++) {
        if (p * kPass * WM * 32 >= left) break;
#pragma unroll
        for (int u = 0; u < kPass; u++)
#pragma unroll
            for (int v = 0; v < S::kBlocksC; v++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    f32x4 y;
#pragma unroll
                    for (int i = 0; i < 4; i++) y[i] = acc[p * kPass + u][v][g * 4 + i];
                    sums[(u * 32 + (lane & 31)) * (kCols / 4) +
                         ((v * 8 + g * 2 + (lane >> 5)) ^ (lane & 15 & (kCols / 4 - 1)))] = y;
                }
        asm volatile("" ::: "memory");
        const int64_t c = c0 + wc * kCols;
        const auto row_of = [&](int r) { return m0 + ((p * kPass + (r >> 5)) * WM + wm) * 32 + (r & 31); };
        // eight columns of row r of the pass, from the row's chunk `at` on
        const auto take = [&](int r, int at, float(&y)[8]) {
            const f32x4 lo = sums[r * (kCols / 4) + (at ^ (r & 15 & (kCols / 4 - 1)))];
            const f32x4 hi = sums[r * (kCols / 4) + ((at + 1) ^ (r & 15 & (kCols / 4 - 1)))];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                y[i] = lo[i];
                y[i + 4] = hi[i];
            }
        };
        if constexpr (KIND == kForward) {
            const int per = glu ? kCols / 16 : kCols / 8;  // lanes a row
            for (int r = lane / per; r < kPass * 32; r += kWave / per) {
                const int64_t m = row_of(r);
                const int q = lane % per;
                if (m >= M) continue;
                // gated: blocks of 16 gate and 16 up columns alternate
                const int at = glu ? (q >> 1) * 8 + (q & 1) * 2 : q * 2;
                const int64_t n = (glu ? c / 2 : c) + q * 8, row = row0 + m;
                if (n >= a.N) continue;
                float y[8];
                take(r, at, y);
                const uint16_t *bias = bias0 + (int64_t)j * a.NW + n;
                uint16_t *pre = pre0 + row * a.NW + n;
                if (a.has_bias) add8<T>(y, bias);
                if (a.has_pre) put8<T>(pre, y);
                if (glu) {
                    float up[8];
                    take(r, at + 4, up);
                    if (a.has_bias) add8<T>(up, bias + a.N);
                    if (a.has_pre) put8<T>(pre + a.N, up);
#pragma unroll
                    for (int i = 0; i < 8; i++) y[i] = y[i] * sigmoid(y[i]) * up[i];
                } else if (a.act != A2AV_ACT_NONE) {
#pragma unroll
                    for (int i = 0; i < 8; i++) y[i] = act_of(a.act, y[i]);
                }
                if (a.has_residual) add8<T>(y, residual0 + row * a.N + n);
                put8<T>(out0 + row * a.N + n, y);
            }
        } else {
            // several rows' LDS reads in flight
            constexpr int kPer = kCols / 8, kRows = kWave / kPer, kTimes = kPass * 32 / kRows;
            constexpr int kBatch = kTimes < 4 ? kTimes : 4;
            const int q = lane % kPer;
            const bool in_c = c + q * 8 < C;
            uint16_t *const at = out0 + (KIND == kDx ? row0 : (int64_t)j * a.NW) * a.K + c + q * 8;
#pragma unroll
            for (int r0 = 0; r0 < kPass * 32; r0 += kBatch * kRows) {
                float y[kBatch][8];
#pragma unroll
                for (int i = 0; i < kBatch; i++) take(r0 + i * kRows + lane / kPer, q * 2, y[i]);
#pragma unroll
                for (int i = 0; i < kBatch; i++) {
                    const int64_t m = row_of(r0 + i * kRows + lane / kPer);
                    if (m < M && in_c) put8<T, KIND == kDweight>(at + m * a.K, y[i]);
                }
            }
        }
        asm volatile("" ::: "memory");
    }
}

// ------------------------------------------------------------------ few rows
// Experts with a few rows each (decoded tokens): what has to move is the
// weights, once, so they go from memory to the matrix cores' operands without
// LDS. A workgroup has 16 output columns (gated: the 16 gate and the 16 up
// rows behind them) of one tile of up to 16 rows; its four waves take blocks
// of 128 contraction elements in turn, every load of two blocks in flight, and
// their sums meet in LDS in wave order. Bound by the weights' bytes.
constexpr int kFewRows = 16, kFewStep = 128;

template <typename T>
__device__ __forceinline__ typename T::frag load_frag(rsrc_t b, uint32_t off) {
    return __builtin_bit_cast(typename T::frag, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}

template <typename T, bool GLU>
__global__ __launch_bounds__(256) void k_expert_few(const ExpertArgs a) {
    constexpr int kHalves = GLU ? 2 : 1;
    __shared__ f32x4 sums[4][kHalves][kWave];
    if (status_at_entry(a.status)) return;
    const uint32_t t = blockIdx.x / (uint32_t)a.cols, ct = blockIdx.x - t * a.cols;
    if ((int)t >= a.tiles[0]) return;
    const int e = a.tiles[2 + 2 * t], mt = a.tiles[3 + 2 * t];
    const int d = e / a.P, j = e - d * a.P;
    const int64_t *ends = a.offsets + (int64_t)d * (a.P + 1) + j;
    const int64_t row0 = ends[0] + (int64_t)mt * kFewRows, n0 = (int64_t)ct * 16;
    const int rows = (int)min(ends[1] - row0, (int64_t)kFewRows), cols = (int)min(a.N - n0, (int64_t)16);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t stride = (uint32_t)a.K * 2;
    const uint16_t *w = (const uint16_t *)a.b[d] + ((int64_t)j * a.NW + n0) * a.K;
    const rsrc_t bx = buffer((const uint16_t *)a.a[d] + row0 * a.K, (uint32_t)rows * stride);
    const rsrc_t bw = buffer(w, (uint32_t)cols * stride), bu = buffer(w + (GLU ? a.N * a.K : 0), (uint32_t)cols * stride);
    const int K = (int)a.K;
    const uint32_t line = (uint32_t)(lane & 15) * stride;
    f32x4 acc[kHalves] = {};
    constexpr int kFrags = kFewStep / 32, kDeep = 2;
    for (int k0 = wave * kFewStep; k0 < K; k0 += 4 * kFewStep * kDeep) {
        typename T::frag x[kDeep][kFrags], g[kDeep][kFrags], u[kDeep][kFrags];
#pragma unroll
        for (int s = 0; s < kDeep; s++)
#pragma unroll
            for (int i = 0; i < kFrags; i++) {
                const int k = k0 + s * 4 * kFewStep + i * 32 + (lane >> 4) * 8;
                const uint32_t at = k < K ? line + k * 2 : kOutside;
                g[s][i] = load_frag<T>(bw, at);
                if (GLU) u[s][i] = load_frag<T>(bu, at);
                x[s][i] = load_frag<T>(bx, at);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < kDeep; s++)
#pragma unroll
            for (int i = 0; i < kFrags; i++) {
                acc[0] = T::mfma(g[s][i], x[s][i], acc[0]);
                if (GLU) acc[kHalves - 1] = T::mfma(u[s][i], x[s][i], acc[kHalves - 1]);
            }
    }
#pragma unroll
    for (int h = 0; h < kHalves; h++) sums[wave][h][lane] = acc[h];
    __syncthreads();
    if (wave != 0) return;
    f32x4 y[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; h++) {
        y[h] = sums[0][h][lane];
#pragma unroll
        for (int i = 1; i < 4; i++) y[h] += sums[i][h][lane];
    }
    // a lane holds columns (lane / 16) * 4 .. + 3 of row lane % 16
    const int m = lane & 15, c = (lane >> 4) * 4;
    if (m >= rows || c >= cols) return;
    const int64_t row = row0 + m, n = n0 + c;
    typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
    u16x4 o;
#pragma unroll
    for (int h = 0; h < kHalves; h++) {
        if (a.has_bias) {
            const u16x4 b = *(const u16x4 *)((const uint16_t *)a.bias[d] + (int64_t)j * a.NW + h * a.N + n);
#pragma unroll
            for (int i = 0; i < 4; i++) y[h][i] += T::to_float(b[i]);
        }
        if (a.has_pre) {
#pragma unroll
            for (int i = 0; i < 4; i++) o[i] = T::from_float(y[h][i]);
            *(u16x4 *)((uint16_t *)a.pre[d] + row * a.NW + h * a.N + n) = o;
        }
    }
    u16x4 r = {};
    if (a.has_residual) r = *(const u16x4 *)((const uint16_t *)a.residual[d] + row * a.N + n);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float v = GLU ? y[0][i] * sigmoid(y[0][i]) * y[kHalves - 1][i] : act_of(a.act, y[0][i]);
        if (a.has_residual) v += T::to_float(r[i]);
        o[i] = T::from_float(v);
    }
    *(u16x4 *)((uint16_t *)a.out[d] + row * a.N + n) = o;
}

// ------------------------------------------------------------------ d_pre and the bias
constexpr int kBlockRows = 64;  // rows of a block of the bias sums
constexpr int kVecCols = 64;    // columns of a workgroup of the 16-byte form

struct DpreArgs {
    const void *pre[A2AV_MAX_W];
    const void *d_out[A2AV_MAX_W];
    void *d_pre[A2AV_MAX_W];
    void *d_bias[A2AV_MAX_W];
    const int64_t *offsets;
    const int32_t *tiles;
    const int32_t *first;
    float *part;  // [tile][blocks][NW] bias sums of the row blocks
    const int32_t *status;
    int64_t N, NW;
    int W, P;
    int act;
    int has_bias;
    int blocks;   // row blocks a tile
};

// d_pre of one element (and, gated, of its up half) from fp32 values.
__device__ __forceinline__ void dpre_of(int act, float g, float h, float up, float &dh, float &du) {
    if (act == A2AV_ACT_SWIGLU) {
        const float s = sigmoid(h);
        dh = g * up * (s * (1.0f + h * (1.0f - s)));
        du = g * h * s;
    } else {
        dh = g * act_slope(act, h);
    }
}

// One workgroup per row block and 64 output columns (VEC) or 256. VEC: a
// thread has 8 neighbouring columns of two rows (16-byte loads and stores, all
// of them in flight together), and the rows' sums meet in LDS in a fixed
// order; otherwise a thread walks one column down the block's rows. Bound by
// the bytes, which it reads and writes once.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_expert_dpre(const DpreArgs a) {
    if (status_at_entry(a.status)) return;
    const int64_t b = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
    const int t = (int)(b / a.blocks);
    if (t >= a.tiles[0]) return;
    const int e = a.tiles[2 + 2 * t], mt = a.tiles[3 + 2 * t];
    const int d = e / a.P, j = e - d * a.P;
    const int64_t *off = a.offsets + (int64_t)d * (a.P + 1) + j;
    const int64_t r0 = off[0] + ((int64_t)mt * a.blocks + b % a.blocks) * kBlockRows;
    const int64_t r1 = r0 + kBlockRows < off[1] ? r0 + kBlockRows : off[1];
    if (r0 >= r1) return;  // the same in the whole workgroup
    const int act = a.act;
    const bool glu = act == A2AV_ACT_SWIGLU, none = act == A2AV_ACT_NONE;
    const uint16_t *d_out = (const uint16_t *)a.d_out[d], *pre = (const uint16_t *)a.pre[d];
    uint16_t *d_pre = (uint16_t *)a.d_pre[d];
    if constexpr (VEC) {
        constexpr int kLanes = kVecCols / 8, kGroups = 256 / kLanes, kRows = kBlockRows / kGroups;
        __shared__ float part[2][kGroups][kVecCols];
        const int col = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
        const int64_t n = (int64_t)blockIdx.x * kVecCols + col * 8, r = r0 + group;
        float s0[8] = {}, s1[8] = {};
        if (n < a.N && r < r1) {
            u16x8 g[kRows], h[kRows], up[kRows];
#pragma unroll
            for (int i = 0; i < kRows; i++) {
                const int64_t row = r + i * kGroups < r1 ? r + i * kGroups : r;  // past the block: row r again, not used
                g[i] = *(const u16x8 *)(d_out + row * a.N + n);
                if (!none) h[i] = *(const u16x8 *)(pre + row * a.NW + n);
                if (glu) up[i] = *(const u16x8 *)(pre + row * a.NW + a.N + n);
            }
#pragma unroll
            for (int i = 0; i < kRows; i++) {
                const int64_t row = r + i * kGroups;
                if (row >= r1) break;
                float dh[8], du[8];
#pragma unroll
                for (int c = 0; c < 8; c++) {
                    dh[c] = T::to_float(g[i][c]);
                    du[c] = 0.0f;
                    if (!none)
                        dpre_of(act, dh[c], T::to_float(h[i][c]), glu ? T::to_float(up[i][c]) : 0.0f, dh[c], du[c]);
                    s0[c] += dh[c];
                    s1[c] += du[c];
                }
                if (!none) put8<T>(d_pre + row * a.NW + n, dh);
                if (glu) put8<T>(d_pre + row * a.NW + a.N + n, du);
            }
        }
        if (!a.has_bias) return;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            part[0][group][col * 8 + c] = s0[c];
            part[1][group][col * 8 + c] = s1[c];
        }
        __syncthreads();
        const int64_t m = (int64_t)blockIdx.x * kVecCols + threadIdx.x;
        if (threadIdx.x >= kVecCols || m >= a.N) return;
        float x = 0.0f, y = 0.0f;
#pragma unroll 8
        for (int i = 0; i < kGroups; i++) {
            x += part[0][i][threadIdx.x];
            y += part[1][i][threadIdx.x];
        }
        a.part[b * a.NW + m] = x;
        if (glu) a.part[b * a.NW + a.N + m] = y;
    } else {
        const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (n >= a.N) return;
        float s0 = 0.0f, s1 = 0.0f;
        for (int64_t r = r0; r < r1; r++) {
            float dh = T::to_float(d_out[r * a.N + n]), du = 0.0f;
            if (!none) {
                dpre_of(act, dh, T::to_float(pre[r * a.NW + n]), glu ? T::to_float(pre[r * a.NW + a.N + n]) : 0.0f, dh,
                        du);
                d_pre[r * a.NW + n] = T::from_float(dh);
                if (glu) d_pre[r * a.NW + a.N + n] = T::from_float(du);
            }
            s0 += dh;
            s1 += du;
        }
        if (a.has_bias) {
            a.part[b * a.NW + n] = s0;
            if (glu) a.part[b * a.NW + a.N + n] = s1;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_expert_dbias(const DpreArgs a) {
    if (status_at_entry(a.status)) return;
    const int e = blockIdx.y, d = e / a.P, j = e - d * a.P;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= a.NW) return;
    const int64_t *off = a.offsets + (int64_t)d * (a.P + 1) + j;
    const int64_t blocks = (off[1] - off[0] + kBlockRows - 1) / kBlockRows, b0 = (int64_t)a.first[e] * a.blocks;
    float s = 0.0f;
    for (int64_t b = 0; b < blocks; b++) s += a.part[(b0 + b) * a.NW + n];
    ((uint16_t *)a.d_bias[d])[(int64_t)j * a.NW + n] = T::from_float(s);
}

// ------------------------------------------------------------------ host
static size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// Row tiles of tile_rows that W * P experts with these rows can have, at most;
// -1 for sizes that are not valid.
static int64_t tile_bound(int W, int P, int64_t K, int64_t N, int act, const int64_t *x_rows, int tile_rows) {
    if (W < 1 || W > A2AV_MAX_W || P < 1 || (int64_t)W * P > A2AV_MAX_EXPERTS || K < 1 || N < 1 || !x_rows)
        return -1;
    if (act < A2AV_ACT_NONE || act > A2AV_ACT_SWIGLU) return -1;
    if (K > A2AV_MAX_WIDTH || N > A2AV_MAX_WIDTH) return -1;
    int64_t total = 0;
    for (int d = 0; d < W; d++) {
        if (x_rows[d] < 0 || x_rows[d] > ((int64_t)1 << 30)) return -1;
        total += x_rows[d];
    }
    const int64_t t = total / tile_rows + (int64_t)W * P;
    return t <= (1 << 30) ? t : -1;
}

// Tile shapes of the fast products, largest first.
constexpr int64_t kMostGroups = 1 << 22;  // workgroups of a launch, times 512 threads inside 32 bits
enum { kBig, kMid, kSmall, kFew };
constexpr int kTile[] = {256, 128, 64, kFewRows};
constexpr int kMostBlocks = 4;  // row blocks of the largest tile
static_assert(kTile[kBig] == kMostBlocks * kBlockRows && kTile[kSmall] == kBlockRows && kAny == kBlockRows, "");

struct Layout {
    int64_t tiles;      // most tiles, of the smallest size
    size_t first, part; // byte offsets
    size_t total;
};

// The workspace holds the list of the smallest tiles, so that it does not
// depend on the shape that a call takes.
static bool plan_layout(int W, int P, int64_t K, int64_t N, int act, const int64_t *x_rows, bool with_part,
                        Layout *l) {
    l->tiles = tile_bound(W, P, K, N, act, x_rows, kBlockRows);
    const int64_t few = tile_bound(W, P, K, N, act, x_rows, kFewRows);
    if (few < 0) return false;
    l->first = round256((size_t)(few + 1) * 8);
    l->part = l->first + round256(((size_t)W * P + 1) * 4);
    const int64_t NW = act == A2AV_ACT_SWIGLU ? 2 * N : N;
    const size_t blocks = (size_t)l->tiles + (size_t)(kMostBlocks - 1) * W * P;
    l->total = l->part + (with_part ? round256(blocks * (size_t)NW * 4) : 0) + 256;
    return true;
}

// The largest tile of which the product has enough to fill the compute units;
// R rows over n experts, M x C the product of one of them (M = 0: its rows).
static int shape_of(int64_t R, int64_t n, int64_t M, int64_t C) {
    for (int s = kBig; s < kSmall; s++) {
        const int64_t t = kTile[s], cols = (C + t - 1) / t;
        const int64_t tiles = M ? n * ((M + t - 1) / t) : R <= n ? R : R / t + (R % (n * t) ? n / 2 : 0);
        if (tiles * cols >= 200) return s;
    }
    return kSmall;
}

static void launch_plan(int W, int P, const int64_t *x_rows, const int64_t *offsets, int tile_rows,
                        unsigned char *ws, const Layout &l, int32_t *status, hipStream_t stream) {
    PlanArgs p;
    std::memset(&p, 0, sizeof(p));
    for (int d = 0; d < W; d++) p.x_rows[d] = x_rows[d];
    p.offsets = offsets;
    p.tiles = (int32_t *)ws;
    p.first = (int32_t *)(ws + l.first);
    p.status = status;
    p.W = W;
    p.P = P;
    p.tile_rows = tile_rows;
    hipLaunchKernelGGL(k_expert_plan, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

// Tiles over the y and z dimensions of a grid.
static dim3 tile_grid(int64_t columns, int64_t tiles) {
    const int64_t y = tiles < 32768 ? tiles : 32768;
    return dim3((unsigned)columns, (unsigned)y, (unsigned)((tiles + y - 1) / y));
}

// Columns of a product, and column tiles of a shape.
template <int KIND>
static int64_t columns_of(const ExpertArgs &a) {
    return KIND != kForward ? a.K : a.act == A2AV_ACT_SWIGLU ? (a.N + 15) / 16 * 32 : a.N;
}
template <int KIND>
static int64_t column_tiles(const ExpertArgs &a, int shape) {
    if (shape == kFew) return (a.N + 15) / 16;
    return (columns_of<KIND>(a) + kTile[shape] - 1) / kTile[shape];
}

// The shape's workgroups fit one launch of the tile kernels (k_expert_any has a
// grid of three dimensions and takes any number).
template <int KIND>
static bool launches(const ExpertArgs &a, int shape, int64_t tiles) {
    if (KIND == kDweight) tiles = (int64_t)a.W * a.P * ((a.NW + kTile[shape] - 1) / kTile[shape]);
    return tiles * column_tiles<KIND>(a, shape) <= kMostGroups;
}

template <int KIND, typename T>
static void launch_product(ExpertArgs &a, int shape, bool fast, int64_t tiles, hipStream_t stream) {
    const int64_t t = fast ? kTile[shape] : kAny;
    a.cols = (int)(fast ? column_tiles<KIND>(a, shape) : (columns_of<KIND>(a) + kAny - 1) / kAny);
    a.row_tiles = (int)((a.NW + t - 1) / t);
    if (!fast) {
        const dim3 g = KIND == kDweight ? dim3(a.cols, a.row_tiles, a.W * a.P) : tile_grid(a.cols, tiles);
        hipLaunchKernelGGL((k_expert_any<KIND, T>), g, dim3(256), 0, stream, a);
        return;
    }
    if constexpr (KIND == kForward) {
        if (shape == kFew) {
            const dim3 g((unsigned)(tiles * a.cols));
            if (a.act == A2AV_ACT_SWIGLU) hipLaunchKernelGGL((k_expert_few<T, true>), g, dim3(256), 0, stream, a);
            else hipLaunchKernelGGL((k_expert_few<T, false>), g, dim3(256), 0, stream, a);
            return;
        }
    }
    if (KIND == kDweight) tiles = (int64_t)a.W * a.P * a.row_tiles;
    const dim3 g((unsigned)((tiles * a.cols + 7) / 8 * 8));
    if (shape == kBig) hipLaunchKernelGGL((k_expert_tile<KIND, T, 256, 256, 2, 4, 64>), g, dim3(512), 0, stream, a);
    else if (shape == kMid)
        hipLaunchKernelGGL((k_expert_tile<KIND, T, 128, 128, 2, 2, KIND == kDweight ? 32 : 64>), g, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_expert_tile<KIND, T, 64, 64, 2, 2, 64>), g, dim3(256), 0, stream, a);
}

template <int KIND>
static void launch_product(ExpertArgs &a, int type, int shape, bool fast, int64_t tiles, hipStream_t stream) {
    if (type == A2AV_DT_BF16) launch_product<KIND, Bf16>(a, shape, fast, tiles, stream);
    else launch_product<KIND, Fp16>(a, shape, fast, tiles, stream);
}

// Most tiles of `rows` rows that a product's row tiles can be.
static int64_t most_tiles(const int64_t *x_rows, int W, int P, int rows) {
    int64_t total = 0;
    for (int d = 0; d < W; d++) total += x_rows[d];
    return total / rows + (int64_t)W * P;
}

static bool aligned16(const void *p) { return (uintptr_t)p % 16 == 0; }

static bool fits(int64_t rows, int64_t width) {
    return (uint64_t)rows <= (uint64_t)INT64_MAX / 4 / (uint64_t)width;
}

}  // namespace a2av

using namespace a2av;

A2AV_API size_t moe_expert_linear_workspace_bytes(int W, int P, int64_t K, int64_t N, int act,
                                                  const int64_t *x_rows) {
    Layout l;
    return plan_layout(W, P, K, N, act, x_rows, false, &l) ? l.total : 0;
}

A2AV_API int moe_expert_linear(int W, int P, int64_t K, int64_t N, int type, int act,
                               const void *const *x, const int64_t *x_rows,
                               const int64_t *expert_offsets, const void *const *weight,
                               const void *const *bias, const void *const *residual,
                               void *const *out, void *const *pre, void *workspace,
                               size_t workspace_bytes, int32_t *status, hipStream_t stream) {
    Layout l;
    if (!plan_layout(W, P, K, N, act, x_rows, false, &l)) return A2AV_EARG;
    if ((type != A2AV_DT_BF16 && type != A2AV_DT_F16) || !x || !expert_offsets || !weight || !out || !status)
        return A2AV_EARG;
    if (!workspace || (uintptr_t)workspace % 8 != 0 || workspace_bytes < l.total) return A2AV_EARG;
    ExpertArgs a;
    std::memset(&a, 0, sizeof(a));
    a.K = K;
    a.N = N;
    a.NW = act == A2AV_ACT_SWIGLU ? 2 * N : N;
    int64_t R = 0;
    bool fast = K % 8 == 0 && N % 8 == 0;
    for (int d = 0; d < W; d++) {
        R += x_rows[d];
        if (!fits(x_rows[d], K) || !fits(x_rows[d], a.NW)) return A2AV_EARG;
        if (!weight[d] || (bias && !bias[d])) return A2AV_EARG;
        if (x_rows[d] > 0 && (!x[d] || !out[d] || (residual && !residual[d]) || (pre && !pre[d])))
            return A2AV_EARG;
        // other tiles still read x; pre is written before the residual is read
        if (x_rows[d] > 0 && (out[d] == x[d] || (pre && (pre[d] == x[d] || pre[d] == out[d]))))
            return A2AV_EARG;
        if (x_rows[d] > 0 && pre && residual && pre[d] == residual[d]) return A2AV_EARG;
        a.a[d] = x[d];
        a.b[d] = weight[d];
        a.bias[d] = bias ? bias[d] : nullptr;
        a.residual[d] = residual ? residual[d] : nullptr;
        a.out[d] = out[d];
        a.pre[d] = pre ? pre[d] : nullptr;
        fast = fast && aligned16(a.a[d]) && aligned16(a.b[d]) && aligned16(a.bias[d]) && aligned16(a.residual[d]) &&
               aligned16(a.out[d]) && aligned16(a.pre[d]);
    }
    a.offsets = expert_offsets;
    a.tiles = (const int32_t *)workspace;
    a.first = (const int32_t *)((unsigned char *)workspace + l.first);
    a.status = status;
    a.W = W;
    a.P = P;
    a.act = act;
    a.has_bias = bias != nullptr;
    a.has_residual = residual != nullptr;
    a.has_pre = pre != nullptr;
    const int64_t n = (int64_t)W * P;
    // Few rows an expert and long weight rows: without LDS. (SwiGLU of 8 rows
    // on 8 of 32 experts, K 7168, N 2048, bf16: 72 against 107 us; no gate,
    // 8 experts: 44 against 58 us at K 7168, 55.5 against 55 at K 4096, 58
    // against 44 at K 2048; 12 rows an expert at K 7168: 210 against 172 us.)
    // The rows are those that x_rows allows. All of them on one expert: its
    // weights are read once for every 16 rows, from the L2 then (128 rows of 32
    // experts, NW 4096: 82 us against 119 of one row more by tiles; 1024 of 256,
    // NW 1024: 155 against 121).
    int shape = R <= 4 * n && K >= 4096 ? kFew : shape_of(R, n, 0, a.NW);
    const auto tiles = [&] { return most_tiles(x_rows, W, P, kTile[shape]); };
    if (shape == kFew && !launches<kForward>(a, shape, tiles())) shape = shape_of(R, n, 0, a.NW);
    fast = fast && launches<kForward>(a, shape, tiles());
    if (!fast) shape = kSmall;
    launch_plan(W, P, x_rows, expert_offsets, kTile[shape], (unsigned char *)workspace, l, status, stream);
    launch_product<kForward>(a, type, shape, fast, tiles(), stream);
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}

A2AV_API size_t moe_expert_linear_backward_workspace_bytes(int W, int P, int64_t K, int64_t N,
                                                           int act, const int64_t *x_rows) {
    Layout l;
    return plan_layout(W, P, K, N, act, x_rows, true, &l) ? l.total : 0;
}

A2AV_API int moe_expert_linear_backward(int W, int P, int64_t K, int64_t N, int type, int act,
                                        const void *const *x, const int64_t *x_rows,
                                        const int64_t *expert_offsets, const void *const *weight,
                                        const void *const *pre, const void *const *d_out,
                                        void *const *d_pre, void *const *d_x, void *const *d_weight,
                                        void *const *d_bias, void *workspace,
                                        size_t workspace_bytes, int32_t *status,
                                        hipStream_t stream) {
    Layout l;
    if (!plan_layout(W, P, K, N, act, x_rows, true, &l)) return A2AV_EARG;
    const bool none = act == A2AV_ACT_NONE;
    if ((type != A2AV_DT_BF16 && type != A2AV_DT_F16) || !x || !expert_offsets || !weight || !d_out || !status)
        return A2AV_EARG;
    if (none ? (pre || d_pre) : (!pre || !d_pre)) return A2AV_EARG;
    if (!workspace || (uintptr_t)workspace % 8 != 0 || workspace_bytes < l.total) return A2AV_EARG;
    unsigned char *ws = (unsigned char *)workspace;
    ExpertArgs a, b;
    DpreArgs g;
    std::memset(&a, 0, sizeof(a));
    std::memset(&b, 0, sizeof(b));
    std::memset(&g, 0, sizeof(g));
    a.K = K;
    a.N = g.N = N;
    a.NW = g.NW = act == A2AV_ACT_SWIGLU ? 2 * N : N;
    a.offsets = g.offsets = expert_offsets;
    a.tiles = g.tiles = (const int32_t *)ws;
    a.first = g.first = (const int32_t *)(ws + l.first);
    a.status = g.status = status;
    a.W = g.W = W;
    a.P = g.P = P;
    a.act = g.act = act;
    b = a;
    g.part = (float *)(ws + l.part);
    g.has_bias = d_bias != nullptr;
    int64_t R = 0;
    bool fast = K % 8 == 0 && N % 8 == 0, vec = N % 8 == 0;
    for (int d = 0; d < W; d++) {
        R += x_rows[d];
        if (!fits(x_rows[d], K) || !fits(x_rows[d], a.NW)) return A2AV_EARG;
        if (!weight[d] || (d_weight && !d_weight[d]) || (d_bias && !d_bias[d])) return A2AV_EARG;
        if (x_rows[d] > 0 && (!x[d] || !d_out[d] || (!none && (!pre[d] || !d_pre[d])) || (d_x && !d_x[d])))
            return A2AV_EARG;
        // other tiles still read d_pre, and d_weight x
        if (x_rows[d] > 0 && d_x && (d_x[d] == x[d] || d_x[d] == (none ? d_out[d] : d_pre[d]))) return A2AV_EARG;
        if (x_rows[d] > 0 && !none && d_pre[d] == x[d]) return A2AV_EARG;
        // d_pre's rows are wider than those of d_out that are still to be read
        if (x_rows[d] > 0 && act == A2AV_ACT_SWIGLU && d_pre[d] == d_out[d]) return A2AV_EARG;
        g.pre[d] = none ? nullptr : pre[d];
        g.d_out[d] = d_out[d];
        g.d_pre[d] = none ? nullptr : d_pre[d];
        g.d_bias[d] = d_bias ? d_bias[d] : nullptr;
        a.a[d] = b.a[d] = none ? d_out[d] : d_pre[d];
        a.b[d] = weight[d];
        a.out[d] = d_x ? d_x[d] : nullptr;
        b.b[d] = x[d];
        b.out[d] = d_weight ? d_weight[d] : nullptr;
        vec = vec && aligned16(g.pre[d]) && aligned16(d_out[d]) && aligned16(g.d_pre[d]);
        fast = fast && aligned16(a.a[d]) && aligned16(a.b[d]) && aligned16(a.out[d]) && aligned16(b.b[d]) &&
               aligned16(b.out[d]);
    }
    const int64_t n = (int64_t)W * P;
    int shape = shape_of(R, n, 0, K);
    const bool fast_x = fast && launches<kDx>(a, shape, most_tiles(x_rows, W, P, kTile[shape]));
    if (!fast_x) shape = kSmall;
    const int64_t tiles = most_tiles(x_rows, W, P, kTile[shape]);
    g.blocks = kTile[shape] / kBlockRows;
    launch_plan(W, P, x_rows, expert_offsets, kTile[shape], ws, l, status, stream);
    if (!none || d_bias) {
        const dim3 grid = tile_grid(vec ? (N + kVecCols - 1) / kVecCols : (N + 255) / 256, tiles * g.blocks);
        if (type == A2AV_DT_BF16 && vec) hipLaunchKernelGGL((k_expert_dpre<Bf16, true>), grid, dim3(256), 0, stream, g);
        else if (type == A2AV_DT_BF16) hipLaunchKernelGGL((k_expert_dpre<Bf16, false>), grid, dim3(256), 0, stream, g);
        else if (vec) hipLaunchKernelGGL((k_expert_dpre<Fp16, true>), grid, dim3(256), 0, stream, g);
        else hipLaunchKernelGGL((k_expert_dpre<Fp16, false>), grid, dim3(256), 0, stream, g);
    }
    if (d_bias) {
        const dim3 grid((unsigned)((a.NW + 255) / 256), W * P);
        if (type == A2AV_DT_BF16) hipLaunchKernelGGL(k_expert_dbias<Bf16>, grid, dim3(256), 0, stream, g);
        else hipLaunchKernelGGL(k_expert_dbias<Fp16>, grid, dim3(256), 0, stream, g);
    }
    if (d_x) launch_product<kDx>(a, type, shape, fast_x, tiles, stream);
    if (d_weight) {
        // Few rows an expert: the tile's sums are short and its stores long, and
        // four workgroups of the middle size on a compute unit cover the one
        // with the other. (K 7168, bf16: 186 against 222 us at 64 rows an expert
        // and NW 2048; with NW 4096 758 against 769 at 256, 1173 against 1115 at
        // 512, 985 against 921 at 1024. Tiles of 256 x 128, with three quarters
        // of the L2's reads, take as long as the middle size.)
        int s = shape_of(R, n, a.NW, K);
        if (s == kBig && R < 384 * n && launches<kDweight>(b, kMid, 0)) s = kMid;
        launch_product<kDweight>(b, type, s, fast && launches<kDweight>(b, s, 0), 0, stream);
    }
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
