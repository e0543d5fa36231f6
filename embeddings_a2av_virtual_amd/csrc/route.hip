// route.hip — the router in front of the MoE pack, and its gradient (gfx950).
//
//   k_moe_route           expert ids and gate weights, 16 or 64 lanes a token
//   k_moe_route_exact     the same by one wave a token, for any size
//   k_route_check         range check of the ids the gradient scatters to
//   k_moe_route_backward  the gradient of the weights in the logits, 16 or 64
//                         lanes a token
//   k_moe_route_backward_any  the same by one wave a token, for any size
#include <hip/hip_runtime.h>

#include <cstring>

#include "common.hpp"

namespace a2av {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxGroups = 64;

struct RouteArgs {
    const void *z[A2AV_MAX_W];
    int32_t *ids[A2AV_MAX_W];
    float *w[A2AV_MAX_W];
    const float *bias;
    const int32_t *status;
    int64_t T;
    int W, k, E;
    int groups, topk_groups, group_top;
    int sigmoid, renorm;
    float scale;
};

// Element i of a logits row as fp32 (exact for every type).
template <int TYPE>
__device__ __forceinline__ float logit_at(const void *row, int64_t i) {
    if constexpr (TYPE == A2AV_DT_F32) return ((const float *)row)[i];
    if constexpr (TYPE == A2AV_DT_BF16) return bf16_lo(((const uint16_t *)row)[i]);
    return (float)((const _Float16 *)row)[i];
}

template <int TYPE>
__device__ __forceinline__ const void *logit_row(const void *base, int64_t row, int E) {
    return (const unsigned char *)base + (uint64_t)row * E * (TYPE == A2AV_DT_F32 ? 4 : 2);
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmax(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// One token's ids by one wave, every comparison in double as the result is
// defined: scores and keys of all experts into LDS, the groups' scores by one
// lane each, then k rounds of a wave-wide argmax. Lane j returns id j; *bad
// tells a token that has NaN weights.
template <int TYPE>
__device__ __forceinline__ int route_exact(const RouteArgs &a, const void *row, double *key, int lane, bool *bad) {
    const double inf = __builtin_huge_val(), nan = __builtin_nan("");
    const int E = a.E;
    double m = -inf;
    int off = 0;
#pragma unroll 1
    for (int e = lane; e < E; e += kWave) {
        const double z = logit_at<TYPE>(row, e);
        off |= z != z || (!a.sigmoid && z == inf);
        m = fmax(m, z);
    }
    *bad = __ballot(off) != 0;
    if (*bad) return lane;
    double sum = 0;
    if (!a.sigmoid) {
        m = wave_max(m);
#pragma unroll 1
        for (int e = lane; e < E; e += kWave) {
            const double z = logit_at<TYPE>(row, e);
            if (z != -inf) sum += exp(z - m);
        }
        sum = wave_sum(sum);
    }
#pragma unroll 1
    for (int e = lane; e < E; e += kWave) {
        const double z = logit_at<TYPE>(row, e);
        double c = a.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - m) / sum;
        if (a.bias) c += a.bias[e];
        if (z == -inf || c != c) c = -inf;
        key[e] = c;
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (a.groups > 1) {
        const int per = E / a.groups;
        double gs = -inf;
        if (lane < a.groups) {
            double t1 = -inf, t2 = -inf;
#pragma unroll 1
            for (int i = 0; i < per; i++) {
                const double c = key[lane * per + i];
                if (c > t1) {
                    t2 = t1;
                    t1 = c;
                } else if (c > t2) {
                    t2 = c;
                }
            }
            gs = a.group_top == 1 ? t1 : t1 + t2;
            if (gs != gs) gs = -inf;
        }
        int before = 0;
#pragma unroll 1
        for (int g = 0; g < a.groups; g++) {
            const double o = __shfl(gs, g);
            before += o > gs || (o == gs && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.groups && before < a.topk_groups);
#pragma unroll 1
        for (int e = lane; e < E; e += kWave)
            if (!((kept >> (e / per)) & 1)) key[e] = nan;
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    int id = 0;
#pragma unroll 1
    for (int j = 0; j < a.k; j++) {
        double c = -inf;
        float z = -__builtin_huge_valf();
        int best = E;  // no expert: behind every real one
#pragma unroll 1
        for (int e = lane; e < E; e += kWave) {
            const double o = key[e];
            if (o != o) continue;  // taken, or of a dropped group
            const float oz = logit_at<TYPE>(row, e);
            if (best == E || o > c || (o == c && oz > z)) {
                c = o;
                z = oz;
                best = e;
            }
        }
#pragma unroll 1
        for (int o = 32; o; o >>= 1) {
            const double oc = __shfl_xor(c, o);
            const float oz = __shfl_xor(z, o);
            const int oe = __shfl_xor(best, o);
            const bool take = oe != E && (best == E || oc > c || (oc == c && (oz > z || (oz == z && oe < best))));
            c = take ? oc : c;
            z = take ? oz : z;
            best = take ? oe : best;
        }
        if (lane == j) id = best;
        if (lane == 0) key[best] = nan;
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    return id;
}

// Reductions over the L lanes of a token (16: a DPP row), in an order that is
// the same for all of them.
template <int L, typename F>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t x, F op) {
    x = op(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xf, 0xf, true));  // row_ror:8
    x = op(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 0xf, 0xf, true));
    x = op(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 0xf, 0xf, true));
    x = op(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 0xf, 0xf, true));
    if constexpr (L == 64) {
        x = op(x, (uint32_t)__shfl_xor((int)x, 16));
        x = op(x, (uint32_t)__shfl_xor((int)x, 32));
    }
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v) {
    return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// A token's logits over its L lanes: lane sub has 4 neighbours of every 4 * L,
// -inf past the last.
template <int TYPE, int L, int V>
__device__ __forceinline__ void load_logits(const void *row, int E, int sub, bool vec, float (&z)[V]) {
    const float inf = __builtin_huge_valf();
    if (vec) {
#pragma unroll
        for (int c = 0; c < V / 4; c++) {
            const int e = (c * L + sub) * 4;
            if constexpr (TYPE == A2AV_DT_F32) {
                f32x4 v = {-inf, -inf, -inf, -inf};
                if (e < E) v = *(const f32x4 *)((const float *)row + e);
#pragma unroll
                for (int q = 0; q < 4; q++) z[c * 4 + q] = v[q];
            } else {
                u32x2 v = {0, 0};
                if (e < E) v = *(const u32x2 *)((const uint16_t *)row + e);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint16_t h = (uint16_t)(v[q / 2] >> (q % 2 * 16));
                    z[c * 4 + q] = e < E ? logit_at<TYPE>(&h, 0) : -inf;
                }
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int e = ((v / 4) * L + sub) * 4 + v % 4;
            z[v] = e < E ? logit_at<TYPE>(row, e) : -inf;
        }
    }
}

// The weights of the ids that lanes 0 .. k - 1 of a token (and those after
// them, L apart) hold in sel: fp32, from the chosen logits relative to the
// largest of them, so that scores outside fp32's range still have ratios; what
// is 0 in double (e^-709 and less) is 0 here. m: the largest of all logits,
// for softmax; sum: the softmax's, without renorm.
template <int TYPE, int L>
__device__ __forceinline__ void route_weights(const RouteArgs &a, const void *row, const int *sel, int sub, bool bad,
                                              float m, float sum, int32_t *ids, float *w, bool store) {
    const float inf = __builtin_huge_valf();
    // k <= L in earnest: a lane's first logit stays in a register
    const int id0 = sub < a.k ? sel[sub] : 0;
    const float z0 = logit_at<TYPE>(row, id0);
    float top = sub < a.k ? z0 : -inf;
    for (int j = sub + L; j < a.k; j += L) top = fmaxf(top, logit_at<TYPE>(row, sel[j]));
    top = lanes_max<L>(top);
    const float least = a.sigmoid ? -709.0f : m - 745.0f;
    const bool nothing = !(top >= least) || top == -inf;
    const float ref = a.sigmoid ? fminf(top, 0.0f) : a.renorm ? top : m;
    const auto score = [&](float z) {
        if (z == -inf || z < least) return 0.0f;
        if (!a.sigmoid) return expf(z - ref);
        if (z >= 0.0f) return 1.0f / (1.0f + expf(-z));
        return expf(a.renorm ? z - ref : z) / (1.0f + expf(z));
    };
    const float s0 = score(z0);
    float S = a.sigmoid ? 1.0f : sum;
    if (a.renorm) {
        S = sub < a.k ? s0 : 0.0f;
        for (int j = sub + L; j < a.k; j += L) S += score(logit_at<TYPE>(row, sel[j]));
        S = lanes_sum<L>(S);
    }
    const auto put = [&](int j, int id, float s) {
        float v = nothing ? 0.0f : s / S * a.scale;
        if (bad) v = __builtin_nanf("");
        if (store) {
            ids[j] = id;
            w[j] = v;
        }
    };
    if (sub < a.k) put(sub, id0, s0);
    for (int j = sub + L; j < a.k; j += L) put(j, sel[j], score(logit_at<TYPE>(row, sel[j])));
}

// m and sum of a whole row by one wave, as route_weights wants them.
template <int TYPE>
__device__ __forceinline__ void row_sum(const RouteArgs &a, const void *row, int lane, float *m, float *sum) {
    *m = *sum = 0.0f;
    if (a.sigmoid) return;
    float x = -__builtin_huge_valf(), s = 0.0f;
    for (int e = lane; e < a.E; e += kWave) x = fmaxf(x, logit_at<TYPE>(row, e));
    x = lanes_max<kWave>(x);
    *m = x;
    if (a.renorm) return;
    for (int e = lane; e < a.E; e += kWave) {
        const float z = logit_at<TYPE>(row, e);
        s += z == -__builtin_huge_valf() ? 0.0f : expf(z - x);
    }
    *sum = lanes_sum<kWave>(s);
}

// One wave per token: any size. Bound by the rounds, each of which walks all the
// keys: 8 x 1024 tokens, top 8, 325 us of 2048 experts and 1.18 ms of 4096.
template <int TYPE>
__global__ __launch_bounds__(256) void k_moe_route_exact(const RouteArgs a) {
    extern __shared__ double keys[];
    __shared__ int sel[4][kWave];
    if (status_at_entry(a.status)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int waves = blockDim.x / kWave;
    double *key = keys + (size_t)wave * a.E;
    const int64_t n = (int64_t)a.W * a.T;
    for (int64_t i = (int64_t)blockIdx.x * waves + wave; i < n; i += (int64_t)gridDim.x * waves) {
        const int r = (int)(i / a.T);
        const int64_t t = i - (int64_t)r * a.T;
        const void *row = logit_row<TYPE>(a.z[r], t, a.E);
        bool bad;
        float m, sum;
        sel[wave][lane] = route_exact<TYPE>(a, row, key, lane, &bad);
        row_sum<TYPE>(a, row, lane, &m, &sum);
        route_weights<TYPE, kWave>(a, row, sel[wave], lane, bad, m, sum, a.ids[r] + t * a.k, a.w[r] + t * a.k, true);
    }
}

constexpr int kCands = 80;  // candidates of a token that are put in order at most

// Doubles of LDS a wave needs: the exact keys of one token or of its tokens'
// candidates, or its tokens' fp32 keys.
__host__ __device__ inline int route_keys(int E, int tokens, int keys) {
    const int a = E > kCands * tokens ? E : kCands * tokens, b = keys * tokens / 2;
    const int c = a > b ? a : b;
    return c + (c & 1);  // 16-byte multiples
}

// L lanes per token, V logits per lane (blocks of 4 neighbours, L blocks
// apart), so E <= L * V. Each lane sorts its keys, and the rounds of the
// selection compare the lanes' heads: 4 DPP steps a round for the four tokens
// of a wave at 16 lanes each. The keys are compared as 32-bit integers whose
// low bits hold the place:
//   BY_LOGIT (no bias, no group sums: the keys' order is the logits')  16-bit
//     logits leave 13 bits for the whole id, and ties are decided; fp32
//     logits lose 4 bits to the place in the lane
//   else  keys in fp32, whose distance from the exact ones is bounded
// Where two neighbours are nearer than what was lost, the rounds go on past k
// until the gap behind the last is wide enough, and the candidates so far are
// put in order by their exact keys. Groups too near each other at their border
// (and more than kCands candidates) leave the token to route_exact: the result
// is always the defined one. Moves E logits per token; bound by the VALU work
// of the sort and the rounds: 30 us for 8 x 8192 tokens of 256 fp32 experts,
// top 8 (11.5 us of bytes; the VALUs issue in 61 % of the cycles, 203
// instructions a token). 8 x 4096 bf16 tokens in groups with a bias 35-45 us, by
// how many near neighbours the inputs hold: 410 instructions a token, 42 % of the
// cycles, the rest waits for the group sums' LDS reads, one after the other.
// 16 lanes a token share a wave's DPP steps among four tokens; one wave a token
// with every comparison in double (k_moe_route_exact) took 265 and 148.
template <int TYPE, int L, int V, bool BY_LOGIT>
__global__ __launch_bounds__(256) void k_moe_route(const RouteArgs a, bool vec, int64_t block0) {
    constexpr bool kIds = BY_LOGIT && TYPE != A2AV_DT_F32;   // whole ids in the keys
    constexpr uint32_t kLow = kIds ? 0x1fff : V - 1;
    constexpr int kTokens = kWave / L, kWaves = 4;
    extern __shared__ __align__(16) double keys[];  // a wave's exact keys of one token, or its tokens' fp32 keys
    constexpr int kSorted = V * kWave > kTokens * kCands ? V : (kTokens * kCands + kWave - 1) / kWave;
    __shared__ uint32_t sorted[kWaves][kSorted][kWave];      // or the candidates in order
    __shared__ int sel[kWaves][kTokens][kCands];
    if (status_at_entry(a.status)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int sub = lane & (L - 1), mine = lane / L;
    const int E = a.E, k = a.k;
    const float inf = __builtin_huge_valf();
    double *key = keys + (size_t)wave * route_keys(E, kTokens, a.groups > 1 ? L * V : 0);
    float *group_keys = (float *)key + mine * (L * V);
    const int64_t n = (int64_t)a.W * a.T;
    const bool full = !a.sigmoid && (!BY_LOGIT || !a.renorm);  // needs the softmax's sum
    const uint64_t my_lanes = L == 64 ? ~0ull : 0xffffull << (lane & 48);
    // no loop over tokens: the compiler would keep the constants of the double
    // exponentials in registers across it
    const int64_t i0 = (block0 + (int64_t)blockIdx.x) * (kWaves * kTokens) + wave * kTokens;
    if (i0 < n) {
        const bool store = i0 + mine < n;
        const int64_t i = store ? i0 + mine : n - 1;
        const int r = (int)(i / a.T);
        const int64_t t = i - (int64_t)r * a.T;
        const void *row = logit_row<TYPE>(a.z[r], t, E);
        float z[V];
        int bad = 0;
        load_logits<TYPE, L, V>(row, E, sub, vec, z);
        float m = -inf;
#pragma unroll
        for (int v = 0; v < V; v++) {
            bad |= z[v] != z[v] || (!a.sigmoid && z[v] == inf);
            m = fmaxf(m, z[v]);
        }
        const bool is_bad = (__ballot(bad) & my_lanes) != 0;
        float sum = 0.0f, key_err = 0.0f;
        float c[V];
        m = lanes_max<L>(m);
        if (full) {
#pragma unroll
            for (int v = 0; v < V; v++) {
                c[v] = z[v] == -inf ? 0.0f : __expf(z[v] - m);
                sum += c[v];
            }
            sum = lanes_sum<L>(sum);
        }
        if constexpr (BY_LOGIT) {
#pragma unroll
            for (int v = 0; v < V; v++) c[v] = z[v];
        } else {
            // sigmoid: the exponential's relative error is |z| 2^-23 at most and
            // s (1 - s) |z| < 0.23, with a step each of the exponential, the sum
            // and the reciprocal 0.23 + 0.25 + 1 + 1 steps of 2^-23; softmax: a step for every term of
            // the sum and a few more, relative to at most 1 / sum
            key_err = a.sigmoid ? 0x1p-21f : (V + 40) * 0x1p-23f / sum;
            if (a.sigmoid) {
#pragma unroll
                for (int v = 0; v < V; v++) c[v] = __builtin_amdgcn_rcpf(1.0f + __expf(-z[v]));
            } else {
                const float scale = 1.0f / sum;
#pragma unroll
                for (int v = 0; v < V; v++) c[v] *= scale;
            }
            if (a.bias) {
                float b[V];
                load_logits<A2AV_DT_F32, L, V>(a.bias, E, sub, vec, b);
#pragma unroll
                for (int v = 0; v < V; v++) c[v] += b[v];
            }
#pragma unroll
            for (int v = 0; v < V; v++) c[v] = z[v] == -inf || c[v] != c[v] ? -inf : c[v];
        }
        bool unsure = false;  // of the groups
        uint32_t kept = ~0u;
        if (a.groups > 1) {
            const int per = E / a.groups;
#pragma unroll
            for (int v = 0; v < V; v += 4)
                *(f32x4 *)(group_keys + (v / 4 * L + sub) * 4) = f32x4{c[v], c[v + 1], c[v + 2], c[v + 3]};
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            float t1 = -inf, t2 = -inf;
            if (sub < a.groups) {
                int at = sub % per;  // the lanes start at different banks
#pragma unroll 8
                for (int q = 0; q < per; q++) {
                    const float x = group_keys[sub * per + at];
                    t2 = fmaxf(t2, fminf(t1, x));
                    t1 = fmaxf(t1, x);
                    at = at + 1 == per ? 0 : at + 1;
                }
            }
            float gs = a.group_top == 1 ? t1 : t1 + t2;
            if (gs != gs) gs = -inf;
            int before = 0;
#pragma unroll 4
            for (int g = 0; g < a.groups; g++) {
                const float o = __shfl(gs, g, L);
                before += o > gs || (o == gs && g < sub);
            }
            const bool in = sub < a.groups && before < a.topk_groups;
            kept = (uint32_t)((__ballot(in) >> (L == 64 ? 0 : lane & 48)));
            if constexpr (BY_LOGIT) {
                // Logits that differ may have equal scores in double, which leave
                // the choice to the group's number: saturated, vanished or tiny
                // ones. From 2^-20 to 16 (softmax: at most 64 below the largest)
                // the nearest other logit is 2^-24 of it away or more, and the
                // scores then differ by over 2^-46 of a score of 1, or of the
                // score itself: far above the errors of double. Where that holds
                // for the last group kept, its score is no other logit's.
                const float low = -lanes_max<L>(in ? -gs : -inf);
                const float size = fabsf(low);
                unsure = !(low == -inf || (size >= 0x1p-20f && (a.sigmoid ? size <= 16.0f : m - low <= 64.0f)));
            } else {
                // The least that a kept group's exact score can be, against the
                // most of a dropped one. A key is off by key_err and half a step
                // of itself (the bias's sum), however small the two keys' sum is;
                // twice that and more for the sum's own rounding and those here.
                // Infinite scores are what they are; beyond fp32's range a
                // dropped one is above every kept one.
                const float off = 2 * key_err + 0x1p-22f * (fabsf(t1) + (a.group_top == 1 ? 0.0f : fabsf(t2)));
                const bool exact = fabsf(gs) == inf;
                const float low = -lanes_max<L>(in ? (exact ? -gs : off - gs) : -inf);
                const float high = lanes_max<L>(sub < a.groups && !in ? (exact ? gs : gs + off) : -inf);
                unsure = !(low > high);
            }
        }
        uint32_t s[V];
        const float per_group = a.groups > 1 ? 1.0f / (float)(E / a.groups) : 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int e = ((v / 4) * L + sub) * 4 + v % 4;
            const uint32_t u = __float_as_uint(c[v] + 0.0f);  // -0 counts as 0
            const uint32_t o = u ^ ((int)u < 0 ? 0xffffffffu : 0x80000000u);
            s[v] = (o & ~kLow) | (kIds ? kLow - e : kLow - v);
            bool live = e < E;
            if (a.groups > 1) live = live && ((kept >> (int)(((float)e + 0.5f) * per_group)) & 1);
            s[v] = live ? s[v] : 0;
        }
        // Batcher's odd-even merge sort, descending
#pragma unroll
        for (int p = 1; p < V; p *= 2)
#pragma unroll
            for (int q = p; q >= 1; q /= 2)
#pragma unroll
                for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                    for (int x = 0; x < q; x++)
                        if (x + j + q < V && (x + j) / (2 * p) == (x + j + q) / (2 * p)) {
                            const uint32_t hi = max(s[x + j], s[x + j + q]), lo = min(s[x + j], s[x + j + q]);
                            s[x + j] = hi;
                            s[x + j + q] = lo;
                        }
#pragma unroll
        for (int v = 0; v < V; v++) sorted[wave][v][lane] = s[v];
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        uint32_t head = s[0], last = 0;
        int at = 0, count = 0;
        bool mixed = false, closed = false;  // two candidates too near each other; the last one found
        const uint64_t below = (1ull << lane) - 1;
        for (int j = 0; j < kCands; j++) {
            const uint32_t top = lanes_max_u32<L>(head);
            bool near = false;
            if constexpr (!kIds) {
                if (BY_LOGIT) {
                    near = (top & ~kLow) == (last & ~kLow);
                } else {
                    // what the low bits hid is under 2^-19 of a key
                    const uint32_t x = last & ~kLow, y = top & ~kLow;
                    const float hi = __uint_as_float(x ^ ((int)x < 0 ? 0x80000000u : 0xffffffffu));
                    const float lo = __uint_as_float(y ^ ((int)y < 0 ? 0x80000000u : 0xffffffffu));
                    near = !(hi - lo > 2 * key_err + 0x1.01p-19f * fmaxf(fabsf(hi), fabsf(lo)));
                }
                near = near && j > 0;
                last = top;
            }
            near = near && top != 0;  // 0: no expert is left
            closed = closed || (j >= k && !near);
            if (__ballot(!closed) == 0) break;
            if (!closed) {
                mixed |= near;
                count = j + 1;
            }
            // of equal heads the first lane's goes
            const bool top_head = head == top && !closed;
            const uint64_t won = __ballot(top_head) & my_lanes;
            if (top_head && (won & below) == 0) {
                const int v = (int)(kLow - (top & kLow));
                sel[wave][mine][j] = kIds ? v : ((v / 4) * L + sub) * 4 + v % 4;
                at++;
                head = at < V ? sorted[wave][at][lane] : 0;
            }
        }
        unsure |= !closed;  // more candidates than there is room for
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (is_bad || !store) {
            for (int j = sub; j < k; j += L) sel[wave][mine][j] = j;
            unsure = mixed = false;
        }
        mixed = mixed && !unsure;
        if (!kIds && __ballot(mixed) != 0) {
            // loops that keep nothing in registers: this is seldom reached, and
            // its registers would cost every wave
            double total = 1.0;
            if (!BY_LOGIT && !a.sigmoid) {
                total = 0.0;
#pragma unroll 1
                for (int e = sub; e < E; e += L) {
                    const float x = logit_at<TYPE>(row, e);
                    if (x != -inf) total += exp((double)x - m);
                }
#pragma unroll 1
                for (int o = L / 2; o; o >>= 1) total += __shfl_xor(total, o);
            }
            double *mine_key = key + mine * kCands;
            int *ids = sel[wave][mine], *in_order = (int *)&sorted[wave][0][0] + mine * kCands;
            if (mixed) {
#pragma unroll 1
                for (int j = sub; j < count; j += L) {
                    const double x = logit_at<TYPE>(row, ids[j]);
                    double y = x;
                    if (!BY_LOGIT) {
                        y = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / total;
                        if (a.bias) y += a.bias[ids[j]];
                        if (x == -inf || y != y) y = -inf;
                    }
                    mine_key[j] = y;
                }
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (mixed) {
#pragma unroll 1
                for (int j = sub; j < count; j += L) {
                    const double y = mine_key[j];
                    const int id = ids[j];
                    int rank = 0;
#pragma unroll 1
                    for (int q = 0; q < count; q++) {
                        const double o = mine_key[q];
                        bool first = o > y;
                        if (o == y && q != j) {
                            const int oid = ids[q];
                            const float x = logit_at<TYPE>(row, id), ox = logit_at<TYPE>(row, oid);
                            first = ox > x || (ox == x && oid < id);
                        }
                        rank += first;
                    }
                    in_order[rank] = id;
                }
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (mixed)
                for (int j = sub; j < k; j += L) ids[j] = in_order[j];
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        // tokens to do again, one after the other, by the whole wave
        uint64_t again = __ballot(unsure && sub == 0);
        while (again) {
            const int l = __builtin_ctzll(again);
            again &= again - 1;
            const int64_t i2 = i0 + l / L;
            const int r2 = (int)(i2 / a.T);
            const void *row2 = logit_row<TYPE>(a.z[r2], i2 - (int64_t)r2 * a.T, E);
            bool none;
            const int id = route_exact<TYPE>(a, row2, key, lane, &none);
            if (lane < k) sel[wave][l / L][lane] = id;
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        route_weights<TYPE, L>(a, row, sel[wave][mine], sub, is_bad, m, sum, a.ids[r] + t * k, a.w[r] + t * k, store);
    }
}

// ------------------------------------------------------------------ gradient
struct RouteGradArgs {
    const void *z[A2AV_MAX_W];
    const int32_t *ids[A2AV_MAX_W];
    const float *w[A2AV_MAX_W];
    const float *dw[A2AV_MAX_W];
    void *dz[A2AV_MAX_W];
    int32_t *status;
    int64_t T;
    int W, k, E;
    int sigmoid, renorm;
    float scale;
};

__global__ __launch_bounds__(256) void k_route_check(const RouteGradArgs a) {
    if (status_poisoned(a.status)) return;
    const int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t Q = a.T * a.k;
    int bad = 0;
    if (q < Q) bad = (unsigned)a.ids[blockIdx.y][q] >= (unsigned)a.E;
    if (__ballot(bad) != 0 && (threadIdx.x & (kWave - 1)) == 0) atomicOr(a.status, A2AV_ST_BAD_EXPERT);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

// fp32 -> an element of d_logits.
template <int TYPE>
__device__ __forceinline__ void store_logit(void *row, int64_t i, float v) {
    if constexpr (TYPE == A2AV_DT_F32) ((float *)row)[i] = v;
    else if constexpr (TYPE == A2AV_DT_BF16) ((uint16_t *)row)[i] = (uint16_t)to_bf16(v);
    else ((_Float16 *)row)[i] = (_Float16)v;
}

// One wave per token (84 us for 8 x 1024 tokens of 2048 fp32 experts, 161 of
// 4096). Lane j holds ds_j * s_j of chosen expert j (scale taken out of the
// weights, so that s_j / S is w_j / scale), and every lane adds up what falls on
// its experts, in slot order.
template <int TYPE>
__global__ __launch_bounds__(256) void k_moe_route_backward_any(const RouteGradArgs a) {
    if (status_at_entry(a.status)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int waves = blockDim.x / kWave;
    const int64_t n = (int64_t)a.W * a.T;
    const float inf = __builtin_huge_valf();
    for (int64_t i = (int64_t)blockIdx.x * waves + wave; i < n; i += (int64_t)gridDim.x * waves) {
        const int r = (int)(i / a.T);
        const int64_t t = i - (int64_t)r * a.T;
        const void *row = logit_row<TYPE>(a.z[r], t, a.E);
        void *out = (void *)logit_row<TYPE>(a.dz[r], t, a.E);
        const bool on = lane < a.k;
        const int id = on ? a.ids[r][t * a.k + lane] : -1;
        const float w = on ? a.w[r][t * a.k + lane] : 0.0f;
        const float g = on ? a.dw[r][t * a.k + lane] : 0.0f;
        // v = ds_j * s_j, and for softmax without renorm their sum
        const float dot = wave_sum(g * w);
        float v = w * g;
        if (a.renorm) v = a.scale == 0 ? 0.0f : w * (g - dot / a.scale);
        if (a.sigmoid && on) v *= 1.0f / (1.0f + expf(logit_at<TYPE>(row, id)));
        float m = 0.0f, f = 0.0f;
        const bool full = !a.sigmoid && !a.renorm;
        const auto part = [&](float z) { return z == -inf ? 0.0f : expf(z - m); };
        if (full) {
            m = -inf;
            for (int e = lane; e < a.E; e += kWave) m = fmaxf(m, logit_at<TYPE>(row, e));
            m = wave_max(m);
            float sum = 0.0f;
            // a row of -inf has no gradient; NaN passes on
            for (int e = lane; e < a.E; e += kWave) sum += part(logit_at<TYPE>(row, e));
            sum = wave_sum(sum);
            f = sum == 0.0f ? 0.0f : dot / sum;
        }
        for (int e0 = 0; e0 < a.E; e0 += kWave) {
            const int e = e0 + lane;
            float d = 0.0f;
            for (int j = 0; j < a.k; j++) {
                const int ej = __shfl(id, j);
                const float vj = __shfl(v, j);
                d += ej == e ? vj : 0.0f;
            }
            if (e < a.E) {
                if (full) d -= f * part(logit_at<TYPE>(row, e));
                store_logit<TYPE>(out, e, d);
            }
        }
    }
}

// L lanes per token, V logits per lane, as k_moe_route. Lane j holds ds_j * s_j
// of chosen expert j; the first of equal ids collects their sum (in slot
// order), so that the row's gradients meet in LDS without atomics. Writes E
// values per token and reads them where softmax is not renormalised; bound by
// those bytes: 30 us for 8 x 8192 tokens of 256 fp32 experts (22.7 us at the
// rate of a plain copy; one wave a token 83).
template <int TYPE, int L, int V>
__global__ __launch_bounds__(256) void k_moe_route_backward(const RouteGradArgs a, bool vec) {
    constexpr int kTokens = kWave / L, kWaves = 4;
    __shared__ __align__(16) float rows[kWaves][kTokens][L * V];
    __shared__ int ids[kWaves][kTokens][kWave];
    __shared__ float vals[kWaves][kTokens][kWave];
    if (status_at_entry(a.status)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int sub = lane & (L - 1), mine = lane / L;
    const int E = a.E, k = a.k;
    const float inf = __builtin_huge_valf();
    const int64_t n = (int64_t)a.W * a.T;
    const bool full = !a.sigmoid && !a.renorm;
    float *d = rows[wave][mine], *val = vals[wave][mine];
    int *id = ids[wave][mine];
    for (int64_t i0 = ((int64_t)blockIdx.x * kWaves + wave) * kTokens; i0 < n; i0 += (int64_t)gridDim.x * kWaves * kTokens) {
        const bool store = i0 + mine < n;
        const int64_t i = store ? i0 + mine : n - 1;
        const int r = (int)(i / a.T);
        const int64_t t = i - (int64_t)r * a.T;
        const void *row = logit_row<TYPE>(a.z[r], t, E);
        void *out = (void *)logit_row<TYPE>(a.dz[r], t, E);
        float z[V];
        if (full) {
            load_logits<TYPE, L, V>(row, E, sub, vec, z);
        }
        float dot = 0.0f;
        for (int j = sub; j < k; j += L) dot += a.dw[r][t * k + j] * a.w[r][t * k + j];
        dot = lanes_sum<L>(dot);
        for (int j = sub; j < k; j += L) {
            const int e = a.ids[r][t * k + j];
            const float w = a.w[r][t * k + j], g = a.dw[r][t * k + j];
            float v = w * g;
            if (a.renorm) v = a.scale == 0 ? 0.0f : w * (g - dot / a.scale);
            if (a.sigmoid) v *= 1.0f / (1.0f + expf(logit_at<TYPE>(row, e)));
            id[j] = e;
            val[j] = v;
        }
#pragma unroll
        for (int v = 0; v < V; v += 4) *(f32x4 *)(d + (v / 4 * L + sub) * 4) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int j = sub; j < k; j += L) {
            float v = 0.0f;
            bool first = true;
            const int e = id[j];
            for (int q = 0; q < k; q++) {
                const bool same = id[q] == e;
                first = first && !(same && q < j);
                v += same ? val[q] : 0.0f;
            }
            if (first) d[e] = v;
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float f = 0.0f;
        if (full) {
            float m = -inf, sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) m = fmaxf(m, z[v]);
            m = lanes_max<L>(m);
#pragma unroll
            for (int v = 0; v < V; v++) {
                // a row of -inf has no gradient; NaN passes on
                z[v] = z[v] == -inf ? 0.0f : __expf(z[v] - m);
                sum += z[v];
            }
            sum = lanes_sum<L>(sum);
            f = sum == 0.0f ? 0.0f : dot / sum;
        }
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const int e = (v / 4 * L + sub) * 4;
            f32x4 y = *(const f32x4 *)(d + e);
            if (full) {
#pragma unroll
                for (int q = 0; q < 4; q++) y[q] -= f * z[v + q];
            }
            if (!store) continue;
            if (vec) {
                if (e < E) {
                    if constexpr (TYPE == A2AV_DT_F32) {
                        *(f32x4 *)((float *)out + e) = y;
                    } else {
                        uint16_t h[4];
#pragma unroll
                        for (int q = 0; q < 4; q++) store_logit<TYPE>(h, q, y[q]);
                        u32x2 o;
                        o.x = h[0] | (uint32_t)h[1] << 16;
                        o.y = h[2] | (uint32_t)h[3] << 16;
                        *(u32x2 *)((uint16_t *)out + e) = o;
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (e + q < E) store_logit<TYPE>(out, e + q, y[q]);
            }
        }
    }
}

static bool route_sizes_ok(int W, int64_t T, int k, int E, int type, int score) {
    if (W < 1 || W > A2AV_MAX_W || T < 0 || k < 1 || k > kWave || E < 1 || E > A2AV_MAX_EXPERTS) return false;
    if (type < A2AV_DT_F32 || type > A2AV_DT_F16) return false;
    if (score != A2AV_SCORE_SOFTMAX && score != A2AV_SCORE_SIGMOID) return false;
    return T <= ((int64_t)1 << 31) / k && T * k < ((int64_t)1 << 31);
}

static unsigned wave_grid(int64_t waves, int per_block) {
    uint64_t blocks = ((uint64_t)waves + per_block - 1) / per_block;
    if (blocks > max_grid()) blocks = max_grid();  // the wave loop strides over the rest
    return (unsigned)blocks;
}

template <int TYPE, int L, int V>
static void launch_route(const RouteArgs &a, bool by_logit, bool vec, hipStream_t stream) {
    const int64_t tokens = 4 * kWave / L, all = ((int64_t)a.W * a.T + tokens - 1) / tokens;
    const unsigned lds = (unsigned)(4 * route_keys(a.E, kWave / L, a.groups > 1 ? L * V : 0) * sizeof(double));
    for (int64_t b = 0; b < all; b += max_grid()) {
        const dim3 g((unsigned)(all - b < max_grid() ? all - b : max_grid()));
        if (by_logit) hipLaunchKernelGGL((k_moe_route<TYPE, L, V, true>), g, dim3(256), lds, stream, a, vec, b);
        else hipLaunchKernelGGL((k_moe_route<TYPE, L, V, false>), g, dim3(256), lds, stream, a, vec, b);
    }
}

template <int TYPE>
static void launch_route(const RouteArgs &a, bool vec, hipStream_t stream) {
    // the order of the keys is that of the logits: no bias, and no sums of scores
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    const int E = a.E;
    if (E > 1024 || (a.groups > 1 && a.groups > (E <= 256 ? 16 : 32))) {
        const int waves = E <= 1024 ? 4 : 1;
        hipLaunchKernelGGL(k_moe_route_exact<TYPE>, dim3(wave_grid((int64_t)a.W * a.T, waves)), dim3(waves * kWave),
                           (unsigned)(waves * E * sizeof(double)), stream, a);
    } else if (E <= 64) {
        launch_route<TYPE, 16, 4>(a, by_logit, vec, stream);
    } else if (E <= 128) {
        launch_route<TYPE, 16, 8>(a, by_logit, vec, stream);
    } else if (E <= 256) {
        launch_route<TYPE, 16, 16>(a, by_logit, vec, stream);
    } else {
        launch_route<TYPE, 64, 16>(a, by_logit, vec, stream);
    }
}

template <int TYPE, int L, int V>
static void launch_route_backward(const RouteGradArgs &a, bool vec, hipStream_t stream) {
    const unsigned blocks = wave_grid(((int64_t)a.W * a.T * L + kWave - 1) / kWave, 4);
    hipLaunchKernelGGL((k_moe_route_backward<TYPE, L, V>), dim3(blocks), dim3(256), 0, stream, a, vec);
}

template <int TYPE>
static void launch_route_backward(const RouteGradArgs &a, bool vec, hipStream_t stream) {
    if (a.E > 1024) {
        const unsigned blocks = wave_grid((int64_t)a.W * a.T, 4);
        hipLaunchKernelGGL(k_moe_route_backward_any<TYPE>, dim3(blocks), dim3(256), 0, stream, a);
    } else if (a.E <= 64) {
        launch_route_backward<TYPE, 16, 4>(a, vec, stream);
    } else if (a.E <= 128) {
        launch_route_backward<TYPE, 16, 8>(a, vec, stream);
    } else if (a.E <= 256) {
        launch_route_backward<TYPE, 16, 16>(a, vec, stream);
    } else {
        launch_route_backward<TYPE, 64, 16>(a, vec, stream);
    }
}

}  // namespace a2av

using namespace a2av;

A2AV_API int moe_route(int W, int64_t T, int k, int E, int type, int score,
                       const void *const *logits, const float *bias, int groups, int topk_groups,
                       int group_top, int renorm, float scale, int32_t *const *ids,
                       float *const *weights, int32_t *status, hipStream_t stream) {
    if (!route_sizes_ok(W, T, k, E, type, score) || !logits || !ids || !weights || !status)
        return A2AV_EARG;
    if (groups < 1 || groups > kMaxGroups || E % groups != 0 || topk_groups < 1 ||
        topk_groups > groups || group_top < 1 || group_top > 2 || group_top > E / groups ||
        k > topk_groups * (E / groups))
        return A2AV_EARG;
    RouteArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int r = 0; r < W; r++) {
        if (T > 0 && (!logits[r] || !ids[r] || !weights[r])) return A2AV_EARG;
        a.z[r] = logits[r];
        a.ids[r] = ids[r];
        a.w[r] = weights[r];
    }
    a.bias = bias;
    a.status = status;
    a.T = T;
    a.W = W;
    a.k = k;
    a.E = E;
    a.groups = topk_groups == groups ? 1 : groups;  // keeping every group is no grouping
    a.topk_groups = topk_groups;
    a.group_top = group_top;
    a.sigmoid = score == A2AV_SCORE_SIGMOID;
    a.renorm = renorm != 0;
    a.scale = scale;
    if (T == 0) return A2AV_OK;
    bool vec = E % 4 == 0 && (uintptr_t)bias % 16 == 0;
    for (int r = 0; r < W; r++) vec = vec && (uintptr_t)logits[r] % 16 == 0;
    switch (type) {
    case A2AV_DT_F32: launch_route<A2AV_DT_F32>(a, vec, stream); break;
    case A2AV_DT_BF16: launch_route<A2AV_DT_BF16>(a, vec, stream); break;
    default: launch_route<A2AV_DT_F16>(a, vec, stream); break;
    }
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}

A2AV_API int moe_route_backward(int W, int64_t T, int k, int E, int type, int score,
                                const void *const *logits, const int32_t *const *ids,
                                const float *const *weights, int renorm, float scale,
                                const float *const *d_weights, void *const *d_logits,
                                int32_t *status, hipStream_t stream) {
    if (!route_sizes_ok(W, T, k, E, type, score) || !logits || !ids || !weights || !d_weights ||
        !d_logits || !status)
        return A2AV_EARG;
    RouteGradArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int r = 0; r < W; r++) {
        if (T > 0 && (!logits[r] || !ids[r] || !weights[r] || !d_weights[r] || !d_logits[r]))
            return A2AV_EARG;
        a.z[r] = logits[r];
        a.ids[r] = ids[r];
        a.w[r] = weights[r];
        a.dw[r] = d_weights[r];
        a.dz[r] = d_logits[r];
    }
    a.status = status;
    a.T = T;
    a.W = W;
    a.k = k;
    a.E = E;
    a.sigmoid = score == A2AV_SCORE_SIGMOID;
    a.renorm = renorm != 0;
    a.scale = scale;
    if (T == 0) return A2AV_OK;
    hipLaunchKernelGGL(k_route_check, dim3((unsigned)((T * k + 255) / 256), W), dim3(256), 0, stream, a);
    bool vec = E % 4 == 0;
    for (int r = 0; r < W; r++)
        vec = vec && (uintptr_t)logits[r] % 16 == 0 && (uintptr_t)d_logits[r] % 16 == 0;
    switch (type) {
    case A2AV_DT_F32: launch_route_backward<A2AV_DT_F32>(a, vec, stream); break;
    case A2AV_DT_BF16: launch_route_backward<A2AV_DT_BF16>(a, vec, stream); break;
    default: launch_route_backward<A2AV_DT_F16>(a, vec, stream); break;
    }
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
