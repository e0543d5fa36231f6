// route.hip — the router in front of the MoE pack, and its gradient (gfx950).
//
//   k_moe_route           expert ids and gate weights of every token
//   k_route_check         range check of the ids the gradient scatters to
//   k_moe_route_backward  the gradient of the weights in the logits
#include <hip/hip_runtime.h>

#include <cstring>

#include "common.hpp"

namespace a2av {

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

// One token by one wave, every comparison in double as the result is defined:
// scores and keys of all experts into LDS, the groups' scores by one lane
// each, then k rounds of a wave-wide argmax. Lane j ends with id j and its
// score in *id and *p; the return value tells a token that has NaN weights.
template <int TYPE>
__device__ __forceinline__ bool route_exact(const RouteArgs &a, const void *row, double *key,
                                            int lane, int *id, double *p) {
    const double inf = __builtin_huge_val(), nan = __builtin_nan("");
    const int E = a.E;
    double m = -inf;
    int bad = 0;
    for (int e = lane; e < E; e += kWave) {
        const double z = logit_at<TYPE>(row, e);
        bad |= z != z || (!a.sigmoid && z == inf);
        m = fmax(m, z);
    }
    *id = lane;
    *p = nan;
    if (__ballot(bad)) return true;
    double inv = 1.0;
    if (!a.sigmoid) {
        m = wave_max(m);
        double sum = 0;
        for (int e = lane; e < E; e += kWave) {
            const double z = logit_at<TYPE>(row, e);
            if (z != -inf) sum += exp(z - m);
        }
        sum = wave_sum(sum);
        inv = sum;
    }
    const auto score = [&](double z) {
        if (z == -inf) return 0.0;
        return a.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - m) / inv;
    };
    for (int e = lane; e < E; e += kWave) {
        const double z = logit_at<TYPE>(row, e);
        double c = score(z) + (a.bias ? (double)a.bias[e] : 0.0);
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
        for (int g = 0; g < a.groups; g++) {
            const double o = __shfl(gs, g);
            before += o > gs || (o == gs && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.groups && before < a.topk_groups);
        for (int e = lane; e < E; e += kWave)
            if (!((kept >> (e / per)) & 1)) key[e] = nan;
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    for (int j = 0; j < a.k; j++) {
        double c = -inf;
        float z = -__builtin_huge_valf();
        int best = E;  // no expert: behind every real one
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
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const double oc = __shfl_xor(c, o);
            const float oz = __shfl_xor(z, o);
            const int oe = __shfl_xor(best, o);
            const bool take = oe != E && (best == E || oc > c || (oc == c && (oz > z || (oz == z && oe < best))));
            c = take ? oc : c;
            z = take ? oz : z;
            best = take ? oe : best;
        }
        if (lane == j) {
            *id = best;
            *p = score(z);
        }
        if (lane == 0) key[best] = nan;
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    return false;
}

// One wave per token.
template <int TYPE>
__global__ __launch_bounds__(256) void k_moe_route(const RouteArgs a) {
    extern __shared__ double keys[];
    if (status_at_entry(a.status)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int waves = blockDim.x / kWave;
    double *key = keys + (size_t)wave * a.E;
    const int64_t n = (int64_t)a.W * a.T;
    for (int64_t i = (int64_t)blockIdx.x * waves + wave; i < n; i += (int64_t)gridDim.x * waves) {
        const int r = (int)(i / a.T);
        const int64_t t = i - (int64_t)r * a.T;
        int id;
        double p;
        route_exact<TYPE>(a, logit_row<TYPE>(a.z[r], t, a.E), key, lane, &id, &p);
        if (a.renorm) {
            const double S = wave_sum(lane < a.k ? p : 0.0);
            p = S == 0 ? 0.0 : p / S;
        }
        if (lane < a.k) {
            a.ids[r][t * a.k + lane] = id;
            a.w[r][t * a.k + lane] = (float)(p * a.scale);
        }
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

// One wave per token. Lane j holds ds_j * s_j of chosen expert j (scale taken
// out of the weights, so that s_j / S is w_j / scale), and every lane adds up
// what falls on its experts, in slot order.
template <int TYPE>
__global__ __launch_bounds__(256) void k_moe_route_backward(const RouteGradArgs a) {
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
        if (full) {
            m = -inf;
            for (int e = lane; e < a.E; e += kWave) m = fmaxf(m, logit_at<TYPE>(row, e));
            m = wave_max(m);
            float sum = 0.0f;
            for (int e = lane; e < a.E; e += kWave) sum += m == -inf ? 0.0f : expf(logit_at<TYPE>(row, e) - m);
            sum = wave_sum(sum);
            f = sum > 0 ? dot / sum : 0.0f;
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
                if (full && m != -inf) d -= f * expf(logit_at<TYPE>(row, e) - m);
                store_logit<TYPE>(out, e, d);
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
    const int waves = E <= 1024 ? 4 : 1;
    const unsigned blocks = wave_grid((int64_t)W * T, waves), lds = (unsigned)(waves * E * sizeof(double));
    switch (type) {
    case A2AV_DT_F32: hipLaunchKernelGGL(k_moe_route<A2AV_DT_F32>, dim3(blocks), dim3(waves * kWave), lds, stream, a); break;
    case A2AV_DT_BF16: hipLaunchKernelGGL(k_moe_route<A2AV_DT_BF16>, dim3(blocks), dim3(waves * kWave), lds, stream, a); break;
    default: hipLaunchKernelGGL(k_moe_route<A2AV_DT_F16>, dim3(blocks), dim3(waves * kWave), lds, stream, a); break;
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
    const unsigned blocks = wave_grid((int64_t)W * T, 4);
    switch (type) {
    case A2AV_DT_F32: hipLaunchKernelGGL(k_moe_route_backward<A2AV_DT_F32>, dim3(blocks), dim3(256), 0, stream, a); break;
    case A2AV_DT_BF16: hipLaunchKernelGGL(k_moe_route_backward<A2AV_DT_BF16>, dim3(blocks), dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL(k_moe_route_backward<A2AV_DT_F16>, dim3(blocks), dim3(256), 0, stream, a); break;
    }
    return hipGetLastError() == hipSuccess ? A2AV_OK : A2AV_EHIP;
}
