// Routing to experts: one wavefront per token.
//
//   score[e] = exp(l[e] - max) / sum exp(l - max)   or   1 / (1 + exp(-l[e]))
//   choice[e] = score[e] + bias[e];  the top_groups groups with the largest sum
//   of their group_best largest choices stay;  the k largest choices of them
//   (ties: the lowest index) are the token's experts, with the weights
//   score[e] (/ their sum) * scale.
//
// Two scores that differ in the last bit of f32 decide which expert runs, so
// everything that a choice depends on is f64 (full rate on this chip); where
// the choice is the order of the logits themselves (no bias, and no group sums
// of more than one) they are compared as they are.  Lane l holds the
// experts l, l + 64, ...: the largest choice is a wavefront maximum, its first
// holder a ballot per 64 experts.  Bound by the k rounds of that (some 30
// instructions each) from a few hundred tokens on, below by the launch.
#include <cfloat>

#include "qlin_device.h"
#include "w4_internal.h"

namespace qlin {

namespace {

constexpr int kRouteWaves = 4;

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp_i<CTRL>((int)(uint32_t)b), hi = (uint32_t)dpp_i<CTRL>((int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_d(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_max(double v) {
    v = fmax(v, dpp_d<0xB1>(v));
    v = fmax(v, dpp_d<0x4E>(v));
    v = fmax(v, dpp_d<0x141>(v));
    v = fmax(v, dpp_d<0x140>(v));
    return fmax(fmax(lane_d(v, 0), lane_d(v, 16)), fmax(lane_d(v, 32), lane_d(v, 48)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_f<0xB1>(v));
    v = fmaxf(v, dpp_f<0x4E>(v));
    v = fmaxf(v, dpp_f<0x141>(v));
    v = fmaxf(v, dpp_f<0x140>(v));
    auto at = [v](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
    return fmaxf(fmaxf(at(0), at(16)), fmaxf(at(32), at(48)));
}
__device__ __forceinline__ int wave_max(int v) {
    v = max(v, dpp_i<0xB1>(v));
    v = max(v, dpp_i<0x4E>(v));
    v = max(v, dpp_i<0x141>(v));
    v = max(v, dpp_i<0x140>(v));
    auto at = [v](int l) { return __builtin_amdgcn_readlane(v, l); };
    return max(max(at(0), at(16)), max(at(32), at(48)));
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_d<0xB1>(v);
    v += dpp_d<0x4E>(v);
    v += dpp_d<0x141>(v);
    v += dpp_d<0x140>(v);
    return (lane_d(v, 0) + lane_d(v, 16)) + (lane_d(v, 32) + lane_d(v, 48));
}

// The choices in their order, as numbers of type Key.  Below every choice of
// an expert that takes part: kMasked (an expert that is masked out comes after
// every other expert of the groups that stay), and below that kGone (experts of
// dropped groups, and those taken already).
template <class Key> struct Order;
template <> struct Order<double> {           // scores and biases: no NaN, no infinity
    static constexpr double kGone = -INFINITY, kMasked = -DBL_MAX;
    static __device__ __forceinline__ double of(double v) { return v >= -DBL_MAX ? fmin(v, DBL_MAX) : -DBL_MAX; }
};
template <> struct Order<int> {              // logits: the bits of a float, in the order of its values
    static constexpr int kGone = INT32_MIN, kMasked = INT32_MIN + 1;
    static __device__ __forceinline__ int of(float v) {
        const int b = __float_as_int(v + 0.0f);   // -0 equals 0
        return b ^ ((b >> 31) & 0x7FFFFFFF);
    }
};

// V: experts per lane.  Key: the type of the choice (double: from the scores,
// int: the logits).
template <int V, class Key, class Logit>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(
    const Logit* __restrict__ logits, int64_t T, int E, int k, int score, const float* __restrict__ bias, int groups,
    int top_groups, int group_best, bool renorm, float scale, int32_t* __restrict__ ids, float* __restrict__ weights) {
    __shared__ double lds[kRouteWaves][V * 64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= T) return;   // wavefronts share nothing: no barrier below
    double* __restrict__ mine = lds[wave];

    float l[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 64 + lane;
        float v = -INFINITY;
        if (e < E) {
            if constexpr (sizeof(Logit) == 2) v = bf16_lo(logits[t * E + e]);
            else v = logits[t * E + e];
        }
        l[j] = v >= -FLT_MAX ? fminf(v, FLT_MAX) : -INFINITY;   // NaN: as -infinity
    }

    // scores (not divided by the softmax's sum yet)
    double p[V], total = 1.0;
    if (score == 0) {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
        m = wave_max(m);
        double z = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[j] = l[j] == -INFINITY ? 0.0 : exp((double)l[j] - (double)m);
            z += p[j];
        }
        total = wave_sum(z);
        if (total == 0.0) total = 1.0;   // every expert masked out
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = l[j] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[j]));
    }

    Key c[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 64 + lane;
        if constexpr (sizeof(Key) == 8) {
            double v = score == 0 ? p[j] / total : p[j];
            if (bias && e < E) v += (double)bias[e];
            c[j] = Order<Key>::of(v);
        } else {
            c[j] = Order<Key>::of(l[j]);
        }
        if (l[j] == -INFINITY) c[j] = Order<Key>::kMasked;
        if (e >= E) c[j] = Order<Key>::kGone;
    }

    if (groups > 1) {
        const int size = E / groups;
#pragma unroll
        for (int j = 0; j < V; ++j) mine[j * 64 + lane] = sizeof(Key) == 8 ? (double)c[j] : l[j] == -INFINITY ? -DBL_MAX : (double)l[j];
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
        // P lanes per group walk its experts and keep the two best
        int P = 64;
        while (P * groups > 64) P >>= 1;
        const int g = lane / P, part = lane % P;
        double a = -INFINITY, b = -INFINITY;
        if (g < groups)
            for (int i = part; i < size; i += P) {
                const double v = mine[g * size + i];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
        for (int d = 1; d < P; d <<= 1) {
            const double oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        double worth = group_best == 2 && size > 1 ? Order<double>::of(a + b) : a;
        // a group stays if fewer than top_groups groups come before it
        int before = 0;
        for (int o = 0; o < groups; ++o) {
            const double w = lane_d(worth, o * P);
            before += w > worth || (w == worth && o < g);
        }
        const uint64_t kept = __ballot(g < groups && before < top_groups);
        const uint32_t magic = ((1u << 21) + size - 1) / size;   // e / size for e, size <= 1024
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 64 + lane;
            const int of = (int)(((uint64_t)e * magic) >> 21);
            if (e < E && !((kept >> (of * P)) & 1)) c[j] = Order<Key>::kGone;
        }
        __threadfence_block();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) mine[j * 64 + lane] = p[j];

    int chosen = 0;   // lane r: the token's choice r
    for (int r = 0; r < k; ++r) {
        Key m = c[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = m > c[j] ? m : c[j];
        m = wave_max(m);
        int at = -1;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint64_t b = __ballot(c[j] == m);
            if (at < 0 && b) at = j * 64 + __builtin_ctzll(b);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j * 64 + lane == at) c[j] = Order<Key>::kGone;
        if (lane == r) chosen = at;
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double w = lane < k ? mine[chosen] : 0.0;
    if (renorm) {
        const double s = wave_sum(w);
        w = s > 0.0 ? w / s : 0.0;
    } else if (score == 0) {
        w /= total;
    }
    if (lane < k) {
        ids[t * k + lane] = chosen;
        weights[t * k + lane] = (float)(w * (double)scale);
    }
}

template <int V, class Key>
hipError_t run(const void* logits, bool f32, int64_t T, int E, int k, int score, const float* bias, int groups,
               int top_groups, int group_best, bool renorm, float scale, int32_t* ids, float* weights, hipStream_t st) {
    const unsigned grid = (unsigned)((T + kRouteWaves - 1) / kRouteWaves);
    if (f32)
        route_kernel<V, Key, float><<<grid, kRouteWaves * 64, 0, st>>>(static_cast<const float*>(logits), T, E, k, score, bias,
                                                                       groups, top_groups, group_best, renorm, scale, ids, weights);
    else
        route_kernel<V, Key, uint16_t><<<grid, kRouteWaves * 64, 0, st>>>(static_cast<const uint16_t*>(logits), T, E, k, score,
                                                                          bias, groups, top_groups, group_best, renorm, scale, ids,
                                                                          weights);
    return hipGetLastError();
}

template <class Key, class... A>
hipError_t by_experts(int E, A... a) {
    if (E <= 64) return run<1, Key>(a...);
    if (E <= 128) return run<2, Key>(a...);
    if (E <= 256) return run<4, Key>(a...);
    if (E <= 512) return run<8, Key>(a...);
    return run<16, Key>(a...);
}

}  // namespace

hipError_t launch_route(const void* logits, bool f32, int64_t T, int E, int k, int score, const float* bias, int groups,
                        int top_groups, int group_best, bool renorm, float scale, int32_t* ids, float* weights,
                        hipStream_t st) {
    const bool by_score = bias != nullptr || (groups > 1 && group_best > 1);
    if (by_score)
        return by_experts<double>(E, logits, f32, T, E, k, score, bias, groups, top_groups, group_best, renorm, scale, ids,
                                  weights, st);
    return by_experts<int>(E, logits, f32, T, E, k, score, bias, groups, top_groups, group_best, renorm, scale, ids, weights,
                             st);
}

}  // namespace qlin
