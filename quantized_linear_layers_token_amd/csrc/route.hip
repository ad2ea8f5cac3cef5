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
// of more than one) they are compared as they are.  Lane l holds the experts
// l, l + 64, ....  A round of the selection takes the wavefront maximum of
// 32-bit keys (the choices rounded to f32, or the logits, as integers in their
// order) and a ballot of its holders; only where several experts share the key
// are their f64 choices compared.  Bound by vector instructions from some
// thousand tokens on, below by the launch: 4096 tokens, 256 experts, sigmoid
// and bias, the best 4 of 8 groups, 8 of 256: 9.6 us (12.6 with f64 keys
// throughout); one token 2.6 us, an empty kernel 2.8.
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

// Keys: the bits of a float as an integer in the order of its values.  Below
// that of every expert that takes part: kMasked (an expert that is masked out
// comes after every other expert of the groups that stay), and below that kGone
// (experts of dropped groups, and those taken already).
constexpr int kGone = INT32_MIN, kMasked = INT32_MIN + 1;
__device__ __forceinline__ int key_of(float v) {
    const int b = __float_as_int(v + 0.0f);   // -0 equals 0
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
// A choice without NaN and infinities.
__device__ __forceinline__ double finite(double v) { return v >= -DBL_MAX ? fmin(v, DBL_MAX) : -DBL_MAX; }

// 1 / (1 + e^-l); 0 below l = -708, where e^-l nears the end of f64.
__device__ __forceinline__ double sigmoid(float l) {
    const double d = 1.0 + exp(-(double)fmaxf(l, -708.0f));
    double r = __builtin_amdgcn_rcp(d);       // two Newton steps: within a unit or two of the last place
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    return l < -708.0f ? 0.0 : r;
}

// The two largest of two lanes' two largest.
template <int CTRL>
__device__ __forceinline__ void merge_dpp(double& a, double& b) {
    const double oa = dpp_d<CTRL>(a), ob = dpp_d<CTRL>(b);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
}

// V: experts per lane.  SCORES: the choices are f64 values from the scores
// (else the logits).
template <int V, bool SCORES, class Logit>
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
        if (m == -INFINITY) m = 0.0f;    // every expert masked out: scores of zero
        double z = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[j] = exp((double)l[j] - (double)m);
            z += p[j];
        }
        total = wave_sum(z);
        if (total == 0.0) total = 1.0;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = sigmoid(l[j]);
    }

    int key[V];
    double c[SCORES ? V : 1];
    const double inv = 1.0 / total;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 64 + lane;
        if constexpr (SCORES) {
            double v = p[j] * inv;
            if (bias && e < E) v += (double)bias[e];
            c[j] = l[j] == -INFINITY ? -INFINITY : finite(v);   // masked out: below every choice
            // f32 rounding keeps the order; past its range every choice shares the last key
            key[j] = key_of((float)fmax(fmin(c[j], (double)FLT_MAX), -(double)FLT_MAX));
        } else {
            key[j] = key_of(l[j]);
        }
        if (l[j] == -INFINITY) key[j] = kMasked;
        if (e >= E) key[j] = kGone;
    }

    if (groups > 1) {
        const int size = E / groups;
#pragma unroll
        for (int j = 0; j < V; ++j) mine[j * 64 + lane] = SCORES ? c[SCORES ? j : 0] : (double)l[j];
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
        if (P > 1) merge_dpp<0xB1>(a, b);
        if (P > 2) merge_dpp<0x4E>(a, b);
        if (P > 4) merge_dpp<0x141>(a, b);
        if (P > 8) merge_dpp<0x140>(a, b);
        for (int d = 16; d < P; d <<= 1) {
            const double oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        // of the experts that take part: one alone is its group's worth, and a
        // group without any stays at -infinity, after every other
        const double worth = group_best == 2 && b != -INFINITY ? finite(a + b) : a;
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
            if (e < E && !((kept >> (of * P)) & 1)) key[j] = kGone;
        }
        __threadfence_block();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) mine[j * 64 + lane] = p[j];

    int chosen = 0;   // lane r: the token's choice r
    for (int r = 0; r < k; ++r) {
        int m = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = max(m, key[j]);
        m = wave_max(m);
        uint64_t held[V];
        int holders = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            held[j] = __ballot(key[j] == m);
            holders += __popcll(held[j]);
        }
        if constexpr (SCORES) {
            if (holders > 1 && m > kMasked) {   // (masked experts are equal)
                double best = -INFINITY;
#pragma unroll
                for (int j = 0; j < V; ++j) best = fmax(best, key[j] == m ? c[j] : -INFINITY);
                best = wave_max(best);
#pragma unroll
                for (int j = 0; j < V; ++j) held[j] = __ballot(key[j] == m && c[j] == best);
            }
        }
        int at = -1;   // the first holder
#pragma unroll
        for (int j = V - 1; j >= 0; --j)
            if (held[j]) at = j * 64 + __builtin_ctzll(held[j]);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j * 64 + lane == at) key[j] = kGone;
        if (lane == r) chosen = at;
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double w = lane < k ? mine[chosen] : 0.0;
    if (renorm) {
        const double s = wave_sum(w);
        w = s > 0.0 ? w / s : 0.0;
    } else if (score == 0) {
        w *= inv;
    }
    if (lane < k) {
        ids[t * k + lane] = chosen;
        weights[t * k + lane] = (float)(w * (double)scale);
    }
}

template <int V, bool SCORES>
hipError_t run(const void* logits, bool f32, int64_t T, int E, int k, int score, const float* bias, int groups,
               int top_groups, int group_best, bool renorm, float scale, int32_t* ids, float* weights, hipStream_t st) {
    const unsigned grid = (unsigned)((T + kRouteWaves - 1) / kRouteWaves);
    if (f32)
        route_kernel<V, SCORES, float><<<grid, kRouteWaves * 64, 0, st>>>(static_cast<const float*>(logits), T, E, k, score, bias,
                                                                       groups, top_groups, group_best, renorm, scale, ids, weights);
    else
        route_kernel<V, SCORES, uint16_t><<<grid, kRouteWaves * 64, 0, st>>>(static_cast<const uint16_t*>(logits), T, E, k, score,
                                                                          bias, groups, top_groups, group_best, renorm, scale, ids,
                                                                          weights);
    return hipGetLastError();
}

template <bool SCORES, class... A>
hipError_t by_experts(int E, A... a) {
    if (E <= 64) return run<1, SCORES>(a...);
    if (E <= 128) return run<2, SCORES>(a...);
    if (E <= 256) return run<4, SCORES>(a...);
    if (E <= 512) return run<8, SCORES>(a...);
    return run<16, SCORES>(a...);
}

}  // namespace

hipError_t launch_route(const void* logits, bool f32, int64_t T, int E, int k, int score, const float* bias, int groups,
                        int top_groups, int group_best, bool renorm, float scale, int32_t* ids, float* weights,
                        hipStream_t st) {
    const bool by_score = bias != nullptr || (groups > 1 && group_best > 1);
    if (by_score)
        return by_experts<true>(E, logits, f32, T, E, k, score, bias, groups, top_groups, group_best, renorm, scale, ids,
                                  weights, st);
    return by_experts<false>(E, logits, f32, T, E, k, score, bias, groups, top_groups, group_best, renorm, scale, ids, weights,
                             st);
}

}  // namespace qlin
