// Queries, keys and values between the q/k/v projection and attention: norm
// and rotation of the heads, keys and values rounded into the paged cache (one
// launch for the three), and cache rows read back.
//
// A workgroup takes one token, or as many as its threads hold at once where the
// heads are few: the cosines and sines of a position are formed once, by
// dims / 2 threads, and shared by all of its heads through LDS.
// LANES lanes hold a head, eight channels each, so that the sum of squares and
// the absmax are reductions within 8, 16 or 32 lanes.  A lane's channels are
// two runs of four: both channels of each of its pairs, so that nothing is
// exchanged for the rotation, and its cosines and sines are the same for every
// head of the token and stay in registers.
//
// Bound by memory for many tokens: 4096 tokens of 32 heads of 128, normalised
// and rotated, 13.7 us (67 MB, 4.9 TB/s; without the norm 11.9); with 8 key and
// value heads rounded to int8 as well 20 us (92 MB).  With eight channels of a
// lane side by side, the partner's exchanged by LDS permutes and normalised a
// second time, and two more divisions to a head, vector instructions bounded
// it (17.7 and 29 us).  Rows read back: 65536 of 8 heads of 128 in E4M3, 77 us
// (407 MB, 5.3 TB/s); sixteen channels to a lane, whose stores leave half a line
// each, took 94.
#include <type_traits>

#include "layer_device.h"
#include "layer_forms.h"

namespace qlin {

namespace {

constexpr int kThreads = kHeadsThreads;
constexpr int kAhead = 3;   // heads of each thread whose loads are under way together

// Cosine and sine of position * frequency, times strength.  The product is
// reduced in f64 by multiples of 2 pi in two parts (the first exact to 53
// bits, the second what that leaves of 2 pi): |r| <= pi, off by less than one
// unit of f32 for any int32 position.
__device__ __forceinline__ float2 turn(int position, double frequency, float strength) {
    const double angle = (double)position * frequency;
    const double k = __builtin_rint(angle * 0.15915494309189535);
    double r = __builtin_fma(-k, 6.283185307179586, angle);
    r = __builtin_fma(-k, 2.4492935982947064e-16, r);
    float s, c;
    sincosf((float)r, &s, &c);
    return make_float2(c * strength, s * strength);
}

// TOKENS: those of a workgroup; more than one only where a token's heads take
// at most kThreads / TOKENS threads.
template <int LANES, int KIND, bool ROTATE, bool NEIGHBOURS, int TOKENS>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsCall a) {
    extern __shared__ float2 turns[];        // [TOKENS][dims / 2]
    constexpr int kPer = kThreads / LANES / TOKENS;   // heads of a token that the workgroup takes at once
    static_assert(kPer > 0, "a token has a head");
    const int c = threadIdx.x % LANES, first = threadIdx.x / LANES % kPer;
    const int of = TOKENS > 1 ? threadIdx.x / LANES / kPer : 0;   // the thread's token
    const int64_t t = (int64_t)blockIdx.x * TOKENS + of;
    const bool mine = c < a.dim / 8 && (TOKENS == 1 || t < a.T);
    // the lane's channels: lo .. lo + 3 and hi .. hi + 3
    const int pairs = ROTATE ? a.rope.dims / 2 : 0;
    int lo = 8 * c, hi = 8 * c + 4;
    bool turned = ROTATE && 8 * c < 2 * pairs;
    if constexpr (ROTATE && !NEIGHBOURS) {
        if (turned) lo = 4 * c, hi = 4 * c + pairs;
    }
    const int all = a.heads + 2 * a.kv_heads;
    const uint16_t *q = a.q + t * a.q_stride, *k = a.k + t * a.k_stride, *v = a.v + t * a.v_stride;
    const v2u none = v2u{0, 0};
    v2u gamma[2][2] = {{none, none}, {none, none}};   // of queries and keys
    const bool normed = a.q_gamma || a.k_gamma;
    if (normed && mine) {
        if (a.q_gamma) gamma[0][0] = *reinterpret_cast<const v2u*>(a.q_gamma + lo), gamma[0][1] = *reinterpret_cast<const v2u*>(a.q_gamma + hi);
        if (a.k_gamma) gamma[1][0] = *reinterpret_cast<const v2u*>(a.k_gamma + lo), gamma[1][1] = *reinterpret_cast<const v2u*>(a.k_gamma + hi);
    }
    const int slot = a.kv_heads && (TOKENS == 1 || t < a.T) ? a.slots[t] : -1;
    int64_t row0 = -1;    // row of the cache of the token's first head
    float2 w[4];

    for (int base = 0; base < all; base += kAhead * kPer) {
        v2u raw[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = base + u * kPer + first;
            raw[u][0] = raw[u][1] = none;
            if (mine && h < all) {
                const uint16_t* p = h < a.heads ? q + h * a.dim
                                  : h < a.heads + a.kv_heads ? k + (h - a.heads) * a.dim
                                                             : v + (h - a.heads - a.kv_heads) * a.dim;
                raw[u][0] = *reinterpret_cast<const v2u*>(p + lo);
                raw[u][1] = *reinterpret_cast<const v2u*>(p + hi);
            }
        }
        if (base == 0) {
            if constexpr (ROTATE) {
                if constexpr (TOKENS == 1) {
                    if (threadIdx.x < pairs) turns[threadIdx.x] = turn(a.positions[t], a.rope.frequencies[threadIdx.x], a.rope.strength);
                } else {
                    for (int i = threadIdx.x; i < TOKENS * pairs; i += kThreads) {
                        const int64_t token = (int64_t)blockIdx.x * TOKENS + i / pairs;
                        if (token < a.T) turns[i] = turn(a.positions[token], a.rope.frequencies[i % pairs], a.rope.strength);
                    }
                }
                __syncthreads();
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = turns[of * pairs + 4 * c + i];
                }
            }
            if (slot >= 0 && slot < a.cache.pages * a.cache.page_size)
                row0 = (int64_t)(slot / a.cache.page_size) * a.kv_heads * a.cache.page_size + slot % a.cache.page_size;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = base + u * kPer + first;
            if (base + u * kPer >= all) break;      // the same for the whole workgroup
            const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(raw[u][i / 2][i % 2]), f[2 * i + 1] = bf16_hi(raw[u][i / 2][i % 2]);
            float d = 1.0f;   // what remains to be multiplied
            if (normed) {
                float squares = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) squares = __builtin_fmaf(f[i], f[i], squares);
                squares = lanes_sum<LANES>(squares);
                if (!is_v && (is_q ? a.q_gamma : a.k_gamma)) {
                    d = __builtin_amdgcn_rsqf(__builtin_fmaf(squares, a.inv_dim, a.eps));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t g = is_q ? gamma[0][i / 2][i % 2] : gamma[1][i / 2][i % 2];
                        f[2 * i] *= bf16_lo(g), f[2 * i + 1] *= bf16_hi(g);
                    }
                }
            }
            if constexpr (ROTATE) {
                if (turned && !is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = NEIGHBOURS ? 2 * i : i, n = NEIGHBOURS ? 2 * i + 1 : i + 4;
                        const float x = f[m], y = f[n];
                        f[m] = x * w[i].x - y * w[i].y;
                        f[n] = y * w[i].x + x * w[i].y;
                    }
                }
            }
            float amax = 0.0f;
            if constexpr (KIND != QLIN_CACHE_BF16) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = larger(amax, fabsf(f[i]));
                amax = lanes_absmax<LANES>(amax);
            }
            if (!mine || h >= all) continue;
            const int head = is_q ? h : h - a.heads - (is_v ? a.kv_heads : 0);
            if (is_q || KIND == QLIN_CACHE_BF16) {
                if (!is_q && row0 < 0) continue;
                uint16_t* to = is_q ? a.q_out + t * a.q_out_stride + head * a.dim
                                    : static_cast<uint16_t*>(is_v ? a.cache.v : a.cache.k) + (row0 + (int64_t)head * a.cache.page_size) * a.dim;
                if (normed) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= d;
                }
                *reinterpret_cast<v2u*>(to + lo) = v2u{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])};
                *reinterpret_cast<v2u*>(to + hi) = v2u{bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
            } else if (row0 >= 0) {
                // as in the norm, the codes are those of f: d is left to the scale
                constexpr bool kFp8 = KIND == QLIN_CACHE_FP8;
                const int64_t row = row0 + (int64_t)head * a.cache.page_size;
                uint8_t* to = static_cast<uint8_t*>(is_v ? a.cache.v : a.cache.k) + row * a.dim;
                const v2u codes = codes8<kFp8>(f, rounding<kFp8>(amax));
                *reinterpret_cast<uint32_t*>(to + lo) = codes.x;
                *reinterpret_cast<uint32_t*>(to + hi) = codes.y;
                if (c == 0) (is_v ? a.cache.v_scale : a.cache.k_scale)[row] = scale_of<kFp8>(amax * d);
            }
        }
    }
}

constexpr int kReadAhead = 4;   // rows of a thread whose loads are under way together

// Eight codes times their scale, rounded to bf16.
template <int KIND>
__device__ __forceinline__ v4u widen_codes(uint32_t a, uint32_t b, float s) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t d = i ? b : a;
        if constexpr (KIND == QLIN_CACHE_FP8) {
            const v2f lo = e4m3_unpack2<false>(d), hi = e4m3_unpack2<true>(d);
            f[4 * i] = lo.x * s, f[4 * i + 1] = lo.y * s, f[4 * i + 2] = hi.x * s, f[4 * i + 3] = hi.y * s;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * i + j] = (float)(int8_t)(d >> (8 * j)) * s;
        }
    }
    return narrow8(f);
}

// A thread takes eight channels of a head, of its keys and its values, in every
// `step`-th row of the workgroup's.
template <int KIND>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(qlin_kv_cache a, const int* __restrict__ slots, int64_t n, int rows,
                                                              uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
    constexpr int kBytes = KIND == QLIN_CACHE_BF16 ? 16 : 8;   // of eight channels
    const int parts = a.dim / 8, per_row = a.kv_heads * parts;
    const int across = per_row < kThreads ? per_row : kThreads, step = kThreads / across;
    const int r0 = threadIdx.x / across;
    const int64_t first = (int64_t)blockIdx.x * rows, last = first + rows < n ? first + rows : n;
    const int total = (int)(a.pages * a.page_size);
    if (r0 >= step) return;
    for (int i = threadIdx.x - r0 * across; i < per_row; i += across) {
        const int head = i / parts, part = i - head * parts;
        for (int64_t at = first + r0; at < last; at += kReadAhead * step) {
            v4u kw[kReadAhead], vw[kReadAhead];
            float ks[kReadAhead], vs[kReadAhead];
            bool live[kReadAhead];
            int slot[kReadAhead];
#pragma unroll
            for (int u = 0; u < kReadAhead; ++u) slot[u] = at + u * step < last ? slots[at + u * step] : -1;
#pragma unroll
            for (int u = 0; u < kReadAhead; ++u) {
                live[u] = slot[u] >= 0 && slot[u] < total;
                if (!live[u]) continue;
                const int page = slot[u] / a.page_size, place = slot[u] - page * a.page_size;
                const int64_t row = ((int64_t)page * a.kv_heads + head) * a.page_size + place;
                const int64_t from = (row * parts + part) * kBytes;
                if constexpr (KIND == QLIN_CACHE_BF16) {
                    kw[u] = *reinterpret_cast<const v4u*>(static_cast<const uint8_t*>(a.k) + from);
                    vw[u] = *reinterpret_cast<const v4u*>(static_cast<const uint8_t*>(a.v) + from);
                } else {
                    const v2u x = *reinterpret_cast<const v2u*>(static_cast<const uint8_t*>(a.k) + from);
                    const v2u y = *reinterpret_cast<const v2u*>(static_cast<const uint8_t*>(a.v) + from);
                    kw[u].x = x.x, kw[u].y = x.y, vw[u].x = y.x, vw[u].y = y.y;
                    ks[u] = a.k_scale[row], vs[u] = a.v_scale[row];
                }
            }
#pragma unroll
            for (int u = 0; u < kReadAhead; ++u) {
                if (!live[u]) continue;
                const int64_t to = (at + u * step) * per_row + i;
                if constexpr (KIND != QLIN_CACHE_BF16) {
                    kw[u] = widen_codes<KIND>(kw[u].x, kw[u].y, ks[u]);
                    vw[u] = widen_codes<KIND>(vw[u].x, vw[u].y, vs[u]);
                }
                __builtin_nontemporal_store(kw[u], reinterpret_cast<v4u*>(k) + to);
                __builtin_nontemporal_store(vw[u], reinterpret_cast<v4u*>(v) + to);
            }
        }
    }
}

template <int LANES, int KIND, bool ROTATE, bool NEIGHBOURS>
void launch_form(const HeadsCall& c, hipStream_t st) {
    constexpr bool kAlone = ROTATE && KIND == QLIN_CACHE_BF16;
    auto go = [&](auto of) {
        constexpr int kTokens = decltype(of)::value;
        const size_t lds = ROTATE ? (size_t)kTokens * (c.rope.dims / 2) * sizeof(float2) : 0;
        hipLaunchKernelGGL((heads_kernel<LANES, KIND, ROTATE, NEIGHBOURS, kTokens>), dim3((unsigned)((c.T + kTokens - 1) / kTokens)), dim3(kThreads), lds, st,
                           c);
    };
    const int tokens = heads_tokens(LANES, c.heads + 2 * c.kv_heads, c.T);
    if constexpr (heads_fit(16, LANES, kAlone)) {
        if (tokens == 16) return go(std::integral_constant<int, 16>{});
    }
    if constexpr (heads_fit(4, LANES, kAlone)) {
        if (tokens == 4) return go(std::integral_constant<int, 4>{});
    }
    go(std::integral_constant<int, 1>{});
}
template <int LANES, int KIND>
void launch_lanes(const HeadsCall& c, hipStream_t st) {
    if (!c.rope.frequencies) launch_form<LANES, KIND, false, false>(c, st);
    else if (c.rope.interleaved) launch_form<LANES, KIND, true, true>(c, st);
    else launch_form<LANES, KIND, true, false>(c, st);
}
template <int KIND>
void launch_kind(const HeadsCall& c, hipStream_t st) {
    switch (heads_lanes(c.dim)) {
        case 8: return launch_lanes<8, KIND>(c, st);
        case 16: return launch_lanes<16, KIND>(c, st);
        default: launch_lanes<32, KIND>(c, st);
    }
}

}  // namespace

// A launch holds 2^32 threads: many tokens take several.
hipError_t launch_heads(const HeadsCall& c, hipStream_t st) {
    constexpr int64_t kTokens = int64_t(1) << 23;
    for (int64_t t = 0; t < c.T; t += kTokens) {
        HeadsCall part = c;
        part.T = c.T - t < kTokens ? c.T - t : kTokens;
        if (c.heads) part.q += t * c.q_stride, part.q_out += t * c.q_out_stride;
        if (c.kv_heads) part.k += t * c.k_stride, part.v += t * c.v_stride, part.slots += t;
        if (c.positions) part.positions += t;
        if (c.kv_heads == 0 || c.cache.kind == QLIN_CACHE_BF16) launch_kind<QLIN_CACHE_BF16>(part, st);
        else if (c.cache.kind == QLIN_CACHE_INT8) launch_kind<QLIN_CACHE_INT8>(part, st);
        else launch_kind<QLIN_CACHE_FP8>(part, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_cache_read(const qlin_kv_cache& cache, const int* slots, int64_t n, uint16_t* k, uint16_t* v, hipStream_t st) {
    const int per_row = cache.kv_heads * (cache.dim / 8), step = per_row < kThreads ? kThreads / per_row : 1;
    const int rows = kReadAhead * step;
    const dim3 grid((unsigned)((n + rows - 1) / rows)), block(kThreads);
    if (cache.kind == QLIN_CACHE_BF16) hipLaunchKernelGGL(cache_read_kernel<QLIN_CACHE_BF16>, grid, block, 0, st, cache, slots, n, rows, k, v);
    else if (cache.kind == QLIN_CACHE_INT8) hipLaunchKernelGGL(cache_read_kernel<QLIN_CACHE_INT8>, grid, block, 0, st, cache, slots, n, rows, k, v);
    else hipLaunchKernelGGL(cache_read_kernel<QLIN_CACHE_FP8>, grid, block, 0, st, cache, slots, n, rows, k, v);
    return hipGetLastError();
}

}  // namespace qlin
