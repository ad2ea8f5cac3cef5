// Queries, keys and values between the q/k/v projection and attention: norm
// and rotation of the heads, keys and values rounded into the paged cache (one
// launch for the three), and cache rows read back.
//
// A workgroup takes one token: the cosines and sines of its position are
// formed once, by dims / 2 threads, and shared by all of its heads through LDS.
// LANES lanes hold a head, eight channels (16 bytes) each, so that the sum of
// squares and the absmax are reductions within 8, 16 or 32 lanes and the other
// channel of a pair is in the lane's own registers (neighbours) or comes from
// one other lane (halves).
#include <type_traits>

#include "layer_device.h"

namespace qlin {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;   // heads of each thread whose loads are under way together

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

template <int LANES, int KIND, bool ROTATE, bool NEIGHBOURS>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsCall a) {
    __shared__ float2 turns[QLIN_MAX_HEAD_DIM / 2];
    constexpr int kPer = kThreads / LANES;   // heads that the workgroup takes at once
    const int64_t t = blockIdx.x;
    const int c = threadIdx.x % LANES, first = threadIdx.x / LANES;
    const int chunks = a.dim / 8;
    const bool mine = c < chunks;
    const int64_t slots = a.cache.pages * a.cache.page_size;
    const int slot = a.kv_heads ? a.slots[t] : -1;
    const bool kept = slot >= 0 && slot < slots;
    // a token that is not kept has no keys and values to do
    const int all = a.heads + (kept ? 2 * a.kv_heads : 0);
    const int page = kept ? slot / a.cache.page_size : 0, place = kept ? slot % a.cache.page_size : 0;
    const int half = a.rope.dims / 16;       // chunks of half of the rotated channels
    const uint16_t *q = a.q + t * a.q_stride, *k = a.k + t * a.k_stride, *v = a.v + t * a.v_stride;

    for (int base = 0; base == 0 || base < all; base += kAhead * kPer) {
        v4u raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = base + u * kPer + first;
            raw[u] = v4u{0, 0, 0, 0};
            if (mine && h < all) {
                const uint16_t* p = h < a.heads ? q + h * a.dim
                                  : h < a.heads + a.kv_heads ? k + (h - a.heads) * a.dim
                                                             : v + (h - a.heads - a.kv_heads) * a.dim;
                raw[u] = *reinterpret_cast<const v4u*>(p + 8 * c);
            }
        }
        if constexpr (ROTATE) {
            if (base == 0) {
                if (threadIdx.x < a.rope.dims / 2)
                    turns[threadIdx.x] = turn(a.positions[t], a.rope.frequencies[threadIdx.x], a.rope.strength);
                __syncthreads();
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = base + u * kPer + first;
            if (base + u * kPer >= all) break;      // the same for the whole workgroup
            const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
            const uint16_t* gamma = is_v ? nullptr : is_q ? a.q_gamma : a.k_gamma;
            float f[8];
            widen8(raw[u], f);
            float other[8];   // halves: the other channels of the lane's pairs
            bool low = false, turned = false;
            if constexpr (ROTATE && !NEIGHBOURS) {
                low = c < half;
                turned = c < 2 * half && !is_v;
                const int lane = threadIdx.x % kWave;
                const int from = turned ? (low ? lane + half : lane - half) : lane;
                v4u o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = __shfl(raw[u][i], from);
                widen8(o, other);
            }
            if (a.q_gamma || a.k_gamma) {
                float squares = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) squares = __builtin_fmaf(f[i], f[i], squares);
                squares = lanes_sum<LANES>(squares);
                if (gamma && mine) {
                    const float d = 1.0f / sqrtf(squares / (float)a.dim + a.eps);
                    float w[8];
                    widen8(*reinterpret_cast<const v4u*>(gamma + 8 * c), w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = f[i] * w[i] * d;
                    if constexpr (ROTATE && !NEIGHBOURS) {
                        if (turned) {
                            widen8(*reinterpret_cast<const v4u*>(gamma + 8 * (low ? c + half : c - half)), w);
#pragma unroll
                            for (int i = 0; i < 8; ++i) other[i] = other[i] * w[i] * d;
                        }
                    }
                }
            }
            if constexpr (ROTATE && !NEIGHBOURS) {
                if (turned) {
                    const float2* w = turns + 8 * (low ? c : c - half);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = f[i] * w[i].x + (low ? -other[i] : other[i]) * w[i].y;
                }
            }
            if constexpr (ROTATE && NEIGHBOURS) {
                if (c < 2 * half && !is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 w = turns[4 * c + i];
                        const float x = f[2 * i], y = f[2 * i + 1];
                        f[2 * i] = x * w.x - y * w.y;
                        f[2 * i + 1] = y * w.x + x * w.y;
                    }
                }
            }
            float amax = 0.0f;
            if constexpr (KIND != QLIN_CACHE_BF16) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
                amax = lanes_max<LANES>(amax);
            }
            if (!mine || h >= all) continue;
            if (is_q) {
                *reinterpret_cast<v4u*>(a.q_out + t * a.q_out_stride + h * a.dim + 8 * c) = narrow8(f);
                continue;
            }
            const int head = h - a.heads - (is_v ? a.kv_heads : 0);
            const int64_t row = ((int64_t)page * a.kv_heads + head) * a.cache.page_size + place;
            void* codes = is_v ? a.cache.v : a.cache.k;
            if constexpr (KIND == QLIN_CACHE_BF16) {
                *reinterpret_cast<v4u*>(static_cast<uint16_t*>(codes) + row * a.dim + 8 * c) = narrow8(f);
            } else {
                constexpr bool kFp8 = KIND == QLIN_CACHE_FP8;
                *reinterpret_cast<v2u*>(static_cast<uint8_t*>(codes) + row * a.dim + 8 * c) = codes8<kFp8>(f, rounding<kFp8>(amax));
                if (c == 0) (is_v ? a.cache.v_scale : a.cache.k_scale)[row] = amax / (kFp8 ? 448.0f : 127.0f);
            }
        }
    }
}

// A workgroup takes `rows` rows of the call; a thread 16 channels of one head
// of a row, keys and values alike.
template <int KIND>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(qlin_kv_cache a, const int* __restrict__ slots, int64_t n, int rows,
                                                              uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
    const unsigned parts = a.dim / 16, per_row = a.kv_heads * parts;
    const int64_t first = (int64_t)blockIdx.x * rows;
    const int64_t total = a.pages * a.page_size;
    for (unsigned i = threadIdx.x; i < rows * per_row; i += kThreads) {
        const unsigned r = i / per_row, rest = i - r * per_row, head = rest / parts, part = rest - head * parts;
        const int64_t at = first + r;
        if (at >= n) break;
        const int slot = slots[at];
        if (slot < 0 || slot >= total) continue;
        const int page = slot / a.page_size, place = slot % a.page_size;
        const int64_t row = ((int64_t)page * a.kv_heads + head) * a.page_size + place;
        const int64_t from = row * a.dim + 16 * part, to = (at * a.kv_heads + head) * a.dim + 16 * part;
        if constexpr (KIND == QLIN_CACHE_BF16) {
            const v4u* ks = reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(a.k) + from);
            const v4u* vs = reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(a.v) + from);
            const v4u k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
            v4u *kt = reinterpret_cast<v4u*>(k + to), *vt = reinterpret_cast<v4u*>(v + to);
            kt[0] = k0, kt[1] = k1, vt[0] = v0, vt[1] = v1;
        } else {
            const v4u kw = *reinterpret_cast<const v4u*>(static_cast<const uint8_t*>(a.k) + from);
            const v4u vw = *reinterpret_cast<const v4u*>(static_cast<const uint8_t*>(a.v) + from);
            const float ks = a.k_scale[row], vs = a.v_scale[row];
            auto widen = [](const v4u& w, float s, uint16_t* to) {
                float f[8];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t d = w[2 * half + i];
                        if constexpr (KIND == QLIN_CACHE_FP8) {
                            const v2f lo = e4m3_unpack2<false>(d), hi = e4m3_unpack2<true>(d);
                            f[4 * i] = lo.x * s, f[4 * i + 1] = lo.y * s, f[4 * i + 2] = hi.x * s, f[4 * i + 3] = hi.y * s;
                        } else {
#pragma unroll
                            for (int b = 0; b < 4; ++b) f[4 * i + b] = (float)(int8_t)(d >> (8 * b)) * s;
                        }
                    }
                    reinterpret_cast<v4u*>(to)[half] = narrow8(f);
                }
            };
            widen(kw, ks, k + to);
            widen(vw, vs, v + to);
        }
    }
}

template <int LANES, int KIND>
void launch_lanes(const HeadsCall& c, hipStream_t st) {
    const dim3 grid((unsigned)c.T), block(kThreads);
    if (!c.rope.frequencies) hipLaunchKernelGGL((heads_kernel<LANES, KIND, false, false>), grid, block, 0, st, c);
    else if (c.rope.interleaved) hipLaunchKernelGGL((heads_kernel<LANES, KIND, true, true>), grid, block, 0, st, c);
    else hipLaunchKernelGGL((heads_kernel<LANES, KIND, true, false>), grid, block, 0, st, c);
}
template <int KIND>
void launch_kind(const HeadsCall& c, hipStream_t st) {
    if (c.dim <= 64) launch_lanes<8, KIND>(c, st);
    else if (c.dim <= 128) launch_lanes<16, KIND>(c, st);
    else launch_lanes<32, KIND>(c, st);
}

}  // namespace

hipError_t launch_heads(const HeadsCall& c, hipStream_t st) {
    if (c.kv_heads == 0 || c.cache.kind == QLIN_CACHE_BF16) launch_kind<QLIN_CACHE_BF16>(c, st);
    else if (c.cache.kind == QLIN_CACHE_INT8) launch_kind<QLIN_CACHE_INT8>(c, st);
    else launch_kind<QLIN_CACHE_FP8>(c, st);
    return hipGetLastError();
}

hipError_t launch_cache_read(const qlin_kv_cache& cache, const int* slots, int64_t n, uint16_t* k, uint16_t* v, hipStream_t st) {
    const int per_row = cache.kv_heads * (cache.dim / 16);
    const int rows = per_row >= 512 ? 1 : 512 / per_row;
    const dim3 grid((unsigned)((n + rows - 1) / rows)), block(kThreads);
    if (cache.kind == QLIN_CACHE_BF16) hipLaunchKernelGGL(cache_read_kernel<QLIN_CACHE_BF16>, grid, block, 0, st, cache, slots, n, rows, k, v);
    else if (cache.kind == QLIN_CACHE_INT8) hipLaunchKernelGGL(cache_read_kernel<QLIN_CACHE_INT8>, grid, block, 0, st, cache, slots, n, rows, k, v);
    else hipLaunchKernelGGL(cache_read_kernel<QLIN_CACHE_FP8>, grid, block, 0, st, cache, slots, n, rows, k, v);
    return hipGetLastError();
}

}  // namespace qlin
