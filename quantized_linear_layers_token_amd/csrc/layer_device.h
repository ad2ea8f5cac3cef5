// Device helpers of the norm, rotary, cache and attention kernels.
#pragma once

#include "layer_internal.h"
#include "qlin_device.h"

namespace qlin {

// The dynamic rounding of a row (group, head) of f32 values with absmax a:
//   s = fl32(a / Q),  inv = fl32(Q * fl32(1 / a)),  code = round(fl32(t * inv))
// and, for a < 2^-64, where inv can exceed the f32 range, t and a scaled by
// 2^64 first.  inv is a reciprocal and a product, as an elementwise evaluation
// in torch has it (a number over a tensor is that there), so that codes equal
// those of a user's own quantizer in torch bit for bit; qlin_round.h divides
// once, which changes the last bit of inv at most.
struct Rounding {
    float pre, inv;
};
template <bool FP8>
__device__ __forceinline__ Rounding rounding(float a) {
    const float q = FP8 ? 448.0f : 127.0f;
    const float pre = a < 0x1p-64f ? 0x1p64f : 1.0f;
    return Rounding{pre, a == 0.0f ? 0.0f : q * (1.0f / (a * pre))};
}
template <bool FP8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, Rounding r) {
    if constexpr (FP8) {
        auto t = [r](float v) { return fminf(fmaxf((v * r.pre) * r.inv, -448.0f), 448.0f); };
        return e4m3_pack_hi(e4m3_pack_lo(t(a), t(b)), t(c), t(d));
    } else {
        auto t = [r](float v) {
            return (uint32_t)(uint8_t)(int8_t)(int)fminf(fmaxf(__builtin_rintf((v * r.pre) * r.inv), -127.0f), 127.0f);
        };
        return t(a) | (t(b) << 8) | (t(c) << 16) | (t(d) << 24);
    }
}
template <bool FP8>
__device__ __forceinline__ v2u codes8(const float (&t)[8], Rounding r) {
    return v2u{codes4<FP8>(t[0], t[1], t[2], t[3], r), codes4<FP8>(t[4], t[5], t[6], t[7], r)};
}

__device__ __forceinline__ void widen8(const v4u& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(v[i]), f[2 * i + 1] = bf16_hi(v[i]);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) { return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16); }
__device__ __forceinline__ v4u narrow8(const float (&f)[8]) {
    return v4u{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// Sum and maximum over runs of N = 8, 16 or 32 lanes; every lane gets the result.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
    v += dpp_f<0xB1>(v);
    v += dpp_f<0x4E>(v);
    v += dpp_f<0x141>(v);
    if constexpr (N >= 16) v += dpp_f<0x140>(v);
    if constexpr (N >= 32) v += __shfl_xor(v, 16);
    return v;
}
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
    v = fmaxf(v, dpp_f<0xB1>(v));
    v = fmaxf(v, dpp_f<0x4E>(v));
    v = fmaxf(v, dpp_f<0x141>(v));
    if constexpr (N >= 16) v = fmaxf(v, dpp_f<0x140>(v));
    if constexpr (N >= 32) v = fmaxf(v, __shfl_xor(v, 16));
    return v;
}

}  // namespace qlin
