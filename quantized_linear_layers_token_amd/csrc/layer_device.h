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

// fl32(a / Q) by the reciprocal of Q and one correction: correctly rounded for
// every mantissa of a and both ranges (1 / a takes a division: the same two
// steps from the hardware's reciprocal miss the last bit of 33 mantissas).
template <bool FP8>
__device__ __forceinline__ float scale_of(float a) {
    constexpr float q = FP8 ? 448.0f : 127.0f, inv = 1.0f / q;
    const float r = a * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, r, a), inv, r);
}
template <bool FP8>
__device__ __forceinline__ Rounding rounding(float a) {
    const float q = FP8 ? 448.0f : 127.0f;
    const float pre = a < 0x1p-64f ? 0x1p64f : 1.0f;
    return Rounding{pre, a == 0.0f ? 0.0f : q * (1.0f / (a * pre))};
}
// Codes of four values.  Nothing saturates: |t * inv| exceeds Q by two units of
// f32 at most, which round to Q.  int8: adding 1.5 * 2^23 rounds to an integer,
// ties to even, and leaves it in the low byte.
template <bool FP8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
#pragma clang fp contract(off)
    if constexpr (FP8) {
        return e4m3_pack_hi(e4m3_pack_lo(a * inv, b * inv), c * inv, d * inv);
    } else {
        constexpr float magic = 12582912.0f;
        auto t = [inv](float v) {
#pragma clang fp contract(off)
            const float x = v * inv;
            return __float_as_uint(x + magic);
        };
        const uint32_t lo = __builtin_amdgcn_perm(t(b), t(a), 0x0C0C0400), hi = __builtin_amdgcn_perm(t(d), t(c), 0x04000C0C);
        return lo | hi;
    }
}
template <bool FP8>
__device__ __forceinline__ v2u codes8(float (&t)[8], Rounding r) {
    if (r.pre != 1.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= r.pre;
    }
    return v2u{codes4<FP8>(t[0], t[1], t[2], t[3], r.inv), codes4<FP8>(t[4], t[5], t[6], t[7], r.inv)};
}

__device__ __forceinline__ void widen8(const v4u& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(v[i]), f[2 * i + 1] = bf16_hi(v[i]);
}
// Two values rounded to bf16 (one instruction).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2bf{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ v4u narrow8(const float (&f)[8]) {
    return v4u{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// The larger of two magnitudes, NaN where one of them is: a row that holds a
// NaN has to get a NaN scale, since int8 codes have none (fmaxf drops it).
// One instruction for two of these.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

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
// The largest of magnitudes, by the order of their bits, in which NaN is above all.
template <int N>
__device__ __forceinline__ float lanes_absmax(float a) {
    uint32_t v = __float_as_uint(a);
    v = max(v, (uint32_t)dpp_i<0xB1>((int)v));
    v = max(v, (uint32_t)dpp_i<0x4E>((int)v));
    v = max(v, (uint32_t)dpp_i<0x141>((int)v));
    if constexpr (N >= 16) v = max(v, (uint32_t)dpp_i<0x140>((int)v));
    if constexpr (N >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    return __uint_as_float(v);
}

}  // namespace qlin
