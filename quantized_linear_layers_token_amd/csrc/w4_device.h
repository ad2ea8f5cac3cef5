// Device helpers of the 4-bit products.
#pragma once

#include "qlin_device.h"
#include "w4_internal.h"

namespace qlin {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// Eight codes of a packed dword as bf16, in the order of their inputs: byte b
// holds input b in its low half and input 4 + b in its high half.  A byte
// 0x00..0x0F read as E4M3 is code * 2^-9 (subnormals below 8, the first
// binade from 8 on: both steps of 2^-9), so with a scale of 2^9 the
// conversion gives the code itself, exactly.  Seven vector instructions for
// eight codes (31 cycles of a SIMD per wavefront measured; shift, mask and or
// into the bf16 mantissa takes eight, 33 cycles, and leaves 16 + code, whose
// correction costs three times the f32 rounding error).
__device__ __forceinline__ v8bf w4_codes(uint32_t w) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return v8bf{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 16 tokens x 32 inputs times 32 inputs x 16 weight rows.  Lane l holds token
// (weight row) l % 16 and inputs 8 (l / 16) .. + 7 of both operands; the
// result's column l % 16 is the weight row, its rows 4 (l / 16) + i the tokens.
__device__ __forceinline__ v4f mfma_bf16(v8bf a, v8bf b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v8bf bf16_const(float v) {
    const __bf16 h = (__bf16)v;
    return v8bf{h, h, h, h, h, h, h, h};
}

// The SUB = 128 / group scales (zero points) of a row in one block.
template <int SUB>
__device__ __forceinline__ void w4_scales(const uint16_t* p, float (&s)[SUB]) {
    if constexpr (SUB == 1) {
        s[0] = bf16_lo(*p);
    } else if constexpr (SUB == 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
        s[0] = bf16_lo(v), s[1] = bf16_hi(v);
    } else {
        const v2u v = *reinterpret_cast<const v2u*>(p);
        s[0] = bf16_lo(v.x), s[1] = bf16_hi(v.x), s[2] = bf16_lo(v.y), s[3] = bf16_hi(v.y);
    }
}
template <int SUB>
__device__ __forceinline__ void w4_minus_zeros(const uint8_t* p, float (&z)[SUB]) {
    uint32_t v;
    if constexpr (SUB == 1) v = *p;
    else if constexpr (SUB == 2) v = *reinterpret_cast<const uint16_t*>(p);
    else v = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < SUB; ++i) z[i] = -(float)((v >> (8 * i)) & 255u);
}

// silu(g) * u of the f32 sums, rounded once.
__device__ __forceinline__ uint16_t swiglu_f32(float g, float u) { return f32_to_bf16(g / (1.0f + __expf(-g)) * u); }

}  // namespace qlin
