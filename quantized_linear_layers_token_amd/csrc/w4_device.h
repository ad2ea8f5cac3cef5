// Device helpers of the 4-bit products.
#pragma once

#include "qlin_device.h"
#include "w4_internal.h"

namespace qlin {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// A pointer to global memory: loads through it stay global loads where the
// compiler cannot see where a pointer comes from.
template <class T> using Global = const __attribute__((address_space(1))) T*;

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

// The SUB = 128 / group scales of a row in one block, as they are packed.
template <int SUB>
struct W4Scales {
    uint32_t v[SUB == 4 ? 2 : 1];
    __device__ __forceinline__ void load(Global<uint16_t> p) {
        if constexpr (SUB == 1) {
            v[0] = *p;
        } else if constexpr (SUB == 2) {
            v[0] = *(Global<uint32_t>)p;
        } else {
            const v2u t = *(Global<v2u>)p;
            v[0] = t.x, v[1] = t.y;
        }
    }
    // the same through a descriptor (a buffer load: no address registers)
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t d, int lane_at, int block_at) {
        if constexpr (SUB == 1) {
            v[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(d, lane_at, block_at, 0);
        } else if constexpr (SUB == 2) {
            v[0] = __builtin_amdgcn_raw_buffer_load_b32(d, lane_at, block_at, 0);
        } else {
            const v2u t = __builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(d, lane_at, block_at, 0));
            v[0] = t.x, v[1] = t.y;
        }
    }
    __device__ __forceinline__ float at(int g) const {
        if constexpr (SUB == 1) return bf16_lo(v[0]);
        else return g & 1 ? bf16_hi(v[g >> 1]) : bf16_lo(v[g >> 1]);
    }
};
// The zero points of a row in one block: that of group g in byte g.
template <int SUB>
__device__ __forceinline__ uint32_t w4_zeros(Global<uint8_t> p) {
    if constexpr (SUB == 1) return *p;
    else if constexpr (SUB == 2) return *(Global<uint16_t>)p;
    else return *(Global<uint32_t>)p;
}

template <int SUB>
__device__ __forceinline__ uint32_t w4_zeros(__amdgpu_buffer_rsrc_t d, int lane_at, int block_at) {
    if constexpr (SUB == 1) return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(d, lane_at, block_at, 0);
    else if constexpr (SUB == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(d, lane_at, block_at, 0);
    else return __builtin_amdgcn_raw_buffer_load_b32(d, lane_at, block_at, 0);
}

// The same value, unpacked anew at every use: held unpacked for the whole
// block, the scales and zero points would take the registers of the sums.
__device__ __forceinline__ uint32_t again(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// silu(g) * u of the f32 sums.
__device__ __forceinline__ float swiglu_f32(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

}  // namespace qlin
