// fsdp_fp8_device.h -- device primitives of the 8-bit blocks: the scale of a
// block and its codes.  Not installed.
#pragma once

#include "fsdp_fp8.h"
#include "fsdp_mx4_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef short s16x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block from the bits of its largest magnitude a: e + 127 for
// the smallest e >= -126 with a <= 448 * 2^e.  448 is 1.75 * 2^8, so that is a's
// exponent less 8, and one more where its significand passes 1.75.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax) {
    const int f = (int)(amax >> 23);
    const int s = f - 8 + ((amax & 0x7fffffu) > 0x600000u);
    return f == 255 ? 255u : (uint32_t)(s < 1 ? 1 : s);
}

// The largest of 16 lanes' values (a row of the wave), in all of them.
__device__ __forceinline__ uint32_t max_of_16(uint32_t a) {
    a = max_of_four(a);
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x141, 0xF, 0xF, true));    // halves of 8 mirrored
    return max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x140, 0xF, 0xF, true));  // the 16 mirrored
}

// Eight elements of a block with scale byte s (not 0) as eight codes, the first
// in the low byte.  gfx950's conversion divides by the power of two and rounds to
// the nearest, ties to even, two elements an instruction; nothing passes 448
// here.  A block with byte 255 has codes 0.
template <int F>
__device__ __forceinline__ u32x2 fp8_codes8(const Raw8<F>& x, uint32_t s) {
    const float f = __uint_as_float((s == 255 ? 127u : s) << 23);
    s16x2 w[2] = {s16x2{0, 0}, s16x2{0, 0}};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (F == FSDP_F32) {
            w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w[k], __uint_as_float(x.w[4 * k]),
                                                            __uint_as_float(x.w[4 * k + 1]), f, 0);
            w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w[k], __uint_as_float(x.w[4 * k + 2]),
                                                            __uint_as_float(x.w[4 * k + 3]), f, 1);
        } else if constexpr (F == FSDP_F16) {
            w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w[k], __builtin_bit_cast(f16x2, x.w[2 * k]), f, 0);
            w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w[k], __builtin_bit_cast(f16x2, x.w[2 * k + 1]), f, 1);
        } else {
            w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w[k], __builtin_bit_cast(bf16x2, x.w[2 * k]), f, 0);
            w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w[k], __builtin_bit_cast(bf16x2, x.w[2 * k + 1]), f, 1);
        }
    }
    return s == 255 ? u32x2{0, 0} : u32x2{__builtin_bit_cast(uint32_t, w[0]), __builtin_bit_cast(uint32_t, w[1])};
}

// Two values rounded to a 16-bit format side by side, the first in the low half.
template <int F>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if constexpr (F == FSDP_BF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
    else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)x, (_Float16)y});
}

}  // namespace fsdp
