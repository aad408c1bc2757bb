// fsdp_mx4_device.h -- device primitives of the 4-bit microscaled blocks: the
// scale of a block, its codes, and loads at any address.  Not installed.
#pragma once

#include "fsdp_any.h"
#include "fsdp_mx4.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const uint32_t f = amax >> 23;
    return f == 255 ? 255u : (f < 2 ? 0u : f - 2);
}
// The factor 2^e of a scale byte; NaN for 255.
__device__ __forceinline__ float from_codes(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7fc00000u : byte << 23));
}

// Eight elements as they lie in memory: 16-bit pairs (the first in the low
// half) or fp32.
template <int F>
struct Raw8 {
    uint32_t w[F == FSDP_F32 ? 8 : 4];
};

// The largest magnitude so far, as a number that grows with it: the bits of a
// fp32 value, or those of two 16-bit values side by side.
template <int F>
__device__ __forceinline__ uint32_t max_mag(uint32_t a, const Raw8<F>& x) {
    if constexpr (F == FSDP_F32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) a = max(a, x.w[k] & 0x7fffffffu);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            a = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                       __builtin_bit_cast(u16x2, x.w[k] & 0x7fff7fffu)));
    }
    return a;
}
// The fp32 bits of what max_mag found.
template <int F>
__device__ __forceinline__ uint32_t mag_bits(uint32_t a) {
    if constexpr (F == FSDP_F32) return a;
    else return __float_as_uint(to_f32<F>(max(a & 0xffffu, a >> 16)));
}

// Eight elements of a block with scale byte s as eight codes, the first in the
// low nibble.  gfx950's conversion divides by the power of two and rounds to
// nearest even, codes above 6 to 6, two elements an instruction; it is not
// asked to divide by the subnormal 2^-127 (byte 0): there the elements are
// multiplied by 2^127, which is exact.  A block with byte 255 has codes 0.
template <int F>
__device__ __forceinline__ uint32_t codes8(const Raw8<F>& x, uint32_t s) {
    uint32_t w = 0;
    if (s == 0) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (F == FSDP_F32) v[k] = __uint_as_float(x.w[k]);
            else v[k] = to_f32<F>(k & 1 ? x.w[k / 2] >> 16 : x.w[k / 2] & 0xffffu);
            v[k] *= 0x1p127f;
        }
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
        return w;
    }
    const float f = __uint_as_float((s == 255 ? 127u : s) << 23);
    if constexpr (F == FSDP_F32) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[0]), __uint_as_float(x.w[1]), f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[2]), __uint_as_float(x.w[3]), f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[4]), __uint_as_float(x.w[5]), f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[6]), __uint_as_float(x.w[7]), f, 3);
    } else if constexpr (F == FSDP_F16) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, x.w[0]), f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, x.w[1]), f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, x.w[2]), f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, x.w[3]), f, 3);
    } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[0]), f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[1]), f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[2]), f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[3]), f, 3);
    }
    return s == 255 ? 0u : w;
}

// The largest of four neighbouring lanes' values, in all four of them.
__device__ __forceinline__ uint32_t max_of_four(uint32_t a) {
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
    return max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// Eight elements at p (any alignment).
template <int F>
__device__ __forceinline__ Raw8<F> load8_raw(const char* p) {
    Raw8<F> x;
#pragma unroll
    for (int j = 0; j < (F == FSDP_F32 ? 2 : 1); ++j) {
        const u32x4 a = *(const u32x4_any*)(p + 16 * j);
        x.w[4 * j] = a.x; x.w[4 * j + 1] = a.y; x.w[4 * j + 2] = a.z; x.w[4 * j + 3] = a.w;
    }
    return x;
}
// n elements at p where n < 8, the rest zero.  Behind the last one it is read
// again: loads under conditions of their own wait for each other.
template <int F>
__device__ __forceinline__ Raw8<F> load_upto8(const char* p, int64_t n) {
    if (n >= 8) return load8_raw<F>(p);
    Raw8<F> x{};
    if (n <= 0) return x;
    const int m = (int)n;
    if constexpr (F == FSDP_F32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x.w[k] = ((const uint32_t*)p)[k < m ? k : m - 1];
#pragma unroll
        for (int k = 1; k < 8; ++k) x.w[k] = k < m ? x.w[k] : 0u;
    } else {
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = ((const uint16_t*)p)[k < m ? k : m - 1];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x.w[k] = (2 * k < m ? e[2 * k] : 0u) | (2 * k + 1 < m ? e[2 * k + 1] << 16 : 0u);
    }
    return x;
}

// The n scales at p, n > 0, at most 16 of them, the rest zero.
__device__ __forceinline__ u32x4 scales16(const uint8_t* p, int n) {
    if (n >= 16) return *(const u32x4_any*)p;
    uint32_t e[16], x[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) e[j] = p[j < n ? j : n - 1];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j / 4] |= j < n ? e[j] << (8 * (j % 4)) : 0u;
    return u32x4{x[0], x[1], x[2], x[3]};
}

}  // namespace fsdp
