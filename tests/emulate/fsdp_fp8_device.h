// What the 8-bit product takes from csrc/fsdp_fp8_device.h, for emulator.h.  Accesses that
// the kernel counts (16-byte stores of results, 16 scales at once) are told to the emulator.
#pragma once

#include "emulator.h"
#include "fsdp_fp8.h"

namespace fsdp {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
constexpr int kRsrcWord3 = 0;

struct Stored16 {
    char at[16];
    void operator=(const u32x4& x) {
        emu::other();
        memcpy(at, &x, 16);
    }
};
#define u32x4_any Stored16

inline uint32_t __float_as_uint(float x) { return __builtin_bit_cast(uint32_t, x); }
using std::min;

// bf16 to the nearest, ties to the even one; fp16 of whole numbers that it holds.
inline uint16_t bits16(int f, float x) {
    const uint32_t u = __float_as_uint(x);
    if (x != x) return f == FSDP_BF16 ? 0x7fc0 : 0x7e00;
    if (f == FSDP_BF16) return (uint16_t)((u + 0x7fff + (u >> 16 & 1)) >> 16);
    if (x == 0) return (uint16_t)(u >> 16);
    const int e = (int)(u >> 23 & 255) - 127;
    emu::check(e >= 0 && e <= 15 && (u & 0x1fff) == 0, "a result that fp16 does not hold");
    return (uint16_t)((u >> 16 & 0x8000) | (e + 15) << 10 | (u >> 13 & 0x3ff));
}
template <int F>
inline uint32_t pack2(float x, float y) { return bits16(F, x) | (uint32_t)bits16(F, y) << 16; }
template <int F>
inline void store1(void* base, int64_t i, float x) {
    if (F == FSDP_F32) ((float*)base)[i] = x;
    else ((uint16_t*)base)[i] = bits16(F, x);
}

// The n scales at p, n > 0, at most 16 of them, the rest zero; 16 are one load.
inline u32x4 scales16(const uint8_t* p, int n) {
    emu::check(n > 0, "scales behind the last block");
    n = n < 16 ? n : 16;
    emu::check(emu::readable(p, n), "scales out of range");
    if (n == 16) emu::other();
    u32x4 x = {0, 0, 0, 0};
    memcpy(&x, p, n);
    return x;
}

template <typename K, typename... Args>
inline void launch_lds(K kernel, dim3 grid, dim3 block, unsigned lds_bytes, hipStream_t, Args... args) {
    emu::check(lds_bytes <= 163840, "more LDS than there is");
    emu::launch(grid.x, block.x, [=]() { kernel(args...); });
}
template <typename K, typename... Args>
inline void launch(K kernel, dim3 grid, dim3 block, hipStream_t st, Args... args) { launch_lds(kernel, grid, block, 0u, st, args...); }

}  // namespace fsdp
