// fsdp_any.h -- device primitives for buffers off the 16-byte grid (a shard of an
// odd size starts every rank's block off it): 8 consecutive elements a lane
// through 16-byte accesses at any address.  Not installed.
#pragma once

#include "fsdp_device.h"

#pragma clang fp contract(off)

namespace fsdp {

// 16 bytes at any address (global accesses need no alignment on this target;
// an address off the 16-byte grid costs a second cache line now and then).
typedef u32x4 u32x4_any __attribute__((aligned(1)));

// 16 bytes at p, with the non-temporal hint or without.
template <bool NT>
__device__ __forceinline__ u32x4 ld_any(const char* p) {
    if constexpr (NT) return __builtin_nontemporal_load((const u32x4_any*)p);
    else return *(const u32x4_any*)p;
}

// 8 consecutive elements of format F at p, at any address, with the non-temporal hint.
template <int F>
__device__ __forceinline__ void load8_any(const char* p, float (&x)[8]) {
    const u32x4 a = ld_any<true>(p);
    uint32_t w[8] = {a.x, a.y, a.z, a.w};
    if constexpr (F == FSDP_F32) {
        const u32x4 b = ld_any<true>(p + 16);
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (F == FSDP_F32) x[k] = __uint_as_float(w[k]);
        else x[k] = to_f32<F>(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
    }
}

// The fold of reduce8 over blocks at any address, four ranks' loads at a time.  What
// a run-time world leaves behind them is loaded and folded one rank after another:
// for N = 3 that is every rank (4.2 TB/s in the norm over units, against 5.5 with
// N = 8 on the 16-byte grid).
template <int NW, int GF, bool FP32R, typename GP>
__device__ __forceinline__ void reduce8_any(const GP& gp, int world, int64_t vi, float (&acc)[8]) {
    constexpr int kBytes = GF == FSDP_F32 ? 32 : 16;
    const int n = NW > 0 ? NW : world;
    load8_any<GF>((const char*)gp(0) + vi * kBytes, acc);
    int q = 1;
    for (; q + 4 <= n; q += 4) {
        float x[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) load8_any<GF>((const char*)gp(q + j) + vi * kBytes, x[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fold<NW, GF, FP32R>(acc[k], x[j][k]);
    }
    for (; q < n; ++q) {
        float x[8];
        load8_any<GF>((const char*)gp(q) + vi * kBytes, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fold<NW, GF, FP32R>(acc[k], x[k]);
    }
}

template <int F>
__device__ __forceinline__ void store8_any(char* p, const float (&x)[8]) {
    if constexpr (F == FSDP_F32) {
        u32x4 a, b;
        a.x = __float_as_uint(x[0]); a.y = __float_as_uint(x[1]);
        a.z = __float_as_uint(x[2]); a.w = __float_as_uint(x[3]);
        b.x = __float_as_uint(x[4]); b.y = __float_as_uint(x[5]);
        b.z = __float_as_uint(x[6]); b.w = __float_as_uint(x[7]);
        *(u32x4_any*)p = a;
        *(u32x4_any*)(p + 16) = b;
    } else {
        u32x4 a;
        a.x = from_f32<F>(x[0]) | (from_f32<F>(x[1]) << 16);
        a.y = from_f32<F>(x[2]) | (from_f32<F>(x[3]) << 16);
        a.z = from_f32<F>(x[4]) | (from_f32<F>(x[5]) << 16);
        a.w = from_f32<F>(x[6]) | (from_f32<F>(x[7]) << 16);
        *(u32x4_any*)p = a;
    }
}

}  // namespace fsdp
