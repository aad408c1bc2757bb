// fsdp_rms_device.h -- device primitives of the norm over features: eight elements
// of a row a lane, in any of the formats, and a row's sums.  Not installed.
#pragma once

#include "fsdp_fp8_device.h"
#include "fsdp_rms.h"

#pragma clang fp contract(off)

namespace fsdp {

template <int F>
__device__ __forceinline__ void to_floats(const Raw8<F>& r, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (F == FSDP_F32) v[k] = __uint_as_float(r.w[k]);
        else v[k] = to_f32<F>(k & 1 ? r.w[k / 2] >> 16 : r.w[k / 2] & 0xffffu);
    }
}

// Elements [c, c + 8) of a row of d, zeros behind it, in two halves: the load, and
// what is done with it once it is there.  No load stands under a condition of its own:
// with WHOLE (d a multiple of 8) a lane behind the row loads its first eight, else a
// lane at or behind the row's end its last eight, and shifts.
template <int F, bool WHOLE>
__device__ __forceinline__ Raw8<F> load_row8(const char* row, int c, int d) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    if constexpr (WHOLE) return load8_raw<F>(row + (c < d ? c : 0) * kEs);
    if (d < 8) return load_upto8<F>(row + (c < d ? c : 0) * kEs, d - c);
    return load8_raw<F>(row + (c < d - 8 ? c : d - 8) * kEs);
}
template <int B>
__device__ __forceinline__ void shift_down(float (&v)[8], bool on) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float x = 0.0f;
        if (k + B < 8) x = v[k + B < 8 ? k + B : 7];
        v[k] = on ? x : v[k];
    }
}
template <int F, bool WHOLE>
__device__ __forceinline__ void row8(const Raw8<F>& r, int c, int d, float (&v)[8]) {
    to_floats<F>(r, v);
    if constexpr (!WHOLE) {
        if (d < 8) return;
        const int s = c > d - 8 ? c - (d - 8) : 0;
        shift_down<4>(v, s & 4);
        shift_down<2>(v, s & 2);
        shift_down<1>(v, s & 1);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c < d ? v[k] : 0.0f;
}

// A format that the launch alone knows.
template <bool WHOLE>
__device__ __forceinline__ void any_row8(const void* row, int dt, int c, int d, float (&v)[8]) {
    if (dt == FSDP_F32) row8<FSDP_F32, WHOLE>(load_row8<FSDP_F32, WHOLE>((const char*)row, c, d), c, d, v);
    else if (dt == FSDP_F16) row8<FSDP_F16, WHOLE>(load_row8<FSDP_F16, WHOLE>((const char*)row, c, d), c, d, v);
    else row8<FSDP_BF16, WHOLE>(load_row8<FSDP_BF16, WHOLE>((const char*)row, c, d), c, d, v);
}

// 16-bit rows are stored with the non-temporal hint (the forward of 4096 x 4096 bf16 27.5
// -> 25.4 us, of 8192 x 1000 16.0 -> 13.2); a lane's two stores of fp32 take half a line
// each, and with it 8191 x 8192 went from 142 to 159.  Codes are not: the product behind
// reads them (norm and product of 200 x 5120 x 5120 26.1 us, 27.8 with the hint).
template <int F, bool WHOLE>
__device__ __forceinline__ void store_row8(char* row, int c, int d, const float (&v)[8]) {
    if (WHOLE ? c < d : c + 8 <= d) {
        if constexpr (F == FSDP_F32)
            store8_any<F>(row + (int64_t)c * 4, v);
        else
            __builtin_nontemporal_store(u32x4{pack2<F>(v[0], v[1]), pack2<F>(v[2], v[3]), pack2<F>(v[4], v[5]), pack2<F>(v[6], v[7])},
                                        (u32x4_any*)(row + (int64_t)c * 2));
    } else if (!WHOLE) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < d) store1<F>(row, c + k, v[k]);
    }
}
template <bool WHOLE>
__device__ __forceinline__ void any_store8(void* row, int dt, int c, int d, const float (&v)[8]) {
    if (dt == FSDP_F32) store_row8<FSDP_F32, WHOLE>((char*)row, c, d, v);
    else if (dt == FSDP_F16) store_row8<FSDP_F16, WHOLE>((char*)row, c, d, v);
    else store_row8<FSDP_BF16, WHOLE>((char*)row, c, d, v);
}

// x of another lane of the row of 16 lanes.
template <int DPP>
__device__ __forceinline__ double moved(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, DPP, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), DPP, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double x, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The sum over a workgroup's lanes, in all of them, in a fixed order.  `part`: a double a
// wave, not written again before every wave has read it.  Lane swaps and scalar reads, not
// the LDS's permutations (gradients of 8192 x 8192 115 -> 110 us, of 1000 x 1600 12.0 ->
// 11.1, a norm of one token 2.7 -> 2.5).
__device__ __forceinline__ double row_sum(double x, double* part) {
    x += moved<0xB1>(x);          // lane ^ 1
    x += moved<0x4E>(x);          // lane ^ 2
    x += moved<0x141>(x);         // halves of 8 mirrored
    x += moved<0x140>(x);         // the 16 mirrored
    x = (lane_of(x, 0) + lane_of(x, 16)) + (lane_of(x, 32) + lane_of(x, 48));
    if (blockDim.x == 64) return x;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
    for (int k = 1; k < (int)blockDim.x >> 6; ++k) x += part[k];
    return x;
}

// A row goes to a workgroup of T lanes, each with eight elements U times: U is 1 up to
// `one` features, and there are the fewest lanes of whole waves that hold the row.
inline int rms_units(int64_t d, int64_t one) { return d <= one ? 1 : (d <= 16384 ? 2 : 4); }
inline int rms_lanes(int64_t d, int64_t one) {
    const int64_t each = 512 * rms_units(d, one);
    return d > 0 ? (int)((d + each - 1) / each * 64) : 64;
}

// Run L<A, B, U, WHOLE>::run(p, stream) for formats a and b and rows of p.d.
template <template <int, int, int, bool> class L, int A, int B, typename P>
static hipError_t by_size(const P& p, hipStream_t st) {
    const int u = rms_units(p.d, L<A, B, 1, true>::kOne);
    if (p.d % 8 == 0) return u == 1 ? L<A, B, 1, true>::run(p, st) : (u == 2 ? L<A, B, 2, true>::run(p, st) : L<A, B, 4, true>::run(p, st));
    return u == 1 ? L<A, B, 1, false>::run(p, st) : (u == 2 ? L<A, B, 2, false>::run(p, st) : L<A, B, 4, false>::run(p, st));
}
template <template <int, int, int, bool> class L, int A, typename P>
static hipError_t by_second(const P& p, int b, hipStream_t st) {
    if (b == FSDP_F32) return by_size<L, A, FSDP_F32>(p, st);
    if (b == FSDP_F16) return by_size<L, A, FSDP_F16>(p, st);
    return by_size<L, A, FSDP_BF16>(p, st);
}
template <template <int, int, int, bool> class L, typename P>
static hipError_t by_formats(const P& p, int a, int b, hipStream_t st) {
    if (a == FSDP_F32) return by_second<L, FSDP_F32>(p, b, st);
    if (a == FSDP_F16) return by_second<L, FSDP_F16>(p, b, st);
    return by_second<L, FSDP_BF16>(p, b, st);
}

}  // namespace fsdp
