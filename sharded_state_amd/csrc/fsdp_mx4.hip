// fsdp_mx4.hip -- gfx950 kernels that turn tensors into 4-bit microscaled
// blocks and back.
//
// A block is 32 consecutive elements that share a power of two.  With
// a = max|x| of the block, e = floor(log2 a) - 2 held in [-127, 127] and
//   code = sign(x) and the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} to |x| / 2^e,
// ties to the code with an even last bit, above 6 to 6; the scale byte is
// e + 127.  floor(log2 a) is a's exponent field, so |x| / 2^e lies in [0, 8)
// and only [7, 8) is off by more than half a step.  A block that holds an
// infinity or a NaN gets the scale byte 255 and stands for NaN; a block of
// zeros gets byte 0.  x is scaled by 2^-e with one exact fp32 product
// (2^-e is a normal number for every e above) and rounded by gfx950's fp4
// conversion with scale 1, two elements an instruction.
// All of this is an HBM stream: 2 to 4 bytes in and 17/32 out an element.
#include "fsdp_device.h"
#include "fsdp_mx4.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const uint32_t f = amax >> 23;
    return f == 255 ? 255u : (f < 2 ? 0u : f - 2);
}
// The factor 2^-e that takes elements into the code's range; 0 for a block that is not finite.
__device__ __forceinline__ float to_codes(uint32_t byte) { return __uint_as_float(byte == 255 ? 0u : (254u - byte) << 23); }
// The factor 2^e of a scale byte; NaN for 255.
__device__ __forceinline__ float from_codes(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7fc00000u : byte << 23));
}

// Eight scaled elements as eight codes, the first in the low nibble.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float f, bool finite) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * f, x[1] * f, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * f, x[3] * f, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * f, x[5] * f, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * f, x[7] * f, 1.0f, 3);
    return finite ? w : 0u;
}

__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// n <= 8 elements at p (any alignment), the rest zero.
template <int F>
__device__ __forceinline__ void load_upto8(const char* p, int64_t n, float (&x)[8]) {
    if (n >= 8) {
        if constexpr (F == FSDP_F32) {
            const u32x4 a = *(const u32x4_any*)p, b = *(const u32x4_any*)(p + 16);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
        } else {
            const u32x4 a = *(const u32x4_any*)p;
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = to_f32<F>(w[k] & 0xffffu);
                x[2 * k + 1] = to_f32<F>(w[k] >> 16);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = k < n ? load1<F>(p, k) : 0.0f;
    }
}

// Blocks along the rows: four lanes a block, eight elements a lane; the
// block's largest magnitude goes round the four with two lane swaps.
template <int F>
__global__ __launch_bounds__(kThreads) void k_mx4_rows(const char* __restrict__ src, int64_t rows, int64_t cols,
                                                       int64_t ld, int64_t nb, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    const int64_t total = rows * nb;
    const int64_t stride = (int64_t)gridDim.x * kThreads / 4;
    const int j = threadIdx.x & 3;
    for (int64_t b = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 2; b < total; b += stride) {
        const int64_t r = rows == 1 ? 0 : b / nb;
        const int64_t c = (b - r * nb) * kMx4Block + j * 8;
        float x[8];
        load_upto8<F>(src + (r * ld + c) * kEs, cols - c, x);
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) a = max(a, mag(x[k]));
        a = max(a, (uint32_t)__shfl_xor((int)a, 1));
        a = max(a, (uint32_t)__shfl_xor((int)a, 2));
        const uint32_t s = scale_byte(a);
        reinterpret_cast<uint32_t*>(codes)[b * 4 + j] = codes8(x, to_codes(s), s != 255);
        if (j == 0) scales[b] = (uint8_t)s;
    }
}

// Blocks along the columns (the rows of the transpose): a lane owns a column
// and takes kColBlocks blocks of 32 rows; the lanes of a wave read 64
// consecutive elements of a row.
constexpr int kColBlocks = 4;
template <int F>
__global__ __launch_bounds__(kThreads) void k_mx4_cols(const char* __restrict__ src, int64_t rows, int64_t cols,
                                                       int64_t ld, int64_t nbr, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    const int64_t col_tiles = (cols + kThreads - 1) / kThreads;
    const int64_t row_tiles = (nbr + kColBlocks - 1) / kColBlocks;
    for (int64_t t = blockIdx.x; t < col_tiles * row_tiles; t += gridDim.x) {
        const int64_t c = t % col_tiles * kThreads + threadIdx.x;
        if (c >= cols) continue;
        const int64_t b0 = t / col_tiles * kColBlocks;
        for (int q = 0; q < kColBlocks && b0 + q < nbr; ++q) {
            const int64_t r0 = (b0 + q) * kMx4Block;
            const char* p = src + (r0 * ld + c) * kEs;
            const int64_t n = rows - r0;
            float x[4][8];
            uint32_t a = 0;
#pragma unroll
            for (int k = 0; k < kMx4Block; ++k) {
                x[k / 8][k % 8] = k < n ? load1<F>(p, (int64_t)k * ld) : 0.0f;
                a = max(a, mag(x[k / 8][k % 8]));
            }
            const uint32_t s = scale_byte(a);
            u32x4 w;
            w.x = codes8(x[0], to_codes(s), s != 255);
            w.y = codes8(x[1], to_codes(s), s != 255);
            w.z = codes8(x[2], to_codes(s), s != 255);
            w.w = codes8(x[3], to_codes(s), s != 255);
            reinterpret_cast<u32x4*>(codes)[c * nbr + b0 + q] = w;
            scales[c * nbr + b0 + q] = (uint8_t)s;
        }
    }
}

// The all-gather of quantised shards into the full buffer of format F: a lane
// turns eight codes into eight elements.  Slots begin wherever q * S puts
// them, so stores take any address.
template <int F>
__global__ __launch_bounds__(kThreads) void k_mx4_gather(Mx4Shards sh, int64_t S, char* __restrict__ out) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    const int q = blockIdx.y;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(sh.codes[q]);
    const uint8_t* scales = sh.scales[q];
    const int64_t nv = (S + 7) / 8;
    for (int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x; v < nv; v += (int64_t)gridDim.x * kThreads) {
        const uint32_t w = codes[v];
        const float f = from_codes(scales[v >> 2]);
        const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        const f32x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
        const f32x2 y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        float x[8] = {y0.x * f, y0.y * f, y1.x * f, y1.y * f, y2.x * f, y2.y * f, y3.x * f, y3.y * f};
        // kept apart from the conversion: fused with it the compiler adds +0 and -0 loses its sign
        if constexpr (F == FSDP_F16) {
#pragma unroll
            for (int k = 0; k < 8; ++k) asm("" : "+v"(x[k]));
        }
        const int64_t i = (int64_t)q * S + v * 8;
        char* o = out + i * kEs;
        if (v * 8 + 8 <= S) {
            if constexpr (F == FSDP_F32) {
                u32x4 a, b;
                a.x = __float_as_uint(x[0]); a.y = __float_as_uint(x[1]);
                a.z = __float_as_uint(x[2]); a.w = __float_as_uint(x[3]);
                b.x = __float_as_uint(x[4]); b.y = __float_as_uint(x[5]);
                b.z = __float_as_uint(x[6]); b.w = __float_as_uint(x[7]);
                *(u32x4_any*)o = a;
                *(u32x4_any*)(o + 16) = b;
            } else {
                u32x4 a;
                a.x = from_f32<F>(x[0]) | (from_f32<F>(x[1]) << 16);
                a.y = from_f32<F>(x[2]) | (from_f32<F>(x[3]) << 16);
                a.z = from_f32<F>(x[4]) | (from_f32<F>(x[5]) << 16);
                a.w = from_f32<F>(x[6]) | (from_f32<F>(x[7]) << 16);
                *(u32x4_any*)o = a;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v * 8 + k < S) store1<F>(out, i + k, x[k]);
        }
    }
}

// ----------------------------------------------------------------- launchers
// A launch holds fewer than 2^32 work items; beyond 2^22 workgroups they loop.
static unsigned capped(int64_t want) {
    const int64_t cap = 1 << 22;
    return (unsigned)(want < 1 ? 1 : (want < cap ? want : cap));
}

template <int F>
static void quantize(const Mx4Quant& q, hipStream_t st) {
    const char* src = (const char*)q.src;
    if (q.codes) {
        int64_t rows = q.rows, cols = q.cols;
        if (q.ld == cols && cols % kMx4Block == 0) {      // whole blocks row after row: one long row
            cols *= rows;
            rows = 1;
        }
        const int64_t nb = mx4_blocks(cols);
        launch(k_mx4_rows<F>, dim3(capped((rows * nb * 4 + kThreads - 1) / kThreads)), dim3(kThreads), st, src, rows,
               cols, q.ld, nb, q.codes, q.scales);
    }
    if (q.codes_t) {
        const int64_t nbr = mx4_blocks(q.rows);
        const int64_t tiles = (q.cols + kThreads - 1) / kThreads * ((nbr + kColBlocks - 1) / kColBlocks);
        launch(k_mx4_cols<F>, dim3(capped(tiles)), dim3(kThreads), st, src, q.rows, q.cols, q.ld, nbr, q.codes_t,
               q.scales_t);
    }
}

hipError_t launch_mx4_quantize(const Mx4Quant& q, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (q.dt == FSDP_F32) quantize<FSDP_F32>(q, st);
    else if (q.dt == FSDP_F16) quantize<FSDP_F16>(q, st);
    else quantize<FSDP_BF16>(q, st);
    return hipGetLastError();
}

hipError_t launch_mx4_gather(const Mx4Shards& s, int world, int64_t S, int dt, void* out, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    int64_t per = ((S + 7) / 8 + kThreads - 1) / kThreads;
    const int64_t cap = (1 << 22) / world;
    const dim3 g((unsigned)(per < cap ? per : cap), (unsigned)world), th(kThreads);
    if (dt == FSDP_F32) launch(k_mx4_gather<FSDP_F32>, g, th, st, s, S, (char*)out);
    else if (dt == FSDP_F16) launch(k_mx4_gather<FSDP_F16>, g, th, st, s, S, (char*)out);
    else launch(k_mx4_gather<FSDP_BF16>, g, th, st, s, S, (char*)out);
    return hipGetLastError();
}

}  // namespace fsdp
