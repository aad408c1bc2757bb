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

// The largest of four neighbouring lanes' values, in all four of them.
__device__ __forceinline__ uint32_t max_of_four(uint32_t a) {
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
    return max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

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
        const uint32_t s = scale_byte(max_of_four(a));
        reinterpret_cast<uint32_t*>(codes)[b * 4 + j] = codes8(x, to_codes(s), s != 255);
        if (j == 0) scales[b] = (uint8_t)s;
    }
}

// Blocks along the columns (the rows of the transpose), and with ROWS along the
// rows too, from one read: a workgroup brings kTile x kTile elements, a lane 8
// of a row at a time.  The rows' blocks are made from registers (four lanes a
// block); for the columns' the tile goes through LDS as it is, and a lane takes
// two columns of 32 rows, one read a row pair.  Workgroups go to the XCDs in
// turn; XCD x takes one run of tiles down the columns, so what neighbouring
// tiles write to a line of the transpose (64 bytes of codes, 4 of scales each)
// meets in one L2.
constexpr int kTile = 128;
template <int F, bool ROWS>
__global__ __launch_bounds__(kThreads) void k_mx4_cols(const char* __restrict__ src, int64_t rows, int64_t cols,
                                                       int64_t ld, uint32_t tiles_r, uint32_t tiles,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                       uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kPass = kThreads / (kTile / 8);            // rows a pass
    __shared__ __attribute__((aligned(16))) uint8_t lds[kTile * kTile * kEs];
    const uint32_t x = blockIdx.x & 7, per = tiles >> 3, more = tiles & 7;
    const uint32_t t = x * per + (x < more ? x : more) + (blockIdx.x >> 3);
    const int64_t r0 = (int64_t)(t % tiles_r) * kTile, c0 = (int64_t)(t / tiles_r) * kTile;
    const int64_t nb = (cols + kMx4Block - 1) / kMx4Block, nbr = (rows + kMx4Block - 1) / kMx4Block;
    const int lr = threadIdx.x / (kTile / 8), lc = threadIdx.x % (kTile / 8) * 8;
#pragma unroll
    for (int q = 0; q < kTile / kPass; ++q) {
        const int64_t r = r0 + q * kPass + lr, c = c0 + lc;
        float v[8];
        load_upto8<F>(src + (r * ld + c) * kEs, r < rows ? cols - c : 0, v);
        uint8_t* o = lds + ((q * kPass + lr) * kTile + lc) * kEs;
        if constexpr (F == FSDP_F32) {
            u32x4 a, b;
            a.x = __float_as_uint(v[0]); a.y = __float_as_uint(v[1]);
            a.z = __float_as_uint(v[2]); a.w = __float_as_uint(v[3]);
            b.x = __float_as_uint(v[4]); b.y = __float_as_uint(v[5]);
            b.z = __float_as_uint(v[6]); b.w = __float_as_uint(v[7]);
            *reinterpret_cast<u32x4*>(o) = a;
            *reinterpret_cast<u32x4*>(o + 16) = b;
        } else {
            u32x4 a;
            a.x = from_f32<F>(v[0]) | (from_f32<F>(v[1]) << 16);
            a.y = from_f32<F>(v[2]) | (from_f32<F>(v[3]) << 16);
            a.z = from_f32<F>(v[4]) | (from_f32<F>(v[5]) << 16);
            a.w = from_f32<F>(v[6]) | (from_f32<F>(v[7]) << 16);
            *reinterpret_cast<u32x4*>(o) = a;
        }
        if constexpr (ROWS) {
            uint32_t a = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) a = max(a, mag(v[k]));
            const uint32_t s = scale_byte(max_of_four(a));
            const uint32_t w = codes8(v, to_codes(s), s != 255);
            if (r < rows && (c >> 5) < nb) {
                const int64_t b = r * nb + (c >> 5);
                reinterpret_cast<uint32_t*>(codes)[b * 4 + (threadIdx.x & 3)] = w;
                if ((threadIdx.x & 3) == 0) scales[b] = (uint8_t)s;
            }
        }
    }
    __syncthreads();
    const int cp = threadIdx.x % (kTile / 2) * 2, rb = threadIdx.x / (kTile / 2);
    const int64_t b = r0 / kMx4Block + rb;
    if (b >= nbr) return;
    float v[2][4][8];
    uint32_t a[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kMx4Block; ++k) {
        const uint8_t* o = lds + ((rb * kMx4Block + k) * kTile + cp) * kEs;
        if constexpr (F == FSDP_F32) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(o);
            v[0][k / 8][k % 8] = __uint_as_float(w.x);
            v[1][k / 8][k % 8] = __uint_as_float(w.y);
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(o);
            v[0][k / 8][k % 8] = to_f32<F>(w & 0xffffu);
            v[1][k / 8][k % 8] = to_f32<F>(w >> 16);
        }
        a[0] = max(a[0], mag(v[0][k / 8][k % 8]));
        a[1] = max(a[1], mag(v[1][k / 8][k % 8]));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t c = c0 + cp + e;
        if (c >= cols) break;
        const uint32_t s = scale_byte(a[e]);
        u32x4 w;
        w.x = codes8(v[e][0], to_codes(s), s != 255);
        w.y = codes8(v[e][1], to_codes(s), s != 255);
        w.z = codes8(v[e][2], to_codes(s), s != 255);
        w.w = codes8(v[e][3], to_codes(s), s != 255);
        reinterpret_cast<u32x4*>(codes_t)[c * nbr + b] = w;
        scales_t[c * nbr + b] = (uint8_t)s;
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
static hipError_t quantize(const Mx4Quant& q, hipStream_t st) {
    const char* src = (const char*)q.src;
    if (q.codes_t) {
        const int64_t tr = (q.rows + kTile - 1) / kTile, tc = (q.cols + kTile - 1) / kTile;
        if (tr > (1 << 24) / tc) return hipErrorInvalidValue;       // 2^38 elements
        const dim3 g((unsigned)(tr * tc)), th(kThreads);
        if (q.codes)
            launch(k_mx4_cols<F, true>, g, th, st, src, q.rows, q.cols, q.ld, (uint32_t)tr, (uint32_t)(tr * tc),
                   q.codes, q.scales, q.codes_t, q.scales_t);
        else
            launch(k_mx4_cols<F, false>, g, th, st, src, q.rows, q.cols, q.ld, (uint32_t)tr, (uint32_t)(tr * tc),
                   q.codes, q.scales, q.codes_t, q.scales_t);
        return hipGetLastError();
    }
    int64_t rows = q.rows, cols = q.cols;
    if (q.ld == cols && cols % kMx4Block == 0) {      // whole blocks row after row: one long row
        cols *= rows;
        rows = 1;
    }
    const int64_t nb = mx4_blocks(cols);
    launch(k_mx4_rows<F>, dim3(capped((rows * nb * 4 + kThreads - 1) / kThreads)), dim3(kThreads), st, src, rows,
           cols, q.ld, nb, q.codes, q.scales);
    return hipGetLastError();
}

hipError_t launch_mx4_quantize(const Mx4Quant& q, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (q.dt == FSDP_F32) return quantize<FSDP_F32>(q, st);
    if (q.dt == FSDP_F16) return quantize<FSDP_F16>(q, st);
    return quantize<FSDP_BF16>(q, st);
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
