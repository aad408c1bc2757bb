// fsdp_fp8_matmul.hip -- the product of two matrices of 8-bit blocks on gfx950's
// scaled matrix instructions.
//
//   C[i][j] = sum over blocks b of 2^(ea(i,b) + eb(j,b)) * sum over the block of qa * qb
//
// Both operands hold their blocks along the summed axis.  v_mfma_scale_f32_32x32x64
// takes from lane l of a wave row l % 32, 32 codes of half l / 32 and a scale byte:
// a block of 128 is two instructions with the same scales.  Sums are fp32 and run in
// a fixed order, so the same call gives the same bits.
#include "fsdp_fp8_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kE4m3 = 0;    // the instruction's code for the format

// A wave makes 32 x 32 results, a workgroup 64 x 64, operands straight from memory.
__global__ __launch_bounds__(256) void k_fp8_product(Fp8Product p, int64_t tm0, int64_t tn0, uint32_t tiles_n) {
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6, h = l >> 5;
    const int64_t m0 = (tm0 + blockIdx.x / tiles_n) * 64 + (w >> 1) * 32;
    const int64_t n0 = (tn0 + blockIdx.x % tiles_n) * 64 + (w & 1) * 32;
    if (m0 >= p.m || n0 >= p.n) return;
    // rows behind a matrix are read as its last one; nobody stores what they give
    const int64_t i = m0 + (l & 31) < p.m ? m0 + (l & 31) : p.m - 1, j = n0 + (l & 31) < p.n ? n0 + (l & 31) : p.n - 1;
    const uint8_t *a = p.a + i * p.nb * kFp8Block, *sa = p.sa + (i >> p.ta) * p.nb;
    const uint8_t *b = p.b + j * p.nb * kFp8Block, *sb = p.sb + (j >> p.tb) * p.nb;
    f32x16 acc = f32x16{0};
    for (int64_t k = 0; k < p.nb; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t at = k * kFp8Block + s * 64 + h * 32;
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(*(const i32x8*)(b + at), *(const i32x8*)(a + at), acc,
                                                                  kE4m3, kE4m3, 0, sb[k], 0, sa[k]);
        }
    const int64_t row = m0 + (l & 31);
    if (row >= p.m) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int64_t col = n0 + e / 4 * 8 + h * 4 + e % 4;
        if (col >= p.n) continue;
        const int64_t o = row * p.ldo + col;
        if (p.dt == FSDP_F32) store1<FSDP_F32>(p.out, o, acc[e]);
        else if (p.dt == FSDP_F16) store1<FSDP_F16>(p.out, o, acc[e]);
        else store1<FSDP_BF16>(p.out, o, acc[e]);
    }
}

hipError_t launch_fp8_matmul(const Fp8Product& p) {
    // a launch holds fewer than 2^32 work items; more tiles go in parts of the result
    constexpr int64_t kMost = (1 << 24) - 1;
    const int64_t tm = (p.m + 63) / 64, tn = (p.n + 63) / 64;
    const int64_t pn = tn < kMost ? tn : kMost, pm = kMost / pn < tm ? kMost / pn : tm;
    for (int64_t i = 0; i < tm; i += pm)
        for (int64_t j = 0; j < tn; j += pn) {
            const int64_t cm = tm - i < pm ? tm - i : pm, cn = tn - j < pn ? tn - j : pn;
            launch(k_fp8_product, dim3((unsigned)(cm * cn)), dim3(256), (hipStream_t)p.stream, p, i, j, (uint32_t)cn);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

}  // namespace fsdp
