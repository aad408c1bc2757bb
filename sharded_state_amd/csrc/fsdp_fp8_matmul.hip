// fsdp_fp8_matmul.hip -- the product of two matrices of 8-bit blocks on gfx950's
// scaled matrix instructions.
//
//   C[i][j] = sum over blocks b of 2^(ea(i,b) + eb(j,b)) * sum over the block of qa * qb
//
// Both operands hold their blocks along the summed axis.  v_mfma_scale_f32_32x32x64
// takes from lane l of a wave row l % 32, 32 codes of half l / 32 and a scale byte:
// a block of 128 is two instructions with the same scales.  Sums are fp32 and run in
// a fixed order, so the same call gives the same bits.
#include "fsdp_fp8_tiles.h"

#pragma clang fp contract(off)

namespace fsdp {

template <int F>
static hipError_t product(const Fp8Product& p) {
    const int64_t enough = p.cus * 5 / 8;
    auto tiles = [&](int64_t t) { return ((p.m + t - 1) / t) * ((p.n + t - 1) / t); };
    if (tiles(256) >= enough) return launch_fp8_tiles<F, 256, 256, 2, 4, 2>(p);
    if (tiles(128) >= enough) return launch_fp8_tiles<F, 128, 128, 2, 2, 4>(p);
    return launch_fp8_tiles<F, 64, 64, 2, 2, 4>(p);
}

hipError_t launch_fp8_matmul(const Fp8Product& p) {
    if (p.dt == FSDP_F32) return product<FSDP_F32>(p);
    if (p.dt == FSDP_F16) return product<FSDP_F16>(p);
    return product<FSDP_BF16>(p);
}

}  // namespace fsdp
