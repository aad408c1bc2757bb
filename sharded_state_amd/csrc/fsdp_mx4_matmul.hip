// fsdp_mx4_matmul.hip -- the product of two matrices of 4-bit microscaled
// blocks on gfx950's scaled matrix instructions.
//
//   C[i][j] = sum over blocks b of 2^(ea(i,b) + eb(j,b)) * sum over the block of qa * qb
//
// Both operands hold their blocks along the summed axis, which is what
// v_mfma_scale_f32_32x32x64_f8f6f4 wants: lane l of a wave brings row l % 32,
// the 32 codes (16 bytes) of block l / 32 and that block's scale byte, and the
// products of 32 x 32 rows over two blocks are added to fp32 sums.  Sums run
// in a fixed order, so the same call gives the same bits.
//
// Tiles (fsdp_mx4_tiles.h).  What bounds the largest one is power: registers
// alone, with random codes, the instruction reaches 5.9 PFLOP/s on this card
// (8.3 with zeros), and the 256 x 256 tile 4.0-4.1 (8192 x 8192 x 10240: 338
// us, 8192 x 10240 x 8192: 337 us, 4096 x 20480 x 5120: 225 us).  A smaller tile
// reads more of each operand (128 x 128: 408 us at 8192 x 8192 x 10240), so it
// is taken only where the large one leaves CUs idle.
#include "fsdp_mx4_tiles.h"

#pragma clang fp contract(off)

namespace fsdp {

// For up to 16 rows of A the product is a read of B, and k_mx4_few reads it with
// more loads on their way than few tiles do (16 rows, us: 8192 x 28672 28.3 against
// 54.7 in tiles, 4096 x 4096 4.7 and 8.3, 10240 x 8192 14.3 and 18.2, 20480 x 5120
// 16.7 and 17.3), until the tiles are many (28672 x 8192 32.1 against 28.8, 40000 x
// 512 7.5 and 5.8).
// Else the largest tile that gives at least 5/8 of the CUs a tile (measured, us):
//   6400 x 1600 x 1000  256: 13.4 (175 tiles)  128: 16.9 (650)   64: 19.1
//   3000 x 5000 x 700   256: 14.9 (240 tiles)  128: 24.6         64: 31.3
//   2048 x 2048 x 2048  256: 16.8 (64 tiles)   128: 10.0 (256)   64: 12.1
//   512 x 8192 x 8192   256: 53.0 (64 tiles)   128: 25.5 (256)   64: 37.6
//   1000 x 1600 x 6400  256: 43.8 (28 tiles)   128: 20.1 (104)   64: 16.1 (400)
//   256 x 5120 x 5120   256: 30.9 (20 tiles)   128: 15.4 (80)    64: 12.4 (320)
// The two smaller ones keep 4 stages in LDS (128 x 128 with 2: 31.5 us instead
// of 25.5 at 512 x 8192 x 8192): with few tiles a CU the loads' latency counts.
template <int F>
static hipError_t product(const Mx4Product& p) {
    auto tiles = [&](int64_t t) { return ((p.m + t - 1) / t) * ((p.n + t - 1) / t); };
    const int64_t enough = p.cus * 5 / 8;
    if (tiles(256) >= enough) return launch_tiles<F, 256, 256, 2, 4, 2>(p);
    if (p.m <= kMx4Few && p.n <= 96 * (int64_t)p.cus)
        return launch_mx4_few(Mx4Few{p.a, p.sa, 0, p.m, p.nb * kMx4Block, 0, p.b, p.sb, p.n, p.nb, p.dt, p.out, p.ldo,
                                     p.cus, p.stream});
    if (tiles(128) >= enough) return launch_tiles<F, 128, 128, 2, 2, 4>(p);
    return launch_tiles<F, 64, 64, 2, 2, 4>(p);
}

hipError_t launch_mx4_matmul(const Mx4Product& p) {
    if (p.dt == FSDP_F32) return product<FSDP_F32>(p);
    if (p.dt == FSDP_F16) return product<FSDP_F16>(p);
    return product<FSDP_BF16>(p);
}

}  // namespace fsdp
