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
// Tiles (fsdp_mx4_tiles.h).  From registers alone, with random codes, the
// instruction reaches 5.9 PFLOP/s on this card (8.3 with zeros), the 256 x 256
// tile 4.0-4.1 where the sum is long (8192 x 8192 x 10240: 331-337 us, 8192 x 10240
// x 8192: 342) and 3.8-3.9 at 4096 x 20480 x 5120 (219-226; 3.4-3.5 with operands
// that the caches do not hold).  Two things bound it, told apart by the same
// product of zero codes (8192 x 8192 x 10240: 266-288 us): as many cycles (643,000
// against 623,000 a CU), but at 2.23 GHz instead of 1.86, so power costs a sixth;
// and of those cycles the matrix cores are busy 53% and waves wait 37% of theirs: a
// stage's last loads are sent just before the wait for them, and with one workgroup
// a CU nothing hides a tile's first loads and its stores.  A smaller tile reads more
// of each operand (128 x 128: 408 us at 8192 x 8192 x 10240), so it is taken only
// where the large one leaves CUs idle.
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
static int64_t tiles(const Mx4Product& p, int64_t t) { return ((p.m + t - 1) / t) * ((p.n + t - 1) / t); }

// The side of a product's tiles; 16 for k_mx4_few.
static int side(const Mx4Product& p) {
    const int64_t enough = p.cus * 5 / 8;
    if (tiles(p, 256) >= enough) return 256;
    if (p.m <= kMx4Few && p.n <= 96 * (int64_t)p.cus) return 16;
    return tiles(p, 128) >= enough ? 128 : 64;
}

template <int F>
static hipError_t product(const Mx4Product& p) {
    switch (side(p)) {
    case 256: return launch_tiles<F, 256, 256, 2, 4, 2>(p);
    case 128: return launch_tiles<F, 128, 128, 2, 2, 4>(p);
    case 64: return launch_tiles<F, 64, 64, 2, 2, 4>(p);
    default:
        return launch_mx4_few(Mx4Few{p.a, p.sa, 0, p.m, p.nb * kMx4Block, 0, p.b, p.sb, p.n, p.nb, p.dt, p.out, p.ldo,
                                     p.cus, p.stream});
    }
}

hipError_t launch_mx4_matmul(const Mx4Product& p) {
    if (p.dt == FSDP_F32) return product<FSDP_F32>(p);
    if (p.dt == FSDP_F16) return product<FSDP_F16>(p);
    return product<FSDP_BF16>(p);
}

// Two products share a launch, the one with the longer sum first: the end of one
// is then the beginning of the other, and a launch boundary costs about 5 us.
// Tiles by their number together, but the largest only where each product has
// half of what is enough: a few long ones would outlast all others (us, apart and
// together by side; m x n x k of a layer's gradients, dx m x k and dw n x k):
//   64 x 1024 x 1024    7.4   64: 4.6    128: 6.4    256: 9.7
//   512 x 5120 x 1280   21.4  64: 15.5   128: 16.9   256: 35.9
//   1000 x 6400 x 1600  34.2  64: 34.5   128: 28.6   256: 47.3 (28 + 175 tiles)
//   2048 x 5120 x 1280  37.1  64: 37.2   128: 28.5   256: 37.0 (40 + 100)
//   1500 x 1500 x 6000  54.4  64: 53.8   128: 44.3   256: 38.7 (144 + 144)
//   100 x 12000 x 3000  52.3  64: 49.9   128: 45.7   256: 86.9 (12 + 564)
//   4096 x 4096 x 4096  83.7  64: 152.7  128: 106.1  256: 78.8 (256 + 256)
//   128 x 8192 x 8192   80.9  64: 101.3  128: 82.9   256: 102.9 (32 + 1024)
hipError_t launch_mx4_two(const Mx4Product& a, const Mx4Product& b) {
    const int64_t enough = a.cus * 5 / 8, ta = tiles(a, 256), tb = tiles(b, 256);
    // apart too where the tiles (four times as many of 128) might pass a launch's work items
    if (side(a) == 16 || side(b) == 16 || ta + tb > (1 << 20)) {
        hipError_t e = launch_mx4_matmul(a);
        return e == hipSuccess ? launch_mx4_matmul(b) : e;
    }
    const Mx4Product &x = a.nb >= b.nb ? a : b, &y = a.nb >= b.nb ? b : a;
    if (ta + tb >= enough && ta >= enough / 2 && tb >= enough / 2) return launch_two<256, 256, 2, 4, 2>(x, y);
    if (tiles(a, 128) + tiles(b, 128) >= enough) return launch_two<128, 128, 2, 2, 4>(x, y);
    return launch_two<64, 64, 2, 2, 4>(x, y);
}

}  // namespace fsdp
