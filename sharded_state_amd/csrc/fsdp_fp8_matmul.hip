// fsdp_fp8_matmul.hip -- the product of two matrices of 8-bit blocks on gfx950's
// scaled matrix instructions.
//
//   C[i][j] = sum over blocks b of 2^(ea(i,b) + eb(j,b)) * sum over the block of qa * qb
//
// Both operands hold their blocks along the summed axis.  v_mfma_scale_f32_32x32x64
// takes from lane l of a wave row l % 32, 32 codes of half l / 32 and a scale byte:
// a block of 128 is two instructions with the same scales.  Sums are fp32 and run in
// a fixed order, so the same call gives the same bits.  Within an instruction eight
// products at a time are cut off under 2^-13 of the largest one's power of two before
// they are added: that is the hardware's, and the price of its rate (1.5e-5 of the
// result's norm with normally distributed operands, whose rounding to e4m3 costs 4e-2).
//
// From registers alone, with codes of normally distributed numbers, the instruction
// reaches 3.9 PFLOP/s on this card (4.8 with zeros: the clock that power allows).
// Products reach 2.7-2.8 where the sum is long (8192^3: 402 us with operands that the
// caches do not hold), 2.6 at 4096 x 20480 x 5120 (332 us).  fsdp_fp8_tiles.h says what
// bounds them.
#include "fsdp_fp8_tiles.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef float f32x4 __attribute__((ext_vector_type(4)));

static int64_t tiles(const Fp8Product& p, int64_t tm, int64_t tn) { return ((p.m + tm - 1) / tm) * ((p.n + tn - 1) / tn); }

// Tiles of a launch are counted in 31 bits: larger results go in parts of 2^20 x 2^20.
constexpr int64_t kPart = 1 << 20;

// The kinds of tiles.  Up to 16 rows of A the product is a read of B, and k_fp8_few has
// more loads on their way than few tiles do (16 rows, us: 8192 x 8192 17.6 against 30.5 in
// tiles, 5120 x 1280 4.4 and 6.8, 1000 x 1000 3.1 and 5.6);
// it holds the scales of 32 rows in LDS, hence kFewBlocks.  Above 96 rows of B a CU the
// tiles are taken, though k_fp8_few is ahead on both sides of that border (16 rows, us:
// 24576 x 8192 42.0 against 48.0, 28672 x 8192 49.4 and 53.0, 50304 x 5120 58.6 and 75.0; one
// row, 28672 x 8192 45.5 and 51.5).  Else the largest tile that gives at least 5/8 of the CUs one (us):
//                       256     128, 2 stages   128, 4 stages   64 x 128   64
//   4096 x 4096 x 4096  56.9    70.2            77.4            105.8      117.7
//   6400 x 1600 x 1000  19.9    18.6            20.8            31.1       27.6
//   1000 x 6400 x 1600  24.6    17.8 (400)      20.6            28.8       26.9
//   2048 x 2048 x 2048  24.1    14.7 (256)      12.9            17.0       18.5
//   512 x 8192 x 8192   100.0   60.2 (256)      42.5            65.3       71.4
//   1000 x 1600 x 6400  60.3    34.8 (104)      27.8            22.5       24.3
//   256 x 5120 x 5120   52.5    31.3 (80)       22.5            19.2       20.9
//   24 x 6400 x 1600    22.3    12.2 (50)       10.9            9.2        7.7
// With more tiles than CUs two workgroups of 128 x 128 and two stages share a CU; with
// fewer, four stages in LDS hide more of the loads' latency.
constexpr int64_t kFewBlocks = 2048;
enum { kFew, k64, k64x128, k128x4, k128, k256 };
static int kind(const Fp8Product& p) {
    const int64_t enough = p.cus * 5 / 8;
    if (tiles(p, 256, 256) >= enough) return k256;
    if (p.m <= kFp8Few && p.nb <= kFewBlocks && p.n <= 96 * (int64_t)p.cus) return kFew;
    const int64_t t = tiles(p, 128, 128);
    if (t >= enough) return t > p.cus ? k128 : k128x4;
    return tiles(p, 64, 128) >= enough ? k64x128 : k64;
}

static hipError_t launch_kind(int kind, const Fp8Product* p, int count, const int* splits) {
    switch (kind) {
    case k256: return launch_fp8_jobs<256, 256, 2, 2, 2>(p, count, splits);
    case k128: return launch_fp8_jobs<128, 128, 2, 2, 2>(p, count, splits);
    case k128x4: return launch_fp8_jobs<128, 128, 2, 2, 4>(p, count, splits);
    case k64x128: return launch_fp8_jobs<64, 128, 2, 2, 4>(p, count, splits);
    default: return launch_fp8_jobs<64, 64, 2, 2, 4>(p, count, splits);
    }
}

// Rounds that a product's sum is split into, none of them empty, each a matrix of fp32
// partial sums that k_fp8_join adds: where even 64 x 64 leaves CUs without a tile, and each
// round keeps 8 blocks (us without and with: 100 x 3008 x 12000 29.3 and 17.6, 32 x 4096 x
// 16384 53.3 and 19.8, 64 x 8192 x 28672 99.0 and 56.6, 24 x 1600 x 6400 17.7 and 10.3; but
// where tiles are more, writing and reading the parts costs more: 256 x 5120 x 5120 19.4
// and 22.8, 1000 x 1600 x 6400 23.0 and 30.4).  Together with another product the tiles are
// larger, and the other's fill the CUs.
static int splits_of(const Fp8Product& p, bool alone) {
    if (p.nb < 16 || kind(p) != k64) return 1;
    const int64_t most = alone ? 2 * p.cus / tiles(p, 64, 64) : p.cus / tiles(p, 128, 128);
    const int64_t s = most < p.nb / 8 ? most : p.nb / 8;
    if (s < 2) return 1;
    const int64_t chunk = (p.nb + s - 1) / s;
    return (int)((p.nb + chunk - 1) / chunk);
}

int64_t fp8_parts_bytes(int64_t m, int64_t n, int64_t nb, int cus) {
    if (m == 0 || n == 0 || m > kPart || n > kPart) return 0;
    Fp8Product p{};
    p.m = m;
    p.n = n;
    p.nb = nb;
    p.cus = cus;
    const int a = splits_of(p, true), b = splits_of(p, false), s = a > b ? a : b;
    return s > 1 ? (s * m * n * 4 + 15) / 16 * 16 : 0;
}

// The sum of a product's partial sums in their order: four columns a lane.
__global__ __launch_bounds__(256) void k_fp8_join(const float* __restrict__ parts, int splits, int64_t m, int64_t n,
                                                  uint32_t across, void* __restrict__ out, int64_t ldo, int dt) {
    const int64_t row = blockIdx.x / across, col = ((int64_t)(blockIdx.x % across) * 256 + threadIdx.x) * 4;
    if (col >= n) return;
    const float* at = parts + row * n + col;
    const int64_t o = row * ldo + col;
    auto put = [&](int64_t i, float x) {
        if (dt == FSDP_F32) store1<FSDP_F32>(out, i, x);
        else if (dt == FSDP_F16) store1<FSDP_F16>(out, i, x);
        else store1<FSDP_BF16>(out, i, x);
    };
    if (col + 4 <= n) {
        typedef f32x4 f32x4_any __attribute__((aligned(4)));
        f32x4 s = *(const f32x4_any*)at;
        for (int k = 1; k < splits; ++k) s += *(const f32x4_any*)(at + k * m * n);
        if (dt == FSDP_F32) {
            *(f32x4_any*)((float*)out + o) = s;
        } else {
            const u32x2 v = dt == FSDP_F16 ? u32x2{pack2<FSDP_F16>(s.x, s.y), pack2<FSDP_F16>(s.z, s.w)}
                                           : u32x2{pack2<FSDP_BF16>(s.x, s.y), pack2<FSDP_BF16>(s.z, s.w)};
            *(u32x2_any*)((uint16_t*)out + o) = v;
        }
    } else {
        for (int c = 0; col + c < n; ++c) {
            float s = at[c];
            for (int k = 1; k < splits; ++k) s += at[c + k * m * n];
            put(o + c, s);
        }
    }
}
static hipError_t join(const Fp8Product& p, int splits) {
    if (splits < 2) return hipSuccess;
    const uint32_t across = (uint32_t)((p.n + 1023) / 1024);
    launch(k_fp8_join, dim3((unsigned)(across * p.m)), dim3(256), (hipStream_t)p.stream, (const float*)p.parts, splits, p.m,
           p.n, across, p.out, p.ldo, p.dt);
    return hipGetLastError();
}

hipError_t launch_fp8_matmul(const Fp8Product& p) {
    for (int64_t i = 0; i < p.m; i += kPart)
        for (int64_t j = 0; j < p.n; j += kPart) {
            Fp8Product c = p;
            c.m = p.m - i < kPart ? p.m - i : kPart;
            c.n = p.n - j < kPart ? p.n - j : kPart;
            c.a = p.a + i * p.nb * kFp8Block;
            c.b = p.b + j * p.nb * kFp8Block;
            c.sa = p.sa + (i >> p.ta) * p.nb;
            c.sb = p.sb + (j >> p.tb) * p.nb;
            c.out = (char*)p.out + (i * p.ldo + j) * dt_bytes(p.dt);
            const int how = kind(c), splits = p.parts ? splits_of(c, true) : 1;
            hipError_t e = how == kFew ? launch_fp8_few(Fp8Few{c.a, c.sa, 0, c.ta, c.m, c.nb * kFp8Block, 0, c.b, c.sb, c.tb, c.n,
                                                               c.nb, c.dt, c.out, c.ldo, c.cus, c.stream})
                                       : launch_kind(how, &c, 1, &splits);
            if (e == hipSuccess) e = join(c, splits);
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

// Two products share a launch, the one with the longer sum first, in tiles by their number
// together, but the largest only where each product has half of what is enough: a few long
// ones would outlast all others.  A layer's gradients with their quantisation (m x n x k, dx
// m x k and dw n x k; us by tile 256, 128, 64):
//   64 x 1024 x 1024     21.1   13.4   11.0
//   512 x 5120 x 1280    62.7   28.5 (41.3 unsplit)   32.5
//   1000 x 6400 x 1600   75.4   53.1   72.7
//   2048 x 5120 x 1280   66.9   49.5   68.7
//   1500 x 1500 x 6000   59.7   57.2   78.4
//   128 x 8192 x 8192    134.5  70.9 (116.9 unsplit)  107.6
//   4096 x 4096 x 4096   134.8  166.1  261.5
//   8192 x 10240 x 8192  1108   1457   2456
hipError_t launch_fp8_two(const Fp8Product& a, const Fp8Product& b) {
    const int64_t enough = a.cus * 5 / 8, ta = tiles(a, 256, 256), tb = tiles(b, 256, 256);
    if (kind(a) == kFew || kind(b) == kFew || a.nb == 0 || b.nb == 0 || ta + tb > (1 << 20)) {
        hipError_t e = launch_fp8_matmul(a);
        return e == hipSuccess ? launch_fp8_matmul(b) : e;
    }
    const Fp8Product p[2] = {a.nb >= b.nb ? a : b, a.nb >= b.nb ? b : a};
    int splits[2] = {1, 1};
    if (ta + tb >= enough && ta >= enough / 2 && tb >= enough / 2) return launch_kind(k256, p, 2, splits);
    if (tiles(a, 128, 128) + tiles(b, 128, 128) < enough) return launch_kind(k64, p, 2, splits);
    for (int q = 0; q < 2; ++q) splits[q] = p[q].parts ? splits_of(p[q], false) : 1;
    hipError_t e = launch_kind(k128, p, 2, splits);
    for (int q = 0; q < 2 && e == hipSuccess; ++q) e = join(p[q], splits[q]);
    return e;
}

}  // namespace fsdp
