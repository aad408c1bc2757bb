// fsdp_fp8.h -- internal interface between the host layer of the 8-bit blocks
// (fsdp_fp8_abi.cpp) and their kernels (fsdp_fp8.hip, fsdp_fp8_matmul.hip).  Not
// installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fsdp_kernels.h"

namespace fsdp {

constexpr int kFp8Block = 128;                           // elements that share a scale, and the side of a tile
inline int64_t fp8_blocks(int64_t cols) { return (cols + kFp8Block - 1) / kFp8Block; }

// Tiles that blocks along the columns are made in; their number is held in 32 bits.
constexpr int64_t kFp8MaxTiles = int64_t(1) << 31;
inline int64_t fp8_tiles(int64_t rows, int64_t cols) { return fp8_blocks(rows) * fp8_blocks(cols); }

struct Fp8Quant {
    const void* src;               // rows x cols, ld elements from row to row
    int dt;
    int64_t rows, cols, ld;
    int tile;                      // a scale for 128 x 128
    uint8_t* codes;                // blocks along the rows, or null
    uint8_t* scales;
    uint8_t* codes_t;              // blocks along the columns, or null
    uint8_t* scales_t;
};
// With `also`, which has q's dt and as q blocks along the columns (and no others),
// neither in tiles, that matrix too in the same launch.
hipError_t launch_fp8_quantize(const Fp8Quant& q, const Fp8Quant* also, void* stream);

struct Fp8Shards {
    const uint8_t* codes[FSDP_MAX_WORLD];
    const uint8_t* scales[FSDP_MAX_WORLD];
};
hipError_t launch_fp8_gather(const Fp8Shards& s, int world, int64_t S, int dt, void* out, void* stream);

struct Fp8Product {
    const uint8_t *a, *sa, *b, *sb;   // codes and scales of A [m][k] and B [n][k], blocks along k
    int ta, tb;                       // log2 of the rows that share a scale: 0, or 7 for tiles
    int64_t m, n, nb;                 // nb blocks of 128 along k
    int dt;
    void* out;                        // [m][n], ldo elements from row to row
    int64_t ldo;
    int cus;
    void* stream;
    float* parts;                     // fp8_parts_bytes(m, n, nb, cus) bytes, or null where that is 0
};
hipError_t launch_fp8_matmul(const Fp8Product& p);
hipError_t launch_fp8_two(const Fp8Product& a, const Fp8Product& b);   // both, in one launch where neither has few rows
// Bytes of a product's partial sums, a multiple of 16: 0 where its sum is not split.
int64_t fp8_parts_bytes(int64_t m, int64_t n, int64_t nb, int cus);

constexpr int kFp8Few = 16;                              // most tokens of launch_fp8_few
// The product for a few tokens: x as it is, or in blocks (sx not null).
struct Fp8Few {
    const void* x;                 // [m][k] of xdt, ldx elements from row to row; or codes [m][nb * 128]
    const uint8_t* sx;             // scales [m >> tx][nb], or null
    int xdt, tx;
    int64_t m, k, ldx;
    const uint8_t *w, *sw;         // codes and scales of W [n][k]
    int tw;
    int64_t n, nb;
    int dt;
    void* out;                     // [m][n], ldo elements from row to row
    int64_t ldo;
    int cus;
    void* stream;
};
hipError_t launch_fp8_few(const Fp8Few& p);

}  // namespace fsdp
