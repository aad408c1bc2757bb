// fsdp_mx4.h -- internal interface between the host layer of the 4-bit
// microscaled blocks (fsdp_mx4_abi.cpp) and their kernels (fsdp_mx4.hip,
// fsdp_mx4_matmul.hip).  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fsdp_kernels.h"

namespace fsdp {

constexpr int kMx4Block = 32;                            // elements that share a scale
inline int64_t mx4_blocks(int64_t cols) { return (cols + kMx4Block - 1) / kMx4Block; }

// Tiles that blocks along the columns are made in; their number is held in 32 bits.
constexpr int kMx4Tile = 128;
constexpr int64_t kMx4MaxColTiles = int64_t(1) << 31;
inline int64_t mx4_col_tiles(int64_t rows, int64_t cols) {
    return ((rows + kMx4Tile - 1) / kMx4Tile) * ((cols + kMx4Tile - 1) / kMx4Tile);
}

struct Mx4Quant {
    const void* src;               // rows x cols, ld elements from row to row
    int dt;
    int64_t rows, cols, ld;
    uint8_t* codes;                // blocks along the rows, or null
    uint8_t* scales;
    uint8_t* codes_t;              // blocks along the columns, or null
    uint8_t* scales_t;
};
// With `also`, which has q's dt and as q blocks along the columns (and no others),
// that matrix too in the same launch.
hipError_t launch_mx4_quantize(const Mx4Quant& q, const Mx4Quant* also, void* stream);

struct Mx4Shards {
    const uint8_t* codes[FSDP_MAX_WORLD];
    const uint8_t* scales[FSDP_MAX_WORLD];
};
hipError_t launch_mx4_gather(const Mx4Shards& s, int world, int64_t S, int dt, void* out, void* stream);

struct Mx4Product {
    const uint8_t *a, *sa, *b, *sb;   // codes and scales of A [m][k] and B [n][k], blocks along k
    int64_t m, n, nb;                 // nb blocks of 32 along k
    int dt;
    void* out;                        // [m][n], ldo elements from row to row
    int64_t ldo;
    int cus;
    void* stream;
};
hipError_t launch_mx4_matmul(const Mx4Product& p);
hipError_t launch_mx4_two(const Mx4Product& a, const Mx4Product& b);   // both, in one launch where neither has few rows

constexpr int kMx4Few = 16;                              // most tokens of launch_mx4_few
// The product for a few tokens: x as it is, or in blocks (sx not null).
struct Mx4Few {
    const void* x;                 // [m][k] of xdt, ldx elements from row to row; or codes [m][nb * 16]
    const uint8_t* sx;             // scales [m][nb], or null
    int xdt;
    int64_t m, k, ldx;
    const uint8_t *w, *sw;         // codes and scales of W [n][k]
    int64_t n, nb;
    int dt;
    void* out;                     // [m][n], ldo elements from row to row
    int64_t ldo;
    int cus;
    void* stream;
};
hipError_t launch_mx4_few(const Mx4Few& p);

}  // namespace fsdp
