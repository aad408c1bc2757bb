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
// zeros gets byte 0.  The largest magnitude is found on the encodings (two
// 16-bit values an instruction), and the elements are divided and rounded by
// gfx950's conversion, two an instruction (fsdp_mx4_device.h).
// All of this is an HBM stream: 2 to 4 bytes in and 17/32 out an element.
#include <type_traits>

#include "fsdp_mx4_device.h"

#pragma clang fp contract(off)

namespace fsdp {

// Blocks along the rows: four lanes a block, eight elements a lane, kRowsU
// blocks a lane with all loads first; the block's largest magnitude goes round
// the four with two lane swaps.  106.8M elements, us by blocks a lane (1, 2,
// 4): bf16 50.4, 46.4 (5.83 TB/s), 48.1; fp32 82.4 (5.88 TB/s), 87.1, 89.6.
template <int F> constexpr int kRowsU = F == FSDP_F32 ? 1 : 2;
template <int F>
__global__ __launch_bounds__(kThreads) void k_mx4_rows(const char* __restrict__ src, int64_t rows, int64_t cols,
                                                       int64_t ld, int64_t nb, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kU = kRowsU<F>;
    constexpr int kPer = kThreads / 4;                       // blocks of a workgroup's pass
    const int64_t total = rows * nb;
    const int j = threadIdx.x & 3;
    for (int64_t b0 = (int64_t)blockIdx.x * (kPer * kU) + (threadIdx.x >> 2); b0 < total;
         b0 += (int64_t)gridDim.x * (kPer * kU)) {
        Raw8<F> x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t b = b0 + u * kPer;
            const int64_t r = rows == 1 ? 0 : b / nb;
            const int64_t c = (b - r * nb) * kMx4Block + j * 8;
            x[u] = load_upto8<F>(src + (r * ld + c) * kEs, b < total ? cols - c : 0);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t b = b0 + u * kPer;
            const uint32_t s = scale_byte(max_of_four(mag_bits<F>(max_mag<F>(0, x[u]))));
            const uint32_t w = codes8<F>(x[u], s);
            if (b < total) {
                reinterpret_cast<uint32_t*>(codes)[b * 4 + j] = w;
                if (j == 0) scales[b] = (uint8_t)s;
            }
        }
    }
}

// Blocks along the columns (the rows of the transpose), and with ROWS along the
// rows too, from one read: a workgroup brings kTile x kTile elements, a lane 8
// of a row at a time.  The rows' blocks are made from registers (four lanes a
// block); for the columns' the tile goes through LDS as it is, and a lane takes
// two columns of 32 rows, one read a row pair.  Workgroups go to the XCDs in
// turn; XCD x takes one run of tiles down the columns, so what neighbouring
// tiles write to a line of the transpose (64 bytes of codes, 4 of scales each)
// meets in one L2.  A lane's eight loads stand under conditions of their own, each
// waited for before the next: that, not the memory, bounds it (8192 x 10240 bf16 47.6
// us, 4.5 TB/s).
constexpr int kTile = kMx4Tile;
struct Mx4Cols {
    Mx4Quant q;
    uint32_t tiles_r, tiles;       // tiles down the rows, and in all
    uint32_t from;                 // the launch's first tile
};
// Tile number `b` of job `j`, in the order of the launch.
template <int F, bool ROWS>
__device__ __forceinline__ void cols_tile(const Mx4Cols& j, uint32_t b, uint8_t* lds) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kPass = kThreads / (kTile / 8);            // rows a pass
    const char* __restrict__ src = (const char*)j.q.src;
    const int64_t rows = j.q.rows, cols = j.q.cols, ld = j.q.ld;
    uint8_t *__restrict__ codes = j.q.codes, *__restrict__ scales = j.q.scales;
    uint8_t *__restrict__ codes_t = j.q.codes_t, *__restrict__ scales_t = j.q.scales_t;
    const uint32_t tiles_r = j.tiles_r, tiles = j.tiles;
    const uint32_t x = b & 7, per = tiles >> 3, more = tiles & 7;
    const uint32_t t = x * per + (x < more ? x : more) + (b >> 3);
    // Tiles go down the rows; with the row form too, kPair columns of them together,
    // so that a row's stores of neighbouring tiles meet in the L2 (bf16 8192 x 10240:
    // 61.6 us, one column at a time 63.3; fp32 110 and 115).  The transpose alone
    // gains nothing by it; four together cost it 20% at 8192 x 8191.
    constexpr uint32_t kPair = ROWS ? 2 : 1;
    const uint32_t tiles_c = tiles / tiles_r, gr = t / (tiles_r * kPair), in = t - gr * tiles_r * kPair;
    const uint32_t gw = kPair == 2 && tiles_c - gr * 2 > 1 ? 2 : 1;
    const int64_t r0 = (int64_t)(in / gw) * kTile, c0 = (int64_t)(gr * kPair + in % gw) * kTile;
    const int64_t nb = (cols + kMx4Block - 1) / kMx4Block, nbr = (rows + kMx4Block - 1) / kMx4Block;
    const int lr = threadIdx.x / (kTile / 8), lc = threadIdx.x % (kTile / 8) * 8;
#pragma unroll
    for (int q = 0; q < kTile / kPass; ++q) {
        const int64_t r = r0 + q * kPass + lr, c = c0 + lc;
        const Raw8<F> v = load_upto8<F>(src + (r * ld + c) * kEs, r < rows ? cols - c : 0);
        u32x4* o = reinterpret_cast<u32x4*>(lds + ((q * kPass + lr) * kTile + lc) * kEs);
#pragma unroll
        for (int j = 0; j < kEs / 2; ++j) o[j] = u32x4{v.w[4 * j], v.w[4 * j + 1], v.w[4 * j + 2], v.w[4 * j + 3]};
        if constexpr (ROWS) {
            const uint32_t s = scale_byte(max_of_four(mag_bits<F>(max_mag<F>(0, v))));
            const uint32_t w = codes8<F>(v, s);
            if (r < rows && (c >> 5) < nb) {
                const int64_t b = r * nb + (c >> 5);
                reinterpret_cast<uint32_t*>(codes)[b * 4 + (threadIdx.x & 3)] = w;
                if ((threadIdx.x & 3) == 0) scales[b] = (uint8_t)s;
            }
        }
    }
    __syncthreads();
    const int cp = threadIdx.x % (kTile / 2) * 2, rb = threadIdx.x / (kTile / 2);
    Raw8<F> v[2][4];
#pragma unroll
    for (int k = 0; k < kMx4Block; k += 2) {
        const uint8_t* o = lds + ((rb * kMx4Block + k) * kTile + cp) * kEs;
        if constexpr (F == FSDP_F32) {
            const u32x2 w0 = *reinterpret_cast<const u32x2*>(o), w1 = *reinterpret_cast<const u32x2*>(o + kTile * kEs);
            v[0][k / 8].w[k % 8] = w0.x;
            v[1][k / 8].w[k % 8] = w0.y;
            v[0][k / 8].w[k % 8 + 1] = w1.x;
            v[1][k / 8].w[k % 8 + 1] = w1.y;
        } else {
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(o);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(o + kTile * kEs);
            v[0][k / 8].w[k % 8 / 2] = __builtin_amdgcn_perm(w1, w0, 0x05040100);    // low halves
            v[1][k / 8].w[k % 8 / 2] = __builtin_amdgcn_perm(w1, w0, 0x07060302);    // high halves
        }
    }
    // The tile's codes of a column are 64 bytes of the transpose, its scales 4:
    // they go through LDS once more, so that four lanes store a column's codes and
    // one its scales (8192 x 10240 bf16: 47.6 us; with 16 bytes and 1 byte stored by
    // each lane 59.4).  A padded row a row block keeps the four lanes' banks apart.
    constexpr int kPitch = kTile * 16 + 64;
    __syncthreads();
    uint8_t* sc = lds + 4 * kPitch;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = max_mag<F>(a, v[e][j]);
        const uint32_t s = scale_byte(mag_bits<F>(a));
        *reinterpret_cast<u32x4*>(lds + rb * kPitch + (cp + e) * 16) =
            u32x4{codes8<F>(v[e][0], s), codes8<F>(v[e][1], s), codes8<F>(v[e][2], s), codes8<F>(v[e][3], s)};
        sc[(cp + e) * 4 + rb] = (uint8_t)s;
    }
    __syncthreads();
    const int64_t b0 = r0 / kMx4Block;
    const int blocks = (int)(nbr - b0 < 4 ? nbr - b0 : 4);
#pragma unroll
    for (int i = threadIdx.x; i < kTile * 4; i += kThreads) {
        const int64_t c = c0 + i / 4;
        if (c < cols && i % 4 < blocks)
            reinterpret_cast<u32x4*>(codes_t)[c * nbr + b0 + i % 4] =
                *reinterpret_cast<const u32x4*>(lds + i % 4 * kPitch + i / 4 * 16);
    }
    if (threadIdx.x < kTile && c0 + threadIdx.x < cols) {
        const int64_t at = (c0 + threadIdx.x) * nbr + b0;
        if (blocks == 4) {
            *(u32_any*)(scales_t + at) = *reinterpret_cast<const uint32_t*>(sc + threadIdx.x * 4);
        } else {
            for (int k = 0; k < blocks; ++k) scales_t[at + k] = sc[threadIdx.x * 4 + k];
        }
    }
}

// With PAIR a second matrix's columns in the same launch, from the next multiple
// of 8 workgroups on (a linear layer's gradients take both operands' at once).
template <int F, bool ROWS, bool PAIR>
__global__ __launch_bounds__(kThreads) void k_mx4_cols(Mx4Cols a, Mx4Cols also) {
    // the tile as it is, later its codes (8.8 KB)
    __shared__ __attribute__((aligned(16))) uint8_t lds[kTile * kTile * (F == FSDP_F32 ? 4 : 2)];
    const uint32_t first = (a.tiles + 7) & ~7u;
    if constexpr (!PAIR) {
        cols_tile<F, ROWS>(a, a.from + blockIdx.x, lds);
    } else if (blockIdx.x < first) {
        if (blockIdx.x < a.tiles) cols_tile<F, ROWS>(a, blockIdx.x, lds);
    } else {
        cols_tile<F, false>(also, blockIdx.x - first, lds);
    }
}

// The all-gather of quantised shards into the full buffer of format F: a lane
// makes two 16-byte vectors of a 16-bit format (8 elements each) or four of
// fp32 (4 elements each), loads first.  With WIDE every slot starts on the 16-byte grid and a wave's
// stores go out as one span with the streamed policy (fsdp_device.h); otherwise
// slots begin wherever q * S puts them, and stores take any address.  Eight
// shards of 106.8M elements, us by vectors a lane (1, 2, 4): bf16 423, 327
// (6.61 TB/s), 370; fp32 819, 652, 604 (6.42 TB/s).
template <int F> constexpr int kGatherU = F == FSDP_F32 ? 4 : 2;
template <int F, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_mx4_gather(Mx4Shards sh, int64_t S, char* __restrict__ out) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kE = 16 / kEs;                             // elements of a vector
    typedef typename std::conditional<kE == 8, uint32_t, uint16_t>::type Codes;
    constexpr int kU = kGatherU<F>;
    const int q = blockIdx.y;
    const Codes* codes = reinterpret_cast<const Codes*>(sh.codes[q]);
    const uint8_t* scales = sh.scales[q];
    const int64_t nv = (S + kE - 1) / kE;
    for (int64_t v0 = (int64_t)blockIdx.x * (kThreads * kU) + threadIdx.x; v0 < nv;
         v0 += (int64_t)gridDim.x * (kThreads * kU)) {
        uint32_t w[kU], sb[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t v = v0 + u * kThreads;
            w[u] = v < nv ? codes[v] : 0;
            sb[u] = v < nv ? scales[v / (kMx4Block / kE)] : 0;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t v = v0 + u * kThreads;
            if (v >= nv) break;
            const float f = from_codes(sb[u]);
            const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0);
            const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
            const f32x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2);
            const f32x2 y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3);
            float x[8] = {y0.x * f, y0.y * f, y1.x * f, y1.y * f, y2.x * f, y2.y * f, y3.x * f, y3.y * f};
            // kept apart from the conversion: fused with it the compiler adds +0 and -0 loses its sign
            if constexpr (F == FSDP_F16) {
#pragma unroll
                for (int k = 0; k < 8; ++k) asm("" : "+v"(x[k]));
            }
            const int64_t i = (int64_t)q * S + v * kE;
            char* o = out + i * kEs;
            if (v * kE + kE <= S) {
                u32x4 a;
                if constexpr (F == FSDP_F32) {
                    a.x = __float_as_uint(x[0]); a.y = __float_as_uint(x[1]);
                    a.z = __float_as_uint(x[2]); a.w = __float_as_uint(x[3]);
                } else {
                    a.x = from_f32<F>(x[0]) | (from_f32<F>(x[1]) << 16);
                    a.y = from_f32<F>(x[2]) | (from_f32<F>(x[3]) << 16);
                    a.z = from_f32<F>(x[4]) | (from_f32<F>(x[5]) << 16);
                    a.w = from_f32<F>(x[6]) | (from_f32<F>(x[7]) << 16);
                }
                if constexpr (WIDE) {
                    const int l = (int)(threadIdx.x & 63);
                    st16_wave(o - 16 * l, l, a);
                } else {
                    *(u32x4_any*)o = a;
                }
            } else {
#pragma unroll
                for (int k = 0; k < kE; ++k)
                    if (v * kE + k < S) store1<F>(out, i + k, x[k]);
            }
        }
    }
}

// ----------------------------------------------------------------- launchers
// A launch holds fewer than 2^32 work items; beyond 2^22 workgroups they loop.
static unsigned capped(int64_t want) {
    const int64_t cap = 1 << 22;
    return (unsigned)(want < 1 ? 1 : (want < cap ? want : cap));
}

// Workgroups of a column launch, a multiple of 8: fewer than 2^32 work items.
constexpr int64_t kMaxTiles = (1 << 23) - 8;

static Mx4Cols cols_job(const Mx4Quant& q) {
    return Mx4Cols{q, (uint32_t)((q.rows + kTile - 1) / kTile), (uint32_t)mx4_col_tiles(q.rows, q.cols), 0};
}

template <int F>
static hipError_t quantize(const Mx4Quant& q, const Mx4Quant* also, hipStream_t st) {
    const char* src = (const char*)q.src;
    const dim3 th(kThreads);
    if (q.codes_t) {
        Mx4Cols a = cols_job(q), b{};
        if (also) b = cols_job(*also);
        const int64_t both = ((int64_t)a.tiles + 7) / 8 * 8 + b.tiles;
        if (also && both <= kMaxTiles) {
            if (q.codes) launch(k_mx4_cols<F, true, true>, dim3((unsigned)both), th, st, a, b);
            else launch(k_mx4_cols<F, false, true>, dim3((unsigned)both), th, st, a, b);
            return hipGetLastError();
        }
        for (int64_t t = 0; t < a.tiles; t += kMaxTiles) {
            const dim3 g((unsigned)(a.tiles - t < kMaxTiles ? a.tiles - t : kMaxTiles));
            a.from = (uint32_t)t;
            if (q.codes) launch(k_mx4_cols<F, true, false>, g, th, st, a, b);
            else launch(k_mx4_cols<F, false, false>, g, th, st, a, b);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return also ? quantize<F>(*also, nullptr, st) : hipSuccess;
    }
    int64_t rows = q.rows, cols = q.cols;
    if (q.ld == cols && cols % kMx4Block == 0) {      // whole blocks row after row: one long row
        cols *= rows;
        rows = 1;
    }
    const int64_t nb = mx4_blocks(cols);
    launch(k_mx4_rows<F>, dim3(capped((rows * nb * 4 + kThreads * kRowsU<F> - 1) / (kThreads * kRowsU<F>))), th, st,
           src, rows, cols, q.ld, nb, q.codes, q.scales);
    return hipGetLastError();
}

hipError_t launch_mx4_quantize(const Mx4Quant& q, const Mx4Quant* also, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (q.dt == FSDP_F32) return quantize<FSDP_F32>(q, also, st);
    if (q.dt == FSDP_F16) return quantize<FSDP_F16>(q, also, st);
    return quantize<FSDP_BF16>(q, also, st);
}

template <int F>
static void gather(const Mx4Shards& s, int world, int64_t S, char* out, hipStream_t st) {
    constexpr int kE = F == FSDP_F32 ? 4 : 8;
    const int64_t per = ((S + kE - 1) / kE + kThreads * kGatherU<F> - 1) / (kThreads * kGatherU<F>), cap = (1 << 22) / world;
    const dim3 g((unsigned)(per < cap ? per : cap), (unsigned)world), th(kThreads);
    if (((uintptr_t)out & 15) == 0 && S % kE == 0) launch(k_mx4_gather<F, true>, g, th, st, s, S, out);
    else launch(k_mx4_gather<F, false>, g, th, st, s, S, out);
}

hipError_t launch_mx4_gather(const Mx4Shards& s, int world, int64_t S, int dt, void* out, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (dt == FSDP_F32) gather<FSDP_F32>(s, world, S, (char*)out, st);
    else if (dt == FSDP_F16) gather<FSDP_F16>(s, world, S, (char*)out, st);
    else gather<FSDP_BF16>(s, world, S, (char*)out, st);
    return hipGetLastError();
}

}  // namespace fsdp
