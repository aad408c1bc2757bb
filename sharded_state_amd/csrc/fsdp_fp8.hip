// fsdp_fp8.hip -- gfx950 kernels that turn tensors into 8-bit blocks and back.
//
// A block is 128 consecutive elements (or a tile of 128 x 128) that share a power
// of two.  With a = max|x| of the block, e is the smallest whole number from -126
// on with a <= 448 * 2^e, and an element is the e4m3 number nearest to x / 2^e,
// ties to the even one; dividing by the power of two is exact, so every element is
// rounded once and none saturates.  The scale byte is e + 127.  A block that holds
// an infinity or a NaN gets byte 255 and codes 0 and stands for NaN.  The largest
// magnitude is found on the encodings (two 16-bit values an instruction).
// All of this is an HBM stream: 2 to 4 bytes in and 129/128 out an element.  Measured: rows,
// 107M fp32 elements 92 us (5.8 TB/s), bf16 57 (5.6); columns of 8192 x 10240 bf16 52 us
// (4.8), both 74 (4.5), in tiles 72 (4.7); 107M elements from each of 8 shards to bf16 400 us
// (6.4).  Codes are stored plainly, since most often a product reads them next: the hint for
// streams makes both forms of 4096 x 4096 bf16 14.3 us from 17.1, but with it the
// gradients of 1000 x 6400 x 1600, which quantise first, take 61.8 from 54.2.
#include <type_traits>

#include "fsdp_fp8_device.h"

#pragma clang fp contract(off)

namespace fsdp {

// Blocks along the rows: 16 lanes a block, eight elements a lane, kFp8RowsU blocks a
// lane with all loads first (107M elements with 1, 2 and 4: fp32 91.5, 95.2 and 98.0 us,
// bf16 60.3, 57.0 and 59.2); the largest magnitude goes round the 16 with four lane swaps.
template <int F> constexpr int kFp8RowsU = F == FSDP_F32 ? 1 : 2;
// I: what counts the blocks; 32 bits where they suffice, since a block's row is a division.
template <int F, typename I>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(const char* __restrict__ src, I total, int64_t cols, int64_t ld,
                                                       I nb, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kU = kFp8RowsU<F>;
    constexpr int kPer = kThreads / 16;                      // blocks of a workgroup's pass
    const int j = threadIdx.x & 15;
    for (I b0 = (I)blockIdx.x * (kPer * kU) + (threadIdx.x >> 4); b0 < total; b0 += (I)gridDim.x * (kPer * kU)) {
        Raw8<F> x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const I b = b0 + u * kPer;
            const I r = total == nb ? 0 : b / nb;
            const int64_t c = (int64_t)(b - r * nb) * kFp8Block + j * 8;
            x[u] = load_upto8<F>(src + ((int64_t)r * ld + c) * kEs, b < total ? cols - c : 0);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const I b = b0 + u * kPer;
            const uint32_t s = fp8_scale_byte(max_of_16(mag_bits<F>(max_mag<F>(0, x[u]))));
            const u32x2 w = fp8_codes8<F>(x[u], s);
            if (b < total) {
                reinterpret_cast<u32x2*>(codes)[(int64_t)b * 16 + j] = w;
                if (j == 0) scales[b] = (uint8_t)s;
            }
        }
    }
}

// Blocks along the columns (the rows of the transpose), and with ROWS along the
// rows too or instead, from one read: a workgroup brings a tile of 128 x 128
// elements, a lane 8 of a row at a time, all its loads first.  The rows' blocks are
// made from registers (16 lanes a block).  For the columns' the tile goes through
// LDS as it is; a lane takes 32 rows of two columns, the four lanes of a column
// agree on its scale through LDS, and its codes go through LDS once more, so that
// eight lanes store a column's 128 bytes.  TILE: one scale for all of it.
// Workgroups go to the XCDs in turn; XCD x takes one run of tiles down the columns,
// so that neighbouring tiles' scales, a byte a column each, meet in one L2.
constexpr int kSide = kFp8Block;
struct Fp8Cols {
    Fp8Quant q;
    uint32_t tiles_r, tiles;       // tiles down the rows, and in all
    uint32_t from;                 // the launch's first tile
};
template <int F> constexpr int kFp8TileLds = kSide * kSide * (F == FSDP_F32 ? 4 : 2);   // the tile, later its codes
constexpr int kCodePitch = kSide + 16;                       // bytes of a column's codes in LDS
static_assert(kSide * kCodePitch <= kFp8TileLds<FSDP_BF16>, "the codes take the tile's place");

template <int F, bool ROWS, bool COLS, bool TILE>
__device__ __forceinline__ void fp8_tile(const Fp8Cols& j, uint32_t b, uint8_t* lds, uint32_t* part) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kPass = kThreads / 16;                     // rows a pass
    constexpr int kN = kSide / kPass;
    const char* __restrict__ src = (const char*)j.q.src;
    const int64_t rows = j.q.rows, cols = j.q.cols, ld = j.q.ld;
    const uint32_t tiles_r = j.tiles_r, tiles = j.tiles;
    const uint32_t x = b & 7, per = tiles >> 3, more = tiles & 7;
    const uint32_t t = x * per + (x < more ? x : more) + (b >> 3);
    const int64_t tc = t / tiles_r, tr = t - (uint32_t)tc * tiles_r;
    const int64_t r0 = tr * kSide, c0 = tc * kSide;
    const int64_t nb = (cols + kSide - 1) / kSide, nbr = (rows + kSide - 1) / kSide;
    const int tid = threadIdx.x, lr = tid / 16, lc = tid % 16 * 8;

    Raw8<F> v[kN];
    const char* at = src + ((r0 + lr) * ld + c0 + lc) * kEs;
    if (r0 + kSide <= rows && c0 + kSide <= cols) {
#pragma unroll
        for (int q = 0; q < kN; ++q) v[q] = load8_raw<F>(at + q * (kPass * kEs) * ld);
    } else {
#pragma unroll
        for (int q = 0; q < kN; ++q)
            v[q] = load_upto8<F>(at + q * (kPass * kEs) * ld, r0 + q * kPass + lr < rows ? cols - c0 - lc : 0);
    }
    if constexpr (COLS) {
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            u32x4* o = reinterpret_cast<u32x4*>(lds + ((q * kPass + lr) * kSide + lc) * kEs);
#pragma unroll
            for (int k = 0; k < kEs / 2; ++k) o[k] = u32x4{v[q].w[4 * k], v[q].w[4 * k + 1], v[q].w[4 * k + 2], v[q].w[4 * k + 3]};
        }
    }
    uint32_t whole = 0;                                      // the tile's scale
    if constexpr (TILE) {
        uint32_t a = 0;
#pragma unroll
        for (int q = 0; q < kN; ++q) a = max_mag<F>(a, v[q]);
        a = max_of_16(mag_bits<F>(a));
        if (tid % 16 == 0) part[tid / 16] = a;
        __syncthreads();
        a = 0;
#pragma unroll
        for (int k = 0; k < kThreads / 16; ++k) a = max(a, part[k]);
        whole = fp8_scale_byte(a);
        if (tid == 0) {
            if (ROWS) j.q.scales[tr * nb + tc] = (uint8_t)whole;
            if (COLS) j.q.scales_t[tc * nbr + tr] = (uint8_t)whole;
        }
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            const int64_t r = r0 + q * kPass + lr;
            const uint32_t s = TILE ? whole : fp8_scale_byte(max_of_16(mag_bits<F>(max_mag<F>(0, v[q]))));
            const u32x2 w = fp8_codes8<F>(v[q], s);
            if (r < rows) {
                *reinterpret_cast<u32x2*>(j.q.codes + (r * nb + tc) * kSide + lc) = w;
                if (!TILE && tid % 16 == 0) j.q.scales[r * nb + tc] = (uint8_t)s;
            }
        }
    }
    if constexpr (COLS) {
        __syncthreads();
        const int cp = tid % (kSide / 2) * 2, rb = tid / (kSide / 2);
        Raw8<F> u[2][4];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const uint8_t* o = lds + ((rb * 32 + k) * kSide + cp) * kEs;
            if constexpr (F == FSDP_F32) {
                const u32x2 w0 = *reinterpret_cast<const u32x2*>(o), w1 = *reinterpret_cast<const u32x2*>(o + kSide * kEs);
                u[0][k / 8].w[k % 8] = w0.x;
                u[1][k / 8].w[k % 8] = w0.y;
                u[0][k / 8].w[k % 8 + 1] = w1.x;
                u[1][k / 8].w[k % 8 + 1] = w1.y;
            } else {
                const uint32_t w0 = *reinterpret_cast<const uint32_t*>(o);
                const uint32_t w1 = *reinterpret_cast<const uint32_t*>(o + kSide * kEs);
                u[0][k / 8].w[k % 8 / 2] = __builtin_amdgcn_perm(w1, w0, 0x05040100);    // low halves
                u[1][k / 8].w[k % 8 / 2] = __builtin_amdgcn_perm(w1, w0, 0x07060302);    // high halves
            }
        }
        if constexpr (!TILE) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t a = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) a = max_mag<F>(a, u[e][k]);
                part[rb * kSide + cp + e] = mag_bits<F>(a);
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t s = whole;
            if constexpr (!TILE) {
                const uint32_t* p = part + cp + e;
                s = fp8_scale_byte(max(max(p[0], p[kSide]), max(p[2 * kSide], p[3 * kSide])));
                if (rb == 0 && c0 + cp + e < cols) j.q.scales_t[(c0 + cp + e) * nbr + tr] = (uint8_t)s;
            }
            u32x2 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = fp8_codes8<F>(u[e][k], s);
            u32x4* o = reinterpret_cast<u32x4*>(lds + (cp + e) * kCodePitch + rb * 32);
            o[0] = u32x4{w[0].x, w[0].y, w[1].x, w[1].y};
            o[1] = u32x4{w[2].x, w[2].y, w[3].x, w[3].y};
        }
        __syncthreads();
#pragma unroll
        for (int i = tid; i < kSide * 8; i += kThreads) {
            const int64_t c = c0 + i / 8;
            if (c < cols)
                *reinterpret_cast<u32x4*>(j.q.codes_t + (c * nbr + tr) * kSide + i % 8 * 16) =
                    *reinterpret_cast<const u32x4*>(lds + i / 8 * kCodePitch + i % 8 * 16);
        }
    }
}

// With PAIR a second matrix's columns in the same launch, from the next multiple
// of 8 workgroups on (a linear layer's gradients take both operands' at once).
template <int F, bool ROWS, bool COLS, bool TILE, bool PAIR>
__global__ __launch_bounds__(kThreads) void k_fp8_tiles(Fp8Cols a, Fp8Cols also) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[COLS ? kFp8TileLds<F> : 16];
    __shared__ uint32_t part[COLS && !TILE ? 4 * kSide : kThreads / 16];
    const uint32_t first = (a.tiles + 7) & ~7u;
    if constexpr (!PAIR) {
        fp8_tile<F, ROWS, COLS, TILE>(a, a.from + blockIdx.x, lds, part);
    } else if (blockIdx.x < first) {
        if (blockIdx.x < a.tiles) fp8_tile<F, ROWS, COLS, TILE>(a, blockIdx.x, lds, part);
    } else {
        fp8_tile<F, false, true, TILE>(also, blockIdx.x - first, lds, part);
    }
}

// The all-gather of quantised shards into the full buffer of format F: a lane
// makes two 16-byte vectors (8 elements of a 16-bit format, 4 of fp32), loads first.  With WIDE every slot starts on the 16-byte grid
// and a wave's stores go out as one span with the streamed policy (fsdp_device.h);
// otherwise slots begin wherever q * S puts them, and stores take any address.  With 1, 2
// and 4 vectors: 8 x 107M elements to bf16 409, 402 and 413 us, 2 x 15.4M to fp16 13.7, 13.2
// and 12.8, 2 x 50M to fp32 70.4, 70.9 and 72.2.
constexpr int kFp8GatherU = 2;
template <int F, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_fp8_gather(Fp8Shards sh, int64_t S, char* __restrict__ out) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int kE = 16 / kEs;                             // elements of a vector
    typedef typename std::conditional<kE == 8, u32x2, uint32_t>::type Codes;
    constexpr int kU = kFp8GatherU;
    const int q = blockIdx.y;
    const Codes* codes = reinterpret_cast<const Codes*>(sh.codes[q]);
    const uint8_t* scales = sh.scales[q];
    const int64_t nv = (S + kE - 1) / kE;
    for (int64_t v0 = (int64_t)blockIdx.x * (kThreads * kU) + threadIdx.x; v0 < nv;
         v0 += (int64_t)gridDim.x * (kThreads * kU)) {
        Codes w[kU];
        uint32_t sb[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t v = v0 + u * kThreads, i = v < nv ? v : nv - 1;
            w[u] = codes[i];
            sb[u] = scales[i / (kFp8Block / kE)];
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t v = v0 + u * kThreads;
            if (v >= nv) break;
            const float f = from_codes(sb[u]);
            float x[kE];
#pragma unroll
            for (int k = 0; k < kE / 4; ++k) {
                uint32_t d;
                if constexpr (kE == 8) d = w[u][k];
                else d = w[u];
                const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(d, 1.0f, 0);
                const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(d, 1.0f, 1);
                x[4 * k] = y0.x * f; x[4 * k + 1] = y0.y * f;
                x[4 * k + 2] = y1.x * f; x[4 * k + 3] = y1.y * f;
            }
            // kept apart from the conversion: fused with it the compiler adds +0 and -0 loses its sign
            if constexpr (F == FSDP_F16) {
#pragma unroll
                for (int k = 0; k < kE; ++k) asm("" : "+v"(x[k]));
            }
            const int64_t i = (int64_t)q * S + v * kE;
            char* o = out + i * kEs;
            if (v * kE + kE <= S) {
                u32x4 a;
                if constexpr (F == FSDP_F32) {
                    a = u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) a[k] = from_f32<F>(x[2 * k]) | (from_f32<F>(x[2 * k + 1]) << 16);
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

// Workgroups of a launch in tiles, a multiple of 8: fewer than 2^32 work items.
constexpr int64_t kMaxTiles = (1 << 23) - 8;

static Fp8Cols tiles_job(const Fp8Quant& q) {
    return Fp8Cols{q, (uint32_t)fp8_blocks(q.rows), (uint32_t)fp8_tiles(q.rows, q.cols), 0};
}

template <int F, bool ROWS, bool COLS, bool TILE>
static hipError_t in_tiles(const Fp8Quant& q, const Fp8Quant* also, hipStream_t st) {
    Fp8Cols a = tiles_job(q), b{};
    if constexpr (COLS && !TILE) {
        if (also) {
            b = tiles_job(*also);
            const int64_t both = ((int64_t)a.tiles + 7) / 8 * 8 + b.tiles;
            if (both <= kMaxTiles) {
                launch(k_fp8_tiles<F, ROWS, COLS, TILE, true>, dim3((unsigned)both), dim3(kThreads), st, a, b);
                return hipGetLastError();
            }
        }
    }
    for (int64_t t = 0; t < a.tiles; t += kMaxTiles) {
        a.from = (uint32_t)t;
        launch(k_fp8_tiles<F, ROWS, COLS, TILE, false>, dim3((unsigned)(a.tiles - t < kMaxTiles ? a.tiles - t : kMaxTiles)),
               dim3(kThreads), st, a, b);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return also ? launch_fp8_quantize(*also, nullptr, st) : hipSuccess;
}

template <int F>
static hipError_t quantize(const Fp8Quant& q, const Fp8Quant* also, hipStream_t st) {
    if (q.tile) {
        if (q.codes && q.codes_t) return in_tiles<F, true, true, true>(q, also, st);
        return q.codes ? in_tiles<F, true, false, true>(q, also, st) : in_tiles<F, false, true, true>(q, also, st);
    }
    if (q.codes_t) return q.codes ? in_tiles<F, true, true, false>(q, also, st) : in_tiles<F, false, true, false>(q, also, st);
    int64_t rows = q.rows, cols = q.cols;
    if (q.ld == cols && cols % kFp8Block == 0) {      // whole blocks row after row: one long row
        cols *= rows;
        rows = 1;
    }
    const char* src = (const char*)q.src;
    const int64_t nb = fp8_blocks(cols), total = rows * nb;
    const dim3 g(capped((total * 16 + kThreads * kFp8RowsU<F> - 1) / (kThreads * kFp8RowsU<F>))), th(kThreads);
    if (total < INT32_MAX / 2) launch(k_fp8_rows<F, uint32_t>, g, th, st, src, (uint32_t)total, cols, q.ld, (uint32_t)nb, q.codes, q.scales);
    else launch(k_fp8_rows<F, int64_t>, g, th, st, src, total, cols, q.ld, nb, q.codes, q.scales);
    return hipGetLastError();
}

hipError_t launch_fp8_quantize(const Fp8Quant& q, const Fp8Quant* also, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (q.dt == FSDP_F32) return quantize<FSDP_F32>(q, also, st);
    if (q.dt == FSDP_F16) return quantize<FSDP_F16>(q, also, st);
    return quantize<FSDP_BF16>(q, also, st);
}

template <int F>
static void gather(const Fp8Shards& s, int world, int64_t S, char* out, hipStream_t st) {
    constexpr int kE = F == FSDP_F32 ? 4 : 8;
    const int64_t per = ((S + kE - 1) / kE + kThreads * kFp8GatherU - 1) / (kThreads * kFp8GatherU), cap = (1 << 22) / world;
    const dim3 g((unsigned)(per < cap ? per : cap), (unsigned)world), th(kThreads);
    if (((uintptr_t)out & 15) == 0 && S % kE == 0) launch(k_fp8_gather<F, true>, g, th, st, s, S, out);
    else launch(k_fp8_gather<F, false>, g, th, st, s, S, out);
}

hipError_t launch_fp8_gather(const Fp8Shards& s, int world, int64_t S, int dt, void* out, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (dt == FSDP_F32) gather<FSDP_F32>(s, world, S, (char*)out, st);
    else if (dt == FSDP_F16) gather<FSDP_F16>(s, world, S, (char*)out, st);
    else gather<FSDP_BF16>(s, world, S, (char*)out, st);
    return hipGetLastError();
}

}  // namespace fsdp
