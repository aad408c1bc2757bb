// fsdp_mx4_tiles.h -- the tiled product of two matrices of 4-bit microscaled
// blocks (fsdp_mx4_matmul.hip instantiates it).  Not installed.
#pragma once

#include <type_traits>

#include "fsdp_mx4_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kFp4 = 4;     // the instruction's code for 4-bit elements
constexpr int kAnyFormat = -1;   // the results' format is p.dt

// Where the tile that workgroup `b` of a product takes lies.  Workgroups go to
// the 8 XCDs in turn, each with an L2 of its own: XCD x takes one run of
// consecutive tiles, and a run walks groups of 4 tile rows column by column,
// so the 32 tiles that an XCD works on at a time share 4 panels of A and 8 of B.
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t tiles = tiles_m * tiles_n;
    const uint32_t x = b & 7, per = tiles >> 3, more = tiles & 7;
    const uint32_t t = x * per + (x < more ? x : more) + (b >> 3);
    const uint32_t g = t / (4 * tiles_n), in = t - g * 4 * tiles_n;
    const uint32_t rows = tiles_m - g * 4 < 4 ? tiles_m - g * 4 : 4;
    tm = g * 4 + in % rows;
    tn = in / rows;
}

// BM x BN results a workgroup of WM x WN waves, BM / WM x BN / WN a wave.  A stage
// is 8 blocks of 32 (a row's 128 bytes, one cache line) of every row; NS stages
// are in LDS, NS - 1 of them on their way.
template <int F, int BM, int BN, int WM, int WN, int NS>
__device__ __forceinline__ void mx4_tile(const Mx4Product& p, uint32_t tiles_m, uint32_t tiles_n, uint32_t block) {
    constexpr int KB = 8;
    constexpr int kWaves = WM * WN;
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;     // fragments of 32 rows a wave
    constexpr int kSteps = KB / 2;                           // steps of 64 along k
    constexpr int kRow = KB * 16;                            // bytes of a row's stage
    constexpr int kLoads = (BM + BN) * KB / 64 / kWaves;     // 1 KB loads a wave a stage
    constexpr int kLoadsA = BM * KB / 64 / kWaves;
    constexpr int kStep = kWaves * 64 / KB;                  // rows from one load of a wave to its next
    constexpr int kStage = (BM + BN) * kRow;
    constexpr int kOutRow = FN * 32 * (F == FSDP_F32 || F == kAnyFormat ? 4 : 2) + 16;   // a result row in LDS, padded
    constexpr int kThreadsWg = 64 * kWaves;
    constexpr int kRows = (BM + BN + kThreadsWg - 1) / kThreadsWg;
    constexpr int kScales = NS * kStage;                     // where the scales lie: 2 x (BM + BN) rows of 16 bytes
    static_assert(kLoadsA * 64 * kWaves == BM * KB && kLoads * 64 * kWaves == (BM + BN) * KB, "whole loads");
    static_assert(WM * WN * 32 * kOutRow <= kScales, "results pass through the stages' LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kScales + 2 * (BM + BN) * 16];

    uint32_t tm, tn;
    tile_of(block, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rows_a = (int)(p.m - m0 < BM ? p.m - m0 : BM), rows_b = (int)(p.n - n0 < BN ? p.n - n0 : BN);
    const int l = threadIdx.x & 63, h = l >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = (int)p.nb, rowbytes = nb * 16;
    const int nk = (nb + KB - 1) / KB;

    // Chunk c (16 bytes: one block) of row r lies at slot c ^ turn(r) of the
    // row's stage: 16 rows' equal chunks then lie in 16 places of the 256 bytes
    // that the banks span.
    auto turn = [](int r) { return (r >> 1) & 7; };

    // Global to LDS: a wave's load fills 1 KB, lane l the 16 bytes at 16 l.  Rows
    // behind the matrix read its last row, blocks behind a row its first one of
    // the stage: what they bring is not stored, or meets scales that take it to 0.
    const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + m0 * rowbytes), 0, rows_a * rowbytes, kRsrcWord3);
    const auto rb = __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + n0 * rowbytes), 0, rows_b * rowbytes, kRsrcWord3);
    const int lrow = (w * 64 + l) / KB;                      // row of load 0; kStep is a multiple of 16
    const int lchunk = ((w * 64 + l) % KB) ^ turn(lrow);
    static_assert(kStep % 16 == 0, "the slots' turn repeats from load to load");
    int voff[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = lrow + (i < kLoadsA ? i : i - kLoadsA) * kStep;
        const int lim = i < kLoadsA ? rows_a : rows_b;
        voff[i] = (r < lim ? r : lim - 1) * rowbytes;
    }
    // Part `part` of `parts` of the loads of stage kt.
    auto load_part = [&](int kt, int part, int parts) {
        const int left = nb - kt * KB;
        const int c = (lchunk < left ? lchunk : 0) * 16;
        const int soff = __builtin_amdgcn_readfirstlane(kt * kRow);
        uint8_t* to = lds + kt % NS * kStage + w * 1024;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (i * parts / kLoads != part) continue;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                i < kLoadsA ? ra : rb, (__attribute__((address_space(3))) void*)(to + i * kWaves * 1024), 16,
                voff[i] + c, soff, 0, 0);
        }
    };

    // Scales: a lane fetches a row's 16 bytes of two stages at once and puts them
    // into LDS, where the waves that share the row read them.  Fetched by each
    // wave for its own fragments they cost more requests than the codes (the
    // address unit 74% busy at 256 x 256; 388 -> 341 us at 8192 x 8192 x 10240).
    // Behind the last block both sides get 2^-127, and what the codes there
    // multiply to vanishes.
    auto fetch_scales = [&](u32x4 (&s)[kRows], int g) {
        const int b0 = g * 16;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = i * kThreadsWg + (int)threadIdx.x;
            if ((i + 1) * kThreadsWg > BM + BN && r >= BM + BN) break;
            const uint8_t* q = r < BM ? p.sa + (m0 + (r < rows_a ? r : rows_a - 1)) * nb
                                      : p.sb + (n0 + (r - BM < rows_b ? r - BM : rows_b - 1)) * nb;
            s[i] = scales16(q + b0, nb - b0);
        }
    };
    auto put_scales = [&](const u32x4 (&s)[kRows], int g) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = i * kThreadsWg + (int)threadIdx.x;
            if ((i + 1) * kThreadsWg > BM + BN && r >= BM + BN) break;
            *reinterpret_cast<u32x4*>(lds + kScales + ((g & 1) * (BM + BN) + r) * 16) = s[i];
        }
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{0};

    const int wm = w / WN, wn = w % WN;
    const int arow = (wm * FM * 32 + (l & 31)) * kRow, brow = (BM + wn * FN * 32 + (l & 31)) * kRow;
    const int tl = turn(l & 31);                             // fragments start at multiples of 32 rows
    const int srow = kScales + (wm * FM * 32 + (l & 31)) * 16, trow = kScales + (BM + wn * FN * 32 + (l & 31)) * 16;
    // a lane needs the scales of its half h: bytes h and h + 2 of a dword for two steps
    const int shift = 8 * h;
    constexpr int kDwords = kSteps / 2;

    u32x4 scales[kRows];
    // Stage kt.  `more`: a stage is left to be loaded while this one is worked on.
    auto stage = [&](int kt, auto more) {
        constexpr bool kMore = decltype(more)::value;
        // Wait for this stage's loads: those of the stages behind it (and no scales) may be on their way.
        if (NS > 2 && kMore) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * kLoads) : "memory");
        else if (NS > 3 && kt + 2 < nk) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLoads) : "memory");
        else if (NS > 2 && kt + 1 < nk) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (kt % 2 == 0) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) asm volatile("" : "+v"(scales[i]));    // not before the wait
            put_scales(scales, kt / 2);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        // every wave's part has arrived, and nobody reads the stage before any more
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt % 2 == 0 && kt + 2 < nk) fetch_scales(scales, kt / 2 + 1);
        const uint8_t* base = lds + kt % NS * kStage;
        const int soff = (kt / 2 & 1) * (BM + BN) * 16 + kt % 2 * 8;
        int sa[FM][kDwords], sb[FN][kDwords];
#pragma unroll
        for (int d = 0; d < kDwords; ++d) {
#pragma unroll
            for (int f = 0; f < FM; ++f)
                sa[f][d] = (int)(*reinterpret_cast<const uint32_t*>(lds + srow + f * 512 + soff + d * 4) >> shift);
#pragma unroll
            for (int f = 0; f < FN; ++f)
                sb[f][d] = (int)(*reinterpret_cast<const uint32_t*>(lds + trow + f * 512 + soff + d * 4) >> shift);
        }
        // A step's instructions go out in rows of FN; between the rows, and kept
        // there, the next step's fragments are read and the next stage's loads sent.
        i32x8 a[2][FM], b[2][FN];
        auto read_a = [&](int s, int f) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(base + arow + f * 32 * kRow +
                                                            ((2 * s + h) ^ tl) * 16);
            a[s & 1][f] = i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        };
        auto read_b = [&](int s, int f) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(base + brow + f * 32 * kRow +
                                                            ((2 * s + h) ^ tl) * 16);
            b[s & 1][f] = i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        };
#pragma unroll
        for (int f = 0; f < FN; ++f) read_b(0, f);
        read_a(0, 0);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (s == 0 && i + 1 < FM) read_a(0, i + 1);
                if (s + 1 < kSteps) {
#pragma unroll
                    for (int f = 0; f < FM + FN; ++f)
                        if (f * FM / (FM + FN) == i) {
                            if (f < FN) read_b(s + 1, f);
                            else read_a(s + 1, f - FN);
                        }
                }
                if (kMore) load_part(kt + NS - 1, s * FM + i, kSteps * FM);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    // rows of B first: a lane then holds runs of four results of one row of A
                    if (s & 1)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            b[1][j], a[1][i], acc[i][j], kFp4, kFp4, 2, sb[j][s / 2], 2, sa[i][s / 2]);
                    else
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            b[0][j], a[0][i], acc[i][j], kFp4, kFp4, 0, sb[j][s / 2], 0, sa[i][s / 2]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    if (nk > 0) {
        fetch_scales(scales, 0);
        load_part(0, 0, 1);
#pragma unroll
        for (int t = 1; t < NS - 1; ++t)
            if (t < nk) load_part(t, 0, 1);
    }
    int kt = 0;
    for (; kt + NS - 1 < nk; ++kt) stage(kt, std::true_type{});
    for (; kt < nk; ++kt) stage(kt, std::false_type{});
    __syncthreads();

    // Results: each wave turns 32 rows at a time through LDS of its own, so
    // that its stores cover whole runs of a row.
    uint8_t* mine = lds + w * 32 * kOutRow;
    const int64_t col0 = n0 + wn * FN * 32;
    auto put = [&](auto format) {
        constexpr int kF = decltype(format)::value, kEs = kF == FSDP_F32 ? 4 : 2;
        constexpr int kLanes = FN * 32 * kEs / 16;           // lanes a row
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint8_t* o = mine + (l & 31) * kOutRow + (j * 32 + q * 8 + h * 4) * kEs;
                    if constexpr (kF == FSDP_F32) {
                        u32x4 v;
                        v.x = __float_as_uint(acc[i][j][4 * q]); v.y = __float_as_uint(acc[i][j][4 * q + 1]);
                        v.z = __float_as_uint(acc[i][j][4 * q + 2]); v.w = __float_as_uint(acc[i][j][4 * q + 3]);
                        *reinterpret_cast<u32x4*>(o) = v;
                    } else {
                        u32x2 v;
                        v.x = from_f32<kF>(acc[i][j][4 * q]) | (from_f32<kF>(acc[i][j][4 * q + 1]) << 16);
                        v.y = from_f32<kF>(acc[i][j][4 * q + 2]) | (from_f32<kF>(acc[i][j][4 * q + 3]) << 16);
                        *reinterpret_cast<u32x2*>(o) = v;
                    }
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int t = 0; t < 32 * kLanes / 64; ++t) {
                const int r = (t * 64 + l) / kLanes, c = (t * 64 + l) % kLanes * (16 / kEs);
                const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * kOutRow + c * kEs);
                const int64_t row = m0 + (wm * FM + i) * 32 + r, col = col0 + c;
                if (row < p.m && col < p.n) {
                    char* o = (char*)p.out + (row * p.ldo + col) * kEs;
                    if (col + 16 / kEs <= p.n) {
                        *(u32x4_any*)o = v;
                    } else {
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 16 / kEs; ++e)
                            if (col + e < p.n) {
                                if constexpr (kF == FSDP_F32) ((uint32_t*)o)[e] = x[e];
                                else ((uint16_t*)o)[e] = (uint16_t)(x[e / 2] >> (16 * (e & 1)));
                            }
                    }
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    };
    if constexpr (F != kAnyFormat) put(std::integral_constant<int, F>{});
    else if (p.dt == FSDP_F32) put(std::integral_constant<int, FSDP_F32>{});
    else if (p.dt == FSDP_F16) put(std::integral_constant<int, FSDP_F16>{});
    else put(std::integral_constant<int, FSDP_BF16>{});
}

template <int F, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void k_mx4_tiles(Mx4Product p, uint32_t tiles_m, uint32_t tiles_n) {
    mx4_tile<F, BM, BN, WM, WN, NS>(p, tiles_m, tiles_n, blockIdx.x);
}

// Two products in one launch, the second from workgroup `first` on (a multiple of
// 8, so that its tiles too go to the XCDs in turn).
template <int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void k_mx4_two(Mx4Product a, Mx4Product b, uint32_t first, uint32_t am,
                                                          uint32_t an, uint32_t bm, uint32_t bn) {
    const bool second = blockIdx.x >= first;
    if (!second && blockIdx.x >= am * an) return;
    Mx4Product p;
    p.a = second ? b.a : a.a;
    p.sa = second ? b.sa : a.sa;
    p.b = second ? b.b : a.b;
    p.sb = second ? b.sb : a.sb;
    p.m = second ? b.m : a.m;
    p.n = second ? b.n : a.n;
    p.nb = second ? b.nb : a.nb;
    p.dt = second ? b.dt : a.dt;
    p.out = second ? b.out : a.out;
    p.ldo = second ? b.ldo : a.ldo;
    mx4_tile<kAnyFormat, BM, BN, WM, WN, NS>(p, second ? bm : am, second ? bn : an,
                                             second ? blockIdx.x - first : blockIdx.x);
}

template <int F, int BM, int BN, int WM, int WN, int NS>
static hipError_t launch_tiles(const Mx4Product& p) {
    // a launch holds fewer than 2^32 work items; more tiles go in parts of the result
    constexpr int64_t kMost = (int64_t(1) << 32) / (64 * WM * WN) - 1;
    const int64_t tm = (p.m + BM - 1) / BM, tn = (p.n + BN - 1) / BN;
    const int64_t pn = tn < kMost ? tn : kMost, pm = kMost / pn < tm ? kMost / pn : tm;
    for (int64_t i = 0; i < tm; i += pm)
        for (int64_t j = 0; j < tn; j += pn) {
            const int64_t m0 = i * BM, n0 = j * BN, cm = tm - i < pm ? tm - i : pm, cn = tn - j < pn ? tn - j : pn;
            Mx4Product c = p;
            c.a = p.a + m0 * p.nb * 16;
            c.sa = p.sa + m0 * p.nb;
            c.b = p.b + n0 * p.nb * 16;
            c.sb = p.sb + n0 * p.nb;
            c.m = p.m - m0 < cm * BM ? p.m - m0 : cm * BM;
            c.n = p.n - n0 < cn * BN ? p.n - n0 : cn * BN;
            c.out = (char*)p.out + (m0 * p.ldo + n0) * dt_bytes(p.dt);
            launch(k_mx4_tiles<F, BM, BN, WM, WN, NS>, dim3((unsigned)(cm * cn)), dim3(64 * WM * WN),
                   (hipStream_t)p.stream, c, (uint32_t)cm, (uint32_t)cn);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

// Of few enough tiles for one launch (launch_mx4_two).
template <int BM, int BN, int WM, int WN, int NS>
static hipError_t launch_two(const Mx4Product& a, const Mx4Product& b) {
    const int64_t am = (a.m + BM - 1) / BM, an = (a.n + BN - 1) / BN, bm = (b.m + BM - 1) / BM, bn = (b.n + BN - 1) / BN;
    const int64_t first = (am * an + 7) / 8 * 8;
    launch(k_mx4_two<BM, BN, WM, WN, NS>, dim3((unsigned)(first + bm * bn)), dim3(64 * WM * WN), (hipStream_t)a.stream,
           a, b, (uint32_t)first, (uint32_t)am, (uint32_t)an, (uint32_t)bm, (uint32_t)bn);
    return hipGetLastError();
}

}  // namespace fsdp
