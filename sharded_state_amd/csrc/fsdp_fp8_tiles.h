// fsdp_fp8_tiles.h -- the tiled product of two matrices of 8-bit blocks
// (fsdp_fp8_matmul.hip instantiates it).  Not installed.
#pragma once

#include "fsdp_fp8_device.h"
#include "fsdp_mx4_tiles.h"    // tile_of and the vector types

#pragma clang fp contract(off)

namespace fsdp {

constexpr int kE4m3 = 0;    // the instruction's code for the format

// BM x BN results a workgroup of WM x WN waves, BM / WM x BN / WN a wave.  A stage
// is a block of every row (128 bytes, one cache line), so a row has one scale in
// it; NS stages are in LDS.
template <int F, int BM, int BN, int WM, int WN, int NS>
__device__ __forceinline__ void fp8_tile_product(const Fp8Product& p, uint32_t tm, uint32_t tn) {
    constexpr int kWaves = WM * WN;
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;     // fragments of 32 rows a wave
    constexpr int kRow = kFp8Block;                          // bytes of a row's stage
    constexpr int kChunks = kRow / 16;
    constexpr int kLoads = (BM + BN) * kChunks / 64 / kWaves;    // 1 KB loads a wave a stage
    constexpr int kLoadsA = BM * kChunks / 64 / kWaves;
    constexpr int kStep = kWaves * 64 / kChunks;             // rows from one load of a wave to its next
    constexpr int kStage = (BM + BN) * kRow;
    constexpr int kOutRow = FN * 32 * (F == FSDP_F32 || F == kAnyFormat ? 4 : 2) + 16;   // a result row in LDS, padded
    constexpr int kThreadsWg = 64 * kWaves;
    constexpr int kRows = (BM + BN + kThreadsWg - 1) / kThreadsWg;
    constexpr int kScales = NS * kStage;                     // where the scales lie: 2 x (BM + BN) rows of 16 bytes
    static_assert(kLoadsA * 64 * kWaves == BM * kChunks && kLoads * 64 * kWaves == (BM + BN) * kChunks, "whole loads");
    static_assert(WM * WN * 32 * kOutRow <= kScales, "results pass through the stages' LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kScales + 2 * (BM + BN) * 16];

    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rows_a = (int)(p.m - m0 < BM ? p.m - m0 : BM), rows_b = (int)(p.n - n0 < BN ? p.n - n0 : BN);
    const int l = threadIdx.x & 63, h = l >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nk = (int)p.nb, rowbytes = nk * kRow;

    // Chunk c (16 bytes) of row r lies at slot c ^ turn(r) of the row's stage: 16 rows'
    // equal chunks then lie in 16 places of the 256 bytes that the banks span.
    auto turn = [](int r) { return (r >> 1) & 7; };

    // Global to LDS: a wave's load fills 1 KB, lane l the 16 bytes at 16 l.  Rows
    // behind the matrix read its last row; what they bring is not stored.
    const int lrow = (w * 64 + l) / kChunks;                 // row of load 0; kStep is a multiple of 16
    const int lchunk = ((w * 64 + l) % kChunks) ^ turn(lrow);
    static_assert(kStep % 16 == 0, "the slots' turn repeats from load to load");
    int voff[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = lrow + (i < kLoadsA ? i : i - kLoadsA) * kStep;
        const int lim = i < kLoadsA ? rows_a : rows_b;
        voff[i] = (r < lim ? r : lim - 1) * rowbytes + lchunk * 16;
    }
    // Part `part` of `parts` of the loads of stage kt into `slot`.  Behind the last stage
    // the buffers are empty: nothing is fetched, and the slot gets zeros.
    auto load_part = [&](int kt, int slot, int part, int parts) {
        const int soff = __builtin_amdgcn_readfirstlane(kt * kRow);
        const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + m0 * rowbytes), 0, kt < nk ? rows_a * rowbytes : 0, kRsrcWord3);
        const auto rb = __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + n0 * rowbytes), 0, kt < nk ? rows_b * rowbytes : 0, kRsrcWord3);
        uint8_t* to = lds + slot * kStage + w * 1024;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (i * parts / kLoads != part) continue;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                i < kLoadsA ? ra : rb, (__attribute__((address_space(3))) void*)(to + i * kWaves * 1024), 16,
                voff[i], soff, 0, 0);
        }
    };

    // Scales: a lane fetches a row's bytes of 16 stages at once and puts them into
    // LDS, where the waves that share the row read them, four stages a read.
    auto fetch_scales = [&](u32x4 (&s)[kRows], int g) {
        const int b0 = g * 16;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = i * kThreadsWg + (int)threadIdx.x;
            if ((i + 1) * kThreadsWg > BM + BN && r >= BM + BN) break;
            const uint8_t* q = r < BM ? p.sa + ((m0 + (r < rows_a ? r : rows_a - 1)) >> p.ta) * nk
                                      : p.sb + ((n0 + (r - BM < rows_b ? r - BM : rows_b - 1)) >> p.tb) * nk;
            s[i] = scales16(q + b0, nk - b0);
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

    // A stage is two steps of 64 along k, a step FM rows of FN instructions.  While a
    // step is multiplied the next one's fragments are read: B's into a second set, A's
    // into the place of the one whose row is done.  Lane half h brings chunks 4 s + h
    // and 4 s + 2 + h of step s on both sides.
    i32x8 a[FM], b[2][FN];
    int sa[FM], sb[FN];
    auto read1 = [&](int at, int s) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(lds + at + ((4 * s + h) ^ tl) * 16);
        const u32x4 y = *reinterpret_cast<const u32x4*>(lds + at + ((4 * s + 2 + h) ^ tl) * 16);
        return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };
    auto read_a = [&](int slot, int s, int f) { a[f] = read1(slot * kStage + arow + f * 32 * kRow, s); };
    auto read_b = [&](int slot, int s, int f) { b[s][f] = read1(slot * kStage + brow + f * 32 * kRow, s); };
    // What of step s of the stage in `slot` is read before row i of the step before it.
    auto read_part = [&](int slot, int s, int i) {
        if (i > 0) read_a(slot, s, i - 1);
#pragma unroll
        for (int f = 0; f < FN; ++f)
            if (f * FM / FN == i) read_b(slot, s, f);
    };
    // The scales of stages kt (even) and kt + 1, a byte each.
    auto read_scales = [&](int kt) {
        const int at = (kt >> 4 & 1) * (BM + BN) * 16 + (kt & 12), by = (kt & 2) * 8;
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[f] = (int)(*reinterpret_cast<const uint32_t*>(lds + srow + f * 512 + at) >> by);
#pragma unroll
        for (int f = 0; f < FN; ++f) sb[f] = (int)(*reinterpret_cast<const uint32_t*>(lds + trow + f * 512 + at) >> by);
    };
    // The wait for a stage's loads, with those of `BEHIND` stages behind it on their way.
    auto arrived = [&](auto behind) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(behind)::value * kLoads) : "memory");
    };
    auto together = [&]() {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // Stage kt + J in `slot`, the fragments of its step 0 read already; `next`: the slot
    // of the stage behind it.
    auto stage = [&](int kt, auto j, int slot, int next) {
        constexpr int J = decltype(j)::value;
        auto multiply = [&](int s, int i) {
#pragma unroll
            for (int f = 0; f < FN; ++f)
                // rows of B first: a lane then holds runs of four results of one row of A
                acc[i][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[s][f], a[i], acc[i][f], kE4m3, kE4m3, J, sb[f],
                                                                            J, sa[i]);
        };
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            read_part(slot, 1, i);
            __builtin_amdgcn_sched_barrier(0);
            multiply(0, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        read_a(slot, 1, FM - 1);
        // one barrier a stage: every wave's part of the next one has arrived, and nobody
        // reads this one any more
        arrived(std::integral_constant<int, NS - 2>{});
        together();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            read_part(next, 0, i);
            load_part(kt + J + NS, slot, i, FM);
            __builtin_amdgcn_sched_barrier(0);
            multiply(1, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        read_a(next, 0, FM - 1);
    };

    if (nk > 0) {
        u32x4 scales[kRows];
        fetch_scales(scales, 0);
#pragma unroll
        for (int t = 0; t < NS; ++t) load_part(t, t, 0, 1);
        arrived(std::integral_constant<int, NS - 1>{});
        put_scales(scales, 0);
        together();
        read_scales(0);
#pragma unroll
        for (int f = 0; f < FN; ++f) read_b(0, 0, f);
#pragma unroll
        for (int f = 0; f < FM; ++f) read_a(0, 0, f);
        // Two stages run without a branch between them (the compiler moves matrix
        // instructions from one block to another, away from their place).  Behind an odd
        // number one of zeros is added, with scales of 2^-127.
        for (int kt = 0; kt < nk; kt += 2) {
            // the next 16 stages' scales: fetched here, put eight stages on, read eight later
            if ((kt & 15) == 0 && kt + 16 < nk) fetch_scales(scales, (kt >> 4) + 1);
            if ((kt & 15) == 8 && kt + 8 < nk) put_scales(scales, (kt >> 4) + 1);
            const int slot = kt % NS;
            stage(kt, std::integral_constant<int, 0>{}, slot, slot + 1);
            stage(kt, std::integral_constant<int, 1>{}, slot + 1, (kt + 2) % NS);
            read_scales(kt + 2);
        }
        arrived(std::integral_constant<int, 0>{});
    }
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
                        *reinterpret_cast<u32x4*>(o) =
                            u32x4{__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                                  __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3])};
                    } else {
                        *reinterpret_cast<u32x2*>(o) =
                            u32x2{from_f32<kF>(acc[i][j][4 * q]) | (from_f32<kF>(acc[i][j][4 * q + 1]) << 16),
                                  from_f32<kF>(acc[i][j][4 * q + 2]) | (from_f32<kF>(acc[i][j][4 * q + 3]) << 16)};
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

// The tiles from (tm0, tn0) on, tiles_m x tiles_n of them.
template <int F, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_tiles(Fp8Product p, uint32_t tm0, uint32_t tn0, uint32_t tiles_m,
                                                            uint32_t tiles_n) {
    uint32_t tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    fp8_tile_product<F, BM, BN, WM, WN, NS>(p, tm0 + tm, tn0 + tn);
}

template <int F, int BM, int BN, int WM, int WN, int NS>
static hipError_t launch_fp8_tiles(const Fp8Product& p) {
    // a launch holds fewer than 2^32 work items; more tiles go in parts of the result
    constexpr int64_t kMost = (int64_t(1) << 32) / (64 * WM * WN) - 1;
    const int64_t tm = (p.m + BM - 1) / BM, tn = (p.n + BN - 1) / BN;
    const int64_t pn = tn < kMost ? tn : kMost, pm = kMost / pn < tm ? kMost / pn : tm;
    for (int64_t i = 0; i < tm; i += pm)
        for (int64_t j = 0; j < tn; j += pn) {
            const int64_t cm = tm - i < pm ? tm - i : pm, cn = tn - j < pn ? tn - j : pn;
            launch(k_fp8_tiles<F, BM, BN, WM, WN, NS>, dim3((unsigned)(cm * cn)), dim3(64 * WM * WN), (hipStream_t)p.stream,
                   p, (uint32_t)i, (uint32_t)j, (uint32_t)cm, (uint32_t)cn);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

}  // namespace fsdp
