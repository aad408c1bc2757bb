// fsdp_fp8_tiles.h -- the tiled product of two matrices of 8-bit blocks
// (fsdp_fp8_matmul.hip instantiates it).  Not installed.
#pragma once

#include "fsdp_fp8_device.h"
#include "fsdp_mx4_tiles.h"    // tile_of and the vector types
#include "fsdp_waits.h"

#pragma clang fp contract(off)

namespace fsdp {

constexpr int kE4m3 = 0;    // the instruction's code for the format

// Up to two products, the tiles of the second behind those of the first.  A product whose
// sum is split is `splits` rounds of its tiles, each over `chunk` blocks along k (the last
// one over what is left) and into a matrix of fp32 partial sums of its own.
struct Fp8Jobs {
    Fp8Product p[2];
    uint32_t tm[2], tn[2], first, tiles;    // tiles of each down and across; of the first, of both, rounds counted
    int splits[2], chunk[2];
};

// One tile of a product, over nk blocks along k.
struct Fp8Tile {
    const uint8_t *a, *b, *sa, *sb;    // the codes of the tile's first rows, and the matrices' scales, from its first block on
    int64_t m0, n0;
    int rows_a, rows_b, nk, nb, ta, tb, round;
    int bytes_a, bytes_b;              // of the tile's rows to the last one's end
    uint32_t tm, tn;
};
template <int BM, int BN>
__device__ __forceinline__ Fp8Tile fp8_tile_at(const Fp8Jobs& j, uint32_t t) {
    const bool second = t >= j.first;
    uint32_t tm = second ? j.tm[1] : j.tm[0], tn = second ? j.tn[1] : j.tn[0], b = second ? t - j.first : t;
    Fp8Tile o;
    o.round = 0;
    for (; b >= tm * tn; b -= tm * tn) ++o.round;
    tile_of(b, tm, tn, o.tm, o.tn);
    o.tm = __builtin_amdgcn_readfirstlane(o.tm);         // tile_of divides, which is vector arithmetic
    o.tn = __builtin_amdgcn_readfirstlane(o.tn);
    o.m0 = (int64_t)o.tm * BM;
    o.n0 = (int64_t)o.tn * BN;
    const int64_t m = (second ? j.p[1].m : j.p[0].m) - o.m0, n = (second ? j.p[1].n : j.p[0].n) - o.n0;
    o.rows_a = m >> 32 ? BM : (int)min((uint32_t)m, (uint32_t)BM);    // no 64-bit compare: those too are vector arithmetic
    o.rows_b = n >> 32 ? BN : (int)min((uint32_t)n, (uint32_t)BN);
    o.nb = (int)(second ? j.p[1].nb : j.p[0].nb);
    const int chunk = second ? j.chunk[1] : j.chunk[0], k0 = o.round * chunk;
    o.nk = min(chunk, o.nb - k0);
    o.a = (second ? j.p[1].a : j.p[0].a) + (o.m0 * o.nb + k0) * kFp8Block;
    o.b = (second ? j.p[1].b : j.p[0].b) + (o.n0 * o.nb + k0) * kFp8Block;
    o.bytes_a = (o.rows_a * o.nb - k0) * kFp8Block;
    o.bytes_b = (o.rows_b * o.nb - k0) * kFp8Block;
    o.sa = (second ? j.p[1].sa : j.p[0].sa) + k0;
    o.sb = (second ? j.p[1].sb : j.p[0].sb) + k0;
    o.ta = second ? j.p[1].ta : j.p[0].ta;
    o.tb = second ? j.p[1].tb : j.p[0].tb;
    return o;
}

// BM x BN results a tile of WM x WN waves, BM / WM x BN / WN a wave.  A stage is a
// block of every row (128 bytes, one cache line), so a row has one scale in it; NS
// stages are in LDS.  A workgroup makes the tiles b, b + grid, ...: the stages of
// all of them are one stream, whose loads run NS stages ahead, so that a tile's end
// and its stores lie behind the next one's first loads.
//
// 256 x 256, four waves of 128 x 128, one a SIMD.  What two stages cost in cycles, from time
// stamps in the kernel: 64 instructions of 64 are 4096, and 4832 go by; 4504 without any
// access to LDS or memory (an instruction of one wave alone takes 68, the rest is the
// loop's head), 40 more with the fragments' reads, 28 with the barriers, 260 with the
// loads, which are sent one before an instruction (all at once: 5-10% slower).  16 stages' scales
// 500-1100 on top, a tile's end 5600.  8192^3 takes 714,000 cycles, 73% of them busy, at
// 1.85 GHz where zeros of the same product run at 2.37: power bounds it as much as the
// loads, which take 352 us alone (256 where the L2 holds all).  Eight waves of 128 x 64
// read half as much again from LDS and need no fewer cycles for it (418 us where four
// took 394); all loads and reads of a row of instructions before it 416 instead of 406.
template <int BM, int BN, int WM, int WN, int NS>
struct Fp8Tiling {
    static constexpr int kWaves = WM * WN, kThreadsWg = 64 * kWaves;
    static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;   // fragments of 32 rows a wave
    static constexpr int kRow = kFp8Block;                       // bytes of a row's stage
    static constexpr int kChunks = kRow / 16;
    static constexpr int kLoads = (BM + BN) * kChunks / 64 / kWaves;    // 1 KB loads a wave a stage
    static constexpr int kLoadsA = BM * kChunks / 64 / kWaves;
    static constexpr int kStep = kWaves * 64 / kChunks;          // rows from one load of a wave to its next
    static constexpr int kStage = (BM + BN) * kRow;
    static constexpr int kScales = NS * kStage;                  // where the scales lie: 2 x 4 x (BM + BN) dwords
    static constexpr int kOutRow = BM == 256 ? 128 : 64;         // bytes of a result row that are turned at a time
    static constexpr int kOut = kScales + 2 * (BM + BN) * 16;    // where results are turned, 32 rows a wave
    static constexpr int kLds = kOut + kWaves * 32 * kOutRow;
    static constexpr int kResident = 163840 / kLds;              // workgroups a CU
    static_assert(kLoadsA * 64 * kWaves == BM * kChunks && kLoads * 64 * kWaves == (BM + BN) * kChunks, "whole loads");
    static_assert(kStep % 16 == 0, "the slots' turn repeats from load to load");
    static_assert(NS % 2 == 0 && kLds <= 163840, "a pair of stages; what a CU has");
};

template <int BM, int BN, int WM, int WN, int NS>
__device__ __forceinline__ void fp8_products(const Fp8Jobs& j) {
    using T = Fp8Tiling<BM, BN, WM, WN, NS>;
    constexpr int FM = T::FM, FN = T::FN, kRow = T::kRow, kLoads = T::kLoads, kStage = T::kStage;
    constexpr int kRows = (BM + BN + T::kThreadsWg - 1) / T::kThreadsWg;
    constexpr int kIns = FM * FN;                            // instructions of a step
    constexpr bool kAhead = BM == 256;                       // lines are brought into the L2 ahead of their loads
    constexpr int kBehind = kAhead;                          // accesses of it behind a stage's loads
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];

    const int l = threadIdx.x & 63, h = l >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // Chunk c (16 bytes) of row r lies at slot c ^ turn(r) of the row's stage: 16 rows'
    // equal chunks then lie in 16 places of the 256 bytes that the banks span.
    auto turn = [](int r) { return (r >> 1) & 7; };

    // Global to LDS: a wave's load fills 1 KB, lane l the 16 bytes at 16 l.  Rows
    // behind the matrix read its last row; what they bring is not stored.
    const int lrow = (w * 64 + l) / T::kChunks;              // row of load 0; kStep is a multiple of 16
    const int lchunk = ((w * 64 + l) % T::kChunks) ^ turn(lrow);
    uint32_t lt = blockIdx.x;                                // the tile that is being loaded, and its next stage
    int lk = 0;
    Fp8Tile ld = fp8_tile_at<BM, BN>(j, lt);
    int voff[kLoads];
    auto aim = [&]() {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = lrow + (i < T::kLoadsA ? i : i - T::kLoadsA) * T::kStep;
            const int lim = i < T::kLoadsA ? ld.rows_a : ld.rows_b;
            voff[i] = (r < lim ? r : lim - 1) * (ld.nb * kRow) + lchunk * 16;
        }
    };
    // Part `part` of `parts` of the loads of stage lk + J of the tile that is loaded,
    // into `slot`.  Behind its last stage, and behind the last tile, the buffers are
    // empty: nothing is fetched, and the slot gets zeros.
    auto load_part = [&](int J, int slot, int part, int parts) {
        const int soff = __builtin_amdgcn_readfirstlane((lk + J) * kRow);
        const bool some = lk + J < ld.nk && lt < j.tiles;
        const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)ld.a, 0, some ? ld.bytes_a : 0, kRsrcWord3);
        const auto rb = __builtin_amdgcn_make_buffer_rsrc((void*)ld.b, 0, some ? ld.bytes_b : 0, kRsrcWord3);
        uint8_t* to = lds + slot * kStage + w * 1024;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (i * parts / kLoads != part) continue;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                i < T::kLoadsA ? ra : rb, (__attribute__((address_space(3))) void*)(to + i * T::kWaves * 1024), 16,
                voff[i], soff, 0, 0);
        }
    };
    // The 32 tiles that an XCD works on at a time share 4 panels of A and 8 of B, so a
    // line comes from memory for 8 or 4 of them at once, and all wait for it.  Each brings
    // its part of the panels into the L2 four stages before it is loaded: a wave two
    // stages of 32 rows, a lane a line.
    int poff = 0;
    auto aim_ahead = [&]() {
        const int r = w == 0 ? (int)(ld.tn & 7) * 32 : (int)(ld.tm & 3) * 64 + (w - 1) * 32;
        poff = (r + (l >> 1)) * (ld.nb * kRow) + (l & 1) * kRow;
    };
    auto ahead = [&]() {
        const int n = w < 3 && lk + 5 < ld.nk && lt < j.tiles ? (w == 0 ? ld.bytes_a : ld.bytes_b) : 0;
        const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)(w == 0 ? ld.a : ld.b), 0, n, kRsrcWord3);
        return __builtin_amdgcn_raw_buffer_load_b32(r, poff, __builtin_amdgcn_readfirstlane((lk + 4) * kRow), 0);
    };
    // Two stages on, and to the next tile behind a tile's last one.
    auto go_on = [&]() {
        lk += 2;
        if (lk >= ld.nk && lt < j.tiles) {
            lk = 0;
            lt += gridDim.x;
            if (lt < j.tiles) {
                ld = fp8_tile_at<BM, BN>(j, lt);
                aim();
                if (kAhead) aim_ahead();
            }
        }
    };

    // Scales: a lane fetches a row's bytes of 16 stages at once and puts them into
    // LDS, a dword for four stages, where the waves that share the row read them.
    // Returns the loads that it left on their way.
    auto fetch_scales = [&](u32x4 (&s)[kRows], const Fp8Tile& t, int g) {
        const int b0 = g * 16;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            int r = i * T::kThreadsWg + (int)threadIdx.x;
            if ((i + 1) * T::kThreadsWg > BM + BN) r = r < BM + BN ? r : BM + BN - 1;
            const uint8_t* q = r < BM ? t.sa + ((t.m0 + (r < t.rows_a ? r : t.rows_a - 1)) >> t.ta) * t.nb
                                      : t.sb + ((t.n0 + (r - BM < t.rows_b ? r - BM : t.rows_b - 1)) >> t.tb) * t.nb;
            s[i] = scales16(q + b0, t.nk - b0);
        }
        return t.nk - b0 >= 16 ? kRows : 0;
    };
    auto put_scales = [&](const u32x4 (&s)[kRows], int half) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = i * T::kThreadsWg + (int)threadIdx.x;
            if ((i + 1) * T::kThreadsWg > BM + BN && r >= BM + BN) break;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                *reinterpret_cast<uint32_t*>(lds + T::kScales + ((half * 4 + d) * (BM + BN) + r) * 4) = s[i][d];
        }
    };

    const int wm = w / WN, wn = w % WN;
    const int arow = (wm * FM * 32 + (l & 31)) * kRow, brow = (BM + wn * FN * 32 + (l & 31)) * kRow;
    const int tl = turn(l & 31);                             // fragments start at multiples of 32 rows
    const int srow = T::kScales + (wm * FM * 32 + (l & 31)) * 4, trow = T::kScales + (BM + wn * FN * 32 + (l & 31)) * 4;

    // A stage is two steps of 64 along k, a step FM rows of FN instructions.  While a
    // step is multiplied the next one's fragments are read, half a fragment (16 bytes a
    // lane) at a time: B's into a second set; A's, where the registers do not hold two
    // of them, into the place of the one whose row is done.  Lane half h brings chunks
    // 4 s + h and 4 s + 2 + h of step s on both sides.
    constexpr int kSetsA = T::kWaves <= 4 ? 2 : 1;
    u32x4 a[kSetsA][FM][2], b[2][FN][2];
    int sa[FM], sb[FN];
    auto read_a = [&](int slot, int s, int f, int c) {
        a[s % kSetsA][f][c] = *reinterpret_cast<const u32x4*>(lds + slot * kStage + arow + f * 32 * kRow + ((4 * s + 2 * c + h) ^ tl) * 16);
    };
    auto read_b = [&](int slot, int s, int f, int c) {
        b[s][f][c] = *reinterpret_cast<const u32x4*>(lds + slot * kStage + brow + f * 32 * kRow + ((4 * s + 2 * c + h) ^ tl) * 16);
    };
    auto whole8 = [](const u32x4 (&x)[2]) {
        return i32x8{(int)x[0].x, (int)x[0].y, (int)x[0].z, (int)x[0].w, (int)x[1].x, (int)x[1].y, (int)x[1].z, (int)x[1].w};
    };
    // What of step s of the stage in `slot` is read before instruction q of the step
    // before it, and behind the last one (q = kIns).
    auto read_part = [&](int slot, int s, int q) {
        if constexpr (kSetsA == 2) {
            constexpr int kN = 2 * (FM + FN), kSpan = kIns > 2 ? kIns - 2 : 1;
#pragma unroll
            for (int x = 0; x < kN; ++x)
                if (x * kSpan / kN == q) {
                    if (x < 2 * FN) read_b(slot, s, x / 2, x % 2);
                    else read_a(slot, s, x / 2 - FN, x % 2);
                }
        } else {
            const int i = q / FN, f = q % FN;
            if (q == kIns) {
                read_a(slot, s, FM - 1, 0);
                read_a(slot, s, FM - 1, 1);
                return;
            }
            if (i > 0) {
                if (FN == 1 || f == 0) read_a(slot, s, i - 1, 0);
                if (FN == 1 || f == 1) read_a(slot, s, i - 1, 1);
            }
#pragma unroll
            for (int x = 0; x < 2 * FN; ++x)
                if (x * kIns / (2 * FN) == q) read_b(slot, s, x / 2, x % 2);
        }
    };
    // The scales of stages kt (even) and kt + 1, a byte each: read among the
    // instructions before them, and put in their place behind the last of these.
    uint32_t sn[FM + FN];
    auto read_scales = [&](int half, int kt) {
        const int at = (half * 4 + (kt >> 2 & 3)) * ((BM + BN) * 4);
#pragma unroll
        for (int f = 0; f < FM; ++f) sn[f] = *reinterpret_cast<const uint32_t*>(lds + srow + f * 128 + at);
#pragma unroll
        for (int f = 0; f < FN; ++f) sn[FM + f] = *reinterpret_cast<const uint32_t*>(lds + trow + f * 128 + at);
    };
    auto take_scales = [&](int kt) {
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[f] = (int)(sn[f] >> ((kt & 2) * 8));
#pragma unroll
        for (int f = 0; f < FN; ++f) sb[f] = (int)(sn[FM + f] >> ((kt & 2) * 8));
    };
    // The wait for a stage's loads, with those of `behind` stages behind it on their way.
    auto arrived = [&](auto behind) { wait_memory<decltype(behind)::value * kLoads>(); };
    // Accesses that went out behind the loads that the next stage 0 waits for: a tile's
    // stores, a fetch of scales.  They need not be over then.  With kAhead one more is there
    // at every such wait, the first one's too: each pair's loads, and the first pair's
    // before the loop, are followed by an access of ahead().
    int newer = 0;
    constexpr int kStored = FM * FN * 2 < 62 - kRows ? FM * FN * 2 : 62 - kRows;    // least stores of a whole tile, a wave: 16 bits
    // The same wait with `n` accesses behind them, 0, kRows, kStored or their sum.
    auto arrived_behind = [&](int n) {
        if constexpr (NS > 2) {
            arrived(std::integral_constant<int, NS - 2>{});
        } else {
            wait_memory_by<kStored, kRows, kBehind, kRows + kBehind, kStored + kBehind>(n);
        }
    };

    f32x16 acc[FM][FN];
    // Stage J of two, in `slot`, the fragments of its step 0 read already; `next`: the
    // slot of the stage behind it.
    auto stage = [&](auto J_, int slot, int next, auto behind_wait, auto behind_barrier) {
        constexpr int J = decltype(J_)::value;
        auto multiply = [&](int s, int q) {
            const int i = q / FN, f = q % FN;
            __builtin_amdgcn_sched_barrier(0);
            // rows of B first: a lane then holds runs of four results of one row of A
            acc[i][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(whole8(b[s][f]), whole8(a[s % kSetsA][i]), acc[i][f],
                                                                        kE4m3, kE4m3, J, sb[f], J, sa[i]);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int q = 0; q < kIns; ++q) {
            read_part(slot, 1, q);
            multiply(0, q);
        }
        read_part(slot, 1, kIns);
        // one barrier a stage: every wave's part of the next one has arrived, and nobody
        // reads this one any more
        if constexpr (J == 0) arrived_behind(newer);
        else arrived(std::integral_constant<int, NS - 2>{});
        behind_wait();
        meet_in_lds();
        behind_barrier();
#pragma unroll
        for (int q = 0; q < kIns; ++q) {
            read_part(next, 0, q);
            load_part(J, slot, q, kIns);
            multiply(1, q);
        }
        read_part(next, 0, kIns);
    };

    // Results: each wave turns 32 rows at a time, kOutRow bytes of each, through LDS of its
    // own, so that its stores cover runs of a row.  Chunk c (16 bytes) of row r lies at
    // slot c ^ turned(r), as in the stages.  LDS takes a wave's accesses in their order: a
    // turn's results are written and read while those of the turn before go out.
    auto store_tile = [&](const Fp8Tile& t, void* to_, int64_t ldo, auto format, auto whole_tile) {
        constexpr int kF = decltype(format)::value, kEs = kF == FSDP_F32 ? 4 : 2, kLanes = T::kOutRow / 16;    // lanes a row
        constexpr int kGroups = T::kOutRow / kEs / 8;        // runs of 8 columns a turn: a fragment has 4, each lane half of one
        constexpr int kStores = 32 * kLanes / 64, kAcross = FN * 4 / kGroups, kTurns = FM * kAcross;
        constexpr bool kWhole = decltype(whole_tile)::value;
        auto turned = [](int r) { return T::kOutRow == 128 ? r >> 1 & 7 : r >> 2 & 3; };
        int le = l;
        unknown(le);                                         // what follows from it is not kept through the stages
        const int r = le & 31, hh = le >> 5;
        uint8_t* const mine = lds + T::kOut + w * 32 * T::kOutRow;
        uint8_t* const to = mine + r * T::kOutRow;
        const int sr0 = le / kLanes, c = le % kLanes;        // what a lane stores: chunk c of rows sr0, sr0 + 64 / kLanes, ...
        const int64_t down = ldo * (64 / kLanes * kEs);
        char* const out = (char*)to_ + ((t.m0 + wm * FM * 32) * ldo + t.n0 + wn * FN * 32) * kEs + (sr0 * ldo * kEs + c * 16);
        u32x4 v[2][kStores];
#pragma unroll
        for (int n = 0; n <= kTurns; ++n) {
            if (n < kTurns) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int at = n % kAcross * kGroups + g, q = at % 4;
                    const f32x16& x = acc[n / kAcross][at / 4];
                    if constexpr (kF == FSDP_F32)
                        *reinterpret_cast<u32x4*>(to + ((2 * g + hh) ^ turned(r)) * 16) =
                            u32x4{__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]), __float_as_uint(x[4 * q + 2]),
                                  __float_as_uint(x[4 * q + 3])};
                    else
                        *reinterpret_cast<u32x2*>(to + (g ^ turned(r)) * 16 + hh * 8) =
                            u32x2{pack2<kF>(x[4 * q], x[4 * q + 1]), pack2<kF>(x[4 * q + 2], x[4 * q + 3])};
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int s = 0; s < kStores; ++s) {
                    const int sr = sr0 + s * (64 / kLanes);
                    v[n & 1][s] = *reinterpret_cast<const u32x4*>(mine + sr * T::kOutRow + (c ^ turned(sr)) * 16);
                }
                __builtin_amdgcn_wave_barrier();
            }
            if (n == 0) continue;
            const int i = (n - 1) / kAcross, c0 = (n - 1) % kAcross * kGroups * 8;    // the turn's rows and first column
            const int left = t.rows_b - wn * FN * 32 - c0 - c * (16 / kEs);
#pragma unroll
            for (int s = 0; s < kStores; ++s) {
                u32x4 x = v[(n - 1) & 1][s];
                char* const o = out + (i * kStores + s) * down + c0 * kEs;
                if constexpr (!kWhole)
                    if ((wm * FM + i) * 32 + sr0 + s * (64 / kLanes) >= t.rows_a) continue;
                if (kWhole || left >= 16 / kEs) {
                    *(u32x4_any*)o = x;
                } else {
#pragma unroll 1
                    for (int e = 0; e < left; ++e) {
                        if constexpr (kF == FSDP_F32) {
                            ((uint32_t*)o)[e] = x.x;
                            x = u32x4{x.y, x.z, x.w, 0};
                        } else {
                            ((uint16_t*)o)[e] = (uint16_t)x.x;
                            x = u32x4{x.x >> 16 | x.y << 16, x.y >> 16 | x.z << 16, x.z >> 16 | x.w << 16, x.w >> 16};
                        }
                    }
                }
            }
        }
    };

    u32x4 scales[kRows];
    uint32_t line = 0;                                       // of those brought ahead
    Fp8Tile at = ld;                                         // the tile that is being made
    int half = 0;                                            // where its 16 stages' scales lie
    if (at.nk > 0) {
        aim();
        if (kAhead) aim_ahead();
        fetch_scales(scales, at, 0);
#pragma unroll
        for (int t = 0; t < NS; t += 2) {
            if (t > 0) go_on();
            load_part(0, t, 0, 1);
            load_part(1, t + 1, 0, 1);
        }
        arrived(std::integral_constant<int, NS - 1>{});
        if (kAhead) line = ahead();
        put_scales(scales, 0);
        meet_in_lds();
        read_scales(0, 0);
        take_scales(0);
#pragma unroll
        for (int x = 0; x < 2 * FN; ++x) read_b(0, 0, x / 2, x % 2);
#pragma unroll
        for (int x = 0; x < 2 * FM; ++x) read_a(0, 0, x / 2, x % 2);
    }
    int pair = 0;                                            // of the stream, modulo NS / 2
    for (uint32_t t = blockIdx.x; t < j.tiles; t += gridDim.x) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) acc[i][f] = f32x16{0};
        const bool second = t >= j.first;
        const Fp8Tile done = at;
        // Two stages run without a branch between or behind them (the compiler moves
        // matrix instructions from one block to another, away from their place).  Behind an
        // odd number one of zeros is added, with scales of 2^-127.
        for (int kt = 0; kt < done.nk; kt += 2) {
            go_on();
            const bool last = kt + 2 >= done.nk, ends = last || (kt & 15) == 14;
            if ((kt & 15) == 0) {
                // the next 16 stages' scales, this tile's or the next one's, go to the other half
                const bool on = kt + 16 < done.nk;
                if (!on && t + gridDim.x < j.tiles) at = fp8_tile_at<BM, BN>(j, t + gridDim.x);
                if (on || t + gridDim.x < j.tiles) newer += fetch_scales(scales, at, on ? (kt >> 4) + 1 : 0);
            }
            const int slot = 2 * pair, other = half ^ 1, then = last ? 0 : kt + 2;
            pair = pair + 1 < NS / 2 ? pair + 1 : 0;
            half = ends ? other : half;
            // the put is done again by every pair, behind a wait that is there anyway: under a
            // condition it would be a branch, and a wait of its own
            stage(std::integral_constant<int, 0>{}, slot, slot + 1, []() {}, []() {});
            stage(std::integral_constant<int, 1>{}, slot + 1, 2 * pair,
                  [&]() {
                      put_scales(scales, other);
                      if (kAhead) needed(line);
                  },
                  [&]() { read_scales(half, then); });
            if (kAhead) line = ahead();
            take_scales(then);
            newer = 0;
        }
        int dt = second ? j.p[1].dt : j.p[0].dt;
        int64_t ldo = second ? j.p[1].ldo : j.p[0].ldo;
        void* out = second ? j.p[1].out : j.p[0].out;
        if ((second ? j.splits[1] : j.splits[0]) > 1) {
            dt = FSDP_F32;
            ldo = second ? j.p[1].n : j.p[0].n;
            out = (second ? j.p[1].parts : j.p[0].parts) + done.round * (second ? j.p[1].m : j.p[0].m) * ldo;
        }
        auto store = [&](auto format) {
            if (done.rows_a == BM && done.rows_b == BN) store_tile(done, out, ldo, format, std::true_type{});
            else store_tile(done, out, ldo, format, std::false_type{});
        };
        if (dt == FSDP_F32) store(std::integral_constant<int, FSDP_F32>{});
        else if (dt == FSDP_F16) store(std::integral_constant<int, FSDP_F16>{});
        else store(std::integral_constant<int, FSDP_BF16>{});
        newer = done.rows_a == BM && done.rows_b == BN ? kStored : 0;
    }
    wait_memory<0>();                                        // loads into LDS end before the workgroup does
}

template <int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_products(Fp8Jobs j) {
    fp8_products<BM, BN, WM, WN, NS>(j);
}

// `count` products in one launch, of fewer than 2^31 tiles together, rounds counted; a sum
// of 0 terms alone.  splits: each one's, or null for 1.  Items that differ in length go a
// workgroup each, in the order in which CUs get free, unless there are many.
template <int BM, int BN, int WM, int WN, int NS>
static hipError_t launch_fp8_jobs(const Fp8Product* p, int count, const int* splits = nullptr) {
    using T = Fp8Tiling<BM, BN, WM, WN, NS>;
    Fp8Jobs j{};
    for (int q = 0; q < count; ++q) {
        j.p[q] = p[q];
        j.tm[q] = (uint32_t)((p[q].m + BM - 1) / BM);
        j.tn[q] = (uint32_t)((p[q].n + BN - 1) / BN);
        j.splits[q] = splits ? splits[q] : 1;
        j.chunk[q] = (int)((p[q].nb + j.splits[q] - 1) / j.splits[q]);
        j.tiles += j.tm[q] * j.tn[q] * (uint32_t)j.splits[q];
        if (q == 0) j.first = j.tiles;
    }
    const uint32_t most = (uint32_t)(p[0].cus * T::kResident) & ~7u;    // whole rounds of the XCDs
    const bool all = j.tiles < most || (count > 1 && j.chunk[0] != j.chunk[1] && j.tiles < 4 * most);
    launch_lds(k_fp8_products<BM, BN, WM, WN, NS>, dim3(all ? j.tiles : most), dim3(T::kThreadsWg), T::kLds,
               (hipStream_t)p[0].stream, j);
    return hipGetLastError();
}

}  // namespace fsdp
