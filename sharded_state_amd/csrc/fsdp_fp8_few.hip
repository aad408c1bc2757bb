// fsdp_fp8_few.hip -- the product with W for a few tokens on gfx950: y = x W^T
// with W in 8-bit blocks along k, and x in such blocks too or quantised on the
// way, in the same launch.
//
// With up to 16 tokens the product is one read of W, a byte an element.  A workgroup
// takes 16 rows of W, a wave every NW-th run of kRun blocks along k of them: 16 rows of
// 256 bytes, which go from memory to LDS without registers, and from there into the
// operands of v_mfma_scale_f32_16x16x128_f8f6f4 (lane l brings row l % 16 and 32 codes
// of the block).  A wave's run is on its way while it multiplies the one before, and no
// barrier stands between runs.  x is quantised by the whole workgroup, 16 lanes a
// block, into LDS, and the rows' scales are brought there, while the first runs are on
// their way; x in blocks comes in runs like W.  The waves' sums are added in LDS in
// their order.
//
// Measured in replayed graphs with W rotated past the caches, one token, us: 28672 x
// 8192 43.4 (5.5 TB/s; quantisation and a product in tiles 57.0), 8192 x 28672 49.6,
// 8192 x 8192 17.1, 5120 x 1280 4.4, 1280 x 5120 5.0; 16 tokens in blocks, 28672 x 8192
// 49.4, 8192 x 8192 17.6.
#include "fsdp_fp8_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRun = 2;                      // blocks along k that a wave takes at a time
constexpr int kRunRow = kRun * kFp8Block;    // a run's bytes of a row: 16 chunks of 16
constexpr int kRunBytes = 16 * kRunRow;
constexpr int kBlocked = -1;                 // x is in blocks already

// Where a workgroup's LDS holds what: the waves' runs of W (and of x in blocks); then
// x's codes [block][token], its scales [token] and W's [row], rows of `pitch` bytes, an
// odd number of 4.
struct FewLds8 {
    int runs, pitch, x, sx, sw, bytes;
};
template <int XF, int NW>
__host__ __device__ __forceinline__ FewLds8 few_lds8(int nb, int m) {
    FewLds8 o;
    o.runs = (nb + kRun - 1) / kRun;
    o.pitch = ((o.runs * kRun + 3) / 4 | 1) * 4;
    o.x = NW * kRunBytes * (XF == kBlocked ? 2 : 1);
    o.sx = o.x + (XF == kBlocked ? 0 : o.runs * kRun * m * kFp8Block);
    o.sw = o.sx + m * o.pitch;
    o.bytes = o.sw + 16 * o.pitch;
    return o;
}

// NW waves; XF: the format of x, or kBlocked.
template <int XF, int NW>
__device__ __forceinline__ void fp8_few(const Fp8Few& p) {
    constexpr int kT = 64 * NW, kF = XF == kBlocked ? FSDP_F32 : XF, kEs = kF == FSDP_F32 ? 4 : 2;
    constexpr int kRing = kRunBytes * (XF == kBlocked ? 2 : 1);
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int tid = threadIdx.x, l = tid & 63, r16 = l & 15, q = l >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int nb = (int)p.nb, m = (int)p.m, rowbytes = nb * kFp8Block;
    const int rows = (int)(p.n - n0 < 16 ? p.n - n0 : 16);
    const FewLds8 at = few_lds8<XF, NW>(nb, m);
    const int tok = r16 < m ? r16 : m - 1;
    uint8_t* ring = lds + w * kRing;

    // Rows behind W and tokens behind x are read as the last ones; nobody stores what
    // they give.  Chunk c of row r of a run lies at slot c ^ r of the row's 256 bytes, so
    // that 16 rows' equal chunks lie in different banks.
    const auto wr = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + n0 * rowbytes), 0, rows * rowbytes, kRsrcWord3);
    const auto xr = __builtin_amdgcn_make_buffer_rsrc((void*)p.x, 0, XF == kBlocked ? m * rowbytes : 0, kRsrcWord3);
    auto send16 = [&](bool of_x, int u) {
        const int left = (nb - u * kRun) * (kFp8Block / 16);     // chunks behind the row: the run's first one again
        const int soff = __builtin_amdgcn_readfirstlane(u * kRunRow), last = (of_x ? m : rows) - 1;
        uint8_t* to = ring + (of_x ? kRunBytes : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + q, c = r16 ^ r;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(of_x ? xr : wr, (__attribute__((address_space(3))) void*)(to + i * 1024), 16,
                                                     (r < last ? r : last) * rowbytes + (c < left ? c : 0) * 16, soff,
                                                     0, 0);
        }
    };
    auto send = [&](int u) {
        send16(false, u);
        if constexpr (XF == kBlocked) send16(true, u);
    };

    // Lane i % 16 of block i / 16: block b of token t is number b * m + t.  Nothing behind the last one.
    auto load_x = [&](int i) {
        const int b = i / 16 / m, t = i / 16 - b * m;
        const int64_t left = p.k - (int64_t)b * kFp8Block - i % 16 * 8;
        return load_upto8<kF>((const char*)p.x + (t * p.ldx + (int64_t)b * kFp8Block + i % 16 * 8) * kEs, left);
    };
    auto put_x = [&](int i, const Raw8<kF>& v) {
        const uint32_t s = fp8_scale_byte(max_of_16(mag_bits<kF>(max_mag<kF>(0, v))));
        const int b = i / 16 / m, t = i / 16 - b * m;
        *reinterpret_cast<u32x2*>(lds + at.x + i / 16 * kFp8Block + ((i % 16 / 2) ^ (t >> 1)) * 16 + i % 2 * 8) =
            fp8_codes8<kF>(v, s);
        if (i % 16 == 0) lds[at.sx + t * at.pitch + b] = (uint8_t)s;
    };
    // The scales of W's rows, and of x in blocks, four at a time.  Behind the last block both
    // sides get 2^-127, and what the codes there multiply to vanishes.
    const int dwords = (at.runs * kRun + 3) / 4;
    auto scales4 = [&](const uint8_t* s, int b) {
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) v |= (uint32_t)s[b + e < nb ? b + e : nb - 1] << (8 * e);
        const int left = nb - b;
        return left >= 4 ? v : (left <= 0 ? 0u : v & ((1u << (8 * left)) - 1));
    };
    auto load_s = [&](int i) {
        const int r = i / dwords, b = (i - r * dwords) * 4;
        if (XF == kBlocked && r >= 16) return scales4(p.sx + ((int64_t)(r - 16) >> p.tx) * nb, b);
        return scales4(p.sw + ((n0 + (r < rows ? r : rows - 1)) >> p.tw) * nb, b);
    };
    auto put_s = [&](int i, uint32_t v) {
        const int r = i / dwords;
        *reinterpret_cast<uint32_t*>(lds + (r < 16 ? at.sw + r * at.pitch : at.sx + (r - 16) * at.pitch) + (i - r * dwords) * 4) = v;
    };

    const bool some = w < at.runs;
    if (nb > 0) {
        // x's and the scales' first loads go out before W's, so that the wait for them is
        // not one for W.  The branches hold the same code: the compiler's wait after a
        // join would be the one of the way without W's loads.
        const int nx = XF == kBlocked ? 0 : at.runs * kRun * m * 16, ns = (XF == kBlocked ? 16 + m : 16) * dwords;
        Raw8<kF> x0{};
        if constexpr (XF != kBlocked) x0 = load_x(tid < nx ? tid : tid & 15);
        const uint32_t s0 = load_s(tid < ns ? tid : 0);
        auto rest = [&]() {
            if (tid < ns) put_s(tid, s0);
            for (int i = tid + kT; i < ns; i += kT) put_s(i, load_s(i));
            if constexpr (XF != kBlocked) {
                if (tid < nx) put_x(tid, x0);
                for (int i = tid + kT; i < nx; i += kT) put_x(i, load_x(i));
            }
        };
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        if (some) {
            send(w);
            __builtin_amdgcn_sched_barrier(0);
            rest();
        } else {
            rest();
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();            // W's loads stay on their way
        asm volatile("" ::: "memory");
    }

    f32x4 acc = f32x4{0, 0, 0, 0};
    for (int u = w; u < at.runs; u += NW) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        u32x4 c[kRun][2], x[kRun][2];
#pragma unroll
        for (int k = 0; k < kRun; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int chunk = k * 8 + e * 4 + q, slot = r16 * kRunRow + (chunk ^ r16) * 16;
                c[k][e] = *reinterpret_cast<const u32x4*>(ring + slot);
                if constexpr (XF == kBlocked) x[k][e] = *reinterpret_cast<const u32x4*>(ring + kRunBytes + slot);
                else
                    x[k][e] = *reinterpret_cast<const u32x4*>(lds + at.x + ((u * kRun + k) * m + tok) * kFp8Block +
                                                              ((e * 4 + q) ^ (tok >> 1)) * 16);
            }
        const uint32_t tw = *reinterpret_cast<const uint16_t*>(lds + at.sw + r16 * at.pitch + u * kRun);
        const uint32_t tx = *reinterpret_cast<const uint16_t*>(lds + at.sx + tok * at.pitch + u * kRun);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // the run's place is free
        __builtin_amdgcn_sched_barrier(0);
        if (u + NW < at.runs) send(u + NW);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const u32x4 *cw = c[k], *cx = x[k];
            const i32x8 aw = i32x8{(int)cw[0].x, (int)cw[0].y, (int)cw[0].z, (int)cw[0].w, (int)cw[1].x, (int)cw[1].y, (int)cw[1].z, (int)cw[1].w};
            const i32x8 bx = i32x8{(int)cx[0].x, (int)cx[0].y, (int)cx[0].z, (int)cx[0].w, (int)cx[1].x, (int)cx[1].y, (int)cx[1].z, (int)cx[1].w};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aw, bx, acc, 0, 0, 0, (int)(tw >> (8 * k)), 0, (int)(tx >> (8 * k)));
        }
    }

    __syncthreads();                                          // the sums take the runs' place
    f32x4* part = reinterpret_cast<f32x4*>(lds);
    part[w * 64 + l] = acc;
    __syncthreads();
    if (w > 0 || r16 >= m) return;
    f32x4 s = part[l];
#pragma unroll
    for (int v = 1; v < NW; ++v) s += part[v * 64 + l];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (4 * q + e >= rows) break;
        const int64_t o = r16 * p.ldo + n0 + 4 * q + e;
        if (p.dt == FSDP_F32) store1<FSDP_F32>(p.out, o, s[e]);
        else if (p.dt == FSDP_F16) store1<FSDP_F16>(p.out, o, s[e]);
        else store1<FSDP_BF16>(p.out, o, s[e]);
    }
}

template <int XF, int NW>
__global__ __launch_bounds__(64 * NW) void k_fp8_few(Fp8Few p) {
    fp8_few<XF, NW>(p);
}

// More rows of W than a launch's work items allow go in launches of kFewRows, a
// multiple of a tile's rows.
constexpr int64_t kFewRows = 1 << 26;
template <int XF, int NW>
static hipError_t few(const Fp8Few& p) {
    const unsigned lds = (unsigned)few_lds8<XF, NW>((int)p.nb, (int)p.m).bytes;
    for (int64_t n0 = 0; n0 < p.n; n0 += kFewRows) {
        Fp8Few c = p;
        c.n = p.n - n0 < kFewRows ? p.n - n0 : kFewRows;
        c.w = p.w + n0 * p.nb * kFp8Block;
        c.sw = p.sw + (n0 >> p.tw) * p.nb;
        c.out = (char*)p.out + n0 * dt_bytes(p.dt);
        launch_lds(k_fp8_few<XF, NW>, dim3((unsigned)((c.n + 15) / 16)), dim3(64 * NW), lds, (hipStream_t)p.stream, c);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Waves: 8 where every one of 4 would have more than a run (x quantised on the way), or for
// at most a workgroup a CU (x in blocks); else 4.
template <int XF>
static hipError_t few_of(const Fp8Few& p) {
    const bool wide = XF == kBlocked ? p.n <= 16 * (int64_t)p.cus : p.nb > 4 * kRun;
    return wide ? few<XF, 8>(p) : few<XF, 4>(p);
}

hipError_t launch_fp8_few(const Fp8Few& p) {
    if (p.sx) return few_of<kBlocked>(p);
    if (p.xdt == FSDP_F32) return few_of<FSDP_F32>(p);
    if (p.xdt == FSDP_F16) return few_of<FSDP_F16>(p);
    return few_of<FSDP_BF16>(p);
}

}  // namespace fsdp
