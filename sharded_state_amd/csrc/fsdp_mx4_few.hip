// fsdp_mx4_few.hip -- the product with W for a few tokens on gfx950: y = x W^T
// with W in 4-bit blocks along k, and x in such blocks too or quantised on the
// way, in the same launch.
//
// With up to 16 tokens the product is one read of W: 17/32 byte an element, two
// operations each.  A workgroup takes 16 rows of W, a wave every NW-th run of 16
// blocks along k of them: a run is 16 rows of 256 bytes, which go from memory to
// LDS without registers, and from there into the operands of
// v_mfma_scale_f32_16x16x128_f8f6f4 (lane l brings row l % 16 and block l / 16 of
// four).  Loaded straight into the operands, 16 lanes of a load lie in 16 rows: 10.1
// million cache accesses instead of 3.5 for one token through 28672 x 8192, and 28.3
// us instead of 24.1.  A wave's run is on its way while it multiplies the
// one before, and no barrier stands between runs.  x is quantised by the whole
// workgroup, a block a lane, into LDS, and the rows' scales are brought there, while
// the first runs are on their way; quantised by every wave for itself, x cost more
// than W (one token through 28672 x 8192 34.3 us, 16 tokens 41.0).  The waves' sums
// are added in LDS in their order.
//
// Measured in replayed graphs with W rotated past the caches, one token, us: 28672
// x 8192 24.1 (5.2 TB/s; quantisation and a product in tiles 34.8), 8192 x 28672
// 25.7 (54.5), 8192 x 8192 9.7 (19.8), 5120 x 1280 4.6 (6.9), 1280 x 5120 4.1 (10.6).
#include "fsdp_mx4_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRun = 16;                 // blocks along k that a wave takes at a time
constexpr int kRunBytes = 16 * kRun * 16;    // a run's codes of 16 rows
constexpr int kBlocked = -1;             // x is in blocks already

// Where a workgroup's LDS holds what: the waves' runs of W (and of x in blocks);
// then x's codes [block][token], its scales [token] and W's [row], rows of `pitch`
// bytes, an odd number of 16.
struct FewLds {
    int runs, pitch, x, sx, sw, bytes;
};
template <int XF, int NW>
__host__ __device__ __forceinline__ FewLds few_lds(int nb, int m) {
    FewLds o;
    o.runs = (nb + kRun - 1) / kRun;
    o.pitch = (o.runs | 1) * kRun;
    o.x = NW * kRunBytes * (XF == kBlocked ? 2 : 1);
    o.sx = o.x + o.runs * kRun * m * 16;
    o.sw = o.sx + m * o.pitch;
    o.bytes = XF == kBlocked ? o.x : o.sw + 16 * o.pitch;
    return o;
}

// NW waves; XF: the format of x, or kBlocked.
template <int XF, int NW>
__device__ __forceinline__ void mx4_few(const Mx4Few& p) {
    constexpr int kT = 64 * NW, kF = XF == kBlocked ? FSDP_F32 : XF, kEs = kF == FSDP_F32 ? 4 : 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int tid = threadIdx.x, l = tid & 63, r16 = l & 15, q = l >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int nb = (int)p.nb, m = (int)p.m, rowbytes = nb * 16;
    const int rows = (int)(p.n - n0 < 16 ? p.n - n0 : 16);
    const FewLds at = few_lds<XF, NW>(nb, m);
    const int tok = r16 < m ? r16 : m - 1;
    uint8_t* ring = lds + w * kRunBytes * (XF == kBlocked ? 2 : 1);

    // Rows behind W and tokens behind x are read as the last ones; nobody stores what
    // they give.  Block c of row r of a run lies at slot c ^ r of the row's 256 bytes,
    // so that 16 rows' equal blocks lie in different banks.
    const auto wr = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + n0 * rowbytes), 0, rows * rowbytes, kRsrcWord3);
    const auto xr = __builtin_amdgcn_make_buffer_rsrc((void*)p.x, 0, XF == kBlocked ? m * rowbytes : 0, kRsrcWord3);
    auto send16 = [&](bool of_x, int u) {
        const int left = nb - u * kRun;          // blocks behind the row: the run's first one again
        const int soff = __builtin_amdgcn_readfirstlane(u * (kRun * 16)), last = (of_x ? m : rows) - 1;
        uint8_t* to = ring + (of_x ? kRunBytes : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + q, c = r16 ^ r;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(of_x ? xr : wr, (__attribute__((address_space(3))) void*)(to + i * 1024), 16,
                                                     (r < last ? r : last) * rowbytes + (c < left ? c : 0) * 16, soff,
                                                     0, 0);
        }
    };
    const uint8_t* const swr = p.sw + (n0 + (r16 < rows ? r16 : rows - 1)) * nb;
    u32x4 sw, sx;                                // the run's scales, where x is in blocks
    auto send = [&](int u) {
        send16(false, u);
        if constexpr (XF == kBlocked) {
            send16(true, u);
            sw = scales16(swr + u * kRun, nb - u * kRun);
            sx = scales16(p.sx + (int64_t)tok * nb + u * kRun, nb - u * kRun);
        }
    };

    struct Block {
        Raw8<kF> v[4];
    };
    // Block i / m of token i % m; nothing behind the last one.
    auto load_x = [&](int i) {
        const int b = i / m, t = i - b * m;
        const int64_t left = p.k - (int64_t)b * kMx4Block;
        const char* x = (const char*)p.x + (t * p.ldx + (int64_t)b * kMx4Block) * kEs;
        Block o{};
        if (left <= 0) return o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (left >= kMx4Block) o.v[j] = load8_raw<kF>(x + j * 8 * kEs);
            else o.v[j] = load_upto8<kF>(x + j * 8 * kEs, left - j * 8);
        }
        return o;
    };
    auto put_x = [&](int i, const Block& o) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = max_mag<kF>(a, o.v[j]);
        const uint32_t s = scale_byte(mag_bits<kF>(a));
        *reinterpret_cast<u32x4*>(lds + at.x + i * 16) =
            u32x4{codes8<kF>(o.v[0], s), codes8<kF>(o.v[1], s), codes8<kF>(o.v[2], s), codes8<kF>(o.v[3], s)};
        lds[at.sx + i % m * at.pitch + i / m] = (uint8_t)s;
    };
    auto load_s = [&](int i) {
        const int r = i / at.runs, b = (i - r * at.runs) * kRun;
        return scales16(p.sw + (n0 + (r < rows ? r : rows - 1)) * nb + b, nb - b);
    };
    auto put_s = [&](int i, u32x4 v) {
        const int r = i / at.runs;
        *reinterpret_cast<u32x4*>(lds + at.sw + r * at.pitch + (i - r * at.runs) * kRun) = v;
    };

    const bool some = w < at.runs;
    if constexpr (XF == kBlocked) {
        if (some) send(w);
    } else if (nb > 0) {
        // x's and the scales' first loads go out before W's, so that the wait for them is
        // not one for W.  The branches hold the same code: the compiler's wait after a
        // join would be the one of the way without W's loads.
        const int nx = at.runs * kRun * m, ns = 16 * at.runs;
        const Block x0 = load_x(tid < nx ? tid : 0);
        const u32x4 s0 = load_s(tid < ns ? tid : 0);
        auto rest = [&]() {
            if (tid < ns) put_s(tid, s0);
            if (tid < nx) put_x(tid, x0);
            for (int i = tid + kT; i < nx; i += kT) put_x(i, load_x(i));
            for (int i = tid + kT; i < ns; i += kT) put_s(i, load_s(i));
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
        u32x4 c[4], x[4], tw, tx;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int slot = r16 * 256 + ((4 * k + q) ^ r16) * 16;
            c[k] = *reinterpret_cast<const u32x4*>(ring + slot);
            if constexpr (XF == kBlocked) x[k] = *reinterpret_cast<const u32x4*>(ring + kRunBytes + slot);
            else x[k] = *reinterpret_cast<const u32x4*>(lds + at.x + ((u * kRun + 4 * k + q) * m + tok) * 16);
        }
        if constexpr (XF == kBlocked) {
            tw = sw;
            tx = sx;
        } else {
            tw = *reinterpret_cast<const u32x4*>(lds + at.sw + r16 * at.pitch + u * kRun);
            tx = *reinterpret_cast<const u32x4*>(lds + at.sx + tok * at.pitch + u * kRun);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // the run's place is free
        __builtin_amdgcn_sched_barrier(0);
        if (u + NW < at.runs) send(u + NW);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // behind the last block both scales are 2^-127, and what the codes there multiply to vanishes
            const i32x8 aw = i32x8{(int)c[k].x, (int)c[k].y, (int)c[k].z, (int)c[k].w, 0, 0, 0, 0};
            const i32x8 bx = i32x8{(int)x[k].x, (int)x[k].y, (int)x[k].z, (int)x[k].w, 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aw, bx, acc, 4, 4, 0, (int)(tw[k] >> (8 * q)), 0,
                                                                  (int)(tx[k] >> (8 * q)));
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
__global__ __launch_bounds__(64 * NW) void k_mx4_few(Mx4Few p) {
    mx4_few<XF, NW>(p);
}

// More rows of W than a launch's work items allow go in launches of kFewRows.
constexpr int64_t kFewRows = 1 << 26;
template <int XF, int NW>
static hipError_t few(const Mx4Few& p) {
    const unsigned lds = (unsigned)few_lds<XF, NW>((int)p.nb, (int)p.m).bytes;
    for (int64_t n0 = 0; n0 < p.n; n0 += kFewRows) {
        Mx4Few c = p;
        c.n = p.n - n0 < kFewRows ? p.n - n0 : kFewRows;
        c.w = p.w + n0 * p.nb * 16;
        c.sw = p.sw + n0 * p.nb;
        c.out = (char*)p.out + n0 * dt_bytes(p.dt);
        launch_lds(k_mx4_few<XF, NW>, dim3((unsigned)((c.n + 15) / 16)), dim3(64 * NW), lds, (hipStream_t)p.stream, c);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Waves.  x quantised on the way: 8, or 4 where no wave would have a run of its own
// (one token, us: 28672 x 8192 24.1 against 26.2, 1280 x 5120 4.1 and 4.5; but 5120 x
// 1280 4.6 with 4, 5.1 with 8).  x in blocks: 8 for at most a workgroup a CU, else 4
// (16 tokens: 1280 x 5120 4.3 against 4.9, 700 x 9000 6.6 and 7.7; but 8192 x 28672
// 28.3 with 4, 32.3 with 8, and 40000 x 512 7.5 and 10.0).
template <int XF>
static hipError_t few_of(const Mx4Few& p) {
    const bool wide = XF == kBlocked ? p.n <= 16 * (int64_t)p.cus : p.nb > 4 * kRun;
    return wide ? few<XF, 8>(p) : few<XF, 4>(p);
}

hipError_t launch_mx4_few(const Mx4Few& p) {
    if (p.sx) return few_of<kBlocked>(p);
    if (p.xdt == FSDP_F32) return few_of<FSDP_F32>(p);
    if (p.xdt == FSDP_F16) return few_of<FSDP_F16>(p);
    return few_of<FSDP_BF16>(p);
}

}  // namespace fsdp
