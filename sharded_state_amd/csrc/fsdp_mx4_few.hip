// fsdp_mx4_few.hip -- the product with W for a few tokens on gfx950: y = x W^T
// with W in 4-bit blocks along k, and x in such blocks too or quantised on the
// way, in the same launch.
//
// With up to 16 tokens the product is one read of W: 17/32 byte an element, two
// operations each.  So nothing of W passes through LDS: a wave takes FR times 16
// rows of W and every NW-th run of 16 blocks along k, fetches the run's codes and
// scales straight into the operands of v_mfma_scale_f32_16x16x128_f8f6f4 (lane l
// brings row l % 16 and block l / 16 of four), one run ahead of the one that it
// multiplies.  x is quantised by the whole workgroup, a block a lane, into LDS
// while the first runs are on their way; quantised by every wave for itself, 16
// lanes a token or none, it cost more than W (one token through 28672 x 8192
// 34.3 us, 16 tokens 41.0).  The waves' sums are added in LDS in their order.
//
// Measured in replayed graphs with W rotated past the caches, one token, us: 28672
// x 8192 27.6 (4.5 TB/s; quantisation and a product in tiles 34.8), 8192 x 28672
// 28.3 (54.5), 8192 x 8192 11.8 (19.8), 5120 x 1280 4.6 (6.9), 1280 x 5120 5.6 (10.6).
#include <type_traits>

#include "fsdp_mx4_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRun = 16;                 // blocks along k that a wave takes at a time
constexpr int kBlocked = -1;             // x is in blocks already

// NW waves, FR x 16 rows of W a wave; XF: the format of x, or kBlocked.
template <int XF, int NW, int FR>
__global__ __launch_bounds__(64 * NW) void k_mx4_few(Mx4Few p) {
    constexpr int kT = 64 * NW;
    extern __shared__ uint8_t lds[];     // x's codes [block][token], its scales; then the sums
    const int l = threadIdx.x & 63, r16 = l & 15, q = l >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * FR);
    const int64_t nb = p.nb;
    const int m = (int)p.m;

    // Rows behind W and tokens behind x are read as the last ones; nobody stores what they give.
    const uint8_t* wrow[FR];
    const uint8_t* srow[FR];
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int64_t r = n0 + f * 16 + r16, row = r < p.n ? r : p.n - 1;
        wrow[f] = p.w + row * nb * 16 + q * 16;
        srow[f] = p.sw + row * nb;
    }
    const int tok = r16 < m ? r16 : m - 1;

    struct Run {
        u32x4 c[FR][4], s[FR];
    };
    // 16 blocks of W from b0 on; with `full` all of them are there.
    auto fetch = [&](Run& r, int64_t b0, auto full) {
        constexpr bool kFull = decltype(full)::value;
#pragma unroll
        for (int f = 0; f < FR; ++f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (kFull || b0 + 4 * k + q < nb) r.c[f][k] = *reinterpret_cast<const u32x4*>(wrow[f] + (b0 + 4 * k) * 16);
                else r.c[f][k] = u32x4{0, 0, 0, 0};
            }
            r.s[f] = scales16(srow[f] + b0, kFull ? kRun : (int)(nb - b0));
        }
    };
    const int64_t whole = nb / kRun, runs = (nb + kRun - 1) / kRun;
    int64_t u = w;
    Run cur;
    if (u < whole) fetch(cur, u * kRun, std::true_type{});
    else if (u < runs) fetch(cur, u * kRun, std::false_type{});

    const uint8_t* xs = lds + nb * m * 16;
    if constexpr (XF != kBlocked) {
        constexpr int kEs = XF == FSDP_F32 ? 4 : 2;
        for (int i = threadIdx.x; i < nb * m; i += kT) {
            const int b = i / m, t = i - b * m;          // tokens of a block next to each other
            const int64_t left = p.k - (int64_t)b * kMx4Block;
            const char* x = (const char*)p.x + (t * p.ldx + (int64_t)b * kMx4Block) * kEs;
            Raw8<XF> v[4];
            uint32_t a = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (left >= kMx4Block) v[j] = load8_raw<XF>(x + j * 8 * kEs);
                else v[j] = load_upto8<XF>(x + j * 8 * kEs, left - j * 8);
                a = max_mag<XF>(a, v[j]);
            }
            const uint32_t s = scale_byte(mag_bits<XF>(a));
            reinterpret_cast<u32x4*>(lds)[i] = u32x4{codes8<XF>(v[0], s), codes8<XF>(v[1], s), codes8<XF>(v[2], s),
                                                     codes8<XF>(v[3], s)};
            lds[nb * m * 16 + i] = (uint8_t)s;
        }
        __syncthreads();
    }

    f32x4 acc[FR];
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[f] = f32x4{0, 0, 0, 0};
    auto multiply = [&](const Run& r, int64_t b0, auto full) {
        constexpr bool kFull = decltype(full)::value;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t b = b0 + 4 * k + q;
            u32x4 c = u32x4{0, 0, 0, 0};
            int sx = 0;
            if (kFull || b < nb) {
                if constexpr (XF == kBlocked) {
                    c = *reinterpret_cast<const u32x4*>((const uint8_t*)p.x + (tok * nb + b) * 16);
                    sx = p.sx[tok * nb + b];
                } else {
                    c = reinterpret_cast<const u32x4*>(lds)[b * m + tok];
                    sx = xs[b * m + tok];
                }
            }
            const i32x8 bx = i32x8{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
#pragma unroll
            for (int f = 0; f < FR; ++f) {
                const i32x8 aw = i32x8{(int)r.c[f][k].x, (int)r.c[f][k].y, (int)r.c[f][k].z, (int)r.c[f][k].w, 0, 0, 0, 0};
                acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aw, bx, acc[f], 4, 4, 0,
                                                                         (int)(r.s[f][k] >> (8 * q)), 0, sx);
            }
        }
    };
    if (u < runs) {
        for (;;) {
            const int64_t v = u + NW;
            Run next;
            if (v < whole) fetch(next, v * kRun, std::true_type{});
            else if (v < runs) fetch(next, v * kRun, std::false_type{});
            if (u < whole) multiply(cur, u * kRun, std::true_type{});
            else multiply(cur, u * kRun, std::false_type{});
            if (v >= runs) break;
            cur = next;
            u = v;
        }
    }

    if constexpr (XF != kBlocked) __syncthreads();           // the sums take x's place
    f32x4* part = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int f = 0; f < FR; ++f) part[(w * FR + f) * 64 + l] = acc[f];
    __syncthreads();
    for (int i = threadIdx.x; i < FR * 64; i += kT) {
        f32x4 s = part[i];
#pragma unroll
        for (int v = 1; v < NW; ++v) s += part[v * FR * 64 + i];
        const int64_t to = i & 15, n = n0 + i / 64 * 16 + (i % 64 >> 4) * 4;
        if (to >= p.m) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= p.n) break;
            const int64_t o = to * p.ldo + n + e;
            if (p.dt == FSDP_F32) store1<FSDP_F32>(p.out, o, s[e]);
            else if (p.dt == FSDP_F16) store1<FSDP_F16>(p.out, o, s[e]);
            else store1<FSDP_BF16>(p.out, o, s[e]);
        }
    }
}

template <int XF, int NW, int FR>
static hipError_t few(const Mx4Few& p) {
    const dim3 g((unsigned)((p.n + 16 * FR - 1) / (16 * FR))), th(64 * NW);
    const unsigned sums = NW * FR * 1024;
    const unsigned x = XF == kBlocked ? 0 : (unsigned)((p.nb * p.m * 17 + 15) / 16 * 16);
    const unsigned lds = x > sums ? x : sums;
    launch_lds(k_mx4_few<XF, NW, FR>, g, th, lds, (hipStream_t)p.stream, p);
    return hipGetLastError();
}

// x quantised on the way: 4 waves of 16 rows, the most workgroups there are (8
// waves: 30.6 us instead of 27.6 at 28672 x 8192, 4.8 instead of 4.6 at 5120 x
// 1280).  x in blocks, 16 tokens: 8 waves, and 32 rows a wave, which share x's
// operands, where 16 would be more than a workgroup a CU (8192 x 28672: 33.9 us
// against 45.0 with 16 rows; 1280 x 5120: 6.0 with 16 rows, 7.3 with 32).
hipError_t launch_mx4_few(const Mx4Few& p) {
    if (p.n / 16 >= (int64_t(1) << 32) / 512 - 1) return hipErrorInvalidValue;   // work items of a launch
    if (p.sx) return p.n > 16 * (int64_t)p.cus ? few<kBlocked, 8, 2>(p) : few<kBlocked, 8, 1>(p);
    if (p.xdt == FSDP_F32) return few<FSDP_F32, 4, 1>(p);
    if (p.xdt == FSDP_F16) return few<FSDP_F16, 4, 1>(p);
    return few<FSDP_BF16, 4, 1>(p);
}

}  // namespace fsdp
