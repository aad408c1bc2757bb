// fsdp_mx4_few.hip -- the linear product for a few tokens on gfx950: y = x W^T
// with W in 4-bit blocks along k and x quantised on the way, one launch.
//
// With up to 32 tokens the product is one read of W: 17/32 byte an element, two
// operations each.  So nothing of W passes through LDS: a wave takes FR times 16
// rows of W and every 8th run of 16 blocks along k, fetches the run's codes and
// scales straight into the operands of v_mfma_scale_f32_16x16x128_f8f6f4 (lane l
// brings row l % 16 and block l / 16 of four), and quantises the tokens' blocks
// itself, a block a lane, while those loads are on their way.  The 8 waves' sums
// are added in LDS in their order.  FR is as large as leaves every CU a
// workgroup: the quantisation of x is shared by the rows of a wave.
#include <type_traits>

#include "fsdp_mx4_device.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 8;
constexpr int kRun = 16;                 // blocks along k that a wave takes at a time

template <int XF, int FR, int FT>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx4_few(Mx4Few p) {
    constexpr int kEs = XF == FSDP_F32 ? 4 : 2;
    __shared__ f32x4 part[kFewWaves][FR][FT][64];
    const int l = threadIdx.x & 63, r16 = l & 15, q = l >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * FR);
    const int64_t nb = p.nb, runs = (nb + kRun - 1) / kRun;

    f32x4 acc[FR][FT];
#pragma unroll
    for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int t = 0; t < FT; ++t) acc[f][t] = f32x4{0, 0, 0, 0};

    // Rows behind W and tokens behind x are read as the last ones; nobody stores what they give.
    const uint8_t* wrow[FR];
    const uint8_t* srow[FR];
    const char* xrow[FT];
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int64_t r = n0 + f * 16 + r16, row = r < p.n ? r : p.n - 1;
        wrow[f] = p.w + row * nb * 16 + q * 16;
        srow[f] = p.sw + row * nb;
    }
#pragma unroll
    for (int t = 0; t < FT; ++t) {
        const int64_t tok = t * 16 + r16 < p.m ? t * 16 + r16 : p.m - 1;
        xrow[t] = (const char*)p.x + (tok * p.ldx + q * kMx4Block) * kEs;
    }
    // 16 blocks from b0 on; with `full` all of them are there, whole.
    auto run = [&](int64_t b0, auto full) {
        constexpr bool kFull = decltype(full)::value;
        u32x4 cw[FR][4];
        uint32_t sw[FR][4];
#pragma unroll
        for (int f = 0; f < FR; ++f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (kFull || b0 + 4 * k + q < nb) cw[f][k] = *reinterpret_cast<const u32x4*>(wrow[f] + (b0 + 4 * k) * 16);
                else cw[f][k] = u32x4{0, 0, 0, 0};
            }
            u32x4 sc = u32x4{0, 0, 0, 0};
            if constexpr (kFull) {
                sc = *(const u32x4_any*)(srow[f] + b0);
            } else {
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (b0 + j < nb) sc[j / 4] |= (uint32_t)srow[f][b0 + j] << (8 * (j % 4));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) sw[f][k] = sc[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            i32x8 bx[FT];
            int sx[FT];
#pragma unroll
            for (int t = 0; t < FT; ++t) {
                const char* x = xrow[t] + (b0 + 4 * k) * (kMx4Block * kEs);
                const int64_t left = p.k - (b0 + 4 * k + q) * kMx4Block;
                Raw8<XF> v[4];
                uint32_t a = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (kFull) v[j] = load8_raw<XF>(x + j * 8 * kEs);
                    else v[j] = load_upto8<XF>(x + j * 8 * kEs, left - j * 8);
                    a = max_mag<XF>(a, v[j]);
                }
                const uint32_t s = scale_byte(mag_bits<XF>(a));
                sx[t] = (int)s;
                bx[t] = i32x8{(int)codes8<XF>(v[0], s), (int)codes8<XF>(v[1], s), (int)codes8<XF>(v[2], s),
                              (int)codes8<XF>(v[3], s), 0, 0, 0, 0};
            }
#pragma unroll
            for (int f = 0; f < FR; ++f) {
                const i32x8 aw = i32x8{(int)cw[f][k].x, (int)cw[f][k].y, (int)cw[f][k].z, (int)cw[f][k].w, 0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < FT; ++t)
                    acc[f][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aw, bx[t], acc[f][t], 4, 4, 0,
                                                                                (int)(sw[f][k] >> (8 * q)), 0, sx[t]);
            }
        }
    };
    const int64_t whole = p.k / (kRun * kMx4Block);
    int64_t u = w;
    for (; u < whole; u += kFewWaves) run(u * kRun, std::true_type{});
    if (u < runs) run(u * kRun, std::false_type{});
#pragma unroll
    for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int t = 0; t < FT; ++t) part[w][f][t][l] = acc[f][t];
    __syncthreads();
    for (int i = threadIdx.x; i < FR * FT * 64; i += 64 * kFewWaves) {
        const f32x4* at = &part[0][0][0][0] + i;
        f32x4 s = at[0];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) s += at[v * FR * FT * 64];
        const int f = i / (FT * 64), t = i / 64 % FT, lane = i % 64;
        const int64_t tok = t * 16 + (lane & 15), n = n0 + f * 16 + (lane >> 4) * 4;
        if (tok >= p.m) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= p.n) break;
            const int64_t o = tok * p.ldo + n + e;
            if (p.dt == FSDP_F32) store1<FSDP_F32>(p.out, o, s[e]);
            else if (p.dt == FSDP_F16) store1<FSDP_F16>(p.out, o, s[e]);
            else store1<FSDP_BF16>(p.out, o, s[e]);
        }
    }
}

template <int XF, int FR>
static hipError_t few_rows(const Mx4Few& p) {
    const dim3 g((unsigned)((p.n + 16 * FR - 1) / (16 * FR))), th(64 * kFewWaves);
    if (p.m <= 16) launch(k_mx4_few<XF, FR, 1>, g, th, (hipStream_t)p.stream, p);
    else launch(k_mx4_few<XF, FR, 2>, g, th, (hipStream_t)p.stream, p);
    return hipGetLastError();
}

template <int XF>
static hipError_t few(const Mx4Few& p) {
    if (p.n >= 64 * (int64_t)p.cus) return few_rows<XF, 4>(p);
    if (p.n >= 32 * (int64_t)p.cus) return few_rows<XF, 2>(p);
    return few_rows<XF, 1>(p);
}

hipError_t launch_mx4_few(const Mx4Few& p) {
    if (p.n / 16 >= (int64_t(1) << 32) / (64 * kFewWaves)) return hipErrorInvalidValue;
    if (p.xdt == FSDP_F32) return few<FSDP_F32>(p);
    if (p.xdt == FSDP_F16) return few<FSDP_F16>(p);
    return few<FSDP_BF16>(p);
}

}  // namespace fsdp
