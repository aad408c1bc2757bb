// fsdp_rms.hip -- gfx950 kernel of the root-mean-square norm over features, with the
// residual's addition before it and 8-bit blocks behind it.
//
//   h = round(x + residual),  r = 1 / sqrt(sum(h^2) / d + eps),  y = (h * r) * w
//
// The memory bounds it: 7 bytes an element in bf16 (3 without a residual), 11 on a fp32
// stream.  A row stays in registers from its one read to its last use, and a workgroup that
// has more of them loads the next before it sums this one.  That holds up to 16384 features.
// Above, nothing is loaded ahead, and the 128 registers that 1024 lanes leave each of them do
// not hold it all: 9 to 41 are spilled, 193 to 391 where rows are ragged (ragged rows with
// fp32 in them spill up to 22 from 4096 features on).  The row's sum is held in 64 bits (a fp32 square overflows above 1.8e19),
// and so is the product, which is rounded to codes once: through fp32 one code in 2^20
// would come out as its neighbour, at a gain of 1 to 8% of the time.
// Measured: 8191 x 8192, bf16 on a fp32 stream, 140 us (5.3 TB/s), with y too 167; 8192 x
// 8192 bf16 89 us (5.3); 4096 x 12288 bf16 70 (5.0); 2048 x 32768 119 (4.0); ragged, 4096 x
// 12287 90 (3.9) and 2048 x 20001 202 (1.4); 1000 x 1600 fp16 5.8; one token of 1280 2.6.
#include "fsdp_rms_device.h"

#pragma clang fp contract(off)

namespace fsdp {

// z cut off after 20 bits behind the leading one, the last of them set where that left
// something out: rounded from there to a format of fewer bits, it is z rounded once, where
// fp32 holds those 20 bits (z from 2^-129 to below 2^128).
__device__ __forceinline__ uint32_t to_odd(double z) {
    const uint64_t b = __builtin_bit_cast(uint64_t, z);
    const uint32_t hi = (uint32_t)(b >> 32) | ((uint32_t)b != 0);
    return __float_as_uint((float)__builtin_bit_cast(double, (uint64_t)hi << 32));
}

// For a block with products that to_odd does not give: from 2^128 on, or with ties between
// codes among fp32's subnormals.  y: the high halves of eight products of a lane, the last
// bit set where the low half is not 0.  Gives the block's scale byte, and in y's place what
// is left of the products divided by the scale, which fp32 holds or is far under a tie.
__device__ __forceinline__ uint32_t far_scale(Raw8<FSDP_F32>& y) {
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) a = max(a, y.w[k] & 0x7fffffffu);
    a = max_of_16(a);
    const int e = (int)(a >> 20) - 1023 + 127 - 8 + ((a & 0xfffffu) > 0xc0000u);     // as fp8_scale_byte
    const uint32_t s = e > 254 ? 255u : (uint32_t)(e < 1 ? 1 : e);
    const double f = __builtin_bit_cast(double, (uint64_t)(1023 + 127 - (int)s) << 52);
#pragma unroll
    for (int k = 0; k < 8; ++k) y.w[k] = __float_as_uint((float)(__builtin_bit_cast(double, (uint64_t)y.w[k] << 32) * f));
    return s;
}

template <int XF, int HF, int U>
struct RmsIn {
    Raw8<XF> x[U];
    Raw8<HF> res[U];
};

template <int XF, int HF, int U, bool WHOLE>
__global__ __launch_bounds__(1024) void k_rms(RmsForward p) {
    constexpr int kXs = XF == FSDP_F32 ? 4 : 2, kHs = HF == FSDP_F32 ? 4 : 2;
    constexpr bool kAhead = U < 4;         // more do not fit the registers twice
    __shared__ double part[2][16];
    const int d = (int)p.d, t = threadIdx.x, T = blockDim.x, nb = (d + kFp8Block - 1) / kFp8Block;
    auto load = [&](int64_t row, RmsIn<XF, HF, U>& o) {
        const char* x = (const char*)p.x + row * p.ldx * kXs;
#pragma unroll
        for (int u = 0; u < U; ++u) o.x[u] = load_row8<XF, WHOLE>(x, (u * T + t) * 8, d);
        if (p.residual) {
            const char* res = (const char*)p.residual + row * p.ldr * kHs;
#pragma unroll
            for (int u = 0; u < U; ++u) o.res[u] = load_row8<HF, WHOLE>(res, (u * T + t) * 8, d);
        }
    };
    RmsIn<XF, HF, U> in;
    float w[U][8];
    load(blockIdx.x, in);
    if (kAhead) {
#pragma unroll
        for (int u = 0; u < U; ++u) any_row8<WHOLE>(p.weight, p.wdt, (u * T + t) * 8, d, w[u]);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        float v[U][8];
        double q = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            row8<XF, WHOLE>(in.x[u], (u * T + t) * 8, d, v[u]);
            if (p.residual) {
                float r[8];
                row8<HF, WHOLE>(in.res[u], (u * T + t) * 8, d, r);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[u][k] = round_to<HF>(v[u][k] + r[k]);
            }
        }
        if (kAhead && row + gridDim.x < p.m) load(row + gridDim.x, in);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 8; ++k) q = __builtin_fma((double)v[u][k], (double)v[u][k], q);
        q = row_sum(q, part[turn]);
        turn ^= 1;
        const double r = 1.0 / __builtin_sqrt(q / (double)d + p.eps);
        if (t == 0 && p.rstd) p.rstd[row] = (float)r;
        // stored only now: h may be the residual, of which every lane has its part by now
        if (p.residual) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                store_row8<HF, WHOLE>((char*)p.h + row * p.ldh * kHs, (u * T + t) * 8, d, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * 8;
            if (!kAhead) any_row8<WHOLE>(p.weight, p.wdt, c, d, w[u]);
            if (p.y) {
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) asm volatile("" : "+v"(v[u][k]), "+v"(w[u][k]));
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = (float)((double)v[u][k] * r * (double)w[u][k]);
                any_store8<WHOLE>((char*)p.y + row * p.ldy * (p.ydt == FSDP_F32 ? 4 : 2), p.ydt, c, d, y);
            }
            Raw8<FSDP_F32> y;
            uint32_t a = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                asm volatile("" : "+v"(v[u][k]), "+v"(w[u][k]));    // widened here, not kept wide
                y.w[k] = to_odd((double)v[u][k] * r * (double)w[u][k]);
                if (c + k >= d) y.w[k] = 0;                  // not 0 * infinity
                a = max(a, y.w[k] & 0x7fffffffu);
            }
            a = max_of_16(a);
            uint32_t s = fp8_scale_byte(a), by = s;
            // a tie is 2^(s - 137) at least, and to_odd needs 2^-129; zeros have none
            if (s == 255 || (s < 8 && a != 0)) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    asm volatile("" : "+v"(v[u][k]), "+v"(w[u][k]));
                    const uint64_t z = __builtin_bit_cast(uint64_t, (double)v[u][k] * r * (double)w[u][k]);
                    y.w[k] = c + k < d ? (uint32_t)(z >> 32) | ((uint32_t)z != 0) : 0u;
                }
                s = far_scale(y);
                by = s == 255 ? 255u : 127u;
            }
            if (c < nb * kFp8Block) {
                *reinterpret_cast<u32x2*>(p.codes + row * nb * kFp8Block + c) = fp8_codes8<FSDP_F32>(y, by);
                if (t % 16 == 0) p.scales[row * nb + c / kFp8Block] = (uint8_t)s;
            }
        }
        if (!kAhead && row + gridDim.x < p.m) load(row + gridDim.x, in);
    }
}

// Workgroups of 24 waves a CU, half as many again as it holds at a time at these registers,
// so that no CU waits long for another's last row (4096 x 4096 bf16: 16 waves 28.7 us,
// 24 27.2, 32 28.4; a workgroup a row 31.3).  Two units a lane above 4096 features leave
// smaller workgroups, of which a CU holds two (8192 x 8192 92 us, 127 with one unit).
template <int XF, int HF, int U, bool WHOLE>
struct Forward {
    static constexpr int kOne = 4096;
    static hipError_t run(const RmsForward& p, hipStream_t st) {
        const int lanes = rms_lanes(p.d, kOne);
        const int64_t most = 256 * 24 / (lanes / 64);
        launch(k_rms<XF, HF, U, WHOLE>, dim3((unsigned)(p.m < most ? p.m : most)), dim3(lanes), st, p);
        return hipGetLastError();
    }
};

hipError_t launch_rms_forward(const RmsForward& p, void* stream) {
    return by_formats<Forward>(p, p.xdt, p.residual ? p.hdt : p.xdt, (hipStream_t)stream);
}

}  // namespace fsdp
