// fsdp_rms_grads.hip -- gfx950 kernels of the gradients of the root-mean-square norm.
//
//   g = dy * w,  dx = r * (g - h * (r^2 * sum(g * h) / d)) + dh,  dw = sum over rows of dy * (h * r)
//
// The memory bounds it: 8 bytes an element in bf16.  A workgroup takes a row at a time, in
// registers from its one read to its last use, with the next one's loads on their way; the
// row's sum is held in 64 bits as the forward's is.  Above 8192 features nothing is loaded
// ahead, and the 128 registers a lane do not hold it all: up to 38 are spilled, 73 to 289
// where rows are ragged or longer than 16384 (ragged rows with fp32 in them spill up to 22
// below 8192 too).  4096 x 12288 bf16 112 us (3.6 TB/s), with fp32 h 342 (2.1), 4096 x 12287
// bf16 245 (1.7), 2048 x 20001 390 (0.8).
// dw is added up by each workgroup over its rows in 32 bits, and the workgroups' sums by a
// second launch in their order: no atomics, so the same call gives the same bits.  Measured:
// 8192 x 8192 bf16 108 us (5.0 TB/s), 8191 x 8192 with fp32 h, dh and dx 184 us (5.1),
// 1000 x 1600 fp16 11.1 us, of which the second launch has a third.
#include "fsdp_rms_device.h"

#pragma clang fp contract(off)

namespace fsdp {

template <int DF, int HF, int U>
struct RmsRow {
    Raw8<DF> dy[U];
    Raw8<HF> h[U], dh[U];
    float r;
};

// Part b of the partial sums of dw: rows b, b + grid, ...
template <int DF, int HF, int U, bool WHOLE>
__global__ __launch_bounds__(1024) void k_rms_grads(RmsBackward p) {
    constexpr int kDs = DF == FSDP_F32 ? 4 : 2, kHs = HF == FSDP_F32 ? 4 : 2;
    __shared__ double part[2][16];
    const int d = (int)p.d, t = threadIdx.x, T = blockDim.x;
    float acc[U][8] = {}, w[U][8];
    auto load = [&](int64_t row) {
        RmsRow<DF, HF, U> o;
        const char *dy = (const char*)p.dy + row * p.ldy * kDs, *h = (const char*)p.h + row * p.ldh * kHs;
#pragma unroll
        for (int u = 0; u < U; ++u) o.dy[u] = load_row8<DF, WHOLE>(dy, (u * T + t) * 8, d);
#pragma unroll
        for (int u = 0; u < U; ++u) o.h[u] = load_row8<HF, WHOLE>(h, (u * T + t) * 8, d);
        // without dh: h's lines once more, whose values nobody uses
        const char* dh = p.dh ? (const char*)p.dh + row * p.lddh * kHs : h;
#pragma unroll
        for (int u = 0; u < U; ++u) o.dh[u] = load_row8<HF, WHOLE>(dh, (u * T + t) * 8, d);
        o.r = p.rstd[row];
        return o;
    };
    int turn = 0;
    constexpr bool kAhead = U == 1;        // more do not fit the registers twice
    RmsRow<DF, HF, U> next;
    if (kAhead) next = load(blockIdx.x);
#pragma unroll
    for (int u = 0; u < U; ++u) any_row8<WHOLE>(p.weight, p.wdt, (u * T + t) * 8, d, w[u]);
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        RmsRow<DF, HF, U> x = kAhead ? next : load(row);
        if (kAhead && row + gridDim.x < p.m) next = load(row + gridDim.x);
        double q = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float y[8], v[8];
            row8<DF, WHOLE>(x.dy[u], (u * T + t) * 8, d, y);
            row8<HF, WHOLE>(x.h[u], (u * T + t) * 8, d, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                q = __builtin_fma((double)(y[k] * w[u][k]), (double)v[k], q);
                acc[u][k] += y[k] * (v[k] * x.r);
            }
        }
        if (!p.dx) continue;
        // dx may be dh, and a ragged row's last lanes load what others will store: not only
        // dy and h, of which the sum was made, but dh too is here before the sum's barrier
        if constexpr (!WHOLE) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < (HF == FSDP_F32 ? 8 : 4); ++k) asm volatile("" : "+v"(x.dh[u].w[k]));
        }
        q = row_sum(q, part[turn]);
        turn ^= 1;
        const float f = (float)(q / (double)d * (double)x.r * (double)x.r);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * 8;
            float y[8], v[8], e[8];
            row8<DF, WHOLE>(x.dy[u], c, d, y);
            row8<HF, WHOLE>(x.h[u], c, d, v);
            row8<HF, WHOLE>(x.dh[u], c, d, e);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = x.r * (y[k] * w[u][k] - v[k] * f);
                if (p.dh) v[k] += e[k];
            }
            store_row8<HF, WHOLE>((char*)p.dx + row * p.lddx * kHs, c, d, v);
        }
    }
    if (!p.dw) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * T + t) * 8;
        if (p.parts) store_row8<FSDP_F32, WHOLE>((char*)(p.parts + (int64_t)blockIdx.x * d), c, d, acc[u]);
        else any_store8<WHOLE>(p.dw, p.dwdt, c, d, acc[u]);
    }
}

// dw from its partial sums: a workgroup takes 64 columns, 16 lanes of four columns for
// each of 64 shares of the parts, whose sums are added in LDS in their order.
__global__ __launch_bounds__(1024) void k_rms_dw(const float* __restrict__ parts, int n, int d, void* __restrict__ dw, int dt) {
    __shared__ float sums[64][65];
    const int g = threadIdx.x / 16, c = threadIdx.x % 16 * 4, col = blockIdx.x * 64 + c;
    float s[4] = {};
    if (col + 4 <= d) {
#pragma unroll 8
        for (int i = g; i < n; i += 64) {
            const u32x4 v = *(const u32x4_any*)(parts + (int64_t)i * d + col);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += __uint_as_float(v[k]);
        }
    } else {
        for (int i = g; i < n; i += 64)
            for (int k = 0; k < 4; ++k)
                if (col + k < d) s[k] += parts[(int64_t)i * d + col + k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[g][c + k] = s[k];
    __syncthreads();
    const int64_t o = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x >= 64 || o >= d) return;
    float x = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 64; ++i) x += sums[i][threadIdx.x];
    if (dt == FSDP_F32) store1<FSDP_F32>(dw, o, x);
    else if (dt == FSDP_F16) store1<FSDP_F16>(dw, o, x);
    else store1<FSDP_BF16>(dw, o, x);
}

// Up to 1024 lanes with a unit each, and the next row's loads ahead; with two units those
// do not fit (8192 x 8192 with fp32 h: 185 us against 326 with two units and none ahead).
constexpr int kOneUnit = 8192;

// Workgroups, each with a partial sum of dw: enough waves for the CUs, but no more than an
// eighth of the rows, whose partial sums then cost an eighth of the rows' own bytes, where
// that leaves a workgroup a CU.
int64_t rms_parts(int64_t m, int64_t d) {
    const int64_t waves = rms_lanes(d, kOneUnit) / 64, most = 4096 / waves < kRmsParts ? 4096 / waves : kRmsParts;
    const int64_t want = m / 8 > 256 ? m / 8 : (m < 256 ? m : 256);
    return want < most ? want : most;
}

template <int DF, int HF, int U, bool WHOLE>
struct Backward {
    static constexpr int kOne = kOneUnit;
    static hipError_t run(const RmsBackward& p, hipStream_t st) {
        launch(k_rms_grads<DF, HF, U, WHOLE>, dim3((unsigned)rms_parts(p.m, p.d)), dim3(rms_lanes(p.d, kOne)), st, p);
        return hipGetLastError();
    }
};

hipError_t launch_rms_backward(const RmsBackward& p, void* stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (p.m > 0) {
        hipError_t e = by_formats<Backward>(p, p.ydt, p.hdt, st);
        if (e != hipSuccess) return e;
    }
    if (p.dw && p.m != 1) {
        launch(k_rms_dw, dim3((unsigned)((p.d + 63) / 64)), dim3(1024), st, (const float*)p.parts, (int)rms_parts(p.m, p.d),
               (int)p.d, p.dw, p.dwdt);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace fsdp
