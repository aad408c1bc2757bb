// fsdp_rms.hip -- gfx950 kernels of the root-mean-square norm over features, with
// the residual's addition before it and 8-bit blocks behind it, and of its
// gradients.
//
//   h = round(x + residual),  r = 1 / sqrt(sum(h^2) / d + eps),  y = (h * r) * w
//   g = dy * w,  dx = r * (g - h * (r^2 * sum(g * h) / d)) + dh,  dw = sum over rows of dy * (h * r)
//
// A row stays in registers from its one read to its last use: eight elements a
// lane, U times.  Its two sums are held in 64 bits (a fp32 square overflows above
// 1.8e19), which costs nothing beside the memory: at 7 bytes an element a CU has
// some 80 lane-operations for each.  dw is added up by each workgroup over its rows
// in 32 bits, and the workgroups' sums by a second launch in their order: no
// atomics, so the same call gives the same bits.
#include <type_traits>

#include "fsdp_fp8_device.h"
#include "fsdp_rms.h"

#pragma clang fp contract(off)

namespace fsdp {

// Eight elements of a row of any of the formats as they lie in memory.
typedef Raw8<FSDP_F32> Raw;

template <int F>
__device__ __forceinline__ void to_floats(const Raw8<F>& r, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (F == FSDP_F32) v[k] = __uint_as_float(r.w[k]);
        else v[k] = to_f32<F>(k & 1 ? r.w[k / 2] >> 16 : r.w[k / 2] & 0xffffu);
    }
}

// Elements [c, c + 8) of a row of d, zeros behind it, in two halves: the load, and
// what is done with it once it is there.  A lane at or behind the row's end loads
// its last eight and shifts: no load stands under a condition of its own.
template <int F>
__device__ __forceinline__ Raw8<F> load_row8(const char* row, int c, int d) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    if (d < 8) return load_upto8<F>(row + (c < d ? c : 0) * kEs, d - c);
    return load8_raw<F>(row + (int64_t)(c < d - 8 ? c : d - 8) * kEs);
}
__device__ __forceinline__ void to_place(float (&v)[8], int c, int d) {
    if (d < 8) return;
    if (d & 7) {
        const int s = c - (d - 8);
        if (s > 0) {
#pragma unroll
            for (int b = 4; b > 0; b >>= 1)
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = s & b ? (k + b < 8 ? v[k + b] : 0.0f) : v[k];
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c < d ? v[k] : 0.0f;
}
template <int F>
__device__ __forceinline__ void row8(const Raw8<F>& r, int c, int d, float (&v)[8]) {
    to_floats<F>(r, v);
    to_place(v, c, d);
}

// The same for a format that the launch alone knows.
__device__ __forceinline__ Raw load_row8(const void* row, int dt, int c, int d) {
    Raw o{};
    if (dt == FSDP_F32) {
        o = load_row8<FSDP_F32>((const char*)row, c, d);
    } else {
        const Raw8<FSDP_BF16> h = load_row8<FSDP_BF16>((const char*)row, c, d);   // 16 bits of any kind
#pragma unroll
        for (int k = 0; k < 4; ++k) o.w[k] = h.w[k];
    }
    return o;
}
__device__ __forceinline__ void row8(const Raw& r, int dt, int c, int d, float (&v)[8]) {
    if (dt == FSDP_F32) {
        to_floats<FSDP_F32>(r, v);
    } else {
        Raw8<FSDP_F16> h;
#pragma unroll
        for (int k = 0; k < 4; ++k) h.w[k] = r.w[k];
        if (dt == FSDP_F16) {
            to_floats<FSDP_F16>(h, v);
        } else {
            Raw8<FSDP_BF16> b;
#pragma unroll
            for (int k = 0; k < 4; ++k) b.w[k] = r.w[k];
            to_floats<FSDP_BF16>(b, v);
        }
    }
    to_place(v, c, d);
}

template <int F>
__device__ __forceinline__ void store_row8(char* row, int c, int d, const float (&v)[8]) {
    if (c + 8 <= d) {
        store8_any<F>(row + (int64_t)c * (F == FSDP_F32 ? 4 : 2), v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < d) store1<F>(row, c + k, v[k]);
    }
}
__device__ __forceinline__ void store_row8(void* row, int dt, int c, int d, const float (&v)[8]) {
    if (dt == FSDP_F32) store_row8<FSDP_F32>((char*)row, c, d, v);
    else if (dt == FSDP_F16) store_row8<FSDP_F16>((char*)row, c, d, v);
    else store_row8<FSDP_BF16>((char*)row, c, d, v);
}

// The sum over the T lanes of a row, in all of them, in a fixed order.  `part`: a
// double a wave, not written again before every wave has read it.
template <int T>
__device__ __forceinline__ double row_sum(double x, double* part) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
        __syncthreads();
        x = part[0];
#pragma unroll
        for (int k = 1; k < T / 64; ++k) x += part[k];
    }
    return x;
}

constexpr int rms_block(int T) { return T < 256 ? 256 : T; }   // lanes of a workgroup with T a row

template <int XF, int HF, int T, int U>
__global__ __launch_bounds__(rms_block(T)) void k_rms(RmsForward p) {
    constexpr int kRows = rms_block(T) / T, kXs = XF == FSDP_F32 ? 4 : 2, kHs = HF == FSDP_F32 ? 4 : 2;
    __shared__ double part[2][T / 64];
    const int d = (int)p.d, t = threadIdx.x % T, nb = (d + kFp8Block - 1) / kFp8Block;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T; row < p.m; row += (int64_t)gridDim.x * kRows) {
        const char* x = (const char*)p.x + row * p.ldx * kXs;
        const char* res = p.residual ? (const char*)p.residual + row * p.ldr * kHs : nullptr;
        Raw8<XF> xr[U];
        Raw8<HF> rr[U];
        Raw wr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) xr[u] = load_row8<XF>(x, (u * T + t) * 8, d);
        if (res) {
#pragma unroll
            for (int u = 0; u < U; ++u) rr[u] = load_row8<HF>(res, (u * T + t) * 8, d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) wr[u] = load_row8(p.weight, p.wdt, (u * T + t) * 8, d);
        float v[U][8];
        double q = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * 8;
            row8<XF>(xr[u], c, d, v[u]);
            if (res) {
                float r[8];
                row8<HF>(rr[u], c, d, r);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[u][k] = round_to<HF>(v[u][k] + r[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) q = __builtin_fma((double)v[u][k], (double)v[u][k], q);
        }
        q = row_sum<T>(q, part[turn]);
        turn ^= 1;
        const float r = (float)(1.0 / __builtin_sqrt(q / (double)d + p.eps));
        if (t == 0 && p.rstd) p.rstd[row] = r;
        // stored only now: h may be the residual, of which every lane has its part by now
        if (res) {
#pragma unroll
            for (int u = 0; u < U; ++u) store_row8<HF>((char*)p.h + row * p.ldh * kHs, (u * T + t) * 8, d, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * 8;
            float w[8];
            row8(wr[u], p.wdt, c, d, w);
            Raw y;
            uint32_t a = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[u][k] = v[u][k] * r * w[k];
                if (c + k >= d) v[u][k] = 0.0f;              // not 0 * infinity
                y.w[k] = __float_as_uint(v[u][k]);
                a = max(a, y.w[k] & 0x7fffffffu);
            }
            if (p.y) store_row8((char*)p.y + row * p.ldy * (p.ydt == FSDP_F32 ? 4 : 2), p.ydt, c, d, v[u]);
            const uint32_t s = fp8_scale_byte(max_of_16(a));
            if (c < nb * kFp8Block) {
                *reinterpret_cast<u32x2*>(p.codes + row * nb * kFp8Block + c) = fp8_codes8<FSDP_F32>(y, s);
                if (t % 16 == 0) p.scales[row * nb + c / kFp8Block] = (uint8_t)s;
            }
        }
    }
}

// P lanes' worth of rows go to each partial sum of dw: part b takes rows b, b + P, ...
template <int DF, int HF, int T, int U>
__global__ __launch_bounds__(rms_block(T)) void k_rms_grads(RmsBackward p) {
    constexpr int kRows = rms_block(T) / T, kDs = DF == FSDP_F32 ? 4 : 2, kHs = HF == FSDP_F32 ? 4 : 2;
    __shared__ double part[2][T / 64];
    const int d = (int)p.d, t = threadIdx.x % T;
    const int64_t b = (int64_t)blockIdx.x * kRows + threadIdx.x / T, parts = (int64_t)gridDim.x * kRows;
    float acc[U][8] = {};
    int turn = 0;
    for (int64_t row = b; row < p.m; row += parts) {
        const char *dy = (const char*)p.dy + row * p.ldy * kDs, *h = (const char*)p.h + row * p.ldh * kHs;
        const char* dh = p.dh && p.dx ? (const char*)p.dh + row * p.lddh * kHs : nullptr;
        const float r = p.rstd[row];
        Raw8<DF> yr[U];
        Raw8<HF> hr[U], er[U];
#pragma unroll
        for (int u = 0; u < U; ++u) yr[u] = load_row8<DF>(dy, (u * T + t) * 8, d);
#pragma unroll
        for (int u = 0; u < U; ++u) hr[u] = load_row8<HF>(h, (u * T + t) * 8, d);
        if (dh) {
#pragma unroll
            for (int u = 0; u < U; ++u) er[u] = load_row8<HF>(dh, (u * T + t) * 8, d);
        }
        double q = 0.0;
        float g[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * 8;
            float y[8], v[8], w[8];
            row8(load_row8(p.weight, p.wdt, c, d), p.wdt, c, d, w);
            row8<DF>(yr[u], c, d, y);
            row8<HF>(hr[u], c, d, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[u][k] = y[k] * w[k];
                q = __builtin_fma((double)g[u][k], (double)v[k], q);
                acc[u][k] += y[k] * (v[k] * r);
            }
        }
        if (!p.dx) continue;
        q = row_sum<T>(q, part[turn]);
        turn ^= 1;
        const float f = (float)(q / (double)d * (double)r * (double)r);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * 8;
            float v[8], e[8];
            row8<HF>(hr[u], c, d, v);
            if (dh) row8<HF>(er[u], c, d, e);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = r * (g[u][k] - v[k] * f);
                if (dh) v[k] += e[k];
            }
            store_row8<HF>((char*)p.dx + row * p.lddx * kHs, c, d, v);
        }
    }
    if (!p.dw) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * T + t) * 8;
        if (p.parts) store_row8<FSDP_F32>((char*)(p.parts + b * d), c, d, acc[u]);
        else if (b == 0) store_row8(p.dw, p.dwdt, c, d, acc[u]);
    }
}

// dw from its partial sums: a workgroup takes 64 columns, 16 lanes of four columns
// for each sixteenth of the parts, whose sums are added in LDS in their order.
__global__ __launch_bounds__(256) void k_rms_dw(const float* __restrict__ parts, int n, int d, void* __restrict__ dw, int dt) {
    __shared__ float sums[16][64];
    const int g = threadIdx.x / 16, c = threadIdx.x % 16 * 4, c0 = blockIdx.x * 64;
    float s[4] = {};
    for (int i = g; i < n; i += 16)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c0 + c + k < d) s[k] += parts[(int64_t)i * d + c0 + c + k];
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[g][c + k] = s[k];
    __syncthreads();
    if (threadIdx.x >= 64 || c0 + (int)threadIdx.x >= d) return;
    float x = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 16; ++i) x += sums[i][threadIdx.x];
    const int64_t o = c0 + threadIdx.x;
    if (dt == FSDP_F32) store1<FSDP_F32>(dw, o, x);
    else if (dt == FSDP_F16) store1<FSDP_F16>(dw, o, x);
    else store1<FSDP_BF16>(dw, o, x);
}

// ----------------------------------------------------------------- launchers
// Lanes a row (T) and eights of elements a lane (U): the fewest that hold it.
template <template <int, int> class K, typename P>
static hipError_t by_size(const P& p, hipStream_t st) {
    if (p.d <= 512) return K<64, 1>::run(p, st);
    if (p.d <= 1024) return K<64, 2>::run(p, st);
    if (p.d <= 2048) return K<256, 1>::run(p, st);
    if (p.d <= 4096) return K<256, 2>::run(p, st);
    if (p.d <= 6144) return K<256, 3>::run(p, st);
    if (p.d <= 8192) return K<256, 4>::run(p, st);
    if (p.d <= 16384) return K<512, 4>::run(p, st);
    return K<1024, 4>::run(p, st);
}
static int row_lanes(int64_t d) { return d <= 1024 ? 64 : (d <= 8192 ? 256 : (d <= 16384 ? 512 : 1024)); }

// A launch holds fewer than 2^32 work items; beyond that workgroups loop.
constexpr int64_t kMaxRowGrid = 1 << 21;

template <int XF, int HF>
struct Forward {
    template <int T, int U>
    struct K {
        static hipError_t run(const RmsForward& p, hipStream_t st) {
            constexpr int kRows = rms_block(T) / T;
            const int64_t want = (p.m + kRows - 1) / kRows;
            launch(k_rms<XF, HF, T, U>, dim3((unsigned)(want < kMaxRowGrid ? want : kMaxRowGrid)), dim3(rms_block(T)), st, p);
            return hipGetLastError();
        }
    };
};

int64_t rms_parts(int64_t m, int64_t d) {
    const int64_t rows = rms_block(row_lanes(d)) / row_lanes(d);
    return m <= 1 ? m : ((m < kRmsParts ? m : kRmsParts) + rows - 1) / rows * rows;
}

template <int DF, int HF>
struct Backward {
    template <int T, int U>
    struct K {
        static hipError_t run(const RmsBackward& p, hipStream_t st) {
            constexpr int kRows = rms_block(T) / T;
            const int64_t parts = rms_parts(p.m, p.d);
            launch(k_rms_grads<DF, HF, T, U>, dim3((unsigned)((parts + kRows - 1) / kRows)), dim3(rms_block(T)), st, p);
            return hipGetLastError();
        }
    };
};

template <template <int, int> class Op, int A, typename P>
static hipError_t by_format(const P& p, int b, hipStream_t st) {
    if (b == FSDP_F32) return by_size<Op<A, FSDP_F32>::template K>(p, st);
    if (b == FSDP_F16) return by_size<Op<A, FSDP_F16>::template K>(p, st);
    return by_size<Op<A, FSDP_BF16>::template K>(p, st);
}
template <template <int, int> class Op, typename P>
static hipError_t by_formats(const P& p, int a, int b, hipStream_t st) {
    if (a == FSDP_F32) return by_format<Op, FSDP_F32>(p, b, st);
    if (a == FSDP_F16) return by_format<Op, FSDP_F16>(p, b, st);
    return by_format<Op, FSDP_BF16>(p, b, st);
}

hipError_t launch_rms_forward(const RmsForward& p, void* stream) {
    return by_formats<Forward>(p, p.xdt, p.residual ? p.hdt : p.xdt, (hipStream_t)stream);
}

hipError_t launch_rms_backward(const RmsBackward& p, void* stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (p.m > 0) {
        hipError_t e = by_formats<Backward>(p, p.ydt, p.hdt, st);
        if (e != hipSuccess) return e;
    }
    if (p.dw && p.m != 1) {
        launch(k_rms_dw, dim3((unsigned)((p.d + 63) / 64)), dim3(256), st, (const float*)p.parts, (int)rms_parts(p.m, p.d),
               (int)p.d, p.dw, p.dwdt);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace fsdp
