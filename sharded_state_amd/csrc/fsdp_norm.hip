// fsdp_norm.hip -- gfx950 kernels of the global gradient norm and of clipping.
//
//   q = sum over tensors and elements of x^2,  norm = sqrt(q),
//   coef = min(1, max_norm / (norm + 1e-6)),   x <- round(x * coef)
//
// Squares and sums are held in 64 bits: a 16-bit or fp32 value is exact in a
// double, its square neither overflows nor vanishes there (fp32 squares do
// beyond 1.8e19 and below 1e-23), and 10^9 terms lose about 1e-13 of the sum.
// The three operations an element that this costs (widen, convert, fma) run at
// a quarter of what the VALU could issue while HBM delivers the elements, so
// the sum stays an HBM stream.
// Workgroup b adds the chunks b, b + grid, ... in that order and writes one
// partial sum; a second launch of one workgroup adds the partial sums in their
// order.  No atomics: the result depends on the sizes and the device alone.
#include "fsdp_any.h"
#include "fsdp_norm.h"

#pragma clang fp contract(off)

namespace fsdp {

__device__ __forceinline__ double sq(float x, double acc) {
    const double d = (double)x;
    return __builtin_fma(d, d, acc);
}

// The squares of the elements of one 16-byte vector of format F.
template <int F>
__device__ __forceinline__ void sq16(u32x4 v, double& a, double& b) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (F == FSDP_F32) {
            if (k & 1) b = sq(to_f32<F>(w[k]), b);
            else a = sq(to_f32<F>(w[k]), a);
        } else {
            a = sq(to_f32<F>(w[k] & 0xffffu), a);
            b = sq(to_f32<F>(w[k] >> 16), b);
        }
    }
}

// The sum of `x` over the workgroup, in a fixed order; thread 0 has it.
template <int THREADS>
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[THREADS / 64];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[w] = x;
    __syncthreads();
    double s = part[0];
#pragma unroll
    for (int k = 1; k < THREADS / 64; ++k) s += part[k];
    return s;
}

__device__ __forceinline__ void write_norm(double q, const NormOut& o) {
    const double n = __builtin_sqrt(q);
    if (o.sumsq) *o.sumsq = q;
    if (o.norm) *o.norm = (float)n;
    if (o.coef) {
        const double c = o.max_norm / (n + 1e-6);
        *o.coef = (float)(c > 1.0 ? 1.0 : c);      // a NaN norm stays NaN
    }
}

// The tensor of a table that owns chunk c.
__device__ __forceinline__ int tensor_of(const TensorTable& T, int64_t c) {
    int lo = 0, hi = T.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (T.chunk_begin[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int F, bool STREAM, bool FINISH>
__global__ __launch_bounds__(kThreads) void k_sumsq(TensorTable T, double* __restrict__ partial, NormOut fin) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int64_t kElems = kSumChunkBytes / kEs;
    constexpr int kU = (int)(kSumChunkBytes / 16 / kThreads);
    const int64_t chunks = T.chunk_begin[T.count];
    double a = 0.0, b = 0.0;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int k = tensor_of(T, c);
        const int64_t start = (c - T.chunk_begin[k]) * kElems;
        const int64_t n = T.n[k] - start;
        const char* p = (const char*)T.p[k] + start * kEs;
        if (n >= kElems) {
            u32x4 v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) v[u] = ld_any<STREAM>(p + ((int64_t)u * kThreads + threadIdx.x) * 16);
#pragma unroll
            for (int u = 0; u < kU; ++u) sq16<F>(v[u], a, b);
        } else {
            const int64_t nv = n * kEs / 16;
            for (int64_t i = threadIdx.x; i < nv; i += kThreads) sq16<F>(*(const u32x4_any*)(p + i * 16), a, b);
            for (int64_t i = nv * (16 / kEs) + threadIdx.x; i < n; i += kThreads) a = sq(load1<F>(p, i), a);
        }
    }
    const double s = block_sum<kThreads>(a + b);
    if (threadIdx.x == 0) {
        if constexpr (FINISH) write_norm(s, fin);
        else partial[blockIdx.x] = s;
    }
}

// 1024 lanes with their loads first: the launch is a chain of latencies.
constexpr int kFinishThreads = 1024;
constexpr int kFinishU = kNormSlots / kFinishThreads;
__global__ __launch_bounds__(kFinishThreads) void k_norm_finish(const double* __restrict__ partial, int n, NormOut o) {
    double s = 0.0;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += kFinishThreads * kFinishU) {
        double v[kFinishU];
#pragma unroll
        for (int u = 0; u < kFinishU; ++u) v[u] = i0 + u * kFinishThreads < n ? partial[i0 + u * kFinishThreads] : 0.0;
#pragma unroll
        for (int u = 0; u < kFinishU; ++u) s += v[u];
    }
    s = block_sum<kFinishThreads>(s);
    if (threadIdx.x == 0) write_norm(s, o);
}

// The sum over the averaged gradient of a table of units: the reduce-scatter's
// fold (fsdp_device.h) with the squares added as its epilogue, and the shard
// stored where the caller wants it.  Vectors in the group layout for an fp32
// shard, 8 consecutive elements for a 16-bit one, as k_reduce_scatter has them;
// a unit with a buffer off the 16-byte grid (a shard of an odd size) goes 8
// consecutive elements at a time through accesses at any address.
template <int NW, int GF, bool FP32R>
__global__ __launch_bounds__(kThreads) void k_norm_units(NormUnits<NW> B, ReduceScalars rs,
                                                         double* __restrict__ partial) {
    constexpr int OF = (FP32R || GF == FSDP_F32) ? FSDP_F32 : GF;
    constexpr bool kGroup = OF == FSDP_F32;
    const int64_t tiles = B.tile_begin[B.count];
    const int world = NW > 0 ? NW : B.world;
    double a = 0.0, b = 0.0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int lo = 0, hi = B.count - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (B.tile_begin[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        const int u = lo;
        const auto gp = [&](int q) -> const void* { return B.g[u * world + q]; };
        const int64_t j = t - B.tile_begin[u];
        const int64_t nvec = B.nvec[u];
        const int64_t tv = (nvec + kThreads - 1) / kThreads;
        void* out = B.out[u];
        if (j < tv) {
            const int64_t vi = j * kThreads + threadIdx.x;
            if (vi < nvec) {
                float x[8];
                if (B.wide[u]) reduce8<NW, GF, FP32R, true, kGroup>(gp, world, vi, x);
                else reduce8_any<NW, GF, FP32R>(gp, world, vi, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = finish<NW, GF, FP32R>(x[k], rs);
                if (out && B.wide[u]) store8x<OF, kGroup>(out, vi, x);
                else if (out) store8_any<OF>((char*)out + vi * (OF == FSDP_F32 ? 32 : 16), x);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    a = sq(x[k], a);
                    b = sq(x[k + 1], b);
                }
            }
        } else {
            const int64_t i = nvec * 8 + (j - tv) * kThreads + threadIdx.x;
            if (i < B.S[u]) {
                const float x = finish<NW, GF, FP32R>(reduce1<NW, GF, FP32R>(gp, world, i), rs);
                if (out) store1<OF>(out, i, x);
                a = sq(x, a);
            }
        }
    }
    const double s = block_sum<kThreads>(a + b);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// round(x * c).  The product is kept apart from the conversion: fused into one
// mixed-precision fma the compiler adds +0 to it, and a product of -0 loses its
// sign.
template <int F>
__device__ __forceinline__ uint32_t scaled(uint32_t bits, float c) {
    float y = to_f32<F>(bits) * c;
    if constexpr (F == FSDP_F16) asm("" : "+v"(y));
    return from_f32<F>(y);
}

// Clipping in place: one 16-byte vector a lane, as the segmented copies.  A
// coefficient of exactly 1 leaves every element as it is, so those launches
// end after one scalar load; a NaN coefficient (a NaN norm) is applied.
// STREAM (see streams()): a wave's stores go out as one span with the streamed
// policy, and the sum's loads carry the non-temporal hint.  Norm and clip of the
// 13B block's 629 MB 347 -> 283 us (norm 108 -> 94, 6.7 TB/s), of 246 MB 145 ->
// 120; of 39 MB, which the memory-side cache keeps from the sum to the clip,
// 26.0 us without and 28 with.
template <int F, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_clip(TensorTable T, const float* __restrict__ coef) {
    constexpr int kEs = F == FSDP_F32 ? 4 : 2;
    constexpr int64_t kElems = kClipChunkBytes / kEs;
    const float c = *coef;
    if (c == 1.0f) return;
    const int64_t chunks = T.chunk_begin[T.count];
    for (int64_t b = blockIdx.x; b < chunks; b += gridDim.x) {
        const int k = tensor_of(T, b);
        const int64_t start = (b - T.chunk_begin[k]) * kElems;
        int64_t n = T.n[k] - start;
        if (n > kElems) n = kElems;
        char* p = (char*)T.p[k] + start * kEs;
        const int64_t nv = n * kEs / 16;
        if (threadIdx.x < nv) {
            const u32x4 v = *(const u32x4_any*)(p + threadIdx.x * 16);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (F == FSDP_F32) w[j] = scaled<F>(w[j], c);
                else w[j] = scaled<F>(w[j] & 0xffffu, c) | (scaled<F>(w[j] >> 16, c) << 16);
            }
            u32x4 r;
            r.x = w[0]; r.y = w[1]; r.z = w[2]; r.w = w[3];
            const int l = threadIdx.x & 63;
            if (STREAM && ((uintptr_t)p & 15) == 0) st16_wave(p + (threadIdx.x - l) * 16, l, r);
            else *(u32x4_any*)(p + threadIdx.x * 16) = r;
        }
        // fewer than one vector's elements are left
        const int64_t i = nv * (16 / kEs) + threadIdx.x;
        if (i < n) {
            if constexpr (F == FSDP_F32) ((uint32_t*)p)[i] = scaled<F>(((uint32_t*)p)[i], c);
            else ((uint16_t*)p)[i] = (uint16_t)scaled<F>(((uint16_t*)p)[i], c);
        }
    }
}

// ----------------------------------------------------------------- launchers
// Whether a call's tensors are more than the memory-side cache (256 MB) could
// hand from one pass to the next.
static bool streams(int64_t bytes) { return bytes > (int64_t(128) << 20); }

// Workgroups of a summing launch, `per` a CU.  A list: 4 (13B block, non-temporal
// loads: 93.7 us, with 8 96.0).  Units: 8 for few ranks, whose lanes have few
// loads each, 4 from four ranks on, 3 where eight ranks' shards are stored too
// (us with 3, 4, 8: N = 1 fp32 92.3, 75.4, 62.2; N = 2 bf16 97.0, 80.1, 64.2; N = 4
// fp16 40.8, 38.0, 39.2; N = 8 bf16 271.6, 264.3 (6.5 TB/s), 278.9, and with its
// shard stored 343.9, 361.6, 380.9).
static int units_per_cu(int world, bool store) { return world < 4 ? 8 : world >= 8 && store ? 3 : 4; }
static int sum_grid(int64_t chunks, int slots, int cus, int per) {
    int64_t g = (int64_t)cus * per;
    if (g > slots) g = slots;
    if (g > chunks) g = chunks;
    return g < 1 ? 1 : (int)g;
}

template <int F>
static void sumsq(const TensorTable& t, double* partial, int g, const NormOut* fin, bool stream, hipStream_t st) {
    const NormOut none{};
    if (fin) launch(k_sumsq<F, false, true>, dim3(1), dim3(kThreads), st, t, partial, *fin);
    else if (stream) launch(k_sumsq<F, true, false>, dim3(g), dim3(kThreads), st, t, partial, none);
    else launch(k_sumsq<F, false, false>, dim3(g), dim3(kThreads), st, t, partial, none);
}

hipError_t launch_sumsq(const TensorTable& t, int dt, int64_t bytes, double* partial, int slots, const NormOut* fin,
                        int cus, int* used, void* stream) {
    const int64_t chunks = t.chunk_begin[t.count];
    *used = 0;
    if (chunks <= 0) return hipSuccess;
    hipStream_t st = (hipStream_t)stream;
    const int g = sum_grid(chunks, slots, cus, 4);
    if (g > 1) fin = nullptr;
    *used = fin ? 0 : g;
    if (dt == FSDP_F32) sumsq<FSDP_F32>(t, partial, g, fin, streams(bytes), st);
    else if (dt == FSDP_F16) sumsq<FSDP_F16>(t, partial, g, fin, streams(bytes), st);
    else sumsq<FSDP_BF16>(t, partial, g, fin, streams(bytes), st);
    return hipGetLastError();
}

template <int NW>
static hipError_t norm_units_all(const NormUnitArgs* units, int n, int world, int grad_dt, int fp32_reduce,
                                 const ReduceScalars& rs, double* partial, int slots, int cus, int* used,
                                 void* stream) {
    const int kMax = norm_units_max(world);
    const int launches = (n + kMax - 1) / kMax;
    const int per = slots / (launches > 0 ? launches : 1);
    const bool f32r = fp32_reduce || grad_dt == FSDP_F32;
    *used = 0;
    for (int done = 0; done < n; done += kMax) {
        NormUnits<NW> B{};
        B.world = world;
        const int c = n - done < kMax ? n - done : kMax;
        int64_t tiles = 0;
        for (int k = 0; k < c; ++k) {
            const NormUnitArgs& a = units[done + k];
            const int64_t nvec = a.S / 8 & ~int64_t(63);  // whole groups; the rest joins the tail
            B.tile_begin[k] = tiles;
            B.nvec[k] = nvec;
            B.S[k] = a.S;
            B.out[k] = a.out;
            B.wide[k] = a.wide;
            for (int q = 0; q < world; ++q) B.g[k * world + q] = a.grads[q];
            tiles += (nvec + kThreads - 1) / kThreads + (a.S - 8 * nvec + kThreads - 1) / kThreads;
        }
        B.count = c;
        B.tile_begin[c] = tiles;
        if (tiles == 0) continue;
        const dim3 g((unsigned)sum_grid(tiles, per, cus, units_per_cu(world, units[done].out != nullptr))), th(kThreads);
        hipStream_t st = (hipStream_t)stream;
        double* out = partial + *used;
        if (grad_dt == FSDP_F32) launch(k_norm_units<NW, FSDP_F32, true>, g, th, st, B, rs, out);
        else if (grad_dt == FSDP_F16 && f32r) launch(k_norm_units<NW, FSDP_F16, true>, g, th, st, B, rs, out);
        else if (grad_dt == FSDP_F16) launch(k_norm_units<NW, FSDP_F16, false>, g, th, st, B, rs, out);
        else if (f32r) launch(k_norm_units<NW, FSDP_BF16, true>, g, th, st, B, rs, out);
        else launch(k_norm_units<NW, FSDP_BF16, false>, g, th, st, B, rs, out);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        *used += (int)g.x;
    }
    return hipSuccess;
}

hipError_t launch_norm_units(const NormUnitArgs* units, int n, int world, int grad_dt, int fp32_reduce,
                             const ReduceScalars& rs, double* partial, int slots, int cus, int* used, void* stream) {
    switch (world) {
    case 1: return norm_units_all<1>(units, n, world, grad_dt, fp32_reduce, rs, partial, slots, cus, used, stream);
    case 2: return norm_units_all<2>(units, n, world, grad_dt, fp32_reduce, rs, partial, slots, cus, used, stream);
    case 4: return norm_units_all<4>(units, n, world, grad_dt, fp32_reduce, rs, partial, slots, cus, used, stream);
    case 8: return norm_units_all<8>(units, n, world, grad_dt, fp32_reduce, rs, partial, slots, cus, used, stream);
    default: return norm_units_all<0>(units, n, world, grad_dt, fp32_reduce, rs, partial, slots, cus, used, stream);
    }
}

hipError_t launch_norm_finish(const double* partial, int n, const NormOut& out, void* stream) {
    launch(k_norm_finish, dim3(1), dim3(kFinishThreads), (hipStream_t)stream, partial, n, out);
    return hipGetLastError();
}

template <int F>
static void clip(const TensorTable& t, const float* coef, dim3 g, bool stream, hipStream_t st) {
    if (stream) launch(k_clip<F, true>, g, dim3(kThreads), st, t, coef);
    else launch(k_clip<F, false>, g, dim3(kThreads), st, t, coef);
}

hipError_t launch_clip(const TensorTable& t, int dt, int64_t bytes, const float* coef, void* stream) {
    const int64_t chunks = t.chunk_begin[t.count];
    if (chunks <= 0) return hipSuccess;
    // a launch holds fewer than 2^32 work items; beyond 2^22 workgroups they loop
    const dim3 g((unsigned)(chunks < (1 << 22) ? chunks : (1 << 22)));
    hipStream_t st = (hipStream_t)stream;
    if (dt == FSDP_F32) clip<FSDP_F32>(t, coef, g, streams(bytes), st);
    else if (dt == FSDP_F16) clip<FSDP_F16>(t, coef, g, streams(bytes), st);
    else clip<FSDP_BF16>(t, coef, g, streams(bytes), st);
    return hipGetLastError();
}

}  // namespace fsdp
