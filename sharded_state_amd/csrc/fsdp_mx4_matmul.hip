// fsdp_mx4_matmul.hip -- the product of two matrices of 4-bit microscaled
// blocks on gfx950's scaled matrix instructions.
//
//   C[i][j] = sum over blocks b of 2^(ea(i,b) + eb(j,b)) * sum over the block of qa * qb
//
// Both operands hold their blocks along the summed axis, which is what
// v_mfma_scale_f32_32x32x64_f8f6f4 wants: lane l of a wave brings row l % 32,
// the 32 codes (16 bytes) of block l / 32 and that block's scale byte, and the
// products of 32 x 32 rows over two blocks are added to fp32 sums.
#include "fsdp_device.h"
#include "fsdp_mx4.h"

#pragma clang fp contract(off)

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kFp4 = 4;     // the instruction's code for 4-bit elements

// A lane's part of an operand: 16 bytes of codes and a scale byte; zeros with scale 1 outside the matrix.
__device__ __forceinline__ void load_frag(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t rows,
                                          int64_t kb, int64_t nb, i32x8& f, int& s) {
    f = i32x8{0, 0, 0, 0, 0, 0, 0, 0};
    s = 127;
    if (row < rows && kb < nb) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(codes + (row * nb + kb) * 16);
        f[0] = (int)w.x; f[1] = (int)w.y; f[2] = (int)w.z; f[3] = (int)w.w;
        s = scales[row * nb + kb];
    }
}

template <int F>
__global__ __launch_bounds__(64) void k_mx4_matmul(Mx4Product p) {
    const int64_t tiles_n = (p.n + 31) / 32;
    const int64_t tiles = (p.m + 31) / 32 * tiles_n;
    const int l = threadIdx.x, h = l >> 5;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m0 = t / tiles_n * 32, n0 = t % tiles_n * 32;
        f32x16 acc = {0};
        for (int64_t kb = 0; kb < p.nb; kb += 2) {
            i32x8 a, b;
            int sa, sb;
            load_frag(p.a, p.sa, m0 + (l & 31), p.m, kb + h, p.nb, a, sa);
            load_frag(p.b, p.sb, n0 + (l & 31), p.n, kb + h, p.nb, b, sb);
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, kFp4, kFp4, 0, sa, 0, sb);
        }
        const int64_t j = n0 + (l & 31);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int64_t i = m0 + 8 * (r / 4) + 4 * h + r % 4;
            if (i < p.m && j < p.n) store1<F>(p.out, i * p.ldo + j, acc[r]);
        }
    }
}

hipError_t launch_mx4_matmul(const Mx4Product& p) {
    const int64_t tiles = (p.m + 31) / 32 * ((p.n + 31) / 32);
    const dim3 g((unsigned)(tiles < (1 << 22) ? tiles : (1 << 22)));
    hipStream_t st = (hipStream_t)p.stream;
    if (p.dt == FSDP_F32) launch(k_mx4_matmul<FSDP_F32>, g, dim3(64), st, p);
    else if (p.dt == FSDP_F16) launch(k_mx4_matmul<FSDP_F16>, g, dim3(64), st, p);
    else launch(k_mx4_matmul<FSDP_BF16>, g, dim3(64), st, p);
    return hipGetLastError();
}

}  // namespace fsdp
