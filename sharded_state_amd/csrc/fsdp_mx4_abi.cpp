// fsdp_mx4_abi.cpp -- host layer of the 4-bit microscaled blocks: argument
// validation and launches for the entry points of include/fsdp_shard.h.  Every
// check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <exception>
#include <vector>

#include "fsdp_internal.h"
#include "fsdp_mx4.h"
#include "fsdp_shard.h"

namespace {

using namespace fsdp;

template <typename F>
int guarded(const char* fn, F&& body) {
    try {
        return body();
    } catch (const std::exception& e) {
        return fail(FSDP_E_SIZE, "%s: %s", fn, e.what());   // the host's tables did not fit
    }
}

// Sizes of a matrix: not negative, and small enough that no byte offset wraps.
int check_matrix(const char* fn, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(FSDP_E_INVAL, "%s: a size is negative", fn);
    // padded to whole blocks a row has fewer than cols + 32 elements
    if (rows > 0 && cols > kMaxElems / rows - kMx4Block) return fail(FSDP_E_SIZE, "%s: the matrix is too large", fn);
    return FSDP_OK;
}

}  // namespace

extern "C" {

int fsdp_mx4_quantize(const void* src, fsdp_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* codes,
                      void* scales, void* codes_t, void* scales_t, void* stream) {
    const char* fn = "fsdp_mx4_quantize";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dt);
        int rc = check_matrix(fn, rows, cols);
        if (!rc) rc = check_matrix(fn, cols, rows);
        if (rc) return rc;
        if (rows > 1 && ld < cols) return fail(FSDP_E_INVAL, "%s: ld is smaller than a row", fn);
        if (rows > 1 && ld > kMaxElems / rows) return fail(FSDP_E_SIZE, "%s: ld is too large", fn);
        if (rows == 0 || cols == 0) return ok();
        if (!codes != !scales || !codes_t != !scales_t)
            return fail(FSDP_E_INVAL, "%s: codes and scales come together", fn);
        if (!codes && !codes_t) return fail(FSDP_E_INVAL, "%s: no output", fn);
        if (!aligned16(codes) || !aligned16(codes_t))
            return fail(FSDP_E_INVAL, "%s: codes must be 16-byte aligned", fn);
        if (!src) return fail(FSDP_E_INVAL, "%s: src is NULL", fn);
        const int64_t nb = mx4_blocks(cols), nbr = mx4_blocks(rows);
        std::vector<Range> outs;
        if (codes) {
            outs.push_back(range(codes, rows * nb, 16));
            outs.push_back(range(scales, rows * nb, 1));
        }
        if (codes_t) {
            outs.push_back(range(codes_t, cols * nbr, 16));
            outs.push_back(range(scales_t, cols * nbr, 1));
        }
        const Range in = range(src, (rows - 1) * (rows > 1 ? ld : 0) + cols, dt_size(dt));
        if (!disjoint(outs, {in})) return fail(FSDP_E_ALIAS, "%s: an output overlaps src or another output", fn);
        const Mx4Quant q{src, (int)dt, rows, cols, rows > 1 ? ld : cols, (uint8_t*)codes, (uint8_t*)scales,
                         (uint8_t*)codes_t, (uint8_t*)scales_t};
        (void)hipGetLastError();
        hipError_t e = launch_mx4_quantize(q, stream);
        if (e != hipSuccess) return hip_fail(e, "quantize launch");
        return ok();
    });
}

int fsdp_mx4_gather(const void* const* codes, const void* const* scales, int32_t world, int64_t shard_numel,
                    fsdp_dtype dt, void* full_out, void* stream) {
    const char* fn = "fsdp_mx4_gather";
    return guarded(fn, [&]() -> int {
        int rc = check_world(world, 0, shard_numel);
        if (!rc) rc = check_matrix(fn, world, shard_numel);
        if (rc) return rc;
        if (!valid_dtype(dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dt);
        if (shard_numel == 0) return ok();
        if (!codes || !scales || !full_out) return fail(FSDP_E_INVAL, "%s: an array or full_out is NULL", fn);
        const int64_t nb = mx4_blocks(shard_numel);
        std::vector<Range> ins;
        Mx4Shards s{};
        for (int q = 0; q < world; ++q) {
            if (!codes[q] || !scales[q]) return fail(FSDP_E_INVAL, "%s: shard %d is NULL", fn, q);
            if (!aligned16(codes[q])) return fail(FSDP_E_INVAL, "%s: codes[%d] must be 16-byte aligned", fn, q);
            ins.push_back(range(codes[q], nb, 16));
            ins.push_back(range(scales[q], nb, 1));
            s.codes[q] = (const uint8_t*)codes[q];
            s.scales[q] = (const uint8_t*)scales[q];
        }
        if (!disjoint({range(full_out, (int64_t)world * shard_numel, dt_size(dt))}, ins))
            return fail(FSDP_E_ALIAS, "%s: full_out overlaps a shard", fn);
        (void)hipGetLastError();
        hipError_t e = launch_mx4_gather(s, world, shard_numel, (int)dt, full_out, stream);
        if (e != hipSuccess) return hip_fail(e, "gather launch");
        return ok();
    });
}

int fsdp_mx4_gather_packed(const void* const* codes, const void* const* scales, int32_t world, int64_t shard_numel,
                           void* full_codes, void* full_scales, void* stream) {
    const char* fn = "fsdp_mx4_gather_packed";
    return guarded(fn, [&]() -> int {
        int rc = check_world(world, 0, shard_numel);
        if (!rc) rc = check_matrix(fn, world, shard_numel);
        if (rc) return rc;
        if (shard_numel % kMx4Block)
            return fail(FSDP_E_SIZE, "%s: shard_numel = %lld is not a multiple of %d: the shards' blocks do not join",
                        fn, (long long)shard_numel, kMx4Block);
        if (shard_numel == 0) return ok();
        if (!codes || !scales || !full_codes || !full_scales)
            return fail(FSDP_E_INVAL, "%s: an array or an output is NULL", fn);
        if (!aligned16(full_codes)) return fail(FSDP_E_INVAL, "%s: full_codes must be 16-byte aligned", fn);
        const int64_t nb = shard_numel / kMx4Block;
        const Range fc = range(full_codes, world * nb, 16), fs = range(full_scales, world * nb, 1);
        std::vector<Range> ins;
        CopyBatch b;
        std::vector<CopyBatch> batches;
        b.count = 0;
        auto add = [&](const void* src, char* dst, int64_t bytes) {
            if (src == dst) return;             // already in place
            ins.push_back(range(src, bytes, 1));
            b.src[b.count] = (const char*)src;
            b.dst[b.count] = dst;
            b.bytes[b.count] = bytes;
            if (++b.count == CopyBatch::kMax) {
                batches.push_back(b);
                b.count = 0;
            }
        };
        for (int q = 0; q < world; ++q) {
            if (!codes[q] || !scales[q]) return fail(FSDP_E_INVAL, "%s: shard %d is NULL", fn, q);
            add(codes[q], (char*)full_codes + q * nb * 16, nb * 16);
            add(scales[q], (char*)full_scales + q * nb, nb);
        }
        if (b.count > 0) batches.push_back(b);
        if (!disjoint({fc, fs}, ins))
            return fail(FSDP_E_ALIAS, "%s: an output overlaps the other one or a shard outside its own slot", fn);
        (void)hipGetLastError();
        for (const CopyBatch& c : batches) {
            hipError_t e = launch_copies(c, cu_count(), stream);
            if (e != hipSuccess) return hip_fail(e, "gather launch");
        }
        return ok();
    });
}

int fsdp_mx4_linear_few(const void* x, fsdp_dtype x_dt, int64_t m, int64_t k, int64_t ldx, const void* w_codes,
                        const void* w_scales, int64_t n, fsdp_dtype out_dt, void* out, int64_t ldo, void* stream) {
    const char* fn = "fsdp_mx4_linear_few";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(x_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)x_dt);
        if (!valid_dtype(out_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)out_dt);
        if (m > FSDP_MX4_FEW) return fail(FSDP_E_SIZE, "%s: m = %lld > %d", fn, (long long)m, FSDP_MX4_FEW);
        int rc = check_matrix(fn, m, k);
        if (!rc) rc = check_matrix(fn, n, k);
        if (!rc) rc = check_matrix(fn, m, n);
        if (rc) return rc;
        if (k > FSDP_MX4_MAX_K) return fail(FSDP_E_SIZE, "%s: k = %lld > %d", fn, (long long)k, FSDP_MX4_MAX_K);
        if (m * mx4_blocks(k) > FSDP_MX4_FEW_BLOCKS)
            return fail(FSDP_E_SIZE, "%s: m = %lld rows of k = %lld are more than %d blocks", fn, (long long)m,
                        (long long)k, FSDP_MX4_FEW_BLOCKS);
        if (m == 0 || n == 0) return ok();
        if (!out) return fail(FSDP_E_INVAL, "%s: out is NULL", fn);
        if (m > 1 && (ldo < n || ldx < k)) return fail(FSDP_E_INVAL, "%s: ldo or ldx is smaller than a row", fn);
        if (m > 1 && (ldo > kMaxElems / m || ldx > kMaxElems / m))
            return fail(FSDP_E_SIZE, "%s: ldo or ldx is too large", fn);
        if (k > 0 && (!x || !w_codes || !w_scales)) return fail(FSDP_E_INVAL, "%s: an operand is NULL", fn);
        if (!aligned16(w_codes)) return fail(FSDP_E_INVAL, "%s: codes must be 16-byte aligned", fn);
        const int64_t nb = mx4_blocks(k), xs = m > 1 ? ldx : k, os = m > 1 ? ldo : n;
        const std::vector<Range> ins = {range(x, (m - 1) * xs + k, dt_size(x_dt)), range(w_codes, n * nb, 16),
                                        range(w_scales, n * nb, 1)};
        if (!disjoint({range(out, (m - 1) * os + n, dt_size(out_dt))}, ins))
            return fail(FSDP_E_ALIAS, "%s: out overlaps an operand", fn);
        const Mx4Few p{x, nullptr, (int)x_dt, m, k, xs, (const uint8_t*)w_codes, (const uint8_t*)w_scales, n, nb, (int)out_dt,
                       out, os, cu_count(), stream};
        (void)hipGetLastError();
        hipError_t e = launch_mx4_few(p);
        if (e != hipSuccess) return hip_fail(e, "product launch");
        return ok();
    });
}

int fsdp_mx4_matmul(const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales, int64_t m,
                    int64_t n, int64_t k, fsdp_dtype out_dt, void* out, int64_t ldo, void* stream) {
    const char* fn = "fsdp_mx4_matmul";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(out_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)out_dt);
        int rc = check_matrix(fn, m, k);
        if (!rc) rc = check_matrix(fn, n, k);
        if (!rc) rc = check_matrix(fn, m, n);
        if (rc) return rc;
        if (k > FSDP_MX4_MAX_K) return fail(FSDP_E_SIZE, "%s: k = %lld > %d", fn, (long long)k, FSDP_MX4_MAX_K);
        if (m == 0 || n == 0) return ok();
        if (!out) return fail(FSDP_E_INVAL, "%s: out is NULL", fn);
        if (m > 1 && ldo < n) return fail(FSDP_E_INVAL, "%s: ldo is smaller than a row", fn);
        if (m > 1 && ldo > kMaxElems / m) return fail(FSDP_E_SIZE, "%s: ldo is too large", fn);
        if (k > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))
            return fail(FSDP_E_INVAL, "%s: an operand is NULL", fn);
        if (!aligned16(a_codes) || !aligned16(b_codes))
            return fail(FSDP_E_INVAL, "%s: codes must be 16-byte aligned", fn);
        const int64_t nb = mx4_blocks(k);
        const std::vector<Range> ins = {range(a_codes, m * nb, 16), range(a_scales, m * nb, 1),
                                        range(b_codes, n * nb, 16), range(b_scales, n * nb, 1)};
        const int64_t step = m > 1 ? ldo : n;
        if (!disjoint({range(out, (m - 1) * step + n, dt_size(out_dt))}, ins))
            return fail(FSDP_E_ALIAS, "%s: out overlaps an operand", fn);
        const Mx4Product p{(const uint8_t*)a_codes, (const uint8_t*)a_scales, (const uint8_t*)b_codes,
                           (const uint8_t*)b_scales, m, n, nb, (int)out_dt, out, step, cu_count(), stream};
        (void)hipGetLastError();
        hipError_t e = launch_mx4_matmul(p);
        if (e != hipSuccess) return hip_fail(e, "product launch");
        return ok();
    });
}

}  // extern "C"
