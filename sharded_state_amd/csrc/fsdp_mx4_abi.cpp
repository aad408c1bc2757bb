// fsdp_mx4_abi.cpp -- host layer of the 4-bit microscaled blocks: argument
// validation and launches for the entry points of include/fsdp_shard.h.  Every
// check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <vector>

#include "fsdp_checks.h"
#include "fsdp_mx4.h"
#include "fsdp_shard.h"

namespace {

using namespace fsdp;

// Sizes of a matrix: not negative, and small enough that no byte offset wraps.
int check_matrix(const char* fn, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(FSDP_E_INVAL, "%s: a size is negative", fn);
    // padded to whole blocks a row has fewer than cols + 32 elements
    if (rows > kMaxElems || cols > kMaxElems || (rows > 0 && cols > kMaxElems / rows - kMx4Block)) return fail(FSDP_E_SIZE, "%s: the matrix is too large", fn);
    return FSDP_OK;
}

// A matrix to be quantised along its columns.
int check_columns(const char* fn, int64_t rows, int64_t cols) {
    if (rows > 0 && cols > 0 && mx4_col_tiles(rows, cols) > kMx4MaxColTiles)
        return fail(FSDP_E_SIZE, "%s: blocks along the columns of %lld x %lld: too many tiles", fn, (long long)rows,
                    (long long)cols);
    return FSDP_OK;
}

// Longest summed axis of a product.
int check_sum(const char* fn, int64_t k) {
    if (k > FSDP_MX4_MAX_K) return fail(FSDP_E_SIZE, "%s: a sum of %lld > %d terms", fn, (long long)k, FSDP_MX4_MAX_K);
    return FSDP_OK;
}

// A matrix in blocks, recorded as spans.
int check_blocked(const char* fn, const char* name, const void* codes, const void* scales, int64_t rows, int64_t cols,
                  std::vector<Span>& spans) {
    if (rows > 0 && cols > 0 && (!codes || !scales)) return fail(FSDP_E_INVAL, "%s: %s is NULL", fn, name);
    if (!aligned16(codes)) return fail(FSDP_E_INVAL, "%s: codes of %s must be 16-byte aligned", fn, name);
    const uint64_t blocks = (uint64_t)rows * (uint64_t)mx4_blocks(cols);
    spans.push_back(span(codes, blocks * 16));
    spans.push_back(span(scales, blocks));
    return FSDP_OK;
}

// Bytes of a matrix in blocks in a workspace, codes then scales, so that the next one is aligned.
int64_t blocked_bytes(int64_t rows, int64_t cols) { return (rows * mx4_blocks(cols) * 17 + 15) / 16 * 16; }

// Whether a linear product quantises x on the way (fsdp_mx4_few.hip).  Every
// workgroup then does, which costs m blocks for 16 of W; a launch of its own 2.4
// us.  Up to 3 tokens it pays at the sizes measured (us, on the way and apart, W
// rotated past the caches: one token, 8192 x 28672 25.6 and 27.3, 28672 x 8192 25.2
// and 36.4; 3 tokens, 8192 x 8192 11.8 and 13.4, 28672 x 8192 31.9 and 33.9; but 8
// tokens 45.8 and 32.4), as far as LDS holds the blocks; for more where the blocks
// are few (16 tokens, 1000 x 1000 (512 blocks) 4.0 and 5.1; a tie from 600 on: 5120 x
// 1280 (640) 6.4 and 6.5, 6400 x 1600 (800) 6.9 and 7.0).  The rule does not look at
// n, and with many rows of W and 16 tokens it is the slower side: 28672 x 1024 (512)
// 12.5 and 9.4, 20480 x 1280 (640) 12.1 and 11.2; not so 40000 x 512 (256) 9.6 and 10.9.
bool linear_few(int64_t m, int64_t k) {
    const int64_t blocks = m * mx4_blocks(k);
    return (m <= 3 && blocks <= 2048) || (m <= kMx4Few && blocks <= 640);
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
        if (codes_t) rc = check_columns(fn, rows, cols);
        if (rc) return rc;
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
        hipError_t e = launch_mx4_quantize(q, nullptr, stream);
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

int64_t fsdp_mx4_linear_workspace(int64_t m, int64_t k) {
    if (m < 0 || k < 0 || check_matrix("fsdp_mx4_linear_workspace", m, k)) return -1;
    ok();
    return linear_few(m, k) ? 0 : blocked_bytes(m, k);
}

int fsdp_mx4_linear(const void* x, fsdp_dtype x_dt, int64_t m, int64_t k, int64_t ldx, const void* w_codes,
                    const void* w_scales, int64_t n, fsdp_dtype out_dt, void* out, int64_t ldo, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    const char* fn = "fsdp_mx4_linear";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(x_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)x_dt);
        if (!valid_dtype(out_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)out_dt);
        int rc = check_matrix(fn, m, k);
        if (!rc) rc = check_matrix(fn, n, k);
        if (!rc) rc = check_matrix(fn, m, n);
        if (!rc) rc = check_sum(fn, k);
        if (rc) return rc;
        if (m == 0 || n == 0) return ok();
        std::vector<Span> ins, outs;
        Rows xr, yr;
        rc = check_rows(fn, "x", x, x_dt, m, k, ldx, k > 0, xr, ins);
        if (!rc) rc = check_rows(fn, "out", out, out_dt, m, n, ldo, true, yr, outs);
        if (!rc) rc = check_blocked(fn, "w", w_codes, w_scales, n, k, ins);
        if (rc) return rc;
        const bool few = linear_few(m, k);
        if (!few) {
            rc = check_space(fn, workspace, workspace_bytes, blocked_bytes(m, k), outs);
            if (rc) return rc;
        }
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output or the workspace overlaps another buffer", fn);
        const int64_t nb = mx4_blocks(k);
        (void)hipGetLastError();
        hipError_t e;
        if (few) {
            e = launch_mx4_few(Mx4Few{x, nullptr, (int)x_dt, m, k, xr.ld, (const uint8_t*)w_codes,
                                      (const uint8_t*)w_scales, n, nb, (int)out_dt, out, yr.ld, cu_count(), stream});
        } else {
            uint8_t* c = (uint8_t*)workspace;
            e = hipSuccess;
            if (nb > 0)
                e = launch_mx4_quantize(Mx4Quant{x, (int)x_dt, m, k, xr.ld, c, c + m * nb * 16, nullptr, nullptr}, nullptr, stream);
            if (e == hipSuccess)
                e = launch_mx4_matmul(Mx4Product{c, c + m * nb * 16, (const uint8_t*)w_codes, (const uint8_t*)w_scales, m,
                                                 n, nb, (int)out_dt, out, yr.ld, cu_count(), stream});
        }
        if (e != hipSuccess) return hip_fail(e, "linear launch");
        return ok();
    });
}

int64_t fsdp_mx4_linear_grads_workspace(int64_t m, int64_t n, int64_t k, int32_t want_dx, int32_t want_dw) {
    const char* fn = "fsdp_mx4_linear_grads_workspace";
    if (m < 0 || n < 0 || k < 0 || check_matrix(fn, m, n) || check_matrix(fn, n, m) || check_matrix(fn, k, m)) return -1;
    ok();
    return (want_dx ? blocked_bytes(m, n) : 0) + (want_dw ? blocked_bytes(n, m) + blocked_bytes(k, m) : 0);
}

int fsdp_mx4_linear_grads(const void* dy, fsdp_dtype dy_dt, int64_t lddy, const void* x, fsdp_dtype x_dt, int64_t ldx,
                          int64_t m, int64_t n, int64_t k, const void* wt_codes, const void* wt_scales,
                          fsdp_dtype dx_dt, void* dx, int64_t lddx, fsdp_dtype dw_dt, void* dw, int64_t lddw,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fsdp_mx4_linear_grads";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(dy_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dy_dt);
        if (dw && !valid_dtype(x_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)x_dt);
        if (dx && !valid_dtype(dx_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dx_dt);
        if (dw && !valid_dtype(dw_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dw_dt);
        int rc = check_matrix(fn, m, n);
        if (!rc) rc = check_matrix(fn, n, m);
        if (!rc) rc = check_matrix(fn, m, k);
        if (!rc) rc = check_matrix(fn, k, m);
        if (!rc) rc = check_matrix(fn, k, n);
        if (!rc) rc = check_matrix(fn, n, k);
        if (!rc && dx) rc = check_sum(fn, n);
        if (!rc && dw) rc = check_sum(fn, m);
        if (!rc && dw) rc = check_columns(fn, m, n);
        if (!rc && dw) rc = check_columns(fn, m, k);
        if (rc) return rc;
        const bool want_dx = dx && m > 0 && k > 0, want_dw = dw && n > 0 && k > 0;
        if (!want_dx && !want_dw) return ok();
        std::vector<Span> ins, outs;
        Rows dyr, xr, dxr, dwr;
        rc = check_rows(fn, "dy", dy, dy_dt, m, n, lddy, m > 0 && n > 0, dyr, ins);
        if (!rc && want_dw) rc = check_rows(fn, "x", x, x_dt, m, k, ldx, m > 0, xr, ins);
        if (!rc && want_dx) rc = check_rows(fn, "dx", dx, dx_dt, m, k, lddx, true, dxr, outs);
        if (!rc && want_dw) rc = check_rows(fn, "dw", dw, dw_dt, n, k, lddw, true, dwr, outs);
        if (!rc && want_dx) rc = check_blocked(fn, "wt", wt_codes, wt_scales, k, n, ins);
        if (!rc)
            rc = check_space(fn, workspace, workspace_bytes,
                             (want_dx ? blocked_bytes(m, n) : 0) + (want_dw ? blocked_bytes(n, m) + blocked_bytes(k, m) : 0),
                             outs);
        if (rc) return rc;
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output or the workspace overlaps another buffer", fn);
        const int64_t nbn = mx4_blocks(n), nbm = mx4_blocks(m);
        uint8_t* at = (uint8_t*)workspace;
        uint8_t *q = nullptr, *sq = nullptr, *qt = nullptr, *st = nullptr, *xt = nullptr, *sx = nullptr;
        if (want_dx) {
            q = at;
            sq = q + m * nbn * 16;
            at += blocked_bytes(m, n);
        }
        if (want_dw) {
            qt = at;
            st = qt + n * nbm * 16;
            xt = at + blocked_bytes(n, m);
            sx = xt + k * nbm * 16;
        }
        const int cus = cu_count();
        hipError_t e = hipSuccess;
        (void)hipGetLastError();
        const Mx4Quant of_dy{dy, (int)dy_dt, m, n, dyr.ld, q, sq, qt, st};
        const Mx4Quant of_x{x, (int)x_dt, m, k, xr.ld, nullptr, nullptr, xt, sx};
        // both operands in one launch where they have one format (1000 x 6400 x 1600 51.2 ->
        // 45.3 us, 64 x 1024 x 1024 17.0 -> 13.0, 8192 x 10240 x 8192 822 -> 817)
        const bool once = want_dw && m > 0 && n > 0 && dy_dt == x_dt;
        if (m > 0 && n > 0) e = launch_mx4_quantize(of_dy, once ? &of_x : nullptr, stream);
        if (e == hipSuccess && want_dw && m > 0 && !once) e = launch_mx4_quantize(of_x, nullptr, stream);
        const Mx4Product of_dx{q, sq, (const uint8_t*)wt_codes, (const uint8_t*)wt_scales, m, k, nbn, (int)dx_dt, dx,
                               dxr.ld, cus, stream};
        const Mx4Product of_dw{qt, st, xt, sx, n, k, nbm, (int)dw_dt, dw, dwr.ld, cus, stream};
        if (e == hipSuccess && want_dx && want_dw) e = launch_mx4_two(of_dx, of_dw);
        else if (e == hipSuccess) e = launch_mx4_matmul(want_dx ? of_dx : of_dw);
        if (e != hipSuccess) return hip_fail(e, "linear launch");
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
        rc = check_sum(fn, k);
        if (rc) return rc;
        if (m == 0 || n == 0) return ok();
        std::vector<Span> ins, outs;
        Rows r;
        rc = check_rows(fn, "out", out, out_dt, m, n, ldo, true, r, outs);
        if (!rc) rc = check_blocked(fn, "a", a_codes, a_scales, m, k, ins);
        if (!rc) rc = check_blocked(fn, "b", b_codes, b_scales, n, k, ins);
        if (rc) return rc;
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: out overlaps an operand", fn);
        const Mx4Product p{(const uint8_t*)a_codes, (const uint8_t*)a_scales, (const uint8_t*)b_codes,
                           (const uint8_t*)b_scales, m, n, mx4_blocks(k), (int)out_dt, out, r.ld, cu_count(), stream};
        (void)hipGetLastError();
        hipError_t e = launch_mx4_matmul(p);
        if (e != hipSuccess) return hip_fail(e, "product launch");
        return ok();
    });
}

}  // extern "C"
