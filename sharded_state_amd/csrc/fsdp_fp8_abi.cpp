// fsdp_fp8_abi.cpp -- host layer of the 8-bit blocks: argument validation and
// launches for the entry points of include/fsdp_shard.h.  Every check runs before
// anything is enqueued.

#include <hip/hip_runtime.h>

#include <vector>

#include "fsdp_checks.h"
#include "fsdp_fp8.h"
#include "fsdp_shard.h"

namespace {

using namespace fsdp;

// Sizes of a matrix: not negative, and small enough that no byte offset wraps.
int check_matrix(const char* fn, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(FSDP_E_INVAL, "%s: a size is negative", fn);
    // padded to whole blocks a row has fewer than cols + 128 elements
    if (rows > kMaxElems || cols > kMaxElems || (rows > 0 && cols > kMaxElems / rows - kFp8Block))
        return fail(FSDP_E_SIZE, "%s: the matrix is too large", fn);
    return FSDP_OK;
}

// A matrix that is quantised in tiles.
int check_tiles(const char* fn, int64_t rows, int64_t cols) {
    if (rows > 0 && cols > 0 && fp8_blocks(rows) > kFp8MaxTiles / fp8_blocks(cols))
        return fail(FSDP_E_SIZE, "%s: %lld x %lld: too many tiles", fn, (long long)rows, (long long)cols);
    return FSDP_OK;
}

// The sizes of a product.
int check_product(const char* fn, int64_t m, int64_t n, int64_t k) {
    int rc = check_matrix(fn, m, k);
    if (!rc) rc = check_matrix(fn, n, k);
    if (!rc) rc = check_matrix(fn, m, n);
    if (!rc && k > FSDP_FP8_MAX_K)
        return fail(FSDP_E_SIZE, "%s: a sum of %lld > %d terms", fn, (long long)k, FSDP_FP8_MAX_K);
    return rc;
}

// Rows of a matrix's table of scales.
int64_t scale_rows(int64_t rows, bool tile) { return tile ? fp8_blocks(rows) : rows; }
int shift(int32_t tile) { return tile ? 7 : 0; }

// A matrix in blocks, recorded as spans.
int check_blocked(const char* fn, const char* name, const void* codes, const void* scales, bool tile, int64_t rows,
                  int64_t cols, std::vector<Span>& spans) {
    if (rows > 0 && cols > 0 && (!codes || !scales)) return fail(FSDP_E_INVAL, "%s: %s is NULL", fn, name);
    if (!aligned16(codes)) return fail(FSDP_E_INVAL, "%s: codes of %s must be 16-byte aligned", fn, name);
    const uint64_t nb = (uint64_t)fp8_blocks(cols);
    spans.push_back(span(codes, (uint64_t)rows * nb * kFp8Block));
    spans.push_back(span(scales, (uint64_t)scale_rows(rows, tile) * nb));
    return FSDP_OK;
}

// Bytes of a matrix in blocks in a workspace, codes then scales, so that the next one is aligned.
int64_t blocked_bytes(int64_t rows, int64_t cols) {
    return (rows * fp8_blocks(cols) * (kFp8Block + 1) + 15) / 16 * 16;
}

// Whether a linear product quantises x on the way (fsdp_fp8_few.hip).  Every workgroup
// then does; a launch of its own costs 2 us (us, on the way and apart: one token, 28672 x
// 8192 43.4 and 47, 8192 x 8192 17.1 and 19.7, 5120 x 1280 4.4 and 6.0; 4 tokens, 28672 x
// 8192 53.5 and 57.8; 16 tokens, 2048 x 512 (64 blocks) 4.2 and 5.1, but 1000 x 1000 (128)
// 5.7 and 5.3, 5120 x 1280 (160) 7.0 and 6.6).
bool linear_few(int64_t m, int64_t k) {
    const int64_t blocks = m * fp8_blocks(k);
    return (m <= 4 && blocks <= 256) || (m <= kFp8Few && blocks <= 64);
}

}  // namespace

extern "C" {

int fsdp_fp8_quantize(const void* src, fsdp_dtype dt, int64_t rows, int64_t cols, int64_t ld, int32_t tile,
                      void* codes, void* scales, void* codes_t, void* scales_t, void* stream) {
    const char* fn = "fsdp_fp8_quantize";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dt);
        int rc = check_matrix(fn, rows, cols);
        if (!rc) rc = check_matrix(fn, cols, rows);
        if (rc) return rc;
        if (!codes != !scales || !codes_t != !scales_t)
            return fail(FSDP_E_INVAL, "%s: codes and scales come together", fn);
        if (!aligned16(codes) || !aligned16(codes_t))
            return fail(FSDP_E_INVAL, "%s: codes must be 16-byte aligned", fn);
        std::vector<Span> ins, outs;
        Rows r;
        const bool some = rows > 0 && cols > 0;
        rc = check_rows(fn, "src", src, dt, rows, cols, ld, some, r, ins);
        if (rc) return rc;
        if (!some) return ok();
        if (!codes && !codes_t) return fail(FSDP_E_INVAL, "%s: no output", fn);
        if (codes_t || tile) rc = check_tiles(fn, rows, cols);
        if (!rc && codes) rc = check_blocked(fn, "out", codes, scales, tile, rows, cols, outs);
        if (!rc && codes_t) rc = check_blocked(fn, "out_t", codes_t, scales_t, tile, cols, rows, outs);
        if (rc) return rc;
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output overlaps src or another output", fn);
        const Fp8Quant q{src, (int)dt, rows, cols, r.ld, tile != 0, (uint8_t*)codes, (uint8_t*)scales,
                         (uint8_t*)codes_t, (uint8_t*)scales_t};
        (void)hipGetLastError();
        hipError_t e = launch_fp8_quantize(q, nullptr, stream);
        if (e != hipSuccess) return hip_fail(e, "quantize launch");
        return ok();
    });
}

int fsdp_fp8_gather(const void* const* codes, const void* const* scales, int32_t world, int64_t shard_numel,
                    fsdp_dtype dt, void* full_out, void* stream) {
    const char* fn = "fsdp_fp8_gather";
    return guarded(fn, [&]() -> int {
        int rc = check_world(world, 0, shard_numel);
        if (!rc) rc = check_matrix(fn, world, shard_numel);
        if (rc) return rc;
        if (!valid_dtype(dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dt);
        if (shard_numel == 0) return ok();
        if (!codes || !scales || !full_out) return fail(FSDP_E_INVAL, "%s: an array or full_out is NULL", fn);
        std::vector<Span> ins;
        Fp8Shards s{};
        for (int q = 0; q < world; ++q) {
            rc = check_blocked(fn, "a shard", codes[q], scales[q], false, 1, shard_numel, ins);
            if (rc) return rc;
            s.codes[q] = (const uint8_t*)codes[q];
            s.scales[q] = (const uint8_t*)scales[q];
        }
        if (!apart({span(full_out, (uint64_t)world * (uint64_t)shard_numel * (uint64_t)dt_size(dt))}, ins))
            return fail(FSDP_E_ALIAS, "%s: full_out overlaps a shard", fn);
        (void)hipGetLastError();
        hipError_t e = launch_fp8_gather(s, world, shard_numel, (int)dt, full_out, stream);
        if (e != hipSuccess) return hip_fail(e, "gather launch");
        return ok();
    });
}

int fsdp_fp8_gather_packed(const void* const* codes, const void* const* scales, int32_t world, int64_t shard_numel,
                           void* full_codes, void* full_scales, void* stream) {
    const char* fn = "fsdp_fp8_gather_packed";
    return guarded(fn, [&]() -> int {
        int rc = check_world(world, 0, shard_numel);
        if (!rc) rc = check_matrix(fn, world, shard_numel);
        if (rc) return rc;
        if (shard_numel % kFp8Block)
            return fail(FSDP_E_SIZE, "%s: shard_numel = %lld is not a multiple of %d: the shards' blocks do not join",
                        fn, (long long)shard_numel, kFp8Block);
        if (shard_numel == 0) return ok();
        if (!codes || !scales) return fail(FSDP_E_INVAL, "%s: an array is NULL", fn);
        std::vector<Span> outs, ins;
        rc = check_blocked(fn, "full", full_codes, full_scales, false, 1, (int64_t)world * shard_numel, outs);
        if (rc) return rc;
        const int64_t nb = shard_numel / kFp8Block;
        CopyBatch b;
        std::vector<CopyBatch> batches;
        b.count = 0;
        auto add = [&](const void* src, char* dst, int64_t bytes) {
            if (src == dst) return;             // already in place
            ins.push_back(span(src, (uint64_t)bytes));
            b.src[b.count] = (const char*)src;
            b.dst[b.count] = dst;
            b.bytes[b.count] = bytes;
            if (++b.count == CopyBatch::kMax) {
                batches.push_back(b);
                b.count = 0;
            }
        };
        for (int q = 0; q < world; ++q) {
            std::vector<Span> one;
            rc = check_blocked(fn, "a shard", codes[q], scales[q], false, 1, shard_numel, one);
            if (rc) return rc;
            add(codes[q], (char*)full_codes + q * shard_numel, shard_numel);
            add(scales[q], (char*)full_scales + q * nb, nb);
        }
        if (b.count > 0) batches.push_back(b);
        if (!apart(outs, ins))
            return fail(FSDP_E_ALIAS, "%s: an output overlaps the other one or a shard outside its own slot", fn);
        (void)hipGetLastError();
        for (const CopyBatch& c : batches) {
            hipError_t e = launch_copies(c, cu_count(), stream);
            if (e != hipSuccess) return hip_fail(e, "gather launch");
        }
        return ok();
    });
}

int64_t fsdp_fp8_matmul_workspace(int64_t m, int64_t n, int64_t k) {
    if (check_product("fsdp_fp8_matmul_workspace", m, n, k)) return -1;
    ok();
    return fp8_parts_bytes(m, n, fp8_blocks(k), cu_count());
}

int fsdp_fp8_matmul(const void* a_codes, const void* a_scales, int32_t a_tile, const void* b_codes,
                    const void* b_scales, int32_t b_tile, int64_t m, int64_t n, int64_t k, fsdp_dtype out_dt, void* out,
                    int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fsdp_fp8_matmul";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(out_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)out_dt);
        int rc = check_product(fn, m, n, k);
        if (rc) return rc;
        if (m == 0 || n == 0) return ok();
        std::vector<Span> ins, outs;
        Rows r;
        rc = check_rows(fn, "out", out, out_dt, m, n, ldo, true, r, outs);
        if (!rc) rc = check_blocked(fn, "a", a_codes, a_scales, a_tile, m, k, ins);
        if (!rc) rc = check_blocked(fn, "b", b_codes, b_scales, b_tile, n, k, ins);
        const int cus = cu_count();
        const int64_t parts = fp8_parts_bytes(m, n, fp8_blocks(k), cus);
        if (!rc) rc = check_space(fn, workspace, workspace_bytes, parts, outs);
        if (rc) return rc;
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: out or the workspace overlaps another buffer", fn);
        const Fp8Product p{(const uint8_t*)a_codes, (const uint8_t*)a_scales, (const uint8_t*)b_codes,
                           (const uint8_t*)b_scales, shift(a_tile), shift(b_tile), m, n, fp8_blocks(k), (int)out_dt,
                           out, r.ld, cus, stream, parts > 0 ? (float*)workspace : nullptr};
        (void)hipGetLastError();
        hipError_t e = launch_fp8_matmul(p);
        if (e != hipSuccess) return hip_fail(e, "product launch");
        return ok();
    });
}

int64_t fsdp_fp8_linear_workspace(int64_t m, int64_t n, int64_t k) {
    if (check_product("fsdp_fp8_linear_workspace", m, n, k)) return -1;
    ok();
    return linear_few(m, k) ? 0 : blocked_bytes(m, k) + fp8_parts_bytes(m, n, fp8_blocks(k), cu_count());
}

int fsdp_fp8_linear(const void* x, fsdp_dtype x_dt, int64_t m, int64_t k, int64_t ldx, const void* w_codes,
                    const void* w_scales, int32_t w_tile, int64_t n, fsdp_dtype out_dt, void* out, int64_t ldo,
                    void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fsdp_fp8_linear";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(x_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)x_dt);
        if (!valid_dtype(out_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)out_dt);
        int rc = check_product(fn, m, n, k);
        if (rc) return rc;
        if (m == 0 || n == 0) return ok();
        std::vector<Span> ins, outs;
        Rows xr, yr;
        rc = check_rows(fn, "x", x, x_dt, m, k, ldx, k > 0, xr, ins);
        if (!rc) rc = check_rows(fn, "out", out, out_dt, m, n, ldo, true, yr, outs);
        if (!rc) rc = check_blocked(fn, "w", w_codes, w_scales, w_tile, n, k, ins);
        const bool few = linear_few(m, k);
        const int cus = cu_count();
        const int64_t blocked = few ? 0 : blocked_bytes(m, k), parts = few ? 0 : fp8_parts_bytes(m, n, fp8_blocks(k), cus);
        if (!rc) rc = check_space(fn, workspace, workspace_bytes, blocked + parts, outs);
        if (rc) return rc;
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output or the workspace overlaps another buffer", fn);
        const int64_t nb = fp8_blocks(k);
        (void)hipGetLastError();
        hipError_t e = hipSuccess;
        if (few) {
            e = launch_fp8_few(Fp8Few{x, nullptr, (int)x_dt, 0, m, k, xr.ld, (const uint8_t*)w_codes, (const uint8_t*)w_scales,
                                      shift(w_tile), n, nb, (int)out_dt, out, yr.ld, cus, stream});
        } else {
            uint8_t *c = (uint8_t*)workspace, *s = c + m * nb * kFp8Block;
            if (nb > 0) e = launch_fp8_quantize(Fp8Quant{x, (int)x_dt, m, k, xr.ld, 0, c, s, nullptr, nullptr}, nullptr, stream);
            if (e == hipSuccess)
                e = launch_fp8_matmul(Fp8Product{c, s, (const uint8_t*)w_codes, (const uint8_t*)w_scales, 0, shift(w_tile), m,
                                                 n, nb, (int)out_dt, out, yr.ld, cus, stream,
                                                 parts > 0 ? (float*)(c + blocked) : nullptr});
        }
        if (e != hipSuccess) return hip_fail(e, "linear launch");
        return ok();
    });
}

// Sizes of a product's gradients.
static int check_grads(const char* fn, int64_t m, int64_t n, int64_t k, bool dx, bool dw) {
    int rc = check_matrix(fn, m, n);
    if (!rc) rc = check_matrix(fn, n, m);
    if (!rc) rc = check_matrix(fn, m, k);
    if (!rc) rc = check_matrix(fn, k, m);
    if (!rc) rc = check_matrix(fn, k, n);
    if (!rc) rc = check_matrix(fn, n, k);
    if (!rc && dx) rc = check_product(fn, m, k, n);
    if (!rc && dw) rc = check_product(fn, n, k, m);
    if (!rc && dw) rc = check_tiles(fn, m, n);
    if (!rc && dw) rc = check_tiles(fn, m, k);
    return rc;
}

// What the workspace holds: dy's blocks, dy's and x's along the tokens, partial sums of each product.
struct GradSpace {
    int64_t dy, dy_t, x_t, dx_parts, dw_parts, bytes;
};
static GradSpace grad_space(int64_t m, int64_t n, int64_t k, bool dx, bool dw) {
    const int cus = cu_count();
    GradSpace g{};
    if (dx) {
        g.dy = blocked_bytes(m, n);
        g.dx_parts = fp8_parts_bytes(m, k, fp8_blocks(n), cus);
    }
    if (dw) {
        g.dy_t = blocked_bytes(n, m);
        g.x_t = blocked_bytes(k, m);
        g.dw_parts = fp8_parts_bytes(n, k, fp8_blocks(m), cus);
    }
    g.bytes = g.dy + g.dy_t + g.x_t + g.dx_parts + g.dw_parts;
    return g;
}

int64_t fsdp_fp8_linear_grads_workspace(int64_t m, int64_t n, int64_t k, int32_t want_dx, int32_t want_dw) {
    if (check_grads("fsdp_fp8_linear_grads_workspace", m, n, k, want_dx, want_dw)) return -1;
    ok();
    return grad_space(m, n, k, want_dx, want_dw).bytes;
}

int fsdp_fp8_linear_grads(const void* dy, fsdp_dtype dy_dt, int64_t lddy, const void* x, fsdp_dtype x_dt, int64_t ldx,
                          int64_t m, int64_t n, int64_t k, const void* wt_codes, const void* wt_scales, int32_t wt_tile,
                          fsdp_dtype dx_dt, void* dx, int64_t lddx, fsdp_dtype dw_dt, void* dw, int64_t lddw,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fsdp_fp8_linear_grads";
    return guarded(fn, [&]() -> int {
        if (!valid_dtype(dy_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dy_dt);
        if (dw && !valid_dtype(x_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)x_dt);
        if (dx && !valid_dtype(dx_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dx_dt);
        if (dw && !valid_dtype(dw_dt)) return fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, (int)dw_dt);
        int rc = check_grads(fn, m, n, k, dx, dw);
        if (rc) return rc;
        const bool want_dx = dx && m > 0 && k > 0, want_dw = dw && n > 0 && k > 0;
        if (!want_dx && !want_dw) return ok();
        std::vector<Span> ins, outs;
        Rows dyr, xr, dxr, dwr;
        rc = check_rows(fn, "dy", dy, dy_dt, m, n, lddy, m > 0 && n > 0, dyr, ins);
        if (!rc && want_dw) rc = check_rows(fn, "x", x, x_dt, m, k, ldx, m > 0, xr, ins);
        if (!rc && want_dx) rc = check_rows(fn, "dx", dx, dx_dt, m, k, lddx, true, dxr, outs);
        if (!rc && want_dw) rc = check_rows(fn, "dw", dw, dw_dt, n, k, lddw, true, dwr, outs);
        if (!rc && want_dx) rc = check_blocked(fn, "wt", wt_codes, wt_scales, wt_tile, k, n, ins);
        const GradSpace g = grad_space(m, n, k, want_dx, want_dw);
        if (!rc) rc = check_space(fn, workspace, workspace_bytes, g.bytes, outs);
        if (rc) return rc;
        if (!apart(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output or the workspace overlaps another buffer", fn);
        const int64_t nbn = fp8_blocks(n), nbm = fp8_blocks(m);
        uint8_t* at = (uint8_t*)workspace;
        auto take = [&](int64_t bytes) {
            uint8_t* p = bytes > 0 ? at : nullptr;
            at += bytes;
            return p;
        };
        uint8_t *q = take(g.dy), *qt = take(g.dy_t), *xt = take(g.x_t);
        float *dxp = (float*)take(g.dx_parts), *dwp = (float*)take(g.dw_parts);
        uint8_t *sq = q ? q + m * nbn * kFp8Block : nullptr, *st = qt ? qt + n * nbm * kFp8Block : nullptr,
                *sx = xt ? xt + k * nbm * kFp8Block : nullptr;
        const int cus = cu_count();
        hipError_t e = hipSuccess;
        (void)hipGetLastError();
        const Fp8Quant of_dy{dy, (int)dy_dt, m, n, dyr.ld, 0, q, sq, qt, st};
        const Fp8Quant of_x{x, (int)x_dt, m, k, xr.ld, 0, nullptr, nullptr, xt, sx};
        const bool once = want_dw && m > 0 && n > 0 && dy_dt == x_dt;    // both operands in one launch
        if (m > 0 && n > 0) e = launch_fp8_quantize(of_dy, once ? &of_x : nullptr, stream);
        if (e == hipSuccess && want_dw && m > 0 && !once) e = launch_fp8_quantize(of_x, nullptr, stream);
        const Fp8Product of_dx{q, sq, (const uint8_t*)wt_codes, (const uint8_t*)wt_scales, 0, shift(wt_tile), m, k, nbn,
                               (int)dx_dt, dx, dxr.ld, cus, stream, dxp};
        const Fp8Product of_dw{qt, st, xt, sx, 0, 0, n, k, nbm, (int)dw_dt, dw, dwr.ld, cus, stream, dwp};
        if (e == hipSuccess && want_dx && want_dw) e = launch_fp8_two(of_dx, of_dw);
        else if (e == hipSuccess) e = launch_fp8_matmul(want_dx ? of_dx : of_dw);
        if (e != hipSuccess) return hip_fail(e, "linear launch");
        return ok();
    });
}

}  // extern "C"
