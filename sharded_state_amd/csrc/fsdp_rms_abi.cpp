// fsdp_rms_abi.cpp -- host layer of the norm over features and its gradients:
// argument validation and launches for the entry points of include/fsdp_shard.h.
// Every check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <cmath>
#include <vector>

#include "fsdp_checks.h"
#include "fsdp_fp8.h"
#include "fsdp_rms.h"
#include "fsdp_shard.h"

namespace {

using namespace fsdp;

int check_sizes(const char* fn, int64_t m, int64_t d) {
    if (m < 0 || d < 0) return fail(FSDP_E_INVAL, "%s: a size is negative", fn);
    if (d > FSDP_RMS_MAX_D) return fail(FSDP_E_SIZE, "%s: %lld > %d features", fn, (long long)d, FSDP_RMS_MAX_D);
    if (m > kMaxElems / (FSDP_RMS_MAX_D + kFp8Block)) return fail(FSDP_E_SIZE, "%s: too many rows", fn);
    return FSDP_OK;
}

int check_type(const char* fn, int dt) {
    return valid_dtype(dt) ? FSDP_OK : fail(FSDP_E_DTYPE, "%s: dtype %d unsupported", fn, dt);
}

// Whether an output may lie on an input: the very same rows of the same type, each
// element of which is read before it is written.
bool same_rows(const void* a, int adt, int64_t lda, const void* b, int bdt, int64_t ldb) {
    return a == b && lda == ldb && dt_size(adt) == dt_size(bdt);
}

int64_t parts_bytes(int64_t m, int64_t d, bool dw) { return dw && m > 1 ? (rms_parts(m, d) * d * 4 + 15) / 16 * 16 : 0; }

}  // namespace

extern "C" {

int fsdp_rms_norm_fp8(const void* x, fsdp_dtype x_dt, int64_t ldx, const void* residual, fsdp_dtype h_dt, int64_t ldr,
                      int64_t m, int64_t d, const void* weight, fsdp_dtype w_dt, double eps, void* h, int64_t ldh,
                      fsdp_dtype y_dt, void* y, int64_t ldy, void* codes, void* scales, float* rstd, void* stream) {
    const char* fn = "fsdp_rms_norm_fp8";
    return guarded(fn, [&]() -> int {
        int rc = check_type(fn, x_dt);
        if (!rc && residual) rc = check_type(fn, h_dt);
        if (!rc) rc = check_type(fn, w_dt);
        if (!rc && y) rc = check_type(fn, y_dt);
        if (!rc) rc = check_sizes(fn, m, d);
        if (rc) return rc;
        if (!(std::isfinite(eps) && eps >= 0.0)) return fail(FSDP_E_INVAL, "%s: eps must be finite and >= 0", fn);
        if (!residual != !h) return fail(FSDP_E_INVAL, "%s: residual and h come together", fn);
        if ((uintptr_t)rstd & 3) return fail(FSDP_E_INVAL, "%s: rstd is not aligned to its type", fn);
        if (m == 0 || d == 0) return ok();
        std::vector<Span> ins, outs;
        Rows xr, rr, hr, yr;
        rc = check_rows(fn, "x", x, x_dt, m, d, ldx, true, xr, ins);
        if (!rc && residual) rc = check_rows(fn, "residual", residual, h_dt, m, d, ldr, true, rr, ins);
        if (!rc && !weight) rc = fail(FSDP_E_INVAL, "%s: weight is NULL", fn);
        if (!rc && h) rc = check_rows(fn, "h", h, h_dt, m, d, ldh, true, hr, outs);
        if (rc) return rc;
        if (!codes || !scales) return fail(FSDP_E_INVAL, "%s: codes or scales is NULL", fn);
        if (!aligned16(codes)) return fail(FSDP_E_INVAL, "%s: codes must be 16-byte aligned", fn);
        ins.push_back(span(weight, (uint64_t)(d * dt_size(w_dt))));
        if (h) {
            // h may be the residual or x, and then meets nothing else
            std::vector<Span> rest{ins.back()};
            if (!same_rows(h, h_dt, hr.ld, x, x_dt, xr.ld)) rest.push_back(ins[0]);
            if (!same_rows(h, h_dt, hr.ld, residual, h_dt, rr.ld)) rest.push_back(ins[1]);
            if (!apart({outs[0]}, rest)) return fail(FSDP_E_ALIAS, "%s: h overlaps an input that it is not", fn);
        }
        if (y) rc = check_rows(fn, "y", y, y_dt, m, d, ldy, true, yr, outs);
        if (rc) return rc;
        const uint64_t blocks = (uint64_t)m * (uint64_t)fp8_blocks(d);
        outs.push_back(span(codes, blocks * kFp8Block));
        outs.push_back(span(scales, blocks));
        outs.push_back(span(rstd, rstd ? (uint64_t)m * 4 : 0));
        if (!apart(outs, {}) || !apart(std::vector<Span>(outs.begin() + (h ? 1 : 0), outs.end()), ins))
            return fail(FSDP_E_ALIAS, "%s: an output overlaps another buffer", fn);
        const RmsForward p{x, residual, (int)x_dt, residual ? (int)h_dt : (int)x_dt, xr.ld, rr.ld, m, d, weight, (int)w_dt,
                           eps, h, hr.ld, y, (int)y_dt, yr.ld, (uint8_t*)codes, (uint8_t*)scales, rstd};
        (void)hipGetLastError();
        hipError_t e = launch_rms_forward(p, stream);
        if (e != hipSuccess) return hip_fail(e, "norm launch");
        return ok();
    });
}

int64_t fsdp_rms_norm_grads_workspace(int64_t m, int64_t d, int32_t want_dw) {
    if (check_sizes("fsdp_rms_norm_grads_workspace", m, d)) return -1;
    ok();
    return parts_bytes(m, d, want_dw);
}

int fsdp_rms_norm_grads(const void* dy, fsdp_dtype dy_dt, int64_t lddy, const void* h, fsdp_dtype h_dt, int64_t ldh,
                        int64_t m, int64_t d, const void* weight, fsdp_dtype w_dt, const float* rstd, const void* dh,
                        int64_t lddh, void* dx, int64_t lddx, fsdp_dtype dw_dt, void* dw, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    const char* fn = "fsdp_rms_norm_grads";
    return guarded(fn, [&]() -> int {
        int rc = check_type(fn, dy_dt);
        if (!rc) rc = check_type(fn, h_dt);
        if (!rc) rc = check_type(fn, w_dt);
        if (!rc && dw) rc = check_type(fn, dw_dt);
        if (!rc) rc = check_sizes(fn, m, d);
        if (rc) return rc;
        if ((uintptr_t)rstd & 3) return fail(FSDP_E_INVAL, "%s: rstd is not aligned to its type", fn);
        if (d == 0 || (m == 0 && !dw) || (!dx && !dw)) return ok();
        std::vector<Span> ins, outs;
        Rows yr, hr, er, xr;
        const bool some = m > 0;
        rc = check_rows(fn, "dy", dy, dy_dt, m, d, lddy, some, yr, ins);
        if (!rc) rc = check_rows(fn, "h", h, h_dt, m, d, ldh, some, hr, ins);
        if (!rc && some && (!weight || !rstd)) rc = fail(FSDP_E_INVAL, "%s: weight or rstd is NULL", fn);
        if (rc) return rc;
        if (some) {
            ins.push_back(span(weight, (uint64_t)(d * dt_size(w_dt))));
            ins.push_back(span(rstd, (uint64_t)m * 4));
        }
        std::vector<Span> rest(ins.begin() + (some ? 1 : 0), ins.end());    // what dx meets nowhere
        const bool want_dx = dx && some;
        if (dh && want_dx) rc = check_rows(fn, "dh", dh, h_dt, m, d, lddh, true, er, ins);
        if (!rc && want_dx) rc = check_rows(fn, "dx", dx, h_dt, m, d, lddx, true, xr, outs);
        if (rc) return rc;
        if (want_dx) {
            if (!same_rows(dx, h_dt, xr.ld, dy, dy_dt, yr.ld)) rest.push_back(ins[0]);
            if (dh && !same_rows(dx, h_dt, xr.ld, dh, h_dt, er.ld)) rest.push_back(ins.back());
            if (!apart(outs, rest)) return fail(FSDP_E_ALIAS, "%s: dx overlaps an input that it is not", fn);
        }
        if (dw) outs.push_back(span(dw, (uint64_t)(d * dt_size(dw_dt))));
        rc = check_space(fn, workspace, workspace_bytes, parts_bytes(m, d, dw), outs);
        if (rc) return rc;
        if (!apart(outs, {}) || !apart(std::vector<Span>(outs.begin() + (want_dx ? 1 : 0), outs.end()), ins))
            return fail(FSDP_E_ALIAS, "%s: an output or the workspace overlaps another buffer", fn);
        const RmsBackward p{dy, h, (int)dy_dt, (int)h_dt, yr.ld, hr.ld, m, d, weight, (int)w_dt, rstd, want_dx ? dh : nullptr,
                            er.ld, want_dx ? dx : nullptr, xr.ld, dw, (int)dw_dt,
                            parts_bytes(m, d, dw) > 0 ? (float*)workspace : nullptr};
        (void)hipGetLastError();
        hipError_t e = launch_rms_backward(p, stream);
        if (e != hipSuccess) return hip_fail(e, "norm launch");
        return ok();
    });
}

}  // extern "C"
