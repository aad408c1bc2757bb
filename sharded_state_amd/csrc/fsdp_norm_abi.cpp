// fsdp_norm_abi.cpp -- host layer of the gradient norm and clipping: argument
// validation, tables and launches for the entry points of
// include/fsdp_shard.h.  Every check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <cmath>
#include <exception>
#include <vector>

#include "fsdp_internal.h"
#include "fsdp_norm.h"
#include "fsdp_shard.h"

namespace {

using namespace fsdp;

// Nothing is thrown across the ABI: what the host's tables cannot hold is
// reported as FSDP_E_SIZE.
template <typename F>
int guarded(const char* fn, F&& body) {
    try {
        return body();
    } catch (const std::exception& e) {
        return fail(FSDP_E_SIZE, "%s: %s", fn, e.what());
    }
}

// The outputs of a norm call.
int check_out(const char* fn, double max_norm, double* sumsq, float* norm, float* coef, NormOut& o,
              std::vector<Range>& outs) {
    if (!sumsq && !norm && !coef) return fail(FSDP_E_INVAL, "%s: no output", fn);
    if (((uintptr_t)sumsq & 7) || ((uintptr_t)norm & 3) || ((uintptr_t)coef & 3))
        return fail(FSDP_E_INVAL, "%s: an output is not aligned to its type", fn);
    if (coef && !(std::isfinite(max_norm) && max_norm >= 0.0))
        return fail(FSDP_E_INVAL, "%s: max_norm must be finite and >= 0", fn);
    o = NormOut{sumsq, norm, coef, max_norm};
    if (sumsq) outs.push_back(range(sumsq, 1, 8));
    if (norm) outs.push_back(range(norm, 1, 4));
    if (coef) outs.push_back(range(coef, 1, 4));
    return FSDP_OK;
}

int check_workspace(const char* fn, void* ws, std::vector<Range>& outs) {
    if (!ws) return fail(FSDP_E_INVAL, "%s: workspace is NULL", fn);
    if ((uintptr_t)ws & 7) return fail(FSDP_E_INVAL, "%s: workspace is not 8-byte aligned", fn);
    outs.push_back(range(ws, FSDP_NORM_WORKSPACE_BYTES, 1));
    return FSDP_OK;
}

int64_t total_bytes(const std::vector<Range>& rs) {
    uint64_t n = 0;
    for (const Range& r : rs) n += r.n;
    return (int64_t)n;
}

// Validate a list of tensors and put it into tables, format by format.
int tensor_tables(const char* fn, const void* const* ptrs, const int64_t* numels, const fsdp_dtype* dts, int32_t n,
                  int64_t chunk_bytes, std::vector<TensorTable>& tables, std::vector<int>& formats,
                  std::vector<Range>& ranges) {
    if (n < 0) return fail(FSDP_E_INVAL, "%s: n_tensors = %d < 0", fn, n);
    if (n > 0 && (!ptrs || !numels || !dts)) return fail(FSDP_E_INVAL, "%s: a host array is NULL", fn);
    int64_t total = 0;
    for (int32_t k = 0; k < n; ++k) {
        if (!valid_dtype(dts[k])) return fail(FSDP_E_DTYPE, "%s: tensor %d: dtype %d unsupported", fn, k, (int)dts[k]);
        if (numels[k] < 0) return fail(FSDP_E_INVAL, "%s: numels[%d] < 0", fn, k);
        if (numels[k] > kMaxElems - total) return fail(FSDP_E_SIZE, "%s: the tensors are too large", fn);
        total += numels[k];
        if (numels[k] > 0 && !ptrs[k]) return fail(FSDP_E_INVAL, "%s: tensor %d is NULL", fn, k);
        if (numels[k] > 0) ranges.push_back(range(ptrs[k], numels[k], dt_size(dts[k])));
    }
    for (int dt : {FSDP_F32, FSDP_F16, FSDP_BF16}) {
        bool open = false;
        for (int32_t k = 0; k < n; ++k) {
            if (dts[k] != dt || numels[k] == 0) continue;
            if (!open || tables.back().count == TensorTable::kMax) {
                tables.emplace_back();
                tables.back().count = 0;
                tables.back().chunk_begin[0] = 0;
                formats.push_back(dt);
                open = true;
            }
            TensorTable& t = tables.back();
            t.p[t.count] = const_cast<void*>(ptrs[k]);
            t.n[t.count] = numels[k];
            t.chunk_begin[t.count + 1] =
                t.chunk_begin[t.count] + (numels[k] * dt_size(dt) + chunk_bytes - 1) / chunk_bytes;
            ++t.count;
        }
    }
    return FSDP_OK;
}

}  // namespace

extern "C" {

int fsdp_grad_norm(const void* const* srcs, const int64_t* numels, const fsdp_dtype* dts, int32_t n_tensors,
                   double max_norm, double* sumsq_out, float* norm_out, float* coef_out, void* workspace,
                   void* stream) {
    const char* fn = "fsdp_grad_norm";
    return guarded(fn, [&]() -> int {
        NormOut o;
        std::vector<Range> ins, outs;
        std::vector<TensorTable> tables;
        std::vector<int> formats;
        int rc = check_out(fn, max_norm, sumsq_out, norm_out, coef_out, o, outs);
        if (!rc) rc = check_workspace(fn, workspace, outs);
        if (!rc) rc = tensor_tables(fn, srcs, numels, dts, n_tensors, kSumChunkBytes, tables, formats, ins);
        if (rc) return rc;
        if (!disjoint(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output overlaps an input or another output", fn);
        if (tables.size() > (size_t)kNormSlots)
            return fail(FSDP_E_SIZE, "%s: %d tensors need more launches than the workspace holds sums", fn, n_tensors);
        const int cus = cu_count();
        double* partial = (double*)workspace;
        int used = 0;
        (void)hipGetLastError();
        for (size_t t = 0; t < tables.size(); ++t) {
            int got = 0;
            hipError_t e = launch_sumsq(tables[t], formats[t], total_bytes(ins), partial + used, kNormSlots / (int)tables.size(),
                                        tables.size() == 1 ? &o : nullptr, cus, &got, stream);
            if (e != hipSuccess) return hip_fail(e, "norm launch");
            if (got == 0) return ok();          // that launch wrote the result itself
            used += got;
        }
        hipError_t e = launch_norm_finish(partial, used, o, stream);
        if (e != hipSuccess) return hip_fail(e, "norm launch");
        return ok();
    });
}

int fsdp_grad_norm_units(const fsdp_norm_unit* units, int32_t n_units, int32_t world, int32_t rank,
                         fsdp_dtype grad_dt, int32_t fp32_reduce, double max_norm, double* sumsq_out,
                         float* norm_out, float* coef_out, void* workspace, void* stream) {
    const char* fn = "fsdp_grad_norm_units";
    return guarded(fn, [&]() -> int {
        NormOut o;
        std::vector<Range> ins, outs;
        int rc = check_out(fn, max_norm, sumsq_out, norm_out, coef_out, o, outs);
        if (!rc) rc = check_workspace(fn, workspace, outs);
        if (!rc) rc = check_world(world, rank, 0);
        if (rc) return rc;
        if (n_units < 0) return fail(FSDP_E_INVAL, "%s: n_units = %d < 0", fn, n_units);
        if (n_units > 0 && !units) return fail(FSDP_E_INVAL, "%s: units is NULL", fn);
        if (!valid_dtype(grad_dt)) return fail(FSDP_E_DTYPE, "%s: grad dtype %d unsupported", fn, (int)grad_dt);
        const int out_dt = (fp32_reduce || grad_dt == FSDP_F32) ? FSDP_F32 : grad_dt;
        std::vector<std::vector<const void*>> blocks(n_units);
        std::vector<NormUnitArgs> args;
        args.reserve(n_units);
        for (int32_t k = 0; k < n_units; ++k) {
            const fsdp_norm_unit& u = units[k];
            rc = check_world(world, rank, u.shard_numel);
            if (!rc) rc = grad_blocks(u.rank_grads, world, rank, u.shard_numel, grad_dt, blocks[k], ins);
            if (rc) return rc;
            if (u.shard_numel == 0) continue;
            bool vec = !u.grad_shard || aligned16(u.grad_shard);
            for (int q = 0; q < world; ++q) vec = vec && aligned16(blocks[k][q]);
            if (u.grad_shard) outs.push_back(range(u.grad_shard, u.shard_numel, dt_size(out_dt)));
            args.push_back(NormUnitArgs{blocks[k].data(), u.grad_shard, u.shard_numel, vec});
        }
        if (!disjoint(outs, ins)) return fail(FSDP_E_ALIAS, "%s: an output overlaps an input or another output", fn);
        const int launches = ((int)args.size() + norm_units_max(world) - 1) / norm_units_max(world);
        if (launches > kNormSlots)
            return fail(FSDP_E_SIZE, "%s: %d units need more launches than the workspace holds sums", fn, n_units);
        int used = 0;
        (void)hipGetLastError();
        hipError_t e = launch_norm_units(args.data(), (int)args.size(), world, grad_dt, fp32_reduce != 0,
                                         reduce_scalars(world), (double*)workspace, kNormSlots, cu_count(), &used,
                                         stream);
        if (e == hipSuccess) e = launch_norm_finish((const double*)workspace, used, o, stream);
        if (e != hipSuccess) return hip_fail(e, "norm launch");
        return ok();
    });
}

int fsdp_grad_norm_combine(const double* sumsqs, int32_t n, double max_norm, double* sumsq_out, float* norm_out,
                           float* coef_out, void* stream) {
    const char* fn = "fsdp_grad_norm_combine";
    return guarded(fn, [&]() -> int {
        NormOut o;
        std::vector<Range> outs;
        int rc = check_out(fn, max_norm, sumsq_out, norm_out, coef_out, o, outs);
        if (rc) return rc;
        if (n < 0) return fail(FSDP_E_INVAL, "%s: n = %d < 0", fn, n);
        if (n > 0 && !sumsqs) return fail(FSDP_E_INVAL, "%s: sumsqs is NULL", fn);
        if ((uintptr_t)sumsqs & 7) return fail(FSDP_E_INVAL, "%s: sumsqs is not 8-byte aligned", fn);
        if (!disjoint(outs, {range(sumsqs, n, 8)}))
            return fail(FSDP_E_ALIAS, "%s: an output overlaps the sums or another output", fn);
        (void)hipGetLastError();
        hipError_t e = launch_norm_finish(sumsqs, n, o, stream);
        if (e != hipSuccess) return hip_fail(e, "norm launch");
        return ok();
    });
}

int fsdp_clip_grads(void* const* tensors, const int64_t* numels, const fsdp_dtype* dts, int32_t n_tensors,
                    const float* coef, void* stream) {
    const char* fn = "fsdp_clip_grads";
    return guarded(fn, [&]() -> int {
        std::vector<Range> outs;
        std::vector<TensorTable> tables;
        std::vector<int> formats;
        if (!coef) return fail(FSDP_E_INVAL, "%s: coef is NULL", fn);
        if ((uintptr_t)coef & 3) return fail(FSDP_E_INVAL, "%s: coef is not 4-byte aligned", fn);
        int rc = tensor_tables(fn, tensors, numels, dts, n_tensors, kClipChunkBytes, tables, formats, outs);
        if (rc) return rc;
        if (!disjoint(outs, {range(coef, 1, 4)}))
            return fail(FSDP_E_ALIAS, "%s: a tensor overlaps another one or the coefficient", fn);
        (void)hipGetLastError();
        for (size_t t = 0; t < tables.size(); ++t) {
            hipError_t e = launch_clip(tables[t], formats[t], total_bytes(outs), coef, stream);
            if (e != hipSuccess) return hip_fail(e, "clip launch");
        }
        return ok();
    });
}

}  // extern "C"
