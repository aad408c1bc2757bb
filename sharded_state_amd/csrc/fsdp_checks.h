// fsdp_checks.h -- argument checks shared by the host layers of the block
// formats and the norms over features (fsdp_mx4_abi.cpp, fsdp_fp8_abi.cpp,
// fsdp_rms_abi.cpp): matrices with strided rows, workspaces, and whether
// buffers meet.  Not installed.
#pragma once

#include <exception>
#include <vector>

#include "fsdp_internal.h"

namespace fsdp {

// Nothing is thrown across the ABI.
template <typename F>
inline int guarded(const char* fn, F&& body) {
    try {
        return body();
    } catch (const std::exception& e) {
        return fail(FSDP_E_SIZE, "%s: %s", fn, e.what());   // the host's tables did not fit
    }
}

// A buffer of a product: `rows` rows of `n` bytes, `pitch` bytes from one to the next.
struct Span {
    uintptr_t lo;
    uint64_t n, pitch, rows;
};
inline Span span(const void* p, uint64_t bytes) { return Span{(uintptr_t)p, bytes, bytes, 1}; }

inline bool meet(const Span& x, const Span& y) {
    if (x.n == 0 || y.n == 0 || x.rows == 0 || y.rows == 0) return false;
    if (x.lo >= y.lo + (y.rows - 1) * y.pitch + y.n || y.lo >= x.lo + (x.rows - 1) * x.pitch + x.n) return false;
    const Span &a = x.rows > 1 ? x : y, &b = x.rows > 1 ? y : x;
    if (a.rows == 1 || (b.rows > 1 && b.pitch != a.pitch)) return true;
    // where b's rows begin within a's pitch: column slices of one buffer lie side by side there
    const uint64_t d = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
    return d < a.n || d + b.n > a.pitch;
}

// No two outputs meet and no output meets an input.
inline bool apart(const std::vector<Span>& outs, const std::vector<Span>& ins) {
    for (size_t i = 0; i < outs.size(); ++i) {
        for (size_t j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return false;
        for (const Span& r : ins)
            if (meet(outs[i], r)) return false;
    }
    return true;
}

// A matrix with strided rows, recorded as a span; `used`: it is read or written.
struct Rows {
    int64_t ld = 0;
};
inline int check_rows(const char* fn, const char* name, const void* p, int dt, int64_t rows, int64_t cols, int64_t ld,
               bool used, Rows& r, std::vector<Span>& spans) {
    if (used && !p) return fail(FSDP_E_INVAL, "%s: %s is NULL", fn, name);
    if (rows > 1 && ld < cols) return fail(FSDP_E_INVAL, "%s: the rows of %s overlap", fn, name);
    if (rows > 1 && ld > kMaxElems / rows) return fail(FSDP_E_SIZE, "%s: %s is too large", fn, name);
    r.ld = rows > 1 ? ld : cols;
    const uint64_t es = dt_size(dt);
    if (rows > 0 && cols > 0)
        spans.push_back(Span{(uintptr_t)p, (uint64_t)cols * es, (uint64_t)r.ld * es, (uint64_t)rows});
    return FSDP_OK;
}

// A workspace of at least `need` bytes, recorded as a span.
inline int check_space(const char* fn, void* ws, int64_t have, int64_t need, std::vector<Span>& spans) {
    if (need == 0) return FSDP_OK;
    if (!ws) return fail(FSDP_E_INVAL, "%s: workspace is NULL", fn);
    if (!aligned16(ws)) return fail(FSDP_E_INVAL, "%s: workspace must be 16-byte aligned", fn);
    if (have < need)
        return fail(FSDP_E_SIZE, "%s: the workspace has %lld bytes, %lld are needed", fn, (long long)have, (long long)need);
    spans.push_back(span(ws, (uint64_t)need));
    return FSDP_OK;
}

}  // namespace fsdp
