// layer_checks.cpp -- the host layer of the 8-bit blocks, their products and the
// norms over features under the sanitizers: argument validation, workspaces and
// launch planning with device pointers that nothing dereferences.  Without a
// device every launch is refused by the runtime, after it was planned.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#include "fsdp_internal.h"
#include "fsdp_kernels.h"
#include "fsdp_shard.h"

// The unit step's kernels are not part of these checks.
namespace fsdp {
hipError_t launch_units_adamw(const UnitArgs*, int, const UnitLaunch&) { return hipSuccess; }
hipError_t launch_units_sgd(const UnitArgs*, int, const UnitLaunch&) { return hipSuccess; }
hipError_t launch_units_adamax(const UnitArgs*, int, const UnitLaunch&) { return hipSuccess; }
hipError_t launch_units_adadelta(const UnitArgs*, int, const UnitLaunch&) { return hipSuccess; }
}  // namespace fsdp

static int g_checks = 0;
#define CHECK(x)                                                           \
    do {                                                                   \
        ++g_checks;                                                        \
        if (!(x)) {                                                        \
            fprintf(stderr, "%s:%d: %s (%s)\n", __FILE__, __LINE__, #x, fsdp_last_error()); \
            exit(1);                                                       \
        }                                                                  \
    } while (0)

static void* at(uint64_t gb, uint64_t off = 0) { return (void*)((uint64_t(1) << 42) + (gb << 30) + off); }
// A call that passes its checks: launched, or refused by the runtime.
static bool planned(int rc) { return rc == FSDP_OK || rc == FSDP_E_HIP; }

static const int64_t kLim = int64_t(1) << 36;
static bool fits(int64_t r, int64_t c) { return r >= 0 && c >= 0 && r <= kLim && c <= kLim && (r == 0 || c <= kLim / r - 128); }

static void blocks(bool device) {
    const int64_t sizes[] = {0, 1, 16, 17, 127, 128, 129, 4096, 28672, (1 << 20) + 1, (1 << 22), (1 << 22) + 1,
                             int64_t(1) << 33, int64_t(1) << 45, INT64_MAX / 128, INT64_MAX, -1, INT64_MIN};
    for (int64_t r : sizes)
        for (int64_t c : sizes) {
            const bool small = fits(r, c) && fits(c, r);
            for (int form = 1; form < 4; ++form)
                for (int tile : {0, 1}) {
                    if (device && small) continue;
                    const int rc = fsdp_fp8_quantize(at(0), form % 3, r, c, c, tile, form & 1 ? at(1024) : nullptr,
                                                     form & 1 ? at(2048) : nullptr, form & 2 ? at(3000) : nullptr,
                                                     form & 2 ? at(4096) : nullptr, nullptr);
                    CHECK(small ? planned(rc) || rc == FSDP_E_SIZE : rc <= 0);
                }
            for (int64_t k : sizes) {
                const bool all = small && fits(r, k) && fits(c, k) && fits(k, r) && fits(k, c);
                const bool product = all && k <= FSDP_FP8_MAX_K;
                const int64_t a = fsdp_fp8_matmul_workspace(r, c, k), b = fsdp_fp8_linear_workspace(r, c, k);
                CHECK(a >= -1 && b >= -1 && a % 16 <= 0 && b % 16 <= 0);
                if (product) CHECK(a >= 0);
                for (int want = 1; want < 4; ++want) {
                    const int64_t g = fsdp_fp8_linear_grads_workspace(r, c, k, want & 1, want >> 1);
                    CHECK(g >= -1 && g % 16 <= 0);
                    if (device && all) continue;
                    const int rc = fsdp_fp8_linear_grads(at(0), 2, c, at(512), 2, k, r, c, k, at(1024), at(2048), want & 1, 2,
                                                         want & 1 ? at(3000) : nullptr, k, 0, want & 2 ? at(4096) : nullptr, k,
                                                         at(8192), INT64_MAX, nullptr);
                    CHECK(rc <= 0);
                }
                if (device && all) continue;
                const int rc = fsdp_fp8_matmul(at(0), at(1024), 0, at(2048), at(3000), 1, r, c, k, 1, at(4096), c, at(8192),
                                               INT64_MAX, nullptr);
                CHECK(product ? planned(rc) : rc <= 0);
                const int l = fsdp_fp8_linear(at(0), 2, r, k, k, at(1024), at(2048), 1, c, 0, at(3000), c, at(8192), INT64_MAX,
                                              nullptr);
                CHECK(product ? planned(l) || l == FSDP_E_SIZE : l <= 0);
                // a byte less than the workspace, and an address off its grid
                if (product && a > 0 && r > 0 && c > 0) {
                    CHECK(fsdp_fp8_matmul(at(0), at(1024), 0, at(2048), at(3000), 1, r, c, k, 1, at(4096), c, at(8192), a - 1,
                                          nullptr) == FSDP_E_SIZE);
                    CHECK(fsdp_fp8_matmul(at(0), at(1024), 0, at(2048), at(3000), 1, r, c, k, 1, at(4096), c, at(8192, 8), a,
                                          nullptr) == FSDP_E_INVAL);
                    CHECK(fsdp_fp8_matmul(at(0), at(1024), 0, at(2048), at(3000), 1, r, c, k, 1, at(4096), c, at(4096), a,
                                          nullptr) == FSDP_E_ALIAS);
                }
            }
        }
    for (int world : {1, 2, 63, 64, 65, 128})
        for (int64_t S : {int64_t(0), int64_t(1), int64_t(128), int64_t(300), int64_t(4096), int64_t(1) << 40, INT64_MAX}) {
            std::vector<const void*> c(world), s(world);
            for (int q = 0; q < world; ++q) {
                c[q] = at(q, 0);
                s[q] = at(200 + q, 1);
            }
            if (device && S < (int64_t(1) << 40)) continue;
            const int a = fsdp_fp8_gather(c.data(), s.data(), world, S, 2, at(500), nullptr);
            const int b = fsdp_fp8_gather_packed(c.data(), s.data(), world, S, at(600), at(700, 3), nullptr);
            CHECK(S < 10000 ? planned(a) : a <= 0);
            CHECK(S < 10000 && S % 128 == 0 ? planned(b) : b <= 0);
        }
}

static void norms(bool device) {
    const int64_t rows[] = {0, 1, 2, 255, 256, 2047, 2048, 2049, 8192, 70000, int64_t(1) << 33, INT64_MAX / 40000, INT64_MAX, -1};
    const int64_t widths[] = {0, 1, 7, 8, 511, 512, 4096, 4097, 8192, 8193, 16384, 16385, FSDP_RMS_MAX_D, FSDP_RMS_MAX_D + 1,
                              INT64_MAX, -1};
    for (int64_t m : rows)
        for (int64_t d : widths) {
            const bool ok = m >= 0 && d >= 0 && d <= FSDP_RMS_MAX_D && m <= 70000;
            const int64_t ws = fsdp_rms_norm_grads_workspace(m, d, 1);
            CHECK(ws >= -1 && fsdp_rms_norm_grads_workspace(m, d, 0) <= 0);
            if (ok) CHECK(ws >= 0 && ws <= int64_t(1024) * FSDP_RMS_MAX_D * 4 && (m < 2 || d == 0 || ws > 0));
            if (device && ok) continue;
            for (int dt = 0; dt < 3; ++dt) {
                const int a = fsdp_rms_norm_fp8(at(0), dt, d, at(100), (fsdp_dtype)((dt + 1) % 3), d, m, d, at(200), dt, 1e-6,
                                                at(300), d, dt, dt ? at(400) : nullptr, d, at(500), at(600), (float*)at(700), nullptr);
                const int b = fsdp_rms_norm_fp8(at(0), dt, d, nullptr, dt, 0, m, d, at(200), dt, 0.0, nullptr, 0, dt, nullptr, 0,
                                                at(500), at(600), nullptr, nullptr);
                const int c = fsdp_rms_norm_grads(at(0), dt, d, at(100), (fsdp_dtype)((dt + 1) % 3), d, m, d, at(200), dt,
                                                  (float*)at(300), dt ? at(400) : nullptr, d, at(500), d, dt, at(600), at(700),
                                                  INT64_MAX, nullptr);
                CHECK(ok ? planned(a) && planned(b) && planned(c) : a <= 0 && b <= 0 && c <= 0);
            }
            if (ok && ws > 0)
                CHECK(fsdp_rms_norm_grads(at(0), 0, d, at(100), 0, d, m, d, at(200), 0, (float*)at(300), nullptr, 0, at(500), d, 0,
                                          at(600), at(700), ws - 1, nullptr) == FSDP_E_SIZE);
        }
    auto norm = [](double eps, void* h, void* y, void* codes) {
        return fsdp_rms_norm_fp8(at(0), 0, 64, at(100), 0, 64, 8, 64, at(200), 0, eps, h, 64, 0, y, 64, codes, at(600), nullptr, nullptr);
    };
    for (double eps : {-1e-9, (double)NAN, (double)INFINITY}) CHECK(norm(eps, at(300), nullptr, at(500)) == FSDP_E_INVAL);
    CHECK(norm(0.0, nullptr, nullptr, at(500)) == FSDP_E_INVAL && norm(0.0, at(300), nullptr, at(500, 8)) == FSDP_E_INVAL);
    CHECK(norm(0.0, at(300), at(100), at(500)) == FSDP_E_ALIAS && norm(0.0, at(300), nullptr, at(300)) == FSDP_E_ALIAS);
    CHECK(norm(0.0, at(100, 4), nullptr, at(500)) == FSDP_E_ALIAS);
    if (!device) CHECK(planned(norm(0.0, at(100), nullptr, at(500))) && planned(norm(0.0, at(0), nullptr, at(500))));
}

int main() {
    int devices = 0;
    const bool device = hipGetDeviceCount(&devices) == hipSuccess && devices > 0;
    blocks(device);
    norms(device);
    std::vector<std::thread> t;                  // calls at once keep their errors apart
    for (int i = 0; i < 4; ++i)
        t.emplace_back([i] {
            for (int k = 0; k < 200; ++k)
                if (fsdp_rms_norm_grads_workspace(i % 2 ? -1 : 64, 64, 1) != (i % 2 ? -1 : 64 * 64 * 4)) exit(1);
        });
    for (auto& x : t) x.join();
    printf("layer sanitizer checks: %d checks ok\n", g_checks);
    return 0;
}
