// ops_checks.cpp -- the host layer of the gradient norm, clipping and the 4-bit
// microscaled blocks under the sanitizers: argument validation, table building
// and launch planning with device pointers that nothing dereferences.  Without
// a device every launch is refused by the runtime, after the tables were built.
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

static void* at(uint64_t gb, uint64_t off = 0) { return (void*)((uint64_t(1) << 40) + (gb << 30) + off); }
// A call that passes its checks: launched, or refused by the runtime.
static bool planned(int rc) { return rc == FSDP_OK || rc == FSDP_E_HIP; }

static void norms(bool device) {
    double* sum = (double*)at(900);
    float *norm = (float*)at(901), *coef = (float*)at(902);
    void* ws = at(903);
    for (int n : {0, 1, 2, 159, 160, 161, 1000}) {
        std::vector<const void*> p(n);
        std::vector<int64_t> s(n);
        std::vector<fsdp_dtype> d(n);
        for (int k = 0; k < n; ++k) {
            p[k] = at(0, (uint64_t)k << 22);
            s[k] = (k * 7919) % 100003;
            d[k] = k % 3;
        }
        if (!device) {
            CHECK(planned(fsdp_grad_norm(p.data(), s.data(), d.data(), n, 1.0, sum, norm, coef, ws, nullptr)));
            CHECK(planned(fsdp_clip_grads((void* const*)p.data(), s.data(), d.data(), n, coef, nullptr)));
        }
        if (n > 1) {
            d[n - 1] = 3;
            CHECK(fsdp_grad_norm(p.data(), s.data(), d.data(), n, 1.0, sum, norm, coef, ws, nullptr) == FSDP_E_DTYPE);
            d[n - 1] = 0;
            s[n - 1] = INT64_MAX;
            CHECK(fsdp_grad_norm(p.data(), s.data(), d.data(), n, 1.0, sum, norm, coef, ws, nullptr) == FSDP_E_SIZE);
            CHECK(fsdp_clip_grads((void* const*)p.data(), s.data(), d.data(), n, coef, nullptr) == FSDP_E_SIZE);
        }
    }
    CHECK(fsdp_grad_norm(nullptr, nullptr, nullptr, 3, 1.0, sum, norm, coef, ws, nullptr) == FSDP_E_INVAL);
    CHECK(fsdp_grad_norm(nullptr, nullptr, nullptr, 0, NAN, sum, norm, coef, ws, nullptr) == FSDP_E_INVAL);
    for (int world : {1, 2, 3, 4, 5, 8, 100, 128})
        for (int units : {0, 1, 39, 71, 200}) {
            std::vector<std::vector<const void*>> g(units);
            std::vector<fsdp_norm_unit> u(units);
            for (int k = 0; k < units; ++k) {
                for (int q = 0; q < world; ++q) g[k].push_back(at(q, (uint64_t)k << 21));
                u[k] = fsdp_norm_unit{g[k].data(), k % 2 ? at(500, (uint64_t)k << 20) : nullptr, k * 37 % 1000};
            }
            for (int dt = 0; dt < 3; ++dt)
                for (int f32 : {0, 1})
                    if (!device)
                        CHECK(planned(fsdp_grad_norm_units(u.data(), units, world, world - 1, dt, f32, 1.0, sum, norm,
                                                           coef, ws, nullptr)));
            if (units) {
                u[units - 1].shard_numel = INT64_MAX / 2;
                CHECK(fsdp_grad_norm_units(u.data(), units, world, 0, 0, 1, 1.0, sum, norm, coef, ws, nullptr) ==
                      FSDP_E_SIZE);
                u[units - 1].shard_numel = -1;
                CHECK(fsdp_grad_norm_units(u.data(), units, world, 0, 0, 1, 1.0, sum, norm, coef, ws, nullptr) ==
                      FSDP_E_INVAL);
            }
        }
    CHECK(fsdp_grad_norm_combine((double*)at(0), INT32_MIN, 1.0, sum, nullptr, nullptr, nullptr) == FSDP_E_INVAL);
    if (!device) CHECK(planned(fsdp_grad_norm_combine((double*)at(0), INT32_MAX, 1.0, sum, norm, coef, nullptr)));
}

static void blocks(bool device) {
    const int64_t lim = int64_t(1) << 36;
    const int64_t sizes[] = {0, 1, 15, 16, 17, 31, 32, 33, 255, 4096, 28672, (1 << 23), (1 << 23) + 1, int64_t(1) << 33,
                             int64_t(1) << 45, INT64_MAX / 32, INT64_MAX, -1, INT64_MIN};
    for (int64_t r : sizes)
        for (int64_t c : sizes) {
            const bool small = r >= 0 && c >= 0 && r <= lim && c <= lim && (r == 0 || c <= lim / r);
            if (device && small) continue;
            for (int form = 1; form < 4; ++form) {
                // operands far enough apart for the sizes that pass
                const int rc = fsdp_mx4_quantize(at(0), form % 3, r, c, c, form & 1 ? at(1024) : nullptr,
                                                 form & 1 ? at(2048) : nullptr, form & 2 ? at(3000) : nullptr,
                                                 form & 2 ? at(4096) : nullptr, nullptr);
                if (small) CHECK(planned(rc));
                else CHECK(rc <= 0);
            }
            const int64_t w = fsdp_mx4_linear_workspace(r, c), gw = fsdp_mx4_linear_grads_workspace(r, c, c, 1, 1);
            CHECK(w >= -1 && gw >= -1);
            if (small) CHECK(w >= 0);
            for (int64_t k : sizes) {
                const bool fits = small && k >= 0 && k <= lim && (k == 0 || (r <= lim / k && c <= lim / k));
                if (device && fits) continue;
                const int rc = fsdp_mx4_matmul(at(0), at(1024), at(2048), at(3000), r, c, k, 1, at(4096), c, nullptr);
                CHECK(fits && k <= FSDP_MX4_MAX_K ? planned(rc) : rc <= 0);
                const int l = fsdp_mx4_linear(at(0), 2, r, k, k, at(1024), at(2048), c, 0, at(3000), c, at(4096),
                                              INT64_MAX, nullptr);
                CHECK(fits && k <= FSDP_MX4_MAX_K ? planned(l) : l <= 0);
                const int g = fsdp_mx4_linear_grads(at(0), 2, c, at(512), 2, k, r, c, k, at(1024), at(2048), 2, at(3000),
                                                    k, 0, at(4096), k, at(8192), INT64_MAX, nullptr);
                CHECK(g <= 0);
            }
        }
    for (int world : {1, 2, 63, 64, 65, 128})
        for (int64_t S : {int64_t(0), int64_t(1), int64_t(32), int64_t(100), int64_t(4096), int64_t(1) << 40, INT64_MAX}) {
            std::vector<const void*> c(world), s(world);
            for (int q = 0; q < world; ++q) {
                c[q] = at(q, 0);
                s[q] = at(200 + q, 1);
            }
            if (device && S < (int64_t(1) << 40)) continue;
            const int a = fsdp_mx4_gather(c.data(), s.data(), world, S, 2, at(500), nullptr);
            const int b = fsdp_mx4_gather_packed(c.data(), s.data(), world, S, at(600), at(700, 3), nullptr);
            CHECK(S < 10000 ? planned(a) : a <= 0);
            CHECK(S < 10000 && S % 32 == 0 ? planned(b) : b <= 0);
        }
}

int main() {
    int devices = 0;
    const bool device = hipGetDeviceCount(&devices) == hipSuccess && devices > 0;
    norms(device);
    blocks(device);
    std::vector<std::thread> t;                  // calls at once keep their errors apart
    for (int i = 0; i < 4; ++i)
        t.emplace_back([i] {
            for (int k = 0; k < 200; ++k)
                if (fsdp_mx4_linear_workspace(i % 2 ? -1 : 64, 64) != (i % 2 ? -1 : 64 * 2 * 17)) exit(1);
        });
    for (auto& x : t) x.join();
    printf("ops sanitizer checks: %d checks ok\n", g_checks);
    return 0;
}
