// The tiled product of 8-bit blocks on emulated workgroups: whole numbers, so that every
// result is exact, over sums of few and of many blocks, tiles behind each other in one
// workgroup, ragged edges, split sums and two products in a launch.
#include "fsdp_fp8_matmul.hip"

using namespace fsdp;

hipError_t fsdp::launch_fp8_few(const Fp8Few&) {
    emu::check(false, "not a product in tiles");
    return hipSuccess;
}

namespace {

struct Matrix {
    int64_t rows, nb;
    int tile;
    std::vector<uint8_t> codes, scales;
    std::vector<float> values;
};
Matrix random_matrix(int64_t rows, int64_t nb, bool tile, unsigned seed) {
    static const uint8_t code[4] = {0x00, 0x38, 0xb8, 0x40};      // 0, 1, -1, 2
    static const float value[4] = {0, 1, -1, 2};
    std::mt19937 r(seed);
    Matrix m{rows, nb, tile ? 7 : 0, {}, {}, {}};
    m.codes.resize(rows * nb * 128);
    m.scales.resize((((rows - 1) >> m.tile) + 1) * nb);
    m.values.resize(m.codes.size());
    for (auto& s : m.scales) s = 127 + r() % 2;
    for (size_t i = 0; i < m.codes.size(); ++i) {
        const unsigned c = r() % 4;
        m.codes[i] = code[c];
        m.values[i] = value[c] * (float)(1 << (m.scales[((i / (nb * 128)) >> m.tile) * nb + i / 128 % nb] - 127));
    }
    return m;
}

constexpr size_t kGuard = 4096;
struct Result {
    int dt;
    int64_t m, n, ldo;
    std::vector<uint8_t> held;
    Result(int dt, int64_t m, int64_t n, int64_t gap) : dt(dt), m(m), n(n), ldo(n + gap) {
        held.assign(2 * kGuard + ((m - 1) * ldo + n) * dt_bytes(dt), 0xa5);
    }
    void* at() { return held.data() + kGuard; }
    void compare(const Matrix& a, const Matrix& b) {
        const int es = (int)dt_bytes(dt);
        const int64_t k = a.nb * 128;
        std::vector<uint8_t> seen(held.size(), 0);
        for (int64_t i = 0; i < m; ++i)
            for (int64_t j = 0; j < n; ++j) {
                const float *x = &a.values[i * k], *y = &b.values[j * k];
                float want = 0;                                    // whole numbers under 2^24
                for (int64_t t = 0; t < k; ++t) want += x[t] * y[t];
                const size_t o = kGuard + (i * ldo + j) * es;
                uint32_t u = 0;
                memcpy(&u, &held[o], es);
                memset(&seen[o], 1, es);
                const float got = __builtin_bit_cast(float, dt == FSDP_F32 ? u : u << 16);
                if (dt == FSDP_BF16) want = __builtin_bit_cast(float, (uint32_t)bits16(dt, want) << 16);
                if (got != want) {
                    fprintf(stderr, "%s: element %lld, %lld is %g, not %g\n", emu::what, (long long)i, (long long)j, got, want);
                    exit(1);
                }
            }
        for (size_t o = 0; o < held.size(); ++o) emu::check(seen[o] || held[o] == 0xa5, "a byte beside the result was written");
    }
};

struct Case {
    int64_t m, n, nb;
    int cus;
    bool ta, tb;
    int dt;
};
std::vector<Case> one = {
    // 256 x 256, more tiles than CUs: the second tile of a workgroup too
    {768, 768, 1, 8, false, false, FSDP_F32}, {768, 768, 2, 8, false, true, FSDP_F32}, {768, 768, 3, 8, true, false, FSDP_BF16},
    {640, 700, 5, 8, false, true, FSDP_F32}, {768, 768, 16, 8, false, true, FSDP_F32}, {768, 768, 17, 8, true, true, FSDP_F32},
    {600, 768, 33, 8, false, false, FSDP_F32}, {768, 768, 36, 8, false, true, FSDP_F32},
    // 128 x 128: two stages with a second tile, four stages
    {768, 768, 2, 16, false, true, FSDP_F32}, {768, 768, 18, 16, false, false, FSDP_F32}, {760, 768, 33, 16, true, true, FSDP_F32},
    {384, 384, 2, 16, false, true, FSDP_F32}, {384, 380, 17, 16, true, false, FSDP_F32},
    // 64 x 128, and 64 x 64 with its sum whole and split
    {192, 384, 3, 20, false, true, FSDP_F32}, {192, 380, 18, 20, false, false, FSDP_F32},
    {100, 130, 5, 32, false, true, FSDP_F32}, {100, 130, 35, 32, true, false, FSDP_F32}, {64, 128, 64, 32, false, true, FSDP_F32},
};

Fp8Product product(const Matrix& a, const Matrix& b, Result& r, int cus, std::vector<float>& parts) {
    const int64_t bytes = fp8_parts_bytes(r.m, r.n, a.nb, cus);
    parts.assign(bytes / 4, __builtin_nanf(""));
    return Fp8Product{a.codes.data(), a.scales.data(), b.codes.data(), b.scales.data(), a.tile, b.tile, r.m, r.n, a.nb, r.dt,
                      r.at(), r.ldo, cus, nullptr, bytes ? parts.data() : nullptr};
}
void readable(const Matrix& m) {
    emu::buffers.push_back({m.codes.data(), m.codes.data() + m.codes.size()});
    emu::buffers.push_back({m.scales.data(), m.scales.data() + m.scales.size()});
}
void said(const char* fmt, long long a, long long b, long long c, int cus) {
    static char text[200];
    static const char* how[] = {"late", "early", "random"};
    int n = snprintf(text, sizeof text, fmt, a, b, c, cus);
    snprintf(text + n, sizeof text - n, ", loads %s%s", how[emu::mode], emu::backwards ? ", last wave first" : "");
    emu::what = text;
    printf("%s\n", text);
    fflush(stdout);
}

}  // namespace

// products <part> <of>: every <of>th case from <part> on
int main(int argc, char** argv) {
    const unsigned part = (unsigned)atoi(argv[1]), of = (unsigned)atoi(argv[2]);
    const struct { emu::Mode mode; bool backwards; } ways[] = {{emu::kLate, false}, {emu::kEarly, true}, {emu::kRandom, false}};
    std::vector<float> parts, more;
    for (size_t i = part; i < one.size(); i += of) {
        const Case& c = one[i];
        const Matrix a = random_matrix(c.m, c.nb, c.ta, 1), b = random_matrix(c.n, c.nb, c.tb, 2);
        emu::buffers.clear();
        readable(a);
        readable(b);
        for (auto& way : ways) {
            emu::mode = way.mode;
            emu::backwards = way.backwards;
            said("%lld x %lld, %lld blocks, %d CUs", c.m, c.n, c.nb, c.cus);
            Result r(c.dt, c.m, c.n, c.n % 8 ? 3 : 0);
            (void)launch_fp8_matmul(product(a, b, r, c.cus, parts));
            r.compare(a, b);
        }
    }
    // a layer's gradients: dx m x k, dw n x k
    static const struct { int64_t m, n, k; int cus; } two[] = {{512, 512, 768, 8}, {300, 768, 384, 16}, {64, 100, 128, 32},
                                                               {256, 2304, 256, 16}};
    for (size_t i = part; i < sizeof two / sizeof *two; i += of) {
        const int64_t m = two[i].m, n = two[i].n, k = two[i].k, nbm = (m + 127) / 128, nbn = (n + 127) / 128;
        const Matrix dy = random_matrix(m, nbn, false, 3), wt = random_matrix(k, nbn, true, 4);
        const Matrix dyt = random_matrix(n, nbm, false, 5), xt = random_matrix(k, nbm, false, 6);
        emu::buffers.clear();
        for (const Matrix* x : {&dy, &wt, &dyt, &xt}) readable(*x);
        for (auto& way : ways) {
            emu::mode = way.mode;
            emu::backwards = way.backwards;
            said("gradients of %lld x %lld x %lld, %d CUs", m, n, k, two[i].cus);
            Result dx(FSDP_F32, m, k, 0), dw(FSDP_F32, n, k, 5);
            (void)launch_fp8_two(product(dy, wt, dx, two[i].cus, parts), product(dyt, xt, dw, two[i].cus, more));
            dx.compare(dy, wt);
            dw.compare(dyt, xt);
        }
    }
    printf("products done\n");
    return 0;
}
