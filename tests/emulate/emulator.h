// Workgroups of gfx950 on the CPU, for kernels whose loads into LDS are waited for by
// count: a fiber a lane, waves that run one after the other up to a barrier, and loads
// into LDS that land as late as the waits allow (or at once, or at random).  A load that
// no wait covers is then read before it is there, and one that is sent too early overwrites
// what another wave still reads: either shows in the results.  Every load is checked
// against the buffers.  Lanes' accesses to LDS and global stores happen at once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <deque>
#include <functional>
#include <memory>
#include <random>
#include <vector>

#undef __device__
#undef __global__
#undef __shared__
#undef __forceinline__
#undef __launch_bounds__
#define __device__
#define __global__
#define __shared__
#define __forceinline__ inline
#define __launch_bounds__(...)

namespace fsdp {
alignas(1024) uint8_t lds[163840];
}

namespace emu {

enum Mode { kLate, kEarly, kRandom };
enum State { kRuns, kAtBarrier, kAtWave, kOver };

struct Access {
    bool into_lds;
    uint8_t* to;
    uint8_t data[16];
};
struct Lane {
    ucontext_t at;
    std::unique_ptr<char[]> stack;
    State state;
    std::deque<Access> queue;      // its wave's accesses, oldest first
    float a[2][32], b[2][32];      // the operands of its last two matrix instructions, scaled
    int turn;
};

inline Mode mode;
inline bool backwards;             // the order of the waves
inline std::mt19937 rng(1);
inline std::vector<std::unique_ptr<Lane>> lanes;
inline ucontext_t home;
inline int now;                    // the lane that runs
inline unsigned block, blocks, threads;
inline std::function<void()> body;
inline std::vector<std::pair<const uint8_t*, const uint8_t*>> buffers;
inline const char* what = "";

inline void check(bool ok, const char* why) {
    if (ok) return;
    fflush(stdout);
    fprintf(stderr, "%s: %s (workgroup %u, lane %d)\n", what, why, block, now);
    exit(1);
}
inline bool readable(const void* p, size_t n) {
    for (auto& b : buffers)
        if ((const uint8_t*)p >= b.first && (const uint8_t*)p + n <= b.second) return true;
    return false;
}

inline Lane& me() { return *lanes[now]; }
inline void yield(State s) {
    Lane& l = me();
    l.state = s;
    swapcontext(&l.at, &home);
}
inline void retire(Lane& l, size_t left) {
    while (l.queue.size() > left) {
        const Access& a = l.queue.front();
        if (a.into_lds && mode != kEarly) memcpy(a.to, a.data, 16);
        l.queue.pop_front();
    }
}
inline void issue(const Access& a) {
    Lane& l = me();
    if (a.into_lds && mode == kEarly) memcpy(a.to, a.data, 16);
    l.queue.push_back(a);
    if (mode == kRandom && rng() % 4 == 0) retire(l, rng() % (l.queue.size() + 1));
}
inline void other() { issue(Access{false, nullptr, {}}); }       // a load into registers, a store
inline void wait(int n) { retire(me(), (size_t)n); }
inline void barrier() { yield(kAtBarrier); }
inline void wave() { yield(kAtWave); }                           // the wave's lanes are all here

inline void enter() {
    body();
    for (const Access& a : me().queue) check(!a.into_lds, "a load into LDS outlasts its workgroup");
    yield(kOver);
}
inline void run_wave(unsigned w) {                               // until all its lanes are at a barrier, or over
    for (;;) {
        State s = kRuns;
        for (unsigned l = 64 * w; l < 64 * w + 64; ++l) {
            now = (int)l;
            if (lanes[l]->state == kRuns || lanes[l]->state == kAtWave) {
                lanes[l]->state = kRuns;
                swapcontext(&home, &lanes[l]->at);
            }
            if (l == 64 * w) s = lanes[l]->state;
            check(lanes[l]->state == s, "the wave's lanes are at different places");
        }
        if (s != kAtWave) return;
    }
}
inline void launch(unsigned grid, unsigned size, std::function<void()> f) {
    check(grid > 0 && size % 64 == 0 && size <= 1024, "launch");
    body = f;
    blocks = grid;
    threads = size;
    constexpr size_t kStack = 256 << 10;
    for (block = 0; block < grid; ++block) {
        memset(fsdp::lds, 0xff, sizeof fsdp::lds);               // NaN, as codes and as scales
        while (lanes.size() < size) {
            lanes.emplace_back(new Lane);
            lanes.back()->stack.reset(new char[kStack]);
        }
        for (unsigned l = 0; l < size; ++l) {
            getcontext(&lanes[l]->at);
            lanes[l]->at.uc_stack.ss_sp = lanes[l]->stack.get();
            lanes[l]->at.uc_stack.ss_size = kStack;
            lanes[l]->at.uc_link = nullptr;
            makecontext(&lanes[l]->at, enter, 0);
            lanes[l]->state = kRuns;
            lanes[l]->queue.clear();
            lanes[l]->turn = 0;
        }
        for (;;) {
            for (unsigned w = 0; w < size / 64; ++w) run_wave(backwards ? size / 64 - 1 - w : w);
            const State s = lanes[0]->state;
            for (unsigned l = 0; l < size; ++l) check(lanes[l]->state == s, "the waves are at different places");
            if (s == kOver) break;
            for (unsigned l = 0; l < size; ++l) lanes[l]->state = kRuns;
        }
    }
}

struct Index {
    unsigned x;
};
inline Index thread_index() { return Index{(unsigned)now}; }

// -------------------------------------------------------------- builtins
struct Buffer {
    const uint8_t* base;
    int bytes;
};
inline Buffer make_buffer(void* p, int, int bytes, int) {
    check(bytes >= 0 && (bytes == 0 || readable(p, (size_t)bytes)), "a buffer of more than the operand");
    return Buffer{(const uint8_t*)p, bytes};
}
inline void fetch(const Buffer& b, int voff, int soff, int n, uint8_t* out) {
    check(voff >= 0 && soff >= 0, "a negative offset");
    for (int i = 0; i < n; i += 4) {
        const int64_t at = (int64_t)voff + soff + i;
        if (at + 4 <= b.bytes) memcpy(out + i, b.base + at, 4);
        else memset(out + i, 0, 4);
    }
}
inline void load_to_lds(const Buffer& b, __attribute__((address_space(3))) void* to, int n, int voff, int soff, int, int) {
    Access a{true, (uint8_t*)to + (now & 63) * n, {}};
    check(n == 16 && a.to >= fsdp::lds && a.to + n <= fsdp::lds + sizeof fsdp::lds, "a load behind the LDS");
    fetch(b, voff, soff, n, a.data);
    issue(a);
}
inline uint32_t load_b32(const Buffer& b, int voff, int soff, int) {
    uint32_t x;
    fetch(b, voff, soff, 4, (uint8_t*)&x);
    other();
    return x;
}

typedef int i8 __attribute__((ext_vector_type(8)));
typedef float f16 __attribute__((ext_vector_type(16)));
inline float value_of(uint8_t c) {
    const int e = c >> 3 & 15, m = c & 7;
    const float v = (c & 127) == 127 ? __builtin_nanf("") : (e ? __builtin_ldexpf(1.0f + m / 8.0f, e - 7) : __builtin_ldexpf((float)m, -9));
    return c & 128 ? -v : v;
}
// Lane l brings row l % 32 of either side, 32 codes of half l / 32 and their scale byte; it
// gets column l % 32 (the second side's row) and rows 8 (i / 4) + 4 (l / 32) + i % 4.
inline f16 scaled_product(i8 a, i8 b, f16 acc, int, int, int byte_a, int scale_a, int byte_b, int scale_b) {
    static float values[256];
    static bool made = false;
    if (!made)
        for (int c = 0; c < 256; ++c) values[c] = value_of((uint8_t)c);
    made = true;
    Lane& l = me();
    const int turn = l.turn ^= 1;
    auto put = [&](float* to, const i8& x, uint32_t byte) {
        const float s = byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, (int)byte - 127);
        uint8_t c[32];
        memcpy(c, &x, 32);
        for (int i = 0; i < 32; ++i) to[i] = values[c[i]] * s;
    };
    put(l.a[turn], a, (uint32_t)scale_a >> (8 * byte_a) & 255);
    put(l.b[turn], b, (uint32_t)scale_b >> (8 * byte_b) & 255);
    wave();
    const int w = now & ~63, col = now & 31, half = now >> 5 & 1;
    for (int i = 0; i < 16; ++i) {
        const int row = 8 * (i / 4) + 4 * half + i % 4;
        float s = 0;
        for (int h = 0; h < 2; ++h) {
            const float *x = lanes[w + 32 * h + row]->a[turn], *y = lanes[w + 32 * h + col]->b[turn];
            for (int k = 0; k < 32; ++k) s += x[k] * y[k];
        }
        acc[i] += s;
    }
    return acc;
}

}  // namespace emu

#define threadIdx emu::thread_index()
#define blockIdx (emu::Index{emu::block})
#define gridDim (emu::Index{emu::blocks})
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __builtin_amdgcn_make_buffer_rsrc emu::make_buffer
#define __builtin_amdgcn_raw_ptr_buffer_load_lds emu::load_to_lds
#define __builtin_amdgcn_raw_buffer_load_b32 emu::load_b32
#define __builtin_amdgcn_sched_barrier(x) ((void)0)
#define __builtin_amdgcn_wave_barrier() emu::wave()
#define __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4 emu::scaled_product
#define hipGetLastError() hipSuccess
