// fsdp_rms.h -- internal interface between the host layer of the norms over
// features (fsdp_rms_abi.cpp) and their kernels (fsdp_rms.hip, fsdp_rms_grads.hip).  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fsdp_kernels.h"

namespace fsdp {

struct RmsForward {
    const void* x;                 // [m][d] of xdt, ldx elements from row to row
    const void* residual;          // [m][d] of hdt, or null
    int xdt, hdt;
    int64_t ldx, ldr, m, d;
    const void* weight;            // [d] of wdt
    int wdt;
    double eps;
    void* h;                       // [m][d] of hdt, or null
    int64_t ldh;
    void* y;                       // [m][d] of ydt, or null
    int ydt;
    int64_t ldy;
    uint8_t *codes, *scales;       // blocks along d
    float* rstd;                   // [m], or null
};
hipError_t launch_rms_forward(const RmsForward& p, void* stream);

// Partial sums of dweight, a row of d each, that a call makes at most.
constexpr int64_t kRmsParts = 1024;
int64_t rms_parts(int64_t m, int64_t d);

struct RmsBackward {
    const void* dy;                // [m][d] of ydt
    const void* h;                 // [m][d] of hdt
    int ydt, hdt;
    int64_t ldy, ldh, m, d;
    const void* weight;            // [d] of wdt
    int wdt;
    const float* rstd;             // [m]
    const void* dh;                // [m][d] of hdt, added to dx; or null
    int64_t lddh;
    void* dx;                      // [m][d] of hdt, or null
    int64_t lddx;
    void* dw;                      // [d] of dwdt, or null
    int dwdt;
    float* parts;                  // [rms_parts(m, d)][d], or null where that is at most 1
};
hipError_t launch_rms_backward(const RmsBackward& p, void* stream);

}  // namespace fsdp
