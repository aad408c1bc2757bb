// fsdp_norm.h -- internal interface between the host layer of the gradient
// norm and clipping (fsdp_norm_abi.cpp) and their kernels (fsdp_norm.hip).
// Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fsdp_kernels.h"

namespace fsdp {

// Partial sums that one call may write: doubles of its workspace.
constexpr int kNormSlots = FSDP_NORM_WORKSPACE_BYTES / 8;

// Tensors of one launch (all of one format), as chunks of a fixed number of
// bytes: tensor k owns chunks [chunk_begin[k], chunk_begin[k + 1]).
struct TensorTable {
    static constexpr int kMax = 160;
    int32_t count;
    int64_t chunk_begin[kMax + 1];
    void* p[kMax];
    int64_t n[kMax];               // elements
};
static_assert(sizeof(TensorTable) <= 4000, "tables travel in kernel arguments");

// Units of one launch whose averaged gradient is summed (and stored where out
// is not null), in tiles: nvec vectors of 8 elements, then single elements.
// The units' gradient pointers lie one after the other, world of them each.
template <int NW>
struct NormUnits {
    static constexpr int kMax = NW == 0 ? 40 : (NW <= 2 ? 70 : (NW <= 4 ? 54 : 38));
    static constexpr int kPtrs = NW > 0 ? NW * kMax : 280;
    int32_t count;
    int32_t world;
    int64_t tile_begin[kMax + 1];
    int64_t nvec[kMax];
    int64_t S[kMax];
    void* out[kMax];
    const void* g[kPtrs];
    bool wide[kMax];               // every buffer starts on the 16-byte grid
};
static_assert(sizeof(NormUnits<1>) <= 4000 && sizeof(NormUnits<2>) <= 4000 && sizeof(NormUnits<4>) <= 4000 &&
                  sizeof(NormUnits<8>) <= 4000 && sizeof(NormUnits<0>) <= 4000,
              "tables travel in kernel arguments");
static_assert(NormUnits<0>::kPtrs >= FSDP_MAX_WORLD, "a unit of any world fits");

struct NormUnitArgs {
    const void* const* grads;      // world pointers, already offset to block `rank`
    void* out;                     // averaged shard, or null
    int64_t S;
    bool wide;
};

// Where a norm goes: sums of squares, their root and the clipping coefficient
// (device, each may be null).
struct NormOut {
    double* sumsq;
    float* norm;
    float* coef;
    double max_norm;
};

// Bytes of a tensor that a workgroup takes at a time when it sums.
constexpr int64_t kSumChunkBytes = 16384;
// Bytes of a tensor that a workgroup scales: one 16-byte vector a lane.
constexpr int64_t kClipChunkBytes = 4096;

inline int norm_units_max(int world) {
    return world == 1 || world == 2 ? NormUnits<2>::kMax : world == 4 ? NormUnits<4>::kMax
         : world == 8 ? NormUnits<8>::kMax
         : NormUnits<0>::kPtrs / world < NormUnits<0>::kMax ? NormUnits<0>::kPtrs / world : NormUnits<0>::kMax;
}

// Sums of squares of the tables' tensors into partial[0 .. *used) (`slots` at
// most), in a fixed order.  With `fin` not null the one workgroup of a launch
// that has just one writes the result itself (*used = 0).  bytes: those of all
// the call's tensors.
hipError_t launch_sumsq(const TensorTable& t, int dt, int64_t bytes, double* partial, int slots, const NormOut* fin,
                        int cus, int* used, void* stream);
hipError_t launch_norm_units(const NormUnitArgs* units, int n, int world, int grad_dt, int fp32_reduce,
                             const ReduceScalars& rs, double* partial, int slots, int cus, int* used, void* stream);
hipError_t launch_norm_finish(const double* partial, int n, const NormOut& out, void* stream);
hipError_t launch_clip(const TensorTable& t, int dt, int64_t bytes, const float* coef, void* stream);

}  // namespace fsdp
