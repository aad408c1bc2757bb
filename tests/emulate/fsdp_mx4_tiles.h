// What the 8-bit product takes from csrc/fsdp_mx4_tiles.h, for emulator.h.
#pragma once

#include <type_traits>

#include "fsdp_fp8_device.h"

namespace fsdp {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

inline void tile_of(uint32_t b, uint32_t, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    tm = b / tiles_n;
    tn = b % tiles_n;
}

}  // namespace fsdp
