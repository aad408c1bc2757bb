// The waits of csrc/fsdp_waits.h for the emulated lanes of emulator.h.
#pragma once

#include "emulator.h"

namespace fsdp {

template <int N>
inline void wait_memory() { emu::wait(N); }
template <int MANY_FROM, int SOME_FROM, int FEW, int SOME, int MANY>
inline void wait_memory_by(int n) { emu::wait(n >= MANY_FROM ? MANY : (n >= SOME_FROM ? SOME : FEW)); }
inline void meet_in_lds() { emu::barrier(); }
inline void unknown(int&) {}
inline void needed(uint32_t) {}

}  // namespace fsdp
