// Loads from memory straight to LDS, and the waits for them.
#pragma once

#include "psgd_internal.h"

#define LDS __attribute__((address_space(3)))

namespace psgd {
namespace {

// 16 bytes per lane from base + off (bytes) straight to LDS: lane x writes at l + 16 x. As asm, since
// with the builtin the compiler waits for every such load before each transposing LDS read; the
// waits are written out below (wait_loads). The load has no register output.
__device__ __forceinline__ void load_lds16(const GLOBAL uint16_t* base, uint32_t off, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(l), "v"(off), "s"(base) : "m0", "memory");
}

// All but the wave's n newest loads have landed, and its LDS reads have been answered. The builtin
// rather than asm: the compiler then knows that the fragments are there. The empty asm keeps LDS
// reads from moving across.
template <int N> __device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace psgd
