// lds_copy.hpp -- direct copies from global memory to LDS for tile kernels whose
// stages lie at one uniform base.
#pragma once

#include "device.hpp"

namespace archead {

// lds_dma16 from a uniform base (in scalar registers) and a 32-bit byte offset
// per lane, with dst a byte address in LDS (uniform): no vector arithmetic.
// Inline assembly, and waited for by its callers, for lds_dma16's reasons.
__device__ __forceinline__ void lds_dma16_from(const void *base, uint32_t offset, uint32_t dst)
{
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, %2\n\ts_nop 0\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "v"(offset), "s"(base), "s"(dst)
                 : "memory");
}

// byte address in LDS of a __shared__ object
__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

} // namespace archead
