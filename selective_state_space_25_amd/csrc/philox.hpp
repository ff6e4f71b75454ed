// philox.hpp -- Philox4x32-10, the counter-based generator of Salmon, Moraes,
// Dror and Shaw ("Parallel random numbers: as easy as 1, 2, 3", 2011): ten
// rounds of two 32 x 32 -> 64 bit products and xors with a key that moves by
// fixed odd steps.  Any word of the stream comes from its index alone, so a
// dropout mask is computed again wherever it is needed and never stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace selscan {

__device__ __forceinline__ void philox4(uint64_t index, uint64_t offset, uint64_t seed, uint32_t w[4]) {
    uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u;
        const uint64_t p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

}  // namespace selscan
