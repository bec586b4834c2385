// pair.cuh -- what the kernels on pairs of CTAs share: bounded waits of their
// roles, places in a ring, stores of whole sectors.
#pragma once

#include <cuda_bf16.h>

#include "sm100.cuh"

namespace dsa {
namespace sm100 {

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store_sector(void* p, const uint32_t* x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

constexpr long long kWaitCycles = 4000000000ll;  // about 2 s

// A place in the ring and the parity of its use, one block after the other.
struct Place {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void step(int ring) {
        if (++at == ring) { at = 0; parity ^= 1; }
    }
};

// A wait that ends early when another role gave up.  The clock is the SM's: reading
// the global timer between two tries cost up to 2,000 cycles after the arrival.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (*abort != 0 || clock64() - t0 > kWaitCycles) return false;
    return true;
}
// The same made by a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
    return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

}  // namespace sm100
}  // namespace dsa
