// What the decode operators' kernels share beside the row kernels' helpers.
#pragma once

#include "ks_kernels.cuh"

namespace ks {

// Fault bit (KS_FAULT_BAD_INDEX): a slot, page or length read on the device was out of range; its
// access was left out.
constexpr unsigned int kFaultBadIndex = KS_FAULT_BAD_INDEX;

// a / b for a, b >= 0: by 32 bits where they fit (a fifth of the time of the 64-bit routine).
__device__ inline int64_t quotient(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// n / d for n below 2^27 by a multiplication: with k = floor(log2 d) and m = floor(2^(31 + k) / d) + 1, m d is at most
// d < 2^(k + 1) above 2^(31 + k), and n times that is below 2^(28 + k), too little to reach the next whole number.
struct Divisor {
    uint32_t magic;
    int32_t shift;
    __host__ static Divisor of(uint32_t d) {
        Divisor v = {0, 0};
        while (d >> (v.shift + 1)) ++v.shift;
        if (d) v.magic = (uint32_t)((1ull << (31 + v.shift)) / d) + 1;
        return v;
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return __umulhi(2 * n, magic) >> shift; }
};

}  // namespace ks
