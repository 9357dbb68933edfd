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

}  // namespace ks
