// What the decode operators' kernels share beside the row kernels' helpers.
#pragma once

#include "ks_kernels.cuh"

namespace ks {

// Fault bit (KS_FAULT_BAD_INDEX): a slot, page or length read on the device was out of range; its
// access was left out.
constexpr unsigned int kFaultBadIndex = KS_FAULT_BAD_INDEX;

}  // namespace ks
