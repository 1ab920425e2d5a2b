// The second half of a product whose K is split (see gemm_split_kernel).
#pragma once

#include "epilogue.hpp"

namespace ts {

// Enqueues the sum over the splits and the epilogue, C of type c (ELT_*).
hipError_t launch_split_finish(const SplitArgs& g, int c, hipStream_t stream);

}  // namespace ts
