// The second half of a product whose K is split (see gemm_split_kernel).
#pragma once

#include "epilogue.hpp"

namespace ts {

// Enqueues the sum over the splits and the epilogue, C of type c (ELT_*); false if that failed.
bool launch_split_finish(SplitArgs& g, int c, hipStream_t stream);

}  // namespace ts
