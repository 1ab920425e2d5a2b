// Limits that the kernels' launches and the Python module (binding.cpp, no HIP) both count on.
#pragma once

namespace ts {

// Longest rows that the norms' gradients hold in the registers of a workgroup (1024 threads of four and of two
// groups of eight columns).  Longer ones need a workspace for numbers of each row, whether or not column sums are
// asked for.
constexpr long long kRmsGradRow = 32768, kLayerGradRow = 16384;

}  // namespace ts
