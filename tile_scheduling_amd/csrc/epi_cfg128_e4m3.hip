// Kernel instances with the fused epilogue: the 128x128 tile, e4m3 operands (K steps of 128
// values), A stored [M][K] and B [N][K].
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_kernels_cfg128_e4m3(int out, int path, int kind) {
    switch (out) {
        case ELT_F16: return epi_kernel<Cfg128, InE4M3, OutF16>(path, kind);
        case ELT_BF16: return epi_kernel<Cfg128, InE4M3, OutBF16>(path, kind);
        default: return epi_kernel<Cfg128, InE4M3, OutF32>(path, kind);
    }
}
}  // namespace ts
