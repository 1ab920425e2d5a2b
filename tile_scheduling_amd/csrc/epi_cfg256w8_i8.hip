// Kernel instances with the fused epilogue: the 256x256 (8 waves) tile, int8 operands (K steps of 128
// values), A stored [M][K] and B [N][K].
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_kernels_cfg256w8_i8(int out, int path, int kind) {
    switch (out) {
        case ELT_F16: return epi_kernel<Cfg256w8, InI8, OutF16>(path, kind);
        case ELT_BF16: return epi_kernel<Cfg256w8, InI8, OutBF16>(path, kind);
        default: return epi_kernel<Cfg256w8, InI8, OutF32>(path, kind);
    }
}
}  // namespace ts
