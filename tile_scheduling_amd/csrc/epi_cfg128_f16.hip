// Kernel instances with the fused epilogue: the 128x128x64 tile, f16 operands, every
// operand layout.
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_kernels_cfg128_f16(int out_f32, int path, int kind) {
    return out_f32 ? epi_kernel<Cfg128, InF16, OutF32>(path, kind) : epi_kernel<Cfg128, InF16, OutF16>(path, kind);
}
}  // namespace ts
