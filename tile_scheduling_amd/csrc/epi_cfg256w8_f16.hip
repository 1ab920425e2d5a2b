// Kernel instances with the fused epilogue: the 256x256x64 (8 waves) tile, f16 operands, every
// operand layout.
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_kernels_cfg256w8_f16(int out_f32, int path, int kind) {
    return out_f32 ? epi_kernel<Cfg256w8, InF16, OutF32>(path, kind) : epi_kernel<Cfg256w8, InF16, OutF16>(path, kind);
}
}  // namespace ts
