// Kernel instances with the fused epilogue: the 128x128x64 tile, bf16 operands, every
// operand layout.
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_kernels_cfg128_bf16(int out_f32, int path, int kind) {
    return out_f32 ? epi_kernel<Cfg128, InBF16, OutF32>(path, kind) : epi_kernel<Cfg128, InBF16, OutBF16>(path, kind);
}
}  // namespace ts
