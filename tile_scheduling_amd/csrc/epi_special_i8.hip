// Special forms of the fused epilogue: the 256x256x64 tile (8 waves), int8 operands, 16-bit C.
#include "epilogue_int8.hpp"

namespace ts {
const void* epi_special_i8(int out, int fam, int residual) {
    if (out == ELT_F16) return residual ? epi_int8_special<OutF16, true>(fam) : epi_int8_special<OutF16, false>(fam);
    return residual ? epi_int8_special<OutBF16, true>(fam) : epi_int8_special<OutBF16, false>(fam);
}
}  // namespace ts
