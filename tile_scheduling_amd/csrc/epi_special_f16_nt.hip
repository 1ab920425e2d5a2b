// Special forms of the fused epilogue: the 256x256x64 tile (8 waves), f16 operands, A [M][K] and
// B [N][K].
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_special_f16_nt(int out_f32, int kind) {
    return out_f32 ? epi_special_by_kind<Cfg256w8, InF16, OutF32, PATH_EDGE_BT>(kind)
                   : epi_special_by_kind<Cfg256w8, InF16, OutF16, PATH_EDGE_BT>(kind);
}
}  // namespace ts
