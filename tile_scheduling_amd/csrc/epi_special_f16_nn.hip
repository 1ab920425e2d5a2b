// Special forms of the fused epilogue: the 256x256x64 tile (8 waves), f16 operands, A [M][K] and
// B [K][N].
#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_special_f16_nn(int out_f32, int kind) {
    return out_f32 ? epi_special_by_kind<Cfg256w8, InF16, OutF32, PATH_EDGE_NN>(kind)
                   : epi_special_by_kind<Cfg256w8, InF16, OutF16, PATH_EDGE_NN>(kind);
}
// A [K][M]: the plain product only, the weight's gradient.
const void* epi_special_f16_tn(int out_f32, int kind) {
    if (kind != EPI_SPECIAL + 4 * AUX_NONE + FAM_NONE) return nullptr;
    return out_f32 ? epi_special<Cfg256w8, InF16, OutF32, PATH_EDGE_AT, FAM_NONE, AUX_NONE>()
                   : epi_special<Cfg256w8, InF16, OutF16, PATH_EDGE_AT, FAM_NONE, AUX_NONE>();
}
}  // namespace ts
