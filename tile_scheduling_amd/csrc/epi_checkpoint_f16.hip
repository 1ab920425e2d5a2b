// Kernel instances with preact in 8 bits: both tiles, fp16 operands; the special forms A stored [M][K].
#include "epilogue_checkpoint.hpp"
#include "internal.hpp"

namespace ts {
const void* epi_checkpoint_f16(int cfg, int out_f32, int path, int fam) {
    if (!out_f32 && fam >= 0 && (path == PATH_EDGE_BT || path == PATH_EDGE_NN)) {
        if (cfg == CFG_128)
            return path == PATH_EDGE_BT ? epi_checkpoint_special<Cfg128, InF16, OutF16, PATH_EDGE_BT>(fam)
                                        : epi_checkpoint_special<Cfg128, InF16, OutF16, PATH_EDGE_NN>(fam);
        return path == PATH_EDGE_BT ? epi_checkpoint_special<Cfg256w8, InF16, OutF16, PATH_EDGE_BT>(fam)
                                    : epi_checkpoint_special<Cfg256w8, InF16, OutF16, PATH_EDGE_NN>(fam);
    }
    if (cfg == CFG_128) return out_f32 ? epi_checkpoint<Cfg128, InF16, OutF32>(path) : epi_checkpoint<Cfg128, InF16, OutF16>(path);
    return out_f32 ? epi_checkpoint<Cfg256w8, InF16, OutF32>(path) : epi_checkpoint<Cfg256w8, InF16, OutF16>(path);
}
}  // namespace ts
