// kivi_paged_stage_2.cu -- the staging kernel for 2-bit codes.
#include "kivi_paged_stage.cuh"

namespace kivi {

KIVI_STAGE(launch_stage_2)
{
    switch (c.G) {
    case 16: return launch_stage_of<2, 16, 0>(c, x, a, weights, grid, s);
    case 32: return launch_stage_of<2, 32, 0>(c, x, a, weights, grid, s);
    case 64: return launch_stage_of<2, 64, 0>(c, x, a, weights, grid, s);
    default: return launch_stage_of<2, 128, 0>(c, x, a, weights, grid, s);
    }
}

}  // namespace kivi
