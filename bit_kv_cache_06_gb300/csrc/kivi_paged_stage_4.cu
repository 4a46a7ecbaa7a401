// kivi_paged_stage_4.cu -- the staging kernel for 4-bit codes.
#include "kivi_paged_stage.cuh"

namespace kivi {

KIVI_STAGE(launch_stage_4)
{
    switch (c.G) {
    case 16: return launch_stage_of<4, 16, 0>(c, x, a, weights, grid, s);
    case 32: return launch_stage_of<4, 32, 0>(c, x, a, weights, grid, s);
    case 64: return launch_stage_of<4, 64, 0>(c, x, a, weights, grid, s);
    default: return launch_stage_of<4, 128, 0>(c, x, a, weights, grid, s);
    }
}

}  // namespace kivi
