// kivi_paged_stage_fp8.cu -- the staging kernel for FP8 pages.
#include "kivi_paged_stage.cuh"

namespace kivi {

KIVI_STAGE(launch_stage_fp8)
{
    return c.fmt == KIVI_FP8_E4M3 ? launch_stage_of<8, 32, KIVI_FP8_E4M3>(c, x, a, weights, grid, s)
                                  : launch_stage_of<8, 32, KIVI_FP8_E5M2>(c, x, a, weights, grid, s);
}

}  // namespace kivi
