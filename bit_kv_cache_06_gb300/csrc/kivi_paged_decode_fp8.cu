// kivi_paged_decode_fp8.cu -- the decode kernel's paged forms for FP8 pages.
#include "kivi_decode_kernels.cuh"

namespace kivi {

// (2-bit, G = 32 only size the per-warp stage buffers, as in kivi_decode_fp8.cu)
cudaError_t launch_paged_decode_fp8(const PagedDecodeArgs &a, int gq, bool weights, int pairs, cudaStream_t s,
                                    int *blocks_per_sm)
{
    return a.c.fmt == KIVI_FP8_E4M3 ? launch_paged_g<2, 32, 0, KIVI_FP8_E4M3>(a, gq, weights, pairs, s, blocks_per_sm)
                                    : launch_paged_g<2, 32, 0, KIVI_FP8_E5M2>(a, gq, weights, pairs, s, blocks_per_sm);
}

}  // namespace kivi
