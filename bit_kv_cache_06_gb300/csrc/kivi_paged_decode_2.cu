// kivi_paged_decode_2.cu -- the decode kernel's paged forms for 2-bit codes
// with fp32 scales and zero points, compiled apart so that they build at once.
#include "kivi_decode_kernels.cuh"

namespace kivi {

cudaError_t launch_paged_decode_2(const PagedDecodeArgs &a, int gq, bool weights, int pairs, cudaStream_t s,
                                     int *blocks_per_sm)
{
    return launch_paged_bits<2, 0>(a, gq, weights, pairs, s, blocks_per_sm);
}

}  // namespace kivi
