// kivi_paged_decode_4_f16.cu -- the decode kernel's paged forms for 4-bit codes
// with fp16 scales and zero points, compiled apart so that they build at once.
#include "kivi_decode_kernels.cuh"

namespace kivi {

cudaError_t launch_paged_decode_4_f16(const PagedDecodeArgs &a, int gq, bool weights, int pairs, cudaStream_t s,
                                     int *blocks_per_sm)
{
    return launch_paged_bits<4, 1>(a, gq, weights, pairs, s, blocks_per_sm);
}

}  // namespace kivi
