// kivi_paged_attend.cuh -- small pieces that the paged cache's kernels share.
#pragma once

#include "kivi_paged.cuh"

namespace kivi {
namespace {

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// {lo half: x0, hi half: x1}, to nearest, saturated to fp16's largest finite
// value (a dequantised value may lie half a step above its group's maximum).
__device__ __forceinline__ uint32_t pack_sat(float x0, float x1)
{
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x1), "f"(x0));
    return d;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Score of q.k in the log2 domain: tau log2(e) q.k, or with a cap
// c log2(e) tanh(tau q.k / c), tanh(y) = 1 - 2 / (e^(2y) + 1) (its absolute error
// of about 2^-23 is what counts here).
__device__ __forceinline__ float score_log2(float dot, const ChunkArgs &x)
{
    if (x.cap_log2 == 0.0f)
        return dot * x.scale_log2;
    const float e = ex2(dot * x.cap_inv * 2.8853900817779268f);      // e^(2y)
    return x.cap_log2 * (1.0f - __fdividef(2.0f, e + 1.0f));
}

}  // namespace
}  // namespace kivi
