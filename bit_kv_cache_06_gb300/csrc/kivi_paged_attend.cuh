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

// tanh(y) = 1 - 2 / (e^(2y) + 1), to 2^-22 absolutely: it leaves a score off by
// 2^-22 of its cap.
__device__ __forceinline__ float tanh_far(float y)
{
    return 1.0f - __fdividef(2.0f, ex2(y * 2.8853900817779268f) + 1.0f);
}

// tanh(y) to about 2^-20 of itself: for |y| < 1/5 the series
// y - y^3/3 + 2 y^5/15 - 17 y^7/315, which is good for 2^-24 there.
__device__ __forceinline__ float tanh_any(float y)
{
    const float y2 = y * y;
    const float near = y * fmaf(y2, fmaf(y2, fmaf(y2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
    return fabsf(y) < 0.2f ? near : tanh_far(y);
}

// Scores in the log2 domain from products q.k times `times`: c log2(e)
// tanh(tau q.k / c).  Small caps (x.cap_small) take the short form: the long one
// cost 9 % of the page weights of 32 tokens and 3 % of an attention of 8.
template <bool SMALL, int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], float times, const ChunkArgs &x)
{
    const float f = x.cap_inv * times;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float y = __uint_as_float(s[k]) * f;
        s[k] = __float_as_uint(x.cap_log2 * (SMALL ? tanh_far(y) : tanh_any(y)));
    }
}

}  // namespace
}  // namespace kivi
