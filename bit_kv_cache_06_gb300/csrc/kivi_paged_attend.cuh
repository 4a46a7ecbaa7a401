// kivi_paged_attend.cuh -- tiles of a paged cache as matrix operands, and the
// pieces the attention and the weights kernels are made of.
#pragma once

#include "kivi_paged.cuh"

namespace kivi {
namespace {

// ------------------------------------------------------- stored elements ---
// Storage formats of a page: KIVI codes of BITS bits with fp32 (MF = 0) or
// fp16 (MF = 1) scales and zero points, or FP8 (FMT) with one scale a tensor.
template <int BITS_, int MF_, int FMT_>
struct PageFmt {
    static constexpr int BITS = BITS_, MF = MF_, FMT = FMT_;
    static constexpr int RB = kHeadDim * BITS / 8;        // code bytes per token row
    static constexpr int MW = MF ? 2 : 4;
    static constexpr int META = FMT ? 0 : 2 * MW * kHeadDim;
};

// A record's geometry for a group size known at run time.
template <class F>
struct RecGeo {
    int G, lgG, SL, VG, sub;
    __device__ explicit RecGeo(int g)
        : G(g), lgG(g == 16 ? 4 : g == 32 ? 5 : g == 64 ? 6 : 7), SL(g < 32 ? g : 32), VG(kHeadDim / g)
    {
        sub = SL * (2 * F::RB + 2 * F::MW * VG);
    }
    __device__ int row(int u) const { return F::META + (u / SL) * sub; }     // its sub-slice
};

template <int FMT>
__device__ __forceinline__ float2 fp8x2_float2(uint16_t x)
{
    uint32_t d;
    if constexpr (FMT == KIVI_FP8_E5M2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(d) : "h"(x));
    else
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(x));
    return __half22float2(*reinterpret_cast<__half2 *>(&d));
}

// Channels 8 c8 .. 8 c8 + 7 of token u of a record, dequantised in fp32:
// (code - z) s, or fp8 * scale.
template <class F>
__device__ __forceinline__ void page_k8(const unsigned char *rec, const RecGeo<F> &geo, int u, int c8,
                                        float scale, float (&x)[8])
{
    if constexpr (F::FMT != 0) {
        const uint2 w = *reinterpret_cast<const uint2 *>(rec + u * kHeadDim + 8 * c8);
        const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = fp8x2_float2<F::FMT>((uint16_t)(ww[i / 2] >> (16 * (i & 1))));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
    } else {
        const unsigned char *row = rec + geo.row(u) + (u % geo.SL) * F::RB + c8 * F::BITS;
        const uint32_t w = F::BITS == 2 ? *reinterpret_cast<const uint16_t *>(row)
                                        : *reinterpret_cast<const uint32_t *>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = meta_load<F::MF>(rec, 8 * c8 + i);
            const float z = meta_load<F::MF>(rec + F::MW * kHeadDim, 8 * c8 + i);
            x[i] = ((float)((w >> (F::BITS * i)) & ((1u << F::BITS) - 1u)) - z) * s;
        }
    }
}

template <class F>
__device__ __forceinline__ void page_v8(const unsigned char *rec, const RecGeo<F> &geo, int u, int c8,
                                        float scale, float (&x)[8])
{
    if constexpr (F::FMT != 0) {
        page_k8<F>(rec + 32 * kHeadDim, geo, u, c8, scale, x);
    } else {
        const unsigned char *base = rec + geo.row(u);
        const unsigned char *row = base + geo.SL * F::RB + (u % geo.SL) * F::RB;
        const unsigned char *vs = base + 2 * geo.SL * F::RB;
        const unsigned char *vz = vs + geo.SL * F::MW * geo.VG;
        const int run = geo.G >> 3;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int ch = 8 * c8 + i;
            const int j = ch >> geo.lgG;
            const int in = ch & (geo.G - 1);
            const int pos = run * F::BITS < 8 ? ch : 16 * (in / run) + run * j + in % run;
            const uint32_t code = (row[pos * F::BITS / 8] >> (pos * F::BITS % 8)) & ((1u << F::BITS) - 1u);
            const int m = (u % geo.SL) * geo.VG + j;
            x[i] = ((float)code - meta_load<F::MF>(vz, m)) * meta_load<F::MF>(vs, m);
        }
    }
}

// ------------------------------------------------------------ mma pieces ---
__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
