// kivi_paged_stage.cuh -- a paged cache's tokens as operand tiles: 128 tokens a
// tile, keys and values dequantised to fp16 as [token][channel], each as two
// panels of 64 channels (128-byte rows, 128-byte swizzle: 16-byte chunk i of
// row r lies at chunk i ^ (r & 7)), the form the matrix instructions of
// kivi_paged_tc.cu take from shared memory.
//
// A pair's page tiles come first, its fp16 tokens (sink, window, new ones)
// follow in tiles of their own, so that one factor per tile undoes what the
// stored numbers are scaled by: pages of codes hold half their values (a group
// that spans fp16's whole range has dequantised values up to 4/3 of it), FP8
// pages hold theirs without the tensor's scale.
//
// Codes become numbers in fp16 pairs:
//   n = code - z       exact: (1024 + code) is the code's bits under an exponent,
//                      and integers up to 2048 are fp16 numbers
//   hi = n fp16(s/2)   one rounding (the scale's is another)
// Runs whose zero point is beyond +-1000 (a narrow group far from zero), or whose
// halved scale is not a normal fp16 number, take fp32 arithmetic instead.  What keys lose to rounding is multiplied by the
// query, and a few channels of keys are far larger than the rest, so
//   attention  the kChannels channels with the largest scales also get
//              lo = (code - z) s/2 - hi, a tile of their own, 32-byte rows
//   weights    (fp32 results) every channel gets it; no values are staged
// The order of channels inside a run of 16 is that in which one mask yields
// pairs of codes -- k and k + 8 (2-bit) or k + 4 (4-bit) -- and the values'
// runs are those of the stored order; queries and outputs follow.
//
// Bound by memory and latency: 96 to 256 bytes read and 512 (+32) written a token.
// 8 pairs of 34816 tokens, 2-bit: 39 us, 152 MB written (most of it into L2), 3.9
// TB/s.
#pragma once

#include "kivi_paged_attend.cuh"
#include "kivi_paged_tc.cuh"

namespace kivi {
namespace {

constexpr int kStageThreads = 256;
constexpr float kLeastScale = 0x1p-14f;          // fp16's smallest normal number

template <int BITS_, int G_, int FMT_>
struct StageCfg {
    static constexpr int BITS = BITS_, G = G_, FMT = FMT_;
    static constexpr int D = kHeadDim;
    static constexpr int NR = kTok / G;                       // records per tile
    static constexpr int SL = G < 32 ? G : 32;
    static constexpr int RB = D * BITS / 8;
    static constexpr int VG = FMT ? 1 : D / G;
    static constexpr int RL = G / 8;                          // value channels of a run
    static constexpr bool NATURAL = RL * BITS < 8;            // value order of the record
    __host__ __device__ static constexpr int sub(int mw) { return FMT ? 0 : SL * (2 * RB + 2 * mw * VG); }
    __host__ __device__ static constexpr int head(int mw) { return FMT ? 0 : 2 * mw * D; }
    __host__ __device__ static constexpr int raw(int mw) { return FMT ? 64 * D : head(mw) + G / SL * sub(mw); }
    static constexpr int RAW = NR * raw(4);
    // element of a run of 16 at place w of the tiles
    __host__ __device__ static constexpr int element(int w) { return run_element(BITS, w); }
};

__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Pair i (0..7) of a run of 16 codes as 1024 + code: places 2i, 2i + 1.
template <int BITS>
__device__ __forceinline__ __half2 code_pair(const uint32_t (&w)[BITS / 2], int i)
{
    const uint32_t x = BITS == 2 ? w[0] >> (2 * i) : w[(i >> 2) & (BITS / 2 - 1)] >> (4 * (i & 3));
    return half2_of((x & (BITS == 2 ? 0x00030003u : 0x000f000fu)) | 0x64006400u);
}

// Code k of a run.
template <int BITS>
__device__ __forceinline__ float code_of(const uint32_t (&w)[BITS / 2], int k)
{
    return (float)((w[k * BITS / 32] >> (k * BITS % 32)) & ((1u << BITS) - 1u));
}

template <int BITS>
__device__ __forceinline__ void run_words(const unsigned char *src, uint32_t (&w)[BITS / 2])
{
    if constexpr (BITS == 2) {
        w[0] = *reinterpret_cast<const uint32_t *>(src);
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(src);
        w[0] = v.x;
        w[1] = v.y;
    }
}

template <int FMT>
__device__ __forceinline__ uint32_t fp8_pair(uint16_t x)
{
    uint32_t d;
    if constexpr (FMT == KIVI_FP8_E5M2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(d) : "h"(x));
    else
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(x));
    return d;
}

__device__ __forceinline__ float scale_of(const unsigned char *base, int mw, int i)
{
    return mw == 4 ? meta_load<0>(base, i) : meta_load<1>(base, i);
}

// Eight pairs (places 16 run .. + 15 of token t) into an image.
__device__ __forceinline__ void image_store(uint8_t *image, int t, int run, const uint32_t (&x)[8])
{
    *reinterpret_cast<uint4 *>(image + image_at(t, 2 * run)) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4 *>(image + image_at(t, 2 * run + 1)) = make_uint4(x[4], x[5], x[6], x[7]);
}

template <class C, bool WEIGHTS>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(PagedArgs c, ChunkArgs x, StageArgs a)
{
    constexpr int D = kHeadDim, BITS = C::BITS, G = C::G, FMT = C::FMT;
    __shared__ __align__(16) unsigned char raw_s[C::RAW];
    __shared__ __align__(16) uint32_t kprm[FMT ? 4 : C::NR * 128];        // [record][s, z][64 pairs]
    __shared__ __align__(16) __half vprm[FMT || WEIGHTS ? 8 : kTok * 2 * C::VG];   // [token][s, z][VG]
    __shared__ unsigned s_kslow[C::NR], s_vslow[4], s_none;
    const int p = a.pair0 + blockIdx.y, b = p / c.Hkv, h = p % c.Hkv, tid = threadIdx.x;
    int first, T;
    PagedState st;
    const bool some = sequence(c, x, b, first, T, st) && T > 0;
    let_next_in();
    wait_for_previous();
    if (!some)
        return;
    const int deep = st.held * G, rowed = st.sink + st.window, shallow = rowed + (x.k ? T : 0);
    const int np = (deep + kTok - 1) / kTok, nf = (shallow + kTok - 1) / kTok;
    if (blockIdx.x >= np + nf)
        return;
    uint8_t *tile = a.tiles + ((int64_t)blockIdx.y * a.tiles_per_pair + blockIdx.x) * kTileBytes;
    const int run = tid & 7, tt = tid >> 3;            // this thread's run of 16 channels, and tokens tt + 32 i

    if (blockIdx.x >= np) {                            // fp16 tokens
        const int base = (blockIdx.x - np) * kTok, count = min(kTok, shallow - base);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tt + 32 * i, u = base + t;
            uint32_t kx[8], vx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                kx[e] = vx[e] = 0u;                    // tokens behind the last one count as zero
            if (t < count) {
                const __half *ks, *vs;
                if (u < rowed) {
                    const int64_t off = ((int64_t)p * c.rows + fp16_row(u, st.sink, c.Ns, c.R, st.head)) * D;
                    ks = c.k_fp16 + off;
                    vs = c.v_fp16 + off;
                } else {
                    const int64_t off = (int64_t)(first + u - rowed) * x.kv_stride + h * D;
                    ks = x.k + off;
                    vs = x.v + off;
                }
                __half k16[16];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    reinterpret_cast<uint4 *>(k16)[q] = reinterpret_cast<const uint4 *>(ks + 16 * run)[q];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    kx[e] = bits_of(__halves2half2(k16[C::element(2 * e)], k16[C::element(2 * e + 1)]));
                if constexpr (!WEIGHTS) {
                    __half v16[16];                    // stored positions 16 run .. + 15, pairs of channels together
#pragma unroll
                    for (int q = 0; q < 16; q += 2)
                        reinterpret_cast<uint32_t *>(v16)[q / 2] =
                            *reinterpret_cast<const uint32_t *>(vs + value_channel(BITS, G, FMT, 16 * run + q));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        vx[e] = bits_of(__halves2half2(v16[C::element(2 * e)], v16[C::element(2 * e + 1)]));
                }
            }
            image_store(tile, t, run, kx);
            if constexpr (!WEIGHTS)
                image_store(tile + kImage, t, run, vx);
        }
        return;
    }

    // the tile's records
    const int mw = c.meta ? 2 : 4, base = blockIdx.x * kTok, count = min(kTok, deep - base);
    const int nr = count / G, sub = C::sub(mw), head = C::head(mw), raw = C::raw(mw), chunks = raw / 16;
    if (tid < C::NR)
        s_kslow[tid] = 0u;
    if (tid < 4)
        s_vslow[tid] = 0u;
    if (tid == 0)
        s_none = 0u;
    __syncthreads();
    for (int i = tid; i < nr * chunks; i += kStageThreads) {
        const int k = i / chunks, off = (i - k * chunks) * 16;
        const unsigned char *rec = page_record(c, p, base / G + k);
        if (!rec) {
            if (off == 0) {
                atomicOr(c.control, KIVI_STATUS_BAD_PAGE);
                atomicOr(&s_none, 1u << k);
            }
            continue;
        }
        if (WEIGHTS && (FMT ? off >= 32 * D : off >= head && (off - head) % sub >= C::SL * C::RB))
            continue;                                  // the keys alone
        *reinterpret_cast<uint4 *>(raw_s + k * raw + off) = __ldcg(reinterpret_cast<const uint4 *>(rec + off));
    }
    __syncthreads();
    const unsigned none = s_none;
    if constexpr (!FMT) {
        for (int i = tid; i < nr * 64; i += kStageThreads) {
            const int k = i >> 6, pair = i & 63;
            const unsigned char *rec = raw_s + k * raw;
            float s[2], z[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ch = (pair >> 3) * 16 + C::element(2 * (pair & 7) + e);
                s[e] = 0.5f * scale_of(rec, mw, ch);
                z[e] = scale_of(rec + mw * D, mw, ch);
            }
            if (!(fabsf(z[0]) <= 1000.0f && fabsf(z[1]) <= 1000.0f && fminf(s[0], s[1]) >= kLeastScale))
                atomicOr(&s_kslow[k], 1u << (pair >> 3));
            kprm[k * 128 + pair] = bits_of(__floats2half2_rn(s[0], s[1]));
            kprm[k * 128 + 64 + pair] = bits_of(__floats2half2_rn(-1024.0f - z[0], -1024.0f - z[1]));
        }
        if constexpr (!WEIGHTS) {
            for (int i = tid; i < count * C::VG; i += kStageThreads) {
                const int t = i / C::VG, j = i % C::VG, u = t % G;
                const unsigned char *vs = raw_s + t / G * raw + head + u / C::SL * sub + 2 * C::SL * C::RB;
                const int at = u % C::SL * C::VG + j;
                const float z = scale_of(vs + C::SL * mw * C::VG, mw, at);
                const float s = 0.5f * scale_of(vs, mw, at);
                if (!(fabsf(z) <= 1000.0f && s >= kLeastScale))
                    atomicOr(&s_vslow[t >> 5], 1u << (t & 31));
                vprm[(2 * t) * C::VG + j] = __float2half_rn(s);
                vprm[(2 * t + 1) * C::VG + j] = __float2half_rn(-1024.0f - z);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = tt + 32 * i, k = t / G, u = t % G;
        const bool there = t < count && !((none >> k) & 1u);
        const unsigned char *rec = raw_s + k * raw;
        uint32_t hi[8], lo[8], v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            hi[e] = lo[e] = v[e] = 0u;
        if constexpr (FMT != 0) {
            if (there) {
#pragma unroll
                for (int part = 0; part < (WEIGHTS ? 1 : 2); ++part) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(rec + part * 32 * D + u * D + 16 * run);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        (part ? v : hi)[e] = fp8_pair<FMT>((uint16_t)(ww[e >> 1] >> (16 * (e & 1))));
                }
            }
        } else if (there) {
            const unsigned char *kc = rec + head + u / C::SL * sub, *vc = kc + C::SL * C::RB;
            const int at = u % C::SL * C::RB + run * 2 * BITS;
            uint32_t w[BITS / 2];
            run_words<BITS>(kc + at, w);
            const bool slow = (s_kslow[k] >> run) & 1u;
            if (!slow) {
                const uint4 *pr = reinterpret_cast<const uint4 *>(kprm + k * 128 + 8 * run);
                const uint4 q[4] = {pr[0], pr[1], pr[16], pr[17]};
                const uint32_t *prm = reinterpret_cast<const uint32_t *>(q);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    hi[e] = bits_of(__hmul2(__hadd2(code_pair<BITS>(w, e), half2_of(prm[8 + e])), half2_of(prm[e])));
            }
            if (slow || WEIGHTS) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int el = C::element(2 * e + q), ch = 16 * run + el;
                        f[q] = 0.5f * ((code_of<BITS>(w, el) - scale_of(rec + mw * D, mw, ch)) * scale_of(rec, mw, ch));
                    }
                    if (slow)
                        hi[e] = pack_sat(f[0], f[1]);
                    const float2 g = __half22float2(half2_of(hi[e]));
                    lo[e] = pack_sat(f[0] - g.x, f[1] - g.y);
                }
            }
            if constexpr (!WEIGHTS) {
                run_words<BITS>(vc + at, w);
                // value group of element el of the run
                auto group = [&](int el) { return C::NATURAL ? run * 16 / G : el / C::RL; };
                if ((s_vslow[t >> 5] >> (t & 31)) & 1u) {
                    const unsigned char *vs = vc + C::SL * C::RB, *vz = vs + C::SL * mw * C::VG;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float f[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int el = C::element(2 * e + q), m = u % C::SL * C::VG + group(el);
                            f[q] = 0.5f * ((code_of<BITS>(w, el) - scale_of(vz, mw, m)) * scale_of(vs, mw, m));
                        }
                        v[e] = pack_sat(f[0], f[1]);
                    }
                } else {
                    struct __align__(2 * C::VG) Halves {
                        __half h[C::VG];
                    };
                    const __half *vp = vprm + 2 * t * C::VG;
                    const Halves vs = *reinterpret_cast<const Halves *>(vp), vz = *reinterpret_cast<const Halves *>(vp + C::VG);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        __half2 s, z;
                        if constexpr (C::NATURAL) {
                            s = __half2half2(vp[run * 16 / G]);
                            z = __half2half2(vp[C::VG + run * 16 / G]);
                        } else {
                            const int ja = C::element(2 * e) / C::RL, jb = C::element(2 * e + 1) / C::RL;
                            s = __halves2half2(vs.h[ja], vs.h[jb]);
                            z = __halves2half2(vz.h[ja], vz.h[jb]);
                        }
                        v[e] = bits_of(__hmul2(__hadd2(code_pair<BITS>(w, e), z), s));
                    }
                }
            }
        }
        image_store(tile, t, run, hi);
        if constexpr (!WEIGHTS)
            image_store(tile + kImage, t, run, v);
        else if constexpr (!FMT)
            image_store(tile + kImage, t, run, lo);
    }
    if constexpr (!WEIGHTS && !FMT) {
        // what the largest channels lose: 16-byte chunk q (8 channels) of token t
        const uint8_t *chan = a.channels + blockIdx.y * kChannels;
        const int t = tid >> 1, q = tid & 1, k = t / G, u = t % G;
        const bool there = t < count && !((none >> k) & 1u);
        const unsigned char *rec = raw_s + k * raw;
        const unsigned char *row = rec + head + u / C::SL * sub + u % C::SL * C::RB;
        uint32_t lo[4] = {0u, 0u, 0u, 0u};
        if (there) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int ch = chan[8 * q + 2 * e + i];
                    const float s = 0.5f * scale_of(rec, mw, ch), z = scale_of(rec + mw * D, mw, ch);
                    const float code = (float)((row[ch * BITS / 8] >> (ch * BITS % 8)) & ((1u << BITS) - 1u));
                    const float value = (code - z) * s;
                    const __half hi = (s_kslow[k] >> (ch >> 4)) & 1u
                                          ? __low2half(half2_of(pack_sat(value, 0.0f)))
                                          : __hmul(__float2half_rn(code - z), __float2half_rn(s));
                    f[i] = value - __half2float(hi);
                }
                lo[e] = pack_sat(f[0], f[1]);
            }
        }
        *reinterpret_cast<uint4 *>(tile + 2 * kImage + low_at(t, q)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

template <int BITS, int G, int FMT>
cudaError_t launch_stage_of(const PagedArgs &c, const ChunkArgs &x, const StageArgs &a, bool weights, dim3 grid,
                            cudaStream_t s)
{
    using C = StageCfg<BITS, G, FMT>;
    if (!weights)
        return launch_dependent(stage_kernel<C, false>, grid, kStageThreads, 0, s, c, x, a);
    stage_kernel<C, true><<<grid, kStageThreads, 0, s>>>(c, x, a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kivi
