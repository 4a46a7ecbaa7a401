// kivi_paged_tc.cu -- attention of long chunks over a paged cache on the
// 5th-generation tensor cores.
//
// A chunk of many new tokens reads every cached token many times (once per 256
// query rows), so the pages are dequantised once, into the workspace, as the
// very images the matrix instructions take from shared memory, and the
// attention itself is a dense one:
//
//  stage_kernel   a pair's tokens in order (pages, sink, window, new tokens),
//                 128 to a tile: the keys as [token][channel], the values
//                 transposed as [channel][token], fp16, each as two panels of
//                 128-byte rows in the 128-byte swizzle (16-byte chunk i of row
//                 r lies at chunk i ^ (r & 7)).  Both operands are then K-major.
//  tc_kernel      256 query rows (two M tiles of 128) of one pair against a
//                 range of its tiles.  Ten warps: one fetches tiles (a bulk copy
//                 of 32 KB per operand, two stages), one issues the matrix
//                 instructions, and a warpgroup per M tile keeps the softmax,
//                 a thread per query row.  S = Q K^T and O += P V accumulate
//                 in tensor memory; P (fp16) overwrites the S it came from, so
//                 one M tile's softmax runs while the other's products do.
//                 O is only rescaled when a row's maximum has grown by more
//                 than 2^8 since the last time: until then 2^(s - m) stays
//                 within fp16 and nothing is lost by an old m.
#include <algorithm>

#include "kivi_paged_attend.cuh"

namespace kivi {
namespace {

constexpr int kTok = 128;                        // tokens per tile
constexpr int kMTile = 128;                      // query rows per M tile
constexpr int kRows = 2 * kMTile;                // query rows per block
constexpr int kImage = kTok * kHeadDim * 2;      // bytes of one operand's tile
constexpr int kTileBytes = 2 * kImage;           // keys, then values
constexpr int kStages = 2;
constexpr int kTcThreads = 320;
constexpr int kStageThreads = 256;
constexpr int kLongRows = 128;                   // query rows per pair from which this path is taken
constexpr int64_t kStageBytes = 1ll << 30;       // staged pairs per launch
constexpr long long kWaitCycles = 1ll << 32;     // about 2 s
constexpr float kRescale = 8.0f;                 // log2 of how far a maximum may run ahead

// ------------------------------------------------------------------ stage ---

struct StageArgs {
    uint8_t *tiles;           // [pairs of this launch][tiles][kTileBytes]
    int tiles_per_pair;
    int pair0;
};

// 16-byte chunk `chunk` (8 elements) of row r of an image.
__device__ __forceinline__ int image_at(int r, int chunk)
{
    return (chunk >> 3) * (kImage / 2) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
}

template <class F>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(PagedArgs c, ChunkArgs x, StageArgs a)
{
    constexpr int D = kHeadDim, VS = D + 8;
    __shared__ __align__(16) __half sv[kTok * VS];
    const int p = a.pair0 + blockIdx.y, b = p / c.Hkv, h = p % c.Hkv, tid = threadIdx.x;
    int first, T;
    PagedState st;
    if (!sequence(c, x, b, first, T, st))
        return;
    const int deep = st.held * c.G, cached = deep + st.sink + st.window;
    const int total = cached + (x.k ? T : 0), base = blockIdx.x * kTok;
    if (base >= total || T == 0)
        return;
    const RecGeo<F> geo(c.G);
    uint8_t *tile = a.tiles + ((int64_t)blockIdx.y * a.tiles_per_pair + blockIdx.x) * kTileBytes;
    for (int i = tid; i < kTok * 16; i += kStageThreads) {
        const int t = i >> 4, c8 = i & 15, u = base + t;
        uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;      // tokens behind the last one count as zero
        if (u < deep) {
            const unsigned char *rec = page_record(c, p, u / c.G);
            if (rec) {
                float f[8];
                page_k8<F>(rec, geo, u % c.G, c8, c.fp8_k_scale, f);
                kv = make_uint4(pack_sat(f[0], f[1]), pack_sat(f[2], f[3]), pack_sat(f[4], f[5]), pack_sat(f[6], f[7]));
                page_v8<F>(rec, geo, u % c.G, c8, c.fp8_v_scale, f);
                vv = make_uint4(pack_sat(f[0], f[1]), pack_sat(f[2], f[3]), pack_sat(f[4], f[5]), pack_sat(f[6], f[7]));
            } else if (c8 == 0) {
                atomicOr(c.control, KIVI_STATUS_BAD_PAGE);
            }
        } else if (u < total) {
            const __half *ks, *vs;
            if (u < cached) {
                const int64_t off = ((int64_t)p * c.rows + fp16_row(u - deep, st.sink, c.Ns, c.R, st.head)) * D;
                ks = c.k_fp16 + off;
                vs = c.v_fp16 + off;
            } else {
                const int64_t off = (int64_t)(first + u - cached) * x.kv_stride + h * D;
                ks = x.k + off;
                vs = x.v + off;
            }
            kv = *reinterpret_cast<const uint4 *>(ks + 8 * c8);
            vv = *reinterpret_cast<const uint4 *>(vs + 8 * c8);
        }
        *reinterpret_cast<uint4 *>(tile + image_at(t, c8)) = kv;
        *reinterpret_cast<uint4 *>(sv + t * VS + 8 * c8) = vv;
    }
    __syncthreads();
    for (int i = tid; i < D * 16; i += kStageThreads) {
        const int ch = i & (D - 1), t8 = i >> 7;              // 8 tokens of one channel
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 v = __halves2half2(sv[(8 * t8 + 2 * k) * VS + ch], sv[(8 * t8 + 2 * k + 1) * VS + ch]);
            w[k] = *reinterpret_cast<const uint32_t *>(&v);
        }
        *reinterpret_cast<uint4 *>(tile + kImage + image_at(ch, t8)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// -------------------------------------------------- barriers, tensor memory ---

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t phase)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(phase) : "memory");
    return ok != 0;
}

// Waits for a phase, about 2 s at most; false, with *failed set for the whole
// block, when it does not come.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t phase, volatile int *failed)
{
    if (bar_try(bar, phase))
        return true;
    const long long start = clock64();
    while (!bar_try(bar, phase)) {
        if (*failed || clock64() - start > kWaitCycles) {
            *failed = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Shared-memory operand: K-major rows of 128 bytes, 128-byte swizzle, groups of
// eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// fp16 x fp16 -> fp32, both K-major, M = 128, N = 128.
constexpr uint32_t kIdesc = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(kIdesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(kIdesc), "r"(accumulate) : "memory");
}

// The barrier completes a phase when every matrix instruction issued so far has.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tm_load32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                 "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                 "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}

__device__ __forceinline__ void tm_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// -------------------------------------------------------------- attention ---

struct TcOut {
    const uint8_t *tiles;
    int tiles_per_pair, pair0, S;
    int rows;                 // query rows a pair has room for in the partial results
    __half *out;
    float *o;                 // [pairs of this launch][rows][S][D] (S > 1)
    float2 *ml;               // [pairs of this launch][rows][S]
};

struct TcSmem {
    uint8_t q[2][kImage];
    uint8_t k[kStages][kImage];
    uint8_t v[kStages][kImage];
    uint64_t k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
    uint64_t s_full[2], p_full[2];
    uint32_t tmem;
    int failed;
};

template <bool CAP>
__global__ void __launch_bounds__(kTcThreads, 1) tc_kernel(PagedArgs c, ChunkArgs x, TcOut d)
{
    constexpr int D = kHeadDim;
    extern __shared__ uint8_t smem_raw[];
    TcSmem &sm = *reinterpret_cast<TcSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int p = d.pair0 + blockIdx.y, b = p / c.Hkv, h = p % c.Hkv;
    int first, T;
    PagedState st;
    if (!sequence(c, x, b, first, T, st)) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0)
            atomicOr(c.control, KIVI_STATUS_BAD_STATE);
        return;
    }
    const int rows = T * c.g, row0 = blockIdx.x * kRows;
    if (row0 >= rows)
        return;
    const int cached = st.held * c.G + st.sink + st.window;
    const int seen = !x.k ? 0 : x.full ? T : min(T, (row0 + kRows - 1) / c.g + 1);
    const int total = cached + seen;
    const int tiles = (total + kTok - 1) / kTok;
    const int t0 = (int)((int64_t)tiles * blockIdx.z / d.S), n = (int)((int64_t)tiles * (blockIdx.z + 1) / d.S) - t0;
    const int mtiles = rows - row0 > kMTile ? 2 : 1;

    // queries, swizzled like the keys; rows behind the last one count as zero
    for (int i = tid; i < mtiles * kMTile * 16; i += kTcThreads) {
        const int r = i >> 4, c8 = i & 15, row = row0 + r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) {
            const int t = row / c.g, hh = row - t * c.g;
            v = *reinterpret_cast<const uint4 *>(x.q + (int64_t)(first + t) * x.q_stride + (h * c.g + hh) * D + 8 * c8);
        }
        *reinterpret_cast<uint4 *>(sm.q[r >> 7] + image_at(r & 127, c8)) = v;
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(smem_addr(&sm.k_full[i]), 1);
            bar_init(smem_addr(&sm.k_free[i]), 1);
            bar_init(smem_addr(&sm.v_full[i]), 1);
            bar_init(smem_addr(&sm.v_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&sm.s_full[i]), 1);
            bar_init(smem_addr(&sm.p_full[i]), kMTile);
        }
        sm.failed = 0;
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tm = sm.tmem;                  // columns: S/P of tile 0, of tile 1, O of tile 0, of tile 1
    volatile int *failed = &sm.failed;

    if (warp == 9) {
        if (lane == 0) {                          // fetches the tiles
            const uint8_t *src = d.tiles + ((int64_t)blockIdx.y * d.tiles_per_pair + t0) * kTileBytes;
            int sent = 0;
            for (int j = 0; j < n; ++j, src += kTileBytes) {
                const int s = j % kStages;
                const uint32_t free_phase = ((j / kStages) & 1) ^ 1;      // the first round passes at once
                if (!bar_wait(smem_addr(&sm.k_free[s]), free_phase, failed))
                    break;
                bar_expect(smem_addr(&sm.k_full[s]), kImage);
                bulk_load(smem_addr(sm.k[s]), src, kImage, smem_addr(&sm.k_full[s]));
                if (!bar_wait(smem_addr(&sm.v_free[s]), free_phase, failed)) {
                    sent = -j - 1;                // the keys of tile j are on their way, its values are not
                    break;
                }
                bar_expect(smem_addr(&sm.v_full[s]), kImage);
                bulk_load(smem_addr(sm.v[s]), src + kImage, kImage, smem_addr(&sm.v_full[s]));
                sent = j + 1;
            }
            if (*failed) {                        // leave no copy in flight: wait, with a limit, for the last ones
                const int upto = sent < 0 ? -sent : sent;
                for (int j = max(0, upto - kStages); j < upto; ++j) {
                    const long long start = clock64();
                    const uint32_t phase = (j / kStages) & 1;
                    while (!bar_try(smem_addr(&sm.k_full[j % kStages]), phase) && clock64() - start < kWaitCycles) {}
                    if (!(sent < 0 && j == upto - 1))
                        while (!bar_try(smem_addr(&sm.v_full[j % kStages]), phase) && clock64() - start < kWaitCycles) {}
                }
            }
        }
    } else if (warp == 8) {
        if (lane == 0 && n > 0) {                 // issues the matrix instructions
            auto qk = [&](int i, int s) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = (ks >> 2) * (kImage / 2) + (ks & 3) * 32;
                    mma_ss(tm + 128 * i, operand(smem_addr(sm.q[i]) + off), operand(smem_addr(sm.k[s]) + off), ks > 0);
                }
            };
            bool ok = bar_wait(smem_addr(&sm.k_full[0]), 0, failed);
            if (ok) {
                for (int i = 0; i < mtiles; ++i) {
                    qk(i, 0);
                    mma_commit(smem_addr(&sm.s_full[i]));
                }
                mma_commit(smem_addr(&sm.k_free[0]));
            }
            for (int j = 0; ok && j < n; ++j) {
                const int s = j % kStages, s1 = (j + 1) % kStages;
                const bool more = j + 1 < n;
                ok = bar_wait(smem_addr(&sm.v_full[s]), (j / kStages) & 1, failed) &&
                     (!more || bar_wait(smem_addr(&sm.k_full[s1]), ((j + 1) / kStages) & 1, failed));
                for (int i = 0; ok && i < mtiles; ++i) {
                    ok = bar_wait(smem_addr(&sm.p_full[i]), j & 1, failed);
                    if (!ok)
                        break;
                    tm_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = (ks >> 2) * (kImage / 2) + (ks & 3) * 32;
                        mma_ts(tm + 256 + 128 * i, tm + 128 * i + 8 * ks, operand(smem_addr(sm.v[s]) + off), j > 0 || ks > 0);
                    }
                    if (more)
                        qk(i, s1);
                    mma_commit(smem_addr(&sm.s_full[i]));
                }
                if (ok) {
                    mma_commit(smem_addr(&sm.v_free[s]));
                    if (more)
                        mma_commit(smem_addr(&sm.k_free[s1]));
                }
            }
        }
    } else if ((warp >> 2) < mtiles) {
        // softmax: warpgroup i owns M tile i, a thread one query row (its TMEM lane)
        const int i = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;             // 32 lanes a warp, lane field from bit 16
        const uint32_t ts = tm + 128 * i + lanes, to = tm + 256 + 128 * i + lanes;
        const int row = row0 + i * kMTile + (warp & 3) * 32 + lane;
        const int tok = row / c.g, hh = row - tok * c.g;
        // tokens this row sees, from the first of this block's range
        const int limit = (row < rows && x.k && !x.full ? min(total, cached + tok + 1) : total) - t0 * kTok;
        const float scale = CAP ? 1.0f : x.scale_log2;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full[i]), j & 1, failed));
            if (!ok)
                break;
            tm_fence_after();
            uint32_t r[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                tm_load32(ts + 32 * q, r[q]);
            tm_wait_load();
            if constexpr (CAP) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        r[q][k] = __float_as_uint(score_log2(__uint_as_float(r[q][k]), x));
            }
            const int left = limit - j * kTok;
            if (left < kTok) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * q + k >= left)
                            r[q][k] = 0xff800000u;                      // -inf
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(r[q][k]));
            const float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grown = (tile_max - m) * scale > kRescale;        // also the first time (m = -inf)
            if (__any_sync(0xffffffffu, grown)) {
                const float m1 = grown ? tile_max : m;
                const float alpha = grown && l > 0.0f ? ex2((m - m1) * scale) : 1.0f;
                m = m1;
                l *= alpha;
                if (j > 0) {
                    // O is at rest: the phase just waited for ends after the last P V
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[32];
                        tm_load32(to + 32 * q, o);
                        tm_wait_load();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        tm_store32(to + 32 * q, o);
                    }
                }
            }
            const float ms = m == -INFINITY ? 0.0f : m * scale;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float a0 = ex2(fmaf(__uint_as_float(r[2 * q + (k >> 4)][2 * (k & 15)]), scale, -ms));
                    const float a1 = ex2(fmaf(__uint_as_float(r[2 * q + (k >> 4)][2 * (k & 15) + 1]), scale, -ms));
                    sum[k & 3] += a0 + a1;
                    pk[k] = pack_sat(a0, a1);
                }
                tm_store32(ts + 32 * q, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tm_wait_store();
            tm_fence_before();
            bar_arrive(smem_addr(&sm.p_full[i]));
        }
        if (n > 0 && ok)
            ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full[i]), n & 1, failed));   // the last P V
        tm_fence_after();
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const int64_t part = (((int64_t)blockIdx.y * d.rows + row) * d.S + blockIdx.z);
        const int64_t at = (int64_t)(first + tok) * (c.Hkv * c.g) + h * c.g + hh;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            __syncwarp();
            if (n > 0) {
                tm_load32(to + 32 * q, o);
                tm_wait_load();
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = 0u;
            }
            if (row < rows) {
                if (d.S == 1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_sat(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                        *reinterpret_cast<uint4 *>(d.out + at * D + 32 * q + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4 *>(d.o + part * D + 32 * q + 4 * k) =
                            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
        }
        if (d.S > 1 && row < rows)
            d.ml[part] = make_float2(m == -INFINITY ? m : m * scale, l);
    }
    tm_fence_before();
    __syncthreads();
    if (tid == 0 && sm.failed)
        atomicOr(c.control, KIVI_STATUS_WAIT_TIMEOUT);
    if (warp == 8) {
        __syncwarp();
        tm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
    }
}

constexpr int kTcSmem = sizeof(TcSmem) + 1024;
constexpr int kTcBlocks = 152;

struct TcPlan {
    int tiles, row_tiles, pairs, splits;      // pairs: staged and attended to per launch
    int64_t pair_bytes;
};

TcPlan tc_plan(const PagedArgs &c, int max_new, int max_cached)
{
    TcPlan p;
    p.tiles = (int)(((int64_t)max_cached + max_new + kTok - 1) / kTok);
    p.row_tiles = (int)(((int64_t)max_new * c.g + kRows - 1) / kRows);
    p.pair_bytes = (int64_t)p.tiles * kTileBytes;
    p.pairs = (int)std::max<int64_t>(1, std::min<int64_t>(c.B * c.Hkv, kStageBytes / p.pair_bytes));
    const int64_t blocks = (int64_t)p.pairs * p.row_tiles;
    // one wave of blocks; a split has four tiles or more
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(kTcBlocks / blocks, p.tiles / 4));
    return p;
}

template <class F>
void launch_stage(const PagedArgs &c, const ChunkArgs &x, const StageArgs &a, dim3 grid, cudaStream_t s)
{
    stage_kernel<F><<<grid, kStageThreads, 0, s>>>(c, x, a);
}

}  // namespace

bool is_long_chunk(const PagedArgs &c, int max_new) { return (int64_t)max_new * c.g >= kLongRows; }

size_t long_chunk_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    if (!is_long_chunk(c, max_new))
        return 0;
    const TcPlan p = tc_plan(c, max_new, max_cached);
    // staged tiles of one launch, and partial results: at most one wave of blocks has them
    const int64_t staged = std::min<int64_t>((int64_t)c.B * c.Hkv * p.pair_bytes, std::max(kStageBytes, p.pair_bytes));
    return (size_t)staged + (size_t)kTcBlocks * kRows * (kHeadDim + 2) * 4;
}

cudaError_t launch_long_chunk(const PagedArgs &c, const ChunkArgs &x, __half *out, void *ws, cudaStream_t s,
                              int *launches)
{
    const TcPlan p = tc_plan(c, x.max_new, x.max_cached);
    const int all = c.B * c.Hkv;
    TcOut d{};
    d.tiles = static_cast<uint8_t *>(ws);
    d.tiles_per_pair = p.tiles;
    d.S = p.splits;
    d.rows = p.row_tiles * kRows;
    d.out = out;
    d.o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.pair_bytes * p.pairs);
    d.ml = reinterpret_cast<float2 *>(d.o + (int64_t)p.pairs * d.rows * p.splits * kHeadDim);
    const void *kernel = x.cap_log2 != 0.0f ? (const void *)tc_kernel<true> : (const void *)tc_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess)
        return e;
    *launches = 0;
    for (int p0 = 0; p0 < all; p0 += p.pairs) {
        const int pairs = std::min(p.pairs, all - p0);
        const StageArgs a{static_cast<uint8_t *>(ws), p.tiles, p0};
        const dim3 grid(p.tiles, pairs);
        if (c.fmt == KIVI_FP8_E4M3)
            launch_stage<PageFmt<8, 0, KIVI_FP8_E4M3>>(c, x, a, grid, s);
        else if (c.fmt == KIVI_FP8_E5M2)
            launch_stage<PageFmt<8, 0, KIVI_FP8_E5M2>>(c, x, a, grid, s);
        else if (c.bits == 2)
            c.meta ? launch_stage<PageFmt<2, 1, 0>>(c, x, a, grid, s) : launch_stage<PageFmt<2, 0, 0>>(c, x, a, grid, s);
        else
            c.meta ? launch_stage<PageFmt<4, 1, 0>>(c, x, a, grid, s) : launch_stage<PageFmt<4, 0, 0>>(c, x, a, grid, s);
        d.pair0 = p0;
        const dim3 tgrid(p.row_tiles, pairs, p.splits);
        if (x.cap_log2 != 0.0f)
            tc_kernel<true><<<tgrid, kTcThreads, kTcSmem, s>>>(c, x, d);
        else
            tc_kernel<false><<<tgrid, kTcThreads, kTcSmem, s>>>(c, x, d);
        *launches += 2;
        if (p.splits > 1) {
            const float *ml = reinterpret_cast<const float *>(d.ml);
            e = launch_join(c, x, Parts{ml, ml + 1, d.o, 2, p.splits, p0, 0, d.rows}, out, pairs, s);
            if (e != cudaSuccess)
                return e;
            *launches += 1;
        }
        e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace kivi
