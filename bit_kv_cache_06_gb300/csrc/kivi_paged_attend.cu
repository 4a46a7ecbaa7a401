// kivi_paged_attend.cu -- attention of new tokens over a paged cache, and the
// softmax weights that its pages get.
//
// The query rows of one (sequence, kv head) pair are its new tokens times the
// g query heads that read the kv head (row r: token r / g, head r mod g), so
// every page is read once for all of them.  A pair's tokens are taken in tiles
// of 64: first the pages (held * G tokens), then the fp16 rows (sink and
// window), then the new tokens with their mask.  A block runs the tiles of one
// split for 64 query rows with a running maximum and sum:
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j        (scores in log2 units),
// and the splits are joined as o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
#include <algorithm>

#include "kivi_paged_attend.cuh"
#include "kivi_paged_decode.cuh"

namespace kivi {
namespace {

constexpr int kTile = 64;              // tokens per tile, query rows per block
constexpr int kAttendThreads = 128;
constexpr int kStride = kHeadDim + 8;  // halves per staged row: rows 4 banks apart
constexpr int kTargetBlocks = 152 * 4;

struct SplitOut {
    __half *out;          // attention: [num_tokens][Hq][D]
    float *o;             // [P][rows][S][D] partial outputs (S > 1)
    float2 *ml;           // [P][rows][S] running maximum and sum
    float *ls;            // weights: [P][rows][units] log2 of a unit's sum
    int S;
    int row0;             // first query row of this launch (attention: 0) ...
    int rows;             // ... and how many it has room for
    int unit, units;      // tokens per unit, units per row
};

// Tiles of one pair in order: pages, fp16 rows, new tokens.
struct Tiles {
    int pages, rows, fresh;
    __device__ int total() const { return pages + rows + fresh; }
};

template <class F, bool WEIGHTS>
__global__ void __launch_bounds__(kAttendThreads) attend_kernel(PagedArgs c, ChunkArgs x, SplitOut d)
{
    constexpr int D = kHeadDim;
    __shared__ __align__(16) __half sk[kTile * kStride];
    __shared__ __align__(16) __half sv[kTile * kStride];   // values; weights: the keys' low parts
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int p = blockIdx.y, b = p / c.Hkv, h = p % c.Hkv;
    int first, T;
    PagedState st;
    if (!sequence(c, x, b, first, T, st)) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0)
            atomicOr(c.control, KIVI_STATUS_BAD_STATE);
        return;
    }
    const int rows = T * c.g;
    const int tile_row0 = d.row0 + blockIdx.z * kTile;
    if (tile_row0 >= rows)
        return;
    const RecGeo<F> geo(c.G);
    const int seen = !x.k ? 0 : x.full ? T : min(T, (tile_row0 + kTile - 1) / c.g + 1);
    const Tiles n{(st.held * c.G + kTile - 1) / kTile, (st.sink + st.window + kTile - 1) / kTile,
                  (seen + kTile - 1) / kTile};
    const int t0 = (int)((int64_t)n.total() * blockIdx.x / d.S);
    const int t1 = (int)((int64_t)n.total() * (blockIdx.x + 1) / d.S);

    // this thread's two query rows and their A fragments
    const int qr = lane >> 2, qc = lane & 3;
    int row[2], tok[2];
    const __half *qp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        row[i] = tile_row0 + warp * 16 + qr + 8 * i;
        tok[i] = row[i] / c.g;
        const int hh = row[i] - tok[i] * c.g;
        qp[i] = row[i] < rows ? x.q + (int64_t)(first + tok[i]) * x.q_stride + (h * c.g + hh) * D : nullptr;
    }
    uint32_t qa[8][4];
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half *src = qp[k & 1];
            qa[s][k] = src ? *reinterpret_cast<const uint32_t *>(src + 16 * s + 2 * qc + 8 * (k >> 1)) : 0u;
        }
    float o[WEIGHTS ? 1 : 16][4];
#pragma unroll
    for (int j = 0; j < (WEIGHTS ? 1 : 16); ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[j][k] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int tile = t0; tile < t1; ++tile) {
        const bool page = tile < n.pages, fresh = tile >= n.pages + n.rows;
        const int base = (page ? tile : fresh ? tile - n.pages - n.rows : tile - n.pages) * kTile;
        const int count = min(kTile, (page ? st.held * c.G : fresh ? T : st.sink + st.window) - base);
        __syncthreads();                                  // the last tile is read
        for (int i = tid; i < kTile * 16; i += kAttendThreads) {
            const int t = i >> 4, c8 = i & 15;
            uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
            if (t < count) {
                if (page) {
                    const int u = base + t;
                    const unsigned char *rec = page_record(c, p, u / c.G);
                    if (rec) {
                        float f[8];
                        page_k8<F>(rec, geo, u % c.G, c8, c.fp8_k_scale, f);
                        kv = make_uint4(pack_sat(f[0], f[1]), pack_sat(f[2], f[3]), pack_sat(f[4], f[5]),
                                        pack_sat(f[6], f[7]));
                        if constexpr (WEIGHTS) {
                            const __half2 *hi = reinterpret_cast<const __half2 *>(&kv);
                            uint32_t lo[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 a = __half22float2(hi[k]);
                                lo[k] = pack_sat(f[2 * k] - a.x, f[2 * k + 1] - a.y);
                            }
                            vv = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        } else {
                            page_v8<F>(rec, geo, u % c.G, c8, c.fp8_v_scale, f);
                            vv = make_uint4(pack_sat(f[0], f[1]), pack_sat(f[2], f[3]), pack_sat(f[4], f[5]),
                                            pack_sat(f[6], f[7]));
                        }
                    } else if (c8 == 0) {
                        atomicOr(c.control, KIVI_STATUS_BAD_PAGE);
                    }
                } else {
                    const __half *ks, *vs;
                    if (fresh) {
                        const int64_t off = (int64_t)(first + base + t) * x.kv_stride + h * D;
                        ks = x.k + off;
                        vs = x.v + off;
                    } else {
                        const int r = fp16_row(base + t, st.sink, c.Ns, c.R, st.head);
                        const int64_t off = ((int64_t)p * c.rows + r) * D;
                        ks = c.k_fp16 + off;
                        vs = c.v_fp16 + off;
                    }
                    kv = *reinterpret_cast<const uint4 *>(ks + 8 * c8);
                    if constexpr (!WEIGHTS)
                        vv = *reinterpret_cast<const uint4 *>(vs + 8 * c8);
                }
            }
            *reinterpret_cast<uint4 *>(sk + t * kStride + 8 * c8) = kv;
            if (!WEIGHTS || page)
                *reinterpret_cast<uint4 *>(sv + t * kStride + 8 * c8) = vv;
        }
        __syncthreads();

        // scores of 16 rows x 64 tokens
        float s[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float hi[4] = {0.0f, 0.0f, 0.0f, 0.0f}, lo[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const uint32_t at = (uint32_t)((8 * j + (lane & 7)) * kStride + (lane >> 3) * 8) * 2;
#pragma unroll
            for (int ks = 0; ks < 8; ks += 2) {
                uint32_t kb[4];
                ldsm_x4(smem_addr(sk) + at + ks * 32, kb);
                mma16816(hi, qa[ks], kb[0], kb[1]);
                mma16816(hi, qa[ks + 1], kb[2], kb[3]);
                if (WEIGHTS && page) {
                    ldsm_x4(smem_addr(sv) + at + ks * 32, kb);
                    mma16816(lo, qa[ks], kb[0], kb[1]);
                    mma16816(lo, qa[ks + 1], kb[2], kb[3]);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int col = 8 * j + 2 * qc + (k & 1), i = k >> 1;
                bool see = col < count;
                if (fresh && !x.full)
                    see = see && base + col <= tok[i];
                s[j][k] = see ? score_log2(hi[k] + lo[k], x) : -INFINITY;
            }
        }

        if constexpr (WEIGHTS) {
            if (page) {
                // log2 of every unit's sum, on its own maximum
                const int per = d.unit >> 3;               // n-tiles of 8 tokens per unit
                for (int u0 = 0; u0 < 8; u0 += per)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float um = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j >= u0 && j < u0 + per)
                                um = fmaxf(um, fmaxf(s[j][2 * i], s[j][2 * i + 1]));
                        um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 1));
                        um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 2));
                        float us = 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j >= u0 && j < u0 + per && um > -INFINITY)
                                us += ex2(s[j][2 * i] - um) + ex2(s[j][2 * i + 1] - um);
                        us += __shfl_xor_sync(0xffffffffu, us, 1);
                        us += __shfl_xor_sync(0xffffffffu, us, 2);
                        const int unit = base / d.unit + u0 / per;
                        if (qc == 0 && row[i] < rows && row[i] - d.row0 < d.rows && 8 * u0 < count)
                            d.ls[((int64_t)p * d.rows + row[i] - d.row0) * d.units + unit] = um + log2f(us);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float tm = m[i];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tm = fmaxf(tm, fmaxf(s[j][2 * i], s[j][2 * i + 1]));
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
            const float base_m = tm == -INFINITY ? 0.0f : tm;   // a row that sees nothing yet
            const float alpha = ex2(m[i] - base_m);
            m[i] = tm;
            l[i] *= alpha;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 2 * i; k < 2 * i + 2; ++k) {
                    s[j][k] = ex2(s[j][k] - base_m);
                    l[i] += s[j][k];
                }
            if constexpr (!WEIGHTS) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    o[j][2 * i] *= alpha;
                    o[j][2 * i + 1] *= alpha;
                }
            }
        }
        if constexpr (!WEIGHTS) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const uint32_t pa[4] = {pack_sat(s[2 * ks][0], s[2 * ks][1]), pack_sat(s[2 * ks][2], s[2 * ks][3]),
                                        pack_sat(s[2 * ks + 1][0], s[2 * ks + 1][1]),
                                        pack_sat(s[2 * ks + 1][2], s[2 * ks + 1][3])};
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    uint32_t vb[4];
                    ldsm_x4_trans(smem_addr(sv) + (uint32_t)((16 * ks + (lane & 15)) * kStride + 8 * j +
                                                            8 * (lane >> 4)) * 2, vb);
                    mma16816(o[j], pa, vb[0], vb[1]);
                    mma16816(o[j + 1], pa, vb[2], vb[3]);
                }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (row[i] >= rows)
            continue;
        if constexpr (WEIGHTS) {
            if (qc == 0 && row[i] - d.row0 < d.rows)
                d.ml[((int64_t)p * d.rows + row[i] - d.row0) * d.S + blockIdx.x] = make_float2(m[i], l[i]);
        } else {
            const int hh = row[i] - tok[i] * c.g;
            const int64_t at = (int64_t)(first + tok[i]) * (c.Hkv * c.g) + h * c.g + hh;
            if (d.S == 1) {
                const float inv = l[i] > 0.0f ? 1.0f / l[i] : 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    *reinterpret_cast<uint32_t *>(d.out + at * D + 8 * j + 2 * qc) =
                        pack_sat(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
            } else {
                const int64_t part = ((int64_t)p * d.rows + row[i]) * d.S + blockIdx.x;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    *reinterpret_cast<float2 *>(d.o + part * D + 8 * j + 2 * qc) =
                        make_float2(o[j][2 * i], o[j][2 * i + 1]);
                if (qc == 0)
                    d.ml[part] = make_float2(m[i], l[i]);
            }
        }
    }
}

// Joins the splits of the attention: a warp per query row, four channels a lane.
__global__ void __launch_bounds__(128) join_kernel(PagedArgs c, ChunkArgs x, Parts d, __half *out)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = d.pair0 + blockIdx.y, b = p / c.Hkv, h = p % c.Hkv;
    int first, T;
    PagedState st;
    if (!sequence(c, x, b, first, T, st))
        return;
    const int row = blockIdx.x * 4 + warp;
    if (row >= T * c.g)
        return;
    const int64_t at = (int64_t)(first + row / c.g) * (c.Hkv * c.g) + h * c.g + row % c.g;
    const int64_t part = ((int64_t)blockIdx.y * d.rows + row) * d.parts;
    float M = -INFINITY, L = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < d.parts; ++i)
        M = fmaxf(M, d.m[(part + i) * d.step]);
    for (int i = 0; i < d.parts; ++i) {
        const float l = d.l[(part + i) * d.step];
        if (!(l > 0.0f))
            continue;
        const float w = ex2(d.m[(part + i) * d.step] - M);
        const float4 v = *reinterpret_cast<const float4 *>(d.o + (part + i) * kHeadDim + 4 * lane);
        L = fmaf(l, w, L);
        O.x = fmaf(v.x, w, O.x);
        O.y = fmaf(v.y, w, O.y);
        O.z = fmaf(v.z, w, O.z);
        O.w = fmaf(v.w, w, O.w);
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    *reinterpret_cast<uint2 *>(out + at * kHeadDim + 4 * lane) =
        make_uint2(pack_sat(O.x * inv, O.y * inv), pack_sat(O.z * inv, O.w * inv));
}

// Adds a page's share of every row: a thread per page, the rows in order.
__global__ void __launch_bounds__(128) weigh_kernel(PagedArgs c, ChunkArgs x, Parts d, const float *page_sums,
                                                    int unit, int units, float *weights)
{
    __shared__ float lse[128];
    const int p = blockIdx.y, b = p / c.Hkv;
    int first, T;
    PagedState st;
    if (!sequence(c, x, b, first, T, st))
        return;
    const int rows = min(d.rows, T * c.g - d.row0);
    const int col = blockIdx.x * 128 + threadIdx.x;
    if (blockIdx.x * 128 >= st.held || rows <= 0)
        return;
    const int per = c.G / unit;
    float sum = 0.0f;
    for (int r0 = 0; r0 < rows; r0 += 128) {
        __syncthreads();
        if (r0 + threadIdx.x < rows) {
            const int64_t part = ((int64_t)p * d.rows + r0 + threadIdx.x) * d.parts;
            float M = -INFINITY, L = 0.0f;
            for (int i = 0; i < d.parts; ++i)
                M = fmaxf(M, d.m[(part + i) * d.step]);
            for (int i = 0; i < d.parts; ++i) {
                const float l = d.l[(part + i) * d.step];
                if (l > 0.0f)
                    L = fmaf(l, ex2(d.m[(part + i) * d.step] - M), L);
            }
            lse[threadIdx.x] = M + log2f(L);
        }
        __syncthreads();
        if (col < st.held)
            for (int r = 0; r < min(128, rows - r0); ++r) {
                const float *ls = page_sums + ((int64_t)p * d.rows + r0 + r) * units + (int64_t)col * per;
                for (int k = 0; k < per; ++k)
                    sum += ex2(ls[k] - lse[r]);
            }
    }
    if (col < st.held)
        weights[(int64_t)p * c.columns + col] += sum;
}

template <bool W>
void launch_attend(const PagedArgs &c, const ChunkArgs &x, const SplitOut &d, dim3 grid, cudaStream_t s)
{
    if (c.fmt == KIVI_FP8_E4M3)
        attend_kernel<PageFmt<8, 0, KIVI_FP8_E4M3>, W><<<grid, kAttendThreads, 0, s>>>(c, x, d);
    else if (c.fmt == KIVI_FP8_E5M2)
        attend_kernel<PageFmt<8, 0, KIVI_FP8_E5M2>, W><<<grid, kAttendThreads, 0, s>>>(c, x, d);
    else if (c.bits == 2 && !c.meta)
        attend_kernel<PageFmt<2, 0, 0>, W><<<grid, kAttendThreads, 0, s>>>(c, x, d);
    else if (c.bits == 2)
        attend_kernel<PageFmt<2, 1, 0>, W><<<grid, kAttendThreads, 0, s>>>(c, x, d);
    else if (!c.meta)
        attend_kernel<PageFmt<4, 0, 0>, W><<<grid, kAttendThreads, 0, s>>>(c, x, d);
    else
        attend_kernel<PageFmt<4, 1, 0>, W><<<grid, kAttendThreads, 0, s>>>(c, x, d);
}

// Splits that fill the GPU: the blocks of one split are `blocks`, and no split
// is shorter than two tiles of the longest sequence.
int split_count(int64_t blocks, int max_new, int max_cached)
{
    const int64_t tiles = ((int64_t)max_cached + max_new + kTile - 1) / kTile;
    return (int)std::max<int64_t>(1, std::min((kTargetBlocks + blocks - 1) / blocks, tiles / 2));
}

constexpr int64_t kWeighBytes = 256ll << 20;     // rows of page sums held at once

// ------------------------------------------------------------------- plans ---
// Few query rows per pair: the decode kernel (kivi_paged_decode.cuh), which
// streams the packed codes into the matrix instructions.  It takes 4 or 8 rows
// and reads the pages again for the next 8.  Groups of 16 tokens it does not
// know.
constexpr int kFewRows = 8;
constexpr int kDecodeBlocks = 4096;              // (pair, row tile, split) blocks of it that the workspace is sized for

bool few_rows(const PagedArgs &c, int max_new) { return c.G >= 32 && (int64_t)max_new * c.g <= kFewRows; }

struct Plan {
    int splits;           // parts of a pair's tokens
    int row_tiles;        // tiles of query rows of the longest chunk, or of one launch
};

Plan attend_plan(const PagedArgs &c, int max_new, int max_cached)
{
    const int64_t pairs = (int64_t)c.B * c.Hkv;
    Plan p;
    p.row_tiles = (int)(((int64_t)max_new * c.g + kTile - 1) / kTile);
    p.splits = split_count(pairs * p.row_tiles, max_new, max_cached);
    return p;
}

int weigh_unit(const PagedArgs &c) { return std::min(c.G, kTile); }

Plan weights_plan(const PagedArgs &c, int max_new, int max_cached)
{
    const int64_t pairs = (int64_t)c.B * c.Hkv;
    const int64_t units = (int64_t)c.columns * c.G / weigh_unit(c);
    const int64_t all = ((int64_t)max_new * c.g + kTile - 1) / kTile;
    Plan p;
    p.row_tiles = (int)std::max<int64_t>(1, std::min(all, kWeighBytes / (pairs * kTile * units * 4)));
    p.splits = split_count(pairs * p.row_tiles, max_new, max_cached);
    return p;
}

cudaError_t paged_decode(const PagedDecodeArgs &a, bool weights, int pairs, cudaStream_t s, int *blocks_per_sm)
{
    const int gq = a.rows <= 4 ? 4 : 8;
    if (a.c.fmt)
        return launch_paged_decode_fp8(a, gq, weights, pairs, s, blocks_per_sm);
    if (a.c.bits == 2)
        return a.c.meta ? launch_paged_decode_2_f16(a, gq, weights, pairs, s, blocks_per_sm)
                        : launch_paged_decode_2(a, gq, weights, pairs, s, blocks_per_sm);
    return a.c.meta ? launch_paged_decode_4_f16(a, gq, weights, pairs, s, blocks_per_sm)
                    : launch_paged_decode_4(a, gq, weights, pairs, s, blocks_per_sm);
}

// Query rows the partial results of a decode launch have room for.
int few_room(const PagedArgs &c, int max_new)
{
    const int rows = max_new * c.g;
    return rows <= 4 ? 4 : (rows + 7) / 8 * 8;
}

// Splits of a decode launch: the count with the smallest waves x (fixed cost +
// chunks per block) for the blocks the GPU holds at once -- the cost model of
// kivi_decode_num_splits, for the longest sequence the bounds allow.
cudaError_t few_splits(const PagedDecodeArgs &a, bool weights, int64_t blocks, int max_cached, int *splits)
{
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = paged_decode(a, weights, 0, nullptr, &per_sm);
    if (e != cudaSuccess)
        return e;
    const int64_t resident = (int64_t)std::max(per_sm, 1) * sms;
    const int64_t chunks = std::max<int64_t>(1, ((int64_t)max_cached + kChunk - 1) / kChunk);
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kDecodeBlocks / blocks, chunks));
    int64_t best = INT64_MAX;
    *splits = 1;
    for (int64_t k = 1; k <= most; ++k) {
        const int64_t cost = (blocks * k + resident - 1) / resident * (12 + (chunks + k - 1) / k);
        if (cost < best) {
            best = cost;
            *splits = (int)k;
        }
    }
    return cudaSuccess;
}

PagedDecodeArgs decode_args_of(const PagedArgs &c, const ChunkArgs &x, int rows)
{
    PagedDecodeArgs a{};
    a.c = c;
    a.x = x;
    a.rows = rows;
    a.cap_log2_inv = x.cap_log2 != 0.0f ? 1.0f / x.cap_log2 : 0.0f;
    a.d.kr = c.k_fp16;
    a.d.vr = c.v_fp16;
    a.d.status = c.control;
    a.d.Ns = c.Ns;
    a.d.R = c.R;
    a.d.rows = c.rows;
    a.d.Hkv = c.Hkv;
    a.d.scale_log2 = x.scale_log2;
    a.d.fp8_k_scale = c.fp8_k_scale;
    a.d.fp8_v_scale = c.fp8_v_scale;
    return a;
}

// Partial results of a decode launch in the workspace: o (attention), m, l.
size_t few_parts(PagedDecodeArgs &a, int64_t pairs, bool weights, void *ws)
{
    const int64_t n = pairs * a.rows * (a.d.S + 1);
    a.d.ws_o = static_cast<float *>(ws);
    a.d.ws_m = a.d.ws_o + (weights ? 0 : n * kHeadDim);
    a.d.ws_l = a.d.ws_m + n;
    return (size_t)n * ((weights ? 0 : kHeadDim) + 2) * 4;
}

// splits * blocks <= max(kDecodeBlocks, blocks), and one more part per row
size_t few_bytes(const PagedArgs &c, int max_new, bool weights)
{
    const int rows = few_room(c, max_new), gq = rows <= 4 ? 4 : 8;
    const int64_t blocks = (int64_t)c.B * c.Hkv * (rows / gq);
    return (size_t)(std::max<int64_t>(kDecodeBlocks, blocks) + blocks) * gq * ((weights ? 0 : kHeadDim) + 2) * 4;
}

}  // namespace

cudaError_t launch_join(const PagedArgs &c, const ChunkArgs &x, const Parts &d, __half *out, int pairs, cudaStream_t s)
{
    join_kernel<<<dim3((unsigned)(((int64_t)x.max_new * c.g + 3) / 4), pairs), 128, 0, s>>>(c, x, d, out);
    return cudaGetLastError();
}

size_t attention_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    // splits * blocks < blocks + target, and more blocks than that mean one split
    const int64_t blocks = std::min<int64_t>((int64_t)c.B * c.Hkv * attend_plan(c, max_new, max_cached).row_tiles,
                                             kTargetBlocks);
    const size_t tiles = (size_t)(kTile * (blocks + kTargetBlocks)) * (kHeadDim + 2) * 4;
    const int few = std::min(max_new, std::max(1, kFewRows / c.g));       // the longest chunk of few rows
    return std::max(tiles, few_bytes(c, few, false));
}

size_t weights_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    const int64_t pairs = (int64_t)c.B * c.Hkv;
    const int64_t units = (int64_t)c.columns * c.G / weigh_unit(c);
    const int64_t tiles = pairs * weights_plan(c, max_new, max_cached).row_tiles;
    const size_t all = (size_t)tiles * kTile * units * 4 + (size_t)kTile * (tiles + kTargetBlocks) * 8;
    const int few = std::min(max_new, std::max(1, kFewRows / c.g));
    const size_t sums = (size_t)pairs * few_room(c, few) * ((size_t)c.columns * c.G / decode_unit(c)) * 4;
    return std::max(all, few_bytes(c, few, true) + sums);
}

cudaError_t launch_paged_attention(const PagedArgs &c, const ChunkArgs &x, __half *out, void *ws, cudaStream_t s,
                                   int *launches)
{
    if (is_long_chunk(c, x.max_new))
        return launch_long_chunk(c, x, out, ws, s, launches);
    const int pairs = c.B * c.Hkv;
    if (few_rows(c, x.max_new)) {
        PagedDecodeArgs a = decode_args_of(c, x, few_room(c, x.max_new));
        const int64_t blocks = (int64_t)pairs * (a.rows <= 4 ? 1 : a.rows / 8);
        cudaError_t e = few_splits(a, false, blocks, x.max_cached, &a.d.S);
        if (e != cudaSuccess)
            return e;
        few_parts(a, pairs, false, ws);
        e = paged_decode(a, false, pairs, s, nullptr);
        if (e != cudaSuccess)
            return e;
        *launches = 2;
        return launch_join(c, x, Parts{a.d.ws_m, a.d.ws_l, a.d.ws_o, 1, a.d.S + 1, 0, 0, a.rows}, out, pairs, s);
    }
    const Plan p = attend_plan(c, x.max_new, x.max_cached);
    SplitOut d{};
    d.out = out;
    d.S = p.splits;
    d.rows = p.row_tiles * kTile;
    d.o = static_cast<float *>(ws);
    d.ml = reinterpret_cast<float2 *>(d.o + (int64_t)pairs * d.rows * p.splits * kHeadDim);
    launch_attend<false>(c, x, d, dim3(p.splits, pairs, p.row_tiles), s);
    *launches = 1;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1)
        return e;
    *launches = 2;
    const float *ml = reinterpret_cast<const float *>(d.ml);
    return launch_join(c, x, Parts{ml, ml + 1, d.o, 2, p.splits, 0, 0, d.rows}, out, pairs, s);
}

cudaError_t launch_paged_weights(const PagedArgs &c, const ChunkArgs &x, float *weights, void *ws, cudaStream_t s,
                                 int *launches)
{
    const int pairs = c.B * c.Hkv;
    const dim3 grid((c.columns + 127) / 128, pairs);
    if (few_rows(c, x.max_new)) {
        PagedDecodeArgs a = decode_args_of(c, x, few_room(c, x.max_new));
        const int64_t blocks = (int64_t)pairs * (a.rows <= 4 ? 1 : a.rows / 8);
        cudaError_t e = few_splits(a, true, blocks, x.max_cached, &a.d.S);
        if (e != cudaSuccess)
            return e;
        const int unit = decode_unit(c);
        a.units = c.columns * c.G / unit;
        a.ls = reinterpret_cast<float *>(static_cast<char *>(ws) + few_parts(a, pairs, true, ws));
        e = paged_decode(a, true, pairs, s, nullptr);
        if (e != cudaSuccess)
            return e;
        weigh_kernel<<<grid, 128, 0, s>>>(c, x, Parts{a.d.ws_m, a.d.ws_l, nullptr, 1, a.d.S + 1, 0, 0, a.rows}, a.ls,
                                          unit, a.units, weights);
        *launches = 2;
        return cudaGetLastError();
    }
    const Plan p = weights_plan(c, x.max_new, x.max_cached);
    SplitOut d{};
    d.S = p.splits;
    d.unit = weigh_unit(c);
    d.units = c.columns * c.G / d.unit;
    d.rows = p.row_tiles * kTile;
    d.ls = static_cast<float *>(ws);
    d.ml = reinterpret_cast<float2 *>(d.ls + (int64_t)pairs * d.rows * d.units);
    const float *ml = reinterpret_cast<const float *>(d.ml);
    *launches = 0;
    for (int64_t r0 = 0; r0 < (int64_t)x.max_new * c.g; r0 += d.rows) {
        d.row0 = (int)r0;
        launch_attend<true>(c, x, d, dim3(p.splits, pairs, p.row_tiles), s);
        weigh_kernel<<<grid, 128, 0, s>>>(c, x, Parts{ml, ml + 1, nullptr, 2, p.splits, 0, d.row0, d.rows}, d.ls, d.unit,
                                          d.units, weights);
        *launches += 2;
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace kivi
