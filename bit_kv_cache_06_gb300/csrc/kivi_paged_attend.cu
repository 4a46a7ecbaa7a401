// kivi_paged_attend.cu -- which kernel an attention or a page-weights call over
// a paged cache takes, and the joins of the parts.
//
//  query rows per pair      kernel
//  up to most_few_rows()    decode kernel (kivi_decode_kernels.cuh), G >= 32
//  more, or G = 16          tcgen05 kernels (kivi_paged_tc.cu)
//
// The parts of a row join as o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,
// M = max_i m_i.
#include <algorithm>
#include <atomic>

#include "kivi_paged_attend.cuh"
#include "kivi_paged_decode.cuh"

namespace kivi {
namespace {

// Joins the splits of the attention: a warp per query row, four channels a lane.
// Latency: 7 us for 256 rows of 8 parts, from cold caches.
__global__ void __launch_bounds__(128) join_kernel(PagedArgs c, ChunkArgs x, Parts d, __half *out)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = d.pair0 + blockIdx.y, b = p / c.Hkv, h = p % c.Hkv;
    int first, T;
    PagedState st;
    const bool some = sequence(c, x, b, first, T, st);
    wait_for_previous();
    const int row = blockIdx.x * 4 + warp;
    if (!some || row >= T * c.g)
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

// Adds a page's share of every row.  A block takes PAGES pages, and 256 / PAGES
// rows at a time; a thread adds up its rows in order, and the threads' sums are
// added in order: equal inputs give equal bits.  Latency: 12 us for 64 rows of 1024
// pages and 4 query rows, 10 us for 16 of 256 and 128 query rows.
constexpr int kWeighRows = 256;        // rows whose normalisers a block holds at once
constexpr int kAhead = 8;              // parts loaded at once

template <int PAGES>
__global__ void __launch_bounds__(256) weigh_kernel(PagedArgs c, ChunkArgs x, Parts d, const float *page_sums, int unit,
                                                    int units, float *weights)
{
    constexpr int LANES = 256 / PAGES;
    __shared__ float lse[kWeighRows], sums[LANES][PAGES];
    const int p = d.pair0 + blockIdx.y, b = p / c.Hkv, at = threadIdx.x % PAGES, lane = threadIdx.x / PAGES;
    int first, T;
    PagedState st;
    const bool some = sequence(c, x, b, first, T, st);
    let_next_in();
    wait_for_previous();
    if (!some)
        return;
    const int rows = min(d.rows, T * c.g - d.row0);
    const int col = blockIdx.x * PAGES + at;
    if (blockIdx.x * PAGES >= st.held || rows <= 0)
        return;
    const int per = c.G / unit;
    float sum = 0.0f;
    for (int r0 = 0; r0 < rows; r0 += kWeighRows) {
        __syncthreads();
        if (r0 + threadIdx.x < rows) {
            const int64_t part = ((int64_t)blockIdx.y * d.rows + r0 + threadIdx.x) * d.parts;
            float M = -INFINITY, L = 0.0f;
            for (int i0 = 0; i0 < d.parts; i0 += kAhead) {
                float m[kAhead], l[kAhead], M1 = M;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const bool in = i0 + k < d.parts;
                    m[k] = in ? d.m[(part + i0 + k) * d.step] : -INFINITY;
                    l[k] = in ? d.l[(part + i0 + k) * d.step] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    M1 = fmaxf(M1, m[k]);
                if (L > 0.0f)
                    L *= ex2(M - M1);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (l[k] > 0.0f)
                        L = fmaf(l[k], ex2(m[k] - M1), L);
                M = M1;
            }
            lse[threadIdx.x] = M + log2f(L);
        }
        __syncthreads();
        if (col < st.held) {
            const float *ls = page_sums + ((int64_t)blockIdx.y * d.rows + r0) * units + (int64_t)col * per;
#pragma unroll 4
            for (int r = lane; r < min(kWeighRows, rows - r0); r += LANES)
                for (int k = 0; k < per; ++k)
                    sum += ex2(ls[(int64_t)r * units + k] - lse[r]);
        }
    }
    sums[lane][at] = sum;
    __syncthreads();
    if (lane == 0 && col < st.held) {
        for (int i = 1; i < LANES; ++i)
            sum += sums[i][at];
        weights[(int64_t)p * c.columns + col] += sum;
    }
}

// ------------------------------------------------------------------- plans ---
// Few query rows per pair: the decode kernel (kivi_paged_decode.cuh), which
// streams the packed codes into the matrix instructions.  It takes 4 or 8 rows
// and reads the pages again for the next 8; the tcgen05 kernels dequantise them
// once, for any number of rows.  Where the two meet (us, decode kernel against
// tcgen05; 32 sequences of up to 8k tokens and 4-bit pages for attention, eight
// of up to 32k and 2-bit pages for weights; FP8: 4 of 16k with 8 heads a kv
// head, and eight of 32k):
//                  8 rows     16         24         32         64         96
//  attention, code                                  319 / 513  492 / 517  713 / 523
//  attention, FP8  64 / 146   114 / 150  140 / 150  186 / 150
//  weights, code                                    249 / 497  415 / 508  589 / 514
//  weights, FP8    171 / 265  314 / 266
// Groups of 16 tokens the decode kernel does not know.
int most_few_rows(const PagedArgs &c, bool weights) { return !c.fmt ? 64 : weights ? 8 : 24; }
constexpr int kDecodeBlocks = 4096;              // (pair, row tile, split) blocks of it that the workspace is sized for

bool few_rows(const PagedArgs &c, int max_new, bool weights)
{
    return c.G >= 32 && (int64_t)max_new * c.g <= most_few_rows(c, weights);
}

// the longest chunk of few rows, max_new at most
int few_new(const PagedArgs &c, int max_new, bool weights)
{
    return std::min(max_new, std::max(1, most_few_rows(c, weights) / c.g));
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

// Blocks of a decode kernel that the current device holds at once; asked once
// per device and kernel.
cudaError_t resident_blocks(const PagedDecodeArgs &a, bool weights, int *blocks)
{
    static std::atomic<int> known[64][128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const PagedArgs &c = a.c;
    const int kind = c.fmt ? c.fmt - 1 : 2 + (c.bits == 4) * 2 + c.meta;             // 0 .. 5
    const int kernel = ((kind * 4 + (c.G == 64 ? 1 : c.G == 128 ? 2 : 0)) * 2 + (a.rows > 4)) * 2 + weights;
    std::atomic<int> *slot = dev < 64 ? &known[dev][kernel] : nullptr;
    *blocks = slot ? slot->load(std::memory_order_relaxed) : 0;
    if (*blocks > 0)
        return cudaSuccess;
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = paged_decode(a, weights, 0, nullptr, &per_sm);
    if (e != cudaSuccess)
        return e;
    *blocks = std::max(per_sm, 1) * sms;
    if (slot)
        slot->store(*blocks, std::memory_order_relaxed);
    return cudaSuccess;
}

// Splits of a decode launch: the count with the smallest waves x (fixed cost +
// chunks per block) for the blocks the GPU holds at once -- the cost model of
// kivi_decode_num_splits, for the longest sequence the bounds allow.
cudaError_t few_splits(const PagedDecodeArgs &a, bool weights, int64_t blocks, int max_cached, int *splits)
{
    int resident = 0;
    const cudaError_t e = resident_blocks(a, weights, &resident);
    if (e != cudaSuccess)
        return e;
    const int64_t chunks = std::max<int64_t>(1, ((int64_t)max_cached + kChunk - 1) / kChunk);
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kDecodeBlocks / blocks, chunks));
    int64_t best = INT64_MAX;
    *splits = 1;
    for (int64_t waves = (blocks + resident - 1) / resident; waves * 13 < best; ++waves) {
        // the most splits that these waves hold, and of those with as many chunks per block the fewest
        const int64_t room = std::max<int64_t>(1, std::min(most, waves * resident / blocks));
        const int64_t per = (chunks + room - 1) / room, k = (chunks + per - 1) / per;
        const int64_t cost = (blocks * k + resident - 1) / resident * (12 + per);
        if (cost < best) {
            best = cost;
            *splits = (int)k;
        }
        if (room == most)
            break;
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
    return launch_dependent(join_kernel, dim3((unsigned)(((int64_t)x.max_new * c.g + 3) / 4), pairs), 128, 0, s, c, x, d, out);
}

cudaError_t launch_weigh(const PagedArgs &c, const ChunkArgs &x, const Parts &d, const float *ls, int unit, int units,
                         float *weights, int pairs, cudaStream_t s)
{
    // 8 pages a block where blocks of 32 would leave SMs idle: two sequences of up to 16k tokens, 128 rows a pair, the call 85 us
    // against 94; eight of 32k, 32 rows, where they do not: 266 against 247, as each block works out the normalisers.
    const int wide = (c.columns + 31) / 32;
    if ((int64_t)wide * pairs >= 512)
        return launch_dependent(weigh_kernel<32>, dim3(wide, pairs), 256, 0, s, c, x, d, ls, unit, units, weights);
    return launch_dependent(weigh_kernel<8>, dim3((c.columns + 7) / 8, pairs), 256, 0, s, c, x, d, ls, unit, units, weights);
}

// The bounds below only grow with max_new and max_cached.
size_t attention_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    const size_t bytes = few_bytes(c, few_new(c, max_new, false), false);
    return few_rows(c, max_new, false) ? bytes : std::max(bytes, long_attention_bytes(c, max_new, max_cached));
}

size_t weights_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    const int few = few_new(c, max_new, true);
    const size_t sums = (size_t)c.B * c.Hkv * few_room(c, few) * ((size_t)c.columns * c.G / decode_unit(c)) * 4;
    const size_t bytes = few_bytes(c, few, true) + sums;
    return few_rows(c, max_new, true) ? bytes : std::max(bytes, long_weights_bytes(c, max_new, max_cached));
}

cudaError_t launch_paged_attention(const PagedArgs &c, const ChunkArgs &x, __half *out, void *ws, cudaStream_t s,
                                   int *launches)
{
    *launches = 0;
    if (!few_rows(c, x.max_new, false))
        return launch_long_attention(c, x, out, ws, s, launches);
    const int pairs = c.B * c.Hkv;
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

cudaError_t launch_paged_weights(const PagedArgs &c, const ChunkArgs &x, float *weights, void *ws, cudaStream_t s,
                                 int *launches)
{
    *launches = 0;
    if (!few_rows(c, x.max_new, true))
        return launch_long_weights(c, x, weights, ws, s, launches);
    const int pairs = c.B * c.Hkv, unit = decode_unit(c);
    PagedDecodeArgs a = decode_args_of(c, x, few_room(c, x.max_new));
    const int64_t blocks = (int64_t)pairs * (a.rows <= 4 ? 1 : a.rows / 8);
    cudaError_t e = few_splits(a, true, blocks, x.max_cached, &a.d.S);
    if (e != cudaSuccess)
        return e;
    a.units = c.columns * c.G / unit;
    a.ls = reinterpret_cast<float *>(static_cast<char *>(ws) + few_parts(a, pairs, true, ws));
    e = paged_decode(a, true, pairs, s, nullptr);
    if (e != cudaSuccess)
        return e;
    *launches = 2;
    return launch_weigh(c, x, Parts{a.d.ws_m, a.d.ws_l, nullptr, 1, a.d.S + 1, 0, 0, a.rows}, a.ls, unit, a.units, weights,
                        pairs, s);
}

}  // namespace kivi
