// kivi_paged_evict.cu -- eviction of the pages with the least accumulated
// attention weight: a selection over each pair's pages and a stable partition
// of its table row.  Nothing but page numbers and weights moves.
//
// One block per (sequence, kv head) pair.  The weights become 32-bit keys in
// their order, kept in shared memory (up to kCached of them; read again from
// memory beyond that).  Three histogram passes of 11, 11 and 10 bits find the
// key T of the last page that stays and how many pages with exactly that key stay
// (the first ones, from the lowest column).  Each warp then owns a run of the
// row: it counts the keys equal to T, then, knowing how many come before its
// run, its kept pages, then writes its pages to their places in a copy of the
// row; the copy goes back when every warp has read its part.
//
// Bound by latency: a row of 1000 pages is 4 KB, and the passes follow one
// another.  64 rows of 1020 pages 11.5 us, 8 rows of 32764 pages 43.5 us (one SM a
// row).  Before the digits were selected by all threads and warps owned runs, the
// calls took 30 and 85 us instead of 17 and 49.
#include <algorithm>

#include "kivi_paged.cuh"

namespace kivi {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopies = 4;             // of the histogram: warps w, w + 4, ... share one
constexpr int kAhead = 8;              // loads in flight per thread
constexpr int kCached = 40960;         // keys in shared memory at most

// Larger weights give larger keys; -0 counts as +0, NaN as the least.
__device__ __forceinline__ unsigned order_key(float w)
{
    if (w != w)
        return 0u;
    const unsigned u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Sums of v over the threads before this one, and over the whole block.
__device__ __forceinline__ int2 block_scan(int v, int *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += up;
    }
    __syncthreads();                       // warp_sums of the scan before are read
    if (lane == 31)
        warp_sums[warp] = incl;
    __syncthreads();
    const int ws = lane < kWarps ? warp_sums[lane] : 0;
    int before = lane < warp ? ws : 0, all = ws;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    return make_int2(before + incl - v, all);
}

struct Moved {
    int32_t id;
    float weight;
};

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(PagedArgs c, float *weights, int budget, int recent,
                                                              Moved *copies, int cached)
{
    extern __shared__ unsigned smem[];
    unsigned *keys = smem;                                   // [cached]
    int *hist = reinterpret_cast<int *>(smem + cached);      // [kCopies][kBins]
    __shared__ int warp_sums[kWarps];
    __shared__ unsigned s_prefix;
    __shared__ int s_need;
    const int p = blockIdx.x, b = p / c.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    PagedState st;
    const bool ok = paged_state(c, b, st);
    const int n = ok ? st.held : 0;
    if (!ok && tid == 0)
        atomicOr(c.control, KIVI_STATUS_BAD_STATE);

    if (n > budget) {
        int32_t *row = c.table + (int64_t)p * c.columns;
        float *w = weights + (int64_t)p * c.columns;
        Moved *copy = copies + (int64_t)p * c.columns;
        const int fixed = min(recent, budget), cand = n - fixed;
        const bool all_cached = n <= cached;
        if (all_cached) {
#pragma unroll 1
            for (int i0 = tid; i0 < n; i0 += kAhead * kEvictThreads) {
                float v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    v[k] = i0 + k * kEvictThreads < n ? w[i0 + k * kEvictThreads] : 0.0f;
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i0 + k * kEvictThreads < n)
                        keys[i0 + k * kEvictThreads] = order_key(v[k]);
            }
        }
        auto key = [&](int i) { return all_cached ? keys[i] : order_key(w[i]); };
        __syncthreads();
        int need = budget - fixed;          // candidates that stay (fewer than cand)
        const bool none = need == 0;
        unsigned prefix = 0u;               // key of the last one that stays, from its highest bits down
        for (int pass = 0; pass < 3 && !none; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 32 : pass == 1 ? 21 : 10;
            const unsigned mask = pass == 2 ? 1023u : 2047u;
            for (int i = tid; i < kCopies * kBins; i += kEvictThreads)
                hist[i] = 0;
            __syncthreads();
            int *mine = hist + (warp % kCopies) * kBins;
#pragma unroll 4
            for (int i = tid; i < cand; i += kEvictThreads) {
                const unsigned k = key(i);
                if (pass == 0 || (k ^ prefix) >> above == 0u)
                    atomicAdd(&mine[(k >> shift) & mask], 1);
            }
            __syncthreads();
            // from the largest digit down: the thread's two, and what lies above them
            const int hi = kBins - 1 - 2 * tid, lo = hi - 1;
            int count[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
                count[0] += hist[k * kBins + hi];
                count[1] += hist[k * kBins + lo];
            }
            int over = block_scan(count[0] + count[1], warp_sums).x;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (over < need && over + count[k] >= need) {
                    s_prefix = prefix | (unsigned)(k ? lo : hi) << shift;
                    s_need = need - over;
                }
                over += count[k];
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;                  // of the keys with this prefix, this many stay
        }
        // this warp's run of columns
        const int per = (n + kWarps - 1) / kWarps, from = min(n, warp * per), to = min(n, from + per);
        int equal = 0;                      // (counts are the same in every lane)
        for (int i = from; i < to; i += 32)
            equal += __popc(__ballot_sync(0xffffffffu, i + lane < min(to, cand) && !none && key(i + lane) == prefix));
        const int equal0 = block_scan(lane == 0 ? equal : 0, warp_sums).x - (lane == 0 ? 0 : equal);
        auto stays = [&](int i, int &seen) {    // column i (any lane's); seen: equal keys before this chunk
            const bool in = i < to, candidate = i < cand;
            const unsigned k = in ? key(i) : 0u;
            const bool same = in && candidate && !none && k == prefix;
            const unsigned votes = __ballot_sync(0xffffffffu, same);
            const int rank = seen + __popc(votes & ((1u << lane) - 1u));
            seen += __popc(votes);
            return in && (!candidate || (!none && (k > prefix || (same && rank < need))));
        };
        int kept = 0, seen = equal0;
        for (int i = from; i < to; i += 32)
            kept += __popc(__ballot_sync(0xffffffffu, stays(i + lane, seen)));
        int kept0 = block_scan(lane == 0 ? kept : 0, warp_sums).x - (lane == 0 ? 0 : kept);
        int gone0 = budget + from - kept0;
        seen = equal0;
#pragma unroll 1
        for (int i0 = from; i0 < to; i0 += 32 * kAhead) {
            Moved m[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + 32 * k + lane;
                m[k] = i < to ? Moved{row[i], w[i]} : Moved{0, 0.0f};
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + 32 * k;
                const bool keep = stays(i + lane, seen);
                const unsigned votes = __ballot_sync(0xffffffffu, keep), below = (1u << lane) - 1u;
                if (i + lane < to) {
                    const int at = keep ? kept0 + __popc(votes & below) : gone0 + __popc(~votes & below);
                    copy[at] = Moved{m[k].id, keep ? m[k].weight : 0.0f};
                }
                kept0 += __popc(votes);
                gone0 += max(0, min(32, to - i)) - __popc(votes);
            }
        }
        __syncthreads();                    // the row is read, the copy written
#pragma unroll 1
        for (int i0 = tid; i0 < n; i0 += kAhead * kEvictThreads) {
            Moved m[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                m[k] = i0 + k * kEvictThreads < n ? copy[i0 + k * kEvictThreads] : Moved{0, 0.0f};
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k * kEvictThreads < n) {
                    row[i0 + k * kEvictThreads] = m[k].id;
                    w[i0 + k * kEvictThreads] = m[k].weight;
                }
        }
    }
    __threadfence();
    __syncthreads();                        // this block has read n_tokens and n_evicted
    if (tid == 0) {
        unsigned *ticket = c.control + 1 + b;
        if (atomicAdd(ticket, 1u) == (unsigned)c.Hkv - 1u) {
            *ticket = 0u;
            if (n > budget)
                c.n_evicted[b] += n - budget;
        }
    }
}

}  // namespace

size_t evict_bytes(const PagedArgs &c) { return (size_t)c.B * c.Hkv * c.columns * sizeof(Moved); }

cudaError_t launch_paged_evict(const PagedArgs &c, float *weights, int budget, int recent, void *ws,
                               cudaStream_t s, int *launches)
{
    const int cached = std::min(c.columns, kCached);
    const int smem = (cached + kCopies * kBins) * 4;
    const cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (kCached + kCopies * kBins) * 4);
    if (e != cudaSuccess)
        return e;
    evict_kernel<<<c.B * c.Hkv, kEvictThreads, smem, s>>>(c, weights, budget, recent, static_cast<Moved *>(ws), cached);
    *launches = 1;
    return cudaGetLastError();
}

}  // namespace kivi
