// kivi_paged_evict.cu -- eviction of the pages with the least accumulated
// attention weight: a selection over each pair's pages and a stable partition
// of its table row.  Nothing but page numbers and weights moves.
//
// One block per (sequence, kv head) pair.  The weights become 32-bit keys in
// their order; four histogram passes of 8 bits find the key T of the last page
// that stays and how many pages with exactly that key stay (the first ones,
// from the lowest column).  One pass over the row in order then writes the kept
// pages in place, to columns at or before the ones already read, and the
// evicted ones to the workspace, from which they follow behind the kept ones.
#include "kivi_paged.cuh"

namespace kivi {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kWarps = kEvictThreads / 32;

// Larger weights give larger keys; -0 counts as +0, NaN as the least.
__device__ __forceinline__ unsigned order_key(float w)
{
    if (w != w)
        return 0u;
    const unsigned u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one, and over the whole block.
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

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(PagedArgs c, float *weights, int budget,
                                                              int recent, int32_t *gone_ids)
{
    __shared__ int hist[256];
    __shared__ int warp_sums[kWarps];
    __shared__ unsigned s_prefix;
    __shared__ int s_need;
    const int p = blockIdx.x, b = p / c.Hkv, tid = threadIdx.x;
    PagedState st;
    const bool ok = paged_state(c, b, st);
    const int n = ok ? st.held : 0;
    if (!ok && tid == 0)
        atomicOr(c.control, KIVI_STATUS_BAD_STATE);
    int32_t *row = c.table + (int64_t)p * c.columns;
    float *w = weights + (int64_t)p * c.columns;
    int32_t *gone = gone_ids + (int64_t)p * c.columns;

    if (n > budget) {
        const int fixed = min(recent, budget), cand = n - fixed;
        int need = budget - fixed;          // candidates that stay (fewer than cand)
        // the key of the last one that stays, from its highest byte down
        unsigned prefix = 0u;
        for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
            if (tid < 256)
                hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < cand; i += kEvictThreads) {
                const unsigned k = order_key(w[i]);
                if (shift == 24 || (k ^ prefix) >> (shift + 8) == 0u)
                    atomicAdd(&hist[(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = need, digit = 255;
                while (digit > 0 && hist[digit] < left)
                    left -= hist[digit--];
                s_prefix = prefix | (unsigned)digit << shift;
                s_need = left;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;                  // of the keys with this prefix, this many stay
        }
        const bool none = budget == fixed;  // no candidate stays
        int kept0 = 0, gone0 = 0, equal0 = 0;
        for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
            const int i = i0 + tid;
            const bool in = i < n;
            const int32_t id = in ? row[i] : 0;
            const float wi = in ? w[i] : 0.0f;
            const unsigned k = order_key(wi);
            const bool candidate = i < cand;
            const bool equal = candidate && !none && k == prefix;
            const int2 eq = block_scan(equal, warp_sums);
            const bool keep = in && (!candidate || (!none && (k > prefix || (equal && equal0 + eq.x < need))));
            const int2 kp = block_scan(keep, warp_sums);   // its barriers: every thread has read row and w
            if (keep) {
                row[kept0 + kp.x] = id;
                w[kept0 + kp.x] = wi;
            } else if (in) {
                gone[gone0 + tid - kp.x] = id;
            }
            equal0 += eq.y;
            kept0 += kp.y;
            gone0 += min(kEvictThreads, n - i0) - kp.y;
        }
        __syncthreads();
        for (int i = tid; i < n - budget; i += kEvictThreads) {
            row[budget + i] = gone[i];
            w[budget + i] = 0.0f;
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

size_t evict_bytes(const PagedArgs &c) { return (size_t)c.B * c.Hkv * c.columns * 4; }

cudaError_t launch_paged_evict(const PagedArgs &c, float *weights, int budget, int recent, void *ws,
                               cudaStream_t s, int *launches)
{
    evict_kernel<<<c.B * c.Hkv, kEvictThreads, 0, s>>>(c, weights, budget, recent, static_cast<int32_t *>(ws));
    *launches = 1;
    return cudaGetLastError();
}

}  // namespace kivi
