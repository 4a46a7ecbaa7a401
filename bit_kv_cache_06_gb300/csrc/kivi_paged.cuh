// kivi_paged.cuh -- what the kernels of the paged cache share: argument
// blocks, the state of a sequence as it follows from its token count, and the
// checks of everything that only the device can see (include/kivi.h, "paged
// cache").
#pragma once

#include "kivi_internal.cuh"

namespace kivi {

struct PagedArgs {
    uint8_t *pool;
    __half *k_fp16, *v_fp16;          // [P][rows][D]
    int32_t *table;                   // [P][columns]
    int32_t *n_tokens, *n_evicted;    // [B]
    unsigned *control;                // status word, then a counter per sequence
    int64_t num_pages;
    int columns;
    int rec_bytes;
    int bits, fmt, meta, G, flush_group;
    int R, Ns, rows;
    int B, Hkv, g;                    // g = query heads per kv head
    float fp8_k_scale, fp8_v_scale;
};

struct ChunkArgs {
    const __half *q, *k, *v;
    const int32_t *offsets;           // [B + 1]
    int64_t q_stride, kv_stride;      // halves from token to token
    int64_t num_tokens;
    int max_new, max_cached;          // bounds of one sequence's new and cached tokens
    float scale_log2;                 // softmax scale * log2(e)
    float cap_log2, cap_inv;          // cap * log2(e) and scale / cap; cap_log2 = 0: no cap
    int cap_small;                    // cap below 64: an error of 2^-22 of it does not show
    int full;                         // every new token sees all of its sequence's
    int v8;                           // k, v rows and the fp16 rows 32-byte aligned
};

// Sequence b as its token count says.
struct PagedState {
    int n;            // tokens seen
    int sink;         // of them in the sink rows
    int flushed;      // key groups quantised so far (held and evicted)
    int held;         // pages held: table columns 0 .. held - 1
    int window;       // tokens in the ring
    int head;         // slot of the oldest of them
};

__device__ __forceinline__ int flushed_groups(const PagedArgs &c, int n)
{
    const int m = n - c.Ns;
    if (c.flush_group)
        return m > c.R ? (m - c.R + c.G - 1) / c.G : 0;
    return m > 0 ? (m - 1) / c.R * (c.R / c.G) : 0;
}

// False when the lengths do not fit the table.
__device__ __forceinline__ bool paged_state(const PagedArgs &c, int b, PagedState &s)
{
    s.n = c.n_tokens[b];
    const int gone = c.n_evicted[b];
    if (s.n < 0 || gone < 0)
        return false;
    s.sink = min(s.n, c.Ns);
    s.flushed = flushed_groups(c, s.n);
    s.held = s.flushed - gone;
    s.window = s.n - s.sink - s.flushed * c.G;
    s.head = (int)((int64_t)s.flushed * c.G % c.R);
    return s.held >= 0 && s.held <= c.columns;
}

// New tokens first .. first + T - 1 of sequence b; false when the offsets are
// not what the header asks for.
__device__ __forceinline__ bool chunk_of(const ChunkArgs &x, int b, int &first, int &T)
{
    const int lo = x.offsets[b], hi = x.offsets[b + 1];
    if (lo < 0 || hi < lo || hi > x.num_tokens || hi - lo > x.max_new)
        return false;
    first = lo;
    T = hi - lo;
    return true;
}

// Sequence b of an attention or a weights call: its new tokens and its state;
// false when the call has to skip it.
__device__ __forceinline__ bool sequence(const PagedArgs &c, const ChunkArgs &x, int b, int &first, int &T,
                                         PagedState &s)
{
    return chunk_of(x, b, first, T) && paged_state(c, b, s) &&
           s.sink + s.held * c.G + s.window <= x.max_cached;
}

// Record in column `col` of pair p, or null when the page number is not one of
// the pool's.
__device__ __forceinline__ unsigned char *page_record(const PagedArgs &c, int p, int col)
{
    const int id = c.table[(int64_t)p * c.columns + col];
    if (id < 0 || id >= c.num_pages)
        return nullptr;
    return c.pool + (int64_t)id * c.rec_bytes;
}

// A kernel that reads what the one before it writes is launched as its
// programmatic dependent: its blocks come in while the earlier ones run and
// wait for the end of that grid and for its writes.  Every block of a dependent
// waits, so a grid's end stands for the end of all before it.
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A... args)
{
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

cudaError_t launch_paged_append(const PagedArgs &c, const ChunkArgs &x, cudaStream_t s, int *launches);

// Workspace bytes, which only grow with max_new and max_cached (both bounds of
// one sequence), and launches that need no more.
size_t attention_bytes(const PagedArgs &c, int max_new, int max_cached);
size_t weights_bytes(const PagedArgs &c, int max_new, int max_cached);
size_t evict_bytes(const PagedArgs &c);

cudaError_t launch_paged_attention(const PagedArgs &c, const ChunkArgs &x, __half *out, void *ws, cudaStream_t s,
                                   int *launches);
cudaError_t launch_paged_weights(const PagedArgs &c, const ChunkArgs &x, float *weights, void *ws, cudaStream_t s,
                                 int *launches);
cudaError_t launch_paged_evict(const PagedArgs &c, float *weights, int budget, int recent, void *ws,
                               cudaStream_t s, int *launches);

// Partial results of the splits: part i of query row r of pair p (the p-th of
// the launch) at index (p rows + r) parts + i, its maximum (log2 units) and sum
// at m, l [index step], its unnormalised output at o[index D].
struct Parts {
    const float *m, *l, *o;
    int step, parts;
    int pair0;                // first pair of the launch
    int row0, rows;           // first query row of the launch, and rows a pair has room for
};

// Joins the parts of launched pairs into out: a warp per query row.
cudaError_t launch_join(const PagedArgs &c, const ChunkArgs &x, const Parts &d, __half *out, int pairs, cudaStream_t s);

// Adds the pages' sums of launched pairs to weights: ls[(p rows + r) units + u]
// holds log2 of the softmax sum of unit u (`unit` tokens) of row r.
cudaError_t launch_weigh(const PagedArgs &c, const ChunkArgs &x, const Parts &d, const float *ls, int unit, int units,
                         float *weights, int pairs, cudaStream_t s);

// Many query rows (kivi_paged_tc.cu).
size_t long_attention_bytes(const PagedArgs &c, int max_new, int max_cached);
bool long_attention_fits(const PagedArgs &c, int max_new, int max_cached);
size_t long_weights_bytes(const PagedArgs &c, int max_new, int max_cached);
cudaError_t launch_long_attention(const PagedArgs &c, const ChunkArgs &x, __half *out, void *ws, cudaStream_t s,
                                  int *launches);
cudaError_t launch_long_weights(const PagedArgs &c, const ChunkArgs &x, float *weights, void *ws, cudaStream_t s,
                                int *launches);

}  // namespace kivi
