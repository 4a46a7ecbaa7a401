// kivi_paged_decode.cuh -- what the decode kernel needs to know of a paged
// cache: its argument block, and the few places where the two kinds of
// argument differ.  What it does and what bounds it (instruction issue) stands in
// kivi_decode_kernels.cuh.  Measured over pages: eight sequences of up to 32768
// tokens, 8 kv heads of 4 query heads, 2-bit: 60 us for 213 MB (3.5 TB/s; the
// contiguous cache of 32768 tokens each: 59 us for 268 MB -- the longest
// sequence's blocks set the time); 32 sequences of up to 8192 tokens, 32 query
// rows in four passes, 4-bit: 322 us.
#pragma once

#include "kivi_paged_attend.cuh"

namespace kivi {

struct PagedDecodeArgs {
    DecodeArgs d;         // split count, scale, partial results; the rest is filled in per block
    PagedArgs c;
    ChunkArgs x;
    float cap_log2_inv;   // 1 / (c log2 e), 0 without a cap
    float *ls;            // weights: [P][rows][units] log2 of a unit's softmax sum
    int units;            // units per row: 32 tokens each, 16 with FP8
    int row0;             // first query row of this launch
    int rows;             // query rows a pair has room for in the partial results
};

// Tokens per unit of the decode kernel's page sums.
inline int decode_unit(const PagedArgs &c) { return c.fmt ? 16 : 32; }

// The decode kernel over a paged cache for query rows row0 .. row0 + rows - 1
// of every pair: its partial results (weights: its page sums too).
// blocks_per_sm set: occupancy query only.  Groups of 32 tokens or more.
#define KIVI_PAGED_DECODE(name) \
    cudaError_t name(const PagedDecodeArgs &a, int gq, bool weights, int pairs, cudaStream_t s, int *blocks_per_sm)
KIVI_PAGED_DECODE(launch_paged_decode_2);
KIVI_PAGED_DECODE(launch_paged_decode_2_f16);
KIVI_PAGED_DECODE(launch_paged_decode_4);
KIVI_PAGED_DECODE(launch_paged_decode_4_f16);
KIVI_PAGED_DECODE(launch_paged_decode_fp8);
#undef KIVI_PAGED_DECODE

namespace {

__device__ __forceinline__ const DecodeArgs &decode_args(const DecodeArgs &arg, const DecodeArgs &) { return arg; }
__device__ __forceinline__ const DecodeArgs &decode_args(const PagedDecodeArgs &, const DecodeArgs &local) { return local; }
__device__ __forceinline__ int paged_rows(const DecodeArgs &) { return 0; }
__device__ __forceinline__ int paged_rows(const PagedDecodeArgs &arg) { return arg.rows; }
__device__ __forceinline__ const __half *fresh_rows(const DecodeArgs &, int) { return nullptr; }
__device__ __forceinline__ const __half *fresh_rows(const PagedDecodeArgs &arg, int value) { return value ? arg.x.v : arg.x.k; }

}  // namespace
}  // namespace kivi
