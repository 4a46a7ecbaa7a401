// kivi_paged_tc.cuh -- the operand tiles that kivi_paged_stage.cuh writes and
// kivi_paged_tc.cu reads.
#pragma once

#include "kivi_paged.cuh"

namespace kivi {

constexpr int kTok = 128;                        // tokens per tile
constexpr int kImage = kTok * kHeadDim * 2;      // bytes of one operand's tile
constexpr int kChannels = 16;                    // key channels that also have a low part
constexpr int kLow = kTok * kChannels * 2;       // bytes of its tile
constexpr int kTileBytes = 2 * kImage + kLow;    // keys | values (weights: keys' low parts) | low parts of some channels

struct StageArgs {
    uint8_t *tiles;           // [pairs of this launch][tiles][kTileBytes]
    const uint8_t *channels;  // [pairs of this launch][kChannels]
    int tiles_per_pair;
    int pair0;                // first pair of this launch
};

// 16-byte chunk `chunk` (8 channels) of row r of an operand image: two panels
// of 128-byte rows, 128-byte swizzle.
__host__ __device__ constexpr int image_at(int r, int chunk)
{
    return (chunk >> 3) * (kImage / 2) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
}

// Chunk (0, 1) of row r of a low tile: 32-byte rows, 32-byte swizzle.
__host__ __device__ constexpr int low_at(int r, int chunk) { return r * 32 + ((chunk ^ ((r >> 2) & 1)) << 4); }

// Element of a run of 16 channels at place w of the tiles, for codes of `bits`
// bits (8: FP8, in order), and the place of element k.
__host__ __device__ constexpr int run_element(int bits, int w)
{
    return bits == 2 ? (w >> 1) + 8 * (w & 1) : bits == 4 ? (w & 8) + ((w >> 1) & 3) + 4 * (w & 1) : w;
}

// Value channel at stored position pos.
__host__ __device__ constexpr int value_channel(int bits, int G, int fmt, int pos)
{
    const int run = G / 8;
    return fmt || run * bits < 8 ? pos : pos % 16 / run * G + pos / 16 * run + pos % run;
}

#define KIVI_STAGE(name) \
    cudaError_t name(const PagedArgs &c, const ChunkArgs &x, const StageArgs &a, bool weights, dim3 grid, cudaStream_t s)
KIVI_STAGE(launch_stage_2);
KIVI_STAGE(launch_stage_4);
KIVI_STAGE(launch_stage_fp8);

}  // namespace kivi
