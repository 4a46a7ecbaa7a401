// kivi_paged_tc.cu -- attention of many query rows over a paged cache, and the
// softmax weights its pages get, on the 5th-generation tensor cores.
//
// Every cached token is read once per 256 query rows, so the pages are
// dequantised once, into the workspace, as the very tiles the matrix
// instructions take from shared memory (kivi_paged_stage.cuh); what runs here is
// a dense attention over them.
//
//  tc_kernel        256 query rows (two M tiles of 128) of one pair against a
//                   range of its tiles.  18 warps: one fetches tiles (bulk
//                   copies, two stages per operand), one issues the matrix
//                   instructions, and two warpgroups per M tile (a team) keep
//                   the softmax: a thread has half the columns of one query row.
//                   S = Q K^T and O += P V accumulate in tensor memory; P (fp16)
//                   overwrites the S it came from, so one team's softmax runs
//                   while the other's products do.  Up to 128 rows there is one M
//                   tile: the teams then take its even and its odd token tiles
//                   and join at the end.
//                   O is only rescaled when a row's maximum has grown by more
//                   than 2^8 since the last time: until then 2^(s - m) stays
//                   within fp16 and nothing is lost by an old m.
//                   Bound by the tensor cores' reads of their operands (S needs
//                   both from shared memory: 128 cycles for 64 of arithmetic)
//                   and by the softmax between the products.  2048 tokens x 4
//                   heads after 32768 tokens, 8 pairs: 787 us, 1440 TFLOP/s,
//                   tensor pipe active 66 %; without any softmax 700 us; issued by
//                   one diverged thread 1085 against 946 us at the time; P and the
//                   queries both in tensor memory, 64-token steps: 943.
//  tc_weigh_kernel  the same without values: every step's S is a tensor-memory
//                   buffer of its own (four in turn), keys have a full low part,
//                   and a thread turns its row's 128 scores into page sums.  16
//                   pairs of up to 16384 tokens, 128 rows: 32 us.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "kivi_paged_attend.cuh"
#include "kivi_paged_tc.cuh"

namespace kivi {
namespace {

constexpr int kMTile = 128;                      // query rows per M tile
constexpr int kRows = 2 * kMTile;                // query rows per block
constexpr int kStages = 2;
constexpr int kTcThreads = 576;              // attention: 16 softmax warps, MMA, fetch
constexpr int kWeighThreads = 320;           // weights: 8, MMA, fetch
constexpr int kTcBlocks = 152;                   // blocks the GPU holds at once
constexpr int kPartBlocks = 4 * kTcBlocks;       // weights: blocks of several splits, at most
constexpr int kJobUnits = 4;                     // what a job costs besides its tiles, in M tiles x token tiles
constexpr int kLeastUnits = 8;                   // fewer are not worth a block
constexpr int64_t kStageBytes = 1ll << 30;       // staged pairs per launch
constexpr int64_t kSumBytes = 256ll << 20;       // page sums held at once
constexpr long long kWaitCycles = 1ll << 32;     // about 2 s
constexpr float kRescale = 8.0f;                 // log2 of how far a maximum may run ahead

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

// Waits for a copy that nobody needs any more, about 2 s at most.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t phase)
{
    const long long start = clock64();
    while (!bar_try(bar, phase) && clock64() - start < kWaitCycles) {}
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ uint64_t operand(uint32_t addr, uint64_t leading, uint64_t stride, uint64_t swizzle)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (leading >> 4) << 16 | (stride >> 4) << 32 | (uint64_t)1 << 46 | swizzle << 61;
}

// Queries and keys: K-major, 128-byte rows and swizzle, eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t by_channel(uint32_t addr) { return operand(addr, 16, 1024, 2); }
// Their low tiles: K-major, 32-byte rows and swizzle, eight rows 256 bytes apart.
__device__ __forceinline__ uint64_t by_channel_low(uint32_t addr) { return operand(addr, 16, 256, 6); }
// Values, [token][channel] with the tokens as K: MN-major, panels of 64 channels
// kImage / 2 apart, eight tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t by_token(uint32_t addr) { return operand(addr, kImage / 2, 1024, 2); }

// fp16 x fp16 -> fp32, M = 128, N = 128; both K-major, or B MN-major.
constexpr uint32_t kIdescK = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kIdescMN = kIdescK | 1u << 16;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(kIdescK), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(kIdescMN), "r"(accumulate) : "memory");
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

__device__ __forceinline__ void tm_load16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

__device__ __forceinline__ void tm_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ----------------------------------------------------------------- common ---

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Largest of 64 scores.
__device__ __forceinline__ float half_max(const uint32_t (&s)[2][32])
{
    float mx[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t *e = &s[q >> 1][16 * (q & 1)];
        mx[q] = fmaxf(__uint_as_float(e[0]), __uint_as_float(e[1]));
#pragma unroll
        for (int k = 2; k < 16; k += 2)
            mx[q] = max3(mx[q], __uint_as_float(e[k]), __uint_as_float(e[k + 1]));
    }
    return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
}

// {lo half: x0, hi half: x1}, to nearest, for values that are in range.
__device__ __forceinline__ uint32_t pack(float x0, float x1)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x1), "f"(x0));
    return d;
}

// Whether any of the 256 threads of team i (barrier 1 + i) says so.
__device__ __forceinline__ bool team_any(int i, bool said)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
                 "barrier.cta.red.or.pred.aligned q, %1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(1 + i), "r"((uint32_t)said) : "memory");
    return any != 0;
}

// An attention launch's work is cut into equal ranges, one per block, without
// regard to where its jobs (256 query rows of one pair) end: a block may finish
// one job, do others and begin the next.  A job's units are kJobUnits and then
// one per M tile and token tile.  The plan, made on the device from the
// sequences' lengths:
struct Plan {
    int blocks;               // that have work
    int start[kTcBlocks + 1]; // job in which a block's range begins
    int units[1];             // [jobs + 1] units before each job
};

struct TcArgs {
    const uint8_t *tiles, *channels;
    const Plan *plan;         // attention
    int jobs, row_tiles;      // attention: jobs of this launch, and per pair
    int tiles_per_pair, pair0, S;
    int row0, rows;           // first query row of this launch, and rows a pair has room for in the results
    __half *out;
    float *o;                 // attention: [2 blocks][256 rows][D] parts of jobs that several blocks share
    float2 *ml;               // attention: [2 blocks][256 rows]; weights: [pairs of this launch][rows][2 S]
    float *ls;                // weights: [pairs of this launch][rows][units]
    int unit, units;
};

// Eight halves of a run of 16 (elements of places 8 half .. 8 half + 7).
template <int BITS>
__device__ __forceinline__ uint4 pick_places(const uint4 (&run)[2], int half)
{
    const __half *e = reinterpret_cast<const __half *>(run);
    uint32_t a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 v = __halves2half2(e[run_element(BITS, 2 * i)], e[run_element(BITS, 2 * i + 1)]);
        a[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return half ? make_uint4(a[4], a[5], a[6], a[7]) : make_uint4(a[0], a[1], a[2], a[3]);
}

// The block's query rows (row0 on, `count` of them exist) as operand images of
// mtiles M tiles, channels in the tiles' order; low: the picked channels alone.
template <int THREADS>
__device__ __forceinline__ void load_queries(const PagedArgs &c, const ChunkArgs &x, int h, int first, int row0, int rows,
                                             int mtiles, uint8_t (*q)[kImage], uint8_t (*q_low)[kLow], const uint8_t *channels)
{
    constexpr int D = kHeadDim;
    auto row_of = [&](int row) {
        const int t = row / c.g;
        return x.q + (int64_t)(first + t) * x.q_stride + (h * c.g + row - t * c.g) * D;
    };
    for (int i = threadIdx.x; i < mtiles * kMTile * 8; i += THREADS) {
        const int r = i >> 3, run = i & 7;
        uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (row0 + r < rows) {
            const uint4 *src = reinterpret_cast<const uint4 *>(row_of(row0 + r) + 16 * run);
            v[0] = src[0];
            v[1] = src[1];
        }
        uint4 a = v[0], b = v[1];
        if (c.bits == 2) {
            a = pick_places<2>(v, 0);
            b = pick_places<2>(v, 1);
        } else if (c.bits == 4) {
            a = pick_places<4>(v, 0);
            b = pick_places<4>(v, 1);
        }
        *reinterpret_cast<uint4 *>(q[r >> 7] + image_at(r & 127, 2 * run)) = a;
        *reinterpret_cast<uint4 *>(q[r >> 7] + image_at(r & 127, 2 * run + 1)) = b;
    }
    if (!q_low)
        return;
    for (int i = threadIdx.x; i < mtiles * kMTile * 2; i += THREADS) {
        const int r = i >> 1, half = i & 1;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (row0 + r < rows) {
            const __half *src = row_of(row0 + r);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 v = __halves2half2(src[channels[8 * half + 2 * e]], src[channels[8 * half + 2 * e + 1]]);
                w[e] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
        *reinterpret_cast<uint4 *>(q_low[r >> 7] + low_at(r & 127, half)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One lane of the warp issues.  The whole warp runs the loops around it, so that
// the operands stay uniform: worked out by one diverged thread, they cost more
// than the products they start.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// S[128 x 128] = Q K^T in tensor memory at d, eight steps of 16 channels.
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t accumulate)
{
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint32_t off = ((ks >> 2) * (kImage / 2) + (ks & 3) * 32) >> 4;
        mma_ss(d, q + off, k + off, accumulate | (ks > 0));
    }
}

// 256 query rows of one pair.
struct Job {
    int p, h, first, T;
    int rows, row0;           // query rows of the pair, first of the job
    int deep, rowed;          // page tokens, other cached tokens
    int np, tiles;            // page tiles, and all tiles that any of the rows sees
};

// Row tile rt of the launch's pair y; false when there are no such rows.
__device__ __forceinline__ bool job_of(const PagedArgs &c, const ChunkArgs &x, int pair0, int y, int row0, int rt, Job &j,
                                       bool &bad)
{
    j.p = pair0 + y;
    j.h = j.p % c.Hkv;
    PagedState st;
    bad = !sequence(c, x, j.p / c.Hkv, j.first, j.T, st);
    if (bad)
        return false;
    j.rows = j.T * c.g;
    j.row0 = row0 + rt * kRows;
    if (j.row0 >= j.rows)
        return false;
    j.deep = st.held * c.G;
    j.rowed = st.sink + st.window;
    const int seen = !x.k ? 0 : x.full ? j.T : min(j.T, (j.row0 + kRows - 1) / c.g + 1);
    j.np = (j.deep + kTok - 1) / kTok;
    j.tiles = j.np + (j.rowed + seen + kTok - 1) / kTok;
    return true;
}

__device__ __forceinline__ int mtiles_of(const Job &j) { return j.rows - j.row0 > kMTile ? 2 : 1; }

// Tile of a job at which unit u of the launch lies.
__device__ __forceinline__ int tile_at(const Job &j, int units0, int64_t u)
{
    const int64_t t = (u - units0 - kJobUnits) / mtiles_of(j);
    return u <= units0 + kJobUnits ? 0 : (int)(t < j.tiles ? t : j.tiles);
}

// First unit of block k.
__device__ __forceinline__ int64_t first_unit(const Plan *plan, int jobs, int k)
{
    return (int64_t)plan->units[jobs] * k / plan->blocks;
}

// Block 0 of the preparing launch: the plan.
__device__ void make_plan(const PagedArgs &c, const ChunkArgs &x, int pair0, int jobs, int row_tiles, int blocks, Plan *plan,
                          int *scan)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int before = 0;
    for (int j0 = 0; j0 < jobs; j0 += 256) {
        const int i = j0 + tid;
        int units = 0;
        if (i < jobs) {
            Job job;
            bool bad;
            const int y = i / row_tiles;
            if (job_of(c, x, pair0, y, 0, i - y * row_tiles, job, bad))
                units = kJobUnits + mtiles_of(job) * job.tiles;
            if (bad)
                atomicOr(c.control, KIVI_STATUS_BAD_STATE);
        }
        int incl = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += up;
        }
        __syncthreads();
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        int all = 0;
        for (int k = 0; k < 8; ++k) {
            if (k < warp)
                incl += scan[k];
            all += scan[k];
        }
        if (i < jobs)
            plan->units[i] = before + incl - units;
        before += all;
    }
    const int used = max(1, min(blocks, before / kLeastUnits));
    if (tid == 0) {
        plan->units[jobs] = before;
        plan->blocks = used;
    }
    __threadfence_block();
    __syncthreads();
    for (int k = tid; k < used; k += 256) {
        // the last job that begins at or before the block's first unit
        const int64_t u = (int64_t)before * k / used;
        int lo = 0, hi = jobs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldcg(&plan->units[mid]) <= u)
                lo = mid;
            else
                hi = mid;
        }
        plan->start[k] = lo;
    }
}

// Its other blocks, one per pair: the 16 key channels of each pair whose keys also get a
// low part, those with the largest scales in up to 32 of its pages (no result
// depends on which they are but for its last bits).
__device__ void pick_channels(const PagedArgs &c, const ChunkArgs &x, int p, uint8_t *channels, float *top)
{
    const int ch = threadIdx.x;
    int first, T;
    PagedState st;
    if (!sequence(c, x, p / c.Hkv, first, T, st))
        return;
    const int n = min(st.held, 32);
    float most = 0.0f;
    for (int i = 0; i < n && ch < kHeadDim; ++i) {
        const unsigned char *rec = page_record(c, p, (int)((int64_t)st.held * i / n));
        if (rec)
            most = fmaxf(most, c.meta ? meta_load<1>(rec, ch) : meta_load<0>(rec, ch));
    }
    if (ch < kHeadDim)
        top[ch] = most;
    __syncthreads();
    if (ch >= kHeadDim)
        return;
    int rank = 0;
    for (int i = 0; i < kHeadDim; ++i)
        rank += top[i] > most || (top[i] == most && i < ch);
    if (rank < kChannels)
        channels[rank] = (uint8_t)ch;
}

__global__ void __launch_bounds__(256) prepare_kernel(PagedArgs c, ChunkArgs x, int pair0, int pairs, int jobs, int row_tiles,
                                                      int blocks, uint8_t *channels, Plan *plan)
{
    __shared__ float top[kHeadDim];
    __shared__ int scan[8];
    let_next_in();
    if (blockIdx.x == 0)
        make_plan(c, x, pair0, jobs, row_tiles, blocks, plan, scan);
    else
        pick_channels(c, x, pair0 + blockIdx.x - 1, channels + (blockIdx.x - 1) * kChannels, top);
}

// fp16 tokens that query row `row` sees.
__device__ __forceinline__ int seen_of(const PagedArgs &c, const ChunkArgs &x, const Job &j, int row)
{
    return j.rowed + (!x.k ? 0 : x.full ? j.T : min(j.T, row / c.g + 1));
}

// -------------------------------------------------------------- attention ---

// A block's share of a job: pair of the launch, first tile, tiles.
struct Share {
    Job job;
    int y, t0, n;
};

struct TcSmem {
    uint8_t q[2][kImage];
    uint8_t k[kStages][kImage];
    uint8_t v[kStages][kImage];
    uint8_t q_low[2][kLow];
    uint8_t k_low[kStages][kLow];
    uint64_t k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
    float rows[2][2][kMTile];     // per team and half: a row's maximum, at the end its sum
    Share share;                  // what the workers are at, while `there`
    bool there;
    float4 other[kMTile];         // team 1's maximum, sum and factor, where the teams share an M tile
    uint64_t s_full[2], p_full[2];
    uint32_t tmem;
    int failed;
};
// the join of the two teams of one M tile: [128][D] floats over the queries, 16-byte chunk i of row r at i ^ (r & 7)
static_assert(kMTile * kHeadDim * 4 <= 2 * kImage, "join buffer");

constexpr int kWorkers = kTcThreads - 32;        // all but the fetching warp: they meet between jobs

// CAP: 0 no cap, 1 a small one, 2 any.
template <int CAP>
__global__ void __launch_bounds__(kTcThreads, 1) tc_kernel(PagedArgs c, ChunkArgs x, TcArgs d)
{
    constexpr int D = kHeadDim;
    extern __shared__ uint8_t smem_raw[];
    TcSmem &sm = *reinterpret_cast<TcSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Plan *plan = d.plan;
    const int block = blockIdx.x;
    let_next_in();
    wait_for_previous();
    if (block >= plan->blocks)
        return;
    const int64_t u0 = first_unit(plan, d.jobs, block), u1 = first_unit(plan, d.jobs, block + 1);
    const bool low = c.fmt == 0;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(smem_addr(&sm.k_full[i]), 1);
            bar_init(smem_addr(&sm.k_free[i]), 1);
            bar_init(smem_addr(&sm.v_full[i]), 1);
            bar_init(smem_addr(&sm.v_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&sm.s_full[i]), 1);
            bar_init(smem_addr(&sm.p_full[i]), 2 * kMTile);
        }
        sm.failed = 0;
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tm = sm.tmem;                  // columns: S/P of warpgroup 0, of 1, O of 0, of 1
    volatile int *failed = &sm.failed;
    // The block's next share of a job, from job i on (rows that see nothing get
    // their zeros from the block in which their job begins).
    auto next_share = [&](int &i, Share &g) {
        for (; i < d.jobs; ++i) {
            const int at = plan->units[i], end = plan->units[i + 1];
            if (at >= u1)
                break;
            if (end == at)
                continue;
            bool bad;
            g.y = i / d.row_tiles;
            job_of(c, x, d.pair0, g.y, 0, i - g.y * d.row_tiles, g.job, bad);
            g.t0 = u0 > at ? tile_at(g.job, at, u0) : 0;
            g.n = (u1 < end ? tile_at(g.job, at, u1) : g.job.tiles) - g.t0;
            if (g.n > 0 || (g.job.tiles == 0 && at >= u0)) {
                ++i;
                return true;
            }
        }
        return false;
    };

    // All but the fetching warp meet between shares.
    auto meet = [&]() {
        __syncwarp();
        asm volatile("barrier.cta.sync.aligned 4, %0;" ::"n"(kWorkers) : "memory");
    };

    if (warp == 17) {
        if (lane == 0) {                          // fetches the tiles, ahead into the next job
            int keys = 0, values = 0;             // tiles asked for
            Share g;
            for (int i = plan->start[block]; !*failed && next_share(i, g);) {
                const uint8_t *src = d.tiles + ((int64_t)g.y * d.tiles_per_pair + g.t0) * kTileBytes;
                for (int j = 0; j < g.n; ++j, src += kTileBytes) {
                    const int s = keys % kStages;
                    const uint32_t free_phase = ((keys / kStages) & 1) ^ 1;   // the first round passes at once
                    if (!bar_wait(smem_addr(&sm.k_free[s]), free_phase, failed))
                        break;
                    const bool with_low = low && g.t0 + j < g.job.np;
                    bar_expect(smem_addr(&sm.k_full[s]), kImage + (with_low ? kLow : 0));
                    bulk_load(smem_addr(sm.k[s]), src, kImage, smem_addr(&sm.k_full[s]));
                    if (with_low)
                        bulk_load(smem_addr(sm.k_low[s]), src + 2 * kImage, kLow, smem_addr(&sm.k_full[s]));
                    ++keys;
                    if (!bar_wait(smem_addr(&sm.v_free[s]), free_phase, failed))
                        break;
                    bar_expect(smem_addr(&sm.v_full[s]), kImage);
                    bulk_load(smem_addr(sm.v[s]), src + kImage, kImage, smem_addr(&sm.v_full[s]));
                    ++values;
                }
            }
            if (*failed) {                        // leave no copy in flight: wait, with a limit, for the last ones
                for (int j = max(0, keys - kStages); j < keys; ++j)
                    bar_drain(smem_addr(&sm.k_full[j % kStages]), (j / kStages) & 1);
                for (int j = max(0, values - kStages); j < values; ++j)
                    bar_drain(smem_addr(&sm.v_full[j % kStages]), (j / kStages) & 1);
            }
        }
    } else if (warp == 16) {                      // issues the matrix instructions, and says what comes next
        int done = 0, tiles0 = 0, tiles1 = 0;     // tiles before this share: all, and each team's
        for (int next = plan->start[block];;) {
            meet();                               // the last share is done with
            if (lane == 0)
                sm.there = next_share(next, sm.share);
            meet();
            if (!sm.there)
                break;
            const Job &job = sm.share.job;
            const int t0 = sm.share.t0, n = sm.share.n, np = job.np;
            const bool two = mtiles_of(job) == 2;     // two M tiles, or one whose tiles the teams share
            auto paged = [&](int j) { return t0 + j < np; };
            load_queries<kWorkers>(c, x, job.h, job.first, job.row0, job.rows, two ? 2 : 1, sm.q, low ? sm.q_low : nullptr,
                                   d.channels + sm.share.y * kChannels);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            meet();
            if (n > 0) {
                const bool leader = elect_one();
                const uint64_t q_at = by_channel(smem_addr(sm.q[0])), k_at = by_channel(smem_addr(sm.k[0]));
                const uint64_t q_low_at = by_channel_low(smem_addr(sm.q_low[0])), k_low_at = by_channel_low(smem_addr(sm.k_low[0]));
                const uint64_t v_at = by_token(smem_addr(sm.v[0]));
                // scores of tile j into S of team i, against M tile m; then (team i of) bar
                auto scores = [&](int i, int m, int j) {
                    const int s = (done + j) % kStages;
                    const bool with_low = low && paged(j);
                    if (leader) {
                        if (with_low)
                            mma_ss(tm + 128 * i, q_low_at + m * (kLow >> 4), k_low_at + s * (kLow >> 4), 0);
                        mma_scores(tm + 128 * i, q_at + m * (kImage >> 4), k_at + s * (kImage >> 4), with_low);
                    }
                };
                auto values = [&](int i, int j, bool first) {
                    const uint64_t v = v_at + ((done + j) % kStages) * (kImage >> 4);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(tm + 256 + 128 * i, tm + 128 * i + 8 * ks, v + (ks * 16 * 128 >> 4), !first || ks > 0);
                    }
                };
                auto commit = [&](uint64_t *bar) {
                    if (leader)
                        mma_commit(smem_addr(bar));
                };
                auto there = [&](uint64_t *bar, int phase) {
                    return (bool)__all_sync(0xffffffffu, bar_wait(smem_addr(bar), phase & 1, failed));
                };
                auto keys_there = [&](int j) { return there(&sm.k_full[(done + j) % kStages], (done + j) / kStages); };
                auto values_there = [&](int j) { return there(&sm.v_full[(done + j) % kStages], (done + j) / kStages); };
                bool ok = keys_there(0);
                if (two) {
                    if (ok) {
                        for (int i = 0; i < 2; ++i) {
                            scores(i, i, 0);
                            commit(&sm.s_full[i]);
                        }
                        commit(&sm.k_free[done % kStages]);
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        const bool more = j + 1 < n;
                        ok = values_there(j) && (!more || keys_there(j + 1));
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            ok = ok && there(&sm.p_full[i], (i ? tiles1 : tiles0) + j);
                            if (!ok)
                                break;
                            tm_fence_after();
                            values(i, j, j == 0);
                            if (more)
                                scores(i, i, j + 1);
                            commit(&sm.s_full[i]);
                        }
                        if (ok) {
                            commit(&sm.v_free[(done + j) % kStages]);
                            if (more)
                                commit(&sm.k_free[(done + j + 1) % kStages]);
                        }
                    }
                } else {
                    // tile j belongs to team j & 1
                    for (int j = 0; ok && j < min(n, 2); ++j) {
                        ok = j == 0 || keys_there(j);
                        if (ok) {
                            scores(j, 0, j);
                            commit(&sm.s_full[j]);
                            commit(&sm.k_free[(done + j) % kStages]);
                        }
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        const int i = j & 1;
                        const bool more = j + 2 < n;
                        ok = values_there(j) && (!more || keys_there(j + 2)) && there(&sm.p_full[i], (i ? tiles1 : tiles0) + (j >> 1));
                        if (!ok)
                            break;
                        tm_fence_after();
                        values(i, j, j < 2);
                        if (more)
                            scores(i, 0, j + 2);
                        commit(&sm.s_full[i]);
                        commit(&sm.v_free[(done + j) % kStages]);
                        if (more)
                            commit(&sm.k_free[(done + j + 2) % kStages]);
                    }
                }
            }
            done += n;
            tiles0 += two ? n : (n + 1) / 2;
            tiles1 += two ? n : n / 2;
        }
    } else {
        int round = 0;                            // phases of this team's s_full before this share
        for (;;) {
            meet();
            meet();
            if (!sm.there)
                break;
            const Job &job = sm.share.job;
            const int t0 = sm.share.t0, n = sm.share.n, np = job.np;
            const bool two = mtiles_of(job) == 2;     // two M tiles, or one whose tiles the teams share
            auto paged = [&](int j) { return t0 + j < np; };
            load_queries<kWorkers>(c, x, job.h, job.first, job.row0, job.rows, two ? 2 : 1, sm.q, low ? sm.q_low : nullptr,
                                   d.channels + sm.share.y * kChannels);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            meet();
            // softmax: a thread has columns 64 half .. + 63 of one query row (its TMEM lane)
            const int i = warp >> 3, half = (warp >> 2) & 1;
            const uint32_t lanes = (uint32_t)(warp & 3) << 21;             // 32 lanes a warp, lane field from bit 16
            const uint32_t ts = tm + 128 * i + lanes, to = tm + 256 + 128 * i + 64 * half + lanes;
            const int r = (warp & 3) * 32 + lane;
            // columns this row sees: of the page tiles, and of the fp16 tiles
            const int deep = job.deep, shallow = seen_of(c, x, job, job.row0 + (two ? i * kMTile : 0) + r);
            const int mine = two ? n : (n - i + 1) / 2;                    // tiles of this team
            const float page_times = low ? 2.0f : c.fp8_k_scale, page_value = low ? 2.0f : c.fp8_v_scale;
            float *shared = sm.rows[i][half], *theirs = sm.rows[i][half ^ 1];
            float m = -INFINITY, l = 0.0f;                                  // l: of this half
            bool in_pages = false, lost = false;                           // O is in units of page_value; a wait gave up
            for (int e = 0; e < mine; ++e) {
                const int j = two ? e : 2 * e + i, t = t0 + j;
                const bool ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full[i]), (round + e) & 1, failed));
                tm_fence_after();
                uint32_t s[2][32];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    tm_load32(ts + 64 * half + 32 * q, s[q]);
                tm_wait_load();
                const float times = paged(j) ? page_times : 1.0f;
                if constexpr (CAP != 0) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        cap_scores<CAP == 1>(s[q], times, x);
                }
                const float scale = CAP != 0 ? 1.0f : x.scale_log2 * times;
                const int left = (paged(j) ? deep - t * kTok : shallow - (t - np) * kTok) - 64 * half;
                if (left < 64) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * q + k >= left)
                                s[q][k] = 0xff800000u;                      // -inf
                }
                const float top = half_max(s) * scale;
                const bool leaves = in_pages && !paged(j);                   // O becomes plain
                in_pages = paged(j);
                // One barrier per tile: both halves have read S (P goes over it), and
                // a maximum that ran ahead (also the first one, m = -inf) is known to
                // the whole team.
                tm_fence_before();
                const bool move = team_any(i, !ok || top - m > kRescale);
                tm_fence_after();
                if (move || leaves) {
                    shared[r] = top;
                    asm volatile("barrier.cta.sync.aligned %0, 256;" ::"r"(1 + i) : "memory");
                    const float both = fmaxf(top, theirs[r]);
                    if (team_any(i, !ok)) {
                        lost = true;
                        break;
                    }
                    const bool grown = both - m > kRescale;
                    const float m1 = grown ? both : m;
                    const float alpha = grown && m > -INFINITY ? ex2(m - m1) : 1.0f;
                    m = m1;
                    l *= alpha;
                    const float factor = leaves ? alpha * page_value : alpha;
                    if (e > 0) {
                        // O is at rest: the phase just waited for ends after the last P V
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t o[16];
                            tm_load16(to + 16 * q, o);
                            tm_wait_load();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * factor);
                            tm_store16(to + 16 * q, o);
                        }
                    }
                }
                const float ms = m == -INFINITY ? 0.0f : m;
                const float2 scale2 = make_float2(scale, scale), ms2 = make_float2(-ms, -ms);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float2 a = __ffma2_rn(make_float2(__uint_as_float(s[q][2 * k]), __uint_as_float(s[q][2 * k + 1])), scale2, ms2);
                        a = make_float2(ex2(a.x), ex2(a.y));
                        sum[k & 1] = __fadd2_rn(sum[k & 1], a);
                        pk[k] = pack(a.x, a.y);
                    }
                    tm_store16(ts + 32 * half + 16 * q, pk);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tm_wait_store();
                tm_fence_before();
                bar_arrive(smem_addr(&sm.p_full[i]));
            }
            if (mine > 0 && !lost)
                __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full[i]), (round + mine) & 1, failed));       // the last P V
            tm_fence_after();
            // the halves' sums, and with one M tile the teams' parts
            float w = in_pages ? page_value : 1.0f, w1 = 0.0f;              // factors of this O and of the other team's
            shared[r] = l;
            asm volatile("barrier.cta.sync.aligned %0, 256;" ::"r"(1 + i) : "memory");
            l += theirs[r];
            uint4 *xo = reinterpret_cast<uint4 *>(sm.q) + r * (D / 4);
            if (!two) {
                // Team 1 hands over its part, if it had a tile.  Its last commit came
                // after the last scores were issued, so the queries are free by then.
                if (i == 1) {
#pragma unroll 1
                    for (int q = 0; q < (mine > 0 ? 4 : 0); ++q) {
                        uint32_t o[16];
                        __syncwarp();
                        tm_load16(to + 16 * q, o);
                        tm_wait_load();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            xo[(16 * half + 4 * q + k) ^ (r & 7)] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                    if (half == 0)
                        sm.other[r] = make_float4(m, l, w, 0.0f);
                }
                asm volatile("barrier.cta.sync.aligned 3, 512;" ::: "memory");
                if (i == 0) {
                    const float4 other = sm.other[r];
                    const float M = fmaxf(m, other.x), at = M == -INFINITY ? 0.0f : M;
                    const float f0 = ex2(m - at), f1 = ex2(other.x - at);
                    w1 = other.z * f1;
                    w *= f0;
                    l = l * f0 + other.y * f1;
                    m = M;
                }
            }
            const int row = job.row0 + (two ? i * kMTile : 0) + r, tok = row / c.g, hh = row - tok * c.g;
            const bool writes = (two || i == 0) && row < job.rows;
            const bool whole = n == job.tiles;
            const float inv = whole ? (l > 0.0f ? 1.0f / l : 0.0f) : 1.0f;
            // a job that began in an earlier block: this block's first part, else its last
            const int64_t part = (int64_t)(2 * block + (t0 > 0 ? 0 : 1)) * kRows + (row - job.row0);
            const int64_t at = (int64_t)(job.first + tok) * (c.Hkv * c.g) + job.h * c.g + hh;
            // a run's places hold the channels of its stored positions, in the run's order
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[16];
                __syncwarp();
                if (mine > 0 && (two || i == 0)) {
                    tm_load16(to + 16 * q, o);
                    tm_wait_load();
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        o[k] = 0u;
                }
                if (!writes)
                    continue;
                float f[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    f[k] = __uint_as_float(o[k]) * w;
                if (w1 != 0.0f) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v = xo[(16 * half + 4 * q + k) ^ (r & 7)];
                        f[4 * k] = fmaf(__uint_as_float(v.x), w1, f[4 * k]);
                        f[4 * k + 1] = fmaf(__uint_as_float(v.y), w1, f[4 * k + 1]);
                        f[4 * k + 2] = fmaf(__uint_as_float(v.z), w1, f[4 * k + 2]);
                        f[4 * k + 3] = fmaf(__uint_as_float(v.w), w1, f[4 * k + 3]);
                    }
                }
                auto put = [&](auto bits) {
                    constexpr int BITS = decltype(bits)::value;
                    // pairs of neighbouring stored positions are neighbouring channels
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        int p0 = 0, p1 = 0;                 // their places in the run
#pragma unroll
                        for (int z = 0; z < 16; ++z) {
                            if (run_element(BITS, z) == k)
                                p0 = z;
                            if (run_element(BITS, z) == k + 1)
                                p1 = z;
                        }
                        const float a0 = f[p0] * inv, a1 = f[p1] * inv;
                        const int ch = value_channel(BITS, c.G, BITS == 8, 64 * half + 16 * q + k);
                        if (whole)
                            *reinterpret_cast<uint32_t *>(d.out + at * D + ch) = pack_sat(a0, a1);
                        else
                            *reinterpret_cast<float2 *>(d.o + part * D + ch) = make_float2(a0, a1);
                    }
                };
                if (c.bits == 2)
                    put(std::integral_constant<int, 2>{});
                else if (c.bits == 4)
                    put(std::integral_constant<int, 4>{});
                else
                    put(std::integral_constant<int, 8>{});
            }
            if (!whole && writes && half == 0)
                d.ml[part] = make_float2(m, l);
            round += mine > 0 ? mine + 1 : 0;
        }
    }
    tm_fence_before();
    __syncthreads();
    if (tid == 0 && sm.failed)
        atomicOr(c.control, KIVI_STATUS_WAIT_TIMEOUT);
    if (warp == 16) {
        __syncwarp();
        tm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
    }
}

constexpr int kJoinRows = 16;                    // rows per block of the join

// Joins the parts of the jobs that several blocks share.  Block k looks at the
// boundary between blocks k and k + 1; the first boundary inside a job joins it.
__global__ void __launch_bounds__(256) tc_join_kernel(PagedArgs c, ChunkArgs x, TcArgs d)
{
    __shared__ int parts[kTcBlocks + 1];         // part numbers of the job, in order
    __shared__ int count;
    __shared__ Job job;
    const Plan *plan = d.plan;
    wait_for_previous();
    const int used = plan->blocks, first_block = blockIdx.x;
    if (first_block >= used - 1)
        return;
    if (threadIdx.x == 0) {
        const int64_t total = plan->units[d.jobs];
        const int i = plan->start[first_block + 1], at = plan->units[i], end = plan->units[i + 1];
        auto first_unit = [&](int k) { return total * k / used; };
        // the tile at which block k's share of this job begins
        auto begin = [&](int k) { return first_unit(k) > at ? tile_at(job, at, first_unit(k)) : 0; };
        auto inside = [&](int k) { return begin(k) > 0 && begin(k) < job.tiles; };
        bool bad;
        count = 0;
        const int y = i / d.row_tiles;
        if (end > at && job_of(c, x, d.pair0, y, 0, i - y * d.row_tiles, job, bad) && inside(first_block + 1) &&
            !inside(first_block)) {
            for (int k = first_block, t = 0; t < job.tiles; ++k) {
                const int next = k < used - 1 && first_unit(k + 1) < end ? begin(k + 1) : job.tiles;
                if (next > t)
                    parts[count++] = 2 * k + (t > 0 ? 0 : 1);
                t = next;
            }
        }
    }
    __syncthreads();
    const int n = count, lane = threadIdx.x & 31;
    const int end = min(job.rows - job.row0, (int)blockIdx.y * kJoinRows + kJoinRows);
    if (n == 0)
        return;
    for (int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5); r < end; r += 8) {
        float M = -INFINITY, L = 0.0f;
        float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < n; ++k)
            M = fmaxf(M, d.ml[(int64_t)parts[k] * kRows + r].x);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const int64_t part = (int64_t)parts[k] * kRows + r;
            const float2 ml = d.ml[part];
            const float4 v = *reinterpret_cast<const float4 *>(d.o + part * kHeadDim + 4 * lane);
            const float w = ml.y > 0.0f ? ex2(ml.x - M) : 0.0f;
            L = fmaf(ml.y, w, L);
            O.x = fmaf(v.x, w, O.x);
            O.y = fmaf(v.y, w, O.y);
            O.z = fmaf(v.z, w, O.z);
            O.w = fmaf(v.w, w, O.w);
        }
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        const int row = job.row0 + r, tok = row / c.g;
        const int64_t to = (int64_t)(job.first + tok) * (c.Hkv * c.g) + job.h * c.g + (row - tok * c.g);
        *reinterpret_cast<uint2 *>(d.out + to * kHeadDim + 4 * lane) =
            make_uint2(pack_sat(O.x * inv, O.y * inv), pack_sat(O.z * inv, O.w * inv));
    }
}

// ---------------------------------------------------------------- weights ---

struct WeighSmem {
    uint8_t q[2][kImage];
    uint8_t k[kStages][kImage];
    uint8_t k_low[kStages][kImage];
    uint64_t k_full[kStages], k_free[kStages];
    uint64_t s_full[4], s_free[4];
    uint32_t tmem;
    int failed;
};

// Step e is the scores of one M tile against one token tile (two M tiles: M tile
// e & 1, tile e / 2; one: tile e), in S buffer e & 3, read by warpgroup e & 1.
template <int CAP, int UNIT>
__global__ void __launch_bounds__(kWeighThreads, 1) tc_weigh_kernel(PagedArgs c, ChunkArgs x, TcArgs d)
{
    extern __shared__ uint8_t smem_raw[];
    WeighSmem &sm = *reinterpret_cast<WeighSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Job job;
    bool bad;
    const bool some = job_of(c, x, d.pair0, blockIdx.y, d.row0, blockIdx.x, job, bad);
    if (bad && tid == 0 && blockIdx.x == 0 && blockIdx.z == 0)
        atomicOr(c.control, KIVI_STATUS_BAD_STATE);
    let_next_in();
    wait_for_previous();
    if (!some)
        return;
    const int t0 = (int)((int64_t)job.tiles * blockIdx.z / d.S), n = (int)((int64_t)job.tiles * (blockIdx.z + 1) / d.S) - t0;
    const bool two = mtiles_of(job) == 2;
    const bool low = c.fmt == 0;
    const int steps = two ? 2 * n : n;

    load_queries<kWeighThreads>(c, x, job.h, job.first, job.row0, job.rows, two ? 2 : 1, sm.q, nullptr, nullptr);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(smem_addr(&sm.k_full[i]), 1);
            bar_init(smem_addr(&sm.k_free[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            bar_init(smem_addr(&sm.s_full[i]), 1);
            bar_init(smem_addr(&sm.s_free[i]), kMTile);
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
    const uint32_t tm = sm.tmem;
    volatile int *failed = &sm.failed;
    auto paged = [&](int j) { return t0 + j < job.np; };

    if (warp == 9) {
        if (lane == 0) {
            const uint8_t *src = d.tiles + ((int64_t)blockIdx.y * d.tiles_per_pair + t0) * kTileBytes;
            int keys = 0;
            for (int j = 0; j < n; ++j, src += kTileBytes) {
                const int s = j % kStages;
                if (!bar_wait(smem_addr(&sm.k_free[s]), ((j / kStages) & 1) ^ 1, failed))
                    break;
                const bool with_low = low && paged(j);
                bar_expect(smem_addr(&sm.k_full[s]), with_low ? 2 * kImage : kImage);
                bulk_load(smem_addr(sm.k[s]), src, kImage, smem_addr(&sm.k_full[s]));
                if (with_low)
                    bulk_load(smem_addr(sm.k_low[s]), src + kImage, kImage, smem_addr(&sm.k_full[s]));
                keys = j + 1;
            }
            if (*failed)
                for (int j = max(0, keys - kStages); j < keys; ++j)
                    bar_drain(smem_addr(&sm.k_full[j % kStages]), (j / kStages) & 1);
        }
    } else if (warp == 8) {
        const bool leader = elect_one();
        const uint64_t q_at = by_channel(smem_addr(sm.q[0])), k_at = by_channel(smem_addr(sm.k[0]));
        const uint64_t k_low_at = by_channel(smem_addr(sm.k_low[0]));
        bool ok = true;
        for (int e = 0; ok && e < steps; ++e) {
            const int j = two ? e >> 1 : e, m = two ? e & 1 : 0, s = j % kStages;
            if (!two || m == 0)
                ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.k_full[s]), (j / kStages) & 1, failed));
            ok = ok && __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_free[e & 3]), ((e >> 2) & 1) ^ 1, failed));
            if (!ok)
                break;
            tm_fence_after();
            const uint32_t to = tm + 128 * (e & 3);
            const bool with_low = low && paged(j);
            if (leader) {
                if (with_low)
                    mma_scores(to, q_at + m * (kImage >> 4), k_low_at + s * (kImage >> 4), 0);
                mma_scores(to, q_at + m * (kImage >> 4), k_at + s * (kImage >> 4), with_low);
                mma_commit(smem_addr(&sm.s_full[e & 3]));
                if (!two || m == 1)
                    mma_commit(smem_addr(&sm.k_free[s]));
            }
        }
    } else {
        const int i = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const int row = job.row0 + (two ? i * kMTile : 0) + (warp & 3) * 32 + lane;
        const int shallow = seen_of(c, x, job, row);
        const bool live = row < job.rows;
        const float page_times = low ? 2.0f : c.fp8_k_scale;
        float *ls = d.ls + ((int64_t)blockIdx.y * d.rows + (row - d.row0)) * d.units;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int e = i; e < steps; e += 2) {
            const int j = two ? e >> 1 : e, t = t0 + j;
            ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full[e & 3]), (e >> 2) & 1, failed));
            if (!ok)
                break;
            tm_fence_after();
            const bool page = paged(j);
            const float times = page ? page_times : 1.0f, scale = CAP != 0 ? 1.0f : x.scale_log2 * times;
            const int left = page ? job.deep - t * kTok : shallow - (t - job.np) * kTok;
            float unit_max[kTok / UNIT], unit_sum[kTok / UNIT];
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                tm_load32(tm + 128 * (e & 3) + lanes + 32 * q, s[q]);
            tm_wait_load();
            tm_fence_before();
            bar_arrive(smem_addr(&sm.s_free[e & 3]));
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (CAP != 0)
                    cap_scores<CAP == 1>(s[q], times, x);
                if (left < 32 * q + 32) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * q + k >= left)
                            s[q][k] = 0xff800000u;
                }
#pragma unroll
                for (int u = 0; u < 32; u += UNIT) {
                    float mx = -INFINITY, sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                    for (int k = u; k < u + UNIT; ++k)
                        mx = fmaxf(mx, __uint_as_float(s[q][k]));
                    mx *= scale;
                    const float ms = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
                    for (int k = u; k < u + UNIT; k += 2) {
                        sum0 += ex2(fmaf(__uint_as_float(s[q][k]), scale, -ms));
                        sum1 += ex2(fmaf(__uint_as_float(s[q][k + 1]), scale, -ms));
                    }
                    unit_max[(32 * q + u) / UNIT] = mx;
                    unit_sum[(32 * q + u) / UNIT] = sum0 + sum1;
                    top = fmaxf(top, mx);
                }
            }
            if (page && live) {
#pragma unroll
                for (int u = 0; u < kTok / UNIT; ++u)
                    if (u * UNIT < left)
                        ls[t * (kTok / UNIT) + u] = unit_max[u] + __log2f(unit_sum[u]);
            }
            const float m1 = fmaxf(m, top), at = m1 == -INFINITY ? 0.0f : m1;
            l *= ex2(m - at);
#pragma unroll
            for (int u = 0; u < kTok / UNIT; ++u)
                l = fmaf(unit_sum[u], ex2(unit_max[u] - at), l);
            m = m1;
        }
        // two parts per split: the warpgroups' (with two M tiles one of them is empty)
        if (live) {
            float2 *ml = d.ml + (((int64_t)blockIdx.y * d.rows + (row - d.row0)) * d.S + blockIdx.z) * 2;
            ml[two ? 0 : i] = make_float2(m, l);
            if (two)
                ml[1] = make_float2(-INFINITY, 0.0f);
        }
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

// --------------------------------------------------------------- launches ---

constexpr int kTcSmem = sizeof(TcSmem) + 1024, kWeighSmem = sizeof(WeighSmem) + 1024;

struct TcPlan {
    int tiles, row_tiles, pairs, splits;      // pairs: staged and worked on per launch; row_tiles, splits: of one launch
    int64_t pair_bytes;
};

// Splits of `blocks` blocks over `tiles` token tiles: the count with the
// smallest waves x (fixed cost of a block, worth about 3 tiles, + its tiles).
int tc_splits(int64_t blocks, int64_t tiles)
{
    int64_t best = INT64_MAX;
    int splits = 1;
    for (int64_t s = 1; s <= std::max<int64_t>(1, std::min(kPartBlocks / blocks, tiles)); ++s) {
        const int64_t cost = (blocks * s + kTcBlocks - 1) / kTcBlocks * (3 + (tiles + s - 1) / s);
        if (cost < best) {
            best = cost;
            splits = (int)s;
        }
    }
    return splits;
}

int64_t row_tiles_of(const PagedArgs &c, int max_new) { return ((int64_t)max_new * c.g + kRows - 1) / kRows; }

int weigh_unit(const PagedArgs &c) { return std::min(c.G, 32); }

// page sums of one block of query rows of every pair
int64_t sum_bytes(const PagedArgs &c, int64_t pairs)
{
    return pairs * kRows * ((int64_t)c.columns * c.G / weigh_unit(c)) * 4;
}

TcPlan tc_plan(const PagedArgs &c, int max_new, int max_cached, bool weights)
{
    TcPlan p;
    // page tiles and fp16 tiles each end in one that may be part empty
    p.tiles = (int)(((int64_t)max_cached + max_new + kTok - 1) / kTok + 1);
    p.pair_bytes = (int64_t)p.tiles * kTileBytes;
    const int64_t all = (int64_t)c.B * c.Hkv, most = std::max<int64_t>(1, std::min(all, kStageBytes / p.pair_bytes));
    const int64_t launches = (all + most - 1) / most;
    p.pairs = (int)((all + launches - 1) / launches);       // launches of equal size
    p.row_tiles = (int)row_tiles_of(c, max_new);
    if (weights)
        p.row_tiles = (int)std::max<int64_t>(1, std::min<int64_t>(p.row_tiles, kSumBytes / sum_bytes(c, p.pairs)));
    p.splits = weights ? tc_splits((int64_t)p.pairs * p.row_tiles, p.tiles) : 1;
    return p;
}

// Bytes of the picked channels and of an attention's plan.
int64_t channel_bytes(int64_t pairs) { return (pairs * kChannels + 255) / 256 * 256; }
int64_t plan_bytes(int64_t jobs) { return ((int64_t)sizeof(Plan) + 4 * jobs + 255) / 256 * 256; }

// Staged tiles of one launch.
int64_t staged_bytes(const PagedArgs &c, const TcPlan &p)
{
    return std::min((int64_t)c.B * c.Hkv * p.pair_bytes, std::max(kStageBytes, p.pair_bytes));
}

cudaError_t stage(const PagedArgs &c, const ChunkArgs &x, const TcPlan &p, int pair0, int pairs, bool weights, void *ws,
                  const uint8_t *channels, cudaStream_t s)
{
    const StageArgs a{static_cast<uint8_t *>(ws), channels, p.tiles, pair0};
    const dim3 grid(p.tiles, pairs);
    if (c.fmt)
        return launch_stage_fp8(c, x, a, weights, grid, s);
    return c.bits == 2 ? launch_stage_2(c, x, a, weights, grid, s) : launch_stage_4(c, x, a, weights, grid, s);
}

TcArgs tc_args(const TcPlan &p, int pairs_at, void *ws, const uint8_t *channels)
{
    TcArgs d{};
    d.tiles = static_cast<const uint8_t *>(ws);
    d.channels = channels;
    d.tiles_per_pair = p.tiles;
    d.pair0 = pairs_at;
    d.S = p.splits;
    d.rows = p.row_tiles * kRows;
    return d;
}

}  // namespace

// Both bounds only grow with max_new and max_cached.
size_t long_attention_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    const TcPlan p = tc_plan(c, max_new, max_cached, false);
    const int64_t all = (int64_t)c.B * c.Hkv;
    return (size_t)(staged_bytes(c, p) + channel_bytes(all) + plan_bytes(all * p.row_tiles)) +
           (size_t)2 * kTcBlocks * kRows * (kHeadDim + 2) * 4;
}

// The plan counts in 32 bits.
bool long_attention_fits(const PagedArgs &c, int max_new, int max_cached)
{
    const TcPlan p = tc_plan(c, max_new, max_cached, false);
    return (int64_t)p.pairs * p.row_tiles <= INT_MAX / (kJobUnits + 2ll * p.tiles);
}

size_t long_weights_bytes(const PagedArgs &c, int max_new, int max_cached)
{
    const TcPlan p = tc_plan(c, max_new, max_cached, true);
    const int64_t all = (int64_t)c.B * c.Hkv, one = sum_bytes(c, all), rows = row_tiles_of(c, max_new);
    const int64_t sums = std::min(one * rows, std::max(kSumBytes, one));
    return (size_t)staged_bytes(c, p) + (size_t)sums + (size_t)(all * rows + kPartBlocks) * kRows * 16;
}

cudaError_t launch_long_attention(const PagedArgs &c, const ChunkArgs &x, __half *out, void *ws, cudaStream_t s,
                                  int *launches)
{
    const TcPlan p = tc_plan(c, x.max_new, x.max_cached, false);
    const int all = c.B * c.Hkv, most_jobs = p.pairs * p.row_tiles;
    uint8_t *channels = static_cast<uint8_t *>(ws) + p.pair_bytes * p.pairs;
    Plan *plan = reinterpret_cast<Plan *>(channels + channel_bytes(p.pairs));
    float *o = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(plan) + plan_bytes(most_jobs));
    auto kernel = x.cap_log2 == 0.0f ? tc_kernel<0> : x.cap_small ? tc_kernel<1> : tc_kernel<2>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess)
        return e;
    const int blocks = std::min(sms, kTcBlocks);
    for (int p0 = 0; p0 < all; p0 += p.pairs) {
        const int pairs = std::min(p.pairs, all - p0);
        TcArgs d = tc_args(p, p0, ws, channels);
        d.plan = plan;
        d.row_tiles = p.row_tiles;
        d.jobs = pairs * p.row_tiles;
        d.out = out;
        d.o = o;
        d.ml = reinterpret_cast<float2 *>(o + (int64_t)2 * kTcBlocks * kRows * kHeadDim);
        prepare_kernel<<<1 + (c.fmt ? 0 : pairs), 256, 0, s>>>(c, x, p0, pairs, d.jobs, p.row_tiles, blocks, channels, plan);
        e = stage(c, x, p, p0, pairs, false, ws, channels, s);
        if (e != cudaSuccess)
            return e;
        e = launch_dependent(kernel, dim3(blocks), kTcThreads, kTcSmem, s, c, x, d);
        if (e == cudaSuccess)
            e = launch_dependent(tc_join_kernel, dim3(blocks, kRows / kJoinRows), 256, 0, s, c, x, d);
        *launches += 4;
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_long_weights(const PagedArgs &c, const ChunkArgs &x, float *weights, void *ws, cudaStream_t s,
                                int *launches)
{
    const TcPlan p = tc_plan(c, x.max_new, x.max_cached, true);
    const int all = c.B * c.Hkv, unit = weigh_unit(c);
    float *ls = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.pair_bytes * p.pairs);
    const int cap = x.cap_log2 == 0.0f ? 0 : x.cap_small ? 1 : 2;
    auto kernel = unit == 16 ? (cap == 0 ? tc_weigh_kernel<0, 16> : cap == 1 ? tc_weigh_kernel<1, 16> : tc_weigh_kernel<2, 16>)
                             : (cap == 0 ? tc_weigh_kernel<0, 32> : cap == 1 ? tc_weigh_kernel<1, 32> : tc_weigh_kernel<2, 32>);
    cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWeighSmem);
    if (e != cudaSuccess)
        return e;
    for (int p0 = 0; p0 < all; p0 += p.pairs) {
        const int pairs = std::min(p.pairs, all - p0);
        e = stage(c, x, p, p0, pairs, true, ws, nullptr, s);
        *launches += 1;
        TcArgs d = tc_args(p, p0, ws, nullptr);
        d.unit = unit;
        d.units = (int)((int64_t)c.columns * c.G / unit);
        d.ls = ls;
        d.ml = reinterpret_cast<float2 *>(ls + ((int64_t)p.pairs * d.rows * d.units + 1) / 2 * 2);
        const float *ml = reinterpret_cast<const float *>(d.ml);
        for (int64_t r0 = 0; e == cudaSuccess && r0 < (int64_t)x.max_new * c.g; r0 += d.rows) {
            d.row0 = (int)r0;
            e = launch_dependent(kernel, dim3(p.row_tiles, pairs, p.splits), kWeighThreads, kWeighSmem, s, c, x, d);
            if (e == cudaSuccess)
                e = launch_weigh(c, x, Parts{ml, ml + 1, nullptr, 2, 2 * p.splits, p0, d.row0, d.rows}, ls, unit, d.units,
                                 weights, pairs, s);
            *launches += 2;
        }
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace kivi
