// experts.cu -- the experts' products over the expert-contiguous rows and their gradients
// (ep_expert_matmul, ep_expert_matmul_dgrad, ep_expert_matmul_wgrad).
//
// One kernel carries the three on the fifth-generation tensor cores. A pair of blocks (a
// cluster of two, one block per SM) computes a tile D[256 features x n rows], n a multiple
// of 32 up to 256:
//
//            D[feature, row]                    M operand (features)   N operand (rows)
//   forward  y^T  = w x^T, reduced over K       w, K contiguous        x, K contiguous
//   dgrad    dx^T = w^T dy^T, reduced over N    w, M contiguous        dy, N contiguous
//   wgrad    dw^T = x^T dy, reduced over rows   x, M contiguous        dy, N contiguous
//
// The features are the instruction's fixed 256 rows and the tokens its free dimension,
// because experts have few and uneven rows: an expert's c rows are cut into ceil(c / 256)
// equal tiles and each runs with just the width it needs, where the other way round a tile
// would be padded to 256 rows. Each block stages its 128 feature rows and half of the token
// rows per step of the reduction (128 bytes wide), so a token row that both blocks multiply is
// staged once.
//
// e4m3 (forward only) is scaled per row and 128 columns and, the weights, per 128 x 128, so the
// product of one 128-wide step cannot stay in the tensor core's accumulator: every step's D goes
// to registers as acc += D * (x_scale * w_scale). Tiles of more than 128 rows have the rows as
// M, D[256 rows x n features]: a lane is a row and needs one scale for each of the tile's two
// weight blocks. With a row a column every thread needs all the columns' scales from shared
// memory, whose bandwidth the operands already take (a step's 32 KiB are written and read once
// in the 512 cycles of its mma): 256 experts of 256 rows, 4096 x 7168, took 1733 us that way and
// take 1480 us this way. Tiles of up to 128 rows are turned across all the same, D[256 features
// x n rows], where a step costs little more than its weights' 16 KiB into the SM: with 4 rows an
// expert 1329 us the one way and 1100 us the other.
//
// What bounds it: bf16 the tensor cores from some 500 rows an expert on (dense 8192^3: 570 us,
// 1930 TFLOP/s, as cuBLAS here) and with fewer the 64 bytes a clock that come into an SM, since
// a step of n = 192 columns brings 28 KiB for 384 cycles of mma; wgrad its output, 4.0 TB/s
// being what this memory takes in writes alone; e4m3 with few rows the weights' way from memory
// and with many the sums, of which a step has 256 cycles to its mma's 512. A lone tile is bound by
// its two SMs' 64 bytes a clock as well, so a handful of tiles with a long reduction is cut along
// it: a cluster of up to four pairs shares a tile, and its parts' sums are read from the others'
// shared memory and added up in a fixed order (kSharedSteps).
//
// Warps: the epilogue's 8 (e4m3: 16), the producer, which walks the tiles, publishes them to
// the others and feeds TMA, one that issues the mma (in the pair's first block), and two helpers
// that load row scales (e4m3) or sum the bias's gradient (wgrad). There are two accumulators in tensor memory (e4m3 across: four), so
// a tile's epilogue, or a step's sums, run under the next one's mma. One thread issues a tile's
// loads and one its mma without leaving its loop: with a branch to lane 0 in every step the
// issue alone took 530 cycles a step. Blocks walk the tiles of all experts in a fixed order
// (persistent, one pair per two SMs); the experts' counts are read from device memory, 32 at a
// time, by the producer itself.
#include <cuda.h>

#include <atomic>

#include "epd_math.cuh"
#include "epd_tcgen05.cuh"

namespace epd {
namespace {

enum { kForward = 0, kDgrad = 1, kWgrad = 2 };

// e4m3 has its sums in registers: 16 epilogue warps of 64 columns each, 16 read at a time. (Eight
// warps of 128 columns: 1795 us at the shape above. 32 columns at a time, or 16 with the next 16
// read ahead, spill: 1915 and 3843 us.)
template <bool FP8>
constexpr int kEpiWarpsOf = FP8 ? 16 : 8;
constexpr int kHelpers = 2;                     // warps that load row scales (e4m3) or sum dbias (wgrad)
template <int MODE, bool FP8>
constexpr int kThreadsOf = (kEpiWarpsOf<FP8> + 2 + (FP8 || MODE == kWgrad ? kHelpers : 0)) * 32;
constexpr int kTileRows = 256;                  // most token rows (wgrad: output rows) of a tile
constexpr int kAcrossRows = 128;                // e4m3: most rows of a tile with the features as M
constexpr int kOperandBytes = 128 * 128;        // 128 rows of 128 bytes: one operand of a stage
constexpr int kStageBytes = 2 * kOperandBytes;
// Staging rows per epilogue warp, 64 bytes each and 80 apart. e4m3 has twice the warps and, with
// half the rows each, room for a sixth stage (few rows an expert: 1130 us with five, 1110 with six).
template <bool FP8>
constexpr int kStagedOf = FP8 ? 16 : 32;
template <bool FP8>
constexpr int kStagingOf = kStagedOf<FP8> * 80;
constexpr int kTailBytes = 768;                 // published tiles and barriers
constexpr int kScaleGroup = 4;                  // reduction steps per group of staged scales
constexpr int kScaleBytes = 2 * kScaleGroup * 128 * 8;  // a row's with each of the tile's two weight blocks
constexpr int kRing = 4;                        // tiles published ahead
constexpr int kCuts = 18;                       // wgrad's boxes: 64, 32, 16 and 1 to 15 rows
constexpr int kGroupTiles = 8;                  // row tiles that share a pass over the features

// n / d rounded up, for n up to INT32_MAX.
__host__ __device__ constexpr int ceil_div(int n, int d) { return (int)(((uint32_t)n + (uint32_t)d - 1) / (uint32_t)d); }

constexpr int kStages = 6;

// A wait's limit, and what each step of the longest reduction adds to it: a wait may be for a whole
// tile, whose steps take 0.1 to 0.5 us each (wgrad of 2^31 rows of one expert: 2^25 steps).
constexpr uint64_t kWaitNs = 2000000000, kWaitStepNs = 2000;
constexpr uint64_t kDrainNs = 1000000000;  // of a wait for what is in flight once another has run out
constexpr uint32_t kConsumed = 0xffffffff;

// Where few tiles leave most SMs idle, up to four pairs share a tile's reduction, which costs
// 1 to 2 us for the larger cluster and the sums' way between blocks, and takes 0.16 us a step
// (e4m3 0.24) off as many steps as the others do. It is done from kSharedSteps / parts steps on,
// and, where a tile has many columns to exchange, from kSharedStepsWide on. One expert, 512 features,
// in four parts and in one, us, bf16:
//      16 rows: K = 1024  6.4  5.7   1536  6.5  6.9   4096  8.4  13.4
//     256 rows: K = 1536 11.9 11.1   2048 12.1 13.1
// in two and in one (64 rows, 7168 features): K = 2048 10.9 and 10.3, 3200 13.6 and 14.1. e4m3:
//      16 rows: K = 1536  7.2  6.6   2048  7.2  7.4   4096  8.1 11.7
//     256 rows: K = 2048 15.1 12.0   3584 16.7 16.7
// in two: K = 3200 11.1 and 11.1, 4096 11.8 and 12.8; with 256 rows, 4096 features, K = 3200 16.6 and
// 16.2, 4096 17.8 and 19.0. wgrad, 256 x 256, rows = 1536 12.7 and 10.5, 4096 13.6 and 21.0.
// How many columns there are the host judges by the buffer's rows. In one that is not full the tiles
// are fewer or narrower than that, and sharing pays all the same (16 rows of 4096, K = 4096, 512
// features: 10.6 and 13.8, e4m3 9.1 and 11.3); wgrad's steps, which the rows are, the kernel looks at
// itself (256 x 256, 16 rows of 4096: 4.7, and 9.2 where that is not done).
template <bool FP8>
constexpr int kSharedSteps = FP8 ? 64 : 96;
template <bool FP8>
constexpr int kSharedStepsWide = FP8 ? 28 : 32;
constexpr int kWideRows = 128;  // more columns of D on average than these are many
template <bool FP8>
__host__ __device__ constexpr bool worth_sharing(int64_t columns, int64_t steps, int parts) {
    return columns > kWideRows ? steps >= kSharedStepsWide<FP8> : steps * parts >= kSharedSteps<FP8>;
}

template <bool FP8>
constexpr int kSmemOf = kStages * kStageBytes + kEpiWarpsOf<FP8> * kStagingOf<FP8> + (FP8 ? kScaleBytes : 0) + kTailBytes;

struct ExpertArgs {
    epd_expert_rows_t rows;
    int K, N;  // features in and out of the product
    int act;
    const float *x_scale, *w_scale;
    int64_t srow, scol, sexp;
    int scale_vec;  // four consecutive scales of a row can be loaded at once
    const float *bias;
    const uint8_t *residual, *preact_in;
    uint8_t *y, *preact;
    const uint8_t *dy;  // wgrad: the rows that dbias sums
    float *dbias;
    int32_t *status;
    uint64_t wait_ns;  // limit of a wait
    int stall;         // a test's: the first tile, of each pair, whose mma are left out (-1: none)
};

// The rows of expert e as they may be read: clipped, with an error where they do not fit.
__device__ __forceinline__ void expert_region(const epd_expert_rows_t &r, int e, int &start, int &count,
                                              int32_t *status) {
    count = r.tokens_per_expert[e];
    const int64_t at = r.expert_start_loc ? (int64_t)r.expert_start_loc[e] : e * r.rows_per_expert;
    if (count < 0 || at < 0) {
        report(status, EPD_ERR_INVALID_ARG);
        count = 0;
    }
    int64_t room = r.capacity_rows - at;
    if (!r.expert_start_loc && room > r.rows_per_expert) room = r.rows_per_expert;
    if (count > 0 && count > room) {
        report(status, EPD_ERR_CAPACITY);
        count = room > 0 ? (int)room : 0;
    }
    start = count > 0 ? (int)at : 0;
}

// The operands' TMA maps. wgrad's reduction runs over a region's rows, whose last step may hold
// fewer than 64: it is loaded in boxes of 32, 16 and 1 to 15 rows, and what is missing to a
// multiple of 16 (one mma's reduction) in a box past the end of the buffer, which reads as zero.
// The other rows of the buffer are never multiplied. A box costs some 33 cycles whatever its
// height (64 experts of 380 rows: 340 us with heights that are powers of two, which take
// five cuts where these take three).
constexpr int cut_rows(int i) { return i < 3 ? 64 >> i : i - 2; }

// Token rows (forward, dgrad), a multiple of 16 up to 128, come in boxes of 128, 64, 32 and 16:
// few boxes, and no row that is not needed. The forward weights' maps are one of 128 rows and,
// gated, one of 64 gate rows and the same features' 64 up rows.
template <int MODE>
struct Maps {
    static constexpr int kM = MODE == kWgrad ? kCuts : MODE == kForward ? 2 : 1, kN = MODE == kWgrad ? kCuts : 4;
    CUtensorMap m[kM], n[kN];
};

// One tile of the work: `rows` valid columns of D from row `row0` (a token row; for wgrad an
// output row of the expert's gradient), n of them computed; features from feat0.
struct alignas(16) Tile {
    int e, start, count;  // e = -1 past the last tile
    int feat0, row0, rows, n;
    int steps;  // of the reduction
    int across; // e4m3: the features are the M operand
    int step0;  // first step of this pair's
    int part, parts;  // of the reduction: this pair's, and how many pairs share it
};

// The producer's tiles, as the other warps of the block get them: a ring in shared memory.
struct Ring {
    const Tile *slots;
    uint32_t full, empty;
    int at = 0;
    uint32_t parity = 0;

    // Waits for the next tile. The slot stays this warp's until drop().
    __device__ __forceinline__ bool next(bool &ok, const ExpertArgs &p) {
        ok = mbar_wait_pipe(full + 8 * at, parity, p.wait_ns);
        return ok && slots[at].e >= 0;
    }
    __device__ __forceinline__ const Tile &tile() const { return slots[at]; }
    __device__ __forceinline__ void drop() {
        __syncwarp();
        if (elect_one()) mbar_arrive_own(empty + 8 * at);
        if (++at == kRing) at = 0, parity ^= 1;
    }
};

// Walks the tiles of one pair, a warp together: lane l holds expert batch + l, and a tile's
// expert is found by a ballot over the running tile counts.
template <int MODE, int STEP, bool FP8>
struct Walker {
    const ExpertArgs &p;
    int lane, feat_tiles, feat_step;
    int batch = -32, before = 0, in_batch = 0;
    int count = 0, start = 0, upto = 0;

    __device__ Walker(const ExpertArgs &args, int feat_step_) : p(args), feat_step(feat_step_) {
        lane = threadIdx.x & 31;
        const int features = MODE == kForward ? p.N : p.K;
        feat_tiles = ceil_div(features, feat_step);
    }

    __device__ bool next(int tile, Tile &t) {
        int local, row_tiles;
        if (MODE == kWgrad) {
            row_tiles = ceil_div(p.N, kTileRows);
            const int per = row_tiles * feat_tiles;
            t.e = tile / per;
            if (t.e >= p.rows.num_experts) return false;
            local = tile - t.e * per;
            expert_region(p.rows, t.e, t.start, t.count, p.status);
        } else {
            while (tile >= before + in_batch) {
                before += in_batch;
                batch += 32;
                in_batch = 0;
                if (batch >= p.rows.num_experts) return false;
                count = start = 0;
                if (batch + lane < p.rows.num_experts)
                    expert_region(p.rows, batch + lane, start, count, p.status);
                upto = ceil_div(count, kTileRows) * feat_tiles;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                in_batch = __shfl_sync(0xffffffffu, upto, 31);
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, tile - before < upto)) - 1;
            t.e = batch + src;
            t.count = __shfl_sync(0xffffffffu, count, src);
            t.start = __shfl_sync(0xffffffffu, start, src);
            row_tiles = ceil_div(t.count, kTileRows);
            local = tile - before - (__shfl_sync(0xffffffffu, upto, src) - row_tiles * feat_tiles);
        }
        // Groups of row tiles pass over the features together, the row tiles fastest, so that the
        // tiles in flight share both operands in L2. Which row tile comes first changes from one
        // feature tile to the next: an expert's last row tile is narrow, and in a fixed order with
        // two of them every second pair of blocks would get nothing else (e4m3, 256 experts of 272
        // rows: 2807 us).
        const int group = local / (kGroupTiles * feat_tiles);
        const int rest = local - group * kGroupTiles * feat_tiles;
        const int width = min(kGroupTiles, row_tiles - group * kGroupTiles);
        const int ft = rest / width;
        const int rt = group * kGroupTiles + (rest - ft * width + __popc(ft)) % width;
        t.feat0 = ft * feat_step;
        const int total = MODE == kWgrad ? p.N : t.count;
        // equal tiles of the least width; e4m3: full tiles of rows, and a last one of at most 128
        // turned across
        const int each = FP8 ? kTileRows : (ceil_div(total, row_tiles) + 31) & ~31;
        t.row0 = rt * each;
        t.rows = min(each, total - t.row0);
        t.across = !FP8 || t.rows <= kAcrossRows;
        if (t.across)
            t.n = t.rows > 0 ? (t.rows + 31) & ~31 : 32;
        else  // feat_step features, gated: and their up
            t.n = feat_step == 128 ? 256 : (min(256, p.N - t.feat0) + 31) & ~31;
        const int red = MODE == kForward ? p.K : MODE == kDgrad ? p.N : t.count;
        t.steps = ceil_div(red, STEP);
        t.step0 = t.part = 0;
        t.parts = 1;
        return true;
    }

    // Leaves part `part` of `parts` of the tile's reduction, in whole groups of staged scales.
    __device__ void cut(Tile &t, int part, int parts) const {
        constexpr int kUnit = FP8 ? kScaleGroup : 1;
        const int units = (t.steps + kUnit - 1) / kUnit;
        t.step0 = part * units / parts * kUnit;
        t.steps = min(t.steps, (part + 1) * units / parts * kUnit) - t.step0;
        t.part = part;
        t.parts = parts;
    }
};

// ---------------------------------------------------------------------------- epilogue
// A warp's 32 features x 32 columns of D are held as fragments f[h][4u + 2i + b]: feature
// 16h + 8b + lane / 4, column 8u + 4i + lane % 4. Packed to bf16 in pairs over i they are 8 x 8
// blocks for stmatrix, whose row j is column 8u + 4 (j % 2) + j / 2 of D; it turns them over, so
// that rows of 32 (a gated product: 16) features lie together and leave for memory 16 bytes a
// lane. In a gated product a block's 128 features are 64 gate features (quadrants 0 and 1) and
// the same features' up (quadrants 2 and 3).
using Frag = float[2][16];

constexpr int kPitch = 80;  // bytes per staged row of 64: eight rows fall in different banks

// Row and 16-byte part of this lane in pass `it` over 32 rows of 64 bytes: the two rows of a
// quarter warp are four apart, which keeps them in different banks.
__device__ __forceinline__ int lane_row(int it) {
    const int lane = threadIdx.x & 31;
    return it * 8 + (lane >> 3) + (lane & 4);
}

// Column of D within its eight that row j of a block is.
__device__ __forceinline__ int block_column(int j) { return 4 * (j & 1) + (j >> 1); }

template <int ACT>
__device__ __forceinline__ void apply(Frag &f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) f[h][r] = activate<ACT>(f[h][r]);
}

// Writes the first `rows` of 32 rows (columns of D), `parts` of their four 16-byte parts each, to
// at + row * pitch, STAGED rows at a time.
template <int STAGED>
__device__ __forceinline__ void put_frag(uint32_t stage, const Frag &f, uint8_t *at, int64_t pitch, int rows,
                                         int parts) {
    const int lane = threadIdx.x & 31, part = lane & 3;
    at += part * 16;
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += STAGED) {
        __syncwarp();
#pragma unroll
        for (int u = r0 / 8; u < (r0 + STAGED) / 8; ++u)
            stmatrix_t(stage + (u * 8 - r0 + block_column(lane & 7)) * kPitch + (lane >> 3) * 16,
                       pack2_bf16(f[0][4 * u], f[0][4 * u + 2]), pack2_bf16(f[0][4 * u + 1], f[0][4 * u + 3]),
                       pack2_bf16(f[1][4 * u], f[1][4 * u + 2]), pack2_bf16(f[1][4 * u + 1], f[1][4 * u + 3]));
        __syncwarp();
#pragma unroll
        for (int it = 0; it < STAGED / 8; ++it) {
            const int row = lane_row(it);
            const uint4 v = lds16(stage + row * kPitch + part * 16);
            if (part < parts && r0 + row < rows) st16(at + (r0 + row) * pitch, v);
        }
    }
}

// The same for 16 features, a half of the warp's.
template <int STAGED>
__device__ __forceinline__ void put_half(uint32_t stage, const float (&f)[16], uint8_t *at, int64_t pitch, int rows, int parts) {
    constexpr int kHalfPitch = 48;
    const int lane = threadIdx.x & 31, part = lane & 1;
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += STAGED) {
        __syncwarp();
#pragma unroll
        for (int u = r0 / 8; u < (r0 + STAGED) / 8; u += 2)
            stmatrix_t(stage + ((u + (lane >> 4)) * 8 - r0 + block_column(lane & 7)) * kHalfPitch + ((lane >> 3) & 1) * 16,
                       pack2_bf16(f[4 * u], f[4 * u + 2]), pack2_bf16(f[4 * u + 1], f[4 * u + 3]),
                       pack2_bf16(f[4 * u + 4], f[4 * u + 6]), pack2_bf16(f[4 * u + 5], f[4 * u + 7]));
        __syncwarp();
#pragma unroll
        for (int it = 0; it < STAGED / 16; ++it) {
            const int row = it * 16 + (lane >> 1);
            const uint4 v = lds16(stage + row * kHalfPitch + part * 16);
            if (part < parts && r0 + row < rows) st16(at + (r0 + row) * pitch + part * 16, v);
        }
    }
}

// 32 rows of 64 bytes of a bf16 operand, fetched ahead of their use and then turned into
// fragments by way of the staging rows. What lies outside is zero.
struct Ahead {
    uint4 v[4];

    __device__ __forceinline__ void fetch(const uint8_t *at, int64_t pitch, int rows, int parts) {
        const int part = threadIdx.x & 3;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int row = lane_row(it);
            v[it] = part < parts && row < rows ? ld_stream16(at + row * pitch + part * 16) : make_uint4(0, 0, 0, 0);
        }
    }

    // Rows r0 .. r0 + STAGED - 1 into the staging rows.
    template <int STAGED>
    __device__ __forceinline__ void stage_rows(uint32_t stage, int r0) const {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < STAGED / 8; ++it)
            sts16(stage + lane_row(it) * kPitch + (threadIdx.x & 3) * 16, v[r0 / 8 + it]);
        __syncwarp();
    }

    template <int STAGED>
    __device__ __forceinline__ void turn(uint32_t stage, uint32_t (&w)[2][8]) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += STAGED) {
            stage_rows<STAGED>(stage, r0);
#pragma unroll
            for (int u = r0 / 8; u < (r0 + STAGED) / 8; ++u)
                ldmatrix_t(stage + (u * 8 - r0 + block_column(lane & 7)) * kPitch + (lane >> 3) * 16, w[0][2 * u],
                           w[0][2 * u + 1], w[1][2 * u], w[1][2 * u + 1]);
        }
    }
};

// Sixteen values a lane to the same lane of the pair's other warp, by way of the staging rows.
template <int STAGED>
__device__ __forceinline__ bool swap_half(uint32_t mine, uint32_t other, uint32_t bar, const float (&out)[16], float (&in)[16],
                                          const ExpertArgs &p) {
    constexpr int kAtOnce = STAGED / 8;  // of the sixteen's four parts: 512 bytes each
    const uint32_t at = (threadIdx.x & 31) * 16;
    bool ok = true;
#pragma unroll
    for (int p0 = 0; p0 < 4; p0 += kAtOnce) {
        __syncwarp();
#pragma unroll
        for (int i = p0; i < p0 + kAtOnce; ++i)
            sts16(mine + (i - p0) * 512 + at,
                  make_uint4(__float_as_uint(out[4 * i]), __float_as_uint(out[4 * i + 1]),
                             __float_as_uint(out[4 * i + 2]), __float_as_uint(out[4 * i + 3])));
        mbar_arrive_own(bar);  // of 64: the barrier's two phases, written and read, end as they began
        ok = ok && mbar_wait_pipe(bar, 0, p.wait_ns);
#pragma unroll
        for (int i = p0; i < p0 + kAtOnce; ++i) {
            const float4 v = lds16f(other + (i - p0) * 512 + at);
            in[4 * i] = v.x, in[4 * i + 1] = v.y, in[4 * i + 2] = v.z, in[4 * i + 3] = v.w;
        }
        mbar_arrive_own(bar);
        ok = ok && mbar_wait_pipe(bar, 1, p.wait_ns);
    }
    return __all_sync(0xffffffffu, ok);
}

// A reduction that several pairs of a cluster share: every pair finishes a part of the tile's
// columns. The others' 32 sums a lane and chunk it leaves in its own shared memory (the stages,
// which nothing fills any more), and fetches what they have left for it. (All by the first pair:
// 256 rows, K = 2048: 14.0 us for 12.1.) e4m3 does it all by the first pair: its sums are in
// registers already, and the code that keeps some and gives others away spills (16 rows, K = 7168,
// SwiGLU: 14.8 us for 13.1).
template <typename F>
__device__ __forceinline__ void park(uint32_t at, F sum) {
    at += (threadIdx.x & 31) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sts16(at + i * 512, make_uint4(__float_as_uint(sum(4 * i)), __float_as_uint(sum(4 * i + 1)),
                                       __float_as_uint(sum(4 * i + 2)), __float_as_uint(sum(4 * i + 3))));
}

// Adds the other parts' sums, in the parts' order.
template <typename F>
__device__ __forceinline__ void add_parked(uint32_t at, const Tile &t, F sum) {
    at += (threadIdx.x & 31) * 16;
    const int rank = cluster_ctarank() & 1;
    for (int s = 0; s < t.parts; ++s) {
        if (s == t.part) continue;
        const uint32_t from = map_to_rank(at, 2 * s + rank);
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = ld_cluster16f(from + (i0 + i) * 512);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * (i0 + i);
                sum(r) += v[i].x, sum(r + 1) += v[i].y, sum(r + 2) += v[i].z, sum(r + 3) += v[i].w;
            }
        }
    }
}

// Arrives on barrier `bar` of the other parts' blocks of this rank, for a warp. (What it needs is read
// where it is needed: e4m3 has no registers to keep it in.)
__device__ __forceinline__ void tell_others(uint32_t bar, const Tile &t) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (lane < t.parts && lane != t.part) mbar_release_cluster(map_to_rank(bar, 2 * lane + (cluster_ctarank() & 1)));
}

// The same for the first pair's alone.
__device__ __forceinline__ void tell_first(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_release_cluster(map_to_rank(bar, cluster_ctarank() & 1));
}

// This warp's sums are left for the others, and theirs are there.
__device__ __forceinline__ bool exchange(uint32_t parked, const Tile &t, const ExpertArgs &p) {
    tell_others(parked, t);
    return __all_sync(0xffffffffu, mbar_wait_pipe<true>(parked, 0, p.wait_ns)) != 0;
}

// Element r of fragments f[h] in the words that Ahead::turn gives.
__device__ __forceinline__ float element(const uint32_t (&w)[8], int r) {
    const uint32_t v = w[(r >> 2) * 2 + (r & 1)];
    return r & 2 ? hi_bf16(v) : lo_bf16(v);
}

// A warp's share of a tile's output.
template <int MODE, bool GATED, int STAGED>
struct Output {
    static constexpr bool kHalf = GATED && MODE == kForward;
    const ExpertArgs &p;
    uint32_t stage, other; // staging rows; a gated product's: of the warp with the other half
    uint32_t bar;          // for the two of them
    bool ok = true;
    int up;                // this warp has up features
    int feat, parts;       // first feature of the warp, and how many octets of them exist
    int rows;              // of the tile
    int64_t pitch;         // bytes between output rows
    int64_t row;           // first row of the tile in the row buffers (wgrad: in dw)
    float bias[2][2];      // of features 16h + 8b + lane / 4
    Ahead a, b;            // the residual, or dgrad's pre-activations (b: their up part)

    __device__ Output(const ExpertArgs &args, uint32_t staging, uint32_t bars, int warp) : p(args) {
        stage = staging + warp * STAGED * kPitch;
        other = staging + (warp ^ 2) * STAGED * kPitch;
        up = kHalf ? (warp >> 1) & 1 : 0;
        bar = bars + 8 * ((warp >> 2) * 2 + (warp & 1));
    }

    __device__ __forceinline__ void begin(const Tile &t, int rank, int quadrant) {
        const int lane = threadIdx.x & 31;
        const int features = MODE == kForward ? p.N : p.K;
        feat = t.feat0 + (kHalf ? rank * 64 + (quadrant & 1) * 32 : rank * 128 + quadrant * 32);
        parts = max(0, min(4, (features - feat) / 8));
        rows = t.rows;
        pitch = (int64_t)features * 2 * (MODE == kDgrad && GATED ? 2 : 1);
        row = (MODE == kWgrad ? (int64_t)t.e * p.N : t.start) + t.row0;
        if (MODE == kForward && p.bias) {
            const float *at = p.bias + (int64_t)t.e * p.N * (GATED ? 2 : 1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int f = feat + 16 * h + 8 * o + lane / 4;
                    bias[h][o] = f < features ? at[f + (up ? p.N : 0)] : 0.0f;
                }
        }
    }

    __device__ __forceinline__ void fetch(int col0) {
        if (MODE == kForward && p.residual)
            a.fetch(p.residual + (row + col0) * pitch + feat * 2, pitch, rows - col0, parts);
        if (MODE == kDgrad && p.act != EPD_ACT_NONE) {
            const uint8_t *z = p.preact_in + (row + col0) * pitch + feat * 2;
            a.fetch(z, pitch, rows - col0, parts);
            if (GATED) b.fetch(z + (int64_t)p.K * 2, pitch, rows - col0, parts);
        }
    }

    template <int ACT>
    __device__ __forceinline__ void times_slope(Frag &f, const uint32_t (&z)[2][8]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 16; ++r) f[h][r] *= activate_grad<ACT>(element(z[h], r));
    }

    // Columns col0 .. col0 + 31; `next` are fetched ahead if there are any.
    __device__ __forceinline__ void finish(Frag &f, int col0, int next) {
        uint8_t *at = p.y + (row + col0) * pitch + feat * 2;
        const int left = rows - col0;
        if (MODE == kWgrad) {
            put_frag<STAGED>(stage, f, at, pitch, left, parts);
            return;
        }
        if (MODE == kDgrad) {
            if (p.act == EPD_ACT_NONE) {
                put_frag<STAGED>(stage, f, at, pitch, left, parts);
                return;
            }
            uint32_t z[2][8];
            a.turn<STAGED>(stage, z);
            if (GATED) {
                uint32_t u[2][8];
                b.turn<STAGED>(stage, u);
                if (next < rows) fetch(next);
                Frag up;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float g = element(z[h], r), w = element(u[h], r);
                        const float s = fast_sigmoid(g);
                        // what has no slope (s = 0) is 0 whatever else there is: the products of d
                        // with the pre-activations, which may overflow, come last
                        up[h][r] = f[h][r] * (g * s);
                        f[h][r] = f[h][r] * (w * (s * (1.0f + g * (1.0f - s))));
                    }
                put_frag<STAGED>(stage, f, at, pitch, left, parts);
                put_frag<STAGED>(stage, up, at + (int64_t)p.K * 2, pitch, left, parts);
                return;
            }
            if (next < rows) fetch(next);
            if (p.act == EPD_ACT_RELU)
                times_slope<EPD_ACT_RELU>(f, z);
            else if (p.act == EPD_ACT_SILU)
                times_slope<EPD_ACT_SILU>(f, z);
            else
                times_slope<EPD_ACT_GELU>(f, z);
            put_frag<STAGED>(stage, f, at, pitch, left, parts);
            return;
        }
        if (p.bias) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 16; ++r) f[h][r] += bias[h][r & 1];
        }
        if (p.preact) {
            const int64_t zp = (int64_t)p.N * 2 * (GATED ? 2 : 1);
            put_frag<STAGED>(stage, f, p.preact + (row + col0) * zp + ((int64_t)feat + (up ? p.N : 0)) * 2, zp, left, parts);
        }
        if (GATED) {
            // the gate warp finishes the first 16 features and the up warp the last: each sends
            // the other what it needs for them
            float in[16];
            if (up) {
                ok = ok && swap_half<STAGED>(stage, other, bar, f[0], in, p);
#pragma unroll
                for (int r = 0; r < 16; ++r) f[1][r] = in[r] * fast_sigmoid(in[r]) * f[1][r];
            } else {
                ok = ok && swap_half<STAGED>(stage, other, bar, f[1], in, p);
#pragma unroll
                for (int r = 0; r < 16; ++r) f[1][r] = f[0][r] * fast_sigmoid(f[0][r]) * in[r];
            }
            if (p.residual) {
                uint32_t z[2][8];
                a.turn<STAGED>(stage, z);
                if (next < rows) fetch(next);
#pragma unroll
                for (int r = 0; r < 16; ++r) f[1][r] += up ? element(z[1], r) : element(z[0], r);
            }
            put_half<STAGED>(stage, f[1], at + up * 32, pitch, left, max(0, min(2, parts - 2 * up)));
            return;
        }
        if (p.act == EPD_ACT_RELU) {
            apply<EPD_ACT_RELU>(f);
        } else if (p.act == EPD_ACT_SILU) {
            apply<EPD_ACT_SILU>(f);
        } else if (p.act == EPD_ACT_GELU) {
            apply<EPD_ACT_GELU>(f);
        }
        if (p.residual) {
            uint32_t z[2][8];
            a.turn<STAGED>(stage, z);
            if (next < rows) fetch(next);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 16; ++r) f[h][r] += element(z[h], r);
        }
        put_frag<STAGED>(stage, f, at, pitch, left, parts);
    }
};

// ---- e4m3: a lane is a row, f[c] its column c of 32.
__device__ __forceinline__ void put_rows(uint32_t stage, const float (&f)[32], uint8_t *at, int64_t pitch, int rows,
                                         int parts) {
    constexpr int kStaged = kStagedOf<true>;
    const int lane = threadIdx.x & 31, part = lane & 3;
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += kStaged) {
        __syncwarp();
        if (lane / kStaged == r0 / kStaged) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sts16(stage + lane % kStaged * kPitch + i * 16,
                      make_uint4(pack2_bf16(f[8 * i], f[8 * i + 1]), pack2_bf16(f[8 * i + 2], f[8 * i + 3]),
                                 pack2_bf16(f[8 * i + 4], f[8 * i + 5]), pack2_bf16(f[8 * i + 6], f[8 * i + 7])));
        }
        __syncwarp();
#pragma unroll
        for (int it = 0; it < kStaged / 8; ++it) {
            const int row = lane_row(it);
            const uint4 v = lds16(stage + row * kPitch + part * 16);
            if (part < parts && r0 + row < rows) st16(at + (r0 + row) * pitch + part * 16, v);
        }
    }
}

// Rows row0 .. row0 + 31 of the tile, columns col0 .. col0 + 31 of its two blocks of features
// (gated: of its gate features and of their up).
template <bool GATED>
__device__ __forceinline__ void finish_rows(const ExpertArgs &p, const Tile &t, int row0, int col0, uint32_t stage,
                                            float (&acc)[2][32]) {
    const int rows = t.rows - row0;
    const int64_t row = (int64_t)t.start + t.row0 + row0, NW = GATED ? 2 * (int64_t)p.N : p.N;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // features of this block: where they begin in a row of the pre-activations, and how many
        const int feat = t.feat0 + col0 + (GATED ? 0 : h * 128);
        const int64_t at = feat + (GATED && h ? (int64_t)p.N : 0);
        const int parts = max(0, min(4, (p.N - feat) / 8));
        float(&f)[32] = acc[h];
        if (p.bias) {
            const float *b = p.bias + t.e * NW + at;
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] += c < parts * 8 ? b[c] : 0.0f;
        }
        if (p.preact) put_rows(stage, f, p.preact + (row * NW + at) * 2, NW * 2, rows, parts);
        if (GATED) {
            if (h == 0) continue;
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] = acc[0][c] * fast_sigmoid(acc[0][c]) * f[c];
        } else if (p.act == EPD_ACT_RELU) {
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] = activate<EPD_ACT_RELU>(f[c]);
        } else if (p.act == EPD_ACT_SILU) {
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] = activate<EPD_ACT_SILU>(f[c]);
        } else if (p.act == EPD_ACT_GELU) {
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] = activate<EPD_ACT_GELU>(f[c]);
        }
        const int64_t pitch = (int64_t)p.N * 2;
        if (p.residual) {
            Ahead r;
            r.fetch(p.residual + row * pitch + (int64_t)feat * 2, pitch, rows, parts);
            constexpr int kStaged = kStagedOf<true>;
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += kStaged) {
                r.stage_rows<kStaged>(stage, r0);
                if (lane / kStaged != r0 / kStaged) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float e[8];
                    unpack8_bf16(lds16(stage + lane % kStaged * kPitch + i * 16), e);
#pragma unroll
                    for (int c = 0; c < 8; ++c) f[8 * i + c] += e[c];
                }
            }
        }
        put_rows(stage, f, p.y + row * pitch + (int64_t)feat * 2, pitch, rows, parts);
    }
}

// dbias[e, n] = the sum of the expert's rows of dy: a warp takes 8 LANES columns of an expert, a
// lane eight of them in every (32 / LANES)th row, and these parts are added up, all in a fixed
// order. The helper warps of wgrad do it beside the products, straight from memory: +12 us at 64
// experts of 384 rows, 4096 x 2048, where a kernel of its own after the product took 37. (Four warps
// a block: +20 us there; with 256 features, where the product is shorter than the sums, 130 us
// become 91.)
template <int LANES>
__device__ __forceinline__ void sum_bias(const ExpertArgs &p, int worker, int workers) {
    constexpr int kRows = 16, kParts = 32 / LANES;  // in flight a lane; rows at a time
    const int lane = threadIdx.x & 31, part = lane / LANES;
    const int groups = ceil_div(p.N, 8 * LANES);
    const int64_t pitch = (int64_t)p.N * 2;
    for (int64_t item = worker; item < (int64_t)groups * p.rows.num_experts; item += workers) {
        const int e = (int)(item / groups), n = (int)(item - (int64_t)e * groups) * (8 * LANES) + (lane % LANES) * 8;
        int start, rows;
        expert_region(p.rows, e, start, rows, p.status);
        const uint32_t count = rows;  // so that a row number past the last, of 2^31 at most, is one
        float sum[8] = {};
        const uint8_t *at = p.dy + ((int64_t)start * p.N + n) * 2;
        for (uint32_t r = part; n < p.N && r < count; r += kParts * kRows) {
            uint4 v[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                v[i] = r + kParts * i < count ? ld_stream16(at + (r + kParts * i) * pitch) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float f[8];
                unpack8_bf16(v[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += f[j];
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int o = LANES; o < 32; o *= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (part == 0 && n < p.N) {
            float *out = p.dbias + (int64_t)e * p.N + n;
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = sum[j];
        }
    }
}

// A wait of this cluster ran out, and nobody in it issues any more. What is in flight lands before
// its blocks go: loads write to their shared memory, matrix instructions to tensor memory. `issued`
// (shared memory of a pair's first block): the steps that each of its producers has issued loads of.
// A function of its own, so that its instructions are not among those that every call fetches (0.1 us).
__device__ __noinline__ void drain(uint32_t full, uint32_t drained, uint32_t issued, int mma_warp) {
    const int rank = (int)cluster_ctarank(), lead = rank & ~1;
    if (rank == lead && threadIdx.x == 0) {
        const uint32_t mine = lds4(issued), other = lds4(issued + 4);
        if (mine != kConsumed && other != kConsumed) {
            const uint32_t both = min(mine, other), any = max(mine, other);
            for (uint32_t i = any > kStages ? any - kStages : 0; i < any; ++i) {
                const uint32_t bar = full + 8 * (i % kStages);
                if (i >= both) mbar_arrive_own(bar);  // for the producer that did not get there
                mbar_wait_pipe(bar, i / kStages & 1, kDrainNs);
            }
        }
    }
    if (rank == lead && threadIdx.x / 32 == mma_warp) {
        if (elect_one()) mma_commit_pair(drained, (uint16_t)(3 << lead));
        __syncwarp();
    }
    if (threadIdx.x == 0) mbar_wait_pipe(drained, 0, kDrainNs);
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
}

template <int MODE, bool FP8, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kThreadsOf<MODE, FP8>, 1)
    expert_kernel(const __grid_constant__ Maps<MODE> maps, const ExpertArgs p) {
    constexpr bool kHalf = GATED && MODE == kForward;  // half of a block's 128 lanes are up features
    // accumulators: two of 256 columns; e4m3, which uses one a step, four of 128 where that is enough
    constexpr int kAccs = FP8 ? 4 : 2;
    constexpr int kEpiWarps = kEpiWarpsOf<FP8>;
    constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kHelperWarp = kEpiWarps + 2;
    constexpr int kStep = FP8 ? 128 : 64;              // reduction elements per stage
    constexpr int kFeatStep = kHalf ? 128 : 256;       // output features per pair
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *after = smem + kStages * kStageBytes;
    const uint32_t staging = smem_addr(after);
    after += kEpiWarps * kStagingOf<FP8>;
    float *scales = reinterpret_cast<float *>(after);
    if (FP8) after += kScaleBytes;
    Tile *slots = reinterpret_cast<Tile *>(after);
    after += kRing * sizeof(Tile);
    uint64_t *bars = reinterpret_cast<uint64_t *>(after);
    constexpr int kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + kAccs,
                  kScFull = kAccEmpty + kAccs, kScEmpty = kScFull + 2, kTileFull = kScEmpty + 2, kTileEmpty = kTileFull + kRing,
                  kSwap = kTileEmpty + kRing, kParked = kSwap + kEpiWarps / 2, kFetched = kParked + 1,
                  kDrained = kFetched + 1, kSlot = kDrained + 1, kFailed = kSlot + 1;
    static_assert((kFailed + 2) * 8 + kRing * sizeof(Tile) <= kTailBytes, "the barriers fit");
    const uint32_t base = smem_addr(smem), bar0 = smem_addr(bars);
    const uint32_t full = bar0, empty = bar0 + 8 * kEmpty, acc_full = bar0 + 8 * kAccFull,
                   acc_empty = bar0 + 8 * kAccEmpty, sc_full = bar0 + 8 * kScFull, sc_empty = bar0 + 8 * kScEmpty;

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    // this block's place in its pair, and the pair's in a cluster that shares a reduction
    const int in_cluster = (int)cluster_ctarank();
    const int rank = SPLIT ? in_cluster & 1 : in_cluster, lead = SPLIT ? in_cluster - rank : 0;
    // [0]: a wait of the cluster's ran out; [1], [2], in the leader: the steps that each block's producer
    // has issued loads of, where it did not see them all consumed. (Not kept: e4m3 has no registers
    // for it.)
    const auto failed = [&] { return reinterpret_cast<volatile uint32_t *>(bars + kFailed); };
    const int part = SPLIT ? lead / 2 : 0, parts = SPLIT ? (int)cluster_blocks() / 2 : 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars + i, 2);           // both blocks' producers
            mbar_init(bars + kEmpty + i, 1);  // a commit
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(bars + kAccFull + i, 1);
            mbar_init(bars + kAccEmpty + i, 2 * kEpiWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kScFull + i, kHelpers);
            mbar_init(bars + kScEmpty + i, kEpiWarps);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bars + kTileFull + i, 1);
            mbar_init(bars + kTileEmpty + i, kEpiWarps + (rank == 0) + (FP8 ? kHelpers : 0));
        }
        for (int i = 0; i < kEpiWarps / 2; ++i) mbar_init(bars + kSwap + i, 64);
        if (SPLIT) {
            mbar_init(bars + kParked, (parts - 1) * kEpiWarps);
            mbar_init(bars + kFetched, (FP8 ? 1 : parts - 1) * kEpiWarps);
        }
        mbar_init(bars + kDrained, 1);
        failed()[0] = 0;
        failed()[1] = failed()[2] = kConsumed;
        mbar_init_fence();
        for (int i = 0; i < Maps<MODE>::kM; ++i) tma_prefetch_map(&maps.m[i]);
        for (int i = 0; i < Maps<MODE>::kN; ++i) tma_prefetch_map(&maps.n[i]);
    }
    if (warp == kMmaWarp) tmem_alloc_pair(bar0 + 8 * kSlot, 512);
    tcgen05_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tcgen05_fence_after();
    const uint32_t tmem = *reinterpret_cast<const volatile uint32_t *>(bars + kSlot);
    pdl_wait();
    pdl_trigger();

    // a cluster's first tile is shared by its pairs; should there be more tiles than clusters, the
    // others are not
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2, first = SPLIT ? pair / parts : pair;
    Walker<MODE, kStep, FP8> walk(p, kFeatStep);
    Tile t;
    bool more = false;
    // Where e4m3's first tile is looked up before the warps part, its epilogue keeps all but two words
    // of what it needs in registers (without gates, 4096 x 7168, 256 experts of 512 rows: 720 us for 772); for the others
    // it only comes later that way (a lone tile +0.3 us).
    constexpr bool kEarly = FP8 && !SPLIT;
    if (kEarly && warp == kProducerWarp) more = walk.next(first, t);
    Ring ring{slots, bar0 + 8 * kTileFull, bar0 + 8 * kTileEmpty};
    bool ok = true;
    if (warp >= kEpiWarps) {
        // e4m3: 640 threads launch with 96 registers each, 61440 in all: 512 x 104 + 128 x 64
        if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kProducerWarp) {
            const uint32_t lead_full = map_to_rank(full, lead);
            int stage = 0, issued = 0;
            uint32_t parity = 1;
            bool cut = false;
            for (int tile = first; ok; tile = SPLIT && tile == first ? pairs / parts + pair : tile + pairs) {
                if (!kEarly || tile != first) more = walk.next(tile, t);
                if (SPLIT && more) {
                    if (tile == first) {
                        // wgrad: the host knows the rows that there is room for, not those that there are
                        cut = MODE != kWgrad || worth_sharing<FP8>(p.N, t.steps, parts);
                        if (cut)
                            walk.cut(t, part, parts);
                        else if (part > 0)
                            continue;
                    } else if (cut && (!FP8 || part > 0)) {  // the stages are free again once the sums are fetched
                        if (!(ok = mbar_wait_pipe<true>(bar0 + 8 * kFetched, 0, p.wait_ns))) break;
                        fence_proxy_async();
                    }
                }
                if (!(ok = mbar_wait_pipe(ring.empty + 8 * ring.at, ring.parity ^ 1, p.wait_ns))) break;
                if (elect_one()) {
                    if (!more) t.e = -1;
                    slots[ring.at] = t;
                    mbar_arrive_own(ring.full + 8 * ring.at);
                }
                if (++ring.at == kRing) ring.at = 0, ring.parity ^= 1;
                if (!more) break;
                // this block's token rows: half of the tile's, or (e4m3, rows as M) its 128 as far as
                // there are any, to a multiple of 16
                const int half = t.across ? t.n / 2 : max(0, min(128, (t.rows - rank * 128 + 15) & ~15));
                const int boxes = (half + 63) / 64;  // wgrad
                const uint32_t bytes = kOperandBytes + (MODE == kWgrad ? boxes * 64 : half) * 128;
                // one thread runs the tile's steps, the warp rejoins for the next tile
                int done = 0;
                if (elect_one()) {
                    // this block's features: gated, 64 and their up, or all 128 of one kind
                    const int feat = t.feat0 + rank * (!t.across ? (kHalf ? p.N : t.n / 2) : kHalf ? 64 : 128);
                    const int row = t.row0 + rank * (t.across ? half : 128);
                    // operand M first; a has the features, b the rows
                    const uint32_t a_at = base + (t.across ? 0 : kOperandBytes);
                    const uint32_t b_at = base + (t.across ? kOperandBytes : 0);
                    for (int i = 0; i < t.steps; ++i) {
                        const int k = SPLIT ? t.step0 + i : i;
                        if (!(ok = mbar_wait_pipe(empty + 8 * stage, parity, p.wait_ns))) break;
                        const uint32_t a = a_at + stage * kStageBytes, b = b_at + stage * kStageBytes;
                        const uint32_t bar = lead_full + 8 * stage;
                        if (MODE == kWgrad) {
                            const int at = t.start + k * kStep, left = t.count - k * kStep;
                            if (left >= kStep) {
                                mbar_arrive_tx_cluster(bar, bytes);
                                tma_2d(a, &maps.m[0], feat, at, bar);
                                tma_2d(a + 8192, &maps.m[0], feat + 64, at, bar);
                                for (int i = 0; i < boxes; ++i) tma_2d(b + i * 8192, &maps.n[0], row + i * 64, at, bar);
                            } else {
                                const int used = (left + 15) & ~15;
                                mbar_arrive_tx_cluster(bar, (2 + boxes) * used * 128);
                                constexpr int kMaps = Maps<MODE>::kM;
                                int r = 0;
#pragma unroll 1
                                for (int c = 0; c < 4; ++c) {
                                    // 32 and 16 rows, the last ones, and the zeros after them
                                    const int rows = c < 2 ? left & (32 >> c) : c == 2 ? left & 15 : used - left;
                                    if (rows == 0) continue;
                                    const int map = (rows >= 16 ? (rows == 32 ? 1 : 2) : rows + 2) % kMaps;
                                    const int from = c < 3 ? at + r : (int)p.rows.capacity_rows;
                                    tma_2d(a + r * 128, &maps.m[map], feat, from, bar);
                                    tma_2d(a + 8192 + r * 128, &maps.m[map], feat + 64, from, bar);
                                    for (int i = 0; i < boxes; ++i)
                                        tma_2d(b + i * 8192 + r * 128, &maps.n[map], row + i * 64, from, bar);
                                    r += rows;
                                }
                            }
                        } else {
                            mbar_arrive_tx_cluster(bar, bytes);
                            if (MODE == kDgrad) {
                                tma_3d(a, &maps.m[0], feat, k * kStep, t.e, bar);
                                tma_3d(a + 8192, &maps.m[0], feat + 64, k * kStep, t.e, bar);
                            } else if (kHalf && t.across) {
                                tma_4d(a, &maps.m[0], k * kStep, feat, 0, t.e, bar);
                            } else {
                                tma_3d(a, &maps.m[Maps<MODE>::kM > 1], k * kStep, feat, t.e, bar);
                            }
                            int r = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (!(half & (128 >> i))) continue;
                                tma_2d(b + r * 128, &maps.n[i], k * kStep, t.start + row + r, bar);
                                r += 128 >> i;
                            }
                        }
                        if (++stage == kStages) stage = 0, parity ^= 1;
                        ++done;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                issued += ok ? t.steps : __reduce_max_sync(0xffffffffu, done);
                stage = __shfl_sync(0xffffffffu, issued % kStages, 0);
                parity = 1 ^ ((issued / kStages) & 1);
            }
            // every stage's last release arrives before this block may go (a stage that was never
            // used counts as released)
            for (int i = 0; ok && i < kStages; ++i) {
                ok = mbar_wait_pipe(empty + 8 * stage, parity, p.wait_ns);
                if (++stage == kStages) stage = 0, parity ^= 1;
            }
            if (!ok && lane == 0) st_cluster(map_to_rank(smem_addr(bars + kFailed) + 4 + 4 * rank, lead), issued);
        } else if (warp == kMmaWarp) {
            const uint16_t pair_mask = (uint16_t)(3 << lead);
            const uint64_t desc_a = smem_desc(base, 8192), desc_b = smem_desc(base + kOperandBytes, 8192);
            int stage = 0, acc = 0, was = -1, tiles = 0;
            uint32_t parity = 0, parities = (1u << kAccs) - 1;  // of each accumulator's next release
            while (rank == 0 && ring.next(ok, p)) {
                const int steps = ring.tile().steps, n = ring.tile().n;
                // wgrad: rows of the region's last step, if it is this pair's and not a full one
                const int left = !SPLIT || ring.tile().part == ring.tile().parts - 1 ? ring.tile().count & 63 : 0;
                const int across = ring.tile().across;
                ring.drop();
                if (tiles++ == p.stall) break;
                if (steps == 0) continue;
                const uint32_t desc = mma_desc<FP8, MODE != kForward, MODE == kWgrad>(n);
                const int accs = FP8 && !across ? 2 : kAccs, columns = 512 / accs;
                if (FP8) acc = 0;
                int st = stage, c = acc;
                uint32_t ph = parity, aph = parities;
                if (elect_one()) {
                    if (FP8 && across != was && was >= 0)  // other accumulators lie where these will
                        for (int i = 0; ok && i < kAccs; ++i) ok = mbar_wait_pipe(acc_empty + 8 * i, (aph >> i) & 1, p.wait_ns);
                    for (int k = 0; ok && k < steps; ++k) {
                        const bool fresh = FP8 || k == 0, last = FP8 || k == steps - 1;
                        if (fresh) {
                            if (!(ok = mbar_wait_pipe(acc_empty + 8 * c, (aph >> c) & 1, p.wait_ns))) break;
                            aph ^= 1u << c;
                        }
                        if (!(ok = mbar_wait_pipe(full + 8 * st, ph, p.wait_ns))) break;
                        tcgen05_fence_after();
                        // a quarter of the stage's reduction: 32 bytes along a K-major row, or
                        // 16 rows of 128 bytes
                        constexpr uint64_t kA = MODE != kForward ? 128 : 2, kB = MODE == kWgrad ? 128 : 2;
                        const uint64_t da = desc_a + (uint32_t)(st * (kStageBytes >> 4));
                        const uint64_t db = desc_b + (uint32_t)(st * (kStageBytes >> 4));
                        const uint32_t d = tmem + c * columns;
                        const int quarters = MODE == kWgrad && left && k == steps - 1 ? (left + 15) / 16 : 4;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (q < quarters) mma_pair<FP8>(d, da + q * kA, db + q * kB, desc, !(fresh && q == 0));
                        mma_commit_pair(empty + 8 * st, pair_mask);
                        if (last) {
                            mma_commit_pair(acc_full + 8 * c, pair_mask);
                            if (++c == accs) c = 0;
                        }
                        if (++st == kStages) st = 0, ph ^= 1;
                    }
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                stage += steps;
                parity ^= (stage / kStages) & 1;
                stage %= kStages;
                was = across;
                // one flip for each use: whole rounds, then the accumulators up to the next
                const int used = FP8 ? steps : 1;
                if (used / accs & 1) parities ^= (1u << accs) - 1;
                for (int i = 0; i < used % accs; ++i) {
                    parities ^= 1u << acc;
                    acc = (acc + 1) % accs;
                }
            }
        } else if (MODE == kWgrad) {
            // 64 columns a warp, or 16 where that leaves warps without any: one expert of 4096 rows,
            // 1024 x 1024, 32.5 us with 64 and 16.5 with 16
            const int worker = blockIdx.x * kHelpers + warp - kHelperWarp, workers = gridDim.x * kHelpers;
            if (p.dbias) {
                if ((int64_t)((p.N + 63) / 64) * p.rows.num_experts < workers)
                    sum_bias<2>(p, worker, workers);
                else
                    sum_bias<8>(p, worker, workers);
            }
        } else if (FP8) {
            const int tid = threadIdx.x - kHelperWarp * 32;
            const int C = p.K / 128;
            const int64_t blocks = ((GATED ? 2 * p.N : p.N) + 127) / 128;
            int buf = 0;
            uint32_t parity = 1;
            while (ok && ring.next(ok, p)) {
                const Tile t = ring.tile();
                ring.drop();
                // the tile's two weight blocks; across: this block's (gated: its gate's and its up's)
                int b0 = (t.feat0 + (t.across ? rank * (kHalf ? 64 : 128) : 0)) / 128;
                int b1 = kHalf ? b0 + p.N / 128 : b0 + (t.across ? 0 : 1);
                if (b0 >= blocks) b0 = 0;  // features past the last: nothing of them is kept
                if (b1 >= blocks) b1 = b0;
                const float *w0 = p.w_scale + ((int64_t)t.e * blocks + b0) * C;
                const float *w1 = p.w_scale + ((int64_t)t.e * blocks + b1) * C;
                const int end = t.step0 + t.steps;
                const int skip = t.across ? 0 : rank * 128, rows = t.rows - skip;
                const float *xs = p.x_scale + ((int64_t)t.start + t.row0 + skip) * p.srow + t.e * p.sexp;
                for (int g = t.step0; g < end; g += kScaleGroup) {
                    float sw[2][kScaleGroup], sx[2][kScaleGroup];
#pragma unroll
                    for (int k = 0; k < kScaleGroup; ++k) {
                        sw[0][k] = g + k < C ? w0[g + k] : 0.0f;
                        sw[1][k] = g + k < C ? w1[g + k] : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = i * 64 + tid;
                        if (c < rows && p.scale_vec) {
                            const float4 v = *reinterpret_cast<const float4 *>(xs + c * p.srow + g);
                            sx[i][0] = v.x, sx[i][1] = v.y, sx[i][2] = v.z, sx[i][3] = v.w;
                        } else {
#pragma unroll
                            for (int k = 0; k < kScaleGroup; ++k)
                                sx[i][k] = c < rows && g + k < C ? xs[c * p.srow + (g + k) * p.scol] : 0.0f;
                        }
                    }
                    if (!(ok = mbar_wait_pipe(sc_empty + 8 * buf, parity, p.wait_ns))) break;
                    if (!t.across) {  // a row's two, side by side
                        float2 *dst = reinterpret_cast<float2 *>(scales) + buf * kScaleGroup * 128 + tid;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int k = 0; k < kScaleGroup; ++k)
                                dst[k * 128 + i * 64] = make_float2(sx[i][k] * sw[0][k], sx[i][k] * sw[1][k]);
                    } else {  // for each weight block, the eight rows of 32 that a lane's fragments hold
                        float *dst = scales + buf * kScaleGroup * 256 + (tid & 32) + 8 * (tid & 3) + ((tid >> 2) & 7);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int k = 0; k < kScaleGroup; ++k) {
                                dst[k * 256 + i * 64] = sx[i][k] * sw[0][k];
                                dst[k * 256 + 128 + i * 64] = sx[i][k] * sw[1][k];
                            }
                    }
                    __syncwarp();
                    if (elect_one()) mbar_arrive_own(sc_full + 8 * buf);
                    buf ^= 1;
                    if (buf == 0) parity ^= 1;
                }
                ok = __all_sync(0xffffffffu, ok);
            }
        }
    } else {
        if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        constexpr int kShare = kEpiWarps / 4;  // warps that share the columns of 32 lanes
        const int quadrant = warp & 3, share = warp >> 2;
        const uint32_t lead_empty = map_to_rank(acc_empty, lead);
        const uint32_t my_tmem = tmem + ((uint32_t)(quadrant * 32) << 16);
        uint32_t parities = 0;  // of each accumulator's next result
        if (FP8) {
            // A lane is a row; the warp's columns are share * 32 .. + 31 of each of the two weight
            // blocks, 16 at a time.
            const float2 *my_scales = reinterpret_cast<const float2 *>(scales) + quadrant * 32 + lane;
            int sbuf = 0;
            uint32_t sparity = 0;
            while (ok && ring.next(ok, p)) {
                const int steps = ring.tile().steps;
                if (ring.tile().across) {
                    // a lane is a feature, in fragments; the warp's columns are share * 32 .. + 31
                    const bool own = share * 32 < ring.tile().n;
                    const float4 *at = reinterpret_cast<const float4 *>(
                        scales + (kHalf && quadrant >= 2 ? 128 : 0) + share * 32 + 8 * (lane & 3));
                    Frag acc;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[h][r] = 0.0f;
                    for (int k = 0; k < steps; ++k) {
                        const int u = k % kScaleGroup, c = k % kAccs;
                        if (u == 0 && !(ok = mbar_wait_pipe(sc_full + 8 * sbuf, sparity, p.wait_ns))) break;
                        if (!(ok = mbar_wait_pipe(acc_full + 8 * c, (parities >> c) & 1, p.wait_ns))) break;
                        parities ^= 1u << c;
                        tcgen05_fence_after();
                        if (own) {
                            const float4 lo = at[(sbuf * kScaleGroup + u) * 64], hi = at[(sbuf * kScaleGroup + u) * 64 + 1];
                            const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};  // columns 4c + lane % 4
                            uint32_t v[2][16];
                            tmem_ld_frag(v[0], my_tmem + c * 128 + share * 32);
                            tmem_ld_frag(v[1], my_tmem + c * 128 + share * 32 + (16u << 16));
                            tmem_wait_ld();
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int r = 0; r < 16; ++r)
                                    acc[h][r] = fmaf(__uint_as_float(v[h][r]), f[r >> 1], acc[h][r]);
                        }
                        tcgen05_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(lead_empty + 8 * c);
                        if (u == kScaleGroup - 1 || k == steps - 1) {
                            if (lane == 0) mbar_arrive_own(sc_empty + 8 * sbuf);
                            sbuf ^= 1;
                            if (sbuf == 0) sparity ^= 1;
                        }
                    }
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (SPLIT && ring.tile().parts > 1) {
                        const uint32_t at = base + warp * 4096;
                        auto sum = [&](int r) -> float & { return acc[r >> 4][r & 15]; };
                        if (ring.tile().part > 0) {
                            if (own) park(at, sum);
                            tell_first(bar0 + 8 * kParked);
                            ring.drop();
                            continue;
                        }
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait_pipe<true>(bar0 + 8 * kParked, 0, p.wait_ns)))) break;
                        if (own) add_parked(at, ring.tile(), sum);
                        tell_others(bar0 + 8 * kFetched, ring.tile());
                    }
                    Output<MODE, GATED, kStagedOf<FP8>> out(p, staging, bar0 + 8 * kSwap, warp);
                    out.begin(ring.tile(), rank, quadrant);
                    if (own) {
                        out.fetch(share * 32);
                        out.finish(acc, share * 32, kTileRows);
                    }
                    ok = out.ok;
                    ring.drop();
                    continue;
                }
                const int blocks = ring.tile().rows - rank * 128 - quadrant * 32 > 0
                                       ? (ring.tile().n - share * 32 + 127) / 128 : 0;  // with columns here
                float acc[2][32];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 32; ++r) acc[h][r] = 0.0f;
                for (int k = 0; k < steps; ++k) {
                    const int u = k % kScaleGroup, c = k & 1;
                    if (u == 0 && !(ok = mbar_wait_pipe(sc_full + 8 * sbuf, sparity, p.wait_ns))) break;
                    const float2 sc = my_scales[(sbuf * kScaleGroup + u) * 128];
                    if (!(ok = mbar_wait_pipe(acc_full + 8 * c, (parities >> c) & 1, p.wait_ns))) break;
                    parities ^= 1u << c;
                    tcgen05_fence_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h < blocks) {
                            const float f = h ? sc.y : sc.x;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                uint32_t v[16];
                                tmem_ld16(v, my_tmem + c * kTileRows + h * 128 + share * 32 + q * 16);
                                tmem_wait_ld();
                                const uint64_t ff = twice(f);
#pragma unroll
                                for (int r = 0; r < 16; r += 2)
                                    fma2(acc[h][q * 16 + r], acc[h][q * 16 + r + 1], v[r], v[r + 1], ff);
                            }
                        }
                    }
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(lead_empty + 8 * c);
                    if (u == kScaleGroup - 1 || k == steps - 1) {
                        if (lane == 0) mbar_arrive_own(sc_empty + 8 * sbuf);
                        sbuf ^= 1;
                        if (sbuf == 0) sparity ^= 1;
                    }
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (SPLIT && ring.tile().parts > 1) {
                    const uint32_t at = base + warp * 8192;
                    auto gate = [&](int r) -> float & { return acc[0][r]; };
                    auto rest = [&](int r) -> float & { return acc[1][r]; };
                    if (ring.tile().part > 0) {
                        if (blocks > 0) park(at, gate), park(at + 4096, rest);
                        tell_first(bar0 + 8 * kParked);
                        ring.drop();
                        continue;
                    }
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait_pipe<true>(bar0 + 8 * kParked, 0, p.wait_ns)))) break;
                    if (blocks > 0) add_parked(at, ring.tile(), gate), add_parked(at + 4096, ring.tile(), rest);
                    tell_others(bar0 + 8 * kFetched, ring.tile());
                }
                if (blocks > 0) finish_rows<GATED>(p, ring.tile(), rank * 128 + quadrant * 32, share * 32,
                                                   staging + warp * kStagingOf<FP8>, acc);
                ring.drop();
            }
        } else {
            Output<MODE, GATED, kStagedOf<FP8>> out(p, staging, bar0 + 8 * kSwap, warp);
            int buf = 0;
            while (ok && ring.next(ok, p)) {
                const Tile &t = ring.tile();
                out.begin(t, rank, quadrant);
                const int chunks = t.n / 32;
                const bool any = t.steps > 0;  // else wgrad of an expert without rows
                Tile part_of;  // parts and this one's number
                part_of.parts = t.parts, part_of.part = t.part;
                const bool shared = SPLIT && t.parts > 1;
                // a shared tile's chunks go round the pairs, as many at a time as its columns are shared by
                const int from = share + (shared ? kShare * part_of.part : 0), by = shared ? kShare * part_of.parts : kShare;
                ring.drop();
                if (from < chunks) out.fetch(from * 32);
                if (any) {
                    if (!(ok = mbar_wait_pipe(acc_full + 8 * buf, (parities >> buf) & 1, p.wait_ns))) break;
                    parities ^= 1u << buf;
                    tcgen05_fence_after();
                }
                auto load = [&](Frag &f, int ch) {
                    uint32_t v[2][16];
                    if (any) {
                        tmem_ld_frag(v[0], my_tmem + buf * kTileRows + ch * 32);
                        tmem_ld_frag(v[1], my_tmem + buf * kTileRows + ch * 32 + (16u << 16));
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 16; ++r) f[h][r] = any ? __uint_as_float(v[h][r]) : 0.0f;
                };
                if (shared) {
                    for (int ch = share; ch < chunks; ch += kShare) {
                        if (ch / kShare % part_of.parts == part_of.part) continue;
                        Frag f;
                        load(f, ch);
                        park(base + (ch * 4 + quadrant) * 4096, [&](int r) -> float & { return f[r >> 4][r & 15]; });
                    }
                    if (!(ok = exchange(bar0 + 8 * kParked, part_of, p))) break;
                }
                for (int ch = from; ch < chunks; ch += by) {
                    Frag f;
                    load(f, ch);
                    if (shared)
                        add_parked(base + (ch * 4 + quadrant) * 4096, part_of,
                                   [&](int r) -> float & { return f[r >> 4][r & 15]; });
                    out.finish(f, ch * 32, (ch + by) * 32);
                }
                if (shared) tell_others(bar0 + 8 * kFetched, part_of);
                if (any) {
                    tcgen05_fence_before();
                    __syncwarp();
                    if (elect_one()) mbar_arrive_cluster(lead_empty + 8 * buf);
                    buf ^= 1;
                }
                ok = __all_sync(0xffffffffu, out.ok);
            }
        }
    }
    if (!ok && lane == 0) {
        report(p.status, EPD_ERR_TIMEOUT);
        for (int i = 0; i < (int)cluster_blocks(); ++i) st_cluster(map_to_rank(smem_addr(bars + kFailed), i), 1);
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tcgen05_fence_after();
    if (*failed()) drain(smem_addr(bars), smem_addr(bars + kDrained), smem_addr(bars + kFailed) + 4, kMmaWarp);
    if (warp == kMmaWarp) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// A map of `dim` dimensions, the innermost contiguous; strides of the others in elements.
bool encode(CUtensorMap *map, bool fp8, int dim, const void *at, const cuuint64_t *size, const int64_t *stride,
            const cuuint32_t *box) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    cuuint64_t bytes[4];
    cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i + 1 < dim; ++i) bytes[i] = (cuuint64_t)stride[i] * (fp8 ? 1 : 2);
    return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dim,
              const_cast<void *>(at), size, bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [count, width] cut into boxes of `rows` rows of 128 bytes.
bool encode_rows(CUtensorMap *map, bool fp8, const void *at, int64_t count, int64_t width, int rows) {
    const cuuint64_t size[2] = {(cuuint64_t)width, (cuuint64_t)(count > 0 ? count : 1)};
    const int64_t stride[1] = {width};
    const cuuint32_t box[2] = {fp8 ? 128u : 64u, (cuuint32_t)rows};
    return encode(map, fp8, 2, at, size, stride, box);
}

// Clusters of `parts` pairs that the device holds at a time (0 where a query fails).
template <int MODE, bool FP8, bool GATED, bool SPLIT>
epd_status_t resident(int parts, int &clusters) {
    static std::atomic<int> cached[3][64];  // one more than the answer, per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return record_cuda_error();
    std::atomic<int> &slot = cached[parts / 2][dev >= 0 && dev < 64 ? dev : 0];
    clusters = slot.load(std::memory_order_relaxed) - 1;
    if (clusters >= 0 && dev < 64) return EPD_OK;
    auto kernel = expert_kernel<MODE, FP8, GATED, SPLIT>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOf<FP8>) != cudaSuccess)
        return record_cuda_error();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count() / (2 * parts) * (2 * parts)));
    cfg.blockDim = dim3(kThreadsOf<MODE, FP8>);
    cfg.dynamicSmemBytes = kSmemOf<FP8>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 0) {
        cudaGetLastError();
        clusters = 0;
    }
    slot.store(clusters + 1, std::memory_order_relaxed);
    return EPD_OK;
}

template <int MODE, bool FP8, bool GATED>
epd_status_t launch(const Maps<MODE> &maps, ExpertArgs p, cudaStream_t stream) {
    const int features = MODE == kForward ? p.N : p.K;
    const int64_t feat_tiles = ceil_div(features, GATED && MODE == kForward ? 128 : 256);
    const int64_t cap = p.rows.capacity_rows, E = p.rows.num_experts;
    const int64_t row_tiles = MODE == kWgrad ? (int64_t)ceil_div(p.N, kTileRows) * E
                              : p.rows.expert_start_loc ? cap / kTileRows + (E < cap ? E : cap)
                                                        : (p.rows.rows_per_expert + kTileRows - 1) / kTileRows * E;
    const int64_t most = row_tiles > 0 ? feat_tiles * row_tiles : 1;
    if (most > INT32_MAX / 2) return EPD_ERR_UNSUPPORTED;
    constexpr int kThreads = kThreadsOf<MODE, FP8>, kSmem = kSmemOf<FP8>;
    int clusters;
    // the columns of D: an expert's rows, as far as there is room on average (wgrad: these are the
    // reduction)
    const int64_t rows = cap / E, columns = MODE == kWgrad ? p.N : rows;
    const int64_t steps = ((MODE == kForward ? p.K : MODE == kDgrad ? p.N : rows) + (FP8 ? 127 : 63)) / (FP8 ? 128 : 64);
    // (wgrad: one expert may have all the rows)
    if (p.wait_ns == 0) p.wait_ns = kWaitNs + (MODE == kWgrad ? (cap + 63) / 64 : steps) * kWaitStepNs;
    for (int parts = 4; parts > 1; parts /= 2) {
        if (!worth_sharing<FP8>(columns, steps, parts)) continue;
        if (most * parts > sm_count() / 2) continue;
        const epd_status_t rc = resident<MODE, FP8, GATED, true>(parts, clusters);
        if (rc != EPD_OK) return rc;
        if (most <= clusters)
            return launch_pdl_cluster(expert_kernel<MODE, FP8, GATED, true>, 2 * parts * (int)most, kThreads, kSmem,
                                      2 * parts, stream, maps, p);
    }
    const epd_status_t rc = resident<MODE, FP8, GATED, false>(1, clusters);
    if (rc != EPD_OK) return rc;
    if (clusters < 1) clusters = 1;
    return launch_pdl_cluster(expert_kernel<MODE, FP8, GATED, false>, 2 * (int)(most < clusters ? most : clusters), kThreads,
                              kSmem, 2, stream, maps, p);
}

bool rows_ok(const epd_expert_rows_t *r) {
    if (!r || r->num_experts < 1 || r->num_experts > EPD_MAX_EXPERTS) return false;
    if (r->capacity_rows < 0 || r->capacity_rows > INT32_MAX) return false;
    if (!r->tokens_per_expert || !aligned4(r->tokens_per_expert)) return false;
    if (r->expert_start_loc) return aligned4(r->expert_start_loc);
    return r->rows_per_expert >= 0 && r->rows_per_expert <= INT32_MAX &&
           r->rows_per_expert * r->num_experts <= r->capacity_rows;
}

bool act_ok(int act) { return act >= EPD_ACT_NONE && act <= EPD_ACT_SWIGLU; }

}  // namespace
}  // namespace epd

namespace epd {
namespace {

epd_status_t forward(const epd_expert_rows_t *rows, const void *x, epd_dtype_t dtype, const float *x_scale,
                     int64_t scale_row_stride, int64_t scale_col_stride, int64_t scale_expert_stride, const void *w,
                     const float *w_scale, int in_features, int out_features, epd_activation_t activation,
                     const float *bias, const void *residual, void *y, void *preact, int32_t *status,
                     epd_stream_t stream, int stall, uint64_t wait_ns) {
    const int K = in_features, N = out_features;
    const bool fp8 = dtype == EPD_FP8_E4M3, gated = activation == EPD_ACT_SWIGLU;
    if (!rows_ok(rows) || !act_ok(activation)) return EPD_ERR_INVALID_ARG;
    if (dtype != EPD_BF16 && !fp8) return EPD_ERR_INVALID_ARG;
    if (K < 1 || N < 1 || K % (fp8 ? 128 : 8) != 0 || N % (gated && fp8 ? 128 : 8) != 0)
        return EPD_ERR_INVALID_ARG;
    if (N > INT32_MAX / 2) return EPD_ERR_UNSUPPORTED;
    if (fp8 != (x_scale != nullptr) || fp8 != (w_scale != nullptr)) return EPD_ERR_INVALID_ARG;
    if (fp8 && (!aligned4(x_scale) || !aligned4(w_scale))) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status) || !w || !aligned16(w) || (bias && !aligned4(bias)))
        return EPD_ERR_INVALID_ARG;
    if (rows->capacity_rows == 0) return EPD_OK;
    if (!x || !aligned16(x) || !y || !aligned16(y) || (residual && !aligned16(residual)) ||
        (preact && !aligned16(preact)))
        return EPD_ERR_INVALID_ARG;
    ExpertArgs p = {};
    p.stall = stall;
    p.wait_ns = wait_ns;
    p.rows = *rows;
    p.act = activation;
    p.x_scale = x_scale;
    p.w_scale = w_scale;
    p.srow = scale_row_stride;
    p.scol = scale_col_stride;
    p.sexp = scale_expert_stride;
    p.K = K;
    p.N = N;
    p.bias = bias;
    p.residual = static_cast<const uint8_t *>(residual);
    p.y = static_cast<uint8_t *>(y);
    p.preact = static_cast<uint8_t *>(preact);
    p.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    p.scale_vec = fp8 && scale_col_stride == 1 && K % 512 == 0 && scale_row_stride % 4 == 0 &&
                  scale_expert_stride % 4 == 0 && aligned16(x_scale);
    Maps<kForward> maps;
    bool done = true;
    for (int i = 0; i < 4; ++i) done = done && encode_rows(&maps.n[i], fp8, x, rows->capacity_rows, K, 128 >> i);
    const cuuint32_t wide = fp8 ? 128 : 64;
    const cuuint64_t E = (cuuint64_t)rows->num_experts;
    const int64_t NW = gated ? 2 * (int64_t)N : N;
    const cuuint64_t size[3] = {(cuuint64_t)K, (cuuint64_t)NW, E};
    const int64_t stride[2] = {K, NW * K};
    const cuuint32_t box[3] = {wide, 128, 1};
    done = done && encode(&maps.m[1], fp8, 3, w, size, stride, box);
    if (gated) {
        const cuuint64_t size2[4] = {(cuuint64_t)K, (cuuint64_t)N, 2, E};
        const int64_t stride2[3] = {K, (int64_t)N * K, NW * K};
        const cuuint32_t box2[4] = {wide, 64, 2, 1};
        done = done && encode(&maps.m[0], fp8, 4, w, size2, stride2, box2);
    } else {
        maps.m[0] = maps.m[1];  // not used
    }
    if (!done) return EPD_ERR_CUDA;
    if (fp8)
        return gated ? launch<kForward, true, true>(maps, p, st) : launch<kForward, true, false>(maps, p, st);
    return gated ? launch<kForward, false, true>(maps, p, st) : launch<kForward, false, false>(maps, p, st);
}

}  // namespace
}  // namespace epd

extern "C" epd_status_t ep_expert_matmul(const epd_expert_rows_t *rows, const void *x,
                                         epd_dtype_t dtype, const float *x_scale,
                                         int64_t scale_row_stride, int64_t scale_col_stride,
                                         int64_t scale_expert_stride, const void *w,
                                         const float *w_scale, int in_features, int out_features,
                                         epd_activation_t activation, const float *bias,
                                         const void *residual, void *y, void *preact,
                                         int32_t *status, epd_stream_t stream) {
    return epd::forward(rows, x, dtype, x_scale, scale_row_stride, scale_col_stride, scale_expert_stride, w, w_scale,
                        in_features, out_features, activation, bias, residual, y, preact, status, stream, -1, 0);
}

extern "C" epd_status_t epd_test_expert_matmul_stalled(
    const epd_expert_rows_t *rows, const void *x, epd_dtype_t dtype, const float *x_scale, int64_t scale_row_stride,
    int64_t scale_col_stride, int64_t scale_expert_stride, const void *w, const float *w_scale, int in_features,
    int out_features, epd_activation_t activation, void *y, int32_t *status, int stalled_tile, int64_t wait_ns,
    epd_stream_t stream) {
    if (wait_ns < 1) return EPD_ERR_INVALID_ARG;
    return epd::forward(rows, x, dtype, x_scale, scale_row_stride, scale_col_stride, scale_expert_stride, w, w_scale,
                        in_features, out_features, activation, nullptr, nullptr, y, nullptr, status, stream,
                        stalled_tile, (uint64_t)wait_ns);
}

extern "C" epd_status_t ep_expert_matmul_dgrad(const epd_expert_rows_t *rows, const void *dy,
                                               const void *w, int in_features, int out_features,
                                               epd_activation_t activation, const void *preact,
                                               void *dx, int32_t *status, epd_stream_t stream) {
    using namespace epd;
    const int K = in_features, N = out_features;
    if (!rows_ok(rows) || !act_ok(activation)) return EPD_ERR_INVALID_ARG;
    if (K < 1 || N < 1 || K % 8 != 0 || N % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (K > INT32_MAX / 2) return EPD_ERR_UNSUPPORTED;
    if ((activation != EPD_ACT_NONE) != (preact != nullptr)) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status) || !w || !aligned16(w)) return EPD_ERR_INVALID_ARG;
    if (rows->capacity_rows == 0) return EPD_OK;
    if (!dy || !aligned16(dy) || !dx || !aligned16(dx) || (preact && !aligned16(preact)))
        return EPD_ERR_INVALID_ARG;
    ExpertArgs p = {};
    p.stall = -1;
    p.rows = *rows;
    p.act = activation;
    p.K = K;
    p.N = N;
    p.preact_in = static_cast<const uint8_t *>(preact);
    p.y = static_cast<uint8_t *>(dx);
    p.status = status;
    Maps<kDgrad> maps;
    const cuuint64_t size[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)rows->num_experts};
    const int64_t stride[2] = {K, (int64_t)N * K};
    const cuuint32_t box[3] = {64, 64, 1};
    bool done = encode(&maps.m[0], false, 3, w, size, stride, box);
    for (int i = 0; i < 4; ++i) done = done && encode_rows(&maps.n[i], false, dy, rows->capacity_rows, N, 128 >> i);
    if (!done) return EPD_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return activation == EPD_ACT_SWIGLU ? launch<kDgrad, false, true>(maps, p, st)
                                        : launch<kDgrad, false, false>(maps, p, st);
}

extern "C" epd_status_t ep_expert_matmul_wgrad(const epd_expert_rows_t *rows, const void *dy,
                                               const void *x, int in_features, int out_features,
                                               void *dw, float *dbias, int32_t *status,
                                               epd_stream_t stream) {
    using namespace epd;
    const int K = in_features, N = out_features;
    if (!rows_ok(rows)) return EPD_ERR_INVALID_ARG;
    if (K < 1 || N < 1 || K % 8 != 0 || N % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (K > INT32_MAX / 2 || N > INT32_MAX / 2) return EPD_ERR_UNSUPPORTED;
    if (!status || !aligned4(status) || !dw || !aligned16(dw) || (dbias && !aligned4(dbias)))
        return EPD_ERR_INVALID_ARG;
    if (rows->capacity_rows > 0 && (!dy || !aligned16(dy) || !x || !aligned16(x)))
        return EPD_ERR_INVALID_ARG;
    ExpertArgs p = {};
    p.stall = -1;
    p.rows = *rows;
    p.K = K;
    p.N = N;
    p.y = static_cast<uint8_t *>(dw);
    p.dy = static_cast<const uint8_t *>(dy);
    p.dbias = dbias;
    p.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // without rows nothing is loaded, but a map has to lie somewhere
    const bool any = rows->capacity_rows > 0;
    Maps<kWgrad> maps;
    for (int i = 0; i < kCuts; ++i)
        if (!encode_rows(&maps.m[i], false, any ? x : dw, rows->capacity_rows, K, cut_rows(i)) ||
            !encode_rows(&maps.n[i], false, any ? dy : dw, rows->capacity_rows, N, cut_rows(i)))
            return EPD_ERR_CUDA;
    return launch<kWgrad, false, false>(maps, p, st);
}
