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
// would be padded to 128 or 256 rows. Each block stages its 128 feature rows and half of the
// token rows per step of the reduction (128 bytes wide), so a token row that both blocks
// multiply is staged once.
//
// Warps: 0-7 epilogue, 8 TMA producer, 9 issues the mma (in the pair's first block), 10 and
// 11 load row scales (e4m3) or clear the ragged end of a region (wgrad). Accumulators are
// double-buffered in tensor memory, so a tile's epilogue runs under the next tile's mma.
// Blocks walk the tiles of all experts in a fixed order (persistent, one pair per two SMs);
// the experts' counts are read from device memory, 32 at a time, by the warps themselves.
//
// e4m3: rows are scaled per 128 columns and weights per 128 x 128, so the product of one
// 128-wide step cannot stay in the tensor core's accumulator: every step's D goes to
// registers as acc += D * (x_scale * w_scale), again through the two tensor-memory buffers.
#include <cuda.h>

#include "epd_math.cuh"
#include "epd_tcgen05.cuh"

namespace epd {
namespace {

enum { kForward = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kAuxWarp = 10, kAuxWarps = 2;
constexpr int kTileRows = 256;                  // most token rows (wgrad: output rows) of a tile
constexpr int kOperandBytes = 128 * 128;        // 128 rows of 128 bytes: one operand of a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kRowBox = 32;                     // token rows per TMA box
constexpr int kStageStride = 36;                // floats per staged row: conflict-free both ways
constexpr int kStageCols = 16;
constexpr int kStagingBytes = kEpilogueWarps * kStageCols * kStageStride * 4;
constexpr int kScaleGroup = 4;                  // reduction steps per group of staged scales
constexpr int kScaleBytes = 2 * kScaleGroup * 2 * kTileRows * 4;
constexpr int kGroupTiles = 8;                  // token tiles that share a pass over the features

template <bool FP8>
constexpr int kStagesOf = FP8 ? 5 : 6;

template <bool FP8>
constexpr int kSmemOf = kStagesOf<FP8> *kStageBytes + kStagingBytes + (FP8 ? kScaleBytes : 0) + 512;

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
    int32_t *status;
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

// One tile of the work: `rows` valid columns of D from row `row0` (a token row; for wgrad an
// output row of the expert's gradient), n of them computed; features from feat0.
struct Tile {
    int e, start, count;
    int feat0, row0, rows, n;
    int steps;  // of the reduction
};

// Walks the tiles of one pair. Every warp that needs them runs its own walker: lane l holds
// expert batch + l, and a tile's expert is found by a ballot over the running tile counts.
template <int MODE, int STEP>
struct Walker {
    const ExpertArgs &p;
    int lane, feat_tiles, feat_step;
    int batch = -32, before = 0, in_batch = 0;
    int count = 0, start = 0, upto = 0;

    __device__ Walker(const ExpertArgs &args, int feat_step_) : p(args), feat_step(feat_step_) {
        lane = threadIdx.x & 31;
        const int features = MODE == kForward ? p.N : p.K;
        feat_tiles = (features + feat_step - 1) / feat_step;
    }

    __device__ bool next(int tile, Tile &t) {
        int local, row_tiles;
        if (MODE == kWgrad) {
            row_tiles = (p.N + kTileRows - 1) / kTileRows;
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
                upto = (count + kTileRows - 1) / kTileRows * feat_tiles;
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
            row_tiles = (t.count + kTileRows - 1) / kTileRows;
            local = tile - before - (__shfl_sync(0xffffffffu, upto, src) - row_tiles * feat_tiles);
        }
        // groups of row tiles pass over the features together, the row tiles fastest, so that
        // the tiles in flight share both operands in L2
        const int group = local / (kGroupTiles * feat_tiles);
        const int rest = local - group * kGroupTiles * feat_tiles;
        const int width = min(kGroupTiles, row_tiles - group * kGroupTiles);
        const int ft = rest / width;
        const int rt = group * kGroupTiles + rest - ft * width;
        t.feat0 = ft * feat_step;
        const int total = MODE == kWgrad ? p.N : t.count;
        const int each = ((total + row_tiles - 1) / row_tiles + 31) & ~31;
        t.row0 = rt * each;
        t.rows = min(each, total - t.row0);
        t.n = t.rows > 0 ? (t.rows + 31) & ~31 : 32;
        const int red = MODE == kForward ? p.K : MODE == kDgrad ? p.N : t.count;
        t.steps = (red + STEP - 1) / STEP;
        return true;
    }
};

// What the epilogue needs of a tile's features, for the octet of features of this lane.
struct Octet {
    float bias[8], bias_up[8];
    int feat;
    bool live;
};

template <int MODE, bool GATED>
__device__ __forceinline__ void finish_octet(const ExpertArgs &p, const Tile &t, const Octet &o, int row,
                                             float (&v)[8], float (&u)[8]) {
    if (MODE == kWgrad) {
        st16(p.y + (((int64_t)t.e * p.N + t.row0 + row) * p.K + o.feat) * 2, pack8_bf16(v));
        return;
    }
    const int64_t s = (int64_t)t.start + t.row0 + row;
    if (MODE == kDgrad) {
        if (GATED) {
            const uint8_t *zr = p.preact_in + (s * 2 * p.K + o.feat) * 2;
            float g[8], up[8];
            unpack8_bf16(ld_stream16(zr), g);
            unpack8_bf16(ld_stream16(zr + (int64_t)p.K * 2), up);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                u[i] = v[i] * g[i] * sigmoid_f32(g[i]);
                v[i] = v[i] * up[i] * activate_grad<EPD_ACT_SWIGLU>(g[i]);
            }
            uint8_t *yr = p.y + (s * 2 * p.K + o.feat) * 2;
            st16(yr, pack8_bf16(v));
            st16(yr + (int64_t)p.K * 2, pack8_bf16(u));
            return;
        }
        const int64_t at = (s * p.K + o.feat) * 2;
        if (p.act != EPD_ACT_NONE) {
            float z[8];
            unpack8_bf16(ld_stream16(p.preact_in + at), z);
            if (p.act == EPD_ACT_RELU) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= activate_grad<EPD_ACT_RELU>(z[i]);
            } else if (p.act == EPD_ACT_SILU) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= activate_grad<EPD_ACT_SILU>(z[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= activate_grad<EPD_ACT_GELU>(z[i]);
            }
        }
        st16(p.y + at, pack8_bf16(v));
        return;
    }
    const int64_t NW = GATED ? 2 * (int64_t)p.N : p.N;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += o.bias[i];
        if (GATED) {
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += o.bias_up[i];
        }
    }
    if (p.preact) {
        uint8_t *zr = p.preact + (s * NW + o.feat) * 2;
        st16(zr, pack8_bf16(v));
        if (GATED) st16(zr + (int64_t)p.N * 2, pack8_bf16(u));
    }
    if (GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid_f32(v[i]) * u[i];
    } else if (p.act == EPD_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate<EPD_ACT_RELU>(v[i]);
    } else if (p.act == EPD_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate<EPD_ACT_SILU>(v[i]);
    } else if (p.act == EPD_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate<EPD_ACT_GELU>(v[i]);
    }
    const int64_t at = (s * p.N + o.feat) * 2;
    if (p.residual) {
        float r[8];
        unpack8_bf16(ld_stream16(p.residual + at), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    st16(p.y + at, pack8_bf16(v));
}

// 32 columns of D (thread = feature, v[c] = column c) turned over in shared memory, so that a
// lane has eight consecutive features of one row and reads and writes 16 bytes at a time. A
// gated warp's lanes 0-15 are 16 gate features and 16-31 the same features' up.
template <int MODE, bool GATED>
__device__ __forceinline__ void finish_columns(const ExpertArgs &p, const Tile &t, const Octet &o, float *stage,
                                               const float (&v)[32], int col0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 32 / kStageCols; ++h) {
        const int c0 = col0 + h * kStageCols;
        if (c0 >= t.rows) break;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kStageCols; ++c) stage[c * kStageStride + lane] = v[h * kStageCols + c];
        __syncwarp();
        constexpr int kOcts = GATED && MODE == kForward ? 2 : 4;
#pragma unroll
        for (int i = 0; i < kStageCols * kOcts / 32; ++i) {
            const int c = (i * 32 + lane) / kOcts;
            const float4 *src = reinterpret_cast<const float4 *>(stage + c * kStageStride + (lane % kOcts) * 8);
            const float4 a = src[0], b = src[1];
            float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            float u[8];
            if (GATED && MODE == kForward) {
                const float4 ua = src[4], ub = src[5];
                u[0] = ua.x, u[1] = ua.y, u[2] = ua.z, u[3] = ua.w;
                u[4] = ub.x, u[5] = ub.y, u[6] = ub.z, u[7] = ub.w;
            }
            if (o.live && c0 + c < t.rows) finish_octet<MODE, GATED>(p, t, o, c0 + c, f, u);
        }
    }
}

template <int MODE, bool GATED>
__device__ __forceinline__ void load_octet(const ExpertArgs &p, const Tile &t, int rank, int quadrant, Octet &o) {
    const int lane = threadIdx.x & 31;
    constexpr bool kHalf = GATED && MODE == kForward;
    o.feat = t.feat0 + (kHalf ? rank * 64 + quadrant * 16 + (lane % 2) * 8 : rank * 128 + quadrant * 32 + (lane % 4) * 8);
    o.live = o.feat < (MODE == kForward ? p.N : p.K);
    if (MODE == kForward && p.bias && o.live) {
        const float *b = p.bias + (int64_t)t.e * (GATED ? 2 * (int64_t)p.N : p.N) + o.feat;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.bias[i] = b[i];
        if (GATED) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o.bias_up[i] = b[p.N + i];
        }
    }
}

template <int MODE, bool FP8, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_kernel(const __grid_constant__ CUtensorMap map_m, const __grid_constant__ CUtensorMap map_n,
                  const ExpertArgs p) {
    constexpr bool kHalf = GATED && MODE == kForward;  // half of a block's 128 lanes are up features
    constexpr int kStages = kStagesOf<FP8>;
    constexpr int kStep = FP8 ? 128 : 64;              // reduction elements per stage
    constexpr int kFeatStep = kHalf ? 128 : 256;       // output features per pair
    extern __shared__ __align__(1024) uint8_t smem[];
    float *staging = reinterpret_cast<float *>(smem + kStages * kStageBytes);
    float *scales = reinterpret_cast<float *>(smem + kStages * kStageBytes + kStagingBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes + kStagingBytes + (FP8 ? kScaleBytes : 0));
    const uint32_t base = smem_addr(smem);
    const uint32_t bar0 = smem_addr(bars);
    const uint32_t full = bar0, empty = full + 8 * kStages, tail = empty + 8 * kStages;
    const uint32_t acc_full = tail + 8 * kStages, acc_empty = acc_full + 16;
    const uint32_t sc_full = acc_empty + 16, sc_empty = sc_full + 16, slot = sc_empty + 16;

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int rank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars + i, 2);                 // both blocks' producers (or tail clearers)
            mbar_init(bars + kStages + i, 1);       // a commit
            mbar_init(bars + 2 * kStages + i, 1);   // this block's own tail loads
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + 3 * kStages + i, 1);
            mbar_init(bars + 3 * kStages + 2 + i, 2 * kEpilogueWarps);
            mbar_init(bars + 3 * kStages + 4 + i, kAuxWarps);
            mbar_init(bars + 3 * kStages + 6 + i, kEpilogueWarps);
        }
        mbar_init_fence();
        tma_prefetch_map(&map_m);
        tma_prefetch_map(&map_n);
    }
    if (warp == kMmaWarp) tmem_alloc_pair(slot, 512);
    tcgen05_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tcgen05_fence_after();
    const uint32_t tmem = *reinterpret_cast<const volatile uint32_t *>(bars + 3 * kStages + 8);
    pdl_wait();
    pdl_trigger();

    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    Walker<MODE, kStep> walk(p, kFeatStep);
    Tile t;
    bool ok = true;

    // 384 threads launch with 168 registers each; the e4m3 sums of 128 columns need more
    if (warp >= kEpilogueWarps) {
    if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kProducerWarp) {
        const uint32_t lead_full = map_to_rank(full, 0), own_tail = map_to_rank(tail, rank);
        int stage = 0, issued = 0;
        uint32_t parity = 1;
        for (int tile = pair; ok && walk.next(tile, t); tile += pairs) {
            const int half = t.n / 2;
            const int boxes = MODE == kWgrad ? (half + 63) / 64 : (half + kRowBox - 1) / kRowBox;
            const uint32_t bytes = kOperandBytes + boxes * (MODE == kWgrad ? 64 : kRowBox) * 128;
            // one thread runs the tile's steps, the warp rejoins for the next tile
            if (elect_one()) {
                const int feat = t.feat0 + rank * (kHalf ? 64 : 128);
                const int row = t.row0 + rank * half;
                int st = stage;
                uint32_t ph = parity;
                for (int k = 0; k < t.steps; ++k) {
                    if (!(ok = mbar_wait_cluster(empty + 8 * st, ph))) break;
                    const uint32_t a = base + st * kStageBytes, b = a + kOperandBytes;
                    // a ragged last step of wgrad completes on this block's own barrier: its
                    // rows past the region are cleared before the pair sees the stage
                    const bool ragged = MODE == kWgrad && k == t.steps - 1 && (t.count & 63) != 0;
                    const uint32_t bar = (ragged ? own_tail : lead_full) + 8 * st;
                    mbar_arrive_tx_cluster(bar, bytes);
                    if (MODE == kForward) {
                        if (kHalf)
                            tma_5d(a, &map_m, k * kStep, 0, 0, feat / 16, t.e, bar);
                        else
                            tma_3d(a, &map_m, k * kStep, feat, t.e, bar);
                    } else if (MODE == kDgrad) {
                        tma_3d(a, &map_m, feat, k * kStep, t.e, bar);
                        tma_3d(a + 8192, &map_m, feat + 64, k * kStep, t.e, bar);
                    } else {
                        tma_2d(a, &map_m, feat, t.start + k * kStep, bar);
                        tma_2d(a + 8192, &map_m, feat + 64, t.start + k * kStep, bar);
                    }
                    for (int i = 0; i < boxes; ++i) {
                        if (MODE == kWgrad)
                            tma_2d(b + i * 8192, &map_n, row + i * 64, t.start + k * kStep, bar);
                        else
                            tma_2d(b + i * kRowBox * 128, &map_n, k * kStep, t.start + row + i * kRowBox, bar);
                    }
                    if (++st == kStages) st = 0, ph ^= 1;
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            issued += t.steps;
            stage += t.steps;
            parity ^= (stage / kStages) & 1;
            stage %= kStages;
        }
        // the last stages' releases arrive before this block may go
        for (int i = 0; ok && i < min(issued, kStages); ++i) {
            ok = mbar_wait_cluster(empty + 8 * stage, parity);
            if (++stage == kStages) stage = 0, parity ^= 1;
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            int stage = 0, buf = 0;
            uint32_t parity = 0, acc_parity = 1;
            const uint64_t desc_a = smem_desc(base, 8192), desc_b = smem_desc(base + kOperandBytes, 8192);
            for (int tile = pair; ok && walk.next(tile, t); tile += pairs) {
                if (t.steps == 0) continue;
                const uint32_t desc = mma_desc<FP8, MODE != kForward, MODE == kWgrad>(t.n);
                if (elect_one()) {
                    int st = stage, bf = buf;
                    uint32_t ph = parity, aph = acc_parity;
                    for (int k = 0; k < t.steps; ++k) {
                        const bool fresh = FP8 || k == 0, last = FP8 || k == t.steps - 1;
                        if (fresh && !(ok = mbar_wait_cluster(acc_empty + 8 * bf, aph))) break;
                        if (!(ok = mbar_wait_cluster(full + 8 * st, ph))) break;
                        if (MODE == kWgrad && k == t.steps - 1 && (t.count & 63)) fence_acquire_cluster();
                        tcgen05_fence_after();
                        // a quarter of the stage's reduction: 32 bytes along a K-major row, or
                        // 16 rows of 128 bytes
                        constexpr uint64_t kA = MODE != kForward ? 128 : 2, kB = MODE == kWgrad ? 128 : 2;
                        const uint64_t da = desc_a + (uint32_t)(st * (kStageBytes >> 4));
                        const uint64_t db = desc_b + (uint32_t)(st * (kStageBytes >> 4));
                        const uint32_t d = tmem + bf * kTileRows;
#pragma unroll
                        for (int q = 0; q < 4; ++q) mma_pair<FP8>(d, da + q * kA, db + q * kB, desc, !(fresh && q == 0));
                        mma_commit_pair(empty + 8 * st);
                        if (last) {
                            mma_commit_pair(acc_full + 8 * bf);
                            bf ^= 1;
                            if (bf == 0) aph ^= 1;
                        }
                        if (++st == kStages) st = 0, ph ^= 1;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                stage += t.steps;
                parity ^= (stage / kStages) & 1;
                stage %= kStages;
                buf += FP8 ? t.steps : 1;
                acc_parity ^= (buf >> 1) & 1;
                buf &= 1;
            }
        }
    } else if (warp >= kAuxWarp) {
        if (FP8) {
            const int tid = threadIdx.x - kAuxWarp * 32;
            const int C = p.K / 128;
            const int NW = GATED ? 2 * p.N : p.N;
            const int64_t blocks = (NW + 127) / 128;
            int buf = 0;
            uint32_t parity = 1;
            for (int tile = pair; ok && walk.next(tile, t); tile += pairs) {
                int b0 = (t.feat0 + rank * (kHalf ? 64 : 128)) / 128;
                int b1 = kHalf ? b0 + p.N / 128 : b0;
                if (b0 >= blocks) b0 = 0;  // a block past the features: nothing of it is kept
                if (b1 >= blocks) b1 = 0;
                const float *w0 = p.w_scale + ((int64_t)t.e * blocks + b0) * C;
                const float *w1 = p.w_scale + ((int64_t)t.e * blocks + b1) * C;
                const float *xs = p.x_scale + ((int64_t)t.start + t.row0) * p.srow + t.e * p.sexp;
                for (int g = 0; g < t.steps; g += kScaleGroup) {
                    float sw[2][kScaleGroup], sx[kTileRows / 64][kScaleGroup];
#pragma unroll
                    for (int k = 0; k < kScaleGroup; ++k) {
                        sw[0][k] = g + k < C ? w0[g + k] : 0.0f;
                        sw[1][k] = g + k < C ? w1[g + k] : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < kTileRows / 64; ++i) {
                        const int c = i * 64 + tid;
                        if (c < t.rows && p.scale_vec) {
                            const float4 v = *reinterpret_cast<const float4 *>(xs + c * p.srow + g);
                            sx[i][0] = v.x, sx[i][1] = v.y, sx[i][2] = v.z, sx[i][3] = v.w;
                        } else {
#pragma unroll
                            for (int k = 0; k < kScaleGroup; ++k)
                                sx[i][k] = c < t.rows && g + k < C ? xs[c * p.srow + (g + k) * p.scol] : 0.0f;
                        }
                    }
                    if (!(ok = mbar_wait_cluster(sc_empty + 8 * buf, parity))) break;
                    float *dst = scales + buf * kScaleGroup * 2 * kTileRows;
#pragma unroll
                    for (int i = 0; i < kTileRows / 64; ++i) {
                        const int c = i * 64 + tid;
                        if (c < t.n) {
#pragma unroll
                            for (int k = 0; k < kScaleGroup; ++k) {
                                dst[(k * 2) * kTileRows + c] = sx[i][k] * sw[0][k];
                                if (kHalf) dst[(k * 2 + 1) * kTileRows + c] = sx[i][k] * sw[1][k];
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_to_rank(sc_full, rank) + 8 * buf);
                    buf ^= 1;
                    if (buf == 0) parity ^= 1;
                }
            }
        } else if (MODE == kWgrad && warp == kAuxWarp) {
            const uint32_t lead_full = map_to_rank(full, 0);
            int at = 0;                // stages used so far, modulo their number
            uint32_t parities = 0;     // of each stage's tail barrier
            for (int tile = pair; ok && walk.next(tile, t); tile += pairs) {
                at = (at + t.steps) % kStages;
                if ((t.count & 63) == 0) continue;
                const int stage = (at + kStages - 1) % kStages;
                if (!(ok = mbar_wait_cluster(tail + 8 * stage, (parities >> stage) & 1))) break;
                parities ^= 1u << stage;
                const int from = t.count & 63;
                const int boxes = 2 + (t.n / 2 + 63) / 64;  // the features' two, then the rows'
                uint8_t *s = smem + stage * kStageBytes;
                for (int i = lane; i < boxes * (64 - from) * 8; i += 32) {
                    const int box = i / ((64 - from) * 8), r = i - box * (64 - from) * 8;
                    *reinterpret_cast<uint4 *>(s + box * 8192 + from * 128 + r * 16) = make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_release_cluster(lead_full + 8 * stage);
            }
        }
    }
    } else {
        if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int quadrant = warp & 3, half = warp >> 2;
        float *stage = staging + warp * kStageCols * kStageStride;
        const uint32_t lead_empty = map_to_rank(acc_empty, 0);
        const uint32_t my_tmem = tmem + ((uint32_t)(quadrant * 32) << 16);
        int buf = 0;
        uint32_t parity = 0;
        int sbuf = 0;
        uint32_t sparity = 0;
        Octet o;
        for (int tile = pair; ok && walk.next(tile, t); tile += pairs) {
            load_octet<MODE, GATED>(p, t, rank, quadrant, o);
            const int chunks = t.n / 32;
            if (FP8) {
                float acc[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 32; ++c) acc[i][c] = 0.0f;
                for (int k = 0; k < t.steps; ++k) {
                    const int kg = k % kScaleGroup;
                    if (kg == 0 && !(ok = mbar_wait_cluster(sc_full + 8 * sbuf, sparity))) break;
                    const float *sc = scales + ((sbuf * kScaleGroup + kg) * 2 + (kHalf && lane >= 16 ? 1 : 0)) * kTileRows;
                    if (!(ok = mbar_wait_cluster(acc_full + 8 * buf, parity))) break;
                    tcgen05_fence_after();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ch = 2 * i + half;
                        if (ch < chunks) {
                            uint32_t v[32];
                            tmem_ld32(v, my_tmem + buf * kTileRows + ch * 32);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 s = *reinterpret_cast<const float4 *>(sc + ch * 32 + c);
                                acc[i][c] = fmaf(__uint_as_float(v[c]), s.x, acc[i][c]);
                                acc[i][c + 1] = fmaf(__uint_as_float(v[c + 1]), s.y, acc[i][c + 1]);
                                acc[i][c + 2] = fmaf(__uint_as_float(v[c + 2]), s.z, acc[i][c + 2]);
                                acc[i][c + 3] = fmaf(__uint_as_float(v[c + 3]), s.w, acc[i][c + 3]);
                            }
                        }
                    }
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(lead_empty + 8 * buf);
                    buf ^= 1;
                    if (buf == 0) parity ^= 1;
                    if (kg == kScaleGroup - 1 || k == t.steps - 1) {
                        if (lane == 0) mbar_arrive_cluster(map_to_rank(sc_empty, rank) + 8 * sbuf);
                        sbuf ^= 1;
                        if (sbuf == 0) sparity ^= 1;
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (2 * i + half < chunks) finish_columns<MODE, GATED>(p, t, o, stage, acc[i], (2 * i + half) * 32);
            } else {
                if (t.steps > 0) {
                    if (!(ok = mbar_wait_cluster(acc_full + 8 * buf, parity))) break;
                    tcgen05_fence_after();
                }
                for (int ch = half; ch < chunks; ch += 2) {
                    uint32_t v[32];
                    float f[32];
                    if (t.steps > 0) {
                        tmem_ld32(v, my_tmem + buf * kTileRows + ch * 32);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) f[c] = __uint_as_float(v[c]);
                    } else {  // wgrad of an expert without rows
#pragma unroll
                        for (int c = 0; c < 32; ++c) f[c] = 0.0f;
                    }
                    finish_columns<MODE, GATED>(p, t, o, stage, f, ch * 32);
                }
                if (t.steps > 0) {
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(lead_empty + 8 * buf);
                    buf ^= 1;
                    if (buf == 0) parity ^= 1;
                }
            }
        }
    }
    if (!ok && lane == 0) report(p.status, EPD_ERR_TIMEOUT);
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tcgen05_fence_after();
    if (warp == kMmaWarp) tmem_free_pair(tmem, 512);
}

// dbias[e, n] = the sum of the expert's rows of dy: a block per 64 columns of an expert, eight
// rows at a time in a fixed order.
__global__ void __launch_bounds__(256) bias_grad_kernel(const epd_expert_rows_t rows, const uint8_t *dy, int N,
                                                        float *dbias, int32_t *status) {
    __shared__ float s_sum[32][64];
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y, oct = threadIdx.x & 7, part = threadIdx.x >> 3;
    const int n = blockIdx.x * 64 + oct * 8;
    int start, count;
    expert_region(rows, e, start, count, status);
    float sum[8] = {};
    if (n < N) {
        for (int r = part; r < count; r += 32) {
            float f[8];
            unpack8_bf16(ld_stream16(dy + (((int64_t)start + r) * N + n) * 2), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += f[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[part][oct * 8 + i] = sum[i];
    __syncthreads();
    if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += s_sum[i][threadIdx.x];
        dbias[(int64_t)e * N + blockIdx.x * 64 + threadIdx.x] = v;
    }
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

template <int MODE, bool FP8, bool GATED>
epd_status_t launch(const CUtensorMap &m, const CUtensorMap &n, const ExpertArgs &p, cudaStream_t stream) {
    constexpr int kSmem = kSmemOf<FP8>;
    auto kernel = expert_kernel<MODE, FP8, GATED>;
    static const int pairs = [&] {
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int found = 0;
        if (cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) != cudaSuccess) found = 0;
        cudaGetLastError();
        return found < 1 ? 1 : found;
    }();
    const int features = MODE == kForward ? p.N : p.K;
    const int64_t feat_tiles = (features + (GATED && MODE == kForward ? 127 : 255)) / (GATED && MODE == kForward ? 128 : 256);
    const int64_t row_tiles = MODE == kWgrad
                                  ? (int64_t)(p.N + kTileRows - 1) / kTileRows * p.rows.num_experts
                                  : p.rows.capacity_rows / kTileRows + (p.rows.num_experts < p.rows.capacity_rows
                                                                            ? p.rows.num_experts
                                                                            : p.rows.capacity_rows);
    const int64_t most = feat_tiles * row_tiles;
    if (most > INT32_MAX / 2) return EPD_ERR_UNSUPPORTED;
    return launch_pdl(kernel, 2 * (int)(most < pairs ? most : pairs), kThreads, kSmem, stream, m, n, p);
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

extern "C" epd_status_t ep_expert_matmul(const epd_expert_rows_t *rows, const void *x,
                                         epd_dtype_t dtype, const float *x_scale,
                                         int64_t scale_row_stride, int64_t scale_col_stride,
                                         int64_t scale_expert_stride, const void *w,
                                         const float *w_scale, int in_features, int out_features,
                                         epd_activation_t activation, const float *bias,
                                         const void *residual, void *y, void *preact,
                                         int32_t *status, epd_stream_t stream) {
    using namespace epd;
    const int K = in_features, N = out_features;
    const bool fp8 = dtype == EPD_FP8_E4M3, gated = activation == EPD_ACT_SWIGLU;
    if (!rows_ok(rows) || !act_ok(activation)) return EPD_ERR_INVALID_ARG;
    if (dtype != EPD_BF16 && !fp8) return EPD_ERR_INVALID_ARG;
    if (K < 1 || N < 1 || K % (fp8 ? 128 : 8) != 0 || N % (gated ? (fp8 ? 128 : 16) : 8) != 0)
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
    CUtensorMap mw, mx;
    bool done = encode_rows(&mx, fp8, x, rows->capacity_rows, K, kRowBox);
    const cuuint32_t wide = fp8 ? 128 : 64;
    const cuuint64_t E = (cuuint64_t)rows->num_experts;
    if (gated) {
        // 16 gate rows, then the same features' 16 up rows: one warp's lanes of the accumulator
        const cuuint64_t size[5] = {(cuuint64_t)K, 16, 2, (cuuint64_t)N / 16, E};
        const int64_t stride[4] = {K, (int64_t)N * K, 16 * (int64_t)K, 2 * (int64_t)N * K};
        const cuuint32_t box[5] = {wide, 16, 2, 4, 1};
        done = done && encode(&mw, fp8, 5, w, size, stride, box);
    } else {
        const cuuint64_t size[3] = {(cuuint64_t)K, (cuuint64_t)N, E};
        const int64_t stride[2] = {K, (int64_t)N * K};
        const cuuint32_t box[3] = {wide, 128, 1};
        done = done && encode(&mw, fp8, 3, w, size, stride, box);
    }
    if (!done) return EPD_ERR_CUDA;
    if (fp8)
        return gated ? launch<kForward, true, true>(mw, mx, p, st) : launch<kForward, true, false>(mw, mx, p, st);
    return gated ? launch<kForward, false, true>(mw, mx, p, st) : launch<kForward, false, false>(mw, mx, p, st);
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
    p.rows = *rows;
    p.act = activation;
    p.K = K;
    p.N = N;
    p.preact_in = static_cast<const uint8_t *>(preact);
    p.y = static_cast<uint8_t *>(dx);
    p.status = status;
    CUtensorMap mw, my;
    const cuuint64_t size[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)rows->num_experts};
    const int64_t stride[2] = {K, (int64_t)N * K};
    const cuuint32_t box[3] = {64, 64, 1};
    if (!encode_rows(&my, false, dy, rows->capacity_rows, N, kRowBox) || !encode(&mw, false, 3, w, size, stride, box))
        return EPD_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return activation == EPD_ACT_SWIGLU ? launch<kDgrad, false, true>(mw, my, p, st)
                                        : launch<kDgrad, false, false>(mw, my, p, st);
}

extern "C" epd_status_t ep_expert_matmul_wgrad(const epd_expert_rows_t *rows, const void *dy,
                                               const void *x, int in_features, int out_features,
                                               void *dw, float *dbias, int32_t *status,
                                               epd_stream_t stream) {
    using namespace epd;
    const int K = in_features, N = out_features;
    if (!rows_ok(rows)) return EPD_ERR_INVALID_ARG;
    if (K < 1 || N < 1 || K % 8 != 0 || N % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status) || !dw || !aligned16(dw) || (dbias && !aligned4(dbias)))
        return EPD_ERR_INVALID_ARG;
    if (rows->capacity_rows > 0 && (!dy || !aligned16(dy) || !x || !aligned16(x)))
        return EPD_ERR_INVALID_ARG;
    ExpertArgs p = {};
    p.rows = *rows;
    p.K = K;
    p.N = N;
    p.y = static_cast<uint8_t *>(dw);
    p.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // without rows nothing is loaded, but a map has to lie somewhere
    const bool any = rows->capacity_rows > 0;
    CUtensorMap mx, my;
    if (!encode_rows(&mx, false, any ? x : dw, rows->capacity_rows, K, 64) ||
        !encode_rows(&my, false, any ? dy : dw, rows->capacity_rows, N, 64))
        return EPD_ERR_CUDA;
    const epd_status_t rc = launch<kWgrad, false, false>(mx, my, p, st);
    if (rc != EPD_OK || !dbias) return rc;
    bias_grad_kernel<<<dim3((N + 63) / 64, rows->num_experts), 256, 0, st>>>(
        *rows, static_cast<const uint8_t *>(dy), N, dbias, status);
    return record_cuda_error();
}
