// attention.cu -- attention of one new token over the paged key-value cache (ep_decode_attention).
//
//   o[b, h] = sum_t softmax_t(scale q[b, h] . k[t, h / G]) v[t, h / G],   G = heads / kv heads
//
// Bound by HBM: every live key and value is read once, for G heads at a time, and G <= 16 heads are
// 16 operations a byte at most. One pass with running maxima and sums.
//
// Split: a block's warps form teams, one for each of up to eight kv heads, so that a block reads
// whole rows of a [page, row, head, dim] cache: of rows of one head alone, 128 bytes out of every KB
// are served at two thirds of the memory's rate (128 sequences of 0 to 8191 tokens in e4m3, 64 heads
// over 8 of 128: 248 us alone, 199 in teams, 205 with the check of the values' scales; their 1.1 GB take 166) and 256 out of every two at 0.95
// (bf16, 32 heads over 8: 345 and 329 us; 2.1 GB take 322). The (sequence, group of heads)
// segments of the batch, each as many tiles of a team's tokens as its length needs, form one line of
// tiles, and every block takes an equal run of it, whatever the lengths are (they are read on the
// device). A segment that lies in one block's run is finished there, by each team for its head; of one
// that several blocks share the parts go to the workspace, and the team that comes last joins its
// head's in the blocks' order. Where the batch has few segments (a long context alone) the teams take
// fewer heads with more warps each, so that the joins have fewer parts and more blocks for them: one
// sequence of 1000 tokens takes 8.5 us (0.6 for its 4 MB: two trips to memory for lengths and pages, one
// for the tile, the counter's and the join's), two of 131072 to 200001 in e4m3, 64 heads over 4, 82.4
// (350 MB take 52; 8 go into start and joins, and the rest is the chain of a tile's instructions, the
// widening of every value before its product among them, with two warps on a scheduler: 36 % of the issue
// slots are used). Teams there made 81.5 into 93 to 122: their joins have few warps and many parts.
//
// A warp has its own tokens of each tile, its own two stages in shared memory, filled by its own
// asynchronous copies one tile ahead (past the ends of segments; page numbers are looked up one tile
// before), and its own statistics; warps meet at a segment's end only, and only a team's. Scores
// and outputs are products on the warp-level matrix instructions with the tokens (of scores) and the
// columns (of outputs) as their 16 rows and 8 query heads as their columns, so that a group of 8
// heads fills them. A bf16 cache's take a fraction of the time that its bytes take (12 % of the tensor pipe),
// and tcgen05's could not make it shorter; of an e4m3 cache with 16 heads, where they and the widening do
// take longer than the bytes, tcgen05 with 128 tokens as its rows and e4m3 operands has not been tried.
//
// Precision: products of bf16 are exact, sums in 32 bits. The weights of a bf16 cache's values are split
// into two bf16 (15 bits at least), so that the output's own rounding is the only one that matters. An
// e4m3 cache is widened to fp16, which holds it exactly; a head's query is scaled by a power of two and
// the weights, with the values' scales in them, by a reference that follows the scales, to fp16's range (11
// bits: an eighth of the output's rounding).
#include <cuda_fp16.h>

#include <type_traits>

#include "cache.cuh"

namespace epd {
namespace {

constexpr int kMaxBlocks = 160;  // blocks that the workspace has room for
constexpr int kMaxHeads = 16;    // query heads of a segment, at most
constexpr int kMaxTeams = 8;
// Tiles of a segment that one block takes whole: a join costs as much as about four of them (256
// sequences of 10 to 300 tokens: 44 us, 76 with all of them cut where the shares end; with 8 tiles one
// sequence of 1000 tokens is left to 8 blocks, and takes 14.8 us instead of 8.5).
constexpr int kUncut = 4;
// Tokens of a segment after which a warp puts its sums aside and starts new ones. The matrix instructions cut
// their sums off where an addition would round, which loses in one direction: 1e-4 of the output over 9000 tokens
// of a bf16 cache in one warp, 3.5e-4 over 30000 and 3.3e-3 (the output's own rounding) over 300000, half of
// that of an e4m3 cache. With runs of 2048 it is 2e-5 whatever the length is.
constexpr int kRunTokens = 2048;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;
// A maximum is moved (and everything summed so far scaled down) only when a score passes it by more
// than a factor: terms up to 2^8 lose nothing in 32 bits, and the scaling is rare. Of an e4m3 cache,
// whose weights are fp16, it is 2^4, the values' scales may pass their reference by 4, and the weights
// are 2^9 as large as they are: 2^15 at most, and off by 2^-11 of their size, or by 2^-34 where that is more and the
// scale is the reference, so that what a quarter of a million tokens of small weights lose is far below the
// output's own rounding.
constexpr float kSlack = 8.0f, kSlackFp8 = 4.0f;
constexpr float kValueSlack = 4.0f, kWeightUp = 512.0f;
// A value's scale goes into its fp16 weight over a reference, a power of two that follows the scales. A tile
// with one above kValueSlack of it, one below kValueRange or none from kValueNear up moves it to the tile's
// largest (never below kValueFall of the segment's largest, so that the sums stay in 32 bits), and the
// scales that are below its range then take another turn over the tile, with a reference of their own: a row of
// zeros has scale 1, and may lie among values of any size. With one reference that only rose, a single such row
// among 1000 of scale 2^-27 left 0.6 % of the output wrong, of 2^-37 26 %; now 0.17 % whatever the scales are
// (the output's own rounding). The check cost 0.5 to 3 % (two of 131072 to 200001 tokens, 64 heads over 4: 81.8 and
// 84.6 us with it); a row of zeros in every 1000 another 1 %, in every 50, where most tiles take two turns, 24 %.
constexpr float kValueRange = 0x1p-8f, kValueNear = 0x1p-3f, kValueFall = 0x1p-64f;
constexpr float kLeastRef = 0x1p-119f;  // of a reference over kWeightUp: its inverse is finite

struct AttnArgs {
    const uint8_t *q;
    int64_t q_stride;  // bytes between tokens
    int QH, group, blocks_of_group;  // segments of a group
    int teams, teams_log, tile_log;  // kv heads at once; log2 of a tile's tokens
    int head_groups;                 // kv heads / teams
    epd_cache_t kv;
    Divisor page;
    const int32_t *lengths;
    int window;
    float scale_log2;
    int aligned;  // every run of 16 positions from a multiple of 16 lies on one page, and tiles begin at such
    uint8_t *out;  // bf16 [B, QH, D]
    float *lse;
    uint32_t *counters;
    float *parts, *aside;
    int32_t *status;
};

// Floats of a warp's sums put aside: of outputs, of weights with their maxima, and the values' reference.
constexpr int aside_floats(int DP, int NH) { return (DP / 16 * NH * 4 + NH * 4 + 4) * 32; }

template <int DP, bool FP8, int NH>
struct Shape {
    static constexpr int kHeads = 8 * NH;                   // of a segment
    static constexpr int kRow = DP * (FP8 ? 1 : 2);         // bytes of a row in shared memory
    static constexpr int kUnits = kRow / 16;
    static constexpr int kChunk = kRow <= 128 ? 32 : 16;    // tokens of a warp's tile
    static constexpr int kTail = (FP8 ? 2 * kChunk * 4 : 0) + 16;  // scales and the live tokens' mask
    static constexpr int kStage = 2 * kChunk * kRow + kTail;
    static constexpr int kWarps = kRow == 512 ? 4 : 8;
    static constexpr bool kQueryInSmem = DP * NH >= 512;    // the query's fragments, where registers have no room
    static constexpr int kQuery = kQueryInSmem ? DP / 16 * NH * 32 * 8 : 0;  // bytes, of a team
    static constexpr int kJoinCols = kQueryInSmem ? (FP8 ? 32 : 64) : DP < 128 ? DP : 128, kJoinRow = kJoinCols + 4;
    static constexpr int kJoin = kWarps * kHeads * kJoinRow * 4;
    // One stage on the way (64 KB a multiprocessor) while another is read. More in flight fill the same
    // memory system, but share it less evenly: of 152 blocks with equal runs, each of one kv head's rows,
    // the fastest then takes 256 us and the slowest 348 (128 sequences, 2.1 GB; 361 us in all), with
    // two stages 303 and 337 (344).
    static constexpr int kStages = 2;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kSmem = kWarps * (kStages * kStage + kQuery) + kJoin;
    static constexpr int kPart = kHeads * (DP + 2);  // floats: the heads' sums, maxima and sums of weights
    static constexpr int kAside = aside_floats(DP, NH);
    static_assert(kSmem <= 226 * 1024 - 2048, "the ring and the join share what a block may have");
};

__device__ __forceinline__ void copy16z(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4z(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// d += a b, 16 x 8 x 16.
template <bool FP8>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (FP8)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 as two pairs of fp16, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Place of 16-byte unit u of a row in shared memory: eight rows of one unit lie in eight bank groups.
template <int UNITS>
__device__ __forceinline__ int swizzle(int row, int u) {
    return UNITS % 8 == 0 ? u ^ (row & 7) : u ^ ((row >> 1) & 3);
}

// The live positions [lo, n) of a sequence and its tiles (one at least: an empty one is written too).
struct Span {
    int lo, n, tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, int len) {
    const int64_t most = cache_positions(a.kv);
    Span s;
    s.n = len < 0 ? 0 : (int64_t)len > most ? (int)most : len;
    s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
    s.tiles = s.n > 0 ? ((s.n - s.lo - 1) >> a.tile_log) + 1 : 1;
    return s;
}

// A place on the line of tiles: tile `tile` of segment (b, heads h * teams and on, block).
struct Cursor {
    int b, h, block, tile, next_len;
    Span span;
    __device__ __forceinline__ void enter(const AttnArgs &a, int len) {
        span = span_of(a, len);
        next_len = b + 1 < a.kv.num_seqs ? __ldg(a.lengths + b + 1) : 0;
    }
    __device__ __forceinline__ void advance(const AttnArgs &a) {
        if (++tile < span.tiles) return;
        tile = 0;
        if (++block < a.blocks_of_group) return;
        block = 0;
        if (++h < a.head_groups) return;
        h = 0;
        ++b;
        enter(a, next_len);
    }
};

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

__device__ __forceinline__ uint32_t add_acq_rel(uint32_t *p, uint32_t v) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// The 8 x 8 matrix of 16-bit values with its rows and columns exchanged.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Joins n parts of a segment: part 0 at `part0`, the others `stride` floats apart from `part1`. A warp
// takes every mates-th row from `sub`, RG of them at a time with the loads of PB parts on the way; lane i
// has the weights of part i.
template <int DP, int HB, int RG, int PB>
__device__ __forceinline__ void combine_parts(const float *part0, const float *part1, int64_t stride, int n, int rows, int sub, int mates,
                                           int D, uint8_t *out, float *lse) {
    constexpr int C = DP / 32;
    const int lane = threadIdx.x & 31, col = lane * C;
    auto at_part = [&](int i) { return i == 0 ? part0 : part1 + (int64_t)(i - 1) * stride; };
    for (int rb = sub; rb < rows; rb += RG * mates) {
        float top[RG], sum[RG], v[RG][C], x[PB][RG][C], m0[RG], l0[RG];
        auto statistic = [&](int i, int j, int which) {
            const int r = rb + j * mates;
            return i < n && r < rows ? __ldcg(at_part(i) + HB * DP + which * HB + r) : which ? 0.0f : -INFINITY;
        };
        auto fetch = [&](int i0) {
#pragma unroll
            for (int i = 0; i < PB; ++i)
#pragma unroll
                for (int j = 0; j < RG; ++j) {
                    const bool has = i0 + i < n && rb + j * mates < rows;
                    const float *src = at_part(i0 + i) + (rb + j * mates) * DP + col;
#pragma unroll
                    for (int k = 0; k < C; k += C < 4 ? 2 : 4) {
                        if (C < 4) {
                            const float2 y = has ? __ldcg(reinterpret_cast<const float2 *>(src)) : make_float2(0.0f, 0.0f);
                            x[i][j][0] = y.x, x[i][j][1] = y.y;
                        } else {
                            const float4 y = has ? __ldcg(reinterpret_cast<const float4 *>(src + k)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            x[i][j][k] = y.x, x[i][j][k + 1] = y.y, x[i][j][(k + 2) % C] = y.z, x[i][j][(k + 3) % C] = y.w;
                        }
                    }
                }
        };
        // all that the first parts need is on its way at once
        fetch(0);
#pragma unroll
        for (int j = 0; j < RG; ++j) {
            m0[j] = statistic(lane, j, 0);
            l0[j] = statistic(lane, j, 1);
            top[j] = m0[j];
            sum[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) v[j][i] = 0.0f;
        }
        for (int i = lane + 32; i < n; i += 32) {
#pragma unroll
            for (int j = 0; j < RG; ++j) top[j] = fmaxf(top[j], statistic(i, j, 0));
        }
#pragma unroll
        for (int j = 0; j < RG; ++j)
#pragma unroll
            for (int d = 16; d; d >>= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(kAll, top[j], d));
        for (int c0 = 0; c0 < n; c0 += 32) {
            float f[RG];
#pragma unroll
            for (int j = 0; j < RG; ++j) {
                const float mi = c0 == 0 ? m0[j] : statistic(c0 + lane, j, 0), li = c0 == 0 ? l0[j] : statistic(c0 + lane, j, 1);
                f[j] = mi == -INFINITY ? 0.0f : fast_exp2(mi - top[j]);
                sum[j] = fmaf(f[j], li, sum[j]);
            }
            const int here = min(32, n - c0);
            for (int i0 = 0; i0 < here; i0 += PB) {
                if (c0 + i0 > 0) fetch(c0 + i0);
#pragma unroll
                for (int i = 0; i < PB; ++i)
#pragma unroll
                    for (int j = 0; j < RG; ++j) {
                        // (what lies past the chunk's 32 parts is never fetched: PB divides 32)
                        const float by = __shfl_sync(kAll, f[j], i0 + i);
#pragma unroll
                        for (int k = 0; k < C; ++k) v[j][k] = fmaf(x[i][j][k], by, v[j][k]);
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < RG; ++j) {
            const int r = rb + j * mates;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum[j] += __shfl_xor_sync(kAll, sum[j], d);
            const float inv = sum[j] > 0.0f ? __fdiv_rn(1.0f, sum[j]) : sum[j];
            if (r >= rows) continue;
            if (lse && lane == 0) lse[r] = (top[j] + log2f(sum[j])) * kLn2;  // -inf of none
            if (col < D) {
#pragma unroll
                for (int k = 0; k < C; k += 2)
                    *reinterpret_cast<uint32_t *>(out + ((int64_t)r * D + col + k) * 2) = pack2_bf16(v[j][k] * inv, v[j][k + 1] * inv);
            }
        }
    }
}

// v, as a value that the compiler does not know.
__device__ __forceinline__ int64_t opaque(int64_t v) {
    asm volatile("" : "+l"(v));
    return v;
}

template <int DP, bool FP8, int NH>
__global__ void __launch_bounds__(Shape<DP, FP8, NH>::kThreads, 1) attention_kernel(AttnArgs a) {
    using S = Shape<DP, FP8, NH>;
    constexpr int W = S::kWarps, UNITS = S::kUnits, CH = S::kChunk, MT = CH / 16, KT = DP / 16;
    constexpr int HB = S::kHeads;
    extern __shared__ uint4 s_dyn[];
    __shared__ int64_t s_scan[W];
    __shared__ float2 s_ml[W][HB], s_all[W][HB];  // maxima and sums of weights, a warp's and a team's
    __shared__ uint32_t s_last[W];
    __shared__ float s_top[W];  // a warp's largest reference of the values' scales in a segment
    // what only a segment's end needs, so that it takes no registers of the loop: each warp's place and the
    // tiles of the sequences before it, and the block's run
    __shared__ Cursor s_cursor[W], s_load[W];
    __shared__ int64_t s_before[W], s_run[5];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int D = a.kv.head_dim, B = a.kv.num_seqs, heads = a.head_groups * a.blocks_of_group;  // segments of a sequence
    // the warp's team, its place there, the team's warps and threads
    const int team = warp & (a.teams - 1), sub = warp >> a.teams_log, mates = W >> a.teams_log, tt = sub * 32 + lane;
    auto team_sync = [&]() {
        if (mates == 1) __syncwarp();
        else named_barrier_sync(1 + team, mates * 32);
    };
    const uint32_t ring = smem_addr(s_dyn) + warp * S::kStages * S::kStage;
    float *const s_join = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(s_dyn) + W * S::kStages * S::kStage);
    uint2 *const s_query = reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(s_join) + S::kJoin + team * S::kQuery);
    // columns past D stay zero
    if (D < DP) {
        uint4 *mine = s_dyn + warp * S::kStages * S::kStage / 16;
        for (int i = lane; i < S::kStages * S::kStage / 16; i += 32) mine[i] = make_uint4(0, 0, 0, 0);
    }
    pdl_wait();
    pdl_trigger();

    // ---- this block's run of the line: the sequences' tiles are summed by the whole block
    int64_t total = 0;
    if (B > S::kThreads) {
        int64_t v = 0;
        for (int b = tid; b < B; b += S::kThreads) v += span_of(a, __ldg(a.lengths + b)).tiles;
        v = warp_scan(v, lane);
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        for (int w = 0; w < W; ++w) total += s_scan[w];
        __syncthreads();
    }
    // The run is [r0, r1) of the line, an equal share of it; a share that begins inside a segment of few tiles
    // begins after it instead, so that no segment is cut whose join would take longer than its tiles.
    int64_t r0 = 0, r1 = 0, before = 0, blocks = gridDim.x;  // blocks: that have a tile
    for (int b0 = 0; b0 < B; b0 += S::kThreads) {
        const int b = b0 + tid;
        const int64_t v = b < B ? span_of(a, __ldg(a.lengths + b)).tiles : 0;
        int64_t incl = warp_scan(v, lane);
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        int64_t sum = 0;
        for (int w = 0; w < W; ++w) {
            if (w < warp) incl += s_scan[w];
            sum += s_scan[w];
        }
        if (b0 == 0) {
            if (B <= S::kThreads) total = sum;
            total *= heads;
            if (total < blocks) blocks = total;
            if (blockIdx.x >= blocks) return;
            r0 = total * blockIdx.x / blocks;
            r1 = total * (blockIdx.x + 1) / blocks;
        }
        incl += before;
        const int64_t seq0 = (incl - v) * heads, seq1 = incl * heads;
        if (seq0 <= r0 && r0 < seq1) {
            const int64_t rest = r0 - seq0;
            Cursor at;
            at.b = b;
            int hh = (int)(rest / v);
            at.tile = (int)(rest - hh * v);
            int64_t first = r0, prefix = incl - v;
            if (at.tile > 0 && v <= kUncut) {
                first += v - at.tile;
                at.tile = 0;
                if (++hh == heads) {
                    hh = 0;
                    ++at.b;
                    prefix = incl;
                }
            }
            at.h = hh / a.blocks_of_group;
            at.block = hh - at.h * a.blocks_of_group;
            s_cursor[0] = at;
            s_before[0] = prefix;
            s_run[0] = first;
        }
        if (seq0 < r1 && r1 <= seq1) {
            const int64_t into = (r1 - seq0) % v;
            s_run[1] = into > 0 && v <= kUncut ? r1 + v - into : r1;
        }
        before += sum;
        __syncthreads();
        if (before * heads >= r1) break;
    }
    const int steps = (int)(s_run[1] - s_run[0]);
    if (steps <= 0) return;
    Cursor ld = s_cursor[0];
    const int64_t prefix0 = s_before[0];
    if (tid == 0) s_run[2] = total, s_run[3] = blocks, s_run[4] = r0;
    ld.enter(a, __ldg(a.lengths + ld.b));
    __syncthreads();
    int left = ld.span.tiles - ld.tile;  // of the segment's tiles
    if (lane == 0) {
        s_cursor[warp] = s_load[warp] = ld;
        s_before[warp] = prefix0;
    }
    __syncthreads();
    if (blockIdx.x == 0) {  // lengths that the pages do not hold
        for (int b = tid; b < B; b += S::kThreads) {
            const int len = __ldg(a.lengths + b);
            if (len < 0) report(a.status, EPD_ERR_INVALID_ARG);
            else if ((int64_t)len > cache_positions(a.kv)) report(a.status, EPD_ERR_CAPACITY);
        }
    }

    // ---- loads: lane l looks after token l % CH of the warp's chunk
    uint32_t position, end;         // of the token, and of its sequence (a tile may end past 2^31 - 1)
    int seq, kv_head, page, inside;  // page: < 0 for a token past the end; inside: its place there
    int64_t head_off;               // of the kv head in its token
    int load_left;                  // tiles of the segment that are still to be loaded
    auto enter = [&](const Cursor &at) {
        position = (uint32_t)at.span.lo + ((uint32_t)at.tile << a.tile_log) + sub * CH + (lane & (CH - 1));
        end = at.span.n;
        seq = at.b;
        kv_head = (at.h << a.teams_log) + team;
        head_off = kv_head * a.kv.head_stride;
        load_left = at.span.tiles - at.tile;
    };
    auto look_up = [&]() {
        const uint32_t nth = divide(position, a.page);
        inside = (int)(position - nth * a.page.d);
        page = position < end ? __ldg(a.kv.page_table + seq * a.kv.table_stride + nth) : -2;
        if (position < end && page < 0) page = INT32_MAX;  // no page either, but reported
    };
    auto go_on = [&]() {
        if (--load_left > 0) {
            position += 1u << a.tile_log;
        } else {
            Cursor at = s_load[warp];
            at.tile = at.span.tiles - 1;
            at.advance(a);
            enter(at);
            __syncwarp();
            if (lane == 0) s_load[warp] = at;
            __syncwarp();
        }
        look_up();
    };
    const int units = D * (FP8 ? 1 : 2) / 16;
    auto load = [&](int stage) {
        const uint32_t at = ring + stage * S::kStage;
        bool live = page >= 0;
        if (live && page >= a.kv.num_pages) {
            report(a.status, EPD_ERR_CAPACITY);
            live = false;
        }
        const int64_t off = live ? ((int64_t)page * a.kv.page_stride + (int64_t)inside * a.kv.token_stride + head_off) * (FP8 ? 1 : 2) : 0;
        const uint32_t mask = __ballot_sync(kAll, live) & (CH == 32 ? kAll : 0xffffu);
        if (a.aligned && mask == (CH == 32 ? kAll : 0xffffu)) {
            // every 16 tokens lie on one page: one address for them, and a constant step
            constexpr int STEP = 32 / UNITS > 0 ? 32 / UNITS : 1;  // rows of one instruction
            // (not kept in registers from step to step)
            const int64_t step = opaque(a.kv.token_stride) * (FP8 ? 1 : 2);
            const int u = lane % UNITS;
            const uint8_t *const k0 = reinterpret_cast<const uint8_t *>(opaque(reinterpret_cast<int64_t>(a.kv.k))) + (lane / UNITS) * step + u * 16;
            const int64_t to_v = opaque((int64_t)(reinterpret_cast<uintptr_t>(a.kv.v) - reinterpret_cast<uintptr_t>(a.kv.k)));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint8_t *src = k0 + __shfl_sync(kAll, off, 16 * t);
#pragma unroll
                for (int i = 0; i < 16 / STEP; ++i) {
                    const int row = t * 16 + i * STEP + lane / UNITS;
                    const uint32_t dst = at + row * S::kRow + swizzle<UNITS>(row, u) * 16;
                    if (u < units) {
                        copy16(dst, src);
                        copy16(dst + CH * S::kRow, src + to_v);
                    }
                    src += STEP * step;
                }
            }
        } else if (mask) {
#pragma unroll
            for (int i = 0; i < CH * UNITS / 32; ++i) {
                const int row = (i * 32 + lane) / UNITS, u = (i * 32 + lane) % UNITS;
                const int64_t o = __shfl_sync(kAll, off, row) + u * 16;
                const bool has = (mask >> row) & 1;
                const uint32_t dst = at + row * S::kRow + swizzle<UNITS>(row, u) * 16;
                if (u < units) {  // a dead row's copy reads nothing and writes zeros
                    copy16z(dst, static_cast<const uint8_t *>(a.kv.k) + (has ? o : 0), has);
                    copy16z(dst + CH * S::kRow, static_cast<const uint8_t *>(a.kv.v) + (has ? o : 0), has);
                }
            }
        }
        if (FP8 && mask) {
            const int64_t so = live ? (int64_t)page * a.kv.scale_page_stride + (int64_t)inside * a.kv.scale_token_stride + kv_head * a.kv.scale_head_stride : 0;
            const uint32_t dst = at + 2 * CH * S::kRow + (lane & (CH - 1)) * 4;
            if (CH == 32 || lane < 16) copy4z(dst, a.kv.k_scale + so, live);
            if (CH == 32 || lane >= 16) copy4z(dst + CH * 4, a.kv.v_scale + so, live);
        }
        if (lane == 0)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + S::kStage - 16), "r"(mask) : "memory");
    };
    enter(ld);
    look_up();
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) {
        if (s < steps) {
            load(s);
            if (s + 1 < steps) go_on();
        }
        copy_commit();
    }

    // ---- the line. o[k][n][i]: column 16 k + g + 8 (i / 2) (e4m3: 16 k + 2 g + i / 2) of head
    // 8 n + 2 c + i % 2; m and l: of heads 8 n + 2 c, 8 n + 2 c + 1, l of the lane's own tokens
    uint32_t q[KT][NH][2];
    float o[KT][NH][4], m[NH][2], l[NH][2], q_scale[NH][2], v_ref = kLeastRef;
    // Fragments of the query: head g, and the columns that the keys' fragments pair with them -- of a
    // 16-byte unit of an e4m3 row a lane holds four neighbours.
    auto load_query = [&](const Cursor &at) {
        const int rows = a.group - at.block * HB;  // heads of the segment, if fewer than HB
        const uint8_t *src = a.q + at.b * a.q_stride + (int64_t)(((at.h << a.teams_log) + team) * a.group + at.block * HB) * D * 2;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = n * 8 + g, col = k * 16 + (FP8 ? 4 * c + i * 2 : 2 * c + i * 8);
                    q[k][n][i] = row < rows && col < D ? __ldg(reinterpret_cast<const uint32_t *>(src + ((int64_t)row * D + col) * 2)) : 0;
                }
    };
    if (!S::kQueryInSmem) load_query(s_cursor[warp]);
    const float *const scales = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(s_dyn) + warp * S::kStages * S::kStage + 2 * CH * S::kRow);
    int stage = 0;
    // One loop over segments around one over tiles: what only a segment's ends need is out of the inner one's
    // registers (with one loop for both, e4m3 heads of 256 spilled: 178 us, 64 sequences, where they take 109).
    for (int step = 0; step < steps;) {
        {  // a segment begins
            if (S::kQueryInSmem) load_query(s_cursor[warp]);
            if (FP8) {
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    float top = 0.0f;
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) top = fmaxf(top, fmaxf(fabsf(lo_bf16(q[k][n][i])), fabsf(hi_bf16(q[k][n][i]))));
                    top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
                    // the head's largest to [2^6, 2^(6+1)): the power of two from the exponent's bits
                    const int e = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -120) : 0;
                    const float up = __uint_as_float((uint32_t)(127 + 6 - e) << 23);
                    const float down = e < 128 ? __uint_as_float((uint32_t)(127 - 6 + e) << 23) * a.scale_log2 : NAN;
                    q_scale[n][0] = __shfl_sync(kAll, down, 8 * c);
                    q_scale[n][1] = __shfl_sync(kAll, down, 8 * c + 4);
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) q[k][n][i] = pack2_f16(lo_bf16(q[k][n][i]) * up, hi_bf16(q[k][n][i]) * up);
                }
            }
            if (S::kQueryInSmem) {
                // every warp of the team has all of it: each writes its share
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int n = 0; n < NH; ++n)
                        if ((k & (mates - 1)) == sub) s_query[(k * NH + n) * 32 + lane] = make_uint2(q[k][n][0], q[k][n][1]);
                team_sync();
            }
#pragma unroll
            for (int n = 0; n < NH; ++n) {
#pragma unroll
                for (int k = 0; k < KT; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.0f;
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
            }
            v_ref = kLeastRef;
            if (FP8 && lane == 0) s_top[warp] = 0.0f;
        }
        // the segment's tiles, in runs after which the sums are put aside
        const int until = step + min(left, steps - step);
        for (bool aside = false;; aside = true) {
            for (const int stop = min(until, step + kRunTokens / CH); step < stop; ++step) {
                copy_wait<S::kStages - 2>();
                __syncwarp();
                if (step + S::kStages - 1 < steps) {
                    load(stage == 0 ? S::kStages - 1 : stage - 1);
                    if (step + S::kStages < steps) go_on();
                }
                copy_commit();

                const uint32_t at = ring + stage * S::kStage;
                uint32_t mask;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(mask) : "r"(at + S::kStage - 16) : "memory");
                // (an e4m3 tile's values' scales from `done` up have had their turn)
                float done = NAN;
                for (bool turn = mask != 0; turn;) {
                    turn = false;
                    // s[t][n][i]: token 16 t + g + 8 (i / 2), head 8 n + 2 c + i % 2
                    float s[MT][NH][4] = {};
                    const int row = lane & 15, right = lane >> 4;
                    auto query = [&](int k, int n) {
                        return S::kQueryInSmem ? s_query[(k * NH + n) * 32 + lane] : make_uint2(q[k][n][0], q[k][n][1]);
                    };
#pragma unroll
                    for (int k = 0; k < UNITS / 2; ++k)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            uint32_t r[4];
                            ldsm4(r, at + (t * 16 + row) * S::kRow + swizzle<UNITS>(row, 2 * k + right) * 16);
                            if (FP8) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t f[4];
                                    widen4(r[2 * h], f[0], f[2]);
                                    widen4(r[2 * h + 1], f[1], f[3]);
#pragma unroll
                                    for (int n = 0; n < NH; ++n) {
                                        const uint2 b = query(2 * k + h, n);
                                        mma<true>(s[t][n], f, b.x, b.y);
                                    }
                                }
                            } else {
#pragma unroll
                                for (int n = 0; n < NH; ++n) {
                                    const uint2 b = query(k, n);
                                    mma<false>(s[t][n], r, b.x, b.y);
                                }
                            }
                        }
                    const float *const sc = scales + stage * (S::kStage / 4);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const float f[2] = {FP8 ? sc[16 * t + g] : a.scale_log2, FP8 ? sc[16 * t + g + 8] : 0.0f};
#pragma unroll
                        for (int n = 0; n < NH; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[t][n][i] *= FP8 ? q_scale[n][i & 1] * f[i >> 1] : f[0];
                    }
                    if (mask != (CH == 32 ? kAll : 0xffffu)) {
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int n = 0; n < NH; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (!((mask >> (16 * t + g + 8 * (i >> 1))) & 1)) s[t][n][i] = -INFINITY;
                    }
                    float top[NH][2];
                    bool more = false;
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            top[n][i] = fmaxf(s[0][n][i], s[0][n][i + 2]);
#pragma unroll
                            for (int t = 1; t < MT; ++t) top[n][i] = fmaxf(top[n][i], fmaxf(s[t][n][i], s[t][n][i + 2]));
                            more |= top[n][i] > m[n][i] + (FP8 ? kSlackFp8 : kSlack);
                        }
                    if (__any_sync(kAll, more)) {
#pragma unroll
                        for (int n = 0; n < NH; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float now = top[n][i];
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1) now = fmaxf(now, __shfl_xor_sync(kAll, now, d));
                                now = fmaxf(now, m[n][i]);
                                const float f = m[n][i] == -INFINITY ? 0.0f : fast_exp2(m[n][i] - now);
                                m[n][i] = now;
                                l[n][i] *= f;
#pragma unroll
                                for (int k = 0; k < KT; ++k) {
                                    o[k][n][i] *= f;
                                    o[k][n][i + 2] *= f;
                                }
                            }
                    }
                    float vs[MT][2];
                    if (FP8) {
                        float most = 0.0f, least = INFINITY;
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                vs[t][i] = sc[CH + 16 * t + g + 8 * i];
                                const float size = fabsf(vs[t][i]);
                                most = fmaxf(most, size);
                                least = fminf(least, size > 0.0f ? size : INFINITY);
                            }
                        const bool out = most > kValueSlack * kWeightUp * v_ref || least < kValueRange * kWeightUp * v_ref;
                        if (__any_sync(kAll, out) || !__any_sync(kAll, most >= kValueNear * kWeightUp * v_ref)) {
                            most = 0.0f;
#pragma unroll
                            for (int t = 0; t < MT; ++t)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    if (fabsf(vs[t][i]) >= done) vs[t][i] = 0.0f;
                                    most = fmaxf(most, fabsf(vs[t][i]));
                                }
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, d));
                            if (most > 0.0f) {
                                most = __uint_as_float(__float_as_uint(most) & 0x7f800000u) / kWeightUp;
                                const float now = fmaxf(fmaxf(most, kLeastRef), s_top[warp] * kValueFall), f = v_ref / now;
                                v_ref = now;
                                __syncwarp();
                                if (lane == 0) s_top[warp] = fmaxf(s_top[warp], now);
                                __syncwarp();
#pragma unroll
                                for (int k = 0; k < KT; ++k)
#pragma unroll
                                    for (int i = 0; i < 4 * NH; ++i) o[k][i >> 2][i & 3] *= f;
                                if (now == most && now < INFINITY) {
                                    const float least = kValueRange * kWeightUp * now;
                                    bool later = false;
#pragma unroll
                                    for (int t = 0; t < MT; ++t)
#pragma unroll
                                        for (int i = 0; i < 2; ++i)
                                            if (fabsf(vs[t][i]) < least && vs[t][i] != 0.0f) {
                                                vs[t][i] = 0.0f;
                                                later = true;
                                            }
                                    turn = __any_sync(kAll, later);
                                }
                            }
                        }
                        const float v_inv = fast_rcp(v_ref);  // exact: a power of two
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) vs[t][i] *= v_inv;
                    }
                    const float counts = done == done ? 0.0f : 1.0f;  // a token's weight counts once
                    // the weights, turned from (token, head) to (head, token) fragments
                    uint32_t p[MT][NH][2], p_lo[MT][NH][2];
#pragma unroll
                    for (int n = 0; n < NH; ++n) {
                        const float base[2] = {m[n][0] == -INFINITY ? 0.0f : m[n][0], m[n][1] == -INFINITY ? 0.0f : m[n][1]};
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float x = fast_exp2(s[t][n][2 * i] - base[0]), y = fast_exp2(s[t][n][2 * i + 1] - base[1]);
                                l[n][0] = FP8 ? fmaf(x, counts, l[n][0]) : l[n][0] + x;
                                l[n][1] = FP8 ? fmaf(y, counts, l[n][1]) : l[n][1] + y;
                                if (FP8) {
                                    p[t][n][i] = transpose8(pack2_f16(x * vs[t][i], y * vs[t][i]));
                                } else {
                                    // the first part is cut off, not rounded, and the second at least 2^-100:
                                    // neither turns an infinite value's product into NaN
                                    const uint32_t hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
                                    p[t][n][i] = transpose8(hi);
                                    p_lo[t][n][i] = transpose8(pack2_bf16(fmaxf(x - lo_bf16(hi), 0x1p-100f), fmaxf(y - hi_bf16(hi), 0x1p-100f)));
                                }
                            }
                    }
                    const uint32_t av = at + CH * S::kRow;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        if (FP8) {
                            // a 16-byte unit is 16 columns: its even ones are the first 8 rows, its odd ones the others
#pragma unroll
                            for (int k = 0; k < UNITS / 2; ++k) {
                                uint32_t r[4];
                                ldsm4t(r, av + (t * 16 + row) * S::kRow + swizzle<UNITS>(row, 2 * k + right) * 16);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t f[4];
                                    widen4(__byte_perm(r[2 * h], 0, 0x3120), f[0], f[1]);
                                    widen4(__byte_perm(r[2 * h + 1], 0, 0x3120), f[2], f[3]);
#pragma unroll
                                    for (int n = 0; n < NH; ++n) mma<true>(o[2 * k + h][n], f, p[t][n][0], p[t][n][1]);
                                }
                            }
                        } else {
                            const int vrow = (lane & 7) + right * 8;
#pragma unroll
                            for (int k = 0; k < KT; ++k) {
                                uint32_t r[4];
                                ldsm4t(r, av + (t * 16 + vrow) * S::kRow + swizzle<UNITS>(vrow, 2 * k + ((lane >> 3) & 1)) * 16);
#pragma unroll
                                for (int n = 0; n < NH; ++n) {
                                    mma<false>(o[k][n], r, p[t][n][0], p[t][n][1]);
                                    mma<false>(o[k][n], r, p_lo[t][n][0], p_lo[t][n][1]);
                                }
                            }
                        }
                    }
                    if (FP8 && turn) done = kValueRange * kWeightUp * v_ref;
                }
                if (++stage == S::kStages) stage = 0;
            }
            if (!aside && step == until) break;
            // ---- the sums so far and those put aside before, brought to the present maxima and reference
            float4 *const kept = reinterpret_cast<float4 *>(a.aside + (int64_t)(blockIdx.x * W + warp) * S::kAside) + lane;
            if (aside) {
                const float fall = FP8 ? kept[(KT + 1) * NH * 32].x / v_ref : 1.0f;
                float by[NH][2];
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    const float4 x = kept[(KT * NH + n) * 32];
                    by[n][0] = x.x == -INFINITY ? 0.0f : fast_exp2(x.x - m[n][0]);
                    by[n][1] = x.y == -INFINITY ? 0.0f : fast_exp2(x.y - m[n][1]);
                    l[n][0] = fmaf(x.z, by[n][0], l[n][0]);
                    l[n][1] = fmaf(x.w, by[n][1], l[n][1]);
                    if (FP8) by[n][0] *= fall, by[n][1] *= fall;
                }
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int n = 0; n < NH; ++n) {
                        const float4 x = kept[(k * NH + n) * 32];
                        o[k][n][0] = fmaf(x.x, by[n][0], o[k][n][0]);
                        o[k][n][1] = fmaf(x.y, by[n][1], o[k][n][1]);
                        o[k][n][2] = fmaf(x.z, by[n][0], o[k][n][2]);
                        o[k][n][3] = fmaf(x.w, by[n][1], o[k][n][3]);
                    }
            }
            if (step == until) break;
            if (FP8) kept[(KT + 1) * NH * 32].x = v_ref;
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                kept[(KT * NH + n) * 32] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
                l[n][0] = l[n][1] = 0.0f;
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    kept[(k * NH + n) * 32] = make_float4(o[k][n][0], o[k][n][1], o[k][n][2], o[k][n][3]);
                    o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.0f;
                }
            }
        }

        {
            // ---- the segment's end here: join the team
            const Cursor cp = s_cursor[warp];
            const int64_t prefix = s_before[warp];
            const int64_t r0 = s_run[0], r1 = s_run[1], total = s_run[2], blocks = s_run[3], share = s_run[4];
            Cursor next = cp;
            next.tile = cp.span.tiles - 1;
            if (step < steps) {
                next.advance(a);
                if (!S::kQueryInSmem) load_query(next);  // on its way meanwhile
            }
            const int h0 = ((cp.h << a.teams_log) + team) * a.group + cp.block * HB, rows = min(HB, a.group - cp.block * HB);
            const int64_t seg0 = prefix * heads + (int64_t)(cp.h * a.blocks_of_group + cp.block) * cp.span.tiles;  // its first tile on the line
            const int64_t seg1 = seg0 + cp.span.tiles;
            const bool whole = r0 <= seg0 && seg1 <= r1;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(kAll, l[n][i], d);
                    if (g == 0) s_ml[warp][n * 8 + 2 * c + i] = make_float2(m[n][i], l[n][i]);
                }
            team_sync();
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = m[n][i];
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (j < mates) top = fmaxf(top, s_ml[team + (j << a.teams_log)][n * 8 + 2 * c + i].x);
                    const float f = m[n][i] == -INFINITY ? 0.0f : fast_exp2(m[n][i] - top);
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int j = i; j < 4; j += 2) {
                            o[k][n][j] *= f;
                            if (FP8) o[k][n][j] *= v_ref;  // (apart: their product may be too small a number)
                        }
                }
            if (tt < HB) {
                float2 x[W];
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    x[j] = j < mates ? s_ml[team + (j << a.teams_log)][tt] : make_float2(-INFINITY, 0.0f);
                    top = fmaxf(top, x[j].x);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) sum += x[j].x == -INFINITY ? x[j].y : x[j].y * fast_exp2(x[j].x - top);  // (0, or NaN of NaN scores alone)
                s_all[team][tt] = make_float2(top, sum);
            }
            const int64_t all_parts = (int64_t)S::kPart << a.teams_log;  // of a block's run: one for every team
            float *const part = a.parts + (2 * blockIdx.x + (share < seg0 ? 1 : 0)) * all_parts + team * S::kPart;
            uint8_t *const out = a.out + ((int64_t)cp.b * a.QH + h0) * D * 2;
            constexpr int JC = S::kJoinCols, JR = S::kJoinRow;
#pragma unroll
            for (int pass = 0; pass < DP / JC; ++pass) {
                if (pass * JC < D) {
                    float *const mine = s_join + warp * HB * JR;
#pragma unroll
                    for (int k = 0; k < JC / 16; ++k)
#pragma unroll
                        for (int n = 0; n < NH; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mine[(n * 8 + 2 * c + (i & 1)) * JR + k * 16 + (FP8 ? 2 * g + (i >> 1) : g + 8 * (i >> 1))] = o[pass * (JC / 16) + k][n][i];
                    team_sync();
                    for (int e = tt; e < rows * (JC / 2); e += mates * 32) {
                        const int r = e / (JC / 2), col = e % (JC / 2) * 2;
                        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            if (j < mates) {
                                const float2 x = *reinterpret_cast<const float2 *>(s_join + ((team + (j << a.teams_log)) * HB + r) * JR + col);
                                v.x += x.x;
                                v.y += x.y;
                            }
                        if (pass * JC + col < D) {
                            if (whole) {
                                const float sum = s_all[team][r].y, inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : sum;
                                *reinterpret_cast<uint32_t *>(out + ((int64_t)r * D + pass * JC + col) * 2) = pack2_bf16(v.x * inv, v.y * inv);
                            } else {
                                *reinterpret_cast<float2 *>(part + r * DP + pass * JC + col) = v;
                            }
                        }
                    }
                    team_sync();
                }
            }
            if (tt < rows) {
                const float top = s_all[team][tt].x, sum = s_all[team][tt].y;
                if (whole) {
                    if (a.lse) a.lse[(int64_t)cp.b * a.QH + h0 + tt] = (top + log2f(sum)) * kLn2;
                } else {
                    part[HB * DP + tt] = top;
                    part[HB * DP + HB + tt] = sum;
                }
            }
            if (!whole) {
                // ---- the parts of the blocks that share the segment, joined by the last of their teams
                const int first = (int)(((seg0 + 1) * blocks - 1) / total), last = (int)((seg1 * blocks - 1) / total);
                uint32_t *const counter = a.counters + first * kMaxTeams + team;  // a block's run has the beginning of one such segment at most
                team_sync();
                if (tt == 0) {  // releases what the team wrote before the barrier, and acquires what the others did
                    const uint32_t seen = add_acq_rel(counter, 1u);
                    s_last[team] = seen == (uint32_t)(last - first);
                    if (s_last[team]) *counter = 0;  // as the next call finds it
                }
                team_sync();
                if (s_last[team]) {
                    const int n = last - first + 1;
                    // the segment is a block's first, or begins inside its run (of the first block only)
                    const float *const part0 = a.parts + (2 * first + (total * first / blocks < seg0 ? 1 : 0)) * all_parts + team * S::kPart;
                    const float *const part1 = a.parts + 2 * (int64_t)(first + 1) * all_parts + team * S::kPart;
                    float *const lse = a.lse ? a.lse + (int64_t)cp.b * a.QH + h0 : nullptr;
                    if (HB <= 2 * mates) combine_parts<DP, HB, 1, DP == 256 ? 8 : 16>(part0, part1, 2 * all_parts, n, rows, sub, mates, D, out, lse);
                    else combine_parts<DP, HB, 4, DP == 256 ? 2 : 4>(part0, part1, 2 * all_parts, n, rows, sub, mates, D, out, lse);
                    team_sync();
                }
            }
            __syncwarp();
            if (lane == 0) {
                s_cursor[warp] = next;
                if (next.b != cp.b) s_before[warp] = prefix + cp.span.tiles;
            }
            __syncwarp();
            left = next.span.tiles;
        }
    }
}

inline int padded_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// The workspace: a counter for every block and team, zero between calls and in the same place whatever
// the sizes are, two parts for every block and team, and what every warp puts aside.
constexpr size_t kCounterBytes = (kMaxBlocks * kMaxTeams * 4 + kAlign - 1) / kAlign * kAlign;

// The most teams that may be: a power of two of them divides the kv heads.
inline int most_teams(int KH) {
    int n = kMaxTeams;
    while (KH % n) n /= 2;
    return n;
}

// The parts' bytes, a multiple of 16.
inline size_t parts_bytes(int group, int KH, int DP) { return (size_t)2 * kMaxBlocks * most_teams(KH) * (group <= 8 ? 8 : kMaxHeads) * (DP + 2) * 4; }

template <int DP, bool FP8, int NH>
epd_status_t launch_heads(AttnArgs &a, cudaStream_t st) {
    using S = Shape<DP, FP8, NH>;
    a.blocks_of_group = (a.group + S::kHeads - 1) / S::kHeads;
    if ((int64_t)a.kv.num_kv_heads * a.blocks_of_group > INT32_MAX) return EPD_ERR_UNSUPPORTED;
    // As many kv heads at once as leave a segment for every fourth multiprocessor. Fewer segments are joined
    // from more parts by fewer warps: one sequence of 32000 bf16 tokens, 32 heads over 8, takes 29 us with
    // teams of one head at a time and 31, 44 and 61 with two, four and eight; eight sequences of 30000
    // in e4m3 99, 95, 93 and 96.
    a.teams = most_teams(a.kv.num_kv_heads);
    if (a.teams > S::kWarps) a.teams = S::kWarps;
    while (a.teams > 1 && (int64_t)a.kv.num_seqs * (a.kv.num_kv_heads / a.teams) * a.blocks_of_group < sm_count() / 4) a.teams /= 2;
    a.teams_log = 0;
    while ((1 << a.teams_log) < a.teams) ++a.teams_log;
    a.tile_log = 4;
    while ((1 << a.tile_log) < S::kChunk * (S::kWarps / a.teams)) ++a.tile_log;
    a.head_groups = a.kv.num_kv_heads / a.teams;
    if (const epd_status_t rc = allow_smem<attention_kernel<DP, FP8, NH>>(S::kSmem)) return rc;
    const int grid = sm_count() < kMaxBlocks ? sm_count() : kMaxBlocks;
    return launch_pdl(attention_kernel<DP, FP8, NH>, grid, S::kThreads, S::kSmem, st, a);
}

// Groups of up to 8 heads take half the registers and matrix instructions; larger ones go 16 heads at a
// time, so that a group of 16 reads the cache once.
template <int DP, bool FP8>
epd_status_t launch_attention(AttnArgs &a, cudaStream_t st) {
    return a.group <= 8 ? launch_heads<DP, FP8, 1>(a, st) : launch_heads<DP, FP8, 2>(a, st);
}

}  // namespace
}  // namespace epd

extern "C" size_t epd_attention_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim) {
    using namespace epd;
    if (num_seqs < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads || head_dim < 8 ||
        head_dim % 8 || head_dim > kMaxHeadDim)
        return 0;
    const int group = num_heads / num_kv_heads;
    return kCounterBytes + parts_bytes(group, num_kv_heads, padded_dim(head_dim)) +
           (size_t)kMaxBlocks * 8 * aside_floats(padded_dim(head_dim), group <= 8 ? 1 : 2) * 4;
}

extern "C" epd_status_t ep_decode_attention(const epd_cache_t *cache, const void *q, int64_t q_token_stride,
                                            int num_heads, const int32_t *lengths, float softmax_scale, int window,
                                            void *workspace, void *out, float *lse, int32_t *status,
                                            epd_stream_t stream) {
    using namespace epd;
    if (const epd_status_t rc = check_cache(cache)) return rc;
    const int B = cache->num_seqs, KH = cache->num_kv_heads, D = cache->head_dim;
    if (num_heads < 1 || num_heads % KH != 0 || window < 0 || q_token_stride < 0 || q_token_stride % 8 != 0 ||
        softmax_scale != softmax_scale)
        return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status)) return EPD_ERR_INVALID_ARG;
    if (B == 0) return EPD_OK;
    if (!q || !out || !lengths || !workspace || !aligned16(q) || !aligned16(out) || !aligned4(lengths) ||
        !aligned4(lse) || !aligned16(workspace))
        return EPD_ERR_INVALID_ARG;
    AttnArgs a;
    a.q = static_cast<const uint8_t *>(q);
    a.q_stride = 2 * q_token_stride;
    a.QH = num_heads;
    a.group = num_heads / KH;
    a.kv = *cache;
    a.page = divisor(cache->page_size);
    a.lengths = lengths;
    a.window = window;
    a.scale_log2 = softmax_scale * kLog2e;
    a.aligned = cache->page_size % 16 == 0 && window == 0;
    a.out = static_cast<uint8_t *>(out);
    a.lse = lse;
    a.counters = static_cast<uint32_t *>(workspace);
    const int DP = padded_dim(D);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    a.aside = a.parts + parts_bytes(a.group, KH, DP) / 4;
    a.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cache->dtype == EPD_FP8_E4M3)
        return DP == 64    ? launch_attention<64, true>(a, st)
               : DP == 128 ? launch_attention<128, true>(a, st)
                           : launch_attention<256, true>(a, st);
    return DP == 64    ? launch_attention<64, false>(a, st)
           : DP == 128 ? launch_attention<128, false>(a, st)
                       : launch_attention<256, false>(a, st);
}
