// attention.cu -- attention of one new token over the paged key-value cache (ep_decode_attention).
//
//   o[b, h] = sum_t softmax_t(scale q[b, h] . k[t, h / G]) v[t, h / G],   G = heads / kv heads
//
// Bound by HBM: every live key and value is read once, for G heads at a time, and G <= 16 heads are
// 16 operations a byte at most. One pass with running maxima and sums.
//
// Split: the (sequence, kv head, block of 16 heads) segments of the batch, each as many tiles of
// 16 tokens a warp as its length needs, form one line of tiles, and every block takes an equal run of
// it, whatever the lengths are (they are read on the device). A segment that lies in one block's run
// is finished there; the parts of one that several blocks share go to the workspace, and the block
// that comes last joins them in the blocks' order.
//
// A warp has its own tokens of each tile, its own ring of stages in shared memory, filled by its own
// asynchronous copies some tiles ahead (past the ends of segments; page numbers are looked up one
// tile before), and its own statistics, and does not wait for the other warps before the segment's
// end. Scores and outputs are products on the warp-level matrix instructions with the tokens (of
// scores) and the columns (of outputs) as their 16 rows and 8 heads as their columns, so that a group
// of 8 heads fills them; with so few heads the 128-row tiles of tcgen05 would be nearly empty, and
// these take a fraction of the time that the bytes take.
//
// Precision: products of bf16 are exact, sums in 32 bits. The weights of a bf16 cache's values are split
// into two bf16 (15 bits at least), so that the output's own rounding is the only one that matters. An
// e4m3 cache is widened to fp16, which holds it exactly; the query is scaled by a power of two and
// the weights, with the values' scales in them, by the largest scale so far, to fp16's range (11
// bits: an eighth of the output's rounding).
#include <cuda_fp16.h>

#include "cache.cuh"

namespace epd {
namespace {

constexpr int kMaxBlocks = 160;  // blocks that the workspace has room for
constexpr int kMaxHeads = 16;    // heads of a segment, at most
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;
// A maximum is moved (and everything summed so far scaled down) only when a score passes it by more
// than 2^8: terms up to 2^8 lose nothing in 32 bits, and the scaling is rare.
constexpr float kSlack = 8.0f;

struct AttnArgs {
    const uint8_t *q;
    int64_t q_stride;  // bytes between tokens
    int QH, group, blocks_of_group;  // segments of a group
    epd_cache_t kv;
    Divisor page;
    const int32_t *lengths;
    int window;
    float scale_log2;
    int aligned;  // every run of 16 positions from a multiple of 16 lies on one page, and tiles begin at such
    uint8_t *out;  // bf16 [B, QH, D]
    float *lse;
    uint32_t *counters;
    float *parts;
    int32_t *status;
};

template <int DP, bool FP8, int NH>
struct Shape {
    static constexpr int kHeads = 8 * NH;                   // of a segment
    static constexpr int kRow = DP * (FP8 ? 1 : 2);         // bytes of a row in shared memory
    static constexpr int kUnits = kRow / 16;
    static constexpr int kChunk = kRow <= 128 ? 32 : 16;    // tokens of a warp's tile
    static constexpr int kTail = (FP8 ? 2 * kChunk * 4 : 0) + 16;  // scales and the live tokens' mask
    static constexpr int kStage = 2 * kChunk * kRow + kTail;
    static constexpr int kWarps = kRow == 512 ? 4 : 8;
    static constexpr int kJoinCols = DP < 128 ? DP : 128, kJoinRow = kJoinCols + 4;
    static constexpr int kJoinSums = kWarps * kHeads * kJoinRow * 4, kJoinWeights = 3 * kMaxBlocks * kHeads * 4;
    static constexpr int kJoin = kJoinSums > kJoinWeights ? kJoinSums : kJoinWeights;
    // One stage on the way (64 KB a multiprocessor) while another is read. More in flight fill the same
    // memory system, but share it less evenly: of 152 blocks with equal runs the fastest then takes
    // 256 us and the slowest 348 (128 sequences, 2.1 GB; 361 us in all), with two stages 303 and 337 (344).
    static constexpr int kStages = 2;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTile = kWarps * kChunk;  // tokens of a tile
    static constexpr int kSmem = kWarps * kStages * kStage + kJoin;
    static constexpr int kPart = kHeads * (DP + 2);  // floats: the heads' sums, maxima and sums of weights
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
template <int TILE>
__device__ __forceinline__ Span span_of(const AttnArgs &a, int len) {
    const int64_t most = cache_positions(a.kv);
    Span s;
    s.n = len < 0 ? 0 : (int64_t)len > most ? (int)most : len;
    s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
    s.tiles = s.n > 0 ? (s.n - s.lo - 1) / TILE + 1 : 1;
    return s;
}

// A place on the line of tiles: tile `tile` of segment (b, h, block).
template <int TILE>
struct Cursor {
    int b, h, block, tile, next_len;
    Span span;
    __device__ __forceinline__ void enter(const AttnArgs &a, int len) {
        span = span_of<TILE>(a, len);
        next_len = b + 1 < a.kv.num_seqs ? __ldg(a.lengths + b + 1) : 0;
    }
    __device__ __forceinline__ void advance(const AttnArgs &a) {
        if (++tile < span.tiles) return;
        tile = 0;
        if (++block < a.blocks_of_group) return;
        block = 0;
        if (++h < a.kv.num_kv_heads) return;
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

template <int DP, bool FP8, int NH>
__global__ void __launch_bounds__(Shape<DP, FP8, NH>::kThreads, 1) attention_kernel(AttnArgs a) {
    using S = Shape<DP, FP8, NH>;
    constexpr int W = S::kWarps, UNITS = S::kUnits, TILE = S::kTile, CH = S::kChunk, MT = CH / 16, KT = DP / 16;
    constexpr int HB = S::kHeads;
    extern __shared__ uint4 s_dyn[];
    __shared__ int64_t s_scan[W];
    __shared__ int64_t s_prefix;
    __shared__ int s_seq;
    __shared__ float s_m[W][HB], s_l[W][HB], s_mall[HB], s_lall[HB];
    __shared__ uint32_t s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int D = a.kv.head_dim, B = a.kv.num_seqs, heads = a.kv.num_kv_heads * a.blocks_of_group;
    const uint32_t ring = smem_addr(s_dyn) + warp * S::kStages * S::kStage;
    float *const s_join = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(s_dyn) + W * S::kStages * S::kStage);
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
        for (int b = tid; b < B; b += S::kThreads) v += span_of<TILE>(a, __ldg(a.lengths + b)).tiles;
        v = warp_scan(v, lane);
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        for (int w = 0; w < W; ++w) total += s_scan[w];
        __syncthreads();
    }
    int64_t r0 = 0, r1 = 0, before = 0, blocks = gridDim.x;  // blocks: that have a tile
    for (int b0 = 0; b0 < B; b0 += S::kThreads) {
        const int b = b0 + tid;
        const int64_t v = b < B ? span_of<TILE>(a, __ldg(a.lengths + b)).tiles : 0;
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
            r0 = total * blockIdx.x / blocks;
            r1 = total * (blockIdx.x + 1) / blocks;
            if (blockIdx.x >= blocks) return;
        }
        incl += before;
        if ((incl - v) * heads <= r0 && r0 < incl * heads) {
            s_seq = b;
            s_prefix = incl - v;
        }
        before += sum;
        __syncthreads();
        if (before * heads > r0) break;
    }
    const int steps = (int)(r1 - r0);
    Cursor<TILE> ld, cp;
    ld.b = s_seq;
    int64_t prefix = s_prefix;  // tiles of the sequences before the compute cursor's
    ld.enter(a, __ldg(a.lengths + ld.b));
    {
        const int64_t rest = r0 - prefix * heads;
        const int hh = (int)(rest / ld.span.tiles);
        ld.tile = (int)(rest - (int64_t)hh * ld.span.tiles);
        ld.h = hh / a.blocks_of_group;
        ld.block = hh - ld.h * a.blocks_of_group;
    }
    cp = ld;
    if (blockIdx.x == 0) {  // lengths that the pages do not hold
        for (int b = tid; b < B; b += S::kThreads) {
            const int len = __ldg(a.lengths + b);
            if (len < 0) report(a.status, EPD_ERR_INVALID_ARG);
            else if ((int64_t)len > cache_positions(a.kv)) report(a.status, EPD_ERR_CAPACITY);
        }
    }

    // ---- loads: lane l looks after token l % CH of the warp's chunk
    int token, page, kv_head;
    auto look_up = [&]() {
        // (a tile may end past 2^31 - 1, where the sequence ends before)
        const uint32_t t = (uint32_t)ld.span.lo + (uint32_t)ld.tile * TILE + warp * CH + (lane & (CH - 1));
        token = t < (uint32_t)ld.span.n ? (int)t : -1;
        kv_head = ld.h;
        page = token >= 0 ? __ldg(a.kv.page_table + ld.b * a.kv.table_stride + divide(t, a.page)) : -1;
    };
    const int units = D * (FP8 ? 1 : 2) / 16;
    auto load = [&](int stage) {
        const uint32_t at = ring + stage * S::kStage;
        bool live = token >= 0;
        if (live && (page < 0 || page >= a.kv.num_pages)) {
            report(a.status, EPD_ERR_CAPACITY);
            live = false;
        }
        const int inside = live ? token - (int)(divide(token, a.page) * a.page.d) : 0;
        const int64_t off = live ? (page * a.kv.page_stride + inside * a.kv.token_stride + kv_head * a.kv.head_stride) * (FP8 ? 1 : 2) : 0;
        const uint32_t mask = __ballot_sync(kAll, live) & (CH == 32 ? kAll : 0xffffu);
        if (a.aligned && mask == (CH == 32 ? kAll : 0xffffu)) {
            // every 16 tokens lie on one page: one address for them, and a constant step
            constexpr int STEP = 32 / UNITS > 0 ? 32 / UNITS : 1;  // rows of one instruction
            const int64_t step = a.kv.token_stride * (FP8 ? 1 : 2);
            const int u = lane % UNITS;
            const uint8_t *const k0 = static_cast<const uint8_t *>(a.kv.k) + (lane / UNITS) * step + u * 16;
            const int64_t to_v = (int64_t)(reinterpret_cast<uintptr_t>(a.kv.v) - reinterpret_cast<uintptr_t>(a.kv.k));
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
            const int64_t so = live ? page * a.kv.scale_page_stride + inside * a.kv.scale_token_stride + kv_head * a.kv.scale_head_stride : 0;
            const uint32_t dst = at + 2 * CH * S::kRow + (lane & (CH - 1)) * 4;
            if (CH == 32 || lane < 16) copy4z(dst, a.kv.k_scale + so, live);
            if (CH == 32 || lane >= 16) copy4z(dst + CH * 4, a.kv.v_scale + so, live);
        }
        if (lane == 0)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + S::kStage - 16), "r"(mask) : "memory");
    };
    __syncwarp();
    look_up();
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) {
        if (s < steps) {
            load(s);
            if (s + 1 < steps) {
                ld.advance(a);
                look_up();
            }
        }
        copy_commit();
    }

    // ---- the line. o[k][n][i]: column 16 k + g + 8 (i / 2) (e4m3: 16 k + 2 g + i / 2) of head
    // 8 n + 2 c + i % 2; m and l: of heads 8 n + 2 c, 8 n + 2 c + 1, l of the lane's own tokens
    uint32_t q[KT][NH][2];
    float o[KT][NH][4], m[NH][2], l[NH][2], q_scale = 1.0f, v_ref = 0.0f, v_inv = 0.0f;
    const float *const scales = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(s_dyn) + warp * S::kStages * S::kStage + 2 * CH * S::kRow);
    bool fresh = true;
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
        if (fresh) {
            fresh = false;
            const int rows = a.group - cp.block * HB;  // heads of the segment, if fewer than HB
            const uint8_t *src = a.q + cp.b * a.q_stride + (int64_t)(cp.h * a.group + cp.block * HB) * D * 2;
            // Fragments of the query: head g, and the columns that the keys' fragments pair with
            // them -- of a 16-byte unit of an e4m3 row a lane holds four neighbours.
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = n * 8 + g, col = k * 16 + (FP8 ? 4 * c + i * 2 : 2 * c + i * 8);
                        q[k][n][i] = row < rows && col < D ? __ldg(reinterpret_cast<const uint32_t *>(src + ((int64_t)row * D + col) * 2)) : 0;
                    }
            if (FP8) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int i = 0; i < 2 * NH; ++i) top = fmaxf(top, fmaxf(fabsf(lo_bf16(q[k][i >> 1][i & 1])), fabsf(hi_bf16(q[k][i >> 1][i & 1]))));
#pragma unroll
                for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
                // to [2^6, 2^7): the power of two from the exponent's bits
                const int e = top > 0.0f ? min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 100) : 0;
                const float up = __uint_as_float((uint32_t)(127 + 6 - e) << 23);
                q_scale = __uint_as_float((uint32_t)(127 - 6 + e) << 23);
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) q[k][n][i] = pack2_f16(lo_bf16(q[k][n][i]) * up, hi_bf16(q[k][n][i]) * up);
            }
#pragma unroll
            for (int n = 0; n < NH; ++n) {
#pragma unroll
                for (int k = 0; k < KT; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.0f;
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
            }
            v_ref = v_inv = 0.0f;
        }
        copy_wait<S::kStages - 2>();
        __syncwarp();
        if (step + S::kStages - 1 < steps) {
            load(stage == 0 ? S::kStages - 1 : stage - 1);
            if (step + S::kStages < steps) {
                ld.advance(a);
                look_up();
            }
        }
        copy_commit();

        const uint32_t at = ring + stage * S::kStage;
        uint32_t mask;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(mask) : "r"(at + S::kStage - 16) : "memory");
        if (mask) {
            // s[t][n][i]: token 16 t + g + 8 (i / 2), head 8 n + 2 c + i % 2
            float s[MT][NH][4] = {};
            const int row = lane & 15, right = lane >> 4;
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
                            for (int n = 0; n < NH; ++n) mma<true>(s[t][n], f, q[2 * k + h][n][0], q[2 * k + h][n][1]);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NH; ++n) mma<false>(s[t][n], r, q[k][n][0], q[k][n][1]);
                    }
                }
            const float *const sc = scales + stage * (S::kStage / 4);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                float f[2] = {a.scale_log2, a.scale_log2};
                if (FP8) {
                    f[0] = f[0] * q_scale * sc[16 * t + g];
                    f[1] = f[1] * q_scale * sc[16 * t + g + 8];
                }
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][n][i] *= f[i >> 1];
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
                    more |= top[n][i] > m[n][i] + kSlack;
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
                // the values' scales over the largest so far (up to 16 times it without moving it)
                bool larger = false;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        vs[t][i] = sc[CH + 16 * t + g + 8 * i];
                        larger |= vs[t][i] > 16.0f * v_ref;
                    }
                if (__any_sync(kAll, larger)) {
                    float most = 0.0f;
#pragma unroll
                    for (int t = 0; t < MT; ++t) most = fmaxf(most, fmaxf(vs[t][0], vs[t][1]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, d));
                    const float f = v_ref / most;
                    v_ref = most;
                    v_inv = 1.0f / most;
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int i = 0; i < 4 * NH; ++i) o[k][i >> 2][i & 3] *= f;
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) vs[t][i] *= v_inv;
            }
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
                        l[n][0] += x;
                        l[n][1] += y;
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
        }
        if (++stage == S::kStages) stage = 0;

        if (cp.tile == cp.span.tiles - 1 || step == steps - 1) {
            // ---- the segment's end here: join the warps
            const int h0 = cp.h * a.group + cp.block * HB, rows = min(HB, a.group - cp.block * HB);
            const int64_t seg0 = prefix * heads + (int64_t)(cp.h * a.blocks_of_group + cp.block) * cp.span.tiles;  // its first tile on the line
            const int64_t seg1 = seg0 + cp.span.tiles;
            const bool whole = r0 <= seg0 && seg1 <= r1;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(kAll, l[n][i], d);
                    if (g == 0) {
                        s_m[warp][n * 8 + 2 * c + i] = m[n][i];
                        s_l[warp][n * 8 + 2 * c + i] = l[n][i];
                    }
                }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][n * 8 + 2 * c + i]);
                    float f = m[n][i] == -INFINITY ? 0.0f : fast_exp2(m[n][i] - top);
                    if (FP8) f *= v_ref;
#pragma unroll
                    for (int k = 0; k < KT; ++k) {
                        o[k][n][i] *= f;
                        o[k][n][i + 2] *= f;
                    }
                }
            if (tid < HB) {
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][tid]);
#pragma unroll
                for (int w = 0; w < W; ++w) sum += s_m[w][tid] == -INFINITY ? 0.0f : s_l[w][tid] * fast_exp2(s_m[w][tid] - top);
                s_mall[tid] = top;
                s_lall[tid] = sum;
            }
            float *const part = a.parts + (2 * blockIdx.x + (r0 < seg0 ? 1 : 0)) * (int64_t)S::kPart;
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
                    __syncthreads();
                    for (int e = tid; e < rows * (JC / 2); e += S::kThreads) {
                        const int r = e / (JC / 2), col = e % (JC / 2) * 2;
                        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const float2 x = *reinterpret_cast<const float2 *>(s_join + (w * HB + r) * JR + col);
                            v.x += x.x;
                            v.y += x.y;
                        }
                        if (pass * JC + col < D) {
                            if (whole) {
                                const float inv = s_lall[r] > 0.0f ? __fdiv_rn(1.0f, s_lall[r]) : s_lall[r];
                                *reinterpret_cast<uint32_t *>(out + ((int64_t)r * D + pass * JC + col) * 2) = pack2_bf16(v.x * inv, v.y * inv);
                            } else {
                                *reinterpret_cast<float2 *>(part + r * DP + pass * JC + col) = v;
                            }
                        }
                    }
                    __syncthreads();
                }
            }
            if (tid < rows) {
                if (whole) {
                    if (a.lse) a.lse[(int64_t)cp.b * a.QH + h0 + tid] = s_mall[tid] == -INFINITY ? -INFINITY : (s_mall[tid] + log2f(s_lall[tid])) * kLn2;
                } else {
                    part[HB * DP + tid] = s_mall[tid];
                    part[HB * DP + HB + tid] = s_lall[tid];
                }
            }
            if (!whole) {
                // ---- the parts of the blocks that share the segment, joined by the last of them
                const int first = (int)(((seg0 + 1) * blocks - 1) / total), last = (int)((seg1 * blocks - 1) / total);
                uint32_t *const counter = a.counters + first;  // a block's run has the beginning of one such segment at most
                __syncthreads();
                if (tid == 0) {  // releases what the block wrote before the barrier, and acquires what the others did
                    const uint32_t seen = add_acq_rel(counter, 1u);
                    s_last = seen == (uint32_t)(last - first);
                    if (s_last) *counter = 0;  // as the next call finds it
                }
                __syncthreads();
                if (s_last) {
                    const int n = last - first + 1;
                    auto part_of = [&](int i) {  // the segment is a block's first, or begins inside its run
                        const int blk = first + i;
                        return a.parts + (2 * blk + (total * blk / blocks < seg0 ? 1 : 0)) * (int64_t)S::kPart;
                    };
                    // only the first block's part can be its second
                    const float *const part0 = part_of(0), *const part1 = a.parts + 2 * (int64_t)(first + 1) * S::kPart;
                    auto at_part = [&](int i) { return i == 0 ? part0 : part1 + 2 * (int64_t)(i - 1) * S::kPart; };
                    // the parts' sums, four columns at a time, sixteen of a thread's on the way
                    constexpr int ITEMS = (HB * DP / 4 + S::kThreads - 1) / S::kThreads, BATCH = 16 / ITEMS;
                    float4 x[BATCH][ITEMS], v[ITEMS];
                    auto fetch = [&](int i0) {
#pragma unroll
                        for (int i = 0; i < BATCH; ++i)
#pragma unroll
                            for (int j = 0; j < ITEMS; ++j) {
                                const int e = tid + j * S::kThreads;
                                x[i][j] = i0 + i < n && e < HB * DP / 4 ? __ldcg(reinterpret_cast<const float4 *>(at_part(i0 + i)) + e) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            }
                    };
                    fetch(0);
                    // meanwhile a weight for every part and head, and the heads' sums
                    float *const s_max = s_join, *const s_sum = s_join + kMaxBlocks * HB, *const s_by = s_sum + kMaxBlocks * HB;
                    for (int e = tid; e < n * HB; e += S::kThreads) {
                        const float *src = at_part(e / HB) + HB * DP + e % HB;
                        s_max[e] = __ldcg(src);
                        s_sum[e] = __ldcg(src + HB);
                    }
                    __syncthreads();
                    const int head = tid % HB;
                    float top = -INFINITY;
#pragma unroll 8
                    for (int i = 0; i < n; ++i) top = fmaxf(top, s_max[i * HB + head]);
                    for (int e = tid; e < n * HB; e += S::kThreads) {  // (kThreads is a multiple of HB: the thread's own head)
                        const float f = s_max[e] == -INFINITY ? 0.0f : fast_exp2(s_max[e] - top);
                        s_by[e] = f;
                        s_sum[e] *= f;
                    }
                    __syncthreads();
                    if (tid < rows) {
                        float sum = 0.0f;
#pragma unroll 8
                        for (int i = 0; i < n; ++i) sum += s_sum[i * HB + tid];
                        s_lall[tid] = sum > 0.0f ? __fdiv_rn(1.0f, sum) : sum;
                        if (a.lse) a.lse[(int64_t)cp.b * a.QH + h0 + tid] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
                    }
#pragma unroll
                    for (int j = 0; j < ITEMS; ++j) v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int i0 = 0; i0 < n; i0 += BATCH) {
                        if (i0 > 0) fetch(i0);
#pragma unroll
                        for (int i = 0; i < BATCH; ++i)
#pragma unroll
                            for (int j = 0; j < ITEMS; ++j) {
                                const int r = (tid + j * S::kThreads) / (DP / 4);
                                const float f = i0 + i < n && r < HB ? s_by[(i0 + i) * HB + r] : 0.0f;
                                v[j].x = fmaf(x[i][j].x, f, v[j].x), v[j].y = fmaf(x[i][j].y, f, v[j].y);
                                v[j].z = fmaf(x[i][j].z, f, v[j].z), v[j].w = fmaf(x[i][j].w, f, v[j].w);
                            }
                    }
                    __syncthreads();
#pragma unroll
                    for (int j = 0; j < ITEMS; ++j) {
                        const int e = tid + j * S::kThreads, r = e / (DP / 4), col = e % (DP / 4) * 4;
                        if (r < rows && col < D)
                            *reinterpret_cast<uint2 *>(out + ((int64_t)r * D + col) * 2) =
                                make_uint2(pack2_bf16(v[j].x * s_lall[r], v[j].y * s_lall[r]), pack2_bf16(v[j].z * s_lall[r], v[j].w * s_lall[r]));
                    }
                    __syncthreads();
                }
            }
            fresh = true;
        }
        if (step + 1 < steps) {
            const int b = cp.b, tiles = cp.span.tiles;
            cp.advance(a);
            if (cp.b != b) prefix += tiles;
        }
    }
}

inline int padded_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// The workspace: a counter for every block, zero between calls and in the same place whatever the
// sizes are, and two parts for every block.
constexpr size_t kCounterBytes = (kMaxBlocks * 4 + kAlign - 1) / kAlign * kAlign;

template <int DP, bool FP8, int NH>
epd_status_t launch_heads(AttnArgs &a, cudaStream_t st) {
    using S = Shape<DP, FP8, NH>;
    a.blocks_of_group = (a.group + S::kHeads - 1) / S::kHeads;
    if ((int64_t)a.kv.num_kv_heads * a.blocks_of_group > INT32_MAX) return EPD_ERR_UNSUPPORTED;
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
    return kCounterBytes + (size_t)2 * kMaxBlocks * kMaxHeads * (padded_dim(head_dim) + 2) * 4;
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
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    a.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int DP = padded_dim(D);
    if (cache->dtype == EPD_FP8_E4M3)
        return DP == 64    ? launch_attention<64, true>(a, st)
               : DP == 128 ? launch_attention<128, true>(a, st)
                           : launch_attention<256, true>(a, st);
    return DP == 64    ? launch_attention<64, false>(a, st)
           : DP == 128 ? launch_attention<128, false>(a, st)
                       : launch_attention<256, false>(a, st);
}
