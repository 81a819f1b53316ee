// rotary.cu -- rotary positions (ep_rotary) and appending to the paged cache with the rotation on
// the way (ep_cache_append).
//
// A pair (a, b) of a head becomes A (a cos - b sin), A (a sin + b cos) with the angle position *
// frequency. The caller gives each pair's frequency as the fraction of a turn that one position adds,
// in units of 2^-64: position * step, in 64-bit integers, is then the whole angle modulo one turn,
// without the cancellation that a product in 32 bits (or a range reduction) has at far positions, and
// without 64-bit floating point, of which this GPU has little.
//
// Bound by HBM: every value is read and written once (16384 tokens of 64 heads of 128: 79.7 us, 80.4 at
// a copy's rate). A head is cut into chunks of V pairs, one a lane, in groups of a power of two of lanes
// a head; a warp takes its token's heads several at a time, with the loads of a few such passes in
// flight, and the lane's sines and cosines serve all of them. What is not rotated is carried over as it is. In an e4m3 cache every token and head has
// its own scale, amax / 448, from the head's lanes by shuffles.
#include <cuda_fp8.h>

#include <type_traits>

#include "cache.cuh"

namespace epd {
namespace {

constexpr int kThreads = 128;
template <int V>
constexpr int kBatch = V == 8 ? 4 : 8;  // passes of ep_rotary whose loads are in flight at once: 128 bytes a lane
constexpr unsigned kAll = 0xffffffffu;

struct Turn {
    const uint64_t *step;  // [R / 2], null for no rotation
    int R, inverse;
    float scale;
};

// How a warp walks over a token's heads.
struct Walk {
    int chunks;     // chunks of a head: the first R / 2V are rotated
    int lanes_log;  // log2 of the lanes of a head
    int heads, passes, parts;  // passes: of a warp; parts: warps of a token
};

// The token and the part of it that a warp has: number `unit` of all parts.
struct Unit {
    int t, part;
    __device__ __forceinline__ Unit(const Divisor &parts) {
        const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        t = (int)divide(unit, parts);
        part = (int)(unit - (uint32_t)t * parts.d);
    }
};

struct RotaryArgs {
    const uint8_t *x;
    uint8_t *out;
    int64_t x_token, x_head, out_token, out_head;  // bytes
    const int32_t *positions;
    int T, D;
    Divisor parts;
    Turn turn;
    Walk walk;
};

struct AppendArgs {
    const uint8_t *q, *k, *v;
    uint8_t *q_out;
    int64_t q_token, k_token, v_token, q_out_token;  // bytes
    const int32_t *positions, *token_seq;
    int T;
    Divisor parts, page;
    epd_cache_t cache;
    Turn turn;
    Walk queries, rows;  // rows: keys, then values
    int32_t *status;
};

// Where the pairs of chunk p lie in a head of D elements: V of their first halves from `a`, V of
// their second halves from `b`; interleaved pairs lie at a + 2 i and a + 2 i + 1.
template <int V, bool INTER>
struct Place {
    int a, b;
    __device__ __forceinline__ Place(int p, int R, int D) {
        if (INTER) {
            a = 2 * V * p;
            b = a + 1;
        } else if (p < R / (2 * V)) {
            a = V * p;
            b = a + R / 2;
        } else {
            a = R + V * (p - R / (2 * V));
            b = a + (D - R) / 2;
        }
    }
};

// The values are read once, and may be written over by the same thread (not the read-only path).
__device__ __forceinline__ uint4 ld16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld8(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// The raw 2 V bf16 values of a chunk: V == 8 halves as two 16-byte words, interleaved V == 4 as one,
// V == 4 halves as two 8-byte words, V == 1 as one 4-byte word.
template <int V, bool INTER>
struct Raw {
    uint32_t w[V] = {};
    __device__ __forceinline__ void load(const uint8_t *head, const Place<V, INTER> &at) {
        if constexpr (V == 8) {
            const uint4 x = ld16(head + 2 * at.a), y = ld16(head + 2 * at.b);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
        } else if constexpr (V == 4 && INTER) {
            const uint4 x = ld16(head + 2 * at.a);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if constexpr (V == 4) {
            const uint2 x = ld8(head + 2 * at.a), y = ld8(head + 2 * at.b);
            w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
        } else if constexpr (INTER) {
            w[0] = *reinterpret_cast<const volatile uint32_t *>(head + 2 * at.a);
        } else {
            const volatile uint16_t *h = reinterpret_cast<const volatile uint16_t *>(head);
            w[0] = (uint32_t)h[at.a] | (uint32_t)h[at.b] << 16;
        }
    }
    // In 32 bits, first halves and second halves.
    __device__ __forceinline__ void values(float (&a)[V], float (&b)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (INTER || V == 1) {
                a[i] = lo_bf16(w[i]);
                b[i] = hi_bf16(w[i]);
            } else {
                a[i] = i & 1 ? hi_bf16(w[i / 2]) : lo_bf16(w[i / 2]);
                b[i] = i & 1 ? hi_bf16(w[V / 2 + i / 2]) : lo_bf16(w[V / 2 + i / 2]);
            }
        }
    }
    // Takes the values if `on`, and stays what it was otherwise.
    __device__ __forceinline__ void take(const float (&a)[V], const float (&b)[V], bool on) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t x = INTER || V == 1 ? pack2_bf16(a[i], b[i]) : i < V / 2 ? pack2_bf16(a[2 * i % V], a[(2 * i + 1) % V])
                                                                                    : pack2_bf16(b[2 * i % V], b[(2 * i + 1) % V]);
            w[i] = on ? x : w[i];
        }
    }
    __device__ __forceinline__ void store(uint8_t *head, const Place<V, INTER> &at) const {
        if constexpr (V == 8) {
            st16(head + 2 * at.a, make_uint4(w[0], w[1], w[2], w[3]));
            st16(head + 2 * at.b, make_uint4(w[4], w[5], w[6], w[7]));
        } else if constexpr (V == 4 && INTER) {
            st16(head + 2 * at.a, make_uint4(w[0], w[1], w[2], w[3]));
        } else if constexpr (V == 4) {
            *reinterpret_cast<uint2 *>(head + 2 * at.a) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(head + 2 * at.b) = make_uint2(w[2], w[3]);
        } else if constexpr (INTER) {
            *reinterpret_cast<uint32_t *>(head + 2 * at.a) = w[0];
        } else {
            reinterpret_cast<uint16_t *>(head)[at.a] = (uint16_t)w[0];
            reinterpret_cast<uint16_t *>(head)[at.b] = (uint16_t)(w[0] >> 16);
        }
    }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <int V, bool INTER>
__device__ __forceinline__ void store_e4m3(uint8_t *head, const Place<V, INTER> &at, float (&a)[V], float (&b)[V], float scale) {
    divide_all(a, scale);
    divide_all(b, scale);
    if constexpr (V == 1) {
        const uint32_t w = e4m3x2(a[0], b[0]);
        head[at.a] = (uint8_t)w;
        head[at.b] = (uint8_t)(w >> 8);
    } else if constexpr (INTER) {
        *reinterpret_cast<uint2 *>(head + at.a) =
            make_uint2(e4m3x2(a[0], b[0]) | e4m3x2(a[1], b[1]) << 16, e4m3x2(a[2], b[2]) | e4m3x2(a[3], b[3]) << 16);
    } else {
        uint32_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            u[i] = e4m3x2(a[4 * i], a[4 * i + 1]) | e4m3x2(a[4 * i + 2], a[4 * i + 3]) << 16;
            u[V / 4 + i] = e4m3x2(b[4 * i], b[4 * i + 1]) | e4m3x2(b[4 * i + 2], b[4 * i + 3]) << 16;
        }
        if constexpr (V == 4) {
            *reinterpret_cast<uint32_t *>(head + at.a) = u[0];
            *reinterpret_cast<uint32_t *>(head + at.b) = u[1];
        } else {
            *reinterpret_cast<uint2 *>(head + at.a) = make_uint2(u[0], u[1]);
            *reinterpret_cast<uint2 *>(head + at.b) = make_uint2(u[2], u[3]);
        }
    }
}

// Cosines and sines of chunk p's pairs at a position, times the scale, where they are rotated.
// The hardware's sine and cosine of an angle within [-pi, pi] are off by 2^-20.5 at most, a 2000th of a
// step of the bf16 that they go into.
template <int V>
__device__ __forceinline__ bool angles(const Turn &t, int p, int position, float (&c)[V], float (&s)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = s[i] = 0.0f;
    if (p >= t.R / (2 * V)) return false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint64_t phase = (uint64_t)(int64_t)position * __ldg(t.step + p * V + i);
        const float angle = (float)(int32_t)(phase >> 32) * 1.4629180792671596e-9f;  // pi / 2^31
        c[i] = __cosf(angle) * t.scale;
        s[i] = __sinf(angle) * (t.inverse ? -t.scale : t.scale);
    }
    return true;
}

template <int V>
__device__ __forceinline__ void rotate(float (&a)[V], float (&b)[V], const float (&c)[V], const float (&s)[V]) {
    if constexpr (V == 1) {
        const float x = a[0], y = b[0];
        a[0] = x * c[0] - y * s[0];
        b[0] = x * s[0] + y * c[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {  // two pairs to an instruction
            const float2 x = make_float2(a[i], a[i + 1]), y = make_float2(b[i], b[i + 1]);
            const float2 cc = make_float2(c[i], c[i + 1]), ss = make_float2(s[i], s[i + 1]);
            const float2 u = __ffma2_rn(x, cc, __fmul2_rn(y, make_float2(-ss.x, -ss.y))), w = __ffma2_rn(x, ss, __fmul2_rn(y, cc));
            a[i] = u.x, a[i + 1] = u.y;
            b[i] = w.x, b[i + 1] = w.y;
        }
    }
}

template <int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const Unit unit(a.parts);
    const int64_t t = unit.t;
    if (t >= a.T) return;
    const int per_pass = 32 >> a.walk.lanes_log, lanes = 1 << a.walk.lanes_log;
    const int first = unit.part * a.walk.passes * per_pass + (lane >> a.walk.lanes_log);
    const int position = __ldg(a.positions + t);
    const uint8_t *x = a.x + t * a.x_token;
    uint8_t *out = a.out + t * a.out_token;
    for (int p = lane & (lanes - 1); p < a.walk.chunks; p += lanes) {
        const Place<V, INTER> at(p, a.turn.R, a.D);
        float c[V], s[V];
        const bool on = angles<V>(a.turn, p, position, c, s);
        for (int i0 = 0; i0 < a.walk.passes; i0 += kBatch<V>) {
            Raw<V, INTER> raw[kBatch<V>];
#pragma unroll
            for (int i = 0; i < kBatch<V>; ++i) {
                const int n = first + (i0 + i) * per_pass;
                if (i0 + i < a.walk.passes && n < a.walk.heads) raw[i].load(x + n * a.x_head, at);
            }
#pragma unroll
            for (int i = 0; i < kBatch<V>; ++i) {
                const int n = first + (i0 + i) * per_pass;
                if (i0 + i < a.walk.passes && n < a.walk.heads) {
                    float u[V], w[V];
                    raw[i].values(u, w);
                    rotate<V>(u, w, c, s);
                    raw[i].take(u, w, on);
                    raw[i].store(out + n * a.out_head, at);
                }
            }
        }
    }
}

// NP: chunks of a head that one lane holds (V == 1 only). Bound by HBM, and by how many warps there are to
// wait for it: 16384 tokens of 64 + 2 x 8 heads of 128 take 99.3 us into an e4m3 cache, half a head rotated
// interleaved (0.64 GB: 96), 99.9 with halves of the whole head, and 100 into a bf16 one (100). With whole
// batches of 8 passes and 90 to 130 registers a thread, five blocks or fewer a multiprocessor, they took 116, 140
// and 108. At these limits the halves' e4m3 instances spill 64 bytes a thread. An e4m3 cache of 16 + 2 x 16 heads
// takes 70.5 (halves), 77 (interleaved; 51) and 79 of 96 elements, 24 of them rotated (38): the conversion's
// instructions, 3 to 5 % of the time the remainders that make its quotients the rounded ones.
template <int V, bool INTER, bool FP8, int NP>
__global__ void __launch_bounds__(kThreads, V == 4 ? 9 : V == 8 ? 6 : 1) append_kernel(AppendArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const Unit unit(a.parts);
    const int64_t t = unit.t;
    if (t >= a.T) return;
    int part = unit.part;
    const epd_cache_t &kv = a.cache;
    const int D = kv.head_dim;
    const int position = __ldg(a.positions + t);
    const int seq = a.token_seq ? __ldg(a.token_seq + t) : (int)t;
    // The token's slot in the cache; false where it has none (padding, or out of range).
    int64_t slot = 0, scale_slot = 0;
    auto find_slot = [&]() {
        if (seq == -1) return false;
        int page = -1, inside = 0;
        if (seq >= 0 && seq < kv.num_seqs && position >= 0 && position < cache_positions(kv)) {
            const int at = (int)divide(position, a.page);
            page = __ldg(kv.page_table + seq * kv.table_stride + at);
            inside = position - at * kv.page_size;
        }
        if (page < 0 || page >= kv.num_pages) {
            if (lane == 0) report(a.status, EPD_ERR_CAPACITY);
            return false;
        }
        slot = page * kv.page_stride + inside * kv.token_stride;
        scale_slot = page * kv.scale_page_stride + inside * kv.scale_token_stride;
        return true;
    };
    const int lanes_log = a.rows.lanes_log, lanes = 1 << lanes_log, per_pass = 32 >> lanes_log;
    const int p0 = lane & (lanes - 1);
    // A warp has queries, keys or values only: from `src`, `turned` or not, to heads `step` apart at `to`
    // (held: in the cache, at the token's slot, with `scales` in an e4m3 one). Keys and values share their
    // code: a warp runs through it once or twice, and waits for instructions where there is more of it.
    auto heads = [&](const uint8_t *src, const Walk &walk, bool turned, auto is_held, uint8_t *to, int64_t step, float *scales) {
        constexpr bool held = decltype(is_held)::value, scaled = held && FP8;
        constexpr int B = NP > 1 ? 1 : scaled ? 2 : 4;
        const int first = part * walk.passes * per_pass + (lane >> lanes_log);
        float c[NP][V], s[NP][V];
        bool on[NP];
#pragma unroll 1
        for (int i0 = 0; i0 < walk.passes; i0 += B) {
            Raw<V, INTER> raw[B][NP];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int n = first + (i0 + i) * per_pass;
                if (i0 + i >= walk.passes || n >= walk.heads) continue;
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    if (p0 + q * lanes < walk.chunks)
                        raw[i][q].load(src + (int64_t)n * D * 2, Place<V, INTER>(p0 + q * lanes, a.turn.R, D));
            }
            if (i0 == 0) {  // with the first values on the way: the slot takes two dependent loads
#pragma unroll
                for (int q = 0; q < NP; ++q) on[q] = angles<V>(a.turn, turned ? p0 + q * lanes : INT32_MAX, position, c[q], s[q]);
                if (!find_slot()) return;
            }
            if constexpr (scaled) {
                // a batch's scales are found together: each is a chain of exchanges
                float u[B][NP][V], w[B][NP][V], scale[B];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    scale[i] = 0.0f;
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        raw[i][q].values(u[i][q], w[i][q]);
                        if (on[q]) rotate<V>(u[i][q], w[i][q], c[q], s[q]);
                        float top = 0.0f;
#pragma unroll
                        for (int j = 0; j < V; ++j) top = fmaxf(top, fmaxf(fabsf(u[i][q][j]), fabsf(w[i][q][j])));
                        if (p0 + q * lanes < walk.chunks) scale[i] = fmaxf(scale[i], top);
                    }
                }
#pragma unroll
                for (int d = 16; d; d >>= 1)
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const float other = __shfl_xor_sync(kAll, scale[i], d);
                        if (d < lanes) scale[i] = fmaxf(scale[i], other);
                    }
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int n = first + (i0 + i) * per_pass;
                    if (i0 + i >= walk.passes || n >= walk.heads) continue;
                    const float by = e4m3_scale(scale[i]);
                    uint8_t *const head = to + slot + n * step;
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        if (p0 + q * lanes < walk.chunks)
                            store_e4m3<V, INTER>(head, Place<V, INTER>(p0 + q * lanes, a.turn.R, D), u[i][q], w[i][q], by);
                    if (p0 == 0) scales[scale_slot + n * kv.scale_head_stride] = by;
                }
            } else {
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int n = first + (i0 + i) * per_pass;
                    if (i0 + i >= walk.passes || n >= walk.heads) continue;
                    uint8_t *const head = to + 2 * (held ? slot : 0) + n * step * 2;
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        float u[V], w[V];
                        raw[i][q].values(u, w);
                        rotate<V>(u, w, c[q], s[q]);
                        raw[i][q].take(u, w, on[q]);
                        if (p0 + q * lanes < walk.chunks) raw[i][q].store(head, Place<V, INTER>(p0 + q * lanes, a.turn.R, D));
                    }
                }
            }
        }
    };
    if (part < a.queries.parts) {
        heads(a.q + t * a.q_token, a.queries, true, std::false_type{}, a.q_out + t * a.q_out_token, D, nullptr);
        return;
    }
    part -= a.queries.parts;
    const bool key = part < a.rows.parts;
    if (!key) part -= a.rows.parts;
    heads(key ? a.k + t * a.k_token : a.v + t * a.v_token, a.rows, key, std::true_type{}, static_cast<uint8_t *>(key ? kv.k : kv.v),
          kv.head_stride, key ? kv.k_scale : kv.v_scale);
}

// Chunks of V pairs: 16-byte words where the rotated part and the rest both split into them, 8-byte
// words where they are multiples of 8, else single pairs.
inline int pairs_of_chunk(int D, int R, bool inter) {
    if (inter) return R % 8 == 0 ? 4 : 1;
    return R % 16 == 0 && (D - R) % 16 == 0 ? 8 : R % 8 == 0 ? 4 : 1;
}

// `columns` of each of `heads` heads of T tokens in chunks of V pairs. A warp takes several passes
// over a token's heads, up to 12 or 16, where that leaves 16 warps for each
// multiprocessor: the sines and cosines are then shared by more heads.
inline Walk walk_of(int T, int heads, int columns, int V) {
    Walk w;
    w.chunks = columns / (2 * V);
    w.lanes_log = 0;
    while ((1 << w.lanes_log) < w.chunks && w.lanes_log < 5) ++w.lanes_log;
    w.heads = heads;
    const int per_pass = 32 >> w.lanes_log, passes = (heads + per_pass - 1) / per_pass, top = V == 8 ? 12 : 16;
    const int64_t share = (int64_t)T * passes / (16 * sm_count());
    const int most = share < 1 ? 1 : share < top ? (int)share : top;
    w.parts = (passes + most - 1) / most;
    w.passes = w.parts > 0 ? (passes + w.parts - 1) / w.parts : 0;
    return w;
}

inline epd_status_t grid_of(int T, int parts, int &grid) {
    const int64_t warps = (int64_t)T * parts;
    if (warps > INT32_MAX - kThreads) return EPD_ERR_UNSUPPORTED;
    grid = (int)((warps + kThreads / 32 - 1) / (kThreads / 32));
    return EPD_OK;
}

template <int V, bool INTER>
epd_status_t launch_append(const AppendArgs &a, int grid, cudaStream_t st) {
    constexpr int NP = V == 1 ? kMaxHeadDim / 2 / 32 : 1;
    return a.cache.dtype == EPD_BF16 ? launch_pdl(append_kernel<V, INTER, false, NP>, grid, kThreads, 0, st, a)
                                     : launch_pdl(append_kernel<V, INTER, true, NP>, grid, kThreads, 0, st, a);
}

inline bool rotation_ok(const uint64_t *steps, int R, int D, float scale) {
    return R >= 0 && R % 2 == 0 && R <= D && (R == 0 || (steps && aligned8(steps))) && scale == scale;
}

}  // namespace
}  // namespace epd

extern "C" epd_status_t ep_rotary(const void *x, int64_t token_stride, int64_t head_stride, const int32_t *positions,
                                  const uint64_t *steps, int num_tokens, int num_heads, int head_dim, int rotary_dim,
                                  int interleaved, float rotary_scale, int inverse, void *out,
                                  int64_t out_token_stride, int64_t out_head_stride, epd_stream_t stream) {
    using namespace epd;
    const int T = num_tokens, N = num_heads, D = head_dim, R = rotary_dim;
    if (T < 0 || N < 0 || D < 8 || D % 8 != 0 || R < 2 || !rotation_ok(steps, R, D, rotary_scale))
        return EPD_ERR_INVALID_ARG;
    for (const int64_t s : {token_stride, head_stride, out_token_stride, out_head_stride})
        if (s < 0 || s % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (D > kMaxHeadDim) return EPD_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return EPD_OK;
    if ((T > 1 && out_token_stride == 0) || (N > 1 && out_head_stride == 0)) return EPD_ERR_INVALID_ARG;
    if (!x || !out || !positions || !aligned16(x) || !aligned16(out) || !aligned4(positions)) return EPD_ERR_INVALID_ARG;
    RotaryArgs a;
    a.x = static_cast<const uint8_t *>(x);
    a.out = static_cast<uint8_t *>(out);
    a.x_token = 2 * token_stride, a.x_head = 2 * head_stride;
    a.out_token = 2 * out_token_stride, a.out_head = 2 * out_head_stride;
    a.positions = positions;
    a.T = T;
    a.D = D;
    a.turn = {steps, R, inverse != 0, rotary_scale};
    const int V = pairs_of_chunk(D, R, interleaved != 0);
    // in place the part that is not rotated stays as it is
    const bool in_place = x == out && token_stride == out_token_stride && head_stride == out_head_stride;
    a.walk = walk_of(T, N, in_place ? R : D, V);
    int grid;
    if (const epd_status_t rc = grid_of(T, a.walk.parts, grid)) return rc;
    a.parts = divisor(a.walk.parts);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (interleaved)
        return V == 4 ? launch_pdl(rotary_kernel<4, true>, grid, kThreads, 0, st, a)
                      : launch_pdl(rotary_kernel<1, true>, grid, kThreads, 0, st, a);
    return V == 8   ? launch_pdl(rotary_kernel<8, false>, grid, kThreads, 0, st, a)
           : V == 4 ? launch_pdl(rotary_kernel<4, false>, grid, kThreads, 0, st, a)
                    : launch_pdl(rotary_kernel<1, false>, grid, kThreads, 0, st, a);
}

extern "C" epd_status_t ep_cache_append(const epd_cache_t *cache, const void *q, int64_t q_token_stride,
                                        int num_heads, const void *k, int64_t k_token_stride, const void *v,
                                        int64_t v_token_stride, const int32_t *positions, const int32_t *token_seq,
                                        int num_tokens, const uint64_t *steps, int rotary_dim, int interleaved,
                                        float rotary_scale, void *q_out, int64_t q_out_token_stride, int32_t *status,
                                        epd_stream_t stream) {
    using namespace epd;
    if (const epd_status_t rc = check_cache(cache)) return rc;
    const int T = num_tokens, D = cache->head_dim, R = rotary_dim, QH = q ? num_heads : 0;
    if (T < 0 || num_heads < 0 || !rotation_ok(steps, R, D, rotary_scale)) return EPD_ERR_INVALID_ARG;
    for (const int64_t s : {q_token_stride, k_token_stride, v_token_stride, q_out_token_stride})
        if (s < 0 || s % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status)) return EPD_ERR_INVALID_ARG;
    if (!rows_apart(*cache) || (T > 1 && QH > 0 && q_out_token_stride == 0)) return EPD_ERR_INVALID_ARG;
    if (!token_seq && T > cache->num_seqs) return EPD_ERR_INVALID_ARG;
    if ((int64_t)QH + 2 * (int64_t)cache->num_kv_heads > INT32_MAX) return EPD_ERR_UNSUPPORTED;
    if (T == 0) return EPD_OK;
    if (!k || !v || !positions || !aligned16(k) || !aligned16(v) || !aligned4(positions) || !aligned4(token_seq))
        return EPD_ERR_INVALID_ARG;
    if (q && (!q_out || !aligned16(q) || !aligned16(q_out))) return EPD_ERR_INVALID_ARG;
    AppendArgs a;
    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.q_token = 2 * q_token_stride, a.k_token = 2 * k_token_stride, a.v_token = 2 * v_token_stride;
    a.q_out_token = 2 * q_out_token_stride;
    a.positions = positions;
    a.token_seq = token_seq;
    a.T = T;
    a.cache = *cache;
    a.turn = {steps, R, 0, rotary_scale};
    a.status = status;
    // without rotation the chunks are runs of 16 bytes
    const bool inter = interleaved || R == 0;
    const int V = pairs_of_chunk(D, R, inter);
    a.queries = walk_of(T, QH, D, V);
    a.rows = walk_of(T, cache->num_kv_heads, D, V);
    int grid;
    const int parts = a.queries.parts + 2 * a.rows.parts;
    if (const epd_status_t rc = grid_of(T, parts, grid)) return rc;
    a.parts = divisor(parts);
    a.page = divisor(cache->page_size);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (inter) return V == 4 ? launch_append<4, true>(a, grid, st) : launch_append<1, true>(a, grid, st);
    return V == 8 ? launch_append<8, false>(a, grid, st)
           : V == 4 ? launch_append<4, false>(a, grid, st)
                    : launch_append<1, false>(a, grid, st);
}
