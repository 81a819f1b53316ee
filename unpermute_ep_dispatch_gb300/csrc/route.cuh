// route.cuh -- what the router and its gradient share: the warp's row layout, its loads and the
// softmax statistics.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "epd_math.cuh"

namespace epd {
namespace {

constexpr int kRouteThreads = 128;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// The largest value of the warp (no NaN among them).
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// s = 1 / (1 + exp(-x)) and its complement c = 1 - s, each to the last place or two: the exponential
// is taken of -|x|, which neither overflows nor loses what is below the smallest normal number, and
// the complement is not a difference (at x = 15 that would be off by a sixth, from 17 on 0).
__device__ __forceinline__ void sigmoid_pair(float x, float &s, float &c) {
    const float e = expf(-fabsf(x)), r = __fdiv_rn(1.0f, 1.0f + e);
    s = x < 0.0f ? e * r : r;
    c = x < 0.0f ? r : e * r;
}

// Scores that are divided by their sum, of picks with sigmoid scores s, complements c and logits x
// (-inf: no pick). Where all logits are negative, s = exp(x) c is taken times exp(-m), m the largest
// logit, which the division takes out again: scores near or below the smallest normal number would
// leave their shares no digits, and the reciprocal of their sum may overflow. 0 where even the
// largest score is 0.
__device__ __forceinline__ void lift_low(float (&s)[2], const float (&c)[2], const float (&x)[2]) {
    const float m = redux_max(fmaxf(x[0], x[1]));
    if (m >= 0.0f) return;
    const bool any = expf(m) > 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = any ? expf(x[h] - m) * c[h] : 0.0f;
}

// A logit as the router reads it: NaN and +inf are reported and count as -inf.
__device__ __forceinline__ float clean_logit(float l, bool &bad) {
    if (!(l < CUDART_INF_F)) {
        bad = true;
        return -CUDART_INF_F;
    }
    return l;
}

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Lane-interleaved row: chunks of C elements, chunk q of lane l being elements
// (32 q + l) C .. + C - 1, so that element i of a lane is expert index_of<C>(i) and a chunk is
// one load of at most 16 bytes.
template <typename T, int V>
struct Layout {
    static constexpr int C = V < (int)(16 / sizeof(T)) ? V : (int)(16 / sizeof(T));
    static constexpr int Q = V / C;
    static __device__ __forceinline__ int index(int i, int lane) { return ((i / C) * 32 + lane) * C + i % C; }
};

// The row as the router reads it; elements past E count as -inf.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *row, int E, bool vec, int lane, float (&l)[V], bool &bad) {
    using L = Layout<T, V>;
#pragma unroll
    for (int q = 0; q < L::Q; ++q) {
        const int e0 = (q * 32 + lane) * L::C;
        if (vec) {  // E is a multiple of C
            alignas(16) T v[L::C];
            if (e0 < E) {
                if (sizeof(v) == 16)
                    *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(row + e0);
                else if (sizeof(v) == 8)
                    *reinterpret_cast<uint2 *>(v) = *reinterpret_cast<const uint2 *>(row + e0);
                else
                    *reinterpret_cast<uint32_t *>(v) = *reinterpret_cast<const uint32_t *>(row + e0);
            }
#pragma unroll
            for (int c = 0; c < L::C; ++c) l[q * L::C + c] = e0 < E ? to_f32(v[c]) : -CUDART_INF_F;
        } else {
#pragma unroll
            for (int c = 0; c < L::C; ++c)
                l[q * L::C + c] = e0 + c < E ? to_f32(row[e0 + c]) : -CUDART_INF_F;
        }
    }
    // one comparison a lane tells whether any of its logits has to be replaced
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
    if (!(top < CUDART_INF_F)) {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = clean_logit(l[i], bad);
    }
}

// A row's maximum and one over its sum of exponentials (0 where nothing is left). KEEP: the
// logits are replaced by the exponentials.
template <bool KEEP, int V>
__device__ __forceinline__ void softmax_stats(float (&l)[V], float &m, float &inv) {
    m = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float z = 0.0f;
    if (m > -CUDART_INF_F) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float e = expf(l[i] - m);
            z += e;
            if (KEEP) l[i] = e;
        }
    }
    z = warp_sum(z);
    inv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
}

// Whether rows of E elements at p can be read in the layout's chunks.
template <typename T, int V>
bool chunked(const void *p, int E) {
    constexpr int C = Layout<T, V>::C;
    return E % C == 0 && reinterpret_cast<uintptr_t>(p) % (C * sizeof(T)) == 0;
}

template <typename F>
epd_status_t by_width(int E, F f) {
    if (E <= 64) return f(std::integral_constant<int, 2>());
    if (E <= 128) return f(std::integral_constant<int, 4>());
    if (E <= 256) return f(std::integral_constant<int, 8>());
    if (E <= 512) return f(std::integral_constant<int, 16>());
    if (E <= 1024) return f(std::integral_constant<int, 32>());
    return f(std::integral_constant<int, EPD_MAX_EXPERTS / 32>());
}

}  // namespace
}  // namespace epd
