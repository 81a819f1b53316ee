// route_backward.cu -- gradient of the router's weights (ep_route_backward).
//
// Sigmoid scores and renormalised softmax weights (the softmax of the picks alone) depend on the
// picks' logits only: the gradient is zero but for them, and the row is not read -- a warp fills
// its row with zeros and its lanes store their picks over them. Softmax weights without
// renormalising depend on the whole row: one pass over it in registers, and the picks over it the
// same way (16383 tokens of 256 experts, top-8: 8.6 us in a graph; the other form 6.2).
#include "route.cuh"

namespace epd {
namespace {

struct RouteGradArgs {
    const float *gw;
    const void *logits;
    const int64_t *idx;
    int T, k, E;
    int renorm, vec;
    float scale;
    void *grad;
    int32_t *status;
};

__device__ __forceinline__ void from_f32(float &p, float v) { p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &p, float v) { p = __float2bfloat16_rn(v); }

// What the two kernels know of a token's picks: lane j % 32 holds pick j (its expert, or -1), its
// logit and its weight's gradient.
template <typename T>
__device__ __forceinline__ void load_picks(const RouteGradArgs &a, int t, const T *row, int lane, int (&pick)[2],
                                           float (&logit)[2], float (&g)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = h * 32 + lane;
        pick[h] = -1;
        g[h] = 0.0f;
        logit[h] = -CUDART_INF_F;
        if (j < a.k) {
            const int64_t id = a.idx[(int64_t)t * a.k + j];
            if (id < -1 || id >= a.E) {
                report(a.status, EPD_ERR_INVALID_EXPERT);
            } else if (id >= 0) {
                bool bad = false;
                pick[h] = (int)id;
                logit[h] = clean_logit(to_f32(row[id]), bad);
                if (bad) report(a.status, EPD_ERR_NONFINITE);
                g[h] = a.gw[(int64_t)t * a.k + j] * a.scale;
            }
        }
    }
}

// Where a row picks an expert more than once, every one of its picks gets the sum of their
// gradients, in the picks' order. once: 0 for all of them but the first.
__device__ __forceinline__ void add_duplicates(int k, const int (&pick)[2], float (&g)[2], float (&once)[2]) {
    const uint32_t same = __match_any_sync(kFull, pick[0]);
    if (k <= 32 && !__any_sync(kFull, pick[0] >= 0 && (same & (same - 1)))) return;
    const int lane = threadIdx.x & 31;
    float d[2] = {0.0f, 0.0f};
    for (int i = 0; i < k; ++i) {
        const int e = __shfl_sync(kFull, i < 32 ? pick[0] : pick[1], i & 31);
        const float v = __shfl_sync(kFull, i < 32 ? g[0] : g[1], i & 31);
        if (e == pick[0]) {
            d[0] += v;
            if (i < lane) once[0] = 0.0f;
        }
        if (e == pick[1]) {
            d[1] += v;
            if (i < lane + 32) once[1] = 0.0f;
        }
    }
    g[0] = d[0];
    g[1] = d[1];
}

template <typename T, int SCORING>
__global__ void __launch_bounds__(kRouteThreads) route_backward_picks_kernel(RouteGradArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.E;
    T *out = static_cast<T *>(a.grad) + (int64_t)t * a.E;
    int pick[2];
    float g[2], x[2];
    load_picks(a, t, row, lane, pick, x, g);
    if (a.vec) {
        constexpr int C = 16 / sizeof(T);
        for (int e = lane * C; e < a.E; e += 32 * C) st16(out + e, make_uint4(0, 0, 0, 0));
    } else {
        for (int e = lane; e < a.E; e += 32) from_f32(out[e], 0.0f);
    }
    const bool two = a.k > 32;
    // what a pick's own logit does to its weight is ds s c: c = 1 - s for the sigmoid, and for the
    // softmax of the picks it is in ds already
    float s[2], c[2] = {1.0f, 1.0f};
    if (SCORING == EPD_SCORE_SOFTMAX) {
        const float m = warp_max(fmaxf(x[0], x[1]));
        s[0] = m > -CUDART_INF_F ? expf(x[0] - m) : 0.0f;
        s[1] = two && m > -CUDART_INF_F ? expf(x[1] - m) : 0.0f;
    } else {
        s[1] = 0.0f;
        sigmoid_pair(x[0], s[0], c[0]);
        if (two) sigmoid_pair(x[1], s[1], c[1]);
        if (a.renorm) lift_low(s, c, x);
    }
    if (a.renorm) {
        // from here on s are the weights, at most 1: their product with ds neither overflows nor
        // has to pass through 1 / sum
        const float sum = warp_sum(s[0] + s[1]);
        const float rs = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        float ds[2] = {0.0f, 0.0f};
        s[0] *= rs;
        s[1] *= rs;
        for (int i = 0; i < min(a.k, 32); ++i) {
            const float gi = __shfl_sync(kFull, g[0], i), pi = __shfl_sync(kFull, s[0], i);
            ds[0] += (g[0] - gi) * pi;
            if (two) ds[1] += (g[1] - gi) * pi;
        }
        for (int i = 32; i < a.k; ++i) {
            const float gi = __shfl_sync(kFull, g[1], i - 32), pi = __shfl_sync(kFull, s[1], i - 32);
            ds[0] += (g[0] - gi) * pi;
            ds[1] += (g[1] - gi) * pi;
        }
        g[0] = ds[0];
        g[1] = ds[1];
    }
    float once[2] = {};
    add_duplicates(a.k, pick, g, once);
    __syncwarp();  // the zeros come first
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (pick[h] >= 0) from_f32(out[pick[h]], g[h] * s[h] * c[h]);
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_backward_row_kernel(RouteGradArgs a) {
    using L = Layout<T, V>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.E;
    int pick[2];
    float g[2], ps[2], s[V];
    load_picks(a, t, row, lane, pick, ps, g);
    bool bad = false;
    load_row<T, V>(row, a.E, a.vec, lane, s, bad);
    if (bad) report(a.status, EPD_ERR_NONFINITE);
    float m, inv;
    softmax_stats<true>(s, m, inv);
    // A pick's gradient is s_j times the sum over all experts of s_i (ds_j - ds_i): with U the scores
    // of all that are not picked, U ds_j plus that sum over the picks. As ds_j - sum of ds_i s_i it
    // would lose its digits as s_j nears one. Of what is not picked it is -s_e times that last sum.
    float p[2], dot = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) p[h] = pick[h] >= 0 && inv > 0.0f ? expf(ps[h] - m) * inv : 0.0f;
    // which of a lane's elements are picked, a bit each
    constexpr int kWords = (V + 31) / 32;
    __shared__ uint32_t s_hit[kRouteWarps][kWords][32];
#pragma unroll
    for (int i = 0; i < kWords; ++i) s_hit[warp][i][lane] = inv > 0.0f ? 0 : kFull;  // nothing left: all are -inf
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (pick[h] >= 0) {
            const int chunk = pick[h] / L::C, i = chunk / 32 * L::C + pick[h] % L::C;
            atomicOr(&s_hit[warp][i / 32][chunk % 32], 1u << (i % 32));
        }
    __syncwarp();
    float rest = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if ((s_hit[warp][i / 32][lane] >> (i % 32)) & 1) s[i] = 0.0f;
        rest += s[i];
    }
    rest = warp_sum(rest) * inv;
    float once[2] = {p[0], p[1]};
    add_duplicates(a.k, pick, g, once);
    float ds[2] = {rest * g[0], rest * g[1]};
    for (int j = 0; j < a.k; ++j) {
        const float gj = __shfl_sync(kFull, j < 32 ? g[0] : g[1], j & 31);
        const float pj = __shfl_sync(kFull, j < 32 ? once[0] : once[1], j & 31);
        dot += gj * pj;
        ds[0] += (g[0] - gj) * pj;
        if (a.k > 32) ds[1] += (g[1] - gj) * pj;
    }
    T *out = static_cast<T *>(a.grad) + (int64_t)t * a.E;
    const float scale = -dot * inv;
#pragma unroll
    for (int q = 0; q < L::Q; ++q) {
        const int e0 = (q * 32 + lane) * L::C;
        alignas(16) T v[L::C];
#pragma unroll
        for (int c = 0; c < L::C; ++c) from_f32(v[c], s[q * L::C + c] * scale);
        if (a.vec) {
            if (e0 < a.E) {
                if (sizeof(v) == 16)
                    *reinterpret_cast<uint4 *>(out + e0) = *reinterpret_cast<const uint4 *>(v);
                else if (sizeof(v) == 8)
                    *reinterpret_cast<uint2 *>(out + e0) = *reinterpret_cast<const uint2 *>(v);
                else
                    *reinterpret_cast<uint32_t *>(out + e0) = *reinterpret_cast<const uint32_t *>(v);
            }
        } else {
#pragma unroll
            for (int c = 0; c < L::C; ++c)
                if (e0 + c < a.E) out[e0 + c] = v[c];
        }
    }
    __syncwarp();  // the picks over what the row has in their places
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (pick[h] >= 0) from_f32(out[pick[h]], ds[h] * p[h]);
}

template <typename T>
epd_status_t launch_route_backward(RouteGradArgs a, int scoring, cudaStream_t st) {
    const int grid = (a.T - 1) / kRouteWarps + 1;
    if (scoring == EPD_SCORE_SOFTMAX && !a.renorm)
        return by_width(a.E, [&](auto width) {
            constexpr int V = decltype(width)::value;
            a.vec = chunked<T, V>(a.logits, a.E) && chunked<T, V>(a.grad, a.E);
            return launch_pdl(route_backward_row_kernel<T, V>, grid, kRouteThreads, 0, st, a);
        });
    a.vec = a.E % (16 / sizeof(T)) == 0 && aligned16(a.grad);
    return launch_pdl(scoring == EPD_SCORE_SIGMOID ? route_backward_picks_kernel<T, EPD_SCORE_SIGMOID>
                                                   : route_backward_picks_kernel<T, EPD_SCORE_SOFTMAX>,
                      grid, kRouteThreads, 0, st, a);
}

}  // namespace
}  // namespace epd

extern "C" epd_status_t ep_route_backward(const float *grad_weights, const void *logits,
                                          epd_dtype_t dtype, const int64_t *topk_idx,
                                          int num_tokens, int num_topk, int num_experts,
                                          epd_scoring_t scoring, int renormalize,
                                          float routed_scale, void *grad_logits, int32_t *status,
                                          epd_stream_t stream) {
    using namespace epd;
    const int T = num_tokens, k = num_topk, E = num_experts;
    if (dtype != EPD_F32 && dtype != EPD_BF16) return EPD_ERR_INVALID_ARG;
    if (scoring != EPD_SCORE_SOFTMAX && scoring != EPD_SCORE_SIGMOID) return EPD_ERR_INVALID_ARG;
    if (T < 0 || E < 1 || E > EPD_MAX_EXPERTS || k < 1 || k > EPD_MAX_TOPK)
        return EPD_ERR_INVALID_ARG;
    if ((int64_t)T * k > INT32_MAX) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status)) return EPD_ERR_INVALID_ARG;
    if (T == 0) return EPD_OK;
    if (!logits || !topk_idx || !grad_weights || !grad_logits) return EPD_ERR_INVALID_ARG;
    const uintptr_t item = dtype == EPD_F32 ? 3u : 1u;
    if (!aligned8(topk_idx) || !aligned4(grad_weights) ||
        (reinterpret_cast<uintptr_t>(logits) & item) || (reinterpret_cast<uintptr_t>(grad_logits) & item))
        return EPD_ERR_INVALID_ARG;
    RouteGradArgs a;
    a.gw = grad_weights;
    a.logits = logits;
    a.idx = topk_idx;
    a.T = T;
    a.k = k;
    a.E = E;
    a.renorm = renormalize != 0;
    a.scale = routed_scale;
    a.grad = grad_logits;
    a.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == EPD_F32 ? launch_route_backward<float>(a, scoring, st)
                            : launch_route_backward<__nv_bfloat16>(a, scoring, st);
}
