// route.cu -- routing to experts and its gradient (ep_route, ep_route_backward).
//
// One warp owns one token: lane l holds experts l, l + 32, ... of the row as keys in
// registers, so a row is read once and every reduction is a warp reduction. A key is the
// choice score c mapped to an unsigned integer of the same order (0 for an expert that
// cannot be chosen), which makes the argmax two integer warp reductions: the largest key,
// then the lowest index that has it -- the tie rule at no extra cost.
#include <math_constants.h>

#include "epd_math.cuh"

namespace epd {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

// Order-preserving key of a float that is neither NaN nor -inf; never 0. Adding +0 makes
// -0 and +0 one value.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

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

// A logit as the router reads it: NaN and +inf are reported and count as -inf.
__device__ __forceinline__ float clean_logit(float l, bool &bad) {
    if (!(l < CUDART_INF_F)) {
        bad = true;
        return -CUDART_INF_F;
    }
    return l;
}

struct RouteArgs {
    const void *logits;
    const float *bias;
    int T, k, E, groups, keep;
    int top2, renorm;
    float scale;
    int64_t *idx;
    float *weights;
    int32_t *status;
};

// The max and the sum of exponentials of a row.
template <int V>
__device__ __forceinline__ void softmax_stats(const float (&l)[V], float &m, float &inv) {
    m = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float z = 0.0f;
    if (m > -CUDART_INF_F) {
#pragma unroll
        for (int i = 0; i < V; ++i) z += expf(l[i] - m);
    }
    z = warp_sum(z);
    inv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
}

template <typename T, int V, int SCORING>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteArgs a) {
    extern __shared__ float s_dyn[];
    __shared__ float s_group[kWarps][EPD_MAX_GROUPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.E;
    float l[V];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        l[i] = e < a.E ? clean_logit(to_f32(row[e]), bad) : -CUDART_INF_F;
    }
    if (bad) report(a.status, EPD_ERR_NONFINITE);
    float m = 0.0f, inv = 0.0f;
    if (SCORING == EPD_SCORE_SOFTMAX) softmax_stats<V>(l, m, inv);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        float c = l[i];
        if (SCORING == EPD_SCORE_SIGMOID)
            c = sigmoid_f32(l[i]);
        else if (a.bias || a.top2)  // compared as scores; otherwise the logits order them
            c = expf(l[i] - m) * inv;
        if (a.bias && e < a.E) c = __fadd_rn(c, a.bias[e]);
        key[i] = l[i] > -CUDART_INF_F ? order_key(c) : 0u;
    }
    if (a.keep < a.groups) {
        // every group is scored by a power-of-two run of lanes from the row in shared memory
        float *s_row = s_dyn + (size_t)warp * a.E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 32 + lane;
            if (e < a.E) s_row[e] = key[i] ? key_value(key[i]) : -CUDART_INF_F;
        }
        __syncwarp();
        const int size = a.E / a.groups;
        int per = 1;
        while (per * 2 * a.groups <= 32) per *= 2;
        const int at_once = 32 / per;
        for (int g0 = 0; g0 < a.groups; g0 += at_once) {
            const int g = g0 + lane / per;
            float b1 = -CUDART_INF_F, b2 = -CUDART_INF_F;
            if (g < a.groups) {
                for (int i = lane % per; i < size; i += per) {
                    const float c = s_row[g * size + i];
                    if (c > b1) {
                        b2 = b1;
                        b1 = c;
                    } else {
                        b2 = fmaxf(b2, c);
                    }
                }
            }
            for (int o = per / 2; o; o >>= 1) {
                const float c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
                b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
                b1 = fmaxf(b1, c1);
            }
            if (g < a.groups && lane % per == 0) {
                float s = b1;
                if (a.top2 && b2 > -CUDART_INF_F) s = __fadd_rn(b1, b2);
                s_group[warp][g] = s;
            }
        }
        __syncwarp();
        uint64_t kept = 0;
        for (int g0 = 0; g0 < a.groups; g0 += 32) {
            const int g = g0 + lane;
            int ahead = 0;
            if (g < a.groups) {
                const float mine = s_group[warp][g];
                for (int o = 0; o < a.groups; ++o) {
                    const float other = s_group[warp][o];
                    ahead += other > mine || (other == mine && o < g);
                }
            }
            kept |= (uint64_t)__ballot_sync(kFull, g < a.groups && ahead < a.keep) << g0;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 32 + lane;
            if (e < a.E && !((kept >> (e / size)) & 1)) key[i] = 0;
            else if (a.top2 && SCORING == EPD_SCORE_SOFTMAX && !a.bias && key[i]) key[i] = order_key(l[i]);
        }
    } else if (a.top2 && SCORING == EPD_SCORE_SOFTMAX && !a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i]) key[i] = order_key(l[i]);
    }
    // k rounds of argmax; lane j % 32 keeps pick j
    int pick[2] = {-1, -1};
    uint32_t best = 0;
    int best_i = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (key[i] > best) best = key[i], best_i = i;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == 0) break;
        const int e = best_i * 32 + lane;
        const int chosen = __reduce_min_sync(kFull, best == top ? e : INT32_MAX);
        if ((j & 31) == lane) pick[j >> 5] = chosen;
        if ((chosen & 31) == lane) {
            best = 0;
            const int gone = chosen >> 5;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i == gone) key[i] = 0;
                if (key[i] > best) best = key[i], best_i = i;
            }
        }
    }
    float s[2];
    float sum = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s[h] = 0.0f;
        if (pick[h] >= 0) {
            const float v = to_f32(row[pick[h]]);
            s[h] = SCORING == EPD_SCORE_SIGMOID ? sigmoid_f32(v) : expf(v - m) * inv;
        }
        sum += s[h];
    }
    if (a.renorm) sum = warp_sum(sum);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = h * 32 + lane;
        if (j < a.k) {
            float w = s[h];
            if (a.renorm) w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
            a.idx[(int64_t)t * a.k + j] = pick[h];
            a.weights[(int64_t)t * a.k + j] = w * a.scale;
        }
    }
}

struct RouteGradArgs {
    const float *gw;
    const void *logits;
    const int64_t *idx;
    int T, k, E;
    int renorm;
    float scale;
    void *grad;
    int32_t *status;
};

__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T, int V, int SCORING>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(RouteGradArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.E;
    float s[V];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        s[i] = e < a.E ? clean_logit(to_f32(row[e]), bad) : -CUDART_INF_F;
    }
    if (bad) report(a.status, EPD_ERR_NONFINITE);
    float m = 0.0f, inv = 0.0f;
    if (SCORING == EPD_SCORE_SOFTMAX) {
        softmax_stats<V>(s, m, inv);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = inv > 0.0f ? expf(s[i] - m) * inv : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = sigmoid_f32(s[i]);
    }
    // the picks: lane j % 32 holds pick j, its score and its weight's gradient
    int pick[2];
    float g[2], ps[2];
    float sum = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = h * 32 + lane;
        pick[h] = -1;
        g[h] = ps[h] = 0.0f;
        if (j < a.k) {
            const int64_t id = a.idx[(int64_t)t * a.k + j];
            if (id < -1 || id >= a.E)
                report(a.status, EPD_ERR_INVALID_EXPERT);
            else
                pick[h] = (int)id;
            if (pick[h] >= 0) {
                bool b = false;
                const float v = clean_logit(to_f32(row[pick[h]]), b);
                ps[h] = SCORING == EPD_SCORE_SIGMOID ? sigmoid_f32(v)
                                                     : (inv > 0.0f ? expf(v - m) * inv : 0.0f);
                g[h] = a.gw[(int64_t)t * a.k + j] * a.scale;
            }
        }
        sum += ps[h];
    }
    if (a.renorm) {
        sum = warp_sum(sum);
        const float rs = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        float ds[2] = {0.0f, 0.0f};
        for (int i = 0; i < a.k; ++i) {
            const float gi = __shfl_sync(kFull, i < 32 ? g[0] : g[1], i & 31);
            const float pi = __shfl_sync(kFull, i < 32 ? ps[0] : ps[1], i & 31) * rs;
            ds[0] += (g[0] - gi) * pi;
            ds[1] += (g[1] - gi) * pi;
        }
        g[0] = ds[0] * rs;
        g[1] = ds[1] * rs;
    }
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int e = __shfl_sync(kFull, j < 32 ? pick[0] : pick[1], j & 31);
        const float v = __shfl_sync(kFull, j < 32 ? g[0] : g[1], j & 31);
        if (e >= 0 && (e & 31) == lane) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == (e >> 5)) d[i] += v;
        }
    }
    T *out = static_cast<T *>(a.grad) + (int64_t)t * a.E;
    float dot = 0.0f;
    if (SCORING == EPD_SCORE_SOFTMAX) {
        if (!a.renorm) {  // renormalised picks: the sum is zero
#pragma unroll
            for (int i = 0; i < V; ++i) dot += d[i] * s[i];
            dot = warp_sum(dot);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const float v = SCORING == EPD_SCORE_SIGMOID ? d[i] * s[i] * (1.0f - s[i]) : s[i] * (d[i] - dot);
        if (e < a.E) store_grad(out + e, v);
    }
}

template <typename T, int V, int SCORING>
epd_status_t launch_route(const RouteArgs &a, cudaStream_t st) {
    const size_t smem = a.keep < a.groups ? (size_t)kWarps * a.E * sizeof(float) : 0;
    const int grid = (a.T + kWarps - 1) / kWarps;
    auto kernel = route_kernel<T, V, SCORING>;
    if (smem > 48 * 1024 - sizeof(float) * kWarps * EPD_MAX_GROUPS) {
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        const epd_status_t rc = record_cuda_error();
        if (rc != EPD_OK) return rc;
    }
    return launch_pdl(kernel, grid, kThreads, smem, st, a);
}

template <typename T, int V, int SCORING>
epd_status_t launch_route_backward(const RouteGradArgs &a, cudaStream_t st) {
    return launch_pdl(route_backward_kernel<T, V, SCORING>, (a.T + kWarps - 1) / kWarps, kThreads, 0, st, a);
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

extern "C" epd_status_t ep_route(const void *logits, epd_dtype_t dtype, const float *bias,
                                 int num_tokens, int num_topk, int num_experts, int num_groups,
                                 int topk_groups, epd_group_score_t group_score,
                                 epd_scoring_t scoring, int renormalize, float routed_scale,
                                 int64_t *topk_idx, float *topk_weights, int32_t *status,
                                 epd_stream_t stream) {
    using namespace epd;
    const int T = num_tokens, k = num_topk, E = num_experts;
    if (dtype != EPD_F32 && dtype != EPD_BF16) return EPD_ERR_INVALID_ARG;
    if (scoring != EPD_SCORE_SOFTMAX && scoring != EPD_SCORE_SIGMOID) return EPD_ERR_INVALID_ARG;
    if (group_score != EPD_GROUP_MAX && group_score != EPD_GROUP_TOP2) return EPD_ERR_INVALID_ARG;
    if (T < 0 || E < 1 || E > EPD_MAX_EXPERTS || k < 1 || k > EPD_MAX_TOPK || k > E)
        return EPD_ERR_INVALID_ARG;
    if (num_groups < 1 || E % num_groups != 0 || topk_groups < 1 || topk_groups > num_groups)
        return EPD_ERR_INVALID_ARG;
    if (num_groups > EPD_MAX_GROUPS) return EPD_ERR_UNSUPPORTED;
    if ((int64_t)T * k > INT32_MAX) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status)) return EPD_ERR_INVALID_ARG;
    if (T == 0) return EPD_OK;
    if (!logits || !topk_idx || !topk_weights) return EPD_ERR_INVALID_ARG;
    if (!aligned8(topk_idx) || !aligned4(topk_weights) || (bias && !aligned4(bias)) ||
        (reinterpret_cast<uintptr_t>(logits) & (dtype == EPD_F32 ? 3u : 1u)))
        return EPD_ERR_INVALID_ARG;
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.T = T;
    a.k = k;
    a.E = E;
    a.groups = num_groups;
    a.keep = topk_groups;
    a.top2 = group_score == EPD_GROUP_TOP2 && topk_groups < num_groups;
    a.renorm = renormalize != 0;
    a.scale = routed_scale;
    a.idx = topk_idx;
    a.weights = topk_weights;
    a.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto type, auto sc) {
        using T_ = decltype(type);
        constexpr int SC = decltype(sc)::value;
        return by_width(E, [&](auto v) { return launch_route<T_, decltype(v)::value, SC>(a, st); });
    };
    if (dtype == EPD_F32)
        return scoring == EPD_SCORE_SOFTMAX ? go(float(), std::integral_constant<int, EPD_SCORE_SOFTMAX>())
                                            : go(float(), std::integral_constant<int, EPD_SCORE_SIGMOID>());
    return scoring == EPD_SCORE_SOFTMAX
               ? go(__nv_bfloat16(), std::integral_constant<int, EPD_SCORE_SOFTMAX>())
               : go(__nv_bfloat16(), std::integral_constant<int, EPD_SCORE_SIGMOID>());
}

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
    auto go = [&](auto type, auto sc) {
        using T_ = decltype(type);
        constexpr int SC = decltype(sc)::value;
        return by_width(E, [&](auto v) { return launch_route_backward<T_, decltype(v)::value, SC>(a, st); });
    };
    if (dtype == EPD_F32)
        return scoring == EPD_SCORE_SOFTMAX ? go(float(), std::integral_constant<int, EPD_SCORE_SOFTMAX>())
                                            : go(float(), std::integral_constant<int, EPD_SCORE_SIGMOID>());
    return scoring == EPD_SCORE_SOFTMAX
               ? go(__nv_bfloat16(), std::integral_constant<int, EPD_SCORE_SOFTMAX>())
               : go(__nv_bfloat16(), std::integral_constant<int, EPD_SCORE_SIGMOID>());
}
