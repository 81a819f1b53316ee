// route.cu -- routing to experts and its gradient (ep_route, ep_route_backward).
//
// One warp owns one token: a row is read once, 16 bytes a lane where its alignment allows, and
// kept in registers as the values that decide the choice. The argmax is two warp reductions: the
// largest value, then the lowest index that has it -- the tie rule at no extra cost. Every lane
// keeps its two largest at hand, so that a pick costs its owner a move and only a lane's second
// pick a new pass over its values.
//
// What bounds it: a row of 256 logits is 1 KiB, 2.7 us for 16384 rows at the copy rate; the
// instructions of k rounds and of the scores (some 700 a token) take longer than that.
#include "route.cuh"

namespace epd {
namespace {

// The largest value of the warp (no NaN among them).
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

struct RouteArgs {
    const void *logits;
    const float *bias;
    int T, k, E, groups, keep, size;  // size: experts per group
    uint32_t by_size;                 // ceil(2^32 / size): e / size = high word of e * by_size
    int top2, renorm, vec, bias_vec;
    float scale;
    int64_t *idx;
    float *weights;
    int32_t *status;
};

__device__ __forceinline__ void merge_top2(float &b1, float &b2, float c1, float c2) {
    b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
    b1 = fmaxf(b1, c1);
}

__device__ __forceinline__ float group_score(float b1, float b2, bool top2) {
    return top2 && b2 > -CUDART_INF_F ? __fadd_rn(b1, b2) : b1;
}

// Which groups stay, as a bit mask, from the scores of groups g0 + lane of each 32.
__device__ __forceinline__ uint64_t keep_groups(const float (&mine)[EPD_MAX_GROUPS / 32], int groups, int keep, int lane) {
    uint64_t kept = 0;
#pragma unroll
    for (int h = 0; h < EPD_MAX_GROUPS / 32; ++h) {
        if (h * 32 >= groups) break;
        int ahead = 0;
        for (int o = 0; o < groups; ++o) {
            const float other = __shfl_sync(kFull, o < 32 ? mine[0] : mine[1], o & 31);
            ahead += other > mine[h] || (other == mine[h] && o < h * 32 + lane);
        }
        kept |= (uint64_t)__ballot_sync(kFull, h * 32 + lane < groups && ahead < keep) << (h * 32);
    }
    return kept;
}

template <typename T, int V, int SCORING>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a) {
    using L = Layout<T, V>;
    extern __shared__ float s_dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.E;
    float c[V];  // what decides the choice; -inf for an expert that cannot be chosen
    bool bad = false;
    load_row<T, V>(row, a.E, a.vec, lane, c, bad);
    if (bad) report(a.status, EPD_ERR_NONFINITE);
    float m = 0.0f, inv = 0.0f;
    const bool grouped = a.keep < a.groups;
    // scores are needed where a bias joins them or groups sum them; otherwise the logits order
    // experts and groups exactly as their scores do
    const bool scored = a.bias != nullptr || (grouped && a.top2);
    // renormalised softmax weights are the softmax of the picks alone
    if (SCORING == EPD_SCORE_SOFTMAX && (scored || !a.renorm)) softmax_stats<false>(c, m, inv);
    if (scored) {
#pragma unroll
        for (int q = 0; q < L::Q; ++q) {
            const int e0 = (q * 32 + lane) * L::C;
            float bias[L::C];
#pragma unroll
            for (int i = 0; i < L::C; ++i) bias[i] = 0.0f;
            if (a.bias) {
                if (a.bias_vec) {
                    if (e0 < a.E) {
#pragma unroll
                        for (int i = 0; i < L::C; i += 4) {
                            const float4 b = *reinterpret_cast<const float4 *>(a.bias + e0 + i);
                            bias[i] = b.x;
                            if (i + 1 < L::C) bias[i + 1] = b.y;
                            if (i + 2 < L::C) bias[i + 2] = b.z;
                            if (i + 3 < L::C) bias[i + 3] = b.w;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < L::C; ++i)
                        if (e0 + i < a.E) bias[i] = a.bias[e0 + i];
                }
            }
#pragma unroll
            for (int i = 0; i < L::C; ++i) {
                float &v = c[q * L::C + i];
                const float score = SCORING == EPD_SCORE_SIGMOID ? fast_sigmoid(v) : __expf(v - m) * inv;
                v = v > -CUDART_INF_F ? __fadd_rn(score, bias[i]) : -CUDART_INF_F;
            }
        }
    }
    if (grouped) {
        float mine[EPD_MAX_GROUPS / 32] = {-CUDART_INF_F, -CUDART_INF_F};
        const int width = a.size / L::C;  // lanes per group, where groups are runs of whole chunks
        const bool runs = width * L::C == a.size && (width & (width - 1)) == 0 && width <= 32 && a.groups <= 32;
        if (runs) {
            const int per = 32 / width;  // groups in each chunk of the warp
#pragma unroll
            for (int q = 0; q < L::Q; ++q) {
                float b1 = c[q * L::C], b2 = -CUDART_INF_F;
#pragma unroll
                for (int i = 1; i < L::C; ++i) {
                    b2 = fmaxf(b2, fminf(b1, c[q * L::C + i]));
                    b1 = fmaxf(b1, c[q * L::C + i]);
                }
                for (int o = width / 2; o; o >>= 1)
                    merge_top2(b1, b2, __shfl_xor_sync(kFull, b1, o), __shfl_xor_sync(kFull, b2, o));
                const float s = __shfl_sync(kFull, group_score(b1, b2, a.top2), (lane & (per - 1)) * width);
                if (lane / per == q) mine[0] = s;
            }
            int ahead = 0;
            for (int o = 0; o < a.groups; ++o) {
                const float other = __shfl_sync(kFull, mine[0], o);
                ahead += other > mine[0] || (other == mine[0] && o < lane);
            }
            const uint32_t kept = __ballot_sync(kFull, lane < a.groups && ahead < a.keep);
#pragma unroll
            for (int q = 0; q < L::Q; ++q) {
                const bool stays = (kept >> ((q * per + lane / width) & 31)) & 1;
#pragma unroll
                for (int i = 0; i < L::C; ++i) c[q * L::C + i] = stays ? c[q * L::C + i] : -CUDART_INF_F;
            }
        } else {
            // any other shape: from the row in shared memory, a power-of-two run of lanes a group
            float *s_row = s_dyn + (size_t)warp * (a.E + EPD_MAX_GROUPS), *s_group = s_row + a.E;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = L::index(i, lane);
                if (e < a.E) s_row[e] = c[i];
            }
            __syncwarp();
            int per = 1;
            while (per * 2 * a.groups <= 32) per *= 2;
            for (int g0 = 0; g0 < a.groups; g0 += 32 / per) {
                const int g = g0 + lane / per;
                float b1 = -CUDART_INF_F, b2 = -CUDART_INF_F;
                if (g < a.groups)
                    for (int i = lane % per; i < a.size; i += per)
                        merge_top2(b1, b2, s_row[g * a.size + i], -CUDART_INF_F);
                for (int o = per / 2; o; o >>= 1)
                    merge_top2(b1, b2, __shfl_xor_sync(kFull, b1, o), __shfl_xor_sync(kFull, b2, o));
                if (g < a.groups && lane % per == 0) s_group[g] = group_score(b1, b2, a.top2);
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < EPD_MAX_GROUPS / 32; ++h)
                if (h * 32 + lane < a.groups) mine[h] = s_group[h * 32 + lane];
            const uint64_t kept = keep_groups(mine, a.groups, a.keep, lane);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t e = (uint32_t)L::index(i, lane);
                const uint32_t g = a.size > 1 ? __umulhi(e, a.by_size) : e;
                const uint32_t half = g & 32 ? (uint32_t)(kept >> 32) : (uint32_t)kept;
                if (!((half >> (g & 31)) & 1)) c[i] = -CUDART_INF_F;
            }
        }
        if (a.top2 && !a.bias) {  // groups are summed scores, experts are ordered by their logits
            float l[V];
            load_row<T, V>(row, a.E, a.vec, lane, l, bad);
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = c[i] > -CUDART_INF_F ? l[i] : -CUDART_INF_F;
        }
    }
    // k rounds of argmax; lane j % 32 keeps pick j. o1, o2: the two largest's places in the lane's
    // part of the row, as index(i, 0)
    int pick[2] = {-1, -1};
    float b1 = -CUDART_INF_F, b2 = -CUDART_INF_F;
    int o1 = 0, o2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = c[i];
        const bool p1 = v > b1, p2 = v > b2;
        b2 = fmaxf(b2, fminf(b1, v));
        o2 = p1 ? o1 : p2 ? L::index(i, 0) : o2;
        b1 = fmaxf(b1, v);
        o1 = p1 ? L::index(i, 0) : o1;
    }
    bool second = true;  // b2, o2 are this lane's next one
    for (int j = 0; j < a.k; ++j) {
        const float top = redux_max(b1);
        if (top == -CUDART_INF_F) break;
        const int e = b1 == top ? o1 + lane * L::C : INT32_MAX;
        const int chosen = __reduce_min_sync(kFull, e);
        if ((j & 31) == lane) pick[j >> 5] = chosen;
        if (e == chosen) {
            if (second) {
                const int gone = o1;
                b1 = b2;
                o1 = o2;
                o2 = gone;
                second = false;
            } else {
                // o2 is the pick before this one; both leave, and the lane looks again
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (L::index(i, 0) == o1 || L::index(i, 0) == o2) c[i] = -CUDART_INF_F;
                b1 = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o1 = c[i] > b1 ? L::index(i, 0) : o1;
                    b1 = fmaxf(b1, c[i]);
                }
                o2 = o1;
            }
        }
    }
    float s[2];
    float sum = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = pick[h] >= 0 ? to_f32(row[pick[h]]) : -CUDART_INF_F;
    if (SCORING == EPD_SCORE_SOFTMAX && a.renorm) {
        m = warp_max(fmaxf(s[0], s[1]));
        inv = 1.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (SCORING == EPD_SCORE_SIGMOID)
            s[h] = sigmoid_f32(s[h]);
        else
            s[h] = pick[h] >= 0 ? expf(s[h] - m) * inv : 0.0f;
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

template <typename T, int V, int SCORING>
epd_status_t launch_route(RouteArgs a, cudaStream_t st) {
    a.vec = chunked<T, V>(a.logits, a.E);
    a.bias_vec = a.vec && Layout<T, V>::C % 4 == 0 && a.bias && aligned16(a.bias);
    const size_t smem = a.keep < a.groups ? (size_t)kRouteWarps * (a.E + EPD_MAX_GROUPS) * sizeof(float) : 0;
    const int grid = (a.T + kRouteWarps - 1) / kRouteWarps;
    auto kernel = route_kernel<T, V, SCORING>;
    if (smem > 48 * 1024) {
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        const epd_status_t rc = record_cuda_error();
        if (rc != EPD_OK) return rc;
    }
    return launch_pdl(kernel, grid, kRouteThreads, smem, st, a);
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
    a.size = E / num_groups;
    a.by_size = a.size > 1 ? (uint32_t)(((1ull << 32) + a.size - 1) / a.size) : 0;
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
