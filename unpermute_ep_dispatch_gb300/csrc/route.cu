// route.cu -- routing to experts (ep_route).
//
// One warp owns one token: a row is read once, 16 bytes a lane where its alignment allows, and
// kept by the lane as the values that decide the choice. The argmax is two warp reductions: the
// largest value, then the lowest index that has it -- the tie rule at no extra cost. Every lane
// keeps its two largest at hand, so that a pick costs its owner a move and only a lane's second
// pick a new pass over its values, for those that come after the pick in the order of picks.
//
// What bounds it: a row of 256 logits is 1 KiB, 2.7 us for 16384 rows at the copy rate; its
// instructions (817 a token with a bias and 4 of 8 groups, 475 for plain softmax; most of
// them compares, selects and maxima at half rate) take 14.6 and 9.6 us back to back in a graph.
// Kernels for rows of up to 256 logits are held to 32 registers a thread, so that sixteen blocks fit
// an SM and a call starts under the end of the one before: 4097 rows 5.6 us from 7.2 in a graph,
// 16384 the same. (From 129 logits on, that spills 32 to 52 bytes a thread.) Rows of more than 1024 logits
// have one form, 128 values a lane in 255 registers with 100 to 170 bytes spilled: 4096 tokens of
// 4096 logits, softmax, 44 us (9.9 of bytes), of 2048 with a bias 75.
#include "route.cuh"

namespace epd {
namespace {

struct RouteArgs {
    const void *logits;
    const float *bias;
    int T, k, E, groups, keep, size;  // size: experts per group
    int run;                          // log2 of the lanes per group, where groups are runs of whole chunks; or -1
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
__global__ void __launch_bounds__(kRouteThreads, V <= 8 ? 16 : 1) route_kernel(RouteArgs a) {
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
        float worst = -CUDART_INF_F;
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
                // expf, for the choice is told apart by these: with the hardware's 2^x of a rounded
                // product neighbouring logits tie from 11 on (16384 tokens grouped: 13.7 us for 14.4 so)
                float score;
                if (SCORING == EPD_SCORE_SIGMOID) {
                    const float e = expf(-fabsf(v));
                    score = (v < 0.0f ? e : 1.0f) * fast_rcp(1.0f + e);
                } else {
                    score = expf(v - m) * inv;
                }
                v = v > -CUDART_INF_F ? __fadd_rn(score, bias[i]) : -CUDART_INF_F;
                worst = max_nan(worst, v);
            }
        }
        if (worst != worst) {  // a NaN bias
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = c[i] == c[i] ? c[i] : -CUDART_INF_F;
            report(a.status, EPD_ERR_NONFINITE);
        }
    }
    if (grouped) {
        if (a.run >= 0) {
            // every lane of a run gets its group's score, and compares it with those of all groups,
            // one a lane and pass
            const int width = 1 << a.run, per = 32 >> a.run;  // per: groups in each chunk of the warp
            float score[L::Q], all = -CUDART_INF_F;           // all: that of group `lane`
            int ahead[L::Q];
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
                score[q] = group_score(b1, b2, a.top2);
                const float s = __shfl_sync(kFull, score[q], (lane & (per - 1)) << a.run);
                if (lane >> (5 - a.run) == q) all = s;
                ahead[q] = 0;
            }
            const uint32_t mine = (0xffffffffu >> (32 - width)) << (lane & -width);  // this run's lanes
            for (int o0 = 0; o0 < a.groups; o0 += width) {
                const int o = o0 + (lane & (width - 1));
                const float other = __shfl_sync(kFull, all, o);
#pragma unroll
                for (int q = 0; q < L::Q; ++q) {
                    const int g = q * per + (lane >> a.run);
                    const bool before = other > score[q] || (other == score[q] && o < g);
                    ahead[q] += __popc(__ballot_sync(kFull, before) & mine);
                }
            }
#pragma unroll
            for (int q = 0; q < L::Q; ++q)
#pragma unroll
                for (int i = 0; i < L::C; ++i) c[q * L::C + i] = ahead[q] < a.keep ? c[q * L::C + i] : -CUDART_INF_F;
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
            float mine[EPD_MAX_GROUPS / 32] = {-CUDART_INF_F, -CUDART_INF_F};
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
    // k rounds of argmax; lane j % 32 keeps pick j. o1, o2: the experts of the lane's two largest
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
    o1 += lane * L::C, o2 += lane * L::C;
    for (int j = 0; j < a.k; ++j) {
        const float top = redux_max(b1);
        if (top == -CUDART_INF_F) break;
        const int e = b1 == top ? o1 : INT32_MAX;
        const int chosen = __reduce_min_sync(kFull, e);
        if (j == lane) pick[0] = chosen;
        if (j == lane + 32) pick[1] = chosen;
        if (e == chosen) {  // its next one; NaN once that is not at hand any more
            b1 = b2;
            o1 = o2;
            b2 = CUDART_NAN_F;
        }
        if (b1 != b1) {
            // the lane looks again, among what comes after the pick: picks come in order
            b1 = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = L::index(i, lane);
                const bool left = c[i] < top || (c[i] == top && at > chosen);
                if (left && c[i] > b1) b1 = c[i], o1 = at;
            }
        }
    }
    const int halves = a.k > 32 ? 2 : 1;
    float x[2] = {-CUDART_INF_F, -CUDART_INF_F}, s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (h < halves && pick[h] >= 0) x[h] = to_f32(row[pick[h]]);
    if (SCORING == EPD_SCORE_SIGMOID) {
        float c[2] = {1.0f, 1.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (h < halves) sigmoid_pair(x[h], s[h], c[h]);
        if (a.renorm) lift_low(s, c, x);
    } else {
        if (a.renorm) {
            m = warp_max(fmaxf(x[0], x[1]));
            inv = 1.0f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (h < halves && pick[h] >= 0) s[h] = expf(x[h] - m) * inv;
    }
    float sum = s[0] + s[1];
    if (a.renorm) sum = warp_sum(sum);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h == halves) break;
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
    const int width = a.size / Layout<T, V>::C;
    a.run = -1;
    if (width * Layout<T, V>::C == a.size && (width & (width - 1)) == 0 && width <= 32 && a.groups <= 32)
        for (a.run = 0; width >> a.run > 1;) ++a.run;
    const size_t smem = a.keep < a.groups && a.run < 0 ? (size_t)kRouteWarps * (a.E + EPD_MAX_GROUPS) * sizeof(float) : 0;
    const int grid = (a.T - 1) / kRouteWarps + 1;
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
