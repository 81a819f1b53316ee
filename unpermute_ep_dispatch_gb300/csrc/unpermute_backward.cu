// unpermute_backward.cu -- gradient of the combine (ep_unpermute).
//
//   grad_expert_out[slot(t, j), h] = bf16( w[t, j] * gy[t, h] )
//   grad_weights[t, j]             = sum over h of gy[t, h] * eo[slot(t, j), h]
//
// Every expert-output row is read once and its gradient row written once, so the kernel is
// bound by HBM: 4 * H bytes per pair. A block owns a token: the token's gradient chunk is
// loaded once for its k picks, whose rows are all in flight before any arithmetic. The dot
// products are summed per thread, per warp and over the block's warps in a fixed order.
#include "epd_math.cuh"

namespace epd {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPicks = 8;  // picks handled at once

struct UnpermuteGradArgs {
    const uint8_t *gy, *eo;
    int64_t capacity;
    const int32_t *index;
    const float *w;
    int T, k;
    int64_t row_vecs;  // H / 8
    uint8_t *geo;
    float *gw;
    int32_t *status;
};

__global__ void __launch_bounds__(kThreads) unpermute_backward_kernel(UnpermuteGradArgs a) {
    __shared__ int s_slot[kPicks];
    __shared__ float s_w[kPicks];
    __shared__ float s_dot[kWarps][kPicks];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int64_t row_bytes = a.row_vecs << 4;
    const int t = blockIdx.x;
    for (int j0 = 0; j0 < a.k; j0 += kPicks) {
        if (tid < kPicks) {
            int slot = -1;
            float w = 0.0f;
            if (j0 + tid < a.k) {
                const int64_t p = (int64_t)t * a.k + j0 + tid;
                slot = a.index[p];
                w = a.w[p];
                if (slot < -1 || (int64_t)slot >= a.capacity) {
                    report(a.status, EPD_ERR_CAPACITY);
                    slot = -1;
                }
            }
            s_slot[tid] = slot;
            s_w[tid] = w;
        }
        __syncthreads();
        float dot[kPicks];
#pragma unroll
        for (int j = 0; j < kPicks; ++j) dot[j] = 0.0f;
        for (int64_t c = tid; c < a.row_vecs; c += kThreads) {
            const uint4 gv = ld_stream16(a.gy + (int64_t)t * row_bytes + (c << 4));
            uint4 v[kPicks];
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                const int slot = s_slot[j];
                v[j] = slot >= 0 ? ld_stream16(a.eo + (int64_t)slot * row_bytes + (c << 4))
                                 : make_uint4(0, 0, 0, 0);
            }
            float g[8];
            unpack8_bf16(gv, g);
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                const int slot = s_slot[j];
                if (slot < 0) continue;
                float f[8], o[8];
                unpack8_bf16(v[j], f);
                const float w = s_w[j];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot[j] = fmaf(g[i], f[i], dot[j]);
                    o[i] = w * g[i];
                }
                st16(a.geo + (int64_t)slot * row_bytes + (c << 4), pack8_bf16(o));
            }
        }
#pragma unroll
        for (int j = 0; j < kPicks; ++j) {
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if (lane == 0) s_dot[warp][j] = dot[j];
        }
        __syncthreads();
        if (tid < kPicks && j0 + tid < a.k) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum += s_dot[i][tid];
            a.gw[(int64_t)t * a.k + j0 + tid] = sum;
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace epd

extern "C" epd_status_t ep_unpermute_backward(const void *grad_y, const void *expert_out,
                                              int64_t capacity_rows, const int32_t *output_index,
                                              const float *topk_weights, int num_tokens,
                                              int num_topk, int hidden, void *grad_expert_out,
                                              float *grad_weights, int32_t *status,
                                              epd_stream_t stream) {
    using namespace epd;
    const int T = num_tokens, k = num_topk, H = hidden;
    if (T < 0 || k < 0 || k > EPD_MAX_TOPK || H <= 0 || H % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (capacity_rows < 0 || capacity_rows > INT32_MAX) return EPD_ERR_INVALID_ARG;
    if ((int64_t)T * k > INT32_MAX) return EPD_ERR_INVALID_ARG;
    if (!status || !aligned4(status)) return EPD_ERR_INVALID_ARG;
    if (T == 0 || k == 0) return EPD_OK;
    if (!grad_y || !aligned16(grad_y) || !output_index || !aligned4(output_index) || !topk_weights ||
        !aligned4(topk_weights) || !grad_weights || !aligned4(grad_weights))
        return EPD_ERR_INVALID_ARG;
    if (capacity_rows > 0 && (!expert_out || !aligned16(expert_out) || !grad_expert_out ||
                              !aligned16(grad_expert_out)))
        return EPD_ERR_INVALID_ARG;
    UnpermuteGradArgs a;
    a.gy = static_cast<const uint8_t *>(grad_y);
    a.eo = static_cast<const uint8_t *>(expert_out);
    a.capacity = capacity_rows;
    a.index = output_index;
    a.w = topk_weights;
    a.T = T;
    a.k = k;
    a.row_vecs = H / 8;
    a.geo = static_cast<uint8_t *>(grad_expert_out);
    a.gw = grad_weights;
    a.status = status;
    return launch_pdl(unpermute_backward_kernel, T, kThreads, 0, reinterpret_cast<cudaStream_t>(stream), a);
}
