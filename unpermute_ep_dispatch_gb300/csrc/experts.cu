// experts.cu -- the experts' products over the expert-contiguous rows and their gradients
// (ep_expert_matmul, ep_expert_matmul_dgrad, ep_expert_matmul_wgrad).
//
// One tiled kernel for the three: C[i, j] = sum over r of A[i, r] * B[j, r], 64 x 64 tiles
// in fp32 on the ordinary cores, blocks walking the tiles of all experts.
#include "epd_math.cuh"

namespace epd {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;
enum { kForward = 0, kDgrad = 1, kWgrad = 2 };

struct ExpertArgs {
    epd_expert_rows_t rows;
    const uint8_t *a;  // x (forward), dy (dgrad, wgrad)
    const uint8_t *b;  // w (forward, dgrad), x (wgrad)
    const float *x_scale, *w_scale;
    int64_t srow, scol, sexp;
    int K, N;  // features in and out of the product
    const float *bias;
    const uint8_t *residual, *preact_in;
    uint8_t *y, *preact;
    float *dbias;
    int32_t *status;
};

__device__ __forceinline__ float load_bf16(const uint8_t *p, int64_t i) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ float load_e4m3(const uint8_t *p, int64_t i) {
    __nv_fp8_e4m3 v;
    v.__x = p[i];
    return static_cast<float>(v);
}
__device__ __forceinline__ void store_bf16(uint8_t *p, int64_t i, float v) {
    reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// The rows of expert e as they may be read: clipped, with an error where they do not fit.
__device__ __forceinline__ void expert_region(const epd_expert_rows_t &r, int e, int64_t &start,
                                              int &count, int32_t *status) {
    count = r.tokens_per_expert[e];
    start = r.expert_start_loc ? r.expert_start_loc[e] : e * r.rows_per_expert;
    if (count < 0 || start < 0) {
        report(status, EPD_ERR_INVALID_ARG);
        count = 0;
        start = 0;
    }
    int64_t room = r.capacity_rows - start;
    if (!r.expert_start_loc && room > r.rows_per_expert) room = r.rows_per_expert;
    if (count > room) {
        report(status, EPD_ERR_CAPACITY);
        count = room > 0 ? (int)room : 0;
    }
}

template <int MODE, bool FP8, int ACT>
__global__ void __launch_bounds__(kThreads) expert_kernel(ExpertArgs p) {
    constexpr bool kGated = ACT == EPD_ACT_SWIGLU;
    constexpr int kSets = (MODE == kForward && kGated) ? 2 : 1;
    __shared__ float sa[kStep][kTile + 1];
    __shared__ float sb[kSets][kStep][kTile + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y;
    int64_t start;
    int count;
    expert_region(p.rows, e, start, count, p.status);
    const int cols = MODE == kForward ? p.N : p.K;
    const int rows = MODE == kWgrad ? p.N : count;
    const int red = MODE == kForward ? p.K : MODE == kDgrad ? p.N : count;
    const int ct = (cols + kTile - 1) / kTile;
    const int64_t tiles = (int64_t)((rows + kTile - 1) / kTile) * ct;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int i0 = (int)(tile / ct) * kTile, j0 = (int)(tile % ct) * kTile;
        float acc[kSets][4][4] = {};
        for (int r0 = 0; r0 < red; r0 += kStep) {
            __syncthreads();
            for (int q = tid; q < kTile * kStep; q += kThreads) {
                // the reduction is contiguous in memory except for wgrad's operands
                const int i = MODE == kWgrad ? q % kTile : q / kStep;
                const int r = MODE == kWgrad ? q / kTile : q % kStep;
                float v = 0.0f;
                if (i0 + i < rows && r0 + r < red) {
                    if (MODE == kWgrad) {
                        v = load_bf16(p.a, (start + r0 + r) * p.N + i0 + i);
                    } else if (FP8) {
                        const int64_t s = start + i0 + i;
                        v = load_e4m3(p.a, s * p.K + r0 + r) *
                            p.x_scale[s * p.srow + (r0 + r) / 128 * p.scol + e * p.sexp];
                    } else {
                        v = load_bf16(p.a, (start + i0 + i) * red + r0 + r);
                    }
                }
                sa[r][i] = v;
#pragma unroll
                for (int z = 0; z < kSets; ++z) {
                    const bool turn = MODE != kForward;
                    const int jj = turn ? q % kTile : q / kStep, rr = turn ? q / kTile : q % kStep;
                    float w = 0.0f;
                    if (j0 + jj < cols && r0 + rr < red) {
                        const int64_t NW = (int64_t)p.N * kSets;
                        const int64_t f = (int64_t)z * p.N + j0 + jj;
                        if (MODE == kWgrad)
                            w = load_bf16(p.b, (start + r0 + rr) * p.K + j0 + jj);
                        else if (MODE == kDgrad)
                            w = load_bf16(p.b, ((int64_t)e * p.N + r0 + rr) * p.K + j0 + jj);
                        else if (FP8)
                            w = load_e4m3(p.b, (e * NW + f) * p.K + r0 + rr) *
                                p.w_scale[(e * ((NW + 127) / 128) + f / 128) * (p.K / 128) + (r0 + rr) / 128];
                        else
                            w = load_bf16(p.b, (e * NW + f) * p.K + r0 + rr);
                    }
                    sb[z][rr][jj] = w;
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kStep; ++r)
#pragma unroll
                for (int z = 0; z < kSets; ++z)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[z][i][j] = fmaf(sa[r][ty + 16 * i], sb[z][r][tx + 16 * j], acc[z][i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ii = i0 + ty + 16 * i;
            if (ii >= rows) continue;
            const int64_t s = start + ii;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int jj = j0 + tx + 16 * j;
                if (jj >= cols) continue;
                float v = acc[0][i][j];
                if (MODE == kWgrad) {
                    store_bf16(p.y, ((int64_t)e * p.N + ii) * p.K + jj, v);
                } else if (MODE == kDgrad) {
                    if (kGated) {
                        const float g = load_bf16(p.preact_in, s * 2 * p.K + jj);
                        const float u = load_bf16(p.preact_in, s * 2 * p.K + p.K + jj);
                        store_bf16(p.y, s * 2 * p.K + jj, v * u * activate_grad<ACT>(g));
                        store_bf16(p.y, s * 2 * p.K + p.K + jj, v * g * sigmoid_f32(g));
                    } else {
                        if (ACT != EPD_ACT_NONE) v *= activate_grad<ACT>(load_bf16(p.preact_in, s * p.K + jj));
                        store_bf16(p.y, s * p.K + jj, v);
                    }
                } else {
                    const int64_t NW = (int64_t)p.N * kSets;
                    if (p.bias) v += p.bias[e * NW + jj];
                    if (p.preact) store_bf16(p.preact, s * NW + jj, v);
                    if (kGated) {
                        float u = acc[kSets - 1][i][j];
                        if (p.bias) u += p.bias[e * NW + p.N + jj];
                        if (p.preact) store_bf16(p.preact, s * NW + p.N + jj, u);
                        v = v * sigmoid_f32(v) * u;
                    } else {
                        v = activate<ACT>(v);
                    }
                    if (p.residual) v += load_bf16(p.residual, s * p.N + jj);
                    store_bf16(p.y, s * p.N + jj, v);
                }
            }
        }
    }
    if (MODE == kWgrad && p.dbias) {
        for (int n = blockIdx.x * kThreads + tid; n < p.N; n += gridDim.x * kThreads) {
            float sum = 0.0f;
            for (int r = 0; r < count; ++r) sum += load_bf16(p.a, (start + r) * p.N + n);
            p.dbias[(int64_t)e * p.N + n] = sum;
        }
    }
}

template <int MODE, bool FP8>
epd_status_t launch(const ExpertArgs &p, int act, cudaStream_t stream) {
    auto kernel = expert_kernel<MODE, FP8, EPD_ACT_NONE>;
    if (MODE != kWgrad) {
        if (act == EPD_ACT_RELU) kernel = expert_kernel<MODE, FP8, EPD_ACT_RELU>;
        if (act == EPD_ACT_SILU) kernel = expert_kernel<MODE, FP8, EPD_ACT_SILU>;
        if (act == EPD_ACT_GELU) kernel = expert_kernel<MODE, FP8, EPD_ACT_GELU>;
        if (act == EPD_ACT_SWIGLU) kernel = expert_kernel<MODE, FP8, EPD_ACT_SWIGLU>;
    }
    kernel<<<dim3(64, p.rows.num_experts), kThreads, 0, stream>>>(p);
    return record_cuda_error();
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
    p.a = static_cast<const uint8_t *>(x);
    p.b = static_cast<const uint8_t *>(w);
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
    return fp8 ? launch<kForward, true>(p, activation, st) : launch<kForward, false>(p, activation, st);
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
    p.a = static_cast<const uint8_t *>(dy);
    p.b = static_cast<const uint8_t *>(w);
    p.K = K;
    p.N = N;
    p.preact_in = static_cast<const uint8_t *>(preact);
    p.y = static_cast<uint8_t *>(dx);
    p.status = status;
    return launch<kDgrad, false>(p, activation, reinterpret_cast<cudaStream_t>(stream));
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
    p.a = static_cast<const uint8_t *>(dy);
    p.b = static_cast<const uint8_t *>(x);
    p.K = K;
    p.N = N;
    p.y = static_cast<uint8_t *>(dw);
    p.dbias = dbias;
    p.status = status;
    return launch<kWgrad, false>(p, EPD_ACT_NONE, reinterpret_cast<cudaStream_t>(stream));
}
