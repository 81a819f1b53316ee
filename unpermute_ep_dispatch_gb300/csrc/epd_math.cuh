// epd_math.cuh -- conversions and activations shared by the router, the experts'
// products and the gradients.
#pragma once

#include <cuda_bf16.h>

#include "epd_common.cuh"

namespace epd {

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Two floats rounded to nearest even, `lo` in the low half.
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}

__device__ __forceinline__ void unpack8_bf16(const uint4 &v, float (&f)[8]) {
    f[0] = lo_bf16(v.x), f[1] = hi_bf16(v.x), f[2] = lo_bf16(v.y), f[3] = hi_bf16(v.y);
    f[4] = lo_bf16(v.z), f[5] = hi_bf16(v.z), f[6] = lo_bf16(v.w), f[7] = hi_bf16(v.w);
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8]) {
    return make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]),
                      pack2_bf16(f[6], f[7]));
}

// 1 / (1 + exp(-x)): 0 for -inf and for the lowest finite value, 1 for +inf.
__device__ __forceinline__ float sigmoid_f32(float x) {
    return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x)));
}

constexpr float kSqrtHalf = 0.70710678118654752440f;
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;

__device__ __forceinline__ float gelu_cdf(float z) { return 0.5f * (1.0f + erff(z * kSqrtHalf)); }

// The sigmoid of the activations, by the hardware's exponential and reciprocal: within a few
// 2^-22 of its value, far below the bf16 it is rounded to (and 0 where it is below 2^-126).
__device__ __forceinline__ float fast_sigmoid(float x) {
    constexpr float kLog2e = 1.4426950408889634f;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -kLog2e));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// act(z) of the ungated activations.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if (ACT == EPD_ACT_RELU) return z < 0.0f ? 0.0f : z;  // keeps NaN
    if (ACT == EPD_ACT_SILU) return z * fast_sigmoid(z);
    if (ACT == EPD_ACT_GELU) return z * gelu_cdf(z);
    return z;
}

// act'(z) of the ungated activations (relu'(0) = 0), and of silu for the gated one.
template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
    if (ACT == EPD_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (ACT == EPD_ACT_SILU || ACT == EPD_ACT_SWIGLU) {
        const float s = fast_sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if (ACT == EPD_ACT_GELU) return gelu_cdf(z) + z * (kInvSqrt2Pi * expf(-0.5f * z * z));
    return 1.0f;
}

}  // namespace epd
