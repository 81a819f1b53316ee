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

// What a division of many numbers by one scale takes: 1 / scale rounded, and -scale (0 for an infinite one,
// by which finite numbers are 0).
struct Quotient {
    float inv, minus;
    __device__ __forceinline__ Quotient(float scale, float inverse) : inv(inverse), minus(scale < INFINITY ? -scale : 0.0f) {}
    // v / scale, rounded as the division is: the product with the inverse is two units off at most, and the
    // remainder, exact in one instruction, sets it right (100 million random quotients were all the
    // division's). Two to an instruction.
    __device__ __forceinline__ float2 operator()(float2 v) const {
        const float2 i = make_float2(inv, inv), q = __fmul2_rn(v, i);
        return __ffma2_rn(__ffma2_rn(q, make_float2(minus, minus), v), i, q);
    }
    __device__ __forceinline__ float operator()(float v) const {
        const float q = v * inv;
        return fmaf(fmaf(q, minus, v), inv, q);
    }
};

// The scale of e4m3 numbers whose largest is amax: amax / 448, 1 of 0; where it would round to 0, the
// smallest number there is.
__device__ __forceinline__ float e4m3_scale(float amax) {
    return amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-149f) : 1.0f;
}

// Scales below this: the remainder, or the scale's inverse, may not fit.
constexpr float kTinyScale = 0x1p-80f;

// v / scale for all of v, by one division; a tiny scale and they are taken 2^100 up first.
template <int N>
__device__ __forceinline__ void divide_all(float (&v)[N], float scale) {
    if (scale < kTinyScale) {
        scale *= 0x1p100f;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= 0x1p100f;
    }
    const Quotient by(scale, __fdiv_rn(1.0f, scale));
    if constexpr (N == 1) {
        v[0] = by(v[0]);
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 q = by(make_float2(v[j], v[j + 1]));
            v[j] = q.x, v[j + 1] = q.y;
        }
    }
}

constexpr float kInvSqrt2Pi = 0.39894228040143267794f;
constexpr float kLog2e = 1.4426950408889634f;

// The hardware's 2^x and 1/x, within 2^-22 and 2^-23 of their values; what is below 2^-126 is 0.
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The sigmoid of the activations. The exponential's argument is a rounded product, so that its error
// grows with |x|: 4 units of 2^-22 of its value at -15, 8 at -30 and 16 at -86, far below the bf16
// that it is rounded to; 0 below -87.3 (2^-126), where z * sigmoid(z) is 10^-36 at most. (The router's
// scores decide between experts and are computed to the last places.)
__device__ __forceinline__ float fast_sigmoid(float x) { return fast_rcp(1.0f + fast_exp2(x * -kLog2e)); }

// The normal distribution function, and e = exp(-z^2 / 2), which its derivative is a multiple of.
// Below zero it is exp(-z^2 / 2) erfcx(|z| / sqrt 2) / 2, and the scaled complementary error
// function over t = 1 / (1 + 9/32 |z|) is smooth for t in (0, 1]: a polynomial fitted to the least
// relative error (1.5e-7) takes it, without branches and with one exponential for both (dgrad into
// GELU, 24 experts of 28 rows, 904 x 520: 7.9 us, with erff and expf 8.9).
// Absolute error 3e-7, relative 1e-6 for z > -3 and 3e-6 for z > -8.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float t = fast_rcp(fmaf(fabsf(z), 0.28125f, 1.0f));
    e = fast_exp2(z * z * (-0.5f * kLog2e));
    float q = 0.02489628456532955f;
    q = fmaf(q, t, -0.09263245016336441f);
    q = fmaf(q, t, 0.08888789266347885f);
    q = fmaf(q, t, -0.004765740130096674f);
    q = fmaf(q, t, 0.07183780521154404f);
    q = fmaf(q, t, 0.08392227441072464f);
    q = fmaf(q, t, 0.1034524142742157f);
    q = fmaf(q, t, 0.11219891905784607f);
    q = fmaf(q, t, 0.11220253258943558f);
    const float tail = t * e * q;
    return z < 0.0f ? tail : 1.0f - tail;
}

// act(z) of the ungated activations.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if (ACT == EPD_ACT_RELU) return z < 0.0f ? 0.0f : z;  // keeps NaN
    if (ACT == EPD_ACT_SILU) return z * fast_sigmoid(z);
    if (ACT == EPD_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
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
    if (ACT == EPD_ACT_GELU) {
        float e;
        const float cdf = normal_cdf(z, e);
        return fmaf(z * e, kInvSqrt2Pi, cdf);
    }
    return 1.0f;
}

}  // namespace epd
