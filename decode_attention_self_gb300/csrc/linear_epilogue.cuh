// What follows a matrix product's sums: activations, residual and the outputs' rows.
#pragma once

#include "dr_device.cuh"
#include "dr_layer.h"

namespace dr {
namespace lin {

// max(x, 0) that keeps a NaN
__device__ __forceinline__ float relu(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / x, within 1 ulp (PTX rcp.approx.ftz.f32)
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x / (1 + e^-x); 0 at -inf (e^-x of a large -x is +inf, whose reciprocal is 0)
__device__ __forceinline__ float silu(float x) {
    const float r = fast_rcp(1.0f + fast_exp2(-1.4426950408889634f * x));
    return x == -INFINITY ? 0.0f : x * r;
}
// x Phi(x) = max(x, 0) - m Q(m), m = |x|, Q the normal distribution's upper tail.  Q(m) e^(m^2/2) is smooth and is fitted
// here by a polynomial in t = 1 / (1 + 0.36 m), the form of Abramowitz and Stegun 7.1.26, with coefficients of its own:
// least squares reweighted to the least largest relative error on [0, 13], 7e-7 (1e-6 in fp32).  No cancellation: the
// sum's error is at most 2e-7 anywhere.  m is cut at 30, where Q is 0 in fp32, so that infinities give their limits.
__device__ __forceinline__ float gelu(float x) {
    const float m = fminf(fabsf(x), 30.0f);
    const float t = fast_rcp(fmaf(0.36f, m, 1.0f));
    float q = 0.047649674117565155f;
    q = fmaf(q, t, -0.18179528415203094f);
    q = fmaf(q, t, 0.18371888995170593f);
    q = fmaf(q, t, 0.024642769247293472f);
    q = fmaf(q, t, 0.14041736721992493f);
    q = fmaf(q, t, 0.14164447784423828f);
    q = fmaf(q, t, 0.14372217655181885f);
    const float e = fast_exp2(m * m * -0.72134752044448170f);   // e^(-m^2 / 2)
    return fmaf(-m * t * q, e, relu(x));
}
// x (1 + tanh u) / 2 = x / (1 + e^-2u), u = sqrt(2 / pi) (x + 0.044715 x^3)
__device__ __forceinline__ float gelu_tanh(float x) {
    const float v = x * fmaf(0.10294324f, x * x, 2.3022082f);   // 2 u log2(e)
    const float r = fast_rcp(1.0f + fast_exp2(-v));
    return x == -INFINITY ? 0.0f : x * r;
}

// act: one of DR_ACT_*, the same for every thread of a launch
template <int n>
__device__ __forceinline__ void activate(float *v, int act) {
    if (act == DR_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = gelu(v[i]);
    } else if (act == DR_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = silu(v[i]);
    } else if (act == DR_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = gelu_tanh(v[i]);
    } else if (act == DR_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = relu(v[i]);
    }
}

__device__ __forceinline__ float bf16_at(const uint16_t *p, int64_t i) {
    return __uint_as_float((uint32_t)__ldg(p + i) << 16);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight columns n .. n+7 (n a multiple of 8) of token t: bias, activation, gating and residual on the sums a (and b, the
// sums of the rows that are multiplied in), stored to the output that holds them.  Columns from N on are left out.
__device__ __forceinline__ void finish8(const LinearParams &p, int t, int n, float (&a)[8], float (&b)[8]) {
    const int have = min(8, p.N - n);
    if (have <= 0) return;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < have) a[i] += bf16_at(p.bias, n + i);
        if (p.gated) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) b[i] += bf16_at(p.bias, (int64_t)p.N + n + i);
        }
    }
    activate<8>(a, p.act);
    if (p.gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= b[i];
    }
    if (p.residual) {
        const int64_t at = (int64_t)t * p.res_stride + n;
        if (p.out_f32) {
            const float *r = static_cast<const float *>(p.residual) + at;
            if (p.vec_res && have == 8) {
                const float4 r0 = *reinterpret_cast<const float4 *>(r), r1 = *reinterpret_cast<const float4 *>(r + 4);
                a[0] += r0.x; a[1] += r0.y; a[2] += r0.z; a[3] += r0.w;
                a[4] += r1.x; a[5] += r1.y; a[6] += r1.z; a[7] += r1.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < have) a[i] += r[i];
            }
        } else {
            const uint16_t *r = static_cast<const uint16_t *>(p.residual) + at;
            if (p.vec_res && have == 8) {
                float f[8];
                unpack8(*reinterpret_cast<const uint4 *>(r), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] += f[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < have) a[i] += __uint_as_float((uint32_t)r[i] << 16);
            }
        }
    }
    int s = 0;
#pragma unroll
    for (int i = 1; i < DR_LINEAR_MAX_OUTS; ++i)
        if (i < p.n_outs && n >= p.out[i].col0) s = i;
    const int64_t at = (int64_t)t * p.out[s].stride + (n - p.out[s].col0);
    if (p.out_f32) {
        float *o = static_cast<float *>(p.out[s].ptr) + at;
        if (p.vec_out && have == 8) {
            *reinterpret_cast<float4 *>(o) = make_float4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<float4 *>(o + 4) = make_float4(a[4], a[5], a[6], a[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) o[i] = a[i];
        }
    } else {
        uint16_t *o = static_cast<uint16_t *>(p.out[s].ptr) + at;
        if (p.vec_out && have == 8) {
            *reinterpret_cast<uint4 *>(o) =
                make_uint4(pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) o[i] = f32_to_bf16_rn(a[i]);
        }
    }
}

}  // namespace lin
}  // namespace dr
