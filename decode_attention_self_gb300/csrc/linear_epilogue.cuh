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
// The activations take two values at a time: the packed fp32 instructions need half the issue slots.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// v r, and 0 at v = -inf, where r is 0
__device__ __forceinline__ float2 times_tail(float2 v, float2 r) {
    return make_float2(v.x == -INFINITY ? 0.0f : v.x * r.x, v.y == -INFINITY ? 0.0f : v.y * r.y);
}
// 1 / (1 + 2^-v); e^-x of a large -x is +inf, whose reciprocal is 0
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 d = __fadd2_rn(make_float2(fast_exp2(-v.x), fast_exp2(-v.y)), both(1.0f));
    return make_float2(fast_rcp(d.x), fast_rcp(d.y));
}
// x / (1 + e^-x)
__device__ __forceinline__ float2 silu(float2 x) { return times_tail(x, sigmoid2(__fmul2_rn(x, both(1.4426950408889634f)))); }
// x (1 + tanh u) / 2 = x / (1 + e^-2u), u = sqrt(2 / pi) (x + 0.044715 x^3)
__device__ __forceinline__ float2 gelu_tanh(float2 x) {
    const float2 c = __ffma2_rn(__fmul2_rn(x, x), both(0.10294324f), both(2.3022082f));   // 2 u log2(e) / x
    return times_tail(x, sigmoid2(__fmul2_rn(x, c)));
}
// x Phi(x) = max(x, 0) - m Q(m), m = |x|, Q the normal distribution's upper tail.  Q(m) e^(m^2/2) is smooth and is fitted
// here by a polynomial in t = 1 / (1 + 0.36 m), the form of Abramowitz and Stegun 7.1.26, with coefficients of its own:
// least squares reweighted to the least largest relative error on [0, 13], 7e-7 (1e-6 in fp32).  No cancellation: the
// sum's error is at most 2e-7 anywhere.  m is cut at 30, where Q is 0 in fp32, so that infinities give their limits.
__device__ __forceinline__ float2 gelu(float2 x) {
    const float2 m = make_float2(fminf(fabsf(x.x), 30.0f), fminf(fabsf(x.y), 30.0f));
    const float2 d = __ffma2_rn(both(0.36f), m, both(1.0f));
    const float2 t = make_float2(fast_rcp(d.x), fast_rcp(d.y));
    float2 q = __ffma2_rn(both(-0.047649674117565155f), t, both(0.18179528415203094f));   // -q: the sign goes with it
    q = __ffma2_rn(q, t, both(-0.18371888995170593f));
    q = __ffma2_rn(q, t, both(-0.024642769247293472f));
    q = __ffma2_rn(q, t, both(-0.14041736721992493f));
    q = __ffma2_rn(q, t, both(-0.14164447784423828f));
    q = __ffma2_rn(q, t, both(-0.14372217655181885f));
    const float2 a = __fmul2_rn(__fmul2_rn(m, both(-0.72134752044448170f)), m);
    const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));   // e^(-m^2 / 2)
    return __ffma2_rn(__fmul2_rn(__fmul2_rn(m, t), q), e, make_float2(relu(x.x), relu(x.y)));
}

// act: one of DR_ACT_*, the same for every thread of a launch
template <int n>
__device__ __forceinline__ void activate(float *v, int act) {
    const auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < n; i += 2) {
            const float2 y = f(make_float2(v[i], v[i + 1]));
            v[i] = y.x;
            v[i + 1] = y.y;
        }
    };
    if (act == DR_ACT_GELU) {
        each([](float2 x) { return gelu(x); });
    } else if (act == DR_ACT_SILU) {
        each([](float2 x) { return silu(x); });
    } else if (act == DR_ACT_GELU_TANH) {
        each([](float2 x) { return gelu_tanh(x); });
    } else if (act == DR_ACT_RELU) {
        each([](float2 x) { return make_float2(relu(x.x), relu(x.y)); });
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

// v[0 .. 8) += bias[i .. i+8); places from `have` on are left out.  bias is 16-byte aligned.
__device__ __forceinline__ void add_bias8(float *v, const uint16_t *bias, int64_t i, int have) {
    if (have >= 8 && i % 8 == 0) {
        float f[8];
        unpack8(ld_ro16(bias + i), f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 y = __fadd2_rn(make_float2(v[j], v[j + 1]), make_float2(f[j], f[j + 1]));
            v[j] = y.x;
            v[j + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < have) v[j] += bf16_at(bias, i + j);
    }
}

// Eight columns n .. n+7 (n a multiple of 8) of token t: bias, activation, gating and residual on the sums a (and b, the
// sums of the rows that are multiplied in), stored to the output that holds them.  Columns from N on are left out.
__device__ __forceinline__ void finish8(const LinearParams &p, int t, int n, float (&a)[8], float (&b)[8]) {
    const int have = min(8, p.N - n);
    if (have <= 0) return;
    if (p.bias) {
        add_bias8(a, p.bias, n, have);
        if (p.gated) add_bias8(b, p.bias, (int64_t)p.N + n, have);
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
