// What follows a matrix product's sums: activations, residual and the outputs' rows.
#pragma once

#include <type_traits>

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

// Plain loads throughout: what another kernel may still be writing while this one starts must not be read before the wait, and
// the compiler may move read-only loads.
__device__ __forceinline__ float bf16_at(const uint16_t *p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The output that holds column n (and by value: constant operands, where a looked-up place of the parameters is a load).
__device__ __forceinline__ int out_of(const LinearParams &p, int n) {
    int s = 0;
    for (int i = 1; i < p.n_outs; ++i)
        if (n >= p.out[i].col0) s = i;
    return s;
}
__device__ __forceinline__ LinearOut output_of(const LinearParams &p, int n) {
    LinearOut o = p.out[0];
    if (p.n_outs > 1)
#pragma unroll
        for (int i = 1; i < DR_LINEAR_MAX_OUTS; ++i)
            if (i < p.n_outs && n >= p.out[i].col0) o = p.out[i];
    return o;
}

template <int n>
__device__ __forceinline__ void add_bias(float *v, const float *bias) {   // bias: 16-byte aligned
#pragma unroll
    for (int j = 0; j < n; j += 4) {
        const float4 b = *reinterpret_cast<const float4 *>(bias + j);
        const float2 x = __fadd2_rn(make_float2(v[j], v[j + 1]), make_float2(b.x, b.y)),
                     y = __fadd2_rn(make_float2(v[j + 2], v[j + 3]), make_float2(b.z, b.w));
        v[j] = x.x;
        v[j + 1] = x.y;
        v[j + 2] = y.x;
        v[j + 3] = y.y;
    }
}

// kN columns of a row as they lie in memory.
template <bool kF32, int kN>
union Columns {
    static constexpr int kWords = kF32 ? kN : kN / 2;   // of 32 bits
    using Piece = typename std::conditional<kWords % 4 == 0, uint4, uint2>::type;
    static constexpr int kPieces = kWords * 4 / (int)sizeof(Piece);
    Piece piece[kPieces];
    uint32_t w[kWords];
};
// The residual of columns n .. n + kN - 1 of token t, where there is one and N has so many; finish() looks at no other.
template <bool kF32, int kN>
__device__ __forceinline__ void load_residual(const LinearParams &p, int t, int n, Columns<kF32, kN> &r) {
    using C = Columns<kF32, kN>;
    if (!p.residual || p.N - n < kN) return;
    const typename C::Piece *from = reinterpret_cast<const typename C::Piece *>(
        static_cast<const uint8_t *>(p.residual) + ((int64_t)t * p.res_stride + n) * (kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) r.piece[i] = from[i];
}

// kN columns n .. n + kN - 1 (4 or 16, n a multiple of it) of token t: bias (of these columns, fp32), activation, gating and
// residual (r, loaded before) on the sums a (and b, the sums of the rows that are multiplied in), stored to the output that holds
// them.  Columns from N on are left out.
template <bool kF32, int kN>
__device__ __forceinline__ void finish(const LinearParams &p, const float *bias_a, const float *bias_b, int t, int n, float (&a)[kN],
                                       float (&b)[kN], const Columns<kF32, kN> &r) {
    using C = Columns<kF32, kN>;
    const int have = p.N - n;
    if (have <= 0) return;
    if (p.bias) {
        add_bias<kN>(a, bias_a);
        if (p.gated) add_bias<kN>(b, bias_b);
    }
    activate<kN>(a, p.act);
    if (p.gated) {
#pragma unroll
        for (int i = 0; i < kN; ++i) a[i] *= b[i];
    }
    if (p.residual && have >= kN) {
#pragma unroll
        for (int i = 0; i < C::kWords; ++i) {
            if constexpr (kF32) {
                a[i] += __uint_as_float(r.w[i]);
            } else {
                a[2 * i] += bf16_lo(r.w[i]);
                a[2 * i + 1] += bf16_hi(r.w[i]);
            }
        }
    } else if (p.residual) {
        const int64_t res_at = (int64_t)t * p.res_stride + n;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (i < have) {
                if constexpr (kF32) a[i] += static_cast<const float *>(p.residual)[res_at + i];
                else a[i] += __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.residual)[res_at + i] << 16);
            }
    }
    const LinearOut o = output_of(p, n);
    const int64_t at = (int64_t)t * o.stride + (n - o.col0);
    if (have >= kN) {
        C y;
#pragma unroll
        for (int i = 0; i < C::kWords; ++i) {
            if constexpr (kF32) y.w[i] = __float_as_uint(a[i]);
            else y.w[i] = pack2(a[2 * i], a[2 * i + 1]);
        }
        typename C::Piece *to = reinterpret_cast<typename C::Piece *>(static_cast<uint8_t *>(o.ptr) + at * (kF32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) to[i] = y.piece[i];
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (i < have) {
                if constexpr (kF32) static_cast<float *>(o.ptr)[at + i] = a[i];
                else static_cast<uint16_t *>(o.ptr)[at + i] = f32_to_bf16_rn(a[i]);
            }
    }
}

// The same for one column n of eight tokens t .. t+7, the first `have` of them: the lanes of a warp take columns side by side,
// where rows are not of whole 16-byte pieces.
template <bool kF32>
__device__ __forceinline__ void finish_column8(const LinearParams &p, float bias_a, float bias_b, int t, int have, int n, float (&a)[8],
                                               float (&b)[8]) {
    if (n >= p.N) return;
    using T = typename std::conditional<kF32, float, uint16_t>::type;
    float r[8];
    if (p.residual) {
        const T *from = static_cast<const T *>(p.residual) + (int64_t)t * p.res_stride + n;
#pragma unroll
        for (int i = 0; i < 8; ++i, from += p.res_stride)
            if (i < have) {
                if constexpr (kF32) r[i] = *from;
                else r[i] = __uint_as_float((uint32_t)*from << 16);
            }
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] += bias_a;
            b[i] += bias_b;
        }
    }
    activate<8>(a, p.act);
    if (p.gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= b[i];
    }
    const LinearOut o = output_of(p, n);
    T *to = static_cast<T *>(o.ptr) + (int64_t)t * o.stride + (n - o.col0);
    const int64_t stride = o.stride;
#pragma unroll
    for (int i = 0; i < 8; ++i, to += stride) {
        if (p.residual) a[i] += r[i];
        if (i < have) {
            if constexpr (kF32) *to = a[i];
            else *to = f32_to_bf16_rn(a[i]);
        }
    }
}

}  // namespace lin
}  // namespace dr
