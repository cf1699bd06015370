// Score and packing helpers shared by the prompt-side attention kernels.
#pragma once

#include "dr_device.cuh"

namespace dr {

// Score cap: s -> cap tanh(u) in log2 units, u = raw c2, c2 = scale / cap.  Two forms, chosen per score:
//   |u| <= 1/2  (raw scale log2 e) P(u^2), P of degree 4, tanh(u) / u to 2^-26 of its value (fitted to the relative error
//               by reweighted least squares, Lawson's method): the uncapped score times a factor near 1
//   beyond      c1 - 2 c1 / (2^(u 2 log2 e) + 1), c1 = cap log2 e
// fp32 stays within 2^-21 of the value of either.  The second alone is off by 2^-22 of the cap whatever the score: at a cap of
// 1e6 by a quarter, and from 1e8 on all scores came out equal.  Infinite scores give the cap, NaN stays NaN.
struct ScoreCap {
    float c1, c2, scale;   // scale: of uncapped scores, scale log2 e
    float small;           // raw scores of the first form
    __device__ __forceinline__ ScoreCap(float c1_, float c2_, float scale_)
        : c1(c1_), c2(fminf(c2_, 3e38f)), scale(scale_), small(0.5f / c2) {}   // finite: a score of 0 stays 0
    __device__ __forceinline__ float2 near(float2 raw) const {
        const auto two = [](float v) { return make_float2(v, v); };
        const float2 u = __fmul2_rn(raw, two(c2)), t = __fmul2_rn(u, u);
        float2 f = __ffma2_rn(t, two(0.0171350781f), two(-0.0529861152f));
        f = __ffma2_rn(f, t, two(0.133247808f));
        f = __ffma2_rn(f, t, two(-0.333330691f));
        f = __ffma2_rn(f, t, two(1.0f));
        return __fmul2_rn(__fmul2_rn(raw, two(scale)), f);
    }
    __device__ __forceinline__ float far(float raw) const {
        return c1 - __fdividef(2.0f * c1, fast_exp2(raw * (2.8853900818f * c2)) + 1.0f);
    }
    // N scores of a thread, by the whole warp: where all of the warp's are of the first form (the usual case) the second is
    // skipped.
    template <int N>
    __device__ __forceinline__ void operator()(float (&s)[N]) const {
        float top[4] = {0.f, 0.f, 0.f, 0.f};   // four chains
#pragma unroll
        for (int c = 0; c < N; ++c) top[c & 3] = fmaxf(top[c & 3], fabsf(s[c]));
        if (__all_sync(0xFFFFFFFFu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) <= small)) {
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 x = near(make_float2(s[c], s[c + 1]));
                s[c] = x.x;
                s[c + 1] = x.y;
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 x = near(make_float2(s[c], s[c + 1]));
                s[c] = fabsf(s[c]) > small ? far(s[c]) : x.x;
                s[c + 1] = fabsf(s[c + 1]) > small ? far(s[c + 1]) : x.y;
            }
        }
    }
};

// The running maximum of a row moves when a score passes it by 2^8 (log2 units): sums are rescaled rarely.
constexpr float kSlack = 8.0f;
// f16 weights are held 2^7 times as large as their ratio to the running maximum: below 2^15, and with steps of 2^-32 of the
// row's largest at least, where 2^-25 would lose thousands of small weights whose sum counts.  (bf16 holds any ratio.)
template <bool kF16>
constexpr float kLift = kF16 ? 7.0f : 0.0f;

// The maximum to store with a softmax state.  m = -inf marks a state without keys, and the maxima drop NaN: a state whose
// scores were all NaN (its sum l is NaN) gets a maximum that no merge takes for an empty one.
__device__ __forceinline__ float state_max(float m, float l) { return m == -INFINITY && l != 0.f ? 0.f : m; }

// The power of two that brings x into [2^14, 2^15), the upper end of f16; 1 for zero, infinite and NaN x.  Exponents are kept where both the
// factor and its reciprocal are normal numbers.
__device__ __forceinline__ float pow2_normaliser(float x) {
    const int e = (int)(__float_as_uint(x) >> 23) & 0xFF;   // x >= 0
    if (x == 0.f || e == 255) return 1.0f;
    const int f = min(max(268 - e, 2), 252);               // 2^(141 - e) has the exponent field 268 - e
    return __uint_as_float((uint32_t)f << 23);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four e4m3 codes -> two f16x2, exact.
__device__ __forceinline__ void codes4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

}  // namespace dr
