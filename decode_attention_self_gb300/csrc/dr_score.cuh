// Score and packing helpers shared by the prompt-side attention kernels.
#pragma once

#include "dr_device.cuh"

namespace dr {

// cap * tanh(raw * scale / cap) in log2 units, c1 = cap log2 e, c2 = 2 log2 e scale / cap:
// tanh y = 1 - 2 / (2^(2 y log2 e) + 1), whose absolute error stays near 2^-23 for every y (the hardware's own tanh
// is off by 2^-11 of its value, which a cap of 50 would turn into 3% of a weight).
__device__ __forceinline__ float capped_score(float raw, float c1, float c2) {
    return c1 - __fdividef(2.0f * c1, fast_exp2(raw * c2) + 1.0f);
}

// The maximum to store with a softmax state.  m = -inf marks a state without keys, and the maxima drop NaN: a state whose
// scores were all NaN (its sum l is NaN) gets a maximum that no merge takes for an empty one.
__device__ __forceinline__ float state_max(float m, float l) { return m == -INFINITY && l != 0.f ? 0.f : m; }

// The power of two that brings x into [0.5, 1); 1 for zero, infinite and NaN x.  Exponents are kept where both the
// factor and its reciprocal are normal numbers.
__device__ __forceinline__ float pow2_normaliser(float x) {
    const int e = (int)(__float_as_uint(x) >> 23) & 0xFF;   // x >= 0
    if (x == 0.f || e == 255) return 1.0f;
    const int f = min(max(253 - e, 2), 252);               // 2^(126 - e) has the exponent field 253 - e
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
