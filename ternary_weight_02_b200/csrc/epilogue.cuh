// epilogue.cuh -- bias, activation and residual on the FP32 sums of a ternary product
// (bonsai_ternary_linear_epilogue): y = act(sum + bias[n]) + residual[m][n], one rounding
// to FP16 at the end.  Every kernel's store goes through epilogue_value when its Epilogue
// is in use.
#pragma once

#include "common.cuh"

namespace bonsai {

// bias (N) and residual (M x N) may be null; residual may be the output itself, each element
// then being read by the thread that writes it.
struct Epilogue {
    const uint16_t *bias = nullptr;
    const uint16_t *residual = nullptr;
    int act = 0;  // bonsai_act
};

// 2^x and 1 / x by the special function unit, relative errors of 2^-22 and 2^-23; a prefill tile's
// epilogue feels every instruction of the exact forms around them.
__device__ __forceinline__ float exp2_unit(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_unit(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2E = 1.4426950408889634f;

// z / (1 + e^-w) for w' = -w log2 e
__device__ __forceinline__ float times_sigmoid(float z, float w2) { return z * rcp_unit(1.f + exp2_unit(w2)); }

// z (1 + erf(z / sqrt 2)) / 2 with the rational approximation 7.1.26 of Abramowitz and Stegun,
// Handbook of Mathematical Functions, for the complementary function of x = |z| / sqrt 2 (its
// five coefficients halved): an absolute error of 1.5e-7, no cancellation for z < 0.
__device__ __forceinline__ float gelu_erf(float z) {
    const float t = rcp_unit(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
    float c = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
    c = fmaf(c, t, 0.5f * 1.421413741f);
    c = fmaf(c, t, 0.5f * -0.284496736f);
    c = fmaf(c, t, 0.5f * 0.254829592f);
    const float h = z * (c * t * exp2_unit(z * z * (-0.5f * kLog2E)));  // z erfc(x) / 2
    return z < 0.f ? h : z - (z < INFINITY ? h : 0.f);  // (at +infinity h is infinity times 0)
}

// A NaN stays a NaN in every branch (the marker of a wait that gave up must not be lost).
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case 1: return z < 0.f ? 0.f : z;
        case 2: return times_sigmoid(z, -kLog2E * z);
        case 3: return gelu_erf(z);
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u), 2 sqrt(2 / pi) = 1.5957691
        case 4: return times_sigmoid(z, (-kLog2E * 1.5957691216057308f) * fmaf(0.044715f * z * z, z, z));
        default: return z;
    }
}

// Bias and residual of one output, read ahead of its sum (a load behind the store of another
// output would wait for it: the residual may be the output buffer, so the two are not
// reordered; through the L2 for the same reason).
struct EpilogueTerms {
    float bias = 0.f, residual = 0.f;
};
__device__ __forceinline__ EpilogueTerms epilogue_terms(const Epilogue &e, int64_t m, int64_t n, int64_t N) {
    EpilogueTerms t;
    if (e.bias) t.bias = half_bits_to_float(__ldcg(e.bias + n));
    if (e.residual) t.residual = half_bits_to_float(__ldcg(e.residual + m * N + n));
    return t;
}
__device__ __forceinline__ float epilogue_value(float v, const Epilogue &e, const EpilogueTerms &t) {
    if (e.bias) v += t.bias;
    v = activate(v, e.act);
    return e.residual ? v + t.residual : v;  // (a -0 stays one without a residual)
}

}  // namespace bonsai
