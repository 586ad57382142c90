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

// A NaN stays a NaN in every branch (the marker of a wait that gave up must not be lost).
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case 1: return z < 0.f ? 0.f : z;
        case 2: return z / (1.f + expf(-z));
        // z (1 + erf(z / sqrt 2)) / 2 by the complementary function: no cancellation for z < 0
        case 3: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u), 2 sqrt(2 / pi) = 1.5957691
        case 4: return z / (1.f + expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)));
        default: return z;
    }
}

// Read through L2: the residual may be the output buffer, which the kernel also writes.
__device__ __forceinline__ float epilogue_value(float v, const Epilogue &e, int64_t m, int64_t n, int64_t N) {
    if (e.bias) v += half_bits_to_float(__ldcg(e.bias + n));
    v = activate(v, e.act);
    if (e.residual) v += half_bits_to_float(__ldcg(e.residual + m * N + n));
    return v;
}

}  // namespace bonsai
