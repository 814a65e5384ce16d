// The gated block's activations and their slopes in float32.
//
// Results go to bfloat16 (half steps of 2^-8), so the hardware's exponential and reciprocal serve: with u = 2^-24, silu is within
// (1.5 |v| + 8) u of itself and gelu within (1.25 v^2 + 20) u, which is where the exponent's argument is rounded; e^x is kept
// below 2^-126 too.  The library's expf, division and erfcf are 40 to 120 instructions a value, and a lane has 64 values of
// a 256 x 128 tile of the gated block.
#pragma once

#include <hip/hip_runtime.h>

#include "muon.h"

namespace muon {
namespace dev {

// e^x for x <= 0 as value * factor: the instruction gives 0 for what is below 2^-126, so 2^-64 is taken out there.
struct Small {
    float value, factor;
    __device__ __forceinline__ float get() const { return value * factor; }
};
__device__ __forceinline__ Small exp_below(float x) {
    const float t = x * 1.44269504088896341f;
    const bool tiny = t < -100.f;
    return {__builtin_amdgcn_exp2f(tiny ? t + 64.f : t), tiny ? 0x1p-64f : 1.f};
}

// P(N < -a) / e^(-a^2 / 2) of a standard normal for a >= 0: a polynomial in 1 / (1 + 0.31 a) without a constant term, fitted here for
// the least relative error on [0, 20] (1.9e-7; in float32, with the reciprocal off by one in its last place, within 10 times 2^-24).
__device__ __forceinline__ float normal_tail(float a) {
    const float t = __builtin_amdgcn_rcpf(1.f + 0.31f * a);
    float s = 0.0359174907f;
    s = fmaf(s, t, -0.141937152f);
    s = fmaf(s, t, 0.155674309f);
    s = fmaf(s, t, -0.0154968156f);
    s = fmaf(s, t, 0.110445343f);
    s = fmaf(s, t, 0.107662246f);
    s = fmaf(s, t, 0.124079071f);
    s = fmaf(s, t, 0.123655602f);
    return s * t;
}

// The value and the slope of act(v); what is not used costs nothing.
template <int ACT>
__device__ __forceinline__ void activate(float v, float& value, float& slope) {
    if constexpr (ACT == MUON_ACT_RELU) {
        value = v <= 0.f ? 0.f : v;                        // (a NaN stays one)
        slope = v <= 0.f ? 0.f : v > 0.f ? 1.f : v;
        return;
    }
    const bool below = v < 0.f;
    if constexpr (ACT == MUON_ACT_SILU) {
        // s = 1 / (1 + e^-v) and 1 - s, each from e = e^-|v| without cancellation
        const Small e = exp_below(-fabsf(v));
        const float r = __builtin_amdgcn_rcpf(1.f + e.get());
        const float s = below ? e.get() * r : r, rest = below ? r : e.get() * r;
        value = v * r * (below ? e.value : 1.f) * (below ? e.factor : 1.f);
        slope = s * (1.f + v * rest);
    } else {
        const float a = fabsf(v);
        const Small e = exp_below(-0.5f * a * a);
        const float tail = normal_tail(a), p = e.get() * tail;
        value = below ? v * tail * e.value * e.factor : v * (1.f - p);
        slope = (below ? p : 1.f - p) + v * (0.3989422804014327f * e.get());
    }
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
    float value, slope;
    activate<ACT>(v, value, slope);
    return value;
}

}  // namespace dev
}  // namespace muon
