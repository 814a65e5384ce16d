// The gated block's activations and their slopes in float32.
#pragma once

#include <hip/hip_runtime.h>

#include "muon.h"

namespace muon {
namespace dev {

// 1 / (1 + e^-v) and 1 minus it, each without cancellation: from e = e^-|v| <= 1.
__device__ __forceinline__ void sigmoids(float v, float& s, float& rest) {
    const float e = expf(-fabsf(v)), r = 1.f / (1.f + e);
    s = v < 0.f ? e * r : r;
    rest = v < 0.f ? r : e * r;
}
// P(N < v) of a standard normal: erfc keeps the digits of its lower end
__device__ __forceinline__ float normal_cdf(float v) { return 0.5f * erfcf(v * -0.70710678118654752f); }

template <int ACT>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == MUON_ACT_SILU) {
        float s, rest;
        sigmoids(v, s, rest);
        return v * s;
    } else if constexpr (ACT == MUON_ACT_GELU) {
        return v * normal_cdf(v);
    } else {
        return v <= 0.f ? 0.f : v;                          // (a NaN stays one)
    }
}

// The value and the slope.
template <int ACT>
__device__ __forceinline__ void activate(float v, float& value, float& slope) {
    if constexpr (ACT == MUON_ACT_SILU) {
        float s, rest;
        sigmoids(v, s, rest);
        value = v * s;
        slope = s * (1.f + v * rest);
    } else if constexpr (ACT == MUON_ACT_GELU) {
        const float p = normal_cdf(v);
        value = v * p;
        slope = p + v * (0.3989422804014327f * expf(-0.5f * v * v));
    } else {
        value = v <= 0.f ? 0.f : v;
        slope = v <= 0.f ? 0.f : v > 0.f ? 1.f : v;
    }
}

}  // namespace dev
}  // namespace muon
