// experts_device.hpp - device helpers that the kernels of the experts' step share.
#pragma once

#include "device_common.hpp"
#include "experts.hpp"

namespace moe {

struct Act {
    float s, c;   // sigmoid and 1 - sigmoid
};

// With t = exp(-|g|) and r = 1 / (1 + t), {s, 1 - s} is {r, t*r} or, for g < 0, {t*r, r}: no step
// overflows and 1 - s keeps its digits where s is near 1.
__device__ __forceinline__ Act sigmoid_of(float g) {
    // exp(-|g|) = 2^(p + q) with p the rounded product -|g| * log2 e and q what it
    // lost, so large |g| keep their digits
    const float a = -fabsf(g);
    constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f;
    const float p = a * kLog2e;
    const float q = __builtin_fmaf(a, kLog2e, -p) + a * kLog2eLow;
    const float e = __builtin_amdgcn_exp2f(p);
    const float t = a < -200.0f ? 0.0f : __builtin_fmaf(e * q, 0.693147182f, e);
    const float r = __builtin_amdgcn_rcpf(1.0f + t);
    const float tr = t * r;
    return g < 0.0f ? Act{tr, r} : Act{r, tr};
}

__device__ __forceinline__ float silu_of(float g) { return g * sigmoid_of(g).s; }

}  // namespace moe
