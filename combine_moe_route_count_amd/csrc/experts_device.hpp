// experts_device.hpp - device helpers that the kernels of the experts' step share.
#pragma once

#include "device_common.hpp"
#include "experts.hpp"

namespace moe {

struct Act {
    float s, c;   // sigmoid and 1 - sigmoid
};

// A constant that is put into a register where it is used.  The compiler keeps the constants of
// instructions that take no literals (fused multiply-adds, medians) in scalar registers over a
// whole kernel, also those that only an epilogue wants.
__device__ __forceinline__ float constant_here(float c) {
    asm volatile("" : "+v"(c));
    return c;
}

// The constants of sigmoid_of.
struct ExpConstants {
    float log2e = 1.44269502f, log2e_low = 1.92596299e-8f, ln2 = 0.693147182f;
    static __device__ __forceinline__ ExpConstants here() {
        const ExpConstants k;
        return {constant_here(k.log2e), constant_here(k.log2e_low), constant_here(k.ln2)};
    }
};

// With t = exp(-|g|) and r = 1 / (1 + t), {s, 1 - s} is {r, t*r} or, for g < 0, {t*r, r}: no step
// overflows and 1 - s keeps its digits where s is near 1.
__device__ __forceinline__ Act sigmoid_of(float g, ExpConstants k = {}) {
    // exp(-|g|) = 2^(p + q) with p the rounded product -|g| * log2 e and q what it
    // lost, so large |g| keep their digits
    const float a = -fabsf(g);
    const float p = a * k.log2e;
    const float q = __builtin_fmaf(a, k.log2e, -p) + a * k.log2e_low;
    const float e = __builtin_amdgcn_exp2f(p);
    const float t = a < -200.0f ? 0.0f : __builtin_fmaf(e * q, k.ln2, e);
    const float r = __builtin_amdgcn_rcpf(1.0f + t);
    const float tr = t * r;
    return g < 0.0f ? Act{tr, r} : Act{r, tr};
}

__device__ __forceinline__ float silu_of(float g, ExpConstants k = {}) { return g * sigmoid_of(g, k).s; }

}  // namespace moe
