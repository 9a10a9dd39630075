// experts_device.hpp - device helpers that the kernels of the experts' step share.
#pragma once

#include "device_common.hpp"
#include "experts.hpp"

namespace moe {

// Ored to an offset below 2^31 it leaves every descriptor's range (2^31 at the most).
__device__ __forceinline__ uint32_t outside_if(bool b) { return (uint32_t)b << 31; }

// A buffer of `rows` rows from `row` on: loads from behind the last one give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, int64_t row, int64_t rows,
                                                          int64_t row_bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((char*)base + row * row_bytes, 0,
                                             (int)(uint32_t)(rows * row_bytes), kRsrcWord3);
}

// All but the last FLYING loads of every wave have landed, and every wave's LDS reads are in
// registers.  The empty asm keeps the compiler from moving memory accesses over the barrier.
template <int FLYING>
__device__ __forceinline__ void stage_sync() {
    static_assert(FLYING < 64, "vmcnt");
    asm volatile("" ::: "memory");
    // simm16 of s_waitcnt: vmcnt in bits 3:0 and 15:14, expcnt 6:4 (none), lgkmcnt 11:8 (0)
    __builtin_amdgcn_s_waitcnt((FLYING & 15) | (FLYING >> 4) << 14 | 0x70);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

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
