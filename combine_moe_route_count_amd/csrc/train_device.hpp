// train_device.hpp - device helpers of the training-side kernels: wave64
// reductions, the total order of f32 values, and lane-units of 8 row elements
// in every row format.
#pragma once

#include "device_common.hpp"
#include "train.hpp"

namespace moe {

// ---------------------------------------------------------------------------
// wave64 reductions (every lane active): DPP row shifts within each 16 lanes,
// then the two row broadcasts; lane 63 holds the result, which is broadcast.
// The order of a sum is fixed by the lane numbers.
// ---------------------------------------------------------------------------
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp(int identity, int x) {
    return __builtin_amdgcn_update_dpp(identity, x, CTRL, ROW_MASK, 0xF, false);
}

template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, T identity, Op op) {
    static_assert(sizeof(T) == 4, "32-bit values");
    const int id = __builtin_bit_cast(int, identity);
#define MOE_DPP_STEP(CTRL, MASK) \
    v = op(v, __builtin_bit_cast(T, dpp<CTRL, MASK>(id, __builtin_bit_cast(int, v))))
    MOE_DPP_STEP(0x111, 0xF);   // row_shr:1
    MOE_DPP_STEP(0x112, 0xF);   // row_shr:2
    MOE_DPP_STEP(0x114, 0xF);   // row_shr:4
    MOE_DPP_STEP(0x118, 0xF);   // row_shr:8
    MOE_DPP_STEP(0x142, 0xA);   // row_bcast:15 into rows 1 and 3
    MOE_DPP_STEP(0x143, 0xC);   // row_bcast:31 into rows 2 and 3
#undef MOE_DPP_STEP
    return readlane(v, kWave - 1);
}

__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, 0.0f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, -__builtin_inff(), [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ int wave_max(int v) {
    return wave_reduce(v, (int)0x80000000, [](int a, int b) { return a > b ? a : b; });
}

// ---------------------------------------------------------------------------
// lane-units: 8 consecutive elements of a row, held as loaded
// ---------------------------------------------------------------------------
template <RowKind KIND>
struct Row8;

template <>
struct Row8<RowKind::Bf16> {
    u32x4 a;
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        a = ld16_stream((const uint16_t*)base + elem);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16lo(a[j]);
            v[2 * j + 1] = bf16hi(a[j]);
        }
    }
};

template <>
struct Row8<RowKind::F32> {
    u32x4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        a = ld16_stream((const float*)base + elem);
        b = ld16_stream((const float*)base + elem + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // through a scalar: a bit cast of a vector element reads element 0
            const uint32_t x = a[j], y = b[j];
            v[j] = __builtin_bit_cast(float, x);
            v[4 + j] = __builtin_bit_cast(float, y);
        }
    }
};

template <>
struct Row8<RowKind::Fp8> {   // e4m3 codes, one byte per element
    u32x2 a;
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        a = ld8_stream((const uint8_t*)base + elem);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            unpack_e4m3x2<false>(a[d], v[4 * d], v[4 * d + 1]);
            unpack_e4m3x2<true>(a[d], v[4 * d + 2], v[4 * d + 3]);
        }
    }
};

template <>
struct Row8<RowKind::Fp4> {   // e2m1 codes, two per byte
    uint32_t a;
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        a = __builtin_nontemporal_load((const uint32_t*)((const uint8_t*)base + elem / 2));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack_e2m1x8(a, v); }
};

constexpr RowKind float_kind(bool f32) { return f32 ? RowKind::F32 : RowKind::Bf16; }

// 8 results as f32 or, rounded to nearest even, bf16; plain write-back stores.
template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t elem, const float (&v)[8]) {
    if constexpr (F32) {
        u32x4 a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __builtin_bit_cast(uint32_t, v[j]);
            b[j] = __builtin_bit_cast(uint32_t, v[4 + j]);
        }
        st16((float*)base + elem, a);
        st16((float*)base + elem + 4, b);
    } else {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        st16((uint16_t*)base + elem, a);
    }
}

inline dim3 capped_grid(int64_t blocks) {
    return dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid));
}

}  // namespace moe
