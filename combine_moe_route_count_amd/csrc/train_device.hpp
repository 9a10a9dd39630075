// train_device.hpp - device helpers of the training-side kernels: wave64
// reductions, lane-units of row elements in every row format, and the mapping of
// work items to workgroups.
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
// lane-units: EL consecutive elements of a row, held as loaded.  load goes past
// the caches' replacement order (rows read once), load_cached through it.
// ---------------------------------------------------------------------------
template <bool STREAM>
__device__ __forceinline__ u32x4 get16(const void* p) {
    return STREAM ? ld16_stream(p) : ld16(p);
}
template <bool STREAM>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
    if constexpr (STREAM) st16_stream(p, v);
    else st16(p, v);
}

// f32 or bf16 elements: 16-byte loads, or one 8-byte load of 4 bf16.
template <bool F32, int EL>
struct FloatUnit {
    static_assert(EL == 4 || EL == 8, "4 or 8 elements");
    static constexpr int W = F32 ? EL : EL / 2;   // words
    uint32_t w[W];
    template <bool STREAM>
    __device__ __forceinline__ void load_as(const void* base, int64_t elem) {
        const char* p = (const char*)base + elem * (F32 ? 4 : 2);
        if constexpr (W == 2) {
            const u32x2 a = STREAM ? ld8_stream(p) : *(const u32x2*)p;
            w[0] = a[0];
            w[1] = a[1];
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const u32x4 a = get16<STREAM>(p + 16 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * i + j] = a[j];
            }
        }
    }
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        load_as<true>(base, elem);
    }
    __device__ __forceinline__ void load_cached(const void* base, int64_t elem) {
        load_as<false>(base, elem);
    }
    __device__ __forceinline__ void get(float (&v)[EL]) const {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (F32) {
                v[i] = __builtin_bit_cast(float, w[i]);
            } else {
                v[2 * i] = bf16lo(w[i]);
                v[2 * i + 1] = bf16hi(w[i]);
            }
        }
    }
};

// 8 elements in any row format.
template <RowKind KIND>
struct Row8;
template <>
struct Row8<RowKind::Bf16> : FloatUnit<false, 8> {};
template <>
struct Row8<RowKind::F32> : FloatUnit<true, 8> {};

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

// EL results as f32 or, rounded to nearest even, bf16.
template <bool F32, bool STREAM, int EL>
__device__ __forceinline__ void store_unit(void* base, int64_t elem, const float (&v)[EL]) {
    static_assert(EL == 4 || EL == 8, "4 or 8 elements");
    if constexpr (F32) {
#pragma unroll
        for (int h = 0; h < EL / 4; ++h) {
            u32x4 a;
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = __builtin_bit_cast(uint32_t, v[4 * h + j]);
            put16<STREAM>((float*)base + elem + 4 * h, a);
        }
    } else if constexpr (EL == 8) {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        put16<STREAM>((uint16_t*)base + elem, a);
    } else {
        const u32x2 a = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        u32x2* p = (u32x2*)((uint16_t*)base + elem);
        if constexpr (STREAM) __builtin_nontemporal_store(a, p);
        else *p = a;
    }
}

// Work item i of n groups of `parts` items -> (group, part).  Workgroups go to the 8
// XCDs round-robin, so in each block of 8 groups the items are laid out part-major:
// the parts of one group run on one XCD and share what they read in its L2.
constexpr int kXcdCount = 8;
__device__ __forceinline__ void xcd_item(int64_t i, int64_t n, int parts, int64_t& group,
                                         int& part) {
    const int64_t grouped = n / kXcdCount * kXcdCount * parts;
    if (i < grouped) {
        const int64_t block = (int64_t)kXcdCount * parts;
        const int64_t b = i / block, r = i - b * block;
        part = (int)(r / kXcdCount);
        group = b * kXcdCount + (r - (int64_t)part * kXcdCount);
    } else {
        group = i / parts;
        part = (int)(i - group * parts);
    }
}

// Threads for rows of `units` lane-units: the fewest passes of at most `most`
// threads, evenly filled waves.
inline int row_threads(int64_t units, int most) {
    const int64_t passes = (units + most - 1) / most;
    const int64_t per = (units + passes - 1) / passes;
    return (int)((per + kWave - 1) / kWave * kWave);
}

inline dim3 capped_grid(int64_t blocks) {
    return dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid));
}

}  // namespace moe
