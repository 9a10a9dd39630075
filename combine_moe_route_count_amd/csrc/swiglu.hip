// swiglu.hip - the activation between an expert's two products, and its gradient from
// what the forward pass kept.
//
// A row of gu holds I gate values g and then I up values u:
//   h = silu(g) * u,  silu(g) = g * s,  s = 1 / (1 + exp(-g))
//   dg = dh * u * s * (1 + g * (1 - s)),  du = dh * silu(g)
//
// The 8-bit checkpoint of gu: e4m3 codes, one f32 scale per 128 elements of a row, the
// smallest power of two that keeps the block's largest finite magnitude within 448.
// Dividing by it is exact, so a kept value is off by one e4m3 rounding and no more.
// (The dispatch's pack keeps scale 1 for small blocks; activations of a layer are
// small, and there a scale that follows them saves up to 8 bits of range.)
//
// Both kernels are one pass over the rows, 8 elements of g and the same of u per lane (4
// where the output is f32, so that a store is 16 bytes a lane and a wave's whole lines),
// HBM bound: 65536 x 2 x 2048 bf16 with the checkpoint 167 us, 6.5 TB/s; the gradient of the
// same from the checkpoint, with h, 242 us, 4.9 TB/s; 16384 x 2 x 2048 f32 gradient 139 us.
// With 8 f32 elements a lane (two stores to a lane, each half of every line) that one took
// 157.  A workgroup is a power of two of lanes along a row times rows of it, so short rows
// share one; rows outside every segment are neither read nor written.
#include <type_traits>

#include "train_device.hpp"
#include "experts_device.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

// Whether a segment owns row r: the last expert e whose segment starts at or before r
// has r - off[e] < cnt[e].
__device__ __forceinline__ bool row_owned(const int32_t* cnt, const int32_t* off, int E,
                                          int64_t r) {
    int lo = 0, n = E;       // off[lo .. lo + n) are to be looked at
    while (n > 1) {
        const int half = n / 2;
        if (off[lo + half] <= r) lo += half;
        n -= half;
    }
    const int64_t slot = r - off[lo];
    return slot >= 0 && slot < cnt[lo];
}

// Max over each aligned group of LANES lanes, 16 or 32.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#define MOE_MAX_STEP(CTRL)                                                                     \
    {                                                                                          \
        const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);   \
        v = v > o ? v : o;                                                                     \
    }
    MOE_MAX_STEP(0xB1)    // lane ^ 1
    MOE_MAX_STEP(0x4E)    // lane ^ 2
    MOE_MAX_STEP(0x141)   // mirrored within 8 lanes
    MOE_MAX_STEP(0x140)   // mirrored within 16 lanes
#undef MOE_MAX_STEP
    if constexpr (LANES == 32) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, 16);
        v = v > o ? v : o;
    }
    return v;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// EL elements of a row of any kind, as f32.
template <RowKind KIND, int EL>
struct Elems {
    std::conditional_t<KIND == RowKind::Fp8, std::conditional_t<EL == 8, Row8<RowKind::Fp8>, uint32_t>,
                       FloatUnit<KIND == RowKind::F32, EL>> u;
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        if constexpr (KIND == RowKind::Fp8 && EL == 4)
            u = __builtin_nontemporal_load((const uint32_t*)((const uint8_t*)base + elem));
        else
            u.load(base, elem);
    }
    __device__ __forceinline__ void get(float (&v)[EL]) const {
        if constexpr (KIND == RowKind::Fp8 && EL == 4) {
            unpack_e4m3x2<false>(u, v[0], v[1]);
            unpack_e4m3x2<true>(u, v[2], v[3]);
        } else {
            u.get(v);
        }
    }
};

// The e4m3 codes of the calling lane's EL values and the scale of its block of 128 / EL
// lanes.  As in the dispatch's pack: infinities saturate, a NaN gets the NaN code with its
// sign.
template <int EL>
__device__ __forceinline__ void checkpoint(const float (&v)[EL], uint32_t (&codes)[EL / 4], float& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < EL; ++j) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu;
        m = m > b ? m : b;
    }
    const bool odd = m >= kInfBits;
    if (odd) {
        m = 0;
#pragma unroll
        for (int j = 0; j < EL; ++j) {
            const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu;
            if (b < kInfBits) m = m > b ? m : b;
        }
    }
    m = group_max<kFp8Block / EL>(m);
    // 448 = 1.75 * 2^8: the exponent of amax, one more past 1.75, less 8; 2^-126 at the least
    const int e = (int)((m + 0x1fffffu) >> 23) - 8;
    const uint32_t se = m == 0 ? 127u : (uint32_t)(e > 1 ? e : 1);
    scale = __builtin_bit_cast(float, se << 23);
    const float inv = __builtin_bit_cast(float, (254u - se) << 23);
    float q[EL];
#pragma unroll
    for (int j = 0; j < EL; ++j) q[j] = v[j] * inv;
    if (odd) {
#pragma unroll
        for (int j = 0; j < EL; ++j)
            if (__builtin_isinf(q[j])) q[j] = __builtin_copysignf(kE4m3Max, q[j]);
    }
#pragma unroll
    for (int i = 0; i < EL / 4; ++i)
        codes[i] = pack_e4m3x4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    if (odd) {
#pragma unroll
        for (int j = 0; j < EL; ++j) {
            const uint32_t b = __builtin_bit_cast(uint32_t, v[j]);
            if ((b & 0x7fffffffu) <= kInfBits) continue;
            const int at = (j & 3) * 8;
            codes[j >> 2] = (codes[j >> 2] & ~(0xffu << at)) | ((0x7fu | (b >> 24 & 0x80u)) << at);
        }
    }
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&c)[N]) {
    if constexpr (N == 2) __builtin_nontemporal_store(u32x2{c[0], c[1]}, (u32x2*)p);
    else __builtin_nontemporal_store(c[0], (uint32_t*)p);
}

constexpr int elems_of(bool out_f32) { return out_f32 ? 4 : 8; }

// Where a thread works: rows first + ty, in steps, and units tx, tx + width, ...
struct Place {
    int width;     // lanes along a row (a power of two, at least 16)
    int64_t row, row_step;
    int unit;
};

__device__ __forceinline__ Place place(int log_width) {
    Place p;
    p.width = 1 << log_width;
    const int per = kThreads >> log_width;
    p.row = (int64_t)blockIdx.x * per + (threadIdx.x >> log_width);
    p.row_step = (int64_t)gridDim.x * per;
    p.unit = (int)(threadIdx.x & (p.width - 1));
    return p;
}

template <bool F32, bool HF32>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(SwigluArgs a, int log_width) {
    constexpr int EL = elems_of(HF32), kLanes = kFp8Block / EL;
    constexpr RowKind KIND = F32 ? RowKind::F32 : RowKind::Bf16;
    const Place p = place(log_width);
    const int units = (int)(a.I / EL);
    for (int64_t r = p.row; r < a.rows; r += p.row_step) {
        if (a.packed_cnt && !row_owned(a.packed_cnt, a.packed_off, a.E, r)) continue;
        for (int u = p.unit; u < units; u += p.width) {
            const int64_t col = (int64_t)u * EL;
            Elems<KIND, EL> gin, uin;
            gin.load(a.gu, r * 2 * a.I + col);
            uin.load(a.gu, r * 2 * a.I + a.I + col);
            float g[EL], up[EL], h[EL];
            gin.get(g);
            uin.get(up);
            if (a.codes) {   // I % 128 == 0 here: all lanes of a block take this together
                uint32_t cg[EL / 4], cu[EL / 4];
                float sg, su;
                checkpoint<EL>(g, cg, sg);
                checkpoint<EL>(up, cu, su);
                uint8_t* at = a.codes + r * 2 * a.I + col;
                store_codes(at, cg);
                store_codes(at + a.I, cu);
                if (u % kLanes == 0) {
                    float* sc = a.scales + r * (a.I / 64) + u / kLanes;
                    sc[0] = sg;
                    sc[a.I / kFp8Block] = su;
                }
            }
#pragma unroll
            for (int j = 0; j < EL; ++j) h[j] = silu_of(g[j]) * up[j];
            store_unit<HF32, true>(a.h, r * a.I + col, h);
        }
    }
}

template <RowKind KIND, bool DF32, bool OF32>
__global__ __launch_bounds__(kThreads) void swiglu_grad_kernel(SwigluGradArgs a, int log_width) {
    constexpr int EL = elems_of(OF32), kLanes = kFp8Block / EL;
    const Place p = place(log_width);
    const int units = (int)(a.I / EL);
    for (int64_t r = p.row; r < a.rows; r += p.row_step) {
        if (a.packed_cnt && !row_owned(a.packed_cnt, a.packed_off, a.E, r)) continue;
        for (int u = p.unit; u < units; u += p.width) {
            const int64_t col = (int64_t)u * EL, at = r * 2 * a.I + col;
            Elems<KIND, EL> gin, uin;
            FloatUnit<DF32, EL> din;
            float sg = 1.0f, su = 1.0f;
            gin.load(a.gu, at);
            uin.load(a.gu, at + a.I);
            din.load(a.dh, r * a.I + col);
            if constexpr (KIND == RowKind::Fp8) {
                const float* sc = a.scales + r * (a.I / 64) + u / kLanes;
                sg = sc[0];
                su = sc[a.I / kFp8Block];
            }
            float g[EL], up[EL], d[EL], h[EL];
            gin.get(g);
            uin.get(up);
            din.get(d);
#pragma unroll
            for (int j = 0; j < EL; ++j) {
                if constexpr (KIND == RowKind::Fp8) {
                    g[j] *= sg;
                    up[j] *= su;
                }
                const Act s = sigmoid_of(g[j]);
                const float act = g[j] * s.s;
                h[j] = act * up[j];
                g[j] = d[j] * up[j] * (s.s * (1.0f + g[j] * s.c));
                up[j] = d[j] * act;
            }
            store_unit<OF32, true>(a.dgu, at, g);
            store_unit<OF32, true>(a.dgu, at + a.I, up);
            if (a.h) store_unit<OF32, true>(a.h, r * a.I + col, h);
        }
    }
}

// Lanes along a row: the smallest power of two that covers its units, at least a block of
// the checkpoint, within a workgroup.  Lanes that leave fewer idle, but take turns on a row,
// were slower: 13796 rows of 1280 bf16 48.4 -> 51.2 us, their gradient 35.2 -> 41.0.
inline int log_width_of(int64_t I, bool out_f32) {
    int l = out_f32 ? 5 : 4;
    while (l < 8 && ((int64_t)elems_of(out_f32) << l) < I) ++l;
    return l;
}

inline dim3 rows_grid(int64_t rows, int log_width) {
    const int64_t per = kThreads >> log_width;
    return capped_grid((rows + per - 1) / per);
}

template <RowKind KIND, bool DF32>
void launch_grad(const SwigluGradArgs& a, hipStream_t s) {
    const int l = log_width_of(a.I, a.out_f32);
    const dim3 grid = rows_grid(a.rows, l);
    if (a.out_f32) swiglu_grad_kernel<KIND, DF32, true><<<grid, kThreads, 0, s>>>(a, l);
    else swiglu_grad_kernel<KIND, DF32, false><<<grid, kThreads, 0, s>>>(a, l);
}

template <RowKind KIND>
void launch_grad(const SwigluGradArgs& a, hipStream_t s) {
    if (a.dh_f32) launch_grad<KIND, true>(a, s);
    else launch_grad<KIND, false>(a, s);
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const int l = log_width_of(a.I, a.h_f32);
    const dim3 grid = rows_grid(a.rows, l);
    if (a.gu_f32) {
        if (a.h_f32) swiglu_kernel<true, true><<<grid, kThreads, 0, s>>>(a, l);
        else swiglu_kernel<true, false><<<grid, kThreads, 0, s>>>(a, l);
    } else {
        if (a.h_f32) swiglu_kernel<false, true><<<grid, kThreads, 0, s>>>(a, l);
        else swiglu_kernel<false, false><<<grid, kThreads, 0, s>>>(a, l);
    }
    return hipGetLastError();
}

hipError_t launch_swiglu_grad(const SwigluGradArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    switch (a.gu_kind) {
        case RowKind::F32: launch_grad<RowKind::F32>(a, s); break;
        case RowKind::Fp8: launch_grad<RowKind::Fp8>(a, s); break;
        default: launch_grad<RowKind::Bf16>(a, s); break;
    }
    return hipGetLastError();
}

}  // namespace moe
