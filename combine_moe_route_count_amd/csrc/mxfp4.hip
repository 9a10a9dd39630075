// mxfp4.hip - rows to and from MXFP4: blocks of 32 consecutive elements as e2m1
// codes with one e8m0 scale, the exponent of a power of two.
//
// With amax the largest finite magnitude of a block, its scale 2^e is the one with
// amax / 2^e in [3.5, 7): the largest code value is 6, and 7 is where a value would
// round away from 6 if the codes went on to 8, so saturating at 6 never moves a value
// further than rounding does.  Codes are x / 2^e rounded to nearest even; the quotient
// is exact, so that is the one rounding.
//
// Rows have no gaps and blocks do not cross rows, so both kernels run over one flat
// array, one pass, HBM bound.  Quantizing, a lane holds 8 elements (4 lanes a block) and
// kUnits such units: 32768 x 7168 f32 take 193 us, 5.5 TB/s.  Dequantizing, it makes 16
// bytes at a time: with 32 (8 f32 elements, two stores to a lane, each half of every line
// past the caches) the same rows took 364 us, now 158 to 170, 6.3 to 6.7 TB/s.
#include <type_traits>

#include "train_device.hpp"
#include "experts.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;   // units of 8 elements per lane, loaded together

// Max over each aligned group of 4 lanes.
__device__ __forceinline__ uint32_t group4_max(uint32_t v) {
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
    return v > o ? v : o;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// The codes of the calling lane's 8 values and the scale byte of its block.
__device__ __forceinline__ void mxfp4_pack8(float (&v)[8], uint32_t& codes, uint32_t& scale) {
    // magnitudes of floats order as their bit patterns
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu;
        m = m > b ? m : b;
    }
    if (m >= kInfBits) {   // over the finite values, unless there is a NaN
        uint32_t f = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu;
            if (b != kInfBits) f = f > b ? f : b;
        }
        m = f;
    }
    m = group4_max(m);
    if (m > kInfBits) {    // a NaN: e2m1 has no code for it, e8m0 has
        codes = 0;
        scale = 0xff;
        return;
    }
    // the exponent of amax, one more from 1.75 on, less 2; 2^-127 at the least
    const int e = (int)((m + 0x200000u) >> 23) - 2;
    scale = m == 0 ? 127u : (uint32_t)(e > 0 ? e : 0);
    const float inv = __builtin_bit_cast(float, (254u - scale) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_fmed3f(v[j] * inv, -kE2m1Max, kE2m1Max);
    codes = pack_e2m1x8(v);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const void* x, int64_t units,
                                                                  uint32_t* codes,
                                                                  uint8_t* scales) {
    constexpr int64_t kStep = kThreads * kUnits;
    for (int64_t base = (int64_t)blockIdx.x * kStep; base < units; base += gridDim.x * kStep) {
        FloatUnit<F32, 8> in[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int64_t u = base + i * kThreads + threadIdx.x;
            if (u < units) in[i].load(x, u * 8);
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            // units is a multiple of 4: the lanes of a block are all inside or all outside
            const int64_t u = base + i * kThreads + threadIdx.x;
            if (u >= units) continue;
            float v[8];
            in[i].get(v);
            uint32_t c, s;
            mxfp4_pack8(v, c, s);
            codes[u] = c;
            if (threadIdx.x % 4 == 0) scales[u / 4] = (uint8_t)s;
        }
    }
}

// The value of a scale byte: 2^(s-127), a subnormal at 0; 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    const uint32_t b = s == 0 ? 0x00400000u : s << 23;
    return __builtin_bit_cast(float, s == 0xff ? 0x7fc00000u : b);
}

// 16 bytes of output per lane: a wave's store covers whole lines.
template <bool F32>
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_kernel(const uint8_t* codes,
                                                                    const uint8_t* scales,
                                                                    int64_t units, void* y) {
    constexpr int EL = F32 ? 4 : 8;
    using Word = std::conditional_t<F32, uint16_t, uint32_t>;
    constexpr int64_t kStep = kThreads * kUnits;
    for (int64_t base = (int64_t)blockIdx.x * kStep; base < units; base += gridDim.x * kStep) {
        uint32_t c[kUnits], s[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int64_t u = base + i * kThreads + threadIdx.x;
            if (u < units) {
                c[i] = __builtin_nontemporal_load((const Word*)codes + u);
                s[i] = scales[u / (kMxBlock / EL)];
            }
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int64_t u = base + i * kThreads + threadIdx.x;
            if (u >= units) continue;
            float v[8], o[EL];
            unpack_e2m1x8(c[i], v);
            const float scale = e8m0_value(s[i]);
#pragma unroll
            for (int j = 0; j < EL; ++j) o[j] = v[j] * scale;
            store_unit<F32, true>(y, u * EL, o);
        }
    }
}

inline dim3 flat_grid(int64_t units) {
    return capped_grid((units + kThreads * kUnits - 1) / (kThreads * kUnits));
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, bool f32, int64_t elems, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
    const int64_t units = elems / 8;
    if (units == 0) return hipSuccess;
    if (f32) mxfp4_quantize_kernel<true><<<flat_grid(units), kThreads, 0, s>>>(x, units, (uint32_t*)codes, scales);
    else mxfp4_quantize_kernel<false><<<flat_grid(units), kThreads, 0, s>>>(x, units, (uint32_t*)codes, scales);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t elems,
                                   void* y, bool f32, hipStream_t s) {
    const int64_t units = elems / (f32 ? 4 : 8);
    if (units == 0) return hipSuccess;
    if (f32) mxfp4_dequantize_kernel<true><<<flat_grid(units), kThreads, 0, s>>>(codes, scales, units, y);
    else mxfp4_dequantize_kernel<false><<<flat_grid(units), kThreads, 0, s>>>(codes, scales, units, y);
    return hipGetLastError();
}

}  // namespace moe
