// experts.hpp - launch interface between the C ABI of the experts' step
// (api_experts.cpp) and its kernels (mxfp4.hip, swiglu.hip, expert_product.hip,
// experts_decode.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "experts_rules.hpp"
#include "train.hpp"

namespace moe {

// MXFP4: blocks of 32 e2m1 codes that share one e8m0 scale.
constexpr int kMxBlock = 32;

hipError_t launch_mxfp4_quantize(const void* x, bool f32, int64_t elems, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t elems,
                                   void* y, bool f32, hipStream_t s);

struct SwigluArgs {
    const void* gu;             // [rows,2I]
    bool gu_f32;
    int64_t rows, I;
    const int32_t* packed_cnt;  // [E], with packed_off [E+1]; null: every row
    const int32_t* packed_off;
    int E;
    void* h;                    // [rows,I]
    bool h_f32;
    uint8_t* codes;             // [rows,2I] e4m3, with scales [rows,2I/128]; or null
    float* scales;
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);

struct SwigluGradArgs {
    const void* dh;             // [rows,I]
    bool dh_f32;
    const void* gu;             // [rows,2I] bf16, f32 or e4m3 codes with scales
    RowKind gu_kind;
    const float* scales;
    int64_t rows, I;
    const int32_t* packed_cnt;
    const int32_t* packed_off;
    int E;
    void* dgu;                  // [rows,2I]
    void* h;                    // [rows,I] or null
    bool out_f32;               // of dgu and h
};
hipError_t launch_swiglu_grad(const SwigluGradArgs& a, hipStream_t s);

struct ProductArgs {
    const uint8_t* a;           // [rows,H/2] codes, a_scales [rows,H/32]
    const uint8_t* a_scales;
    const uint8_t* w;           // [E,N,H/2] codes, w_scales [E,N,H/32]
    const uint8_t* w_scales;
    int64_t rows, H, N;
    const int32_t* packed_cnt;  // [E]
    const int32_t* packed_off;  // [E+1]
    int E;
    bool swiglu;
    void* y;                    // [rows,N], or [rows,N/2] with swiglu
    bool y_f32;
};
hipError_t launch_product(const ProductArgs& a, hipStream_t s);

// The whole experts' step of a few tokens.
constexpr int kDecodeEntries = 1024;              // most T*K
constexpr int64_t kDecodeLength = (int64_t)1 << 20;   // most H and I
struct DecodeArgs {
    const uint16_t* x;          // [T,H] bf16
    int64_t T, H, I;
    const int32_t* idx;         // [T,K]
    const float* w;             // [T,K]
    int K, E;
    const void* w13;            // [E,2I,H] bf16, or codes with s13 [E,2I,H/32]
    const uint8_t* s13;
    const void* w2;             // [E,H,I] bf16, or codes with s2 [E,H,I/32]
    const uint8_t* s2;
    void* out;                  // [T,H]
    bool out_f32;
    void* ws;
};
size_t decode_ws(int64_t T, int K, int64_t H, int64_t I);
hipError_t launch_experts_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace moe
