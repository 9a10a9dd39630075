// train.hpp - launch interface between the training-side C ABI (api_train.cpp)
// and its kernels (gate.hip, grad.hip, embedding.hip).  Not part of the public
// ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct GateArgs {
    const void* logits;  // [T,E] bf16 or f32
    bool f32;
    int64_t T;
    int E, K;
    bool renorm;
    float scale;
    int32_t* idx;        // forward: out; backward: in
    float* w;            // forward out
    const float* dw;     // backward in
    void* dlogits;       // backward out
};
hipError_t launch_gate(const GateArgs& a, hipStream_t s);
hipError_t launch_gate_backward(const GateArgs& a, hipStream_t s);

// How the rows of an expert output are stored.
enum class RowKind { Bf16, F32, Fp8, Fp4 };

struct CombineGradArgs {
    const void* dout;           // [T,H]
    bool dout_f32;
    const float* dout_weights;  // [T] or null
    int64_t T, H;
    const void* y;              // [y_rows,H]; read only if dw
    RowKind y_kind;
    const float* y_scales;      // [y_rows,H/128] or null
    int64_t y_rows;
    const int64_t* tok_map;
    const float* w;             // read only if dy
    int K;
    void* dy;                   // [y_rows,H] or null
    bool dy_f32;
    const int32_t* packed_cnt;  // [E], with packed_off [E+1]; null: unowned rows stay
    const int32_t* packed_off;
    int E;
    float* dw;                  // [T,K] or null
};
hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t s);

struct DispatchGradArgs {
    const void* dpacked;   // [packed_rows,H]
    bool d_f32;
    int64_t packed_rows, H;
    const int64_t* tok_map;
    int64_t T;
    int K;
    const void* residual;  // [T,H] of dx's type, or null; may be dx
    void* dx;
    bool dx_f32;
};
hipError_t launch_dispatch_grad(const DispatchGradArgs& a, hipStream_t s);

struct EmbeddingArgs {
    const void* table;   // [V,H]
    bool table_f32;
    int64_t V, H;
    const void* ids;     // [N] of id_bytes
    int id_bytes;
    int64_t N;
    float scale;
    void* out;
    bool out_f32;
    int32_t* stats;      // [1] or null
};
hipError_t launch_embedding(const EmbeddingArgs& a, hipStream_t s);

struct EmbeddingGradArgs {
    const void* dout;    // [N,H]
    bool dout_f32;
    const void* ids;
    int id_bytes;
    int64_t N, V, H;
    float scale;
    bool accumulate;
    void* dtable;        // [V,H]
    bool dtable_f32;
    void* ws;
};
size_t embedding_grad_ws(int64_t N, int64_t V, int64_t H);
hipError_t launch_embedding_grad(const EmbeddingGradArgs& a, hipStream_t s);

}  // namespace moe
