// api_experts.cpp - the C ABI of moe_experts.h: argument checks and the launch of
// each entry point.  Every check runs before the first launch, so a call that
// returns an error has enqueued nothing.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "moe_experts.h"
#include "api_common.hpp"
#include "experts.hpp"

namespace {

using moe::check_apart;
using moe::check_elems;
using moe::check_float;
using moe::check_row_count;
using moe::check_rows_ptr;
using moe::fail;
using moe::float_bytes;
using moe::is_float;

int check_len(int64_t n, int multiple, const char* name) {
    if (n <= 0 || n % multiple != 0)
        return fail(MOE_ERR_INVALID_ARG, "%s=%lld must be a positive multiple of %d", name,
                    (long long)n, multiple);
    if (n > ((int64_t)1 << 24))
        return fail(MOE_ERR_INVALID_ARG, "%s=%lld exceeds 2^24", name, (long long)n);
    return MOE_OK;
}

// packed_cnt and packed_off, both or (if they may be left out) neither.
int check_segments(const int32_t* cnt, const int32_t* off, int E, bool needed) {
    if ((cnt == nullptr) != (off == nullptr) || (needed && !cnt))
        return fail(MOE_ERR_INVALID_ARG, needed ? "packed_cnt or packed_off is NULL"
                                                : "packed_cnt and packed_off go together");
    if (!cnt) return MOE_OK;
    if (E < 1 || E > 1024) return fail(MOE_ERR_INVALID_ARG, "E=%d must be in [1,1024]", E);
    MOE_TRY(check_elems(cnt, E, 4, "packed_cnt"));
    return check_elems(off, E, 4, "packed_off");
}

struct Buf {
    const void* p;
    int64_t bytes;
    const char* name;
};

// No output shares bytes with an input or with another output.
template <int NO, int NI>
int check_all_apart(const Buf (&out)[NO], const Buf (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Buf& b : in)
            MOE_TRY(check_apart(out[i].p, out[i].bytes, out[i].name, b.p, b.bytes, b.name));
        for (int j = 0; j < i; ++j)
            MOE_TRY(check_apart(out[i].p, out[i].bytes, out[i].name, out[j].p, out[j].bytes,
                                out[j].name));
    }
    return MOE_OK;
}

}  // namespace

MOE_API int moe_mxfp4_quantize(const void* x, moe_dtype x_dt, int64_t rows, int64_t H,
                               void* codes, void* scales, void* stream) {
    MOE_TRY(check_float(x_dt, "x"));
    MOE_TRY(check_len(H, moe::kMxBlock, "H"));
    MOE_TRY(check_row_count(rows, "rows"));
    MOE_TRY(check_rows_ptr(x, rows, "x"));
    MOE_TRY(check_rows_ptr(codes, rows, "codes"));
    MOE_TRY(check_elems(scales, rows, 1, "scales"));
    MOE_TRY(check_all_apart({{codes, rows * (H / 2), "codes"},
                             {scales, rows * (H / moe::kMxBlock), "scales"}},
                            {{x, rows * H * float_bytes(x_dt), "x"}}));
    MOE_HIP(moe::launch_mxfp4_quantize(x, x_dt == MOE_F32, rows * H, (uint8_t*)codes,
                                       (uint8_t*)scales, (hipStream_t)stream),
            "moe_mxfp4_quantize");
    return MOE_OK;
}

MOE_API int moe_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t H,
                                 void* y, moe_dtype y_dt, void* stream) {
    MOE_TRY(check_float(y_dt, "y"));
    MOE_TRY(check_len(H, moe::kMxBlock, "H"));
    MOE_TRY(check_row_count(rows, "rows"));
    MOE_TRY(check_rows_ptr(codes, rows, "codes"));
    MOE_TRY(check_elems(scales, rows, 1, "scales"));
    MOE_TRY(check_rows_ptr(y, rows, "y"));
    MOE_TRY(check_all_apart({{y, rows * H * float_bytes(y_dt), "y"}},
                            {{codes, rows * (H / 2), "codes"},
                             {scales, rows * (H / moe::kMxBlock), "scales"}}));
    MOE_HIP(moe::launch_mxfp4_dequantize((const uint8_t*)codes, (const uint8_t*)scales, rows * H,
                                         y, y_dt == MOE_F32, (hipStream_t)stream),
            "moe_mxfp4_dequantize");
    return MOE_OK;
}

MOE_API int moe_expert_product_mxfp4(const void* a, const void* a_scales, int64_t rows, int64_t H,
                                     const void* w, const void* w_scales, int64_t N,
                                     const int32_t* packed_cnt, const int32_t* packed_off, int E,
                                     int swiglu, void* y, moe_dtype y_dt, void* stream) {
    MOE_TRY(check_float(y_dt, "y"));
    MOE_TRY(check_len(H, moe::kMxBlock, "H"));
    MOE_TRY(check_len(N, swiglu ? 16 : 8, "N"));
    MOE_TRY(check_row_count(rows, "rows"));
    MOE_TRY(check_segments(packed_cnt, packed_off, E, true));
    MOE_TRY(check_rows_ptr(a, rows, "a"));
    MOE_TRY(check_elems(a_scales, rows, 1, "a_scales"));
    MOE_TRY(check_rows_ptr(w, E, "w"));
    MOE_TRY(check_elems(w_scales, E, 1, "w_scales"));
    MOE_TRY(check_rows_ptr(y, rows, "y"));
    const int64_t cols = swiglu ? N / 2 : N;
    MOE_TRY(check_all_apart({{y, rows * cols * float_bytes(y_dt), "y"}},
                            {{a, rows * (H / 2), "a"},
                             {a_scales, rows * (H / moe::kMxBlock), "a_scales"},
                             {w, E * N * (H / 2), "w"},
                             {w_scales, E * N * (H / moe::kMxBlock), "w_scales"},
                             {packed_cnt, (int64_t)E * 4, "packed_cnt"},
                             {packed_off, ((int64_t)E + 1) * 4, "packed_off"}}));
    moe::ProductArgs p{};
    p.a = (const uint8_t*)a;
    p.a_scales = (const uint8_t*)a_scales;
    p.w = (const uint8_t*)w;
    p.w_scales = (const uint8_t*)w_scales;
    p.rows = rows;
    p.H = H;
    p.N = N;
    p.packed_cnt = packed_cnt;
    p.packed_off = packed_off;
    p.E = E;
    p.swiglu = swiglu != 0;
    p.y = y;
    p.y_f32 = y_dt == MOE_F32;
    MOE_HIP(moe::launch_product(p, (hipStream_t)stream), "moe_expert_product_mxfp4");
    return MOE_OK;
}

MOE_API size_t moe_experts_decode_workspace_size(int64_t T, int K, int64_t H, int64_t I) {
    if (T < 0 || K < 1 || K > 16 || T > moe::kDecodeEntries || T * K > moe::kDecodeEntries)
        return 0;
    for (int64_t n : {H, I})
        if (n <= 0 || n % 8 != 0 || n > moe::kDecodeLength) return 0;
    return moe::decode_ws(T, K, H, I);
}

MOE_API int moe_experts_decode(const void* x, int64_t T, int64_t H, const int32_t* idx,
                               const float* w, int K, int E, int64_t I, const void* w13,
                               const void* w13_scales, const void* w2, const void* w2_scales,
                               moe_dtype wt_dt, void* out, moe_dtype out_dt, void* ws,
                               size_t ws_bytes, void* stream) {
    MOE_TRY(check_float(out_dt, "out"));
    const bool mx = wt_dt == MOE_FP4_E2M1;
    if (!mx && wt_dt != MOE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "weight dtype must be MOE_BF16 or MOE_FP4_E2M1");
    MOE_TRY(check_len(H, mx ? moe::kMxBlock : 8, "H"));
    MOE_TRY(check_len(I, mx ? moe::kMxBlock : 8, "I"));
    if (H > moe::kDecodeLength || I > moe::kDecodeLength)
        return fail(MOE_ERR_INVALID_ARG, "H=%lld or I=%lld exceeds 2^20", (long long)H, (long long)I);
    if (K < 1 || K > 16) return fail(MOE_ERR_INVALID_ARG, "K=%d must be in [1,16]", K);
    if (T < 0 || T > moe::kDecodeEntries || T * K > moe::kDecodeEntries)
        return fail(MOE_ERR_INVALID_ARG, "T=%lld with K=%d: T*K must be in [0, %d]", (long long)T, K,
                    moe::kDecodeEntries);
    if (E < 1 || E > 1024) return fail(MOE_ERR_INVALID_ARG, "E=%d must be in [1,1024]", E);
    MOE_TRY(check_rows_ptr(x, T, "x"));
    MOE_TRY(check_elems(idx, T, 4, "idx"));
    MOE_TRY(check_elems(w, T, 4, "w"));
    MOE_TRY(check_rows_ptr(w13, E, "w13"));
    MOE_TRY(check_rows_ptr(w2, E, "w2"));
    if (mx != (w13_scales != nullptr) || mx != (w2_scales != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "w13_scales and w2_scales go with MOE_FP4_E2M1 weights alone");
    MOE_TRY(check_rows_ptr(out, T, "out"));
    const size_t need = moe::decode_ws(T, K, H, I);
    MOE_TRY(moe::check_ws(ws, ws_bytes, need));
    const int64_t wb = (int64_t)E * H * I * (mx ? 1 : 4) / 2, sb = (int64_t)E * H * I / moe::kMxBlock;
    MOE_TRY(check_all_apart({{out, T * H * float_bytes(out_dt), "out"}, {ws, (int64_t)need, "ws"}},
                            {{x, T * H * 2, "x"},
                             {idx, T * K * 4, "idx"},
                             {w, T * K * 4, "w"},
                             {w13, 2 * wb, "w13"},
                             {w13_scales, 2 * sb, "w13_scales"},
                             {w2, wb, "w2"},
                             {w2_scales, sb, "w2_scales"}}));
    moe::DecodeArgs a{};
    a.x = (const uint16_t*)x;
    a.T = T;
    a.H = H;
    a.I = I;
    a.idx = idx;
    a.w = w;
    a.K = K;
    a.E = E;
    a.w13 = w13;
    a.s13 = (const uint8_t*)w13_scales;
    a.w2 = w2;
    a.s2 = (const uint8_t*)w2_scales;
    a.out = out;
    a.out_f32 = out_dt == MOE_F32;
    a.ws = ws;
    MOE_HIP(moe::launch_experts_decode(a, (hipStream_t)stream), "moe_experts_decode");
    return MOE_OK;
}

MOE_API int moe_swiglu(const void* gu, moe_dtype gu_dt, int64_t rows, int64_t I,
                       const int32_t* packed_cnt, const int32_t* packed_off, int E, void* h,
                       moe_dtype h_dt, void* codes, float* scales, void* stream) {
    MOE_TRY(check_float(gu_dt, "gu"));
    MOE_TRY(check_float(h_dt, "h"));
    if ((codes == nullptr) != (scales == nullptr))
        return fail(MOE_ERR_INVALID_ARG, "codes and scales go together");
    MOE_TRY(check_len(I, codes ? 128 : 8, "I"));
    MOE_TRY(check_row_count(rows, "rows"));
    MOE_TRY(check_rows_ptr(gu, rows, "gu"));
    MOE_TRY(check_rows_ptr(h, rows, "h"));
    MOE_TRY(check_rows_ptr(codes, 0, "codes"));
    MOE_TRY(check_elems(scales, 0, 4, "scales"));
    MOE_TRY(check_segments(packed_cnt, packed_off, E, false));
    MOE_TRY(check_all_apart({{h, rows * I * float_bytes(h_dt), "h"},
                             {codes, rows * 2 * I, "codes"},
                             {scales, rows * (I / 64) * 4, "scales"}},
                            {{gu, rows * 2 * I * float_bytes(gu_dt), "gu"},
                             {packed_cnt, (int64_t)E * 4, "packed_cnt"},
                             {packed_off, ((int64_t)E + 1) * 4, "packed_off"}}));
    moe::SwigluArgs a{};
    a.gu = gu;
    a.gu_f32 = gu_dt == MOE_F32;
    a.rows = rows;
    a.I = I;
    a.packed_cnt = packed_cnt;
    a.packed_off = packed_off;
    a.E = E;
    a.h = h;
    a.h_f32 = h_dt == MOE_F32;
    a.codes = (uint8_t*)codes;
    a.scales = scales;
    MOE_HIP(moe::launch_swiglu(a, (hipStream_t)stream), "moe_swiglu");
    return MOE_OK;
}

MOE_API int moe_swiglu_backward(const void* dh, moe_dtype dh_dt, const void* gu, moe_dtype gu_dt,
                                const float* gu_scales, int64_t rows, int64_t I,
                                const int32_t* packed_cnt, const int32_t* packed_off, int E,
                                void* dgu, void* h, moe_dtype out_dt, void* stream) {
    MOE_TRY(check_float(dh_dt, "dh"));
    MOE_TRY(check_float(out_dt, "out"));
    const bool fp8 = gu_dt == MOE_FP8_E4M3;
    if (!fp8 && !is_float(gu_dt))
        return fail(MOE_ERR_INVALID_ARG, "gu dtype must be MOE_BF16, MOE_F32 or MOE_FP8_E4M3");
    MOE_TRY(check_len(I, fp8 ? 128 : 8, "I"));
    MOE_TRY(check_row_count(rows, "rows"));
    MOE_TRY(check_rows_ptr(dh, rows, "dh"));
    MOE_TRY(check_rows_ptr(gu, rows, "gu"));
    if (!fp8 && gu_scales)
        return fail(MOE_ERR_INVALID_ARG, "gu_scales must be NULL unless gu is fp8");
    MOE_TRY(check_elems(gu_scales, fp8 ? rows : 0, 4, "gu_scales"));
    MOE_TRY(check_rows_ptr(dgu, rows, "dgu"));
    MOE_TRY(check_rows_ptr(h, 0, "h"));
    MOE_TRY(check_segments(packed_cnt, packed_off, E, false));
    MOE_TRY(check_all_apart({{dgu, rows * 2 * I * float_bytes(out_dt), "dgu"},
                             {h, rows * I * float_bytes(out_dt), "h"}},
                            {{dh, rows * I * float_bytes(dh_dt), "dh"},
                             {gu, rows * 2 * I * (fp8 ? 1 : float_bytes(gu_dt)), "gu"},
                             {gu_scales, rows * (I / 64) * 4, "gu_scales"},
                             {packed_cnt, (int64_t)E * 4, "packed_cnt"},
                             {packed_off, ((int64_t)E + 1) * 4, "packed_off"}}));
    moe::SwigluGradArgs a{};
    a.dh = dh;
    a.dh_f32 = dh_dt == MOE_F32;
    a.gu = gu;
    a.gu_kind = fp8 ? moe::RowKind::Fp8 : gu_dt == MOE_F32 ? moe::RowKind::F32 : moe::RowKind::Bf16;
    a.scales = gu_scales;
    a.rows = rows;
    a.I = I;
    a.packed_cnt = packed_cnt;
    a.packed_off = packed_off;
    a.E = E;
    a.dgu = dgu;
    a.h = h;
    a.out_f32 = out_dt == MOE_F32;
    MOE_HIP(moe::launch_swiglu_grad(a, (hipStream_t)stream), "moe_swiglu_backward");
    return MOE_OK;
}
