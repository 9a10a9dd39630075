// api_train.cpp - the C ABI of moe_train.h: argument checks and the launch of
// each entry point.  Every check runs before the first launch, so a call that
// returns an error has enqueued nothing.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "moe_train.h"
#include "api_common.hpp"
#include "train.hpp"

namespace {

using moe::aligned;
using moe::check_H;
using moe::check_rows_ptr;
using moe::fail;
using moe::kMaxRows;

bool is_float(moe_dtype d) { return d == MOE_BF16 || d == MOE_F32; }

int64_t float_bytes(moe_dtype d) { return d == MOE_F32 ? 4 : 2; }

int check_float(moe_dtype d, const char* name) {
    if (is_float(d)) return MOE_OK;
    return fail(MOE_ERR_INVALID_ARG, "%s dtype must be MOE_BF16 or MOE_F32", name);
}

int check_elems(const void* p, int64_t n, size_t align, const char* name) {
    if (n > 0 && !p) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    if (p && !aligned(p, align))
        return fail(MOE_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    return MOE_OK;
}

// out and in must not share bytes.
int check_apart(const void* out, int64_t out_bytes, const char* out_name, const void* in,
                int64_t in_bytes, const char* in_name) {
    if (!out || !in || out_bytes <= 0 || in_bytes <= 0) return MOE_OK;
    const uintptr_t a = (uintptr_t)out, b = (uintptr_t)in;
    if (a < b + (uintptr_t)in_bytes && b < a + (uintptr_t)out_bytes)
        return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", out_name, in_name);
    return MOE_OK;
}

int check_entries(int64_t T, int K, const int64_t* tok_map) {
    if (T < 0 || T >= ((int64_t)1 << 31))
        return fail(MOE_ERR_INVALID_ARG, "T=%lld must be in [0, 2^31)", (long long)T);
    if (K < 1 || K > 16) return fail(MOE_ERR_INVALID_ARG, "K=%d must be in [1,16]", K);
    if (T * (int64_t)K >= ((int64_t)1 << 31))
        return fail(MOE_ERR_INVALID_ARG, "T*K=%lld must be < 2^31", (long long)(T * K));
    return check_elems(tok_map, T, 8, "tok_map");
}

int check_row_count(int64_t rows, const char* name) {
    if (rows < 0 || rows > kMaxRows)
        return fail(MOE_ERR_INVALID_ARG, "%s must be in [0, 2^31-1]", name);
    return MOE_OK;
}

int check_gate(const void* logits, moe_dtype l_dt, int64_t T, int E, int K) {
    MOE_TRY(check_float(l_dt, "logits"));
    if (T < 0 || T >= ((int64_t)1 << 31))
        return fail(MOE_ERR_INVALID_ARG, "T=%lld must be in [0, 2^31)", (long long)T);
    if (E < 1 || E > 1024) return fail(MOE_ERR_INVALID_ARG, "E=%d must be in [1,1024]", E);
    if (K < 1 || K > 16 || K > E)
        return fail(MOE_ERR_INVALID_ARG, "K=%d must be in [1,16] and at most E=%d", K, E);
    if (T * (int64_t)K >= ((int64_t)1 << 31))
        return fail(MOE_ERR_INVALID_ARG, "T*K=%lld must be < 2^31", (long long)(T * K));
    return check_elems(logits, T, (size_t)float_bytes(l_dt), "logits");
}

int check_ids(const void* ids, int id_bytes, int64_t N) {
    if (N < 0 || N >= ((int64_t)1 << 31))
        return fail(MOE_ERR_INVALID_ARG, "N=%lld must be in [0, 2^31)", (long long)N);
    if (id_bytes != 4 && id_bytes != 8)
        return fail(MOE_ERR_INVALID_ARG, "id_bytes=%d must be 4 or 8", id_bytes);
    return check_elems(ids, N, (size_t)id_bytes, "ids");
}

int check_vocab(int64_t V) {
    if (V < 1 || V > kMaxRows)
        return fail(MOE_ERR_INVALID_ARG, "V=%lld must be in [1, 2^31-1]", (long long)V);
    return MOE_OK;
}

moe::GateArgs gate_args(const void* logits, moe_dtype l_dt, int64_t T, int E, int K,
                        int renormalize, float scale) {
    moe::GateArgs a{};
    a.logits = logits;
    a.f32 = l_dt == MOE_F32;
    a.T = T;
    a.E = E;
    a.K = K;
    a.renorm = renormalize != 0;
    a.scale = scale;
    return a;
}

}  // namespace

MOE_API int moe_gate(const void* logits, moe_dtype l_dt, int64_t T, int E, int K, int renormalize,
                     float scale, int32_t* idx, float* w, void* stream) {
    MOE_TRY(check_gate(logits, l_dt, T, E, K));
    MOE_TRY(check_elems(idx, T, 4, "idx"));
    MOE_TRY(check_elems(w, T, 4, "w"));
    const int64_t in = T * E * float_bytes(l_dt), out = T * K * 4;
    MOE_TRY(check_apart(idx, out, "idx", logits, in, "logits"));
    MOE_TRY(check_apart(w, out, "w", logits, in, "logits"));
    MOE_TRY(check_apart(idx, out, "idx", w, out, "w"));
    moe::GateArgs a = gate_args(logits, l_dt, T, E, K, renormalize, scale);
    a.idx = idx;
    a.w = w;
    MOE_HIP(moe::launch_gate(a, (hipStream_t)stream), "moe_gate");
    return MOE_OK;
}

MOE_API int moe_gate_backward(const void* logits, moe_dtype l_dt, int64_t T, int E, int K,
                              int renormalize, float scale, const int32_t* idx, const float* dw,
                              void* dlogits, void* stream) {
    MOE_TRY(check_gate(logits, l_dt, T, E, K));
    MOE_TRY(check_elems(idx, T, 4, "idx"));
    MOE_TRY(check_elems(dw, T, 4, "dw"));
    MOE_TRY(check_elems(dlogits, T, (size_t)float_bytes(l_dt), "dlogits"));
    const int64_t lb = T * E * float_bytes(l_dt), kb = T * K * 4;
    MOE_TRY(check_apart(dlogits, lb, "dlogits", logits, lb, "logits"));
    MOE_TRY(check_apart(dlogits, lb, "dlogits", idx, kb, "idx"));
    MOE_TRY(check_apart(dlogits, lb, "dlogits", dw, kb, "dw"));
    moe::GateArgs a = gate_args(logits, l_dt, T, E, K, renormalize, scale);
    a.idx = const_cast<int32_t*>(idx);
    a.dw = dw;
    a.dlogits = dlogits;
    MOE_HIP(moe::launch_gate_backward(a, (hipStream_t)stream), "moe_gate_backward");
    return MOE_OK;
}

MOE_API int moe_combine_backward(const void* dout, moe_dtype dout_dt, const float* dout_weights,
                                 int64_t T, int64_t H, const void* y, moe_dtype y_dt,
                                 const float* y_scales, int64_t y_rows, const int64_t* tok_map,
                                 const float* w, int K, void* dy, moe_dtype dy_dt,
                                 const int32_t* packed_cnt, const int32_t* packed_off, int E,
                                 float* dw, void* stream) {
    MOE_TRY(check_entries(T, K, tok_map));
    MOE_TRY(check_float(dout_dt, "dout"));
    if (!is_float(y_dt) && !moe::quantized(y_dt))
        return fail(MOE_ERR_INVALID_ARG, "unknown y dtype %d", (int)y_dt);
    MOE_TRY(check_H(H, moe::quantized(y_dt)));
    MOE_TRY(check_row_count(y_rows, "y_rows"));
    MOE_TRY(check_rows_ptr(dout, T, "dout"));
    if (dout_weights && !aligned(dout_weights, 4))
        return fail(MOE_ERR_INVALID_ARG, "dout_weights is not 4-byte aligned");
    if (!dy && !dw) return fail(MOE_ERR_INVALID_ARG, "dy and dw are both NULL");
    if (y_scales && !moe::quantized(y_dt))
        return fail(MOE_ERR_INVALID_ARG, "y_scales must be NULL unless y is fp8 or fp4");
    if (y_scales && !aligned(y_scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "y_scales is not 4-byte aligned");
    if (dw) MOE_TRY(check_rows_ptr(y, y_rows, "y"));
    if (dw && !aligned(dw, 4)) return fail(MOE_ERR_INVALID_ARG, "dw is not 4-byte aligned");
    if ((packed_cnt == nullptr) != (packed_off == nullptr))
        return fail(MOE_ERR_INVALID_ARG, "packed_cnt and packed_off go together");
    if (packed_cnt && (E < 1 || E > 1024))
        return fail(MOE_ERR_INVALID_ARG, "E=%d must be in [1,1024]", E);
    if (packed_cnt && (!aligned(packed_cnt, 4) || !aligned(packed_off, 4)))
        return fail(MOE_ERR_INVALID_ARG, "packed_cnt or packed_off is not 4-byte aligned");
    const int64_t dout_bytes = T * H * float_bytes(dout_dt);
    const int64_t y_bytes = !dw ? 0
                            : is_float(y_dt) ? y_rows * H * float_bytes(y_dt)
                                             : y_rows * (y_dt == MOE_FP4_E2M1 ? H / 2 : H);
    if (dy) {
        MOE_TRY(check_float(dy_dt, "dy"));
        MOE_TRY(check_rows_ptr(dy, y_rows, "dy"));
        MOE_TRY(check_elems(w, T, 4, "w"));
    }
    // what the call reads; y and its scales for dw only, w and the segments for dy only
    const struct {
        const void* p;
        int64_t bytes;
        const char* name;
    } in[] = {{dout, dout_bytes, "dout"},
              {dout_weights, dw ? T * 4 : 0, "dout_weights"},
              {y, y_bytes, "y"},
              {y_scales, dw ? y_rows * (H / 128) * 4 : 0, "y_scales"},
              {tok_map, T * K * 8, "tok_map"},
              {w, dy ? T * K * 4 : 0, "w"},
              {packed_cnt, dy ? (int64_t)E * 4 : 0, "packed_cnt"},
              {packed_off, dy ? ((int64_t)E + 1) * 4 : 0, "packed_off"}};
    const int64_t dy_bytes = y_rows * H * float_bytes(dy_dt);
    for (const auto& i : in) {
        MOE_TRY(check_apart(dy, dy_bytes, "dy", i.p, i.bytes, i.name));
        MOE_TRY(check_apart(dw, T * K * 4, "dw", i.p, i.bytes, i.name));
    }
    MOE_TRY(check_apart(dy, dy_bytes, "dy", dw, T * K * 4, "dw"));
    moe::CombineGradArgs a{};
    a.dout = dout;
    a.dout_f32 = dout_dt == MOE_F32;
    a.dout_weights = dout_weights;
    a.T = T;
    a.H = H;
    a.y = y;
    a.y_kind = y_dt == MOE_F32          ? moe::RowKind::F32
               : y_dt == MOE_FP8_E4M3   ? moe::RowKind::Fp8
               : y_dt == MOE_FP4_E2M1   ? moe::RowKind::Fp4
                                        : moe::RowKind::Bf16;
    a.y_scales = y_scales;
    a.y_rows = y_rows;
    a.tok_map = tok_map;
    a.w = w;
    a.K = K;
    a.dy = dy;
    a.dy_f32 = dy_dt == MOE_F32;
    a.packed_cnt = packed_cnt;
    a.packed_off = packed_off;
    a.E = E;
    a.dw = dw;
    MOE_HIP(moe::launch_combine_grad(a, (hipStream_t)stream), "moe_combine_backward");
    return MOE_OK;
}

MOE_API int moe_dispatch_backward(const void* dpacked, moe_dtype d_dt, int64_t packed_rows,
                                  int64_t H, const int64_t* tok_map, int64_t T, int K,
                                  const void* residual, void* dx, moe_dtype dx_dt, void* stream) {
    MOE_TRY(check_entries(T, K, tok_map));
    MOE_TRY(check_float(d_dt, "dpacked"));
    MOE_TRY(check_float(dx_dt, "dx"));
    MOE_TRY(check_H(H, false));
    MOE_TRY(check_row_count(packed_rows, "packed_rows"));
    MOE_TRY(check_rows_ptr(dpacked, packed_rows, "dpacked"));
    MOE_TRY(check_rows_ptr(dx, T, "dx"));
    MOE_TRY(check_rows_ptr(residual, 0, "residual"));
    const int64_t b = T * H * float_bytes(dx_dt);
    MOE_TRY(check_apart(dx, b, "dx", dpacked, packed_rows * H * float_bytes(d_dt), "dpacked"));
    MOE_TRY(check_apart(dx, b, "dx", tok_map, T * K * 8, "tok_map"));
    if (residual != dx) MOE_TRY(check_apart(dx, b, "dx", residual, b, "residual"));
    moe::DispatchGradArgs a{};
    a.dpacked = dpacked;
    a.d_f32 = d_dt == MOE_F32;
    a.packed_rows = packed_rows;
    a.H = H;
    a.tok_map = tok_map;
    a.T = T;
    a.K = K;
    a.residual = residual;
    a.dx = dx;
    a.dx_f32 = dx_dt == MOE_F32;
    MOE_HIP(moe::launch_dispatch_grad(a, (hipStream_t)stream), "moe_dispatch_backward");
    return MOE_OK;
}

MOE_API int moe_embedding(const void* table, moe_dtype table_dt, int64_t V, int64_t H,
                          const void* ids, int id_bytes, int64_t N, float scale, void* out,
                          moe_dtype out_dt, int32_t* stats, void* stream) {
    MOE_TRY(check_float(table_dt, "table"));
    MOE_TRY(check_float(out_dt, "out"));
    MOE_TRY(check_vocab(V));
    MOE_TRY(check_H(H, false));
    MOE_TRY(check_ids(ids, id_bytes, N));
    MOE_TRY(check_rows_ptr(table, V, "table"));
    MOE_TRY(check_rows_ptr(out, N, "out"));
    if (stats && !aligned(stats, 4))
        return fail(MOE_ERR_INVALID_ARG, "stats is not 4-byte aligned");
    const int64_t tb = V * H * float_bytes(table_dt), ob = N * H * float_bytes(out_dt);
    MOE_TRY(check_apart(out, ob, "out", table, tb, "table"));
    MOE_TRY(check_apart(out, ob, "out", ids, N * id_bytes, "ids"));
    MOE_TRY(check_apart(stats, 4, "stats", out, ob, "out"));
    MOE_TRY(check_apart(stats, 4, "stats", table, tb, "table"));
    MOE_TRY(check_apart(stats, 4, "stats", ids, N * id_bytes, "ids"));
    moe::EmbeddingArgs a{};
    a.table = table;
    a.table_f32 = table_dt == MOE_F32;
    a.V = V;
    a.H = H;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.N = N;
    a.scale = scale;
    a.out = out;
    a.out_f32 = out_dt == MOE_F32;
    a.stats = stats;
    MOE_HIP(moe::launch_embedding(a, (hipStream_t)stream), "moe_embedding");
    return MOE_OK;
}

MOE_API size_t moe_embedding_workspace_size(int64_t N, int64_t V, int64_t H) {
    if (N < 0 || N >= ((int64_t)1 << 31) || V < 1 || V > kMaxRows || H <= 0 || H % 8 != 0 ||
        H > ((int64_t)1 << 24))
        return 0;
    return moe::embedding_grad_ws(N, V, H);
}

MOE_API int moe_embedding_backward(const void* dout, moe_dtype dout_dt, const void* ids,
                                   int id_bytes, int64_t N, int64_t V, int64_t H, float scale,
                                   int accumulate, void* dtable, moe_dtype dtable_dt, void* ws,
                                   size_t ws_bytes, void* stream) {
    MOE_TRY(check_float(dout_dt, "dout"));
    MOE_TRY(check_float(dtable_dt, "dtable"));
    MOE_TRY(check_vocab(V));
    MOE_TRY(check_H(H, false));
    MOE_TRY(check_ids(ids, id_bytes, N));
    MOE_TRY(check_rows_ptr(dout, N, "dout"));
    MOE_TRY(check_rows_ptr(dtable, V, "dtable"));
    const size_t need = moe::embedding_grad_ws(N, V, H);
    MOE_TRY(moe::check_ws(ws, ws_bytes, need));
    const int64_t db = N * H * float_bytes(dout_dt), tb = V * H * float_bytes(dtable_dt);
    MOE_TRY(check_apart(dtable, tb, "dtable", dout, db, "dout"));
    MOE_TRY(check_apart(dtable, tb, "dtable", ids, N * id_bytes, "ids"));
    MOE_TRY(check_apart(ws, (int64_t)need, "ws", dout, db, "dout"));
    MOE_TRY(check_apart(ws, (int64_t)need, "ws", ids, N * id_bytes, "ids"));
    MOE_TRY(check_apart(ws, (int64_t)need, "ws", dtable, tb, "dtable"));
    moe::EmbeddingGradArgs a{};
    a.dout = dout;
    a.dout_f32 = dout_dt == MOE_F32;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.N = N;
    a.V = V;
    a.H = H;
    a.scale = scale;
    a.accumulate = accumulate != 0;
    a.dtable = dtable;
    a.dtable_f32 = dtable_dt == MOE_F32;
    a.ws = ws;
    MOE_HIP(moe::launch_embedding_grad(a, (hipStream_t)stream), "moe_embedding_backward");
    return MOE_OK;
}
