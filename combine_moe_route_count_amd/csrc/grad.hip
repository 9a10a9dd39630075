// grad.hip - gradients of the combine and the dispatch.
//
// Combine, out[t] = sum_k w[t,k] * v[r] with r = tok_map[t,k]:
//   dy[r] = w[t,k] * dout[t],   dw[t,k] = <dout[t], v[r]> (+ dout_weights[t]).
// One pass: a workgroup takes a few entries of one token and walks the row; each
// lane holds 8 elements of dout[t], loads those of every v[r], adds the products to
// one f32 sum per entry and writes w*dout to every dy[r].  The sums are joined by
// the wave reduction and then over the waves in LDS, always in the same order.
// HBM bound: per entry one row read and one row written, 3 flops per element.
//
// Dispatch, packed[r] = x[t] for every entry of t: dx[t] = sum_k dpacked[r], the
// combine's gather without weights.
#include "train_device.hpp"
#include "internal.hpp"

namespace moe {

namespace {

constexpr int kGradThreads = 512;   // most of a workgroup

// Rows of dy that no entry owns: [off[e] + cnt[e], off[e+1]) of every expert, and
// [off[E], y_rows).  About kGapGroups workgroups share the experts' rows, at least 8 to
// an expert, and kTailParts those behind the last segment.  Values outside [0, y_rows]
// are clamped.  8 experts of 2048 rows, a quarter owned, rows of 4096 f32: 120 us with
// 8 workgroups per expert, 68 with 1024 in all, 64.5 with 2048, 62 with 4096; 128
// experts and 16 tokens, next to nothing to clear: 9.9, 10.1, 10.2, 11.8.
constexpr int kGapGroups = 2048;
constexpr int kTailParts = 512;
inline int gap_parts(int E) { return kGapGroups / E > 8 ? kGapGroups / E : 8; }

template <bool DYF32>
__device__ __forceinline__ void zero_gap(const CombineGradArgs& a, int64_t item, int expert_parts) {
    int64_t lo, hi;
    int parts, part;
    if (item < (int64_t)a.E * expert_parts) {
        const int e = (int)item / expert_parts;
        parts = expert_parts;
        part = (int)item - e * expert_parts;
        lo = (int64_t)a.packed_off[e] + a.packed_cnt[e];
        hi = a.packed_off[e + 1];
    } else {
        parts = kTailParts;
        part = (int)(item - (int64_t)a.E * expert_parts);
        lo = a.packed_off[a.E];
        hi = a.y_rows;
    }
    if (lo < 0) lo = 0;
    if (hi > a.y_rows) hi = a.y_rows;
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int units = (int)(a.H / 8);
    for (int64_t r = lo + part; r < hi; r += parts)
        for (int u = threadIdx.x; u < units; u += blockDim.x)
            store_unit<DYF32, false>(a.dy, r * a.H + (int64_t)u * 8, zero);
}

// Entries per workgroup and its most threads.  What the rows of one workgroup keep
// in flight decides: two bf16 or f32 rows at up to 512 threads, four rows of codes
// at up to 256.  Measured (us) at T=8192 K=8 H=7168 bf16: 1 entry 464, 2 367-369, 4
// 377, a wave per entry 382; T=8192 K=6 H=4096 f32: 2 entries 352-360, 4 407, a wave
// per entry 391.  Codes, e4m3 and e2m1: T=8192 K=8 H=7168 2 entries 319 and 293, 4 entries
// 313 and 264, at up to 512 threads 366 and 383, 310 and 264; T=501 K=8 H=6144 2 entries
// 21.3 and 21.3, 4 entries 18.4 and 17.6, at up to 512 threads 25.4 and 25.7, 20.0 and 19.8.
constexpr bool is_quant(RowKind k) { return k == RowKind::Fp8 || k == RowKind::Fp4; }
constexpr int grad_entries(RowKind k) { return is_quant(k) ? 4 : 2; }
constexpr int grad_threads(RowKind k) { return is_quant(k) ? 256 : kGradThreads; }

// bf16 rows of dy are stored non-temporally (367 against 384 us at T=8192 K=8
// H=7168), f32 rows through L2 (352 against 360 us at T=8192 K=6 H=4096).
template <RowKind YK, bool DF32, bool DYF32>
__global__ __launch_bounds__(kGradThreads) void combine_grad_kernel(CombineGradArgs a,
                                                                    int groups, int expert_parts,
                                                                    int64_t gap_blocks) {
    constexpr int N = grad_entries(YK);
    __shared__ float wave_dot[kGradThreads / kWave][N];
    const int lane = threadIdx.x % kWave;
    const int wave = threadIdx.x / kWave;
    const int units = (int)(a.H / 8);
    const int64_t nblk = a.H / kFp8Block;
    const int64_t items = a.T * groups;
    for (int64_t b = blockIdx.x; b < items + gap_blocks; b += gridDim.x) {
        if (b >= items) {
            zero_gap<DYF32>(a, b - items, expert_parts);
            continue;
        }
        int64_t t;
        int group;
        xcd_item(b, a.T, groups, t, group);
        // lane i: entry i of this workgroup
        const int k = group * N + lane;
        const int64_t e = t * a.K + k;
        const bool mine = lane < N && k < a.K;
        int my_row = -1;
        float my_w = 0.0f;
        if (mine) {
            const int64_t r = a.tok_map[e];
            if (a.dy) my_w = a.w[e];
            if (r >= 0 && r < a.y_rows) my_row = (int)r;
        }
        int rows[N];
        float w[N], dot[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            rows[i] = readlane(my_row, i);
            w[i] = readlane(my_w, i);
            dot[i] = 0.0f;
        }
        for (int u = threadIdx.x; u < units; u += blockDim.x) {
            const int64_t col = (int64_t)u * 8;
            FloatUnit<DF32, 8> d;
            d.load_cached(a.dout, t * a.H + col);
            Row8<YK> y[N];
            float scale[N];
            if (a.dw) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (rows[i] < 0) continue;
                    y[i].load(a.y, (int64_t)rows[i] * a.H + col);
                    scale[i] = 1.0f;
                    if (is_quant(YK) && a.y_scales)
                        scale[i] = a.y_scales[(int64_t)rows[i] * nblk + u / (kFp8Block / 8)];
                }
            }
            float dv[8];
            d.get(dv);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (rows[i] < 0) continue;
                if (a.dw) {
                    float v[8];
                    y[i].get(v);
                    if (is_quant(YK)) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = v[j] * scale[i];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot[i] = __builtin_fmaf(dv[j], v[j], dot[i]);
                }
                if (a.dy) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = w[i] * dv[j];
                    store_unit<DYF32, !DYF32>(a.dy, (int64_t)rows[i] * a.H + col, o);
                }
            }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = wave_sum(dot[i]);
            if (lane == 0) wave_dot[wave][i] = s;
        }
        __syncthreads();
        if (mine && wave == 0) {
            float s = 0.0f;
            for (int i = 0; i < (int)blockDim.x / kWave; ++i) s += wave_dot[i][lane];
            if (a.dout_weights) s += a.dout_weights[t];
            a.dw[e] = my_row >= 0 ? s : 0.0f;
        }
        __syncthreads();
    }
}

template <RowKind YK, bool DF32, bool DYF32>
void combine_go(const CombineGradArgs& a, hipStream_t s) {
    const int groups = (a.K + grad_entries(YK) - 1) / grad_entries(YK);
    const bool gaps = a.dy && a.packed_off;
    const int expert_parts = gaps ? gap_parts(a.E) : 0;
    const int64_t gap_blocks = gaps ? (int64_t)a.E * expert_parts + kTailParts : 0;
    combine_grad_kernel<YK, DF32, DYF32>
        <<<capped_grid(a.T * groups + gap_blocks), dim3(row_threads(a.H / 8, grad_threads(YK))), 0,
           s>>>(a, groups, expert_parts, gap_blocks);
}

template <RowKind YK>
void combine_by_type(const CombineGradArgs& a, hipStream_t s) {
    if (a.dout_f32) {
        if (a.dy_f32) combine_go<YK, true, true>(a, s);
        else combine_go<YK, true, false>(a, s);
    } else {
        if (a.dy_f32) combine_go<YK, false, true>(a, s);
        else combine_go<YK, false, false>(a, s);
    }
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------

// One workgroup per (token, chunk of the row): lanes below K read the token's rows,
// every lane then has the loads of all rows of its unit in flight and adds them in
// ascending k.  Units of 8 bf16 or 4 f32 elements, one 16-byte load per row.
constexpr int kGatherThreads = 256;
constexpr int gather_unit(bool f32) { return f32 ? 4 : 8; }

template <bool DF32, bool OF32, int KMAX>
__global__ __launch_bounds__(kGatherThreads) void dispatch_grad_kernel(DispatchGradArgs a,
                                                                       int nch) {
    constexpr int EL = gather_unit(DF32);
    const int lane = threadIdx.x % kWave;
    const int units = (int)(a.H / EL);
    const int64_t items = a.T * nch;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        int64_t t;
        int c;
        xcd_item(i, a.T, nch, t, c);
        int my_row = -1;
        if (lane < a.K) {
            const int64_t r = a.tok_map[t * a.K + lane];
            if (r >= 0 && r < a.packed_rows) my_row = (int)r;
        }
        int rows[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k) rows[k] = readlane(my_row, k);
        const int u = c * (int)blockDim.x + (int)threadIdx.x;
        if (u >= units) continue;
        const int64_t col = (int64_t)u * EL;
        FloatUnit<DF32, EL> d[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
            if (rows[k] >= 0) d[k].load(a.dpacked, (int64_t)rows[k] * a.H + col);
        float acc[EL];
#pragma unroll
        for (int j = 0; j < EL; ++j) acc[j] = 0.0f;
        if (a.residual) {
            FloatUnit<OF32, EL> r;
            r.load(a.residual, t * a.H + col);
            r.get(acc);
        }
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
            if (rows[k] < 0) continue;
            float v[EL];
            d[k].get(v);
#pragma unroll
            for (int j = 0; j < EL; ++j) acc[j] += v[j];
        }
        store_unit<OF32, true>(a.dx, t * a.H + col, acc);
    }
}

// Threads of the gather that may share a CU: more of them keep more row loads in
// flight than HBM serves well.  LDS that the launch reserves and never touches holds
// the workgroups back.  Measured uncapped -> capped: T=8192 H=7168 K=8 bf16 177.0 ->
// 174.1 us (182 at 1280 threads), with residual 197.6 -> 192.0; T=16384 H=4096 K=6
// f32 with residual 363 -> 345 us (356 at 1536 threads).
constexpr int gather_threads_per_cu(bool f32) { return f32 ? 1280 : 1536; }
constexpr int kMaxCapped = 16;   // small workgroups run uncapped
inline size_t gather_lds(bool f32, int threads) {
    const int n = gather_threads_per_cu(f32) / threads;
    return n <= kMaxCapped ? kLdsPerCu / n : 0;
}

template <bool DF32, bool OF32, int KMAX>
void dispatch_go(const DispatchGradArgs& a, hipStream_t s) {
    const int64_t units = a.H / gather_unit(DF32);
    const int threads = row_threads(units, kGatherThreads);
    const int nch = (int)((units + threads - 1) / threads);
    dispatch_grad_kernel<DF32, OF32, KMAX>
        <<<capped_grid(a.T * nch), dim3(threads), gather_lds(DF32, threads), s>>>(a, nch);
}

template <bool DF32, bool OF32>
void dispatch_by_k(const DispatchGradArgs& a, hipStream_t s) {
    if (a.K <= 2) dispatch_go<DF32, OF32, 2>(a, s);
    else if (a.K <= 4) dispatch_go<DF32, OF32, 4>(a, s);
    else if (a.K <= 8) dispatch_go<DF32, OF32, 8>(a, s);
    else dispatch_go<DF32, OF32, 16>(a, s);
}

}  // namespace

hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t s) {
    if (a.T == 0 && !(a.dy && a.packed_off)) return hipSuccess;
    switch (a.y_kind) {
        case RowKind::Bf16: combine_by_type<RowKind::Bf16>(a, s); break;
        case RowKind::F32: combine_by_type<RowKind::F32>(a, s); break;
        case RowKind::Fp8: combine_by_type<RowKind::Fp8>(a, s); break;
        case RowKind::Fp4: combine_by_type<RowKind::Fp4>(a, s); break;
    }
    return hipGetLastError();
}

hipError_t launch_dispatch_grad(const DispatchGradArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    if (a.d_f32) {
        if (a.dx_f32) dispatch_by_k<true, true>(a, s);
        else dispatch_by_k<true, false>(a, s);
    } else {
        if (a.dx_f32) dispatch_by_k<false, true>(a, s);
        else dispatch_by_k<false, false>(a, s);
    }
    return hipGetLastError();
}

}  // namespace moe
