// grad.hip - gradients of the combine and the dispatch.
//
// Combine, out[t] = sum_k w[t,k] * v[r] with r = tok_map[t,k]:
//   dy[r] = w[t,k] * dout[t],   dw[t,k] = <dout[t], v[r]> (+ dout_weights[t]).
// One wave per entry (t,k) walks the row in 64 lane-units of 8 elements: it reads
// dout[t] (which the token's other entries find in cache) and v[r], adds their
// product to the lane's f32 sum and writes w*dout to dy[r].
//
// Dispatch, packed[r] = x[t] for every entry of t: dx[t] = sum_k dpacked[r], the
// combine's gather without weights.
#include "train_device.hpp"

namespace moe {

namespace {

constexpr int kGradWaves = 4;
constexpr int kGradThreads = kGradWaves * kWave;

// Rows of dy that no entry owns: [off[e] + cnt[e], off[e+1]) of every expert, and
// [off[E], y_rows).  kGapParts workgroups share one expert's rows, kTailParts the
// rows behind the last segment.  Values outside [0, y_rows] are clamped.
constexpr int kGapParts = 8;
constexpr int kTailParts = 512;

template <bool DYF32>
__device__ __forceinline__ void zero_gap(const CombineGradArgs& a, int64_t item) {
    int64_t lo, hi;
    int parts, part;
    if (item < (int64_t)a.E * kGapParts) {
        const int e = (int)(item / kGapParts);
        parts = kGapParts;
        part = (int)(item % kGapParts);
        lo = (int64_t)a.packed_off[e] + a.packed_cnt[e];
        hi = a.packed_off[e + 1];
    } else {
        parts = kTailParts;
        part = (int)(item - (int64_t)a.E * kGapParts);
        lo = a.packed_off[a.E];
        hi = a.y_rows;
    }
    if (lo < 0) lo = 0;
    if (hi > a.y_rows) hi = a.y_rows;
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int units = (int)(a.H / 8);
    for (int64_t r = lo + part; r < hi; r += parts)
        for (int u = threadIdx.x; u < units; u += kGradThreads)
            store8<DYF32>(a.dy, r * a.H + (int64_t)u * 8, zero);
}

template <RowKind YK, bool DF32, bool DYF32>
__global__ __launch_bounds__(kGradThreads) void combine_grad_kernel(CombineGradArgs a,
                                                                    int64_t entry_blocks,
                                                                    int64_t gap_blocks) {
    const int lane = threadIdx.x % kWave;
    const int64_t n = a.T * a.K;
    const int units = (int)(a.H / 8);
    const int64_t nblk = a.H / kFp8Block;
    for (int64_t b = blockIdx.x; b < entry_blocks + gap_blocks; b += gridDim.x) {
        if (b >= entry_blocks) {
            zero_gap<DYF32>(a, b - entry_blocks);
            continue;
        }
        const int64_t e = b * kGradWaves + threadIdx.x / kWave;
        if (e >= n) continue;
        const int64_t t = e / a.K;
        const int64_t r = a.tok_map[e];
        if (r < 0 || r >= a.y_rows) {
            if (a.dw && lane == 0) a.dw[e] = 0.0f;
            continue;
        }
        const float w = a.dy ? a.w[e] : 0.0f;
        float dot = 0.0f;
        for (int u = lane; u < units; u += kWave) {
            Row8<float_kind(DF32)> d;
            d.load(a.dout, t * a.H + (int64_t)u * 8);
            Row8<YK> y;
            float scale = 1.0f;
            if (a.dw) {
                y.load(a.y, r * a.H + (int64_t)u * 8);
                if (a.y_scales) scale = a.y_scales[r * nblk + u / (kFp8Block / 8)];
            }
            float dv[8];
            d.get(dv);
            if (a.dw) {
                float yv[8];
                y.get(yv);
                if (YK == RowKind::Fp8 || YK == RowKind::Fp4) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) yv[j] = yv[j] * scale;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(dv[j], yv[j], dot);
            }
            if (a.dy) {
#pragma unroll
                for (int j = 0; j < 8; ++j) dv[j] = w * dv[j];
                store8<DYF32>(a.dy, r * a.H + (int64_t)u * 8, dv);
            }
        }
        if (a.dw) {
            const float s = wave_sum(dot);
            if (lane == 0) a.dw[e] = a.dout_weights ? s + a.dout_weights[t] : s;
        }
    }
}

template <RowKind YK, bool DF32, bool DYF32>
void combine_go(const CombineGradArgs& a, hipStream_t s) {
    const int64_t entry_blocks = (a.T * a.K + kGradWaves - 1) / kGradWaves;
    const int64_t gap_blocks =
        a.dy && a.packed_off ? (int64_t)a.E * kGapParts + kTailParts : 0;
    combine_grad_kernel<YK, DF32, DYF32><<<capped_grid(entry_blocks + gap_blocks),
                                           dim3(kGradThreads), 0, s>>>(a, entry_blocks,
                                                                       gap_blocks);
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

template <bool DF32, bool OF32>
__global__ __launch_bounds__(kGradThreads) void dispatch_grad_kernel(DispatchGradArgs a, int nch) {
    const int units = (int)(a.H / 8);
    const int64_t items = a.T * nch;
    for (int64_t wi = blockIdx.x; wi < items; wi += gridDim.x) {
        const int64_t t = wi / nch;
        const int u = (int)(wi - t * nch) * kGradThreads + threadIdx.x;
        if (u >= units) continue;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.residual) {
            Row8<float_kind(OF32)> x;
            x.load(a.residual, t * a.H + (int64_t)u * 8);
            x.get(acc);
        }
        for (int k = 0; k < a.K; ++k) {
            const int64_t r = a.tok_map[t * a.K + k];
            if (r < 0 || r >= a.packed_rows) continue;
            Row8<float_kind(DF32)> x;
            x.load(a.dpacked, r * a.H + (int64_t)u * 8);
            float v[8];
            x.get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += v[j];
        }
        store8<OF32>(a.dx, t * a.H + (int64_t)u * 8, acc);
    }
}

template <bool DF32, bool OF32>
void dispatch_go(const DispatchGradArgs& a, hipStream_t s) {
    const int nch = (int)((a.H / 8 + kGradThreads - 1) / kGradThreads);
    dispatch_grad_kernel<DF32, OF32><<<capped_grid(a.T * nch), dim3(kGradThreads), 0, s>>>(a, nch);
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
        if (a.dx_f32) dispatch_go<true, true>(a, s);
        else dispatch_go<true, false>(a, s);
    } else {
        if (a.dx_f32) dispatch_go<false, true>(a, s);
        else dispatch_go<false, false>(a, s);
    }
    return hipGetLastError();
}

}  // namespace moe
