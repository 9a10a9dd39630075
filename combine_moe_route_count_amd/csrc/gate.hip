// gate.hip - the top-k gate and its gradient: one wave per token.
//
// Lane l holds the V consecutive logits [l*V, l*V + V) of its token, V the
// smallest power of two with 64*V >= E, so the lowest lane that holds a value
// also holds its lowest expert id.  A choice is one wave maximum over ordered
// integer keys, one ballot for the lowest lane that has it, and one readlane for
// the place inside the lane; K choices need no memory.  The softmax follows in
// the same registers: with m the largest logit, p_j = exp(l_j - m) / sum.
#include "train_device.hpp"

namespace moe {

namespace {

constexpr int kGateWaves = 4;                       // tokens per workgroup
constexpr int kGateThreads = kGateWaves * kWave;

// f32 -> int32 so that integer order is value order: -inf lowest, -0 equal to
// +0, and every NaN above +inf.
__device__ __forceinline__ int order_key(float v) {
    if (v != v) return 0x7fffffff;
    const int b = __builtin_bit_cast(int, v + 0.0f);   // -0 + 0 = +0
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) {
    return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff));
}
constexpr int kMaskedKey = (int)0x807fffff;   // order_key(-inf)
constexpr int kTakenKey = (int)0x80000000;

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if (F32) return ((const float*)p)[i];
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
}

// The lane's V logits; -inf for ids past E.
template <int V, bool F32>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int lane,
                                            float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = lane * V + i;
        v[i] = j < E ? load_logit<F32>(logits, t * E + j) : -__builtin_inff();
    }
}

template <int V, bool F32>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a) {
    const int lane = threadIdx.x % kWave;
    const int64_t step = (int64_t)gridDim.x * kGateWaves;
    for (int64_t t = (int64_t)blockIdx.x * kGateWaves + threadIdx.x / kWave; t < a.T; t += step) {
        float v[V];
        load_logits<V, F32>(a.logits, t, a.E, lane, v);
        int key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = order_key(v[i]);
        int my_idx = -1, my_key = kMaskedKey;    // lane k: choice k
        for (int k = 0; k < a.K; ++k) {
            int best = key[0], at = 0;
#pragma unroll
            for (int i = 1; i < V; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i;
                }
            const int m = wave_max(best);
            if (m <= kMaskedKey) break;          // the same in every lane
            const int owner = __builtin_ctzll(ballot64(best == m));
            const int j = owner * V + readlane(at, owner);
            if (lane == k) {
                my_idx = j;
                my_key = m;
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane == owner && i == at) key[i] = kTakenKey;
        }
        const float top = key_value(readlane(my_key, 0));
        float e = my_idx >= 0 ? expf(key_value(my_key) - top) : 0.0f;
        float part = e;
        if (!a.renorm) {
            part = 0.0f;
            if (readlane(my_idx, 0) >= 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) part += expf(v[i] - top);
            }
        }
        const float total = wave_sum(part);
        if (lane < a.K) {
            a.idx[t * a.K + lane] = my_idx;
            a.w[t * a.K + lane] = my_idx >= 0 ? (e / total) * a.scale : 0.0f;
        }
    }
}

template <int V, bool F32>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(GateArgs a) {
    const int lane = threadIdx.x % kWave;
    const int64_t step = (int64_t)gridDim.x * kGateWaves;
    for (int64_t t = (int64_t)blockIdx.x * kGateWaves + threadIdx.x / kWave; t < a.T; t += step) {
        // lane k: entry k's expert, its logit and the gradient of its weight
        int j = -1;
        float l = -__builtin_inff(), dw = 0.0f;
        if (lane < a.K) {
            const int32_t id = a.idx[t * a.K + lane];
            const float g = a.dw[t * a.K + lane];
            if (id >= 0 && id < a.E) {
                j = id;
                dw = g;
                l = load_logit<F32>(a.logits, t * a.E + id);
            }
        }
        float v[V];
        float top = l;
        if (!a.renorm) {
            load_logits<V, F32>(a.logits, t, a.E, lane, v);
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
        }
        top = wave_max(top);
        if (top == -__builtin_inff()) top = 0.0f;      // nothing to choose from: exp gives 0
        const float e = j >= 0 ? expf(l - top) : 0.0f;
        float part = e;
        if (!a.renorm) {
            part = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = expf(v[i] - top);
                part += v[i];
            }
        }
        float total = wave_sum(part);
        if (total == 0.0f) total = 1.0f;
        const float p = e / total;
        const float d = j >= 0 ? (p * dw) * a.scale : 0.0f;
        const float dot = wave_sum(d);
        const float mine = a.renorm ? d - p * dot : d;
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = a.renorm ? 0.0f : -((v[i] / total) * dot);
        for (int k = 0; k < a.K; ++k) {
            const int jk = readlane(j, k);
            if (jk < 0) continue;
            const float x = readlane(mine, k);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i == jk) g[i] += x;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int jj = lane * V + i;
            if (jj >= a.E) continue;
            if (F32) ((float*)a.dlogits)[t * a.E + jj] = g[i];
            else ((uint16_t*)a.dlogits)[t * a.E + jj] = __builtin_bit_cast(uint16_t, (__bf16)g[i]);
        }
    }
}

template <int V, bool F32>
void go(const GateArgs& a, bool backward, hipStream_t s) {
    const dim3 grid = capped_grid((a.T + kGateWaves - 1) / kGateWaves), block(kGateThreads);
    if (backward) gate_backward_kernel<V, F32><<<grid, block, 0, s>>>(a);
    else gate_kernel<V, F32><<<grid, block, 0, s>>>(a);
}

template <bool F32>
void by_e(const GateArgs& a, bool backward, hipStream_t s) {
    if (a.E <= 64) go<1, F32>(a, backward, s);
    else if (a.E <= 128) go<2, F32>(a, backward, s);
    else if (a.E <= 256) go<4, F32>(a, backward, s);
    else if (a.E <= 512) go<8, F32>(a, backward, s);
    else go<16, F32>(a, backward, s);
}

hipError_t launch(const GateArgs& a, bool backward, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    if (a.f32) by_e<true>(a, backward, s);
    else by_e<false>(a, backward, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t s) { return launch(a, false, s); }
hipError_t launch_gate_backward(const GateArgs& a, hipStream_t s) { return launch(a, true, s); }

}  // namespace moe
