// gate.hip - the top-k gate and its gradient: one wave per token.
//
// Lane l holds the V consecutive logits [l*V, l*V + V) of its token, V the smallest
// power of two with 64*V >= E, so the lowest lane that holds a value also holds its
// lowest expert id.  Each lane sorts its logits once, as ordered integer keys, equal
// ones by id.  A choice is then one wave maximum over the lanes' heads and a pop of
// the list it came from; K choices need no memory.  The softmax follows in the same registers: with m the largest logit,
// p_j = exp(l_j - m) / sum.
//
// The launch is bound by the vector instructions of its waves, not by memory.
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

// The lane's V logits; -inf for ids past E.  VEC: E % V == 0 and the rows are aligned
// for it, so a lane's logits are whole vectors.
template <int V, bool F32>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int lane,
                                            bool vec, float (&v)[V]) {
    const int64_t first = t * E + lane * V;
    if (V * (F32 ? 4 : 2) >= 8 && vec) {
        constexpr int W = V * (F32 ? 4 : 2) / 4 > 0 ? V * (F32 ? 4 : 2) / 4 : 1;   // words
        uint32_t w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = F32 ? 0xff800000u : 0xff80ff80u;
        if (lane * V < E) {
            const char* p = (const char*)logits + first * (F32 ? 4 : 2);
            if constexpr (W >= 4) {
#pragma unroll
                for (int h = 0; h < W / 4; ++h) {
                    const u32x4 a = ld16(p + 16 * h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[4 * h + j] = a[j];
                }
            } else if constexpr (W == 2) {
                const u32x2 a = *(const u32x2*)p;
                w[0] = a[0];
                w[1] = a[1];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (F32) v[i] = __builtin_bit_cast(float, w[i % W]);
            else v[i] = (i & 1) ? bf16hi(w[i / 2 % W]) : bf16lo(w[i / 2 % W]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = lane * V + i < E ? load_logit<F32>(logits, first + i) : -__builtin_inff();
}

template <int V, bool F32>
__device__ __forceinline__ void store_logits(void* out, int64_t t, int E, int lane, bool vec,
                                             const float (&v)[V]) {
    const int64_t first = t * E + lane * V;
    if constexpr (V >= 4) {
        if (vec) {
            if (lane * V < E) {
#pragma unroll
                for (int h = 0; h < V; h += 4) {
                    const float part[4] = {v[h], v[h + 1], v[h + 2], v[h + 3]};
                    store_unit<F32, false, 4>(out, first + h, part);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (lane * V + i >= E) continue;
        if (F32) ((float*)out)[first + i] = v[i];
        else ((uint16_t*)out)[first + i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    }
}

// exp(x) for x <= 0 by the hardware's 2^y: rounding y = x*log2(e) costs |x| * 2^-24
// relative, as much as rounding x itself; results below 2^-126 become 0.
__device__ __forceinline__ float exp_neg(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// What a lane has left to choose from.  head() is its largest key; find() says which
// expert the wave's largest key m is and whether it is this lane's; pop() removes
// this lane's head.

// bf16: the low half of a key is free for the id, inverted, so keys differ and ties
// go to the lowest id by themselves.  Sorted once by the odd-even merge network.
template <int V>
struct PackedList {
    int key[V];
    __device__ __forceinline__ PackedList(const float (&v)[V], int lane) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = (order_key(v[i]) & (int)0xffff0000) | (0xffff - (lane * V + i));
#pragma unroll
        for (int p = 1; p < V; p <<= 1)
#pragma unroll
            for (int k = p; k > 0; k >>= 1)
#pragma unroll
                for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                    for (int i = 0; i < k; ++i)
                        if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            const int x = key[i + j], y = key[i + j + k];
                            key[i + j] = x > y ? x : y;
                            key[i + j + k] = x > y ? y : x;
                        }
    }
    __device__ __forceinline__ int head() const { return key[0]; }
    __device__ __forceinline__ bool find(int m, int lane, int& expert) const {
        expert = 0xffff - (m & 0xffff);
        return key[0] == m;
    }
    __device__ __forceinline__ void pop() {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = kTakenKey;
    }
    static __device__ __forceinline__ float value(int m) {
        return key_value(m < 0 ? m | 0xffff : m & (int)0xffff0000);
    }
};

// f32: keys fill the word.  Sorted by neighbours, which keeps equal keys in order of
// their ids, along with the places 0..V-1 they came from (4 bits each, the head's
// lowest).
template <int V>
struct FullList {
    static_assert(V <= 8, "places in one word");
    int key[V];
    uint32_t place;
    __device__ __forceinline__ FullList(const float (&v)[V], int) {
        int from[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = order_key(v[i]);
            from[i] = i;
        }
#pragma unroll
        for (int i = 1; i < V; ++i) {
#pragma unroll
            for (int j = i; j > 0; --j) {
                const bool up = key[j] > key[j - 1];
                const int hi = up ? key[j] : key[j - 1], lo = up ? key[j - 1] : key[j];
                const int fh = up ? from[j] : from[j - 1], fl = up ? from[j - 1] : from[j];
                key[j - 1] = hi;
                key[j] = lo;
                from[j - 1] = fh;
                from[j] = fl;
            }
        }
        place = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) place = place << 4 | (uint32_t)from[i];
    }
    __device__ __forceinline__ int head() const { return key[0]; }
    __device__ __forceinline__ bool find(int m, int lane, int& expert) const {
        const int owner = __builtin_ctzll(ballot64(key[0] == m));
        expert = owner * V + (int)(readlane(place, owner) & 15);
        return lane == owner;
    }
    __device__ __forceinline__ void pop() {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = kTakenKey;
        place >>= 4;
    }
    static __device__ __forceinline__ float value(int m) { return key_value(m); }
};

// f32, more than 8 logits per lane: looking through them for each choice costs less
// than sorting them.
template <int V>
struct FullScan {
    int key[V];
    int best, at;
    __device__ __forceinline__ FullScan(const float (&v)[V], int) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = order_key(v[i]);
        look();
    }
    __device__ __forceinline__ void look() {
        best = key[0];
        at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
    }
    __device__ __forceinline__ int head() const { return best; }
    __device__ __forceinline__ bool find(int m, int lane, int& expert) const {
        const int owner = __builtin_ctzll(ballot64(best == m));
        expert = owner * V + readlane(at, owner);
        return lane == owner;
    }
    __device__ __forceinline__ void pop() {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i == at) key[i] = kTakenKey;
        look();
    }
    static __device__ __forceinline__ float value(int m) { return key_value(m); }
};

template <int V, bool F32>
struct LaneChoice {
    using type = PackedList<V>;
};
template <int V>
struct LaneChoice<V, true> {
    using type = FullList<V>;
};
template <>
struct LaneChoice<8, true> {
    using type = FullScan<8>;
};
template <>
struct LaneChoice<16, true> {
    using type = FullScan<16>;
};

template <int V, bool F32>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a, bool vec) {
    const int lane = threadIdx.x % kWave;
    const int64_t step = (int64_t)gridDim.x * kGateWaves;
    for (int64_t t = (int64_t)blockIdx.x * kGateWaves + threadIdx.x / kWave; t < a.T; t += step) {
        float v[V];
        load_logits<V, F32>(a.logits, t, a.E, lane, vec, v);
        using Choice = typename LaneChoice<V, F32>::type;
        Choice left(v, lane);
        int my_idx = -1, my_key = kMaskedKey;    // lane k: choice k
        for (int k = 0; k < a.K; ++k) {
            const int m = wave_max(left.head());
            if (m <= kMaskedKey) break;          // the same in every lane
            int expert;
            const bool mine = left.find(m, lane, expert);
            if (lane == k) {
                my_idx = expert;
                my_key = m;
            }
            if (mine) left.pop();
        }
        const float top = Choice::value(readlane(my_key, 0));
        const float e = my_idx >= 0 ? exp_neg(Choice::value(my_key) - top) : 0.0f;
        float part = e;
        if (!a.renorm) {
            part = 0.0f;
            if (readlane(my_idx, 0) >= 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) part += exp_neg(v[i] - top);
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
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(GateArgs a, bool vec) {
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
            load_logits<V, F32>(a.logits, t, a.E, lane, vec, v);
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
        }
        top = wave_max(top);
        if (top == -__builtin_inff()) top = 0.0f;      // nothing to choose from: exp gives 0
        const float e = j >= 0 ? exp_neg(l - top) : 0.0f;
        float part = e;
        if (!a.renorm) {
            part = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = exp_neg(v[i] - top);
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
        // in order of k, so an expert named twice gets both in a fixed order
        for (int k = 0; k < a.K; ++k) {
            const int jk = readlane(j, k);
            if (jk < 0) continue;
            const float x = readlane(mine, k);
            if (lane != jk / V) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == jk % V) g[i] += x;
        }
        store_logits<V, F32>(a.dlogits, t, a.E, lane, vec, g);
    }
}

template <int V, bool F32>
void go(const GateArgs& a, bool backward, hipStream_t s) {
    const dim3 grid = capped_grid((a.T + kGateWaves - 1) / kGateWaves), block(kGateThreads);
    const uintptr_t at = (uintptr_t)a.logits | (uintptr_t)(backward ? a.dlogits : nullptr);
    const bool vec = a.E % V == 0 && at % 16 == 0;
    if (backward) gate_backward_kernel<V, F32><<<grid, block, 0, s>>>(a, vec);
    else gate_kernel<V, F32><<<grid, block, 0, s>>>(a, vec);
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
