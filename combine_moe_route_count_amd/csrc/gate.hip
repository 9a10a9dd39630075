// gate.hip - the top-k gate and its gradient.
//
// A token belongs to a group of G lanes: 64, or 16 (four tokens per wave) where its
// logits still fit the registers of 16 lanes well.  Lane l of a group holds the V
// consecutive logits [l*V, l*V + V), V the smallest power of two with G*V >= E, so
// the lowest lane that holds a value also holds its lowest expert id.  Each lane
// sorts its logits once, as ordered integer keys, equal ones by id; with 8 or 16 f32
// logits it looks for its largest instead, again after each of its own that is chosen.
// A choice is then one maximum over the heads of the group's lanes and a pop from the
// lane that had it; K choices need no memory.  The softmax follows in the same
// registers: with m the largest logit, p_j = exp(l_j - m) / sum.
//
// In this form the launch spends its time on the vector instructions of its waves, not
// on memory: T=16384 E=256 K=8 bf16 7.4 us, the bytes alone 1.6.  One round of the
// choice costs about V + 10 instructions for all tokens of the wave with a sorted list,
// several times V where the lane looks again.
#include "train_device.hpp"

namespace moe {

namespace {

constexpr int kGateWaves = 4;
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

// exp(x) for x <= 0 by the hardware's 2^y.  With u = 2^-24, y = x*log2(e) is rounded
// (|x| u relative in the result) and the constant is 0.2 u off, the power adds about
// 2 u; so small weights carry up to |x| times more error than the top one.  Rounding
// x = l - top itself costs another |x| u, where that difference is not exact.  Results
// below 2^-126 become 0.
__device__ __forceinline__ float exp_neg(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// Reductions over the group of G lanes; every lane gets the result, and a sum has one
// order.  16 lanes are one DPP row: pairs, quads, then mirrored halves.
template <int G>
struct Group;
template <>
struct Group<64> {
    template <class T>
    static __device__ __forceinline__ T max(T v) { return wave_max(v); }
    static __device__ __forceinline__ float sum(float v) { return wave_sum(v); }
    template <class T>
    static __device__ __forceinline__ T share(T v, int k) { return readlane(v, k); }
};
template <>
struct Group<16> {
    template <class T, class Op>
    static __device__ __forceinline__ T reduce(T v, Op op) {
        v = op(v, other<0xB1>(v));    // lane ^ 1
        v = op(v, other<0x4E>(v));    // lane ^ 2
        v = op(v, other<0x141>(v));   // 7 - lane, of 8
        return op(v, other<0x140>(v));   // 15 - lane
    }
    template <int CTRL, class T>
    static __device__ __forceinline__ T other(T v) {
        return __builtin_bit_cast(
            T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
    }
    static __device__ __forceinline__ int max(int v) {
        return reduce(v, [](int a, int b) { return a > b ? a : b; });
    }
    static __device__ __forceinline__ float max(float v) {
        return reduce(v, [](float a, float b) { return fmaxf(a, b); });
    }
    static __device__ __forceinline__ float sum(float v) {
        return reduce(v, [](float a, float b) { return a + b; });
    }
    template <class T>
    static __device__ __forceinline__ T share(T v, int k) { return __shfl(v, k, 16); }
};

// What a lane has left to choose from.  head() is its largest key, owns(m) whether the
// group's largest key m is this lane's head, place() which of its logits the head
// is; pop() removes it.

// bf16: the low half of a key is free for the id, inverted, so keys differ and ties
// go to the lowest id by themselves.  Sorted once by the odd-even merge network.
template <int V>
struct PackedList {
    int key[V];
    __device__ __forceinline__ PackedList(const float (&v)[V], int gl) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = (order_key(v[i]) & (int)0xffff0000) | (0xffff - (gl * V + i));
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
    template <int G>
    __device__ __forceinline__ bool owns(int m) const { return key[0] == m; }
    __device__ __forceinline__ int place() const { return (0xffff - (key[0] & 0xffff)) % V; }
    __device__ __forceinline__ void pop() {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = kTakenKey;
    }
    static __device__ __forceinline__ float value(int m) {
        return key_value(m < 0 ? m | 0xffff : m & (int)0xffff0000);
    }
};

// Whether this is the lowest lane of its group that says yes.
template <int G>
__device__ __forceinline__ bool lowest(bool yes) {
    const uint64_t all = ballot64(yes);
    if (G == 64) return yes && lanes_below(all) == 0;
    const int row = (int)(threadIdx.x % kWave) & ~(G - 1);
    const uint32_t mine = (uint32_t)(all >> row) & ((1u << G % 32) - 1u);
    return yes && (mine & ((1u << (threadIdx.x % G)) - 1u)) == 0;
}

// f32: keys fill the word.  Sorted by neighbours, which keeps equal keys in order of
// their ids, along with the places 0..V-1 they came from (4 bits each, the head's
// lowest).
template <int V>
struct FullList {
    static_assert(V <= 8, "places in one word");
    int key[V];
    uint32_t places;
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
        places = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) places = places << 4 | (uint32_t)from[i];
    }
    __device__ __forceinline__ int head() const { return key[0]; }
    template <int G>
    __device__ __forceinline__ bool owns(int m) const { return lowest<G>(key[0] == m); }
    __device__ __forceinline__ int place() const { return (int)(places & 15); }
    __device__ __forceinline__ void pop() {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = kTakenKey;
        places >>= 4;
    }
    static __device__ __forceinline__ float value(int m) { return key_value(m); }
};

// f32, 8 or 16 logits per lane: looking through them for each choice costs less than
// sorting them with their places (T=16384 E=512 K=8: 15 us, sorted 27); with 4 sorting
// does (E=256: 9.9 us, looking 11.0).
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
    template <int G>
    __device__ __forceinline__ bool owns(int m) const { return lowest<G>(best == m); }
    __device__ __forceinline__ int place() const { return at; }
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

// Tokens of the workgroup's wave, G lanes each; a wave whose last tokens are past T
// computes token T - 1 there and stores nothing, so that every lane takes part.
template <int G, int V, bool F32>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a, bool vec) {
    constexpr int kTokens = kGateThreads / G;
    const int gl = threadIdx.x % G;
    for (int64_t b = blockIdx.x; b * kTokens < a.T; b += gridDim.x) {
        const int64_t want = b * kTokens + threadIdx.x / G;
        const bool live = want < a.T;
        const int64_t t = live ? want : a.T - 1;
        float v[V];
        load_logits<V, F32>(a.logits, t, a.E, gl, vec, v);
        using Choice = typename LaneChoice<V, F32>::type;
        Choice left(v, gl);
        int my_key = kMaskedKey, top_key = kMaskedKey;   // lane k: choice k
        for (int k = 0; k < a.K; ++k) {
            const int m = Group<G>::max(left.head());
            if (gl == k) my_key = m;
            if (k == 0) top_key = m;
            if (left.template owns<G>(m) && m > kMaskedKey) {
                if (live) a.idx[t * a.K + k] = gl * V + left.place();
                left.pop();
            }
        }
        const bool some = top_key > kMaskedKey, mine = my_key > kMaskedKey && gl < a.K;
        const float top = Choice::value(top_key);
        const float e = mine ? exp_neg(Choice::value(my_key) - top) : 0.0f;
        float part = e;
        if (!a.renorm) {
            part = 0.0f;
            if (some) {
#pragma unroll
                for (int i = 0; i < V; ++i) part += exp_neg(v[i] - top);
            }
        }
        const float total = Group<G>::sum(part);
        if (gl < a.K && live) {
            if (!mine) a.idx[t * a.K + gl] = -1;
            a.w[t * a.K + gl] = mine ? (e / total) * a.scale : 0.0f;
        }
    }
}

template <int G, int V, bool F32>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(GateArgs a, bool vec) {
    constexpr int kTokens = kGateThreads / G;
    const int gl = threadIdx.x % G;
    for (int64_t b = blockIdx.x; b * kTokens < a.T; b += gridDim.x) {
        const int64_t want = b * kTokens + threadIdx.x / G;
        const bool live = want < a.T;
        const int64_t t = live ? want : a.T - 1;
        float v[V];
        if (!a.renorm) load_logits<V, F32>(a.logits, t, a.E, gl, vec, v);
        // lane k: entry k's expert, its logit and the gradient of its weight
        int j = -1;
        float l = -__builtin_inff(), dw = 0.0f;
        if (gl < a.K) {
            const int32_t id = a.idx[t * a.K + gl];
            const float g = a.dw[t * a.K + gl];
            if (id >= 0 && id < a.E) {
                l = load_logit<F32>(a.logits, t * a.E + id);
                // a masked expert's weight is 0 whatever its logit does next: its entry
                // counts as none, so a non-finite dw there reaches nobody as 0 * dw
                if (l != -__builtin_inff()) {
                    j = id;
                    dw = g;
                }
            }
        }
        float top = l;
        if (!a.renorm) {
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
        }
        top = Group<G>::max(top);
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
        float total = Group<G>::sum(part);
        if (total == 0.0f) total = 1.0f;
        const float p = e / total;
        const float d = j >= 0 ? (p * dw) * a.scale : 0.0f;
        const float dot = Group<G>::sum(d);
        const float mine = a.renorm ? d - p * dot : d;
        float g[V];
        const float all = dot / total;
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = a.renorm ? 0.0f : -(v[i] * all);
        // in order of k, so an expert named twice gets both in a fixed order
        for (int k = 0; k < a.K; ++k) {
            const int jk = Group<G>::share(j, k);
            const float x = Group<G>::share(mine, k);
            if constexpr (G == kWave) {    // one token: jk is the same in every lane
                if (jk < 0) continue;
                const float here = gl == jk / V ? x : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (jk % V == i) g[i] += here;
            } else {
                const int at = jk - gl * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (jk >= 0 && at == i) g[i] += x;
            }
        }
        if (live) store_logits<V, F32>(a.dlogits, t, a.E, gl, vec, g);
    }
}

template <int G, int V, bool F32>
void go(const GateArgs& a, bool backward, hipStream_t s) {
    constexpr int kTokens = kGateThreads / G;
    const dim3 grid = capped_grid((a.T + kTokens - 1) / kTokens), block(kGateThreads);
    const uintptr_t at = (uintptr_t)a.logits | (uintptr_t)(backward ? a.dlogits : nullptr);
    const bool vec = a.E % V == 0 && at % 16 == 0;
    if (backward) gate_backward_kernel<G, V, F32><<<grid, block, 0, s>>>(a, vec);
    else gate_kernel<G, V, F32><<<grid, block, 0, s>>>(a, vec);
}

// 16 lanes per token up to 64 logits; up to 128 f32 or 256 bf16 ones where there are
// tokens enough to fill the chip at four a wave, since the lists of 8 or 16 logits a
// lane make the single token's chain longer.  Measured, us on the GPU, 64 lanes -> 16:
//   T=16384 (a call)  bf16 E=64 7.3 -> 6.2, E=256 8.5 -> 6.1, its gradient 11.4 -> 9.4;
//                     f32 E=64 7.8 -> 6.1, E=128 8.5 -> 6.6, its gradient 9.3 -> 7.2;
//                     but f32 E=256 10.5 -> 11.2, its gradient 12.2 -> 13.5
//   T=8192            bf16 E=256 6.6 -> 5.5; f32 E=128 6.4 -> 6.1, E=16 5.7 -> 3.4
//   T=4096            bf16 E=256 4.8 -> 5.1; f32 E=128 4.8 -> 6.0, E=16 4.2 -> 3.4
//   T=512             bf16 E=256 4.0 -> 4.8; f32 E=128 4.0 -> 6.9, E=16 3.6 -> 3.3
constexpr int64_t kFewTokens = 4096;
template <bool F32>
void by_e(const GateArgs& a, bool backward, hipStream_t s) {
    const bool few = a.T <= kFewTokens;
    if (a.E <= 16) return go<16, 1, F32>(a, backward, s);
    if (a.E <= 32) return go<16, 2, F32>(a, backward, s);
    if (a.E <= 64) return go<16, 4, F32>(a, backward, s);
    if (a.E <= 128) return few ? go<64, 2, F32>(a, backward, s) : go<16, 8, F32>(a, backward, s);
    if (a.E <= 256)
        return F32 || few ? go<64, 4, F32>(a, backward, s) : go<16, 16, false>(a, backward, s);
    if (a.E <= 512) return go<64, 8, F32>(a, backward, s);
    go<64, 16, F32>(a, backward, s);
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
