// experts_decode.hip - the whole experts' step of a few tokens, in two kernels:
//   h[f]   = silu(W1[e] x[t]) * (W3[e] x[t])        for every entry f = t*K + k, e = idx[f]
//   out[t] = sum over k of w[t,k] * W2[e] h[t*K + k]
// There is nothing to do here but to read the weights of the experts in use once; their
// bytes over the HBM rate are the floor.  So no token row is packed or moved: each
// kernel walks the experts in use, streams their weights from HBM straight into matrix
// fragments, 16 weight rows by 16 entries, and looks its entries up.
//
// Weights are the rows of v_mfma 16x16x32 bf16: lane l holds row l % 16 and 8
// consecutive k.  MXFP4 weights are widened to bf16 in registers (e2m1 times a power of
// two is exact in bf16): lane group g = l / 16 takes block g of 4 and uses its 32 codes
// in 4 matrix steps, so its codes are one 16-byte load and its scale one byte.
//
// Up kernel: a workgroup takes (expert, 16 rows of W1 and of W3), its 4 waves a quarter of
// H each; the partial sums are joined in LDS in order of the waves, and h goes to the
// workspace.  Down kernel: a workgroup owns 16 outputs and walks all experts in use, one
// wave an expert (or a part of I where experts are few); every entry's result is kept in
// LDS and a token's are added in ascending k, as moe_combine adds them.
//
// h between the products is held in as many bf16 parts as the result can show: 2 (16 bits
// of significand) for a bf16 result, 3 (24 bits) for an f32 one.  Each part costs one
// matrix instruction per weight fragment, which these kernels have to spare.
#include <type_traits>

#include "train_device.hpp"
#include "experts.hpp"

namespace moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kUpThreads = 256, kUpWaves = kUpThreads / kWave;
constexpr int kDownThreads = 512, kDownWaves = kDownThreads / kWave;
constexpr int kMaxEntries = kDecodeEntries;

// The experts in use and their entries: expert ids[a] has entries ent[start[a]] ..
// ent[start[a+1]-1], in ascending order.
struct Lists {
    int n;
    uint16_t ids[kMaxEntries];
    uint16_t start[kMaxEntries + 1];
    uint16_t ent[kMaxEntries];
};

// Builds the lists from the ids, by the whole workgroup.  cnt and sum are scratch.
template <int THREADS>
__device__ void build_lists(const int32_t* idx, int N, int E, Lists& l, int (&cnt)[1024],
                            int (&sum)[THREADS / kWave][2]) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    for (int e = tid; e < E; e += THREADS) cnt[e] = 0;
    __syncthreads();
    constexpr int kPer = kMaxEntries / THREADS;
    int mine[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int f = tid * kPer + i;
        const int e = f < N ? idx[f] : -1;
        mine[i] = e >= 0 && e < E ? e : -1;
        if (mine[i] >= 0) atomicAdd(&cnt[mine[i]], 1);
    }
    __syncthreads();
    // exclusive sums over the experts, of "in use" and of entries
    constexpr int kPerE = 1024 / THREADS;
    int used = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kPerE; ++i) {
        const int e = tid * kPerE + i;
        const int c = e < E ? cnt[e] : 0;
        used += c > 0;
        total += c;
    }
    int u = used, t = total;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int ou = __shfl_up(u, d), ot = __shfl_up(t, d);
        if (lane >= d) {
            u += ou;
            t += ot;
        }
    }
    if (lane == kWave - 1) {
        sum[wave][0] = u;
        sum[wave][1] = t;
    }
    __syncthreads();
    int a = u - used, at = t - total, all = 0, all_ent = 0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) {
        if (i < wave) {
            a += sum[i][0];
            at += sum[i][1];
        }
        all += sum[i][0];
        all_ent += sum[i][1];
    }
#pragma unroll
    for (int i = 0; i < kPerE; ++i) {
        const int e = tid * kPerE + i;
        const int c = e < E ? cnt[e] : 0;
        if (c > 0) {
            l.ids[a] = (uint16_t)e;
            l.start[a] = (uint16_t)at;
            ++a;
        }
        if (e < E) cnt[e] = at;    // from here on: where the expert's next entry goes
        at += c;
    }
    if (tid == 0) {
        l.n = all;
        l.start[all] = (uint16_t)all_ent;
    }
    __syncthreads();
    // an entry's place among its expert's does not change any result: a column of a
    // matrix fragment does not depend on its neighbours
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (mine[i] >= 0) l.ent[atomicAdd(&cnt[mine[i]], 1)] = (uint16_t)(tid * kPer + i);
    __syncthreads();
}

// ---------------------------------------------------------------------------
// acc[r][c] += A[16 rows of tile r][k0 .. k1) * B[k0 .. k1)[16 entries of tile c], B the sum
// of P parts.  a[r]: the lane's weight row; b[c]: the lane's entry row, part p at + p*part.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ u32x4 zero4() { return u32x4{0, 0, 0, 0}; }

template <int RT, int NT, int P>
__device__ __forceinline__ void stream_bf16(f32x4 (&acc)[RT][NT], const uint16_t* (&a)[RT],
                                            const uint16_t* (&b)[NT], int64_t part, int k0, int k1) {
    constexpr int U = 8 / (RT < 2 ? 1 : RT);   // steps whose loads are in flight together
    const int g8 = (threadIdx.x % kWave) / 16 * 8;
    int k = k0;
    auto step = [&](auto n, auto guarded) {
        constexpr int STEPS = decltype(n)::value;
        constexpr bool GUARD = decltype(guarded)::value;
        u32x4 wa[STEPS][RT];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int at = k + s * 32 + g8;
                wa[s][r] = !GUARD || at < k1 ? ld16_stream(a[r] + at) : zero4();
            }
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const int at = k + s * 32 + g8;
                    const u32x4 v = !GUARD || at < k1 ? ld16(b[c] + p * part + at) : zero4();
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(wa[s][r]), as_bf16(v),
                                                                            acc[r][c], 0, 0, 0);
                }
        k += STEPS * 32;
    };
    while (k + U * 32 <= k1) step(std::integral_constant<int, U>{}, std::false_type{});
    while (k < k1) step(std::integral_constant<int, 1>{}, std::true_type{});
}

// Two e2m1 codes (byte SEL of d) times 2^(scale's exponent), as bf16.
template <int SEL>
__device__ __forceinline__ uint32_t widen2(uint32_t d, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, SEL);
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ u32x4 widen8(uint32_t d, float scale) {
    return u32x4{widen2<0>(d, scale), widen2<1>(d, scale), widen2<2>(d, scale), widen2<3>(d, scale)};
}

// a[r]: codes of the lane's weight row; sc[r]: its scales.
template <int RT, int NT, int P>
__device__ __forceinline__ void stream_mxfp4(f32x4 (&acc)[RT][NT], const uint8_t* (&a)[RT],
                                             const uint8_t* (&sc)[RT], const uint16_t* (&b)[NT],
                                             int64_t part, int k0, int k1) {
    constexpr int U = 4 / (RT < 2 ? 1 : RT);
    const int g = (threadIdx.x % kWave) / 16;
    int k = k0;
    auto step = [&](auto n, auto guarded) {
        constexpr int STEPS = decltype(n)::value;
        constexpr bool GUARD = decltype(guarded)::value;
        u32x4 codes[STEPS][RT];
        uint32_t scale[STEPS][RT];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int blk = (k >> 5) + s * 4 + g;
                const bool in = !GUARD || blk * 32 < k1;
                codes[s][r] = in ? ld16_stream(a[r] + blk * 16) : zero4();
                scale[s][r] = in ? sc[r][blk] : 0u;
            }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int at = k + s * 128 + g * 32;
            const bool in = !GUARD || at < k1;
            float f[RT];
            bool nan[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t e = scale[s][r];
                nan[r] = e == 255u;
                f[r] = __builtin_bit_cast(float, e << 23);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                u32x4 wa[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    wa[r] = widen8(codes[s][r][q], f[r]);
                    if (nan[r]) wa[r] = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
                }
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const u32x4 v = in ? ld16(b[c] + p * part + at + q * 8) : zero4();
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                as_bf16(wa[r]), as_bf16(v), acc[r][c], 0, 0, 0);
                    }
            }
        }
        k += STEPS * 128;
    };
    while (k + U * 128 <= k1) step(std::integral_constant<int, U>{}, std::false_type{});
    while (k < k1) step(std::integral_constant<int, 1>{}, std::true_type{});
}

// The lane's rows of RT tiles of 16 weight rows of [.., K], and their products with the
// entries' rows, over [k0, k1).
template <bool MX, int RT, int NT, int P>
__device__ __forceinline__ void stream(f32x4 (&acc)[RT][NT], const void* w, const uint8_t* scales,
                                       const int64_t (&row)[RT], int64_t K, const uint16_t* (&b)[NT],
                                       int64_t part, int k0, int k1) {
    if constexpr (MX) {
        const uint8_t *a[RT], *sc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            a[r] = (const uint8_t*)w + row[r] * (K / 2);
            sc[r] = scales + row[r] * (K / 32);
        }
        stream_mxfp4<RT, NT, P>(acc, a, sc, b, part, k0, k1);
    } else {
        const uint16_t* a[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) a[r] = (const uint16_t*)w + row[r] * K;
        stream_bf16<RT, NT, P>(acc, a, b, part, k0, k1);
    }
}

// Part `part` of `parts` of [0, K), in whole steps.
template <bool MX>
__device__ __forceinline__ void k_range(int64_t K, int part, int parts, int& k0, int& k1) {
    constexpr int kStep = MX ? 128 : 32;
    const int steps = (int)((K + kStep - 1) / kStep);
    const int per = (steps + parts - 1) / parts;
    const int64_t lo = (int64_t)part * per * kStep, hi = lo + (int64_t)per * kStep;
    k0 = (int)(lo < K ? lo : K);
    k1 = (int)(hi < K ? hi : K);
}

__device__ __forceinline__ float silu_of(float g) {
    // g / (1 + exp(-g)); exp overflows to an infinity below -88, where the quotient is -0
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// v as a sum of P bf16 values, each the rounding of what the ones before it left.
template <int P>
__device__ __forceinline__ void split_store(uint16_t* h, int64_t part, float v) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const __bf16 b = (__bf16)v;
        h[p * part] = __builtin_bit_cast(uint16_t, b);
        // an infinity or a NaN stands in the first part alone
        v = p == 0 && !__builtin_isfinite(v) ? 0.0f : v - (float)b;
    }
}

constexpr int kCols = 4;     // column tiles of 16 entries that are worked on together

template <bool MX, int P>
__global__ __launch_bounds__(kUpThreads) void up_kernel(DecodeArgs a, Lists* out_lists, uint16_t* h) {
    __shared__ Lists l;
    __shared__ int cnt[1024];
    __shared__ int sum[kUpWaves][2];
    __shared__ float red[kUpWaves][2][16][kCols * 16];
    const int N = (int)(a.T * a.K);
    build_lists<kUpThreads>(a.idx, N, a.E, l, cnt, sum);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < (int)(sizeof(Lists) / 4); i += kUpThreads)
            ((uint32_t*)out_lists)[i] = ((const uint32_t*)&l)[i];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t part = (int64_t)N * a.I;
    const int slices = (int)((a.I + 15) / 16);
    int k0, k1;
    k_range<MX>(a.H, wave, kUpWaves, k0, k1);
    for (int item = blockIdx.x; item < l.n * slices; item += gridDim.x) {
        const int who = item / slices, i0 = (item - who * slices) * 16;
        const int e = l.ids[who], first = l.start[who], n = l.start[who + 1] - first;
        int64_t i = i0 + lane % 16;
        if (i >= a.I) i = a.I - 1;            // rows that are not there: computed, not stored
        const int64_t row[2] = {(int64_t)e * 2 * a.I + i, (int64_t)e * 2 * a.I + a.I + i};
        auto columns = [&](auto nt, int c0) {
            constexpr int NT = decltype(nt)::value;
            const uint16_t* b[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                int col = c0 + c * 16 + lane % 16;
                if (col >= n) col = n - 1;    // columns that are not there, likewise
                b[c] = a.x + (int64_t)(l.ent[first + col] / a.K) * a.H;
            }
            f32x4 acc[2][NT] = {};
            stream<MX, 2, NT, 1>(acc, a.w13, a.s13, row, a.H, b, 0, k0, k1);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        red[wave][r][lane / 16 * 4 + q][c * 16 + lane % 16] = acc[r][c][q];
            __syncthreads();
            for (int o = threadIdx.x; o < NT * 256; o += kUpThreads) {
                const int ri = o % 16, col = o / 16;
                if (c0 + col < n && i0 + ri < a.I) {
                    float g = 0.0f, u = 0.0f;
#pragma unroll
                    for (int w = 0; w < kUpWaves; ++w) {
                        g += red[w][0][ri][col];
                        u += red[w][1][ri][col];
                    }
                    split_store<P>(h + (int64_t)l.ent[first + c0 + col] * a.I + i0 + ri, part,
                                   silu_of(g) * u);
                }
            }
            __syncthreads();
        };
        int c0 = 0;
        for (; c0 + 16 < n; c0 += kCols * 16) columns(std::integral_constant<int, kCols>{}, c0);
        if (c0 < n) columns(std::integral_constant<int, 1>{}, c0);
    }
}

template <bool MX, int P, bool F32>
__global__ __launch_bounds__(kDownThreads) void down_kernel(DecodeArgs a, const Lists* lists,
                                                            const uint16_t* h, int max_parts) {
    __shared__ Lists l;
    extern __shared__ __align__(16) float y[];     // [parts][N][16]
    const int N = (int)(a.T * a.K);
    for (int i = threadIdx.x; i < (int)(sizeof(Lists) / 4); i += kDownThreads)
        ((uint32_t*)&l)[i] = ((const uint32_t*)lists)[i];
    __syncthreads();
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t part = (int64_t)N * a.I;
    int parts = l.n > 0 ? (kDownWaves + l.n - 1) / l.n : 1;
    if (parts > max_parts) parts = max_parts;
    const int64_t h0 = (int64_t)blockIdx.x * 16;
    int64_t hr = h0 + lane % 16;
    if (hr >= a.H) hr = a.H - 1;
    for (int item = wave; item < l.n * parts; item += kDownWaves) {
        const int who = item / parts, p = item - who * parts;
        const int e = l.ids[who], first = l.start[who], n = l.start[who + 1] - first;
        const int64_t row[1] = {(int64_t)e * a.H + hr};
        int k0, k1;
        k_range<MX>(a.I, p, parts, k0, k1);
        auto columns = [&](auto nt, int c0) {
            constexpr int NT = decltype(nt)::value;
            const uint16_t* b[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                int col = c0 + c * 16 + lane % 16;
                if (col >= n) col = n - 1;
                b[c] = h + (int64_t)l.ent[first + col] * a.I;
            }
            f32x4 acc[1][NT] = {};
            stream<MX, 1, NT, P>(acc, a.w2, a.s2, row, a.I, b, part, k0, k1);
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const int col = c0 + c * 16 + lane % 16;
                if (col < n)
                    *(f32x4*)(y + ((int64_t)p * N + l.ent[first + col]) * 16 + lane / 16 * 4) = acc[0][c];
            }
        };
        int c0 = 0;
        for (; c0 + 16 < n; c0 += kCols * 16) columns(std::integral_constant<int, kCols>{}, c0);
        if (c0 < n) columns(std::integral_constant<int, 1>{}, c0);
    }
    __syncthreads();
    for (int o = threadIdx.x; o < (int)a.T * 16; o += kDownThreads) {
        const int t = o / 16, ri = o % 16;
        if (h0 + ri >= a.H) continue;
        float v = 0.0f;
        for (int k = 0; k < a.K; ++k) {
            const int f = t * a.K + k;
            const int e = a.idx[f];
            if (e < 0 || e >= a.E) continue;
            float s = y[f * 16 + ri];
            for (int p = 1; p < parts; ++p) s += y[((int64_t)p * N + f) * 16 + ri];
            v += a.w[f] * s;
        }
        const int64_t at = (int64_t)t * a.H + h0 + ri;
        if constexpr (F32) {
            ((float*)a.out)[at] = v;
        } else {
            const __bf16 b = (__bf16)v;
            ((uint16_t*)a.out)[at] = __builtin_bit_cast(uint16_t, b);
        }
    }
}

constexpr size_t kListBytes = (sizeof(Lists) + 255) / 256 * 256;
static_assert(sizeof(Lists) % 4 == 0, "copied by words");

template <bool MX, int P, bool F32>
hipError_t launch(const DecodeArgs& a, hipStream_t s) {
    const int64_t N = a.T * a.K;
    Lists* lists = (Lists*)a.ws;
    uint16_t* h = (uint16_t*)((char*)a.ws + kListBytes);
    const int64_t most = (N < a.E ? N : a.E) * ((a.I + 15) / 16);
    up_kernel<MX, P><<<dim3((unsigned)(most < 2048 ? most : 2048)), kUpThreads, 0, s>>>(a, lists, h);
    const int max_parts = (int)(kMaxEntries / N < kDownWaves ? kMaxEntries / N : kDownWaves);
    const size_t lds = (size_t)max_parts * N * 16 * sizeof(float);
    down_kernel<MX, P, F32><<<dim3((unsigned)((a.H + 15) / 16)), kDownThreads, lds, s>>>(a, lists, h,
                                                                                        max_parts);
    return hipGetLastError();
}

template <bool MX>
hipError_t launch(const DecodeArgs& a, hipStream_t s) {
    return a.out_f32 ? launch<MX, 3, true>(a, s) : launch<MX, 2, false>(a, s);
}

}  // namespace

size_t decode_ws(int64_t T, int K, int64_t I) {
    return kListBytes + (size_t)(T * K) * I * 3 * sizeof(uint16_t);
}

hipError_t launch_experts_decode(const DecodeArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    return a.s13 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
