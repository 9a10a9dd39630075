// experts_decode.hip - the whole experts' step of a few tokens:
//   h[f]   = silu(W1[e] x[t]) * (W3[e] x[t])        for every entry f = t*K + k, e = idx[f]
//   y[f]   = W2[e] h[f]
//   out[t] = sum over k of w[t,k] * y[t*K + k]
// There is nothing to do here but to read the weights of the experts in use once; their
// bytes over the HBM rate are the floor.  So no token row is packed or moved: the two
// products walk the experts in use, 32 weight rows of a wave by 16 entries (or 32) at a
// time, and look their entries up; a short third kernel adds a token's results.
//
// Weights are the rows of v_mfma 16x16x32 bf16: lane l holds row l % 16 and 8 consecutive
// k.  MXFP4 weights are widened to bf16 in registers (e2m1 times a power of two is exact
// in bf16): lane group g = l / 16 takes block g of 4 and uses its 32 codes in 4 matrix
// steps.
//
// K runs in stages of 64 elements (MXFP4: 128 or 256): weight rows and the entries' rows go
// straight into LDS, four stages deep, so that three are in flight while one is used.  What
// runs dry costs most here, so the stages of a workgroup's items (expert, weight rows)
// form one stream: the last stages of an item are used while the first of the next one
// are on their way.  Items have the same number of stages, filled up to a multiple of four
// with stages of zeros, so that every LDS buffer is a fixed one in the code.  Where items
// are few, the waves of a workgroup take the same weight rows of W1 and W3 and a quarter of K
// each, and their sums are added in LDS.
//
// h between the products is held in as many bf16 parts as the result can show: 2 (16 bits
// of significand) for a bf16 result, 3 (24 bits) for an f32 one.  With a third
// part one bf16 result in some hundreds would be its neighbour, and the relative error against 64
// bits is 0.0017 with either; it costs 53 -> 63 us (one token, bf16), 293 -> 315 (128 tokens, MXFP4).
// Each part is one matrix instruction per weight fragment and LDS for its rows.  MXFP4 weights
// must be widened too and leave less room: where experts have few entries the parts are
// columns of one instruction, and the columns of an entry are added at the end.
//
// Measured, bytes of the weights in use over the time: one token and bf16 weights of 8
// experts, 1024 x 6144, 54 us, 5.6 TB/s; 32 tokens and MXFP4 weights of 111 experts, 1024 x
// 7168, 225 to 237 us, 5.5 to 5.8 TB/s; bf16, 1024 x 4096, 476 to 481 us, 5.8 TB/s.
#include <type_traits>

#include "train_device.hpp"
#include "experts_device.hpp"
#include "internal.hpp"

namespace moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

using Lds = __attribute__((address_space(3))) uint8_t;
using LdsWords = __attribute__((address_space(3))) u32x4;

constexpr int kMaxEntries = kDecodeEntries;
constexpr int kGroup = 4;      // stages in LDS
constexpr float kBf16Max = 0x1.fep127f;

// A block of lists (ListLayout), sized by the number of entries, so that few of them leave the LDS
// to the stages.
struct Lists {
    uint16_t *n, *expert, *first, *ent;
    __device__ __forceinline__ Lists(uint16_t* base, int N)
        : n(base), expert(base + ListLayout{N}.expert()), first(base + ListLayout{N}.first()),
          ent(base + ListLayout{N}.ent()) {}
};
constexpr size_t kListBytes = (ListLayout{kMaxEntries}.words32() * 4 + 255) / 256 * 256;

// Scratch of build_lists: how many entries of each expert a chunk of 64 entries has (16
// chunks, 64 at the most), in four arrays of 256 experts each, and sums of the waves.
struct ListScratch {
    static constexpr int kChunks = kMaxEntries / kWave;
    static constexpr int kExperts = 256;
    Lds *count0, *count1, *count2, *count3;
    int (*sum)[2];
    __device__ __forceinline__ Lds* of(int e) const {
        Lds* low = e < kExperts ? count0 : count1;
        Lds* high = e < 3 * kExperts ? count2 : count3;
        return (e < 2 * kExperts ? low : high) + e % kExperts * kChunks;
    }
};

// Builds the lists from the ids, by the whole workgroup; entries of an expert in ascending
// order, the same in every workgroup.  Each wave finds the ranks of entries in its chunks; where
// a chunk's entries go follows from the counts of the chunks before it.
template <int THREADS>
__device__ void build_lists(const int32_t* idx, int N, int E, int width, const Lists& l,
                            const ListScratch& sc, uint16_t* start) {
    constexpr int kWaves = THREADS / kWave, kPer = ListScratch::kChunks / kWaves;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    int e[kPer], rank[kPer], same[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int f = (i * kWaves + wave) * kWave + lane;
        e[i] = f < N ? idx[f] : -1;
        if (e[i] >= E || e[i] < 0) e[i] = -1;
    }
    for (int i = tid; i < E; i += THREADS) *(LdsWords*)sc.of(i) = u32x4{0, 0, 0, 0};
    const int bits = E > 1 ? 32 - __builtin_clz(E - 1) : 1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint64_t lanes = match_key(e[i], bits);
        rank[i] = lanes_below(lanes);
        same[i] = __popcll(lanes);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (e[i] >= 0 && rank[i] == 0) sc.of(e[i])[i * kWaves + wave] = (uint8_t)same[i];
    __syncthreads();
    auto entries = [](u32x4 v) {
        uint32_t n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) n = __builtin_amdgcn_sad_u8(v[j], 0u, n);
        return (int)n;
    };
    // exclusive sums over the experts, of slots and of entries
    constexpr int kPerE = 1024 / THREADS;
    const int per = (E + THREADS - 1) / THREADS;       // experts of a thread
    int cnt[kPerE], slots = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kPerE; ++i) {
        const int x = tid * per + i;
        cnt[i] = i < per && x < E ? entries(*(const LdsWords*)sc.of(x)) : 0;
        slots += (cnt[i] + width - 1) / width;
        total += cnt[i];
    }
    int u = slots, t = total;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int ou = __shfl_up(u, d), ot = __shfl_up(t, d);
        if (lane >= d) {
            u += ou;
            t += ot;
        }
    }
    if (lane == kWave - 1) {
        sc.sum[wave][0] = u;
        sc.sum[wave][1] = t;
    }
    __syncthreads();
    int a = u - slots, at = t - total, all = 0, used = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i < wave) {
            a += sc.sum[i][0];
            at += sc.sum[i][1];
        }
        all += sc.sum[i][0];
        used += sc.sum[i][1];
    }
#pragma unroll
    for (int i = 0; i < kPerE; ++i) {
        const int x = tid * per + i;
        if (cnt[i] == 0) continue;
        for (int j = 0; j < cnt[i]; j += width) {
            l.expert[a] = (uint16_t)x;
            l.first[a] = (uint16_t)(at + j);
            ++a;
        }
        start[x] = (uint16_t)at;
        at += cnt[i];
    }
    if (tid == 0) {
        *l.n = (uint16_t)all;
        l.first[all] = (uint16_t)used;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (e[i] < 0) continue;
        u32x4 before = *(const LdsWords*)sc.of(e[i]);
        const int c = i * kWaves + wave;               // chunks from c on do not count
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int bytes = min(max(c - 4 * j, 0), 4);
            before[j] = bytes == 4 ? before[j] : before[j] & ((1u << (8 * bytes)) - 1);
        }
        l.ent[start[e[i]] + entries(before) + rank[i]] = (uint16_t)((i * kWaves + wave) * kWave + lane);
    }
    __syncthreads();
}

// The same for at most 64 entries, by one wave on its own (experts in the order of their
// first entries): the barriers of build_lists and its passes over the experts' counts cost 4 us
// more.
__device__ void build_short_lists(const int32_t* idx, int N, int E, int width, const Lists& l) {
    const int lane = threadIdx.x % kWave;
    int e = lane < N ? idx[lane] : -1;
    if (e >= E || e < 0) e = -1;
    const uint64_t same = match_key(e, E > 1 ? 32 - __builtin_clz(E - 1) : 1);
    const int rank = lanes_below(same), cnt = __popcll(same);
    const bool leads = e >= 0 && rank == 0;
    const int mine = leads ? (cnt + width - 1) / width << 16 | cnt : 0;    // slots, entries
    int upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    const int before = upto - mine, all = readlane(upto, kWave - 1);
    if (leads)
        for (int j = 0; j < cnt; j += width) {
            const int a = (before >> 16) + j / width;
            l.expert[a] = (uint16_t)e;
            l.first[a] = (uint16_t)((before & 0xffff) + j);
        }
    const int at = __shfl(before & 0xffff, e >= 0 ? __builtin_ctzll(same) : 0);
    if (e >= 0) l.ent[at + rank] = (uint16_t)lane;
    if (lane == 0) {
        *l.n = (uint16_t)(all >> 16);
        l.first[all >> 16] = (uint16_t)(all & 0xffff);
    }
}

// The lists of a product that takes fewer entries at a time, `width`, from those at hand.
__device__ void write_lists(const Lists& l, int width, const Lists& out) {
    const int lane = threadIdx.x % kWave, n = *l.n, used = l.first[n];
    for (int i = threadIdx.x; i < used; i += blockDim.x) out.ent[i] = l.ent[i];
    if (threadIdx.x >= kWave) return;
    int base = 0;
    for (int c = 0; c < n; c += kWave) {
        const int s = c + lane;
        const int first = s < n ? l.first[s] : 0, cnt = s < n ? l.first[s + 1] - first : 0;
        const int mine = (cnt + width - 1) / width;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        for (int j = 0; j < mine; ++j) {
            out.expert[base + upto - mine + j] = l.expert[s];
            out.first[base + upto - mine + j] = (uint16_t)(first + j * width);
        }
        base += readlane(upto, kWave - 1);
    }
    if (lane == 0) {
        *out.n = (uint16_t)base;
        out.first[base] = (uint16_t)used;
    }
}

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

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

// 64 x 16 bytes into LDS.  ONCE: the line is not wanted again (nt).
template <bool ONCE>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (Lds*)lds, 16, (int)off, 0, 0, ONCE ? 2 : 0);
}

// One of the two products.  UP: the rows are those of W1 and W3, a wave has 16 of each, the
// other factor is x (one part); else they are those of W2, 32 of a wave, times the P
// parts of h.  NT: 16 entries per wave and pass times NT.  SK: elements of a stage.
// SPLIT: all waves have the same rows, each its own stretch of K, and their sums are added.
// PACK: the parts of h are columns of their own, 16 / P entries at a time, and the columns
// of an entry are added at the end.
template <bool MX, bool UP, int P, int NT, int SK, int WAVES, bool SPLIT, bool PACK>
struct Stream {
    static_assert(!PACK || (!UP && NT == 1 && !SPLIT), "parts as columns");
    static constexpr int kWidth = PACK ? 16 / P : 16 * NT;      // entries at a time
    static constexpr int kParts = PACK ? 1 : P;                 // of the stages in LDS
    static constexpr int kThreads = WAVES * kWave;
    static constexpr int kStageK = SK;
    static constexpr int kRowBytes = MX ? SK / 2 : SK * 2;      // of a weight row in a stage
    static constexpr bool kLine = kRowBytes == 128;             // a cache line
    static constexpr int kWords = MX ? SK / 128 * kGroup : 4;   // of scales, 4 blocks each, of a group
    static constexpr int kRowChunks = kRowBytes / 16;
    static constexpr int kRowsPer = kWave / kRowChunks;         // weight rows per load
    static constexpr int kLoadsW = 32 / kRowsPer;
    static constexpr int kColChunks = kStageK / 8;              // 16-byte chunks of an entry's row
    static constexpr int kColsPer = kWave / kColChunks;
    static constexpr int kColLoads = 16 * NT / kColsPer;        // loads of one part of all entries
    static constexpr int kLoadsB = SPLIT ? kColLoads : (kColLoads + WAVES - 1) / WAVES;   // of a wave and part
    static constexpr int kPart = 16 * NT * kColChunks * 16;
    static constexpr int kW = WAVES * 32 * kRowBytes;
    static constexpr int kStageBytes = kW + (SPLIT ? WAVES : 1) * kParts * kPart;
    static constexpr int kRows = (SPLIT ? 1 : WAVES) * (UP ? 16 : 32);    // output rows of an item
    static constexpr int kLoads = kLoadsW + kParts * kLoadsB;        // of a wave for a stage
    // waves on a SIMD, as far as the LDS lets the compiler count on them
    static constexpr int kPerSimd = kLdsPerCu / (kGroup * kStageBytes) * WAVES >= 8 ? 2 : 1;
    static_assert(kRowBytes == 128 || kRowBytes == 64, "whole or half cache lines");
};

// Where the stream is: the first weight row of an item and how many there are, and the
// offsets of the entries' rows that the calling lane loads.
template <int LB>
struct Cursor {
    int64_t row;
    int rows;
    uint32_t col[LB];
};

// down_width: entries that the second product takes at a time.  ONCE: a stage of a weight row
// is a cache line, which is not wanted again.
template <bool MX, bool UP, int P, int NT, int SK, int WAVES, bool SPLIT, bool PACK, bool ONCE>
__global__ __launch_bounds__(WAVES * 64, (Stream<MX, UP, P, NT, SK, WAVES, SPLIT, PACK>::kPerSimd))
void stream_kernel(DecodeArgs a, uint32_t* lists, int down_width, uint16_t* h, int64_t h_part, float* y, int h_parts) {
    using S = Stream<MX, UP, P, NT, SK, WAVES, SPLIT, PACK>;
    constexpr int kThreads = S::kThreads, kParts = S::kParts;
    extern __shared__ __align__(16) uint32_t list_block[];
    __shared__ __align__(16) uint8_t lds0[S::kStageBytes], lds1[S::kStageBytes];
    __shared__ __align__(16) uint8_t lds2[S::kStageBytes], lds3[S::kStageBytes];
    __shared__ f32x4 sums[SPLIT ? (WAVES - 1) * 2 * NT * kWave : 1];     // of all waves but the first
    const int N = (int)(a.T * a.K);
    const Lists l((uint16_t*)list_block, N);
    if constexpr (UP) {
        // the scratch of the lists is in the stages' space, which is not in use yet
        constexpr int kCounts = ListScratch::kExperts * ListScratch::kChunks;
        static_assert(kCounts + 2048 <= S::kStageBytes, "scratch");
        const ListScratch scratch{(Lds*)lds0, (Lds*)lds1, (Lds*)lds2, (Lds*)lds3, (int(*)[2])(lds1 + kCounts)};
        if (N > kWave) {
            build_lists<kThreads>(a.idx, N, a.E, 16 * NT, l, scratch, (uint16_t*)(lds0 + kCounts));
        } else {
            if (threadIdx.x < kWave) build_short_lists(a.idx, N, a.E, 16 * NT, l);
            __syncthreads();
        }
        if (blockIdx.x == gridDim.x - 1) {        // has nothing else to do
            write_lists(l, down_width, Lists((uint16_t*)lists, N));
            return;
        }
    } else {
        // (lists that another call on the same workspace has overwritten give wrong results, but
        // no index or address out of range)
        const ListLayout lay{N};
        for (int i = threadIdx.x; i < lay.words32(); i += kThreads) {
            const uint32_t v = lists[i];
            list_block[i] = lay.bounded(2 * i, v & 0xffffu, a.E) | lay.bounded(2 * i + 1, v >> 16, a.E) << 16;
        }
        __syncthreads();
    }
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t K = UP ? a.H : a.I, M = UP ? a.I : a.H;     // sum length, output rows of an expert
    const int blocks = (int)((M + S::kRows - 1) / S::kRows);
    const int items = __builtin_amdgcn_readfirstlane((int)*l.n) * blocks;
    const int workers = (int)gridDim.x - (UP ? 1 : 0);
    const int chunks = (int)(MX ? K / 32 : K / 8), col_chunks = (int)(K / 8);
    constexpr int kGroupK = S::kStageK * kGroup * (SPLIT ? WAVES : 1);
    const int groups = (int)((K + kGroupK - 1) / kGroupK);      // of a wave
    const int row_wave = SPLIT ? 0 : wave;                      // by rows, and by stretches of K
    const int k_wave = SPLIT ? wave : 0;
    const int64_t rb = MX ? K / 2 : K * 2, wrows = UP ? 2 * M : M;

    auto item_rows = [&](int item, int& slot) {
        slot = item / blocks;
        return (int64_t)(item - slot * blocks) * S::kRows;
    };
    auto seek = [&](int item, Cursor<S::kLoadsB>& c) {
        int slot;
        const int64_t r0 = item_rows(item, slot);
        const int e = __builtin_amdgcn_readfirstlane((int)l.expert[slot]);
        const int first = __builtin_amdgcn_readfirstlane((int)l.first[slot]);
        const int n = __builtin_amdgcn_readfirstlane((int)l.first[slot + 1]) - first;
        c.row = (int64_t)e * wrows + r0;
        c.rows = (int)(M - r0 < S::kRows ? M - r0 : S::kRows);
#pragma unroll
        for (int i = 0; i < S::kLoadsB; ++i) {
            const int col = (row_wave * S::kLoadsB + i) % S::kColLoads * S::kColsPer + lane / S::kColChunks;
            // (of PACK, column col is part col / width of entry col % width)
            const int part = PACK ? col / S::kWidth : 0, of = PACK ? col % S::kWidth : col;
            const bool none = of >= n || part >= P;
            const int f = l.ent[none ? 0 : first + of];
            const int64_t row = (UP ? f / a.K : f) + (int64_t)(none ? 0 : part) * N;
            c.col[i] = (uint32_t)(row * K * 2) | outside_if(none);
        }
    };
    // Stage s of an item into LDS.  A row's chunks stand at chunk ^ row bits, so that 8 lanes
    // that read one chunk of 8 rows meet different banks.
    const void* weights = UP ? a.w13 : a.w2;
    auto load_stage = [&](uint8_t* lds, const Cursor<S::kLoadsB>& c, int s) {
        s += k_wave * groups * kGroup;
        const auto first = rows_of(weights, c.row, c.rows, rb);
        const auto second = UP ? rows_of(weights, c.row + M, c.rows, rb) : first;
#pragma unroll
        for (int i = 0; i < S::kLoadsW; ++i) {
            const int r = i * S::kRowsPer + lane / S::kRowChunks;     // of the wave's 32
            const int at = s * S::kRowChunks + ((lane % S::kRowChunks) ^ (S::kLine ? r % 8 : r / 2 % 4));
            const int row = UP ? row_wave * 16 + r % 16 : row_wave * 32 + r;
            to_lds<ONCE>(UP && i * S::kRowsPer >= 16 ? second : first, lds + (wave * 32 + i * S::kRowsPer) * S::kRowBytes,
                   ((uint32_t)row * (uint32_t)rb + (uint32_t)at * 16) | outside_if(at >= chunks));
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const auto src = UP ? rows_of(a.x, 0, a.T, K * 2)
                                : rows_of(h + p * h_part, 0, PACK ? (int64_t)N * P : N, K * 2);
#pragma unroll
            for (int i = 0; i < S::kLoadsB; ++i) {
                const int load = (row_wave * S::kLoadsB + i) % S::kColLoads;
                const int col = load * S::kColsPer + lane / S::kColChunks;
                const int at = s * S::kColChunks + ((lane % S::kColChunks) ^ (col % 8));
                to_lds<false>(src, lds + S::kW + (k_wave * kParts + p) * S::kPart + load * 1024,
                       (c.col[i] + (uint32_t)at * 16) | outside_if(at >= col_chunks));
            }
        }
    };
    // 64 bytes of a row's scales are loaded together (in smaller pieces their cache lines are
    // long gone when the next piece is wanted), 16 by each of the row's four lanes.  They
    // are those of kPerLoad groups of stages; of the group at hand every lane takes a copy:
    // byte g of word i is that of the lane's block in the group's i-th 128 elements.  Rows
    // start at any byte; 16 bytes that would reach behind the item's last row are read
    // that much earlier, and moved when they are taken (a move here would wait for them).
    const int r = lane % 16, g = lane / 16;
    const int nblk = (int)(K / 32);
    constexpr int kPerLoad = 16 / S::kWords;
    u32x4 next_scale[2] = {};
    int next_move[2] = {}, next_valid = 0;     // bytes to drop in front, bytes of the row behind them
    auto load_scales = [&](const Cursor<S::kLoadsB>& c, int group) {
        if constexpr (MX) {
            const int b0 = (k_wave * groups + group) * S::kWords * 4 + g * 16;
            const int end = c.rows * nblk - 16;         // (c.rows is a multiple of 16)
            next_valid = nblk - b0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto src = rows_of(UP ? a.s13 : a.s2, UP && i ? c.row + M : c.row, c.rows, nblk);
                const int row = UP ? row_wave * 16 + r : row_wave * 32 + i * 16 + r;
                const int at = row * nblk + b0;
                next_move[i] = max(at - end, 0);
                next_scale[i] = __builtin_amdgcn_raw_buffer_load_b128(src, min(at, end), 0, 0);
            }
        }
    };
    // v without its first `move` bytes, of what is left the first `valid`; zeros else.
    auto placed = [](u32x4 v, int move, int valid) {
        const int words = min(move, 16) / 4;
        if (words & 1) v = u32x4{v[1], v[2], v[3], 0};
        if (words & 2) v = u32x4{v[2], v[3], 0, 0};
        if (words & 4) v = u32x4{0, 0, 0, 0};
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = __builtin_amdgcn_alignbyte(j < 3 ? v[j + 1] : 0u, v[j], move & 3);
            const int left = min(max(valid - 4 * j, 0), 4);
            o[j] = left == 4 ? w : w & ((1u << (8 * left)) - 1);
        }
        return o;
    };

    // The further parts of h have sums of their own: where a weight is infinite the first part's
    // sum is the result (0 or the other sign, which a further part may have, would make it NaN).
    constexpr int kSums = kParts > 1 ? 2 : 1;
    f32x4 sum[kSums][2][NT];
    auto& acc = sum[0];
    auto clear = [&] {
#pragma unroll
        for (int k = 0; k < kSums; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < NT; ++c) sum[k][i][c] = f32x4{0, 0, 0, 0};
    };
    // first + rest, but first where that is infinite.
    auto add_rest = [](f32x4 (&first)[NT], const f32x4 (&rest)[NT]) {
        float most = 0.0f;
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) most = fmaxf(most, fabsf(first[c][q]));
        if (ballot64(most == __builtin_inff())) {     // rare
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) first[c][q] += __builtin_isinf(first[c][q]) ? 0.0f : rest[c][q];
        } else {
#pragma unroll
            for (int c = 0; c < NT; ++c) first[c] += rest[c];
        }
    };
    u32x4 scales[2] = {};
    uint32_t scale[2][S::kWords] = {};
    bool nan[2] = {};     // whether the lane has met the NaN scale in its row
    auto use_stage = [&](const uint8_t* lds, int stage) {
        const uint8_t* wa = lds + wave * 32 * S::kRowBytes + r * S::kRowBytes;
        const uint8_t* wb = lds + S::kW + k_wave * kParts * S::kPart + r * S::kColChunks * 16;
        auto other = [&](int p, int c, int chunk) {
            return as_bf16(ld16(wb + p * S::kPart + c * 16 * S::kColChunks * 16 + ((chunk ^ (r % 8)) * 16)));
        };
        if constexpr (MX) {
#pragma unroll
            for (int part = 0; part < SK / 128; ++part) {
                u32x4 codes[2];
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = (4 * part + g) ^ (S::kLine ? r % 8 : r / 2 % 4);
                    codes[i] = ld16(wa + i * 16 * S::kRowBytes + at * 16);
                    const uint32_t e = scale[i][stage * (SK / 128) + part] >> (8 * g) & 0xffu;
                    nan[i] |= e == 0xffu;
                    f[i] = __builtin_bit_cast(float, e << 23);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    bf16x8 w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) w[i] = as_bf16(widen8(codes[i][q], f[i]));
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            const bf16x8 b = other(p, c, part * 16 + 4 * g + q);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                sum[p > 0][i][c] =
                                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], b, sum[p > 0][i][c], 0, 0, 0);
                        }
                }
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                bf16x8 w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[i] = as_bf16(ld16(wa + i * 16 * S::kRowBytes + (((4 * q + g) ^ (r % 8)) * 16)));
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const bf16x8 b = other(p, c, 4 * q + g);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            sum[p > 0][i][c] =
                                __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], b, sum[p > 0][i][c], 0, 0, 0);
                    }
            }
        }
    };
    // A lane holds 4 consecutive output rows of one entry.
    auto store_item = [&](int item) {
        int slot;
        const int64_t r0 = item_rows(item, slot);
        const int first = l.first[slot], n = l.first[slot + 1] - first;
        if constexpr (MX) {
            // a NaN scale makes its whole row NaN; bit r of bad: row r
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint64_t bad = ballot64(nan[i]);
                bad |= bad >> 32;
                bad |= bad >> 16;
                nan[i] = false;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (bad >> (4 * g + q) & 1)
#pragma unroll
                        for (int c = 0; c < NT; ++c) acc[i][c][q] = __builtin_nanf("");
            }
        }
        if constexpr (SPLIT) {
            // (the next item's sums come behind barriers that the first wave passes as well)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    if (wave > 0) sums[((wave - 1) * 2 * NT + i * NT + c) * kWave + lane] = acc[i][c];
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xc07f);     // LDS writes are done
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (wave > 0) {
                clear();
                return;
            }
#pragma unroll
            for (int k = 0; k < WAVES - 1; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < NT; ++c) acc[i][c] += sums[(k * 2 * NT + i * NT + c) * kWave + lane];
        }
        if constexpr (PACK) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x4 rest[NT];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    rest[0][q] = __shfl_down(acc[i][0][q], S::kWidth);
#pragma unroll
                    for (int p = 2; p < P; ++p) rest[0][q] += __shfl_down(acc[i][0][q], p * S::kWidth);
                }
                add_rest(acc[i], rest);
            }
        }
        if constexpr (kSums > 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) add_rest(acc[i], sum[1][i]);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const int col = c * 16 + r;
            const int f = l.ent[col < n ? first + col : 0];
            if constexpr (UP) {
                const int64_t i = r0 + row_wave * 16 + 4 * g;
                // (constants over the whole kernel: 237 -> 248 us, 32 tokens of 128 experts in MXFP4)
                const ExpConstants constants = ExpConstants::here();
                const float most = constant_here(kBf16Max);
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = silu_of(acc[0][c][q], constants) * acc[1][c][q];
                for (int p = 0; p < h_parts; ++p) {
                    // a finite h past bf16's largest value has that as its first part; an infinity
                    // or a NaN stands in the first part alone
                    float part[4];
                    bool finite[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        finite[q] = __builtin_isfinite(v[q]);
                        part[q] = finite[q] ? __builtin_amdgcn_fmed3f(v[q], -most, most) : v[q];
                    }
                    const u32x2 b = {pack_bf16x2(part[0], part[1]), pack_bf16x2(part[2], part[3])};
                    if (col < n && i < M) *(u32x2*)(h + p * h_part + f * a.I + i) = b;
                    const float was[4] = {bf16lo(b[0]), bf16hi(b[0]), bf16lo(b[1]), bf16hi(b[1])};
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = finite[q] ? v[q] - was[q] : 0.0f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t row = r0 + row_wave * 32 + i * 16 + 4 * g;
                    if (col < n && row < M) *(f32x4*)(y + f * a.H + row) = acc[i][c];
                }
            }
        }
        clear();
    };

    int item = blockIdx.x;
    if (item >= items) return;
    __syncthreads();      // the lists are done with their scratch
    Cursor<S::kLoadsB> now, next;
    seek(item, now);
    clear();
    load_scales(now, 0);
    load_stage(lds0, now, 0);
    load_stage(lds1, now, 1);
    load_stage(lds2, now, 2);
    for (int group = 0;;) {
        // where the stream goes after this group; behind the last item it loads zeros
        const bool last = group + 1 == groups;
        const int next_item = last ? item + workers : item;
        const int next_group = last ? 0 : group + 1;
        const bool more = next_item < items;
        next = now;
        if (last && more) seek(next_item, next);
        const int beyond = more ? 0 : 1 << 20;
        if constexpr (MX) {
            if (group % kPerLoad == 0) {
                scales[0] = placed(next_scale[0], next_move[0], next_valid);
                scales[1] = placed(next_scale[1], next_move[1], next_valid);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < S::kWords; ++j)
                    scale[i][j] = (uint32_t)__shfl((int)scales[i][j % 4],
                                                   r + 16 * (group % kPerLoad * (S::kWords / 4) + j / 4));
            if (more && next_group % kPerLoad == 0) load_scales(next, next_group);
        }
        stage_sync<2 * S::kLoads>();      // two stages may be in flight
        load_stage(lds3, now, group * kGroup + 3);
        use_stage(lds0, 0);
        stage_sync<2 * S::kLoads>();
        load_stage(lds0, next, next_group * kGroup + beyond);
        use_stage(lds1, 1);
        stage_sync<2 * S::kLoads>();
        load_stage(lds1, next, next_group * kGroup + 1 + beyond);
        use_stage(lds2, 2);
        stage_sync<2 * S::kLoads>();
        load_stage(lds2, next, next_group * kGroup + 2 + beyond);
        use_stage(lds3, 3);
        if (last) store_item(item);
        if (!more) break;
        item = next_item;
        group = next_group;
        now = next;
    }
    // no load into LDS may be in flight when it goes to the next workgroup
    __builtin_amdgcn_s_waitcnt(0);
}

// out[t] = sum over k, ascending, of w[t,k] * y[t*K + k].  y is still in the caches: 3 to 4 us,
// 32 tokens of 8 x 7168 too, most of it the launch and two dependent loads.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void join_kernel(DecodeArgs a, const float* y) {
    const int64_t t = blockIdx.y;
    const int64_t c = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (c >= a.H) return;
    // (the rows of half the largest K are loaded together; a row that no expert has written
    // is read as well, and not used)
    float v[4] = {0, 0, 0, 0};
    constexpr int kBatch = 8;
    for (int k0 = 0; k0 < a.K; k0 += kBatch) {
        f32x4 z[kBatch];
        float w[kBatch];
        bool has[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t f = t * a.K + (k0 + j < a.K ? k0 + j : 0);
            const int e = a.idx[f];
            has[j] = k0 + j < a.K && e >= 0 && e < a.E;
            w[j] = a.w[f];
            z[j] = *(const f32x4*)(y + f * a.H + c);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (has[j])
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += w[j] * z[j][q];
    }
    if (a.out_f32) store_unit<true, false>(a.out, t * a.H + c, v);
    else store_unit<false, false>(a.out, t * a.H + c, v);
}

struct Work {
    uint32_t* lists;
    uint16_t* h;
    int64_t h_part;       // elements of a part
    float* y;
    int parts;            // of h
    StreamForm up, down;
};

// Workgroups: as many as fit the card at once (LDS decides), or one per item.
template <bool MX, bool UP, int P, int NT, int SK, int WAVES, bool SPLIT, bool PACK>
hipError_t launch(const DecodeArgs& a, const Work& w, hipStream_t s) {
    using S = Stream<MX, UP, P, NT, SK, WAVES, SPLIT, PACK>;
    const int64_t N = a.T * a.K, M = UP ? a.I : a.H;
    const int64_t most = N * ((M + S::kRows - 1) / S::kRows);
    const size_t lists_lds = (size_t)ListLayout{(int)N}.words32() * 4;
    const int per_cu = (int)(kLdsPerCu / (kGroup * S::kStageBytes + (SPLIT ? (WAVES - 1) * NT * 2048 : 16) + lists_lds));
    const int64_t fit = (int64_t)kCUs * (per_cu < 1 ? 1 : per_cu);
    // Weights go past the caches where rows are whole lines; a line that two stages share would be
    // fetched twice: 640 us with, 707 without (32 tokens, bf16, 128 experts of 2816 x 2816), 889
    // and 761 (2888 x 2888).
    const int64_t rb = (UP ? a.H : a.I) * 2 / (MX ? 4 : 1);
    const bool once = S::kLine && rb % 128 == 0 && (uintptr_t)(UP ? a.w13 : a.w2) % 128 == 0;
    // (one more writes the lists of the second product)
    const dim3 grid((unsigned)((most < fit ? most : fit) + (UP ? 1 : 0)));
    if (S::kLine && once)
        stream_kernel<MX, UP, P, NT, SK, WAVES, SPLIT, PACK, S::kLine>
            <<<grid, S::kThreads, lists_lds, s>>>(a, w.lists, w.down.width, w.h, w.h_part, w.y, w.parts);
    else
        stream_kernel<MX, UP, P, NT, SK, WAVES, SPLIT, PACK, false>
            <<<grid, S::kThreads, lists_lds, s>>>(a, w.lists, w.down.width, w.h, w.h_part, w.y, w.parts);
    return hipGetLastError();
}

template <bool MX, bool UP, int P, int NT, int SK, bool PACK = false>
hipError_t launch_waves(const DecodeArgs& a, const Work& w, hipStream_t s) {
    return (UP ? w.up : w.down).waves == 4 ? launch<MX, UP, P, NT, SK, 4, false, PACK>(a, w, s)
                                           : launch<MX, UP, P, NT, SK, 2, false, PACK>(a, w, s);
}

template <bool MX>
hipError_t launch_up(const DecodeArgs& a, const Work& w, hipStream_t s) {
    constexpr int kShort = MX ? 128 : 64;
    if (w.up.split) return launch<MX, true, 1, 1, kShort, 4, true, false>(a, w, s);
    if constexpr (MX) {
        if (w.up.width == 32) return launch<MX, true, 1, 2, kShort, 4, false, false>(a, w, s);
        if (w.up.stage == 256) return launch_waves<MX, true, 1, 1, 256>(a, w, s);
    } else {
        if (w.up.width == 32) return launch_waves<MX, true, 1, 2, kShort>(a, w, s);
    }
    return launch_waves<MX, true, 1, 1, kShort>(a, w, s);
}

template <bool MX, int P>
hipError_t launch_down(const DecodeArgs& a, const Work& w, hipStream_t s) {
    constexpr int kShort = MX ? 128 : 64;
    if constexpr (MX) {
        if (w.down.pack)
            return w.down.stage == 256 ? launch_waves<MX, false, P, 1, 256, true>(a, w, s)
                                       : launch_waves<MX, false, P, 1, 128, true>(a, w, s);
        if (w.down.width == 32) return launch<MX, false, P, 2, kShort, 4, false, false>(a, w, s);
    } else {
        if (w.down.width == 32) return launch_waves<MX, false, P, 2, kShort>(a, w, s);
    }
    return launch_waves<MX, false, P, 1, kShort>(a, w, s);
}

template <bool MX>
hipError_t launch_type(const DecodeArgs& a, hipStream_t s) {
    const int64_t N = a.T * a.K;
    Work w{};
    w.lists = (uint32_t*)a.ws;
    w.y = (float*)((char*)a.ws + kListBytes);
    w.h = (uint16_t*)(w.y + N * a.H);
    w.h_part = N * a.I;
    w.parts = a.out_f32 ? 3 : 2;
    const DecodeSize size{a.T, a.H, a.I, a.K, a.E, MX, w.parts};
    w.up = size.up();
    w.down = size.down();
    hipError_t st = launch_up<MX>(a, w, s);
    if (st == hipSuccess) st = a.out_f32 ? launch_down<MX, 3>(a, w, s) : launch_down<MX, 2>(a, w, s);
    if (st != hipSuccess) return st;
    const dim3 grid((unsigned)((a.H + 4 * kJoinThreads - 1) / (4 * kJoinThreads)), (unsigned)a.T);
    join_kernel<<<grid, kJoinThreads, 0, s>>>(a, w.y);
    return hipGetLastError();
}

}  // namespace

size_t decode_ws(int64_t T, int K, int64_t H, int64_t I) {
    return kListBytes + (size_t)(T * K) * ((size_t)H * sizeof(float) + (size_t)I * 3 * sizeof(uint16_t));
}

hipError_t launch_experts_decode(const DecodeArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    return a.s13 ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

}  // namespace moe
