// expert_product.hip - the grouped product of packed rows with their experts' weights,
// both in MXFP4: y[r,n] = sum_h a[r,h] * w[e,n,h] for the rows r of expert e's segment,
// or, with SwiGLU, silu(y[r,i]) * y[r,I+i].
//
// Products of codes run on the scaled matrix instruction, which multiplies 32x64 by
// 64x32 e2m1 codes, applies the two e8m0 scales of each block of 32 and adds in f32.
// Weights are its rows and activations its columns, so a lane ends up with 4
// consecutive n of one row.
//
// A workgroup of 4 waves owns BM rows of one expert and 256 weight rows (with SwiGLU
// 128 gate and 128 up rows, 32 of each in turn, so a lane holds both halves of its
// outputs).  Which expert a workgroup has follows from packed_cnt on the device; the
// grid covers the most tiles that the row count allows, and the rest leave at once.
//
// K runs in stages of 256 elements: 128 bytes of each row, loaded straight into LDS
// while the stage before is multiplied.  The 16-byte chunks of a row are stored at
// (chunk ^ row % 8), so that 8 lanes that read one chunk of 8 rows meet different
// banks.  A stage is four matrix steps; lane half g takes chunks 4g to 4g+3, which puts
// its four scales side by side in memory.  Fragments are read one step ahead of the
// matrix instructions, so one barrier a stage is enough: before the last step every wave
// holds the rest of the stage in registers, its LDS is free for the stage after next,
// and the next stage has landed.
//
// Rows behind a segment, weight rows behind N and chunks behind H are loaded as zeros
// by the range check of the buffer descriptors (their scales too, so a NaN scale of a
// neighbour does not get in); they are never stored.
#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kBN = 256;          // weight rows of a tile
constexpr int kStageChunks = 8;   // 16-byte chunks of a row in a stage: 256 codes
constexpr int kStageBytes = 128;
constexpr int kGroup = 4;         // stages whose scales are loaded together
constexpr int kGroupChunks = kGroup * kStageChunks;
constexpr int kFp4 = 4;           // the matrix instruction's format code of e2m1

// Ored to an offset below 2^31 it leaves every descriptor's range (2^31 at the most).
__device__ __forceinline__ uint32_t outside_if(bool b) { return (uint32_t)b << 31; }

using Lds = __attribute__((address_space(3))) uint8_t;

struct Tile {
    int e;          // expert, or -1: no tile
    int64_t row0;   // first row
    int rows;       // rows of it, at most BM
};

__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

// Rows of expert e inside the buffer.
__device__ __forceinline__ int segment(const ProductArgs& a, int e, int64_t& first) {
    const int64_t lo = a.packed_off[e];
    const int64_t n = a.packed_cnt[e];
    first = lo < 0 ? 0 : lo;
    int64_t hi = lo + n;
    if (hi > a.rows) hi = a.rows;
    return hi > first ? (int)(hi - first) : 0;
}

// The row tile that workgroup b works on: experts in order, BM rows at a time.  Row
// tiles times column tiles are dealt out so that each XCD (workgroups go to them in
// turn) gets one run of neighbours, which share weights and rows in its L2.  Every
// wave finds the tile by itself, 64 experts at a time.
template <int BM>
__device__ __forceinline__ Tile find_tile(const ProductArgs& a, int64_t b, int col_tiles,
                                          int& col) {
    const int lane = threadIdx.x % kWave;
    int total = 0;
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
        int64_t first;
        const int n = e0 + lane < a.E ? segment(a, e0 + lane, first) : 0;
        total += (n + BM - 1) / BM;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) total += __shfl_xor(total, d);
    total = __builtin_amdgcn_readfirstlane(total);
    const int64_t items = (int64_t)total * col_tiles;
    const int64_t per = (items + 7) / 8;
    const int64_t item = (int64_t)(b % 8) * per + b / 8;
    Tile t{-1, 0, 0};
    if (b / 8 >= per || item >= items) return t;
    int at = (int)(item / col_tiles);
    col = (int)(item - (int64_t)at * col_tiles);
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
        int64_t first = 0;
        const int n = e0 + lane < a.E ? segment(a, e0 + lane, first) : 0;
        const int mine = (n + BM - 1) / BM;
        int upto = mine;   // tiles of the experts up to and with this lane's
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const int here = readlane(upto, kWave - 1);
        if (at >= here) {
            at -= here;
            continue;
        }
        const int owner = __builtin_ctzll(ballot64(upto > at));
        const int skip = at - (readlane(upto, owner) - readlane(mine, owner));
        const int cnt = readlane(n, owner);
        const uint64_t f = (uint64_t)first;
        const int64_t start = (int64_t)(((uint64_t)(uint32_t)readlane((int)(f >> 32), owner) << 32) |
                                        (uint32_t)readlane((int)f, owner));
        t.e = e0 + owner;
        t.row0 = start + (int64_t)skip * BM;
        t.rows = cnt - skip * BM < BM ? cnt - skip * BM : BM;
        return t;
    }
    return t;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint8_t* base, int64_t row,
                                                          int64_t rows, int64_t row_bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)(base + row * row_bytes), 0,
                                             (int)(uint32_t)(rows * row_bytes), kRsrcWord3);
}

// 8 rows of a stage into LDS: lane l fetches chunk (l % 8) ^ (l / 8) of row l / 8.
__device__ __forceinline__ void stage8(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (Lds*)lds, 16, (int)off, 0, 0, 0);
}

__device__ __forceinline__ void store4(void* y, bool f32, int64_t at, f32x4 v) {
    if (f32) {
        *(f32x4*)((float*)y + at) = v;
    } else {
        *(u32x2*)((uint16_t*)y + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

__device__ __forceinline__ float silu_of(float g) {
    // g / (1 + exp(-g)); exp overflows to an infinity below -88, where the quotient is -0
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// WM x WN waves: a wave owns BM / WM rows and kBN / WN weight rows.
// WORDS: every row's scales start and end at a whole word.
template <int BM, int WM, bool SWIGLU, bool WORDS>
__global__ __launch_bounds__(kThreads, 1) void product_kernel(ProductArgs a, int col_tiles,
                                                              int64_t base) {
    constexpr int WN = kWaves / WM;
    constexpr int MT = BM / WM / 32, NT = kBN / WN / 32;
    constexpr int kLoadsA = BM / 8 / kWaves, kLoadsW = kBN / 8 / kWaves;
    __shared__ __align__(16) uint8_t lds_a0[BM * kStageBytes], lds_a1[BM * kStageBytes];
    __shared__ __align__(16) uint8_t lds_w0[kBN * kStageBytes], lds_w1[kBN * kStageBytes];

    int col = 0;
    Tile t = find_tile<BM>(a, base + blockIdx.x, col_tiles, col);
    // the same in every lane: into scalar registers, where descriptors have to be
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.row0 = uniform(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    col = __builtin_amdgcn_readfirstlane(col);
    if (t.e < 0) return;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t rb = a.H / 2;            // bytes of a row of codes
    const int nblk = (int)(a.H / kMxBlock);
    const int stages = (nblk + kStageChunks - 1) / kStageChunks;
    const int whole_stages = WORDS && BM > 32 ? nblk / kGroupChunks * kGroup : 0;
    const int64_t NO = SWIGLU ? a.N / 2 : a.N;     // output columns
    const int64_t n0 = (int64_t)col * (SWIGLU ? kBN / 2 : kBN);
    const int64_t wrow = (int64_t)t.e * a.N + n0;
    const int64_t left = NO - n0;
    const int wrows = (int)(left < (SWIGLU ? kBN / 2 : kBN) ? left : (SWIGLU ? kBN / 2 : kBN));

    const auto ra = rows_of(a.a, t.row0, t.rows, rb);
    const auto rw = rows_of(a.w, wrow, wrows, rb);
    const auto ru = SWIGLU ? rows_of(a.w, wrow + NO, wrows, rb) : rw;
    const auto rsa = rows_of(a.a_scales, t.row0, t.rows, nblk);
    const auto rsw = rows_of(a.w_scales, wrow, wrows, nblk);
    const auto rsu = SWIGLU ? rows_of(a.w_scales, wrow + NO, wrows, nblk) : rsw;

    // Weight row (within its half) of tile row r.
    auto weight_row = [](int r) { return SWIGLU ? (r >> 6) * 32 + (r & 31) : r; };

    static_assert(kLoadsW * 8 % 64 == 0, "a wave starts at a gate row");
    const int chunk = (lane % 8) ^ (lane / 8);
    const int spread = chunk % 4 + (chunk / 4) * (kGroupChunks / 2);
    auto load_stage = [&](uint8_t* la, uint8_t* lw, int s) {
        // all by arithmetic: a branch would split the blocks of the main loop
        const int whole = (s - whole_stages) >> 31;     // -1: yes, 0: no
        const int group = s / kGroup * kGroupChunks + s % kGroup * 4;
        const int first = s * kStageChunks + ((group - s * kStageChunks) & whole);
        const uint32_t at = (uint32_t)(first + chunk + ((spread - chunk) & whole));
        const uint32_t bad = outside_if((int)at >= nblk);
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int r8 = (wave * kLoadsA + i) * 8;
            stage8(ra, la + r8 * kStageBytes, ((uint32_t)(r8 + lane / 8) * (uint32_t)rb + at * 16) | bad);
        }
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) {
            const int r8 = (wave * kLoadsW + i) * 8;
            const int row = weight_row(r8) + lane / 8;
            stage8(SWIGLU && (i * 8 & 32) ? ru : rw, lw + r8 * kStageBytes,
                   ((uint32_t)row * (uint32_t)rb + at * 16) | bad);
        }
    };

    const int r = lane % 32, g = lane / 32;
    // The scale bytes of a lane in a group of stages: byte j of word i is that of matrix
    // step j of stage i.
    auto scale16 = [&](__amdgpu_buffer_rsrc_t rs, int row, int group, auto whole) -> u32x4 {
        const uint32_t off = (uint32_t)row * (uint32_t)nblk + (uint32_t)(group * kGroupChunks);
        u32x4 v;
        if constexpr (decltype(whole)::value) {
            v = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(off + (kGroupChunks / 2) * g), 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const int b = i * kStageChunks + 4 * g;
                const int room = nblk - group * kGroupChunks - b;   // blocks from there on
                if constexpr (WORDS) {
                    v[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)((off + b) | outside_if(room <= 0)), 0, 0);
                } else {
                    uint32_t w = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(
                                 rs, (int)((off + b + j) | outside_if(room <= j)), 0, 0) << (8 * j);
                    v[i] = w;
                }
            }
        }
        return v;
    };
    u32x4 sw[NT], sa[MT], next_sw[NT], next_sa[MT];
    auto load_group = [&](int group, auto whole) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int tr = wn * NT + i;
            next_sw[i] = scale16(SWIGLU && (i & 1) ? rsu : rsw, weight_row(tr * 32) + r, group, whole);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) next_sa[i] = scale16(rsa, (wm * MT + i) * 32 + r, group, whole);
    };
    auto load_scales = [&](int group) {
        if (WORDS && BM > 32 && group * kGroup < whole_stages) load_group(group, std::true_type{});
        else load_group(group, std::false_type{});
    };
    auto take_scales = [&] {
#pragma unroll
        for (int i = 0; i < NT; ++i) sw[i] = next_sw[i];
#pragma unroll
        for (int i = 0; i < MT; ++i) sa[i] = next_sa[i];
    };

    i32x8 fw[2][NT], fa[2][MT];
    const uint32_t frag0 = (uint32_t)(r * kStageBytes + (((4 * g) ^ (r & 7)) * 16));
    // The fragments of matrix step `step` into set `set`.
    auto read_frags = [&](int set, int step, const uint8_t* la, const uint8_t* lw) {
        const uint32_t at = frag0 ^ (uint32_t)(step * 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const u32x4 v = *(const u32x4*)(lw + (wn * NT + i) * 32 * kStageBytes + at);
            fw[set][i] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const u32x4 v = *(const u32x4*)(la + (wm * MT + i) * 32 * kStageBytes + at);
            fa[set][i] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
    };

    f32x16 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

// The order of loads and matrix instructions stays as written from step to step.
#define MOE_MX_STEP(FRAGS, STEP, STAGE)                                                       \
    _Pragma("unroll") for (int i = 0; i < NT; ++i)                                          \
        _Pragma("unroll") for (int j = 0; j < MT; ++j)                                      \
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(                    \
                fw[FRAGS][i], fa[FRAGS][j], acc[i][j], kFp4, kFp4, STEP, (int)sw[i][STAGE], \
                STEP, (int)sa[j][STAGE]);                                                    \
    _Pragma("unroll") for (int i = 0; i < NT + MT; ++i) {                                   \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0); /* one LDS read */               \
        __builtin_amdgcn_sched_group_barrier(0x008, NT * MT / (NT + MT), 0);                \
    }                                                                                       \
    __builtin_amdgcn_sched_barrier(0)

    // Every wave's loads into LDS have landed and every wave's reads are in registers.
    auto sync_stage = [] {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
// Stage s, number STAGE of its group, in LDS buffers A, W, its first fragments already
// read; the next stage is on its way into NA, NW.
#define MOE_MX_STAGE(A, W, NA, NW, STAGE) \
    read_frags(1, 1, A, W);               \
    MOE_MX_STEP(0, 0, STAGE);             \
    read_frags(0, 2, A, W);               \
    MOE_MX_STEP(1, 1, STAGE);             \
    read_frags(1, 3, A, W);               \
    MOE_MX_STEP(0, 2, STAGE);             \
    sync_stage();                         \
    load_stage(A, W, s + 2);              \
    read_frags(0, 0, NA, NW);             \
    MOE_MX_STEP(1, 3, STAGE);             \
    ++s

    load_stage(lds_a0, lds_w0, 0);
    load_scales(0);
    sync_stage();
    load_stage(lds_a1, lds_w1, 1);      // past the last stage: zeros
    read_frags(0, 0, lds_a0, lds_w0);
    int s = 0;
    while (s + kGroup <= stages) {
        take_scales();
        load_scales(s / kGroup + 1);
        MOE_MX_STAGE(lds_a0, lds_w0, lds_a1, lds_w1, 0);
        MOE_MX_STAGE(lds_a1, lds_w1, lds_a0, lds_w0, 1);
        MOE_MX_STAGE(lds_a0, lds_w0, lds_a1, lds_w1, 2);
        MOE_MX_STAGE(lds_a1, lds_w1, lds_a0, lds_w0, 3);
    }
    take_scales();
    if (s < stages) {
        MOE_MX_STAGE(lds_a0, lds_w0, lds_a1, lds_w1, 0);
    }
    if (s < stages) {
        MOE_MX_STAGE(lds_a1, lds_w1, lds_a0, lds_w0, 1);
    }
    if (s < stages) {
        MOE_MX_STAGE(lds_a0, lds_w0, lds_a1, lds_w1, 2);
    }
#undef MOE_MX_STAGE
#undef MOE_MX_STEP
    // no load into LDS may be in flight when the workgroup's LDS goes to the next one
    __builtin_amdgcn_s_waitcnt(0);

    // a lane holds columns r of the tile (a row of y) and weight rows 8 * p + 4 * g + 0..3
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int row = (wm * MT + j) * 32 + r;
        if (row >= t.rows) continue;
        const int64_t out = (t.row0 + row) * NO;
        if constexpr (SWIGLU) {
#pragma unroll
            for (int i = 0; i < NT; i += 2)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int64_t n = n0 + (wn * NT + i) / 2 * 32 + 8 * p + 4 * g;
                    if (n >= NO) continue;
                    f32x4 v;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[q] = silu_of(acc[i][j][4 * p + q]) * acc[i + 1][j][4 * p + q];
                    store4(a.y, a.y_f32, out + n, v);
                }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int64_t n = n0 + (wn * NT + i) * 32 + 8 * p + 4 * g;
                    if (n >= NO) continue;
                    const f32x4 v = {acc[i][j][4 * p], acc[i][j][4 * p + 1], acc[i][j][4 * p + 2],
                                     acc[i][j][4 * p + 3]};
                    store4(a.y, a.y_f32, out + n, v);
                }
        }
    }
}

template <int BM, int WM>
hipError_t launch(const ProductArgs& a, hipStream_t s) {
    const int64_t cols = a.swiglu ? a.N / 2 : a.N;
    const int col_tiles = (int)((cols + (a.swiglu ? kBN / 2 : kBN) - 1) / (a.swiglu ? kBN / 2 : kBN));
    const bool words = a.H / kMxBlock % 4 == 0 && ((uintptr_t)a.a_scales | (uintptr_t)a.w_scales) % 4 == 0;
    // every expert may have one tile that is not full
    const int64_t row_tiles = a.rows / BM + (a.E < a.rows ? a.E : a.rows);
    const int64_t blocks = (row_tiles * col_tiles + 7) / 8 * 8;
    for (int64_t base = 0; base < blocks; base += kMaxGrid) {
        const dim3 grid((unsigned)(blocks - base < kMaxGrid ? blocks - base : kMaxGrid));
        if (a.swiglu) {
            if (words) product_kernel<BM, WM, true, true><<<grid, kThreads, 0, s>>>(a, col_tiles, base);
            else product_kernel<BM, WM, true, false><<<grid, kThreads, 0, s>>>(a, col_tiles, base);
        } else {
            if (words) product_kernel<BM, WM, false, true><<<grid, kThreads, 0, s>>>(a, col_tiles, base);
            else product_kernel<BM, WM, false, false><<<grid, kThreads, 0, s>>>(a, col_tiles, base);
        }
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const int64_t mean = a.rows / a.E;
    if (mean <= 32) return launch<32, 1>(a, s);
    if (mean <= 64) return launch<64, 1>(a, s);
    if (mean <= 128) return launch<128, 2>(a, s);
    return launch<256, 2>(a, s);
}

}  // namespace moe
