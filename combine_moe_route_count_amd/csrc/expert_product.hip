// expert_product.hip - the grouped product of packed rows with their experts' weights,
// both in MXFP4: y[r,n] = sum_h a[r,h] * w[e,n,h] for the rows r of expert e's segment,
// or, with SwiGLU, silu(y[r,i]) * y[r,I+i].
//
// Products of codes run on the scaled matrix instruction, which multiplies 32x64 by
// 64x32 e2m1 codes, applies the two e8m0 scales of each block of 32 and adds in f32.
// Weights are its rows and activations its columns, so a lane ends up with 4
// consecutive n of one row.
//
// A workgroup of 4 waves owns BM rows (64, 128 or 256) of one expert and 256 weight rows (with
// SwiGLU 128 gate and 128 up rows, 32 of each in turn, so a lane holds both halves of its
// outputs).  Which expert a workgroup has follows from packed_cnt on the device; the
// grid covers the most tiles that the row count allows, and the rest leave at once.  A tile
// of at most BM / 2 rows runs at half the height.  Where there are few tiles, others of 32
// rows and 64 weight rows take over, whose 4 waves share out K and add their sums in LDS.
//
// K runs in stages of 128 elements: 64 bytes of each row, loaded straight into LDS, four
// stages deep, so that three are in flight while one is multiplied.  The 16-byte chunks of a
// row are stored at (chunk ^ row / 2 % 4), so that 8 lanes that read one chunk of 8 rows meet
// different banks.  A stage is two matrix steps of 64 elements, of which lane half g takes
// chunk g.  The body of a stage is one block without a branch: with one the compiler moves
// the matrix instructions behind it, away from the loads they were to cover.
//
// Scales are loaded for eight stages at once, 16 bytes by each of two lanes, wherever rows start:
// loads of single words kept the address unit busier than the matrix cores.
//
// Measured on random codes: 3.0 to 3.1e15 operations a second (32768 rows x 4096 x 7168 over
// 64 experts, SwiGLU), 3.7 to 3.9e15 (8192 x 8192 x 8192), where the matrix instruction alone runs at
// 6.3e15.  All-zero codes take a quarter less time: that much of it is power, and rows of zeros in a
// tile cost little.  The rest is what a tile does beside its matrix instructions: with 128 or 256 rows
// a CU has one workgroup, so finding the tile, its first loads and its epilogue are covered by nothing
// (at K = 2048, 32768 rows x 7168, 2.2e15; there the 256-row form without SwiGLU also spills
// 16 registers).  6.0 TB/s of weights where experts have two rows each (128 experts, 4096 x 4096).
//
// Rows behind a segment, weight rows behind N and chunks behind H are loaded as zeros
// by the range check of the buffer descriptors (their scales too, so a NaN scale of a
// neighbour does not get in); they are never stored.
#include <type_traits>

#include "device_common.hpp"
#include "experts_device.hpp"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kBN = kTileCols;    // weight rows of a tile
constexpr int kStageChunks = 4;   // 16-byte chunks of a row in a stage: 128 codes
constexpr int kStageBytes = 64;
constexpr int kGroup = 4;         // stages in LDS, and stages whose scales are loaded together
constexpr int kGroupChunks = kGroup * kStageChunks;
constexpr int kFp4 = 4;           // the matrix instruction's format code of e2m1

constexpr int kRowGroup = 4;       // row tiles of an expert that are worked on side by side

using Lds = __attribute__((address_space(3))) uint8_t;

struct Tile {
    int e;          // expert, or -1: no tile
    int64_t row0;   // first row
    int rows;       // rows of it, at most BM
};

// Sum of v over the lanes up to and with the calling one (every lane active).
__device__ __forceinline__ int wave_scan(int v) {
#define MOE_SCAN_STEP(CTRL, MASK) v += __builtin_amdgcn_update_dpp(0, v, CTRL, MASK, 0xF, false)
    MOE_SCAN_STEP(0x111, 0xF);   // row_shr:1
    MOE_SCAN_STEP(0x112, 0xF);   // row_shr:2
    MOE_SCAN_STEP(0x114, 0xF);   // row_shr:4
    MOE_SCAN_STEP(0x118, 0xF);   // row_shr:8
    MOE_SCAN_STEP(0x142, 0xA);   // row_bcast:15 into rows 1 and 3
    MOE_SCAN_STEP(0x143, 0xC);   // row_bcast:31 into rows 2 and 3
#undef MOE_SCAN_STEP
    return v;
}

__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

// Rows of expert e inside the buffer, whatever the segment says.
__device__ __forceinline__ int segment(const ProductArgs& a, int e, int& first) {
    const int lo = a.packed_off[e], cnt = a.packed_cnt[e] > 0 ? a.packed_cnt[e] : 0;
    const int rows = (int)a.rows;
    first = lo > 0 ? lo : 0;
    const int n = lo >= 0 ? min(cnt, rows - lo) : min(lo + cnt, rows);   // neither overflows
    return n > 0 ? n : 0;
}

// The tile that workgroup b works on.  Experts in order; of one expert, kRowGroup row tiles
// at a time, row tiles first, so that tiles that run together share few weight rows and
// few token rows.  The sequence is cut into 8 runs, one for each XCD (workgroups go to
// them in turn), so that neighbours share an L2.  Every wave finds the tile by itself.
template <int BM>
__device__ __forceinline__ Tile find_tile(const ProductArgs& a, int64_t b, int col_tiles,
                                          int& col) {
    constexpr int kChunks = 4;          // of 64 experts, looked at together
    const int lane = threadIdx.x % kWave;
    int upto[kChunks];                  // row tiles of a chunk's experts up to and with this lane's
    auto look_at = [&](int e0) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int e = e0 + c * kWave + lane;
            int first;
            upto[c] = e < a.E ? (int)(((uint32_t)segment(a, e, first) + BM - 1) / BM) : 0;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) upto[c] = wave_scan(upto[c]);
    };
    int total = 0;
    for (int e0 = 0; e0 < a.E; e0 += kChunks * kWave) {
        look_at(e0);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) total += readlane(upto[c], kWave - 1);
    }
    const int64_t items = (int64_t)total * col_tiles;
    const int64_t per = (items + 7) / 8;
    const int64_t item = (int64_t)(b % 8) * per + b / 8;
    Tile t{-1, 0, 0};
    if (b / 8 >= per || item >= items) return t;
    const int at = (int)(item / col_tiles);    // row tile, if an expert's were not grouped
    int before = 0, e = 0, tiles = 0;          // row tiles before expert e, and its own
    for (int e0 = 0; tiles == 0 && e0 < a.E; e0 += kChunks * kWave) {
        if (a.E > kChunks * kWave) look_at(e0);      // else as it was found above
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int here = readlane(upto[c], kWave - 1);
            if (tiles != 0) continue;
            if (at - before >= here) {
                before += here;
                continue;
            }
            const int owner = __builtin_ctzll(ballot64(upto[c] > at - before));
            const int less = owner > 0 ? readlane(upto[c], owner - 1) : 0;
            tiles = readlane(upto[c], owner) - less;
            before += less;
            e = e0 + c * kWave + owner;
        }
    }
    const int64_t local = item - (int64_t)before * col_tiles;
    // counts that change under the call, or whose sum overflows because segments overlap
    if (local < 0 || local >= (int64_t)tiles * col_tiles) return t;
    const int top = (int)(local / ((int64_t)kRowGroup * col_tiles)) * kRowGroup;
    const int rows = tiles - top < kRowGroup ? tiles - top : kRowGroup;
    const int in_group = (int)(local - (int64_t)top * col_tiles);
    col = in_group / rows;
    const int skip = top + in_group - col * rows;
    int first;
    const int cnt = segment(a, e, first);
    t.e = e;
    t.row0 = (int64_t)first + (int64_t)skip * BM;
    t.rows = cnt - skip * BM < BM ? cnt - skip * BM : BM;
    return t;
}

// 16 rows of a stage into LDS, lane l's 16 bytes to l * 16.
__device__ __forceinline__ void stage16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (Lds*)lds, 16, (int)off, 0, 0, 0);
}

// For a bf16 result, whose rounding is 300 times as coarse: exp2's argument is rounded once, off by
// |g| * 2^-24 of the result at the most (exp overflows to an infinity below -88, where the quotient is
// -0).  Every output's silu stands behind the matrix instructions of its tile: with silu_of 640 ->
// 652 us (32768 rows x 4096 x 7168 over 64 experts), 383 -> 399 (16384 rows).
__device__ __forceinline__ float silu_for_bf16(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// Rows of scales from the word on in which the first begins, `skip` bytes before it.  The
// range ends with the word that holds the last byte.
struct Scales {
    __amdgpu_buffer_rsrc_t rs;
    int skip;
};
template <bool WORDS>
__device__ __forceinline__ Scales scales_of(const uint8_t* base, int64_t row, int64_t rows, int64_t nblk) {
    const uint8_t* p = base + row * nblk;
    const int skip = WORDS ? 0 : (int)((uintptr_t)p & 3);
    return Scales{__builtin_amdgcn_make_buffer_rsrc((void*)(p - skip), 0,
                                                    (int)((uint32_t)(skip + rows * nblk + 3) & ~3u), kRsrcWord3),
                  skip};
}

// Waves that share a tile's weight rows.
constexpr int row_waves(int BM) { return BM >= 128 ? 2 : 1; }

// One tile of at most BM rows by kBN weight rows: WM x WN waves, each BM / WM rows and kBN /
// WN weight rows.  WORDS: every row's scales start and end at a whole word.
template <int BM, bool SWIGLU, bool WORDS, int LDS>
__device__ __forceinline__ void product_tile(const ProductArgs& a, const Tile& t, int col,
                                             uint8_t (&lds0)[LDS], uint8_t (&lds1)[LDS],
                                             uint8_t (&lds2)[LDS], uint8_t (&lds3)[LDS]) {
    constexpr int WM = row_waves(BM), WN = kWaves / WM;
    constexpr int MT = BM / WM / 32, NT = kBN / WN / 32;
    constexpr int kLoadsA = (BM / 16 + kWaves - 1) / kWaves, kLoadsW = kBN / 16 / kWaves;
    constexpr int kA = BM * kStageBytes;     // where a stage's weight rows begin
    static_assert(kA + kBN * kStageBytes <= LDS, "a stage fits its buffer");

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t rb = a.H / 2;            // bytes of a row of codes
    const int nblk = (int)(a.H / kMxBlock);
    const int stages = (nblk + kStageChunks - 1) / kStageChunks;
    const int64_t NO = SWIGLU ? a.N / 2 : a.N;     // output columns
    const int64_t n0 = (int64_t)col * (SWIGLU ? kBN / 2 : kBN);
    const int64_t wrow = (int64_t)t.e * a.N + n0;
    const int64_t left = NO - n0;
    const int wrows = (int)(left < (SWIGLU ? kBN / 2 : kBN) ? left : (SWIGLU ? kBN / 2 : kBN));

    const auto ra = rows_of(a.a, t.row0, t.rows, rb);
    const auto rw = rows_of(a.w, wrow, wrows, rb);
    const auto ru = SWIGLU ? rows_of(a.w, wrow + NO, wrows, rb) : rw;
    const Scales rsa = scales_of<WORDS>(a.a_scales, t.row0, t.rows, nblk);
    const Scales rsw = scales_of<WORDS>(a.w_scales, wrow, wrows, nblk);
    const Scales rsu = SWIGLU ? scales_of<WORDS>(a.w_scales, wrow + NO, wrows, nblk) : rsw;

    // Weight row (within its half) of tile row r.
    auto weight_row = [](int r) { return SWIGLU ? (r >> 6) * 32 + (r & 31) : r; };

    static_assert(kLoadsW * 16 % 64 == 0, "a wave starts at a gate row");
    const int chunk = (lane % 4) ^ (lane / 8 % 4);
    auto load_stage = [&](uint8_t* lds, int s) {
        const uint32_t at = (uint32_t)(s * kStageChunks + chunk);
        const uint32_t bad = outside_if((int)at >= nblk);
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            // 32 rows are two loads for four waves: two waves each fetch the same
            const int r16 = (wave * kLoadsA + i) * 16 % BM;
            stage16(ra, lds + r16 * kStageBytes,
                    ((uint32_t)(r16 + lane / 4) * (uint32_t)rb + at * 16) | bad);
        }
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) {
            const int r16 = (wave * kLoadsW + i) * 16;
            const int row = weight_row(r16) + lane / 4;
            stage16(SWIGLU && (i * 16 & 32) ? ru : rw, lds + kA + r16 * kStageBytes,
                    ((uint32_t)row * (uint32_t)rb + at * 16) | bad);
        }
    };

    const int r = lane % 32, g = lane / 32;
    // The scales of a lane's row in a group of stages: bytes 2g and 2g + 1 of word i are
    // those of the two matrix steps of stage i.  Whole groups are loaded in pairs, 32 bytes
    // of a row by two lanes, and taken apart when they are needed.
    // WORDS or not, whole words are loaded (16 bytes that start anywhere in one are taken apart by
    // the address unit: 227 us against 254 for 7782 rows x 8192 x 4128); then a row's 32
    // bytes end in a ninth word.
    struct Pair {
        u32x4 v;
        uint32_t last;
    };
    auto scale_pair = [&](const Scales& sc, int row, int group) -> Pair {
        const int at = ((sc.skip + row * nblk) & ~3) + group * kGroupChunks;
        Pair p;
        p.v = __builtin_amdgcn_raw_buffer_load_b128(sc.rs, at + g * kGroupChunks, 0, 0);
        p.last = WORDS ? 0u : __builtin_amdgcn_raw_buffer_load_b32(sc.rs, at + 2 * kGroupChunks, 0, 0);
        return p;
    };
    // What is left behind the pairs: a word for each stage, or, where rows do not start at whole
    // words, its two bytes as they stand in memory, moved to their place when taken (a move
    // here would wait for the load).  The last two of a row are read where fewer are left.
    auto scale_rest = [&](const Scales& sc, int row, int group) -> u32x4 {
        const auto rs = sc.rs;
        const uint32_t off = (uint32_t)sc.skip + (uint32_t)row * (uint32_t)nblk;
        u32x4 v;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int b = group * kGroupChunks + i * kStageChunks;
            if constexpr (WORDS) {
                v[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)((off + b) | outside_if(b >= nblk)), 0, 0);
            } else {
                const int at = min(b + 2 * g, nblk - 2);
                v[i] = nblk > 1 ? __builtin_amdgcn_raw_buffer_load_b16(rs, (int)(off + at), 0, 0)
                                : __builtin_amdgcn_raw_buffer_load_b8(rs, (int)off, 0, 0) << 8;
            }
        }
        return v;
    };
    // Pairs of groups whose weight scales are loaded at once: a cache line of them, where weight
    // rows are read once, lest the line leave the L2 before its next quarter is wanted (weights
    // of 128 experts, 4096 x 4096: 1222 -> 1040 MB from memory, 176 -> 166 us for 256 rows).
    // 128 rows have no registers left for that: 288 -> 295 us (8192 rows of 64 experts).
    constexpr int kAhead = BM <= 64 ? (WORDS ? 4 : 2) : 1;
    u32x4 qw[NT], qa[MT];
    Pair next_qw[NT], next_qa[MT], ready_qw[kAhead][NT], flying_qw[kAhead][NT];
    auto load_rest = [&](int group) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int tr = wn * NT + i;
            next_qw[i].v = scale_rest(SWIGLU && (i & 1) ? rsu : rsw, weight_row(tr * 32) + r, group);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) next_qa[i].v = scale_rest(rsa, (wm * MT + i) * 32 + r, group);
    };
    auto load_w_pairs = [&](int group) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int tr = wn * NT + i;
                flying_qw[k][i] = scale_pair(SWIGLU && (i & 1) ? rsu : rsw, weight_row(tr * 32) + r, group + 2 * k);
            }
    };
    auto load_a_pair = [&](int group) {
#pragma unroll
        for (int i = 0; i < MT; ++i) next_qa[i] = scale_pair(rsa, (wm * MT + i) * 32 + r, group);
    };
    auto next_pair = [&] {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            next_qw[i] = ready_qw[0][i];
#pragma unroll
            for (int k = 1; k < kAhead; ++k) ready_qw[k - 1][i] = ready_qw[k][i];
        }
    };
    // Both halves of a wave get the lower half's group (HALF 0) or the upper half's, from the
    // byte on at which row r begins (rows of a tile are 32 apart, so all of its like it).
    auto of_half = [](uint32_t v, int half) {
        return (uint32_t)__builtin_amdgcn_permlane32_swap(v, v, false, false)[half];
    };
    auto group_of = [&](const Pair& p, const Scales& sc, auto half) {
        constexpr int HALF = decltype(half)::value;
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = of_half(p.v[i], HALF);
        if constexpr (!WORDS) {
            const uint32_t behind = HALF ? p.last : of_half(p.v[0], 1);
            const int by = (sc.skip + r * nblk) & 3;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_alignbyte(i < 3 ? o[i + 1] : behind, o[i], by);
        }
        return o;
    };
    auto take_half = [&](auto half) {
#pragma unroll
        for (int i = 0; i < NT; ++i) qw[i] = group_of(next_qw[i], SWIGLU && (i & 1) ? rsu : rsw, half);
#pragma unroll
        for (int i = 0; i < MT; ++i) qa[i] = group_of(next_qa[i], rsa, half);
    };
    auto take_rest = [&](int group) {
        auto placed = [&](u32x4 v) {
            if constexpr (!WORDS) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    // bytes that belong to a block in front: none, one or both
                    const int b = group * kGroupChunks + i * kStageChunks + 2 * g;
                    v[i] = (v[i] >> (8 * min(max(b - (nblk - 2), 0), 2))) << (16 * g);
                }
            }
            return v;
        };
#pragma unroll
        for (int i = 0; i < NT; ++i) qw[i] = placed(next_qw[i].v);
#pragma unroll
        for (int i = 0; i < MT; ++i) qa[i] = placed(next_qa[i].v);
    };
    uint32_t sw[NT], sa[MT];      // of one stage: bytes 0 and 1
    auto stage_scales = [&](int i) {
#pragma unroll
        for (int j = 0; j < NT; ++j) sw[j] = qw[j][i] >> (16 * g);
#pragma unroll
        for (int j = 0; j < MT; ++j) sa[j] = qa[j][i] >> (16 * g);
    };

    i32x8 fw[2][NT], fa[2][MT];
    const uint32_t frag0 = (uint32_t)(r * kStageBytes + (((2 * g) ^ (r / 2 & 3)) * 16));
    // The fragments of matrix step `step` into set `step`.
    auto read_frags = [&](int step, const uint8_t* lds) {
        const uint32_t at = frag0 ^ (uint32_t)(step * 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const u32x4 v = *(const u32x4*)(lds + kA + (wn * NT + i) * 32 * kStageBytes + at);
            fw[step][i] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const u32x4 v = *(const u32x4*)(lds + (wm * MT + i) * 32 * kStageBytes + at);
            fa[step][i] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
    };

    f32x16 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

// The order of loads and matrix instructions stays as written from step to step, LDS
// reads spread over the matrix instructions.
#define MOE_MX_STEP(STEP)                                                                   \
    _Pragma("unroll") for (int i = 0; i < NT; ++i)                                          \
        _Pragma("unroll") for (int j = 0; j < MT; ++j)                                      \
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(                    \
                fw[STEP][i], fa[STEP][j], acc[i][j], kFp4, kFp4, STEP, (int)sw[i], STEP,    \
                (int)sa[j]);                                                                \
    _Pragma("unroll") for (int i = 0; i < NT + MT; ++i) {                                   \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0); /* one LDS read */               \
        __builtin_amdgcn_sched_group_barrier(0x008, NT * MT / (NT + MT), 0);                \
    }                                                                                       \
    __builtin_amdgcn_sched_barrier(0)

    constexpr int kLoads = kLoadsA + kLoadsW;    // of a wave for a stage
// Stage s, number I of its group, in LDS buffer LDS, its first fragments already read; the
// next stage is in NEXT, or on its way (s + 2 and s + 3 may be in flight when s + 1 has to be there).
#define MOE_MX_STAGE(LDS, NEXT, I) \
    stage_scales(I);               \
    read_frags(1, LDS);            \
    MOE_MX_STEP(0);                \
    stage_sync<2 * kLoads>();      \
    load_stage(LDS, s + kGroup);   \
    read_frags(0, NEXT);           \
    MOE_MX_STEP(1);                \
    ++s

// The whole group that begins with stage s.
#define MOE_MX_GROUP()              \
    MOE_MX_STAGE(lds0, lds1, 0);    \
    MOE_MX_STAGE(lds1, lds2, 1);    \
    MOE_MX_STAGE(lds2, lds3, 2);    \
    MOE_MX_STAGE(lds3, lds0, 3)

    const int pairs = nblk / (2 * kGroupChunks);
    load_w_pairs(0);
    load_a_pair(0);
    load_stage(lds0, 0);
    load_stage(lds1, 1);      // past the last stage: zeros
    load_stage(lds2, 2);
    load_stage(lds3, 3);
    int s = 0;
    stage_sync<3 * kLoads>();
    read_frags(0, lds0);
    for (int p = 0; p < pairs;) {      // what is loaded behind the last pair is not used
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < NT; ++i) ready_qw[k][i] = flying_qw[k][i];
        load_w_pairs(2 * (p + kAhead));
        const int end = min(p + kAhead, pairs);
#pragma unroll 1
        for (; p < end; ++p) {
            next_pair();
            take_half(std::integral_constant<int, 0>{});
            MOE_MX_GROUP();
            take_half(std::integral_constant<int, 1>{});
            load_a_pair(2 * p + 2);
            MOE_MX_GROUP();
        }
    }
    if (s < stages) load_rest(2 * pairs);
    while (s + kGroup <= stages) {
        take_rest(s / kGroup);
        load_rest(s / kGroup + 1);
        MOE_MX_GROUP();
    }
    take_rest(s / kGroup);
    if (s < stages) {
        MOE_MX_STAGE(lds0, lds1, 0);
    }
    if (s < stages) {
        MOE_MX_STAGE(lds1, lds2, 1);
    }
    if (s < stages) {
        MOE_MX_STAGE(lds2, lds3, 2);
    }
#undef MOE_MX_GROUP
#undef MOE_MX_STAGE
#undef MOE_MX_STEP
    // No load into LDS may be in flight when it is written below, or goes to the next
    // workgroup.
    stage_sync<0>();

    // A lane holds column r of a tile (a row of y) and weight rows 8 * p + 4 * g + 0..3 of it:
    // stores of its own values would be 8 bytes to a row.  Each wave turns 32 rows at a time
    // in its quarter of the LDS and stores whole stretches of a row, 16 bytes a lane.
    constexpr int kCols = NT * 32 / (SWIGLU ? 2 : 1);     // output columns of a wave
    static_assert(32 * (kCols * 4 + 16) <= LDS, "a wave's 32 rows fit one buffer");
    uint8_t* turn = wave == 0 ? lds0 : wave == 1 ? lds1 : wave == 2 ? lds2 : lds3;
    const int64_t c0 = n0 + wn * kCols;
    auto store_rows = [&](auto f32) {
        constexpr bool F32 = decltype(f32)::value;
        constexpr int kEl = F32 ? 4 : 2;
        constexpr int kPitch = kCols * kEl + 16;          // spreads rows over the banks
        constexpr int kLanes = kCols * kEl / 16;          // lanes of a row
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row0 = (wm * MT + j) * 32;
            if (row0 >= t.rows) break;
#pragma unroll
            for (int i = 0; i < NT; i += SWIGLU ? 2 : 1)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float z = acc[i][j][4 * p + q];
                        if constexpr (SWIGLU) v[q] = (F32 ? silu_of(z) : silu_for_bf16(z)) * acc[i + 1][j][4 * p + q];
                        else v[q] = z;
                    }
                    uint8_t* at = turn + r * kPitch + (i / (SWIGLU ? 2 : 1) * 32 + 8 * p + 4 * g) * kEl;
                    if constexpr (F32) *(f32x4*)at = f32x4{v[0], v[1], v[2], v[3]};
                    else *(u32x2*)at = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int k = 0; k < 32 * kLanes / kWave; ++k) {
                const int row = k * (kWave / kLanes) + lane / kLanes;
                const int64_t n = c0 + lane % kLanes * (16 / kEl);
                const u32x4 v = *(const u32x4*)(turn + row * kPitch + lane % kLanes * 16);
                if (row0 + row < t.rows && n < NO)
                    st16((uint8_t*)a.y + ((t.row0 + row0 + row) * NO + n) * kEl, v);
            }
            __builtin_amdgcn_wave_barrier();
        }
    };
    if (a.y_f32) store_rows(std::true_type{});
    else store_rows(std::false_type{});
}

// A tile of up to 128 rows that is half full at the most is worked on as one of half the
// height: 4096 rows of 64 experts (4096 x 7168) 241 -> 232 us, 8192 295 -> 285.  (At 256 rows
// it did not pay: 650 -> 659 us for 32768 rows.)
template <int BM, bool SWIGLU, bool WORDS>
__global__ __launch_bounds__(kThreads, (BM <= 64 ? 2 : 1)) void product_kernel(ProductArgs a, int col_tiles,
                                                              int64_t base) {
    constexpr int kLds = (BM + kBN) * kStageBytes;
    __shared__ __align__(16) uint8_t lds0[kLds], lds1[kLds], lds2[kLds], lds3[kLds];
    int col = 0;
    Tile t = find_tile<BM>(a, base + blockIdx.x, col_tiles, col);
    // the same in every lane: into scalar registers, where descriptors have to be
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.row0 = uniform(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    col = __builtin_amdgcn_readfirstlane(col);
    if (t.e < 0) return;
    constexpr bool kHalves = BM <= 128;
    if (kHalves && t.rows <= BM / 2)
        product_tile<(kHalves ? BM / 2 : BM), SWIGLU, WORDS>(a, t, col, lds0, lds1, lds2, lds3);
    else
        product_tile<BM, SWIGLU, WORDS>(a, t, col, lds0, lds1, lds2, lds3);
}

// ---------------------------------------------------------------------------
// Few rows and few weight rows: tiles of 32 by 64, so that there are enough of them, and K
// is split over the waves of a workgroup.  A wave streams its quarter through LDS buffers
// of its own (stages of 128 elements, four deep), with no barrier until the four sums are
// joined, in the order of the waves.  One row by 8192 x 8192 takes 14.6 us, 2.4 TB/s: the
// latency of 16 stages a wave and the launch (21.5 with tiles of 64 rows by 256).
// ---------------------------------------------------------------------------
template <bool SWIGLU, bool WORDS>
__global__ __launch_bounds__(kThreads, 1) void product_narrow_kernel(ProductArgs a, int col_tiles,
                                                                     int64_t base) {
    constexpr int kA = kNarrowRows * kStageBytes;
    constexpr int kStage = kA + kNarrowCols * kStageBytes;
    __shared__ __align__(16) uint8_t lds0[kWaves * kStage], lds1[kWaves * kStage];
    __shared__ __align__(16) uint8_t lds2[kWaves * kStage], lds3[kWaves * kStage];
    int col = 0;
    Tile t = find_tile<kNarrowRows>(a, base + blockIdx.x, col_tiles, col);
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.row0 = uniform(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    col = __builtin_amdgcn_readfirstlane(col);
    if (t.e < 0) return;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t rb = a.H / 2;
    const int nblk = (int)(a.H / kMxBlock);
    const int stages = (nblk + kStageChunks - 1) / kStageChunks;
    const int per = (stages + kWaves - 1) / kWaves;
    const int s0 = min(wave * per, stages), s1 = min(s0 + per, stages);     // the wave's
    const int64_t NO = SWIGLU ? a.N / 2 : a.N;
    constexpr int kCols = SWIGLU ? kNarrowCols / 2 : kNarrowCols;
    const int64_t n0 = (int64_t)col * kCols;
    const int64_t wrow = (int64_t)t.e * a.N + n0;
    const int wrows = (int)(NO - n0 < kCols ? NO - n0 : kCols);
    const auto ra = rows_of(a.a, t.row0, t.rows, rb);
    const auto rw = rows_of(a.w, wrow, wrows, rb);
    const auto ru = SWIGLU ? rows_of(a.w, wrow + NO, wrows, rb) : rw;
    const auto rsa = rows_of(a.a_scales, t.row0, t.rows, nblk);
    const auto rsw = rows_of(a.w_scales, wrow, wrows, nblk);
    const auto rsu = SWIGLU ? rows_of(a.w_scales, wrow + NO, wrows, nblk) : rsw;

    constexpr int kLoads = kStage / 1024;
    const int chunk = (lane % 4) ^ (lane / 8 % 4);
    auto load_stage = [&](uint8_t* lds, int s) {
        const uint32_t at = (uint32_t)(s * kStageChunks + chunk);
        const uint32_t bad = outside_if((int)at >= nblk) | outside_if(s >= s1);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r16 = i * 16;           // rows 0 to 31: tokens, then weights
            const bool w = r16 >= kNarrowRows, up = SWIGLU && r16 >= kNarrowRows + 32;
            const int row = (up ? r16 - kNarrowRows - 32 : w ? r16 - kNarrowRows : r16) + lane / 4;
            stage16(up ? ru : w ? rw : ra, lds + wave * kStage + r16 * kStageBytes,
                    ((uint32_t)row * (uint32_t)rb + at * 16) | bad);
        }
    };
    const int r = lane % 32, g = lane / 32;
    // scales of four stages from s on: [0], [1] of the weight tiles, [2] of the token rows; as
    // in product_tile where rows do not start at whole words
    u32x4 next[3];
    auto load_scales = [&](int s) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const auto rs = k == 2 ? rsa : SWIGLU && k == 1 ? rsu : rsw;
            const uint32_t off = (uint32_t)(k == 1 && !SWIGLU ? r + 32 : r) * (uint32_t)nblk;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const int b = (s + i) * kStageChunks;
                if constexpr (WORDS) {
                    next[k][i] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)((off + b) | outside_if(b >= nblk)), 0, 0);
                } else {
                    const int at = min(b + 2 * g, nblk - 2);
                    next[k][i] = nblk > 1 ? __builtin_amdgcn_raw_buffer_load_b16(rs, (int)(off + at), 0, 0)
                                          : __builtin_amdgcn_raw_buffer_load_b8(rs, (int)off, 0, 0) << 8;
                }
            }
        }
    };
    f32x16 acc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][q] = 0.0f;
    auto frag = [&](const uint8_t* lds, int tile, int step) {
        const u32x4 v = ld16(lds + wave * kStage + (tile * 32 + r) * kStageBytes +
                             (((2 * g + step) ^ (r / 2 & 3)) * 16));
        return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
    };
    // Stage s has landed (three more may be in flight): multiply it, then fill its buffer.
    auto use_stage = [&](uint8_t* lds, const uint32_t (&sc)[3], int s) {
        constexpr int N = 3 * kLoads;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0xf70);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        i32x8 f[2][3];
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
            for (int k = 0; k < 3; ++k) f[step][k] = frag(lds, k, step);
#define MOE_MX_NARROW(STEP)                                                                    \
    _Pragma("unroll") for (int i = 0; i < 2; ++i)                                              \
        acc[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(                              \
            f[STEP][i + 1], f[STEP][0], acc[i], kFp4, kFp4, STEP, (int)sc[i], STEP, (int)sc[2])
        MOE_MX_NARROW(0);
        MOE_MX_NARROW(1);
#undef MOE_MX_NARROW
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xc07f);      // the reads are in registers
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        load_stage(lds, s + kGroup);
    };

    load_scales(s0);
    load_stage(lds0, s0);
    load_stage(lds1, s0 + 1);
    load_stage(lds2, s0 + 2);
    load_stage(lds3, s0 + 3);
    for (int s = s0; s < s1; s += kGroup) {
        uint32_t sc[kGroup][3];
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if constexpr (WORDS) {
                    sc[i][k] = next[k][i] >> (16 * g);
                } else {
                    const int b = (s + i) * kStageChunks + 2 * g;
                    sc[i][k] = next[k][i] >> (8 * min(max(b - (nblk - 2), 0), 2));
                }
            }
        load_scales(s + kGroup);
        use_stage(lds0, sc[0], s);
        use_stage(lds1, sc[1], s + 1);
        use_stage(lds2, sc[2], s + 2);
        use_stage(lds3, sc[3], s + 3);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();

    // each wave's sums, row by row of y, in one buffer
    constexpr int kPitch = kNarrowCols + 4;
    static_assert(kNarrowRows * kPitch * 4 <= sizeof(lds0), "a wave's sums fit one buffer");
    float* turn = (float*)(wave == 0 ? lds0 : wave == 1 ? lds1 : wave == 2 ? lds2 : lds3);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p)
            *(f32x4*)(turn + r * kPitch + i * 32 + 8 * p + 4 * g) =
                f32x4{acc[i][4 * p], acc[i][4 * p + 1], acc[i][4 * p + 2], acc[i][4 * p + 3]};
    __syncthreads();
    const int row = threadIdx.x / 8, c = threadIdx.x % 8;
    if (row >= t.rows) return;
    auto joined = [&](int n) {
        f32x4 v = *(const f32x4*)((const float*)lds0 + row * kPitch + n);
        v += *(const f32x4*)((const float*)lds1 + row * kPitch + n);
        v += *(const f32x4*)((const float*)lds2 + row * kPitch + n);
        v += *(const f32x4*)((const float*)lds3 + row * kPitch + n);
        return v;
    };
#pragma unroll
    for (int k = 0; k < kCols / 32; ++k) {
        const int n = k * 32 + c * 4;
        if (n0 + n >= NO) continue;
        f32x4 v = joined(n);
        if constexpr (SWIGLU) {
            const f32x4 u = joined(n + 32);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = silu_of(v[q]) * u[q];
        }
        const int64_t at = (t.row0 + row) * NO + n0 + n;
        if (a.y_f32) *(f32x4*)((float*)a.y + at) = v;
        else *(u32x2*)((uint16_t*)a.y + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

bool whole_words(const ProductArgs& a) {
    return a.H / kMxBlock % 4 == 0 && ((uintptr_t)a.a_scales | (uintptr_t)a.w_scales) % 4 == 0;
}

// Launches KERNEL<.., swiglu, whole words> over the most tiles of BM rows by BN weight rows
// that there can be: every expert may have one that is not full.
#define MOE_PRODUCT(BM, BN, KERNEL, ...)                                                           \
    do {                                                                                           \
        const int64_t cols = a.swiglu ? a.N / 2 : a.N, width = a.swiglu ? (BN) / 2 : (BN);         \
        const int col_tiles = (int)((cols + width - 1) / width);                                   \
        const int64_t row_tiles = a.rows / (BM) + (a.E < a.rows ? a.E : a.rows);                   \
        const int64_t blocks = (row_tiles * col_tiles + 7) / 8 * 8;                                \
        for (int64_t base = 0; base < blocks; base += kMaxGrid) {                                  \
            const dim3 grid((unsigned)(blocks - base < kMaxGrid ? blocks - base : kMaxGrid));      \
            const bool words = whole_words(a);                                                     \
            if (a.swiglu && words) KERNEL<__VA_ARGS__ true, true><<<grid, kThreads, 0, s>>>(a, col_tiles, base);   \
            else if (a.swiglu) KERNEL<__VA_ARGS__ true, false><<<grid, kThreads, 0, s>>>(a, col_tiles, base);      \
            else if (words) KERNEL<__VA_ARGS__ false, true><<<grid, kThreads, 0, s>>>(a, col_tiles, base);         \
            else KERNEL<__VA_ARGS__ false, false><<<grid, kThreads, 0, s>>>(a, col_tiles, base);   \
        }                                                                                          \
    } while (0)
#define MOE_COMMA ,

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    switch (ProductSize{a.rows, a.N, a.E}.tile_rows()) {
        case kNarrowRows: MOE_PRODUCT(kNarrowRows, kNarrowCols, product_narrow_kernel); break;
        case 64: MOE_PRODUCT(64, kTileCols, product_kernel, 64 MOE_COMMA); break;
        case 128: MOE_PRODUCT(128, kTileCols, product_kernel, 128 MOE_COMMA); break;
        default: MOE_PRODUCT(256, kTileCols, product_kernel, 256 MOE_COMMA);
    }
    return hipGetLastError();
}

}  // namespace moe
