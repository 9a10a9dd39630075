// experts_rules.hpp - what the experts' step decides with whole numbers alone: which kernels take a
// product or a decode step of a given size, and the layout of the lists in experts_decode's workspace
// with their bounds.  Plain C++, so that it can be checked without a GPU.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define MOE_HOST_DEVICE __host__ __device__
#else
#define MOE_HOST_DEVICE
#endif

namespace moe {

// The work of one pass over an expert's weights: up to a pass's width of its entries.  Slot s
// belongs to expert[s] and has the entries ent[first[s]] .. ent[first[s + 1] - 1].  All
// three, and the number n of slots, are one block of 16-bit words, sized by the number N of
// entries: n, one unused, expert [N], first [N+2], ent [N].
struct ListLayout {
    int N;
    MOE_HOST_DEVICE constexpr int expert() const { return 2; }
    MOE_HOST_DEVICE constexpr int first() const { return 2 + N; }
    MOE_HOST_DEVICE constexpr int ent() const { return 4 + 2 * N; }
    MOE_HOST_DEVICE constexpr int words32() const { return (4 + 3 * N + 1) / 2; }
    // 16-bit word i of a block as it is used, whatever v it holds: n and first at most N, so that
    // first[s + 1] ends every list within ent; ids of experts and entries below E and N.
    MOE_HOST_DEVICE constexpr uint32_t bounded(int i, uint32_t v, int E) const {
        const int most = i >= ent() ? N - 1 : i >= first() || i < expert() ? N : E - 1;
        return v < (uint32_t)most ? v : (uint32_t)most;
    }
};

constexpr int kCUs = 256;

// ---------------------------------------------------------------------------
// expert_product_mxfp4
// ---------------------------------------------------------------------------
constexpr int kNarrowRows = 32, kNarrowCols = 64;    // a tile of product_narrow_kernel
constexpr int kTileCols = 256;                       // weight rows of a tile of product_kernel

// Rows of a product's tiles: 64, 128 or 256, or 32 where narrow tiles take over.
//
// Tile heights 64, 128, 256 by the mean rows of an expert, in us (32 experts with uneven
// loads, 4096 x 4096): mean 24 62, 64, 72; 64 73, 75, 82; 96 91, 90, 94; 192 135, 117, 122;
// 256 163, 148, 128; 384 224, 200, 185.  The mean is that of the buffer's rows, for the host does not
// know the counts: padded segments that are mostly empty get higher tiles than their rows need.  64
// experts with room for 256 rows (4096 x 7168, SwiGLU), tiles of 256 and 64: 12 rows in each 228
// and 188 us, 64 244, 204; 128 271, 287; 200 306, 451.
// A height whose tiles would leave 100 CUs without one gives way to the next lower, in us:
// 120 tiles of 256 rows 22.2 against 16.9 with 128, 136 35.7 and 28.4, 168 23.6 and 27.6,
// 184 37.3 and 44.9; 138 tiles of 128 rows 22.5 against 20.2 with 64, 144 22.8 and 20.8,
// 184 24.9 and 31.2, 192 26.4 and 31.9.
// Narrow tiles where nearly each can have a CU, in us against tiles of 64 rows: 56 of them 9.0
// and 17.8, 160 11.6 and 16.1, 256 17.9 and 27.6, 264 17.2 and 27.2; 320 20.3 and 16.4,
// 512 31.5 and 27.8.
struct ProductSize {
    int64_t rows, N;
    int E;
    constexpr int64_t tiles(int64_t height, int64_t width) const {       // about
        const int64_t used = E < rows ? E : rows;
        const int64_t row_tiles = (2 * rows / height + used) / 2;
        return (row_tiles > used ? row_tiles : used) * ((N + width - 1) / width);
    }
    constexpr int tile_rows() const {
        constexpr int64_t kIdle = 100;
        const int64_t mean = rows / E;
        if (tiles(kNarrowRows, kNarrowCols) <= kCUs + kCUs / 8) return kNarrowRows;
        if (mean <= 64 || tiles(128, kTileCols) < kCUs - kIdle) return 64;
        if (mean < 224 || tiles(256, kTileCols) < kCUs - kIdle) return 128;
        return 256;
    }
};

// ---------------------------------------------------------------------------
// experts_decode
// ---------------------------------------------------------------------------
// The kernel of one of the two products: entries at a time (16 or 32, or as many as fit with the
// parts of h as columns of their own: pack), elements of a row in a stage, waves, and whether these
// share out K (split).
struct StreamForm {
    int width, stage, waves;
    bool split, pack;
};

struct DecodeSize {
    int64_t T, H, I;
    int K, E;
    bool mx;         // MXFP4 weights
    int parts;       // of h: 2, or 3 for an f32 result
    constexpr int64_t entries() const { return T * K; }
    constexpr int64_t used() const { return entries() < E ? entries() : E; }    // experts, at the most
    // Passes over an expert's weights that the entries need, about.
    constexpr int64_t slots(int width) const {
        const int64_t full = (2 * entries() / width + used()) / 2;
        return full > used() ? full : used();
    }
    // The first product's K is split over the waves where that still leaves a CU no more than
    // two items, in us without and with: bf16 64 items 26.3, 18.5, 256 35.0, 28.4, 512 40.6,
    // 39.1, 1088 40.2, 56.2; MXFP4 36 items 47.0, 26.3, 128 23.5, 17.9, 320 33.5, 25.3, 512
    // 26.4, 26.1, 768 22.4, 25.7, 1024 32.6, 41.2.
    constexpr bool split() const { return slots(16) * ((I + 15) / 16) <= 2 * kCUs; }
    // 32 entries at a time instead of 16, in us without and with, by entries per expert: bf16 8 152,
    // 150; 10 59, 60; 16 74, 62; 21 495, 334; 32 113, 84.  MXFP4, whose wide stages are half as long,
    // where 4 waves share them 16 68.6, 69.1; 21 175, 144; 24 92, 84; 32 98, 91; 64 169, 144; where
    // 2 do 10 35, 50; 16 42, 51; 32 57, 62; 128 153, 160 (f32 result 158, 223).
    constexpr bool wide() const {
        if (split()) return false;
        return mx ? entries() > 16 * (int64_t)E && waves(I, 64) == 4 && waves(H, 128) == 4
                  : entries() > 8 * (int64_t)E;
    }
    // Parts of h as columns, in us without and with, by entries per expert: one token of 8 experts 49.1,
    // 45.2 (4 experts a token, f32 result 49.4, 43.8); 2 240, 238 (f32 result 261, 240); 4 272, 270; 8
    // 290, 298, where some experts have too many for one pass.  (The parts are read by one
    // descriptor of less than 2^31 bytes.)
    constexpr bool pack() const {
        return mx && entries() <= 4 * (int64_t)E && entries() * I * 2 * parts < ((int64_t)1 << 31);
    }
    // 4 waves share the entries' rows; 2 where 4 would leave CUs without work (rows: of a workgroup of 4).
    constexpr int waves(int64_t M, int rows) const {
        return used() * ((M + rows - 1) / rows) >= 2 * kCUs ? 4 : 2;
    }
    // Whole cache lines of MXFP4 rows (stages of 256) where a group of stages is not mostly zeros:
    // 163 -> 152 us (111 experts' W1 and W3 of 1024 x 7168), 238 -> 226 both products (32 tokens).
    // Not with the parts of h apart: their stages leave the CU one workgroup, 97 -> 114 us (W2).
    static constexpr int kLong = 768;
    constexpr StreamForm up() const {
        if (split()) return {16, mx ? 128 : 64, 4, true, false};
        const int stage = !mx ? 64 : !wide() && H >= kLong ? 256 : 128;
        return {wide() ? 32 : 16, stage, waves(I, 64), false, false};
    }
    constexpr StreamForm down() const {
        const int stage = !mx ? 64 : pack() && I >= kLong ? 256 : 128;
        return {pack() ? 16 / parts : wide() ? 32 : 16, stage, waves(H, 128), false, pack()};
    }
};

}  // namespace moe
