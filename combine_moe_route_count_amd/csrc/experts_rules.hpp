// experts_rules.hpp - what the experts' step decides with whole numbers alone: which kernel takes a
// product of a given size, and the layout of the lists in experts_decode's workspace
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
// 256 163, 148, 128; 384 224, 200, 185.  (The mean is that of the buffer's rows: the host does not
// know the counts.  Padded segments that are mostly empty get higher tiles than their rows need.)
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

}  // namespace moe
