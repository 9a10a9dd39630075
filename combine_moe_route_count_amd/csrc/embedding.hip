// embedding.hip - embedding lookup with scaling, and its gradient by sorted
// tokens.
//
// Lookup: out[n] = scale * table[ids[n]], a row gather.
//
// Gradient: dtable[v] = scale * sum of dout[n] over the n with ids[n] = v.  The
// positions are sorted by token id, stably, so that each table row owns one run of
// positions in ascending order: no atomics, one fixed order.  The sorted order is
// cut into windows of a few positions.  A workgroup streams the rows of one window,
// whatever runs they belong to, and writes a table row wherever a run ends; the
// parts of runs that cross windows go to f32 rows of the workspace, and a last
// launch joins them in order.  So every workgroup that reads dout has the same work,
// whether a token occurs once or in half of all positions.  The join has not: there one
// workgroup adds all parts of a run for its columns, a part per window.  What that costs
// at 65536 tokens of 4096 into 131072 f32 rows: 459 us with Zipf tokens, 477 with half
// of all positions on one token, 491 with all on it.
//
// The sort: up to kSmallSort positions are ranked by counting, one launch.  More are
// radix sorted by digits of at most 9 bits, with the routing's stable ranks inside
// tiles of 1024 (route_device.hpp): a pass ranks the tiles, and then moves (id,
// position).  Up to kOwnScanTiles tiles, each moving workgroup sums the tiles' counts
// for itself; more tiles go through the one-launch routing (route_fused.hip), whose
// last workgroup scans them.
//
// What bounds it: one read of dout's rows and one write of the table, most of it zeros
// for a large vocabulary.  65536 tokens of 4096 (bf16, Zipf) into 131072 f32 rows, 2.66
// GB: 469 us = 5.7 TB/s, of it zeros 260 us (7.0 TB/s), windows 161 (5.2 TB/s), sort 23
// and join 15.
#include "train_device.hpp"
#include "internal.hpp"
#include "route_device.hpp"

namespace moe {

namespace {

constexpr int kEmbThreads = 256;
constexpr int kSmallSort = 4096;   // positions

// Bits of a digit: at most 9 (512 keys).  Fewer for long inputs: own scans read tiles x
// tiles x keys counts in all, which stay under 2^24; the one-launch routing keeps its
// tiles x keys counts in registers up to 2^14.  Own scans against the routing, the whole
// gradient: 10136 tokens of 80 35.0 and 39.7 us, 65536 of 64 48.9 and 63.2, 131072 of 256
// 65.5 and 82.7, 262144 of 256 115 and 131.  The routing's shorter digits take more passes,
// two launches each: with a table of 131072 rows of 64 f32, 262144 tokens 68 us, 262145 93,
// 524288 135, 2^20 235, 2^22 885.
constexpr int64_t kOwnScanTiles = 256;
constexpr int kDigitMost = 9, kDigitLeast = 4;
constexpr int64_t kRoutedCounts = (int64_t)1 << 14;
inline int digit_bits(int64_t tiles) {
    int bits = kDigitMost;
    while (bits > kDigitLeast && (tiles <= kOwnScanTiles ? (tiles * tiles) << bits > (1 << 24)
                                                         : tiles << bits > kRoutedCounts))
        --bits;
    return bits;
}

// Tiles x keys counts that the workspace holds for ids of id_bits: enough for every sort
// of at most this many tiles, since fewer tiles take longer digits.  Past kLongDigitTiles
// all digits have kDigitLeast bits.
constexpr int64_t kLongDigitTiles = kRoutedCounts >> (kDigitLeast + 1);
inline int64_t count_room(int64_t tiles, int id_bits) {
    const int most = id_bits < kDigitMost ? id_bits : kDigitMost;
    const int least = id_bits < kDigitLeast ? id_bits : kDigitLeast;
    const int64_t few = (tiles < kLongDigitTiles ? tiles : kLongDigitTiles) << most;
    const int64_t many = tiles << least;
    return few > many ? few : many;
}

__device__ __forceinline__ int64_t token_id(const void* ids, int id_bytes, int64_t n) {
    return id_bytes == 8 ? ((const int64_t*)ids)[n] : (int64_t)((const int32_t*)ids)[n];
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
// Workgroup (token, chunk of the row), two units per lane so that both loads of a
// lane are in flight behind the one read of the token id.  Table rows go through
// the caches, since frequent tokens read the same ones again; out is stored
// non-temporally, in 16-byte units: 8 bf16 or 4 f32 elements.  Measured, 16384
// tokens of 7168 from an f32 table of 131072 rows to bf16: streamed loads 128 us,
// cached 95, with non-temporal stores 88, two units per lane 81, workgroups of up to
// 512 threads 80.  f32 to f32 (8192 tokens of 4096): 8-element units 43 us,
// 4-element units 32.4, workgroups of up to 128 threads 31.1.
constexpr int kLookupUnits = 2;
constexpr int lookup_threads(bool out_f32) { return out_f32 ? 128 : 512; }

template <bool TF32, bool OF32>
__global__ __launch_bounds__(lookup_threads(OF32)) void embedding_kernel(EmbeddingArgs a,
                                                                         int nch) {
    constexpr int EL = OF32 ? 4 : 8;
    const int units = (int)(a.H / EL);
    const int64_t items = a.N * nch;
    for (int64_t wi = blockIdx.x; wi < items; wi += gridDim.x) {
        const int64_t n = wi / nch;
        const int c = (int)(wi - n * nch);
        const int64_t id = token_id(a.ids, a.id_bytes, n);
        const bool some = id >= 0 && id < a.V;
        if (a.stats && !some && id != -1 && c == 0 && threadIdx.x == 0) atomicAdd(a.stats, 1);
        const int u0 = c * kLookupUnits * (int)blockDim.x + (int)threadIdx.x;
        FloatUnit<TF32, EL> x[kLookupUnits];
#pragma unroll
        for (int i = 0; i < kLookupUnits; ++i) {
            const int u = u0 + i * (int)blockDim.x;
            if (some && u < units) x[i].load_cached(a.table, id * a.H + (int64_t)u * EL);
        }
#pragma unroll
        for (int i = 0; i < kLookupUnits; ++i) {
            const int u = u0 + i * (int)blockDim.x;
            if (u >= units) continue;
            float v[EL];
#pragma unroll
            for (int j = 0; j < EL; ++j) v[j] = 0.0f;
            if (some) {
                x[i].get(v);
#pragma unroll
                for (int j = 0; j < EL; ++j) v[j] = v[j] * a.scale;
            }
            store_unit<OF32, true>(a.out, n * a.H + (int64_t)u * EL, v);
        }
    }
}

// The count of ids outside [0,V) starts at 0 in a launch of its own: the lookup then
// adds to it for such ids only.
__global__ void clear_count_kernel(int32_t* stats) { *stats = 0; }

template <bool TF32, bool OF32>
void embedding_go(const EmbeddingArgs& a, hipStream_t s) {
    const int64_t units = a.H / (OF32 ? 4 : 8);
    const int threads = row_threads((units + kLookupUnits - 1) / kLookupUnits, lookup_threads(OF32));
    const int nch = (int)((units + threads * kLookupUnits - 1) / (threads * kLookupUnits));
    if (a.stats) clear_count_kernel<<<dim3(1), dim3(1), 0, s>>>(a.stats);
    if (a.N > 0)
        embedding_kernel<TF32, OF32><<<capped_grid(a.N * nch), dim3(threads), 0, s>>>(a, nch);
}

// ---------------------------------------------------------------------------
// gradient: the sort
// ---------------------------------------------------------------------------
// Table rows to clear, kEmbThreads lane-units of 16 bytes per workgroup: several
// narrow rows, or one chunk of a wide one.  One non-temporal store per lane and many
// small workgroups: 7.0 TB/s, against 5.4-6.1 with four stores per lane, 3.9 to 6.3
// in a flat loop, and 4.5 with stores through L2 (131072 rows of 4096 f32).
constexpr int zero_unit(bool f32) { return f32 ? 4 : 8; }

struct ZeroRows {
    int units;     // lane-units of a row
    int rows;      // rows per workgroup, if a row is narrow (else 1)
    int chunks;    // workgroups per row, if it is wide (else 1)
    int64_t blocks;
};

ZeroRows zero_layout(int64_t V, int64_t H, bool f32) {
    ZeroRows z;
    z.units = (int)(H / zero_unit(f32));
    z.rows = z.units < kEmbThreads ? kEmbThreads / z.units : 1;
    z.chunks = (z.units + kEmbThreads - 1) / kEmbThreads;
    z.blocks = (V + z.rows - 1) / z.rows * z.chunks;
    return z;
}

// Row and unit of thread tid of block b; false if it has none.
__device__ __forceinline__ bool zero_place(const ZeroRows& z, int64_t b, int tid, int64_t V,
                                           int64_t& v, int& u) {
    if (z.chunks > 1 || z.rows == 1) {
        v = b / z.chunks;
        u = (int)(b - v * z.chunks) * kEmbThreads + tid;
        return u < z.units;
    }
    const int r = tid / z.units;
    v = b * z.rows + r;
    u = tid - r * z.units;
    return r < z.rows && v < V;
}

template <bool OF32>
__device__ __forceinline__ void zero_store(void* table, int64_t H, int64_t v, int u) {
    constexpr int EL = zero_unit(OF32);
    float z[EL];
#pragma unroll
    for (int j = 0; j < EL; ++j) z[j] = 0.0f;
    store_unit<OF32, true>(table, v * H + (int64_t)u * EL, z);
}

struct MoveArgs {              // one radix pass
    DigitSource d;
    int64_t N;
    int32_t* local_rank;
    int32_t* tile_cnt;         // [tiles][NK] counts; after the one-launch routing, bases
    int32_t* tile_flags;
    int32_t* off;              // [NK+1]
    int tiles, NK, nbits;
    const int32_t* in_pos;     // null: the position is the entry's own number
    int32_t* out_id;
    int32_t* out_pos;
    uint8_t* clear;            // first of several passes: [V] flags to clear, or null
    uint8_t* present;          // last of several passes: flags of the ids that occur, or null
    int64_t V;
    void* dtable;              // table to zero by the workgroups past move_blocks, or null
    bool dtable_f32;
    int64_t H;
    int64_t move_blocks;
    ZeroRows zero;
};

constexpr int kSortThreads = kTile;   // a tile per workgroup, an entry per thread
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int64_t kMaxSortGrid = (int64_t)1 << 20;   // moving, and as many zeroing

__global__ __launch_bounds__(kSortThreads) void digit_rank_kernel(MoveArgs a) {
    extern __shared__ int32_t run_all[];   // [kSortWaves][NK]
    rank_tile<kSortWaves, 1>(DigitKeys{a.d}, a.N, a.NK, a.nbits, (int64_t)blockIdx.x, run_all,
                             a.local_rank, a.tile_cnt, a.tile_flags);
}

// Zeroing and clearing beside a move; false if this workgroup moves nothing.
__device__ __forceinline__ bool beside_move(const MoveArgs& a) {
    constexpr int kParts = kSortThreads / kEmbThreads;
    const int part = threadIdx.x / kEmbThreads, tid = threadIdx.x % kEmbThreads;
    if (blockIdx.x >= a.move_blocks) {
        for (int64_t b = ((int64_t)blockIdx.x - a.move_blocks) * kParts + part; b < a.zero.blocks;
             b += ((int64_t)gridDim.x - a.move_blocks) * kParts) {
            int64_t v;
            int u;
            if (!zero_place(a.zero, b, tid, a.V, v, u)) continue;
            if (a.dtable_f32) zero_store<true>(a.dtable, a.H, v, u);
            else zero_store<false>(a.dtable, a.H, v, u);
        }
        return false;
    }
    if (a.clear) {
        const int64_t step = a.move_blocks * kSortThreads;
        for (int64_t v = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; v < a.V; v += step)
            a.clear[v] = 0;
    }
    return true;
}

__device__ __forceinline__ int32_t entry_id(const DigitSource& d, int64_t f) {
    return d.total ? ((const int32_t*)d.ids)[f] : (int32_t)token_id(d.ids, d.id_bytes, f);
}

__device__ __forceinline__ void move_entry(const MoveArgs& a, int64_t f, int32_t id, int64_t to) {
    a.out_id[to] = id;
    a.out_pos[to] = a.in_pos ? a.in_pos[f] : (int32_t)f;
    if (a.present) a.present[id] = 1;
}

// Move of one tile per workgroup behind its own scan: thread (key, part) sums the counts
// of a stretch of tiles, in all and before this tile.
__global__ __launch_bounds__(kSortThreads) void scan_move_kernel(MoveArgs a) {
    __shared__ int32_t before_lds[kSortThreads], total_lds[kSortThreads];
    __shared__ int32_t wave_sums[kScanThreads / kWave];
    if (!beside_move(a)) return;
    const int tid = threadIdx.x;
    const int tile = blockIdx.x;
    const int64_t f = (int64_t)tile * kTile + tid;
    const int32_t lr = f < a.N ? a.local_rank[f] : -1;
    const int32_t id = lr >= 0 ? entry_id(a.d, f) : 0;
    const int parts = kSortThreads / a.NK, per = (a.tiles + parts - 1) / parts;
    const int key = tid % a.NK, part = tid / a.NK;
    const int t0 = part * per, t1 = t0 + per < a.tiles ? t0 + per : a.tiles;
    int32_t before = 0, total = 0;
#pragma unroll 8
    for (int t = t0; t < t1; ++t) {
        const int32_t c = a.tile_cnt[(int64_t)t * a.NK + key];
        total += c;
        before += t < tile ? c : 0;
    }
    before_lds[tid] = before;
    total_lds[tid] = total;
    __syncthreads();
    if (tid < a.NK)
        for (int p = 1; p < parts; ++p) {
            before += before_lds[p * a.NK + tid];
            total += total_lds[p * a.NK + tid];
        }
    const int32_t first = block_exclusive_scan(tid < a.NK ? total : 0, wave_sums);
    if (tid < a.NK) {
        before_lds[tid] = first + before;     // read by nobody else before the barrier
        if (tile == 0) {
            a.off[tid] = first;
            if (tid == a.NK - 1) a.off[a.NK] = first + total;
        }
    }
    __syncthreads();
    if (lr >= 0)
        move_entry(a, f, id, (int64_t)before_lds[(id >> a.d.shift) & a.d.mask] + lr);
}

// Move behind the one-launch routing, which left the tiles' bases and the offsets.
__global__ __launch_bounds__(kSortThreads) void move_kernel(MoveArgs a) {
    if (!beside_move(a)) return;
    const int64_t step = a.move_blocks * kSortThreads;
    for (int64_t f = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; f < a.N; f += step) {
        const int32_t lr = a.local_rank[f];
        if (lr < 0) continue;
        const int32_t id = entry_id(a.d, f);
        const int key = (id >> a.d.shift) & a.d.mask;
        move_entry(a, f, id, (int64_t)a.off[key] + a.tile_cnt[(f / kTile) * a.NK + key] + lr);
    }
}

// Sort of up to kSmallSort ids by counting: position n goes behind every smaller id
// and behind the equal ids before it.  8 positions per workgroup, 32 threads each;
// the remaining workgroups zero the whole table meanwhile (zero_blocks, none when
// accumulating), so the sums need not know which rows to clear.  The whole gradient
// with 777 tokens took 18.5, 14.9 and 14.7 us at 4, 16 and 32 threads per position.
// By counting and by digits: 3000 tokens into 3000 rows of 256 16.9 and 22.4 us, 4096
// into 50000 rows of 2048 f32 78.6 and 87.5, but into 512 rows of 64 (one digit) 18.2
// and 16.2; 8192 into 50000 rows of 4096 180 and 159.
constexpr int kSortShare = 32;
constexpr int kSortPositions = kEmbThreads / kSortShare;

struct SmallSortArgs {
    const void* ids;
    int id_bytes;
    int64_t N, V, H;
    int32_t* id;
    int32_t* pos;
    int32_t* total;
    void* dtable;
    int sort_blocks;
    ZeroRows zero;      // no blocks when accumulating
};

template <bool OF32>
__global__ __launch_bounds__(kEmbThreads) void small_sort_kernel(SmallSortArgs a) {
    __shared__ __align__(16) int32_t key[kSmallSort];
    const int tid = threadIdx.x;
    for (int64_t b = blockIdx.x; b < a.sort_blocks + a.zero.blocks; b += gridDim.x) {
        if (b >= a.sort_blocks) {
            int64_t v;
            int u;
            if (zero_place(a.zero, b - a.sort_blocks, tid, a.V, v, u))
                zero_store<OF32>(a.dtable, a.H, v, u);
            continue;
        }
        // ids of no row sort last and are not placed
        const int padded = ((int)a.N + 3) & ~3;
        for (int m = tid; m < padded; m += kEmbThreads) {
            const int64_t id = m < a.N ? token_id(a.ids, a.id_bytes, m) : -1;
            key[m] = id >= 0 && id < a.V ? (int32_t)id : INT32_MAX;
        }
        __syncthreads();
        const int n = (int)b * kSortPositions + tid / kSortShare;
        const int own = n < a.N ? key[n] : INT32_MAX;
        const bool placed = own != INT32_MAX;
        const int mine = placed ? own : 0;
        int rank = 0, valid = 0;
        for (int m = (tid % kSortShare) * 4; m < padded; m += kSortShare * 4) {
            const int4 k = *(const int4*)&key[m];
            rank += k.x < mine + (m < n ? 1 : 0);
            rank += k.y < mine + (m + 1 < n ? 1 : 0);
            rank += k.z < mine + (m + 2 < n ? 1 : 0);
            rank += k.w < mine + (m + 3 < n ? 1 : 0);
            valid += (k.x != INT32_MAX) + (k.y != INT32_MAX) + (k.z != INT32_MAX) +
                     (k.w != INT32_MAX);
        }
#pragma unroll
        for (int d = 1; d < kSortShare; d <<= 1) {
            rank += __shfl_xor(rank, d, kWave);
            valid += __shfl_xor(valid, d, kWave);
        }
        if (tid % kSortShare == 0 && placed) {
            a.id[rank] = mine;
            a.pos[rank] = n;
        }
        if (b == 0 && tid == 0) *a.total = valid;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// gradient: the sums
// ---------------------------------------------------------------------------
struct SumArgs {
    EmbeddingGradArgs g;
    const int32_t* id;        // sorted token ids
    const int32_t* pos;       // their positions
    const int32_t* total;     // how many
    float* partial;           // [2 * windows][H]: the entering and the leaving run's part
    int window;               // positions per window
    int64_t windows;
    int nch;                  // chunks of a row
};

// Rows of the ids that do not occur, by the flags of the last move or, where one digit
// is the whole id, by its offsets.  A launch of its own: as more workgroups of the
// sums, under their registers, it ran at half the rate (524 us for both, 257 + 160
// apart, 131072 rows of 4096 f32).
template <bool OF32>
__global__ __launch_bounds__(kEmbThreads) void zero_rows_kernel(void* table, int64_t V, int64_t H,
                                                                const uint8_t* present,
                                                                const int32_t* off, ZeroRows z) {
    for (int64_t b = blockIdx.x; b < z.blocks; b += gridDim.x) {
        int64_t v;
        int u;
        if (!zero_place(z, b, threadIdx.x, V, v, u)) continue;
        const bool some = present ? present[v] != 0 : off[v + 1] != off[v];
        if (!some) zero_store<OF32>(table, H, v, u);
    }
}

// dtable[v] = base + scale * acc, one unit; base (null: 0) as loaded before.
template <bool OF32, int EL>
__device__ __forceinline__ void put_row(const SumArgs& a, int64_t v, int64_t col,
                                        const float (&acc)[EL], const FloatUnit<OF32, EL>* base) {
    float r[EL];
#pragma unroll
    for (int j = 0; j < EL; ++j) r[j] = acc[j] * a.g.scale;
    if (base) {
        float old[EL];
        base->get(old);
#pragma unroll
        for (int j = 0; j < EL; ++j) r[j] = old[j] + r[j];
    }
    store_unit<OF32, false>(a.g.dtable, v * a.g.H + col, r);
}

// Windows: workgroup (window, chunk).  16-byte stores: units of 4 elements where the
// table is f32 (161 us at 65536 tokens of 4096 bf16, 178 with units of 8), else of 8
// (60 against 62 us at 32768 tokens into bf16).  Streamed row loads; through the caches
// 176 and 71 us.  ACC (accumulating): the table rows of the runs that end in a batch are
// loaded with the batch, not one after the other: the call takes 62 us instead of 86 with
// 8192 tokens of 4096 into 131072 f32 rows (252 instead of 242 with 65536 tokens).
constexpr int window_unit(bool dout_f32, bool table_f32) { return dout_f32 || table_f32 ? 4 : 8; }
constexpr int kBatch = 8;   // rows in flight
template <bool DF32, bool OF32, bool ACC>
__global__ __launch_bounds__(kEmbThreads) void windows_kernel(SumArgs a) {
    constexpr int EL = window_unit(DF32, OF32);
    const int lane = threadIdx.x % kWave;
    const int units = (int)(a.g.H / EL);
    const int64_t m = *a.total;
    for (int64_t b = blockIdx.x; b < a.windows * a.nch; b += gridDim.x) {
        int64_t w;
        int c;
        xcd_item(b, a.windows, a.nch, w, c);
        const int64_t lo = w * a.window;
        if (lo >= m) continue;
        const int cnt = m - lo < a.window ? (int)(m - lo) : a.window;
        const int u = c * (int)blockDim.x + (int)threadIdx.x;
        const bool live = u < units;
        const int64_t col = (int64_t)(live ? u : units - 1) * EL;
        // lane i: position lo + i; bit i of ends: a run ends there
        const int64_t at = lo + (lane < cnt ? lane : cnt - 1);
        const int32_t id = a.id[at];
        const int32_t next = at + 1 < m ? a.id[at + 1] : -1;
        const int32_t pos = a.pos[at];
        const int32_t before = lo > 0 ? a.id[lo - 1] : -1;
        const uint64_t ends = ballot64(lane < cnt && id != next);
        bool entered = before == readlane(id, 0);   // the current run began in an earlier window
        float acc[EL];
#pragma unroll
        for (int j = 0; j < EL; ++j) acc[j] = 0.0f;
        for (int i = 0; i < cnt; i += kBatch) {
            FloatUnit<DF32, EL> x[kBatch];
            FloatUnit<OF32, EL> base[ACC ? kBatch : 1];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (i + q >= cnt) continue;
                x[q].load(a.g.dout, (int64_t)readlane(pos, i + q) * a.g.H + col);
                if constexpr (ACC)
                    if ((ends >> (i + q)) & 1)
                        base[q].load(a.g.dtable, (int64_t)readlane(id, i + q) * a.g.H + col);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (i + q >= cnt) continue;
                float v[EL];
                x[q].get(v);
#pragma unroll
                for (int j = 0; j < EL; ++j) acc[j] += v[j];
                if (!((ends >> (i + q)) & 1)) continue;
                if (live) {
                    if (entered) store_unit<true, false>(a.partial, 2 * w * a.g.H + col, acc);
                    else
                        put_row<OF32, EL>(a, readlane(id, i + q), col, acc,
                                          ACC ? &base[ACC ? q : 0] : nullptr);
                }
                entered = false;
#pragma unroll
                for (int j = 0; j < EL; ++j) acc[j] = 0.0f;
            }
        }
        if (live && !((ends >> (cnt - 1)) & 1))
            store_unit<true, false>(a.partial, (2 * w + (entered ? 0 : 1)) * a.g.H + col, acc);
    }
}

// Runs that cross windows: workgroup (window in which the run begins, chunk) adds the
// parts in order.  Where a row leaves threads over, they share the parts: `share`
// stretches of consecutive ones, whose sums are added in order (10136 tokens of 80:
// 34.9 us for the whole gradient with one stretch, 26.6 with 12; 131072 of 256 65.6 and
// 56.5 with 4).  For wide rows the same
// through several units per thread was slower, its registers and LDS cost the short
// runs more: 65536 tokens of 4096 496 -> 525 us, 8192 tokens over 200 rows 37 -> 42.
template <bool OF32>
__global__ __launch_bounds__(kEmbThreads) void join_kernel(SumArgs a, int nch, int share) {
    constexpr int EL = 4;
    __shared__ float stretch[kEmbThreads][EL];
    const int lane = threadIdx.x % kWave;
    const int units = (int)(a.g.H / EL);
    const int64_t m = *a.total;
    for (int64_t b = blockIdx.x; b < a.windows * nch; b += gridDim.x) {
        const int64_t w = b / nch;
        const int64_t lo = w * a.window, hi = lo + a.window;
        if (hi >= m) continue;
        const int32_t v = a.id[hi - 1];
        if (a.id[hi] != v) continue;                                     // no run leaves
        if (a.id[lo] == v && lo > 0 && a.id[lo - 1] == v) continue;      // it began earlier
        // windows after this one whose first position the run holds
        int64_t more = 0;
        for (;;) {
            const int64_t first = (w + 1 + more + lane) * a.window;
            const uint64_t no = ballot64(!(first < m && a.id[first < m ? first : 0] == v));
            if (no == 0) {
                more += kWave;
                continue;
            }
            more += __builtin_ctzll(no);
            break;
        }
        const int s = share > 1 ? (int)threadIdx.x / units : 0;   // this thread's stretch
        const int u = share > 1 ? (int)threadIdx.x - s * units
                                : (int)(b - w * nch) * (int)blockDim.x + (int)threadIdx.x;
        const bool mine = u < units && s < share;
        const int64_t col = (int64_t)u * EL;
        const int64_t per = (more + share - 1) / share;
        const int64_t from = s * per, to = from + per < more ? from + per : more;
        float acc[EL];
#pragma unroll
        for (int j = 0; j < EL; ++j) acc[j] = 0.0f;
        FloatUnit<OF32, EL> base;
        if (mine && s == 0) {
            FloatUnit<true, EL> x0;
            x0.load(a.partial, (2 * w + 1) * a.g.H + col);
            if (a.g.accumulate) base.load(a.g.dtable, (int64_t)v * a.g.H + col);
            x0.get(acc);
        }
        for (int64_t i = from; mine && i < to; i += kBatch) {
            FloatUnit<true, EL> x[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                if (i + q < to) x[q].load(a.partial, 2 * (w + 1 + i + q) * a.g.H + col);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (i + q >= to) continue;
                float p[EL];
                x[q].get(p);
#pragma unroll
                for (int j = 0; j < EL; ++j) acc[j] += p[j];
            }
        }
        if (share > 1) {
            __syncthreads();   // the previous run's stretches are read
#pragma unroll
            for (int j = 0; j < EL; ++j) stretch[threadIdx.x][j] = acc[j];
            __syncthreads();
            if (mine && s == 0)
                for (int i = 1; i < share; ++i)
#pragma unroll
                    for (int j = 0; j < EL; ++j) acc[j] += stretch[i * units + u][j];
        }
        if (mine && s == 0)
            put_row<OF32, EL>(a, v, col, acc, a.g.accumulate ? &base : nullptr);
    }
}

// Positions per window: 64 (one wave's lanes), fewer while there would be less than so
// many waves of 512 elements: shorter windows make more workgroups and longer joins,
// and narrow rows share those.  Measured with 512 / 1024 / 2048 / 4096, us: 65536 tokens
// of 64 - / 44.4 / 39.5 / 39.0, of 264 - / 75.0 / 72.8 / 77.3; 8192 tokens of 1024 over
// 100 rows 24.0 / 26.2 / 33.8 / -, of 4096 over 200 rows 32.6 / 32.5 / 30.3 / -; 4096
// of 1024 over 100 rows 23.0 / 27.0 / 26.9 / -.
constexpr int kShortestWindow = 8;
inline int64_t enough_windows(int64_t H) {
    const int64_t waves = H <= 512 ? 2048 : 512, per_row = (H + 511) / 512;
    return (waves + per_row - 1) / per_row;
}
inline int window_of(int64_t N, int64_t H) {
    int w = kWave;
    while (w > kShortestWindow && (N + w - 1) / w < enough_windows(H)) w /= 2;
    return w;
}

// Windows that the workspace holds: enough for every sort of at most N positions, since
// fewer positions take shorter windows.  A window that was halved leaves less than twice
// enough_windows, because the longer one left less than enough.
inline int64_t window_room(int64_t N, int64_t H) {
    const int64_t full = (N + kWave - 1) / kWave;
    const int64_t shortest = (N + kShortestWindow - 1) / kShortestWindow;
    const int64_t halved = 2 * (enough_windows(H) - 1);
    const int64_t most = shortest < halved ? shortest : halved;
    return most > full ? most : full;
}

struct GradWs {
    size_t ticket, local_rank, tile_cnt, tile_flags, off0, off, id[2], pos[2], present, partial,
        total;
    int64_t tiles, windows;
    int passes, bits;   // digits, and bits of each; no pass: the small sort
    int window;
    bool zero_early;
};

// Up to this many bytes of rows of tokens that occur (at most min(N,V) rows, as f32),
// the whole table is zeroed beside the first move and those rows are written twice;
// past it, the rows of absent tokens get a launch of their own that writes nothing
// twice.  10136 tokens of 80 into 8762 bf16 rows: 39.2 us beside the move, 41.6 apart;
// 65536 of 64 into 131072 f32 rows 64.0, 67.6; 8192 of 4096 into 50000 rows 164, 159.
constexpr int64_t kZeroTwice = (int64_t)64 << 20;

// Every piece is sized so that it does not shrink when N or V grows: a workspace for the
// most positions and the largest vocabulary serves every call of the same H below them.
GradWs grad_ws(int64_t N, int64_t V, int64_t H) {
    GradWs w{};
    int id_bits = 1;
    w.tiles = (N + kTile - 1) / kTile;
    w.window = window_of(N, H);
    w.windows = (N + w.window - 1) / w.window;
    if (N > kSmallSort) {
        while (((int64_t)1 << id_bits) < V) ++id_bits;
        const int most = digit_bits(w.tiles);
        w.passes = (id_bits + most - 1) / most;
        w.bits = (id_bits + w.passes - 1) / w.passes;
        w.zero_early = (N < V ? N : V) * H * 4 <= kZeroTwice;
    }
    size_t total = 0;
    auto take = [&total](size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t n = (size_t)N, offsets = 4 * (((size_t)1 << kDigitMost) + 1);
    // the routing's arrival ticket first: calls of any size that share a workspace
    // find it where the last one left it
    w.ticket = take(sizeof(uint64_t));
    w.off0 = take(offsets);   // behind the last offset: how many ids are valid
    w.id[0] = take(4 * n);
    w.pos[0] = take(4 * n);
    w.partial = take(4 * 2 * (size_t)window_room(N, H) * (size_t)H);
    if (w.passes > 0) {
        w.local_rank = take(4 * n);
        w.tile_cnt = take(4 * (size_t)count_room(w.tiles, id_bits));
        w.tile_flags = take(8 * (size_t)w.tiles);
    }
    if (w.passes > 1) {
        w.off = take(offsets);
        w.id[1] = take(4 * n);
        w.pos[1] = take(4 * n);
        w.present = take((size_t)V);
    }
    w.total = total;
    return w;
}

template <class P>
P* at(void* ws, size_t off) {
    return (P*)((char*)ws + off);
}

inline int chunks(int64_t units, int threads) { return (int)((units + threads - 1) / threads); }

template <bool OF32>
hipError_t small_sort(const EmbeddingGradArgs& g, const SumArgs& a, hipStream_t s) {
    SmallSortArgs m{};
    m.ids = g.ids;
    m.id_bytes = g.id_bytes;
    m.N = g.N;
    m.V = g.V;
    m.H = g.H;
    m.id = const_cast<int32_t*>(a.id);
    m.pos = const_cast<int32_t*>(a.pos);
    m.total = const_cast<int32_t*>(a.total);
    m.dtable = g.dtable;
    m.sort_blocks = (int)((g.N + kSortPositions - 1) / kSortPositions);
    m.zero = zero_layout(g.V, g.H, OF32);
    if (g.accumulate) m.zero.blocks = 0;
    small_sort_kernel<OF32>
        <<<capped_grid(m.sort_blocks + m.zero.blocks), dim3(kEmbThreads), 0, s>>>(m);
    return hipGetLastError();
}

// Ranks of one digit by the one-launch routing, scanned by its last workgroup.
hipError_t route_digit(const MoveArgs& m, uint64_t* ticket, hipStream_t s) {
    RouteFusedArgs fa{};
    fa.kind = KeyKind::Digits;
    fa.digits = m.d;
    fa.N = m.N;
    fa.nbits = m.nbits;
    fa.local_rank = m.local_rank;
    fa.ticket = ticket;
    fa.scan.tile_cnt = m.tile_cnt;
    fa.scan.tile_flags = m.tile_flags;
    fa.scan.tiles = m.tiles;
    fa.scan.NK = m.NK;
    fa.scan.rows_limit = INT64_MAX;
    fa.scan.off_ws = m.off;
    fa.scan.mode = StatsMode::Plain;
    return launch_route_fused(fa, s);
}

// Sorts by one digit after the other; cur: which of the two buffers holds the result.
hipError_t radix_sort(const EmbeddingGradArgs& g, const GradWs& w, int& cur, hipStream_t s) {
    void* ws = g.ws;
    const bool own_scan = w.tiles <= kOwnScanTiles;
    MoveArgs m{};
    m.N = g.N;
    m.V = g.V;
    m.H = g.H;
    m.local_rank = at<int32_t>(ws, w.local_rank);
    m.tile_cnt = at<int32_t>(ws, w.tile_cnt);
    m.tile_flags = at<int32_t>(ws, w.tile_flags);
    m.tiles = (int)w.tiles;
    m.NK = 1 << w.bits;
    m.nbits = w.bits;
    m.d.mask = m.NK - 1;
    cur = 0;
    for (int p = 0; p < w.passes; ++p) {
        const bool first = p == 0, last = p == w.passes - 1;
        m.d.shift = p * w.bits;
        m.d.ids = first ? g.ids : at<int32_t>(ws, w.id[cur]);
        m.d.id_bytes = first ? g.id_bytes : 4;
        m.d.V = g.V;
        m.d.total = first ? nullptr : at<int32_t>(ws, w.off0) + m.NK;
        m.off = at<int32_t>(ws, first ? w.off0 : w.off);
        if (own_scan) {
            digit_rank_kernel<<<dim3((unsigned)w.tiles), dim3(kSortThreads),
                                sizeof(int32_t) * kSortWaves * m.NK, s>>>(m);
        } else {
            const hipError_t e = route_digit(m, at<uint64_t>(ws, w.ticket), s);
            if (e != hipSuccess) return e;
        }
        const int next = first ? 0 : 1 - cur;
        m.in_pos = first ? nullptr : at<int32_t>(ws, w.pos[cur]);
        m.out_id = at<int32_t>(ws, w.id[next]);
        m.out_pos = at<int32_t>(ws, w.pos[next]);
        const bool flags = w.passes > 1 && !w.zero_early && !g.accumulate;
        m.clear = flags && first ? at<uint8_t>(ws, w.present) : nullptr;
        m.present = flags && last ? at<uint8_t>(ws, w.present) : nullptr;
        m.move_blocks = w.tiles < kMaxSortGrid ? w.tiles : kMaxSortGrid;
        int64_t zero_blocks = 0;
        if (first && w.zero_early && !g.accumulate) {
            m.dtable = g.dtable;
            m.dtable_f32 = g.dtable_f32;
            m.zero = zero_layout(g.V, g.H, g.dtable_f32);
            constexpr int kParts = kSortThreads / kEmbThreads;
            zero_blocks = (m.zero.blocks + kParts - 1) / kParts;
            if (zero_blocks > kMaxSortGrid) zero_blocks = kMaxSortGrid;
        }
        const dim3 grid((unsigned)(m.move_blocks + zero_blocks));
        if (own_scan) scan_move_kernel<<<grid, dim3(kSortThreads), 0, s>>>(m);
        else move_kernel<<<grid, dim3(kSortThreads), 0, s>>>(m);
        cur = next;
    }
    return hipGetLastError();
}

template <bool DF32, bool OF32>
hipError_t grad_go(const EmbeddingGradArgs& g, hipStream_t s) {
    const GradWs w = grad_ws(g.N, g.V, g.H);
    SumArgs a{};
    a.g = g;
    a.total = at<int32_t>(g.ws, w.off0) + (1 << w.bits);
    a.partial = at<float>(g.ws, w.partial);
    a.window = w.window;
    a.windows = w.windows;
    int cur = 0;
    if (w.passes > 0) {
        const hipError_t e = radix_sort(g, w, cur, s);
        if (e != hipSuccess) return e;
    }
    a.id = at<int32_t>(g.ws, w.id[cur]);
    a.pos = at<int32_t>(g.ws, w.pos[cur]);
    if (w.passes == 0) {
        const hipError_t e = small_sort<OF32>(g, a, s);
        if (e != hipSuccess || g.N == 0) return e;
    }
    const int64_t units = g.H / window_unit(DF32, OF32);
    const int threads = row_threads(units, kEmbThreads);
    a.nch = chunks(units, threads);
    if (w.passes > 0 && !w.zero_early && !g.accumulate) {
        const ZeroRows z = zero_layout(g.V, g.H, OF32);
        zero_rows_kernel<OF32><<<capped_grid(z.blocks), dim3(kEmbThreads), 0, s>>>(
            g.dtable, g.V, g.H, w.passes > 1 ? at<uint8_t>(g.ws, w.present) : nullptr,
            at<int32_t>(g.ws, w.off0), z);
    }
    const dim3 grid = capped_grid(a.windows * a.nch);
    if (g.accumulate) windows_kernel<DF32, OF32, true><<<grid, dim3(threads), 0, s>>>(a);
    else windows_kernel<DF32, OF32, false><<<grid, dim3(threads), 0, s>>>(a);
    if (a.windows > 1) {
        const int64_t ju = g.H / 4;
        const int share = ju < kEmbThreads ? (int)(kEmbThreads / ju) : 1;
        const int jt = share > 1 ? kEmbThreads : row_threads(ju, kEmbThreads);
        const int jch = chunks(ju, jt);
        join_kernel<OF32><<<capped_grid(a.windows * jch), dim3(jt), 0, s>>>(a, jch, share);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding(const EmbeddingArgs& a, hipStream_t s) {
    if (a.N == 0 && !a.stats) return hipSuccess;
    if (a.table_f32) {
        if (a.out_f32) embedding_go<true, true>(a, s);
        else embedding_go<true, false>(a, s);
    } else {
        if (a.out_f32) embedding_go<false, true>(a, s);
        else embedding_go<false, false>(a, s);
    }
    return hipGetLastError();
}

size_t embedding_grad_ws(int64_t N, int64_t V, int64_t H) { return grad_ws(N, V, H).total; }

hipError_t launch_embedding_grad(const EmbeddingGradArgs& g, hipStream_t s) {
    if (g.N == 0 && g.accumulate) return hipSuccess;
    if (g.dout_f32) return g.dtable_f32 ? grad_go<true, true>(g, s) : grad_go<true, false>(g, s);
    return g.dtable_f32 ? grad_go<false, true>(g, s) : grad_go<false, false>(g, s);
}

}  // namespace moe
