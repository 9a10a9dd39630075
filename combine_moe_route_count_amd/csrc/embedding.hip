// embedding.hip - embedding lookup with scaling, and its gradient by sorted
// tokens.
//
// Lookup: out[n] = scale * table[ids[n]], a row gather.
//
// Gradient: dtable[v] = scale * sum of dout[n] over the n with ids[n] = v.  The
// positions are sorted by token id, stably, so that each table row owns one run
// of positions in ascending order and sums it alone: no atomics, one fixed order.
// The sort is a radix sort of the ids whose digits (at most 9 bits) are the keys
// of the one-launch routing (route_fused.hip): a 131072-row table takes two
// passes.  Launches: per pass the routing and the move of (id, position), then
// the run bounds, the pieces of long runs, and the table rows.
//
// A run longer than kRun positions (frequent tokens) is cut into pieces of kRun
// from its start.  Each piece is summed on its own into an f32 row of the
// workspace, and the table row adds the pieces in order, so one token's
// occurrences do not serialise behind each other.
#include "train_device.hpp"
#include "internal.hpp"

namespace moe {

namespace {

constexpr int kEmbThreads = 256;
constexpr int kRun = 256;
constexpr int kDigitBits = 9;   // 512 keys: the most that the one-launch routing takes

inline int chunks_of(int64_t H) { return (int)((H / 8 + kEmbThreads - 1) / kEmbThreads); }

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
    // the last item counts the ids outside [0,V)
    for (int64_t wi = blockIdx.x; wi < items + (a.stats ? 1 : 0); wi += gridDim.x) {
        if (wi == items) {
            __shared__ int32_t bad;
            if (threadIdx.x == 0) bad = 0;
            __syncthreads();
            int32_t mine = 0;
            for (int64_t n = threadIdx.x; n < a.N; n += blockDim.x) {
                const int64_t id = token_id(a.ids, a.id_bytes, n);
                mine += id < -1 || id >= a.V;
            }
            if (mine) atomicAdd(&bad, mine);
            __syncthreads();
            if (threadIdx.x == 0) a.stats[0] = bad;
            continue;
        }
        const int64_t n = wi / nch;
        const int c = (int)(wi - n * nch);
        const int64_t id = token_id(a.ids, a.id_bytes, n);
        const bool some = id >= 0 && id < a.V;
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

template <bool TF32, bool OF32>
void embedding_go(const EmbeddingArgs& a, hipStream_t s) {
    const int64_t units = a.H / (OF32 ? 4 : 8);
    const int threads = row_threads((units + kLookupUnits - 1) / kLookupUnits, lookup_threads(OF32));
    const int nch = (int)((units + threads * kLookupUnits - 1) / (threads * kLookupUnits));
    embedding_kernel<TF32, OF32>
        <<<capped_grid(a.N * nch + (a.stats ? 1 : 0)), dim3(threads), 0, s>>>(a, nch);
}

// ---------------------------------------------------------------------------
// gradient: the sort
// ---------------------------------------------------------------------------
struct Run {   // positions [start, end) of the sorted order
    int32_t start, end;
};

struct MoveArgs {              // one radix pass's move
    DigitSource d;
    int64_t N;
    const int32_t* local_rank;
    const int32_t* tile_base;  // [tiles][NK]
    const int32_t* off;        // [NK+1]
    int NK;
    const int32_t* in_pos;     // null: the position is the entry's own number
    int32_t* out_id;
    int32_t* out_pos;
    Run* runs;                 // [V] to clear, or null
    int64_t V;
};

__global__ __launch_bounds__(kEmbThreads) void move_kernel(MoveArgs a) {
    const int64_t step = (int64_t)gridDim.x * kEmbThreads;
    const int64_t first = (int64_t)blockIdx.x * kEmbThreads + threadIdx.x;
    if (a.runs)
        for (int64_t v = first; v < a.V; v += step) a.runs[v] = Run{0, 0};
    for (int64_t f = first; f < a.N; f += step) {
        const int32_t lr = a.local_rank[f];
        if (lr < 0) continue;
        const int32_t id = a.d.total ? ((const int32_t*)a.d.ids)[f]
                                     : (int32_t)token_id(a.d.ids, a.d.id_bytes, f);
        const int key = (id >> a.d.shift) & a.d.mask;
        const int64_t to = (int64_t)a.off[key] + a.tile_base[(f / kTile) * a.NK + key] + lr;
        a.out_id[to] = id;
        a.out_pos[to] = a.in_pos ? a.in_pos[f] : (int32_t)f;
    }
}

// The run of each token that occurs: its first and last position say so.
__global__ __launch_bounds__(kEmbThreads) void runs_kernel(const int32_t* id, const int32_t* total,
                                                           Run* runs) {
    const int64_t m = *total;
    const int64_t step = (int64_t)gridDim.x * kEmbThreads;
    for (int64_t i = (int64_t)blockIdx.x * kEmbThreads + threadIdx.x; i < m; i += step) {
        const int32_t v = id[i];
        if (i == 0 || id[i - 1] != v) runs[v].start = (int32_t)i;
        if (i == m - 1 || id[i + 1] != v) runs[v].end = (int32_t)i + 1;
    }
}

// ---------------------------------------------------------------------------
// gradient: the sums
// ---------------------------------------------------------------------------
struct SumArgs {
    EmbeddingGradArgs g;
    const int32_t* id;      // sorted token ids
    const int32_t* pos;     // their positions
    const int32_t* total;   // how many
    const Run* runs;
    float* partial;         // [2 * ceil(N/kRun)][H]
    int nch;
};

// Workspace row of the piece that starts at position p of the sorted order; first
// says whether it is its run's first piece.  Long runs are longer than kRun, so
// no two of them start in the same kRun positions, nor do two later pieces.
__device__ __forceinline__ int64_t piece_slot(int64_t p, bool first) {
    return 2 * (p / kRun) + (first ? 0 : 1);
}

// acc += dout[pos[i]] for i in [lo, hi) ascending, unit u of the rows.  Every lane
// of the wave takes part (u clamped to the row).
template <bool DF32>
__device__ __forceinline__ void sum_rows(const SumArgs& a, int lo, int hi, int u, float (&acc)[8]) {
    const int lane = threadIdx.x % kWave;
    for (int64_t base = lo; base < hi; base += kWave) {
        const int mine = base + lane < hi ? a.pos[base + lane] : 0;
        const int cnt = hi - base < kWave ? (int)(hi - base) : kWave;
        for (int i = 0; i < cnt; ++i) {
            const int64_t n = readlane(mine, i);
            FloatUnit<DF32, 8> x;
            x.load(a.g.dout, n * a.g.H + (int64_t)u * 8);
            float v[8];
            x.get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += v[j];
        }
    }
}

// One piece of a long run: workgroup (block of kRun positions, first / later, chunk).
template <bool DF32>
__global__ __launch_bounds__(kEmbThreads) void pieces_kernel(SumArgs a, int64_t blocks) {
    const int64_t m = *a.total;
    const int units = (int)(a.g.H / 8);
    for (int64_t wi = blockIdx.x; wi < blocks * 2 * a.nch; wi += gridDim.x) {
        const int64_t slot = wi / a.nch;
        const int64_t b0 = (slot / 2) * kRun;
        const bool first = (slot & 1) == 0;
        // a first piece's run also holds the next block's first position, a later
        // piece's run holds this block's
        const int64_t probe = first ? b0 + kRun : b0;
        if (probe >= m) continue;
        const Run run = a.runs[a.id[probe]];
        if (run.end - run.start <= kRun) continue;
        int64_t lo;
        if (first) {
            lo = run.start;
            if (lo < b0) continue;
        } else {
            if (run.start >= b0) continue;
            lo = run.start + (b0 - run.start + kRun - 1) / kRun * kRun;
            if (lo >= run.end) continue;
        }
        const int64_t hi = lo + kRun < run.end ? lo + kRun : run.end;
        const int u = (int)(wi % a.nch) * kEmbThreads + threadIdx.x;
        const int uc = u < units ? u : units - 1;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        sum_rows<DF32>(a, (int)lo, (int)hi, uc, acc);
        if (u < units) store_unit<true, false>(a.partial, slot * a.g.H + (int64_t)u * 8, acc);
    }
}

// Table rows: workgroup (row, chunk).
template <bool DF32, bool OF32>
__global__ __launch_bounds__(kEmbThreads) void table_grad_kernel(SumArgs a) {
    const int units = (int)(a.g.H / 8);
    for (int64_t wi = blockIdx.x; wi < a.g.V * a.nch; wi += gridDim.x) {
        const int64_t v = wi / a.nch;
        const Run run = a.runs[v];
        const int len = run.end - run.start;
        if (len == 0 && a.g.accumulate) continue;
        const int u = (int)(wi % a.nch) * kEmbThreads + threadIdx.x;
        const int uc = u < units ? u : units - 1;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (len > kRun) {
            for (int64_t p = run.start; p < run.end; p += kRun) {
                FloatUnit<true, 8> x;
                x.load(a.partial, piece_slot(p, p == run.start) * a.g.H + (int64_t)uc * 8);
                float pv[8];
                x.get(pv);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += pv[j];
            }
        } else {
            sum_rows<DF32>(a, run.start, run.end, uc, acc);
        }
        if (u >= units) continue;
        const int64_t at = v * a.g.H + (int64_t)u * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = acc[j] * a.g.scale;
        if (a.g.accumulate) {
            FloatUnit<OF32, 8> x;
            x.load(a.g.dtable, at);
            float base[8];
            x.get(base);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = base[j] + acc[j];
        }
        store_unit<OF32, false>(a.g.dtable, at, acc);
    }
}

struct GradWs {
    size_t ticket, local_rank, tile_cnt, tile_flags, off0, off, id[2], pos[2], runs, partial, total;
    int64_t tiles, blocks;
    int passes, bits;   // digits, and bits of each
};

GradWs grad_ws(int64_t N, int64_t V, int64_t H) {
    GradWs w{};
    int bits = 1;
    while (((int64_t)1 << bits) < V) ++bits;
    w.passes = (bits + kDigitBits - 1) / kDigitBits;
    w.bits = (bits + w.passes - 1) / w.passes;
    w.tiles = (N + kTile - 1) / kTile;
    w.blocks = (N + kRun - 1) / kRun;
    size_t total = 0;
    auto take = [&total](size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t n = (size_t)N, nk = (size_t)1 << w.bits;
    w.ticket = take(sizeof(uint64_t));
    w.local_rank = take(4 * n);
    w.tile_cnt = take(4 * (size_t)w.tiles * nk);
    w.tile_flags = take(8 * (size_t)w.tiles);
    w.off0 = take(4 * (nk + 1));
    w.off = take(4 * (nk + 1));
    for (int i = 0; i < 2; ++i) {
        w.id[i] = take(4 * n);
        w.pos[i] = take(4 * n);
    }
    w.runs = take(sizeof(Run) * (size_t)V);
    w.partial = take(4 * 2 * (size_t)w.blocks * (size_t)H);
    w.total = total;
    return w;
}

template <class P>
P* at(void* ws, size_t off) {
    return (P*)((char*)ws + off);
}

inline dim3 flat_grid(int64_t n) { return capped_grid((n + kEmbThreads - 1) / kEmbThreads); }

template <bool DF32>
void sums_go(const SumArgs& a, int64_t blocks, hipStream_t s) {
    if (a.g.N > kRun)
        pieces_kernel<DF32><<<capped_grid(blocks * 2 * a.nch), dim3(kEmbThreads), 0, s>>>(a, blocks);
    const dim3 grid = capped_grid(a.g.V * a.nch);
    if (a.g.dtable_f32) table_grad_kernel<DF32, true><<<grid, dim3(kEmbThreads), 0, s>>>(a);
    else table_grad_kernel<DF32, false><<<grid, dim3(kEmbThreads), 0, s>>>(a);
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
    const GradWs w = grad_ws(g.N, g.V, g.H);
    void* ws = g.ws;
    Run* runs = at<Run>(ws, w.runs);
    int cur = 0;
    for (int p = 0; p < w.passes; ++p) {
        const int NK = 1 << w.bits;
        DigitSource d{};
        d.shift = p * w.bits;
        d.mask = NK - 1;
        if (p == 0) {
            d.ids = g.ids;
            d.id_bytes = g.id_bytes;
            d.V = g.V;
        } else {
            d.ids = at<int32_t>(ws, w.id[cur]);
            d.total = at<int32_t>(ws, w.off0) + NK;
        }
        int32_t* off = at<int32_t>(ws, p == 0 ? w.off0 : w.off);
        if (g.N > 0) {
            RouteFusedArgs fa{};
            fa.kind = KeyKind::Digits;
            fa.digits = d;
            fa.N = g.N;
            fa.nbits = w.bits;
            fa.local_rank = at<int32_t>(ws, w.local_rank);
            fa.ticket = at<uint64_t>(ws, w.ticket);
            fa.scan.tile_cnt = at<int32_t>(ws, w.tile_cnt);
            fa.scan.tile_flags = at<int32_t>(ws, w.tile_flags);
            fa.scan.tiles = (int)w.tiles;
            fa.scan.NK = NK;
            fa.scan.rows_limit = INT64_MAX;
            fa.scan.off_ws = off;
            fa.scan.mode = StatsMode::Plain;
            const hipError_t e = launch_route_fused(fa, s);
            if (e != hipSuccess) return e;
        }
        MoveArgs m{};
        m.d = d;
        m.N = g.N;
        m.local_rank = at<int32_t>(ws, w.local_rank);
        m.tile_base = at<int32_t>(ws, w.tile_cnt);
        m.off = off;
        m.NK = NK;
        const int next = p == 0 ? 0 : 1 - cur;
        m.in_pos = p == 0 ? nullptr : at<int32_t>(ws, w.pos[cur]);
        m.out_id = at<int32_t>(ws, w.id[next]);
        m.out_pos = at<int32_t>(ws, w.pos[next]);
        m.runs = p == 0 ? runs : nullptr;
        m.V = g.V;
        move_kernel<<<flat_grid(p == 0 && g.V > g.N ? g.V : g.N), dim3(kEmbThreads), 0, s>>>(m);
        cur = next;
        if (g.N == 0) break;
    }
    SumArgs a{};
    a.g = g;
    a.id = at<int32_t>(ws, w.id[cur]);
    a.pos = at<int32_t>(ws, w.pos[cur]);
    a.total = at<int32_t>(ws, w.off0) + (1 << w.bits);
    a.runs = runs;
    a.partial = at<float>(ws, w.partial);
    a.nch = chunks_of(g.H);
    if (g.N > 0) runs_kernel<<<flat_grid(g.N), dim3(kEmbThreads), 0, s>>>(a.id, a.total, runs);
    if (g.dout_f32) sums_go<true>(a, w.blocks, s);
    else sums_go<false>(a, w.blocks, s);
    return hipGetLastError();
}

}  // namespace moe
