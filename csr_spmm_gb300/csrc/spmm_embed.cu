// Embedding lookup out[t, :] = scale * table[ids[t], :] and its gradient
// dtable[v, :] = beta * dtable[v, :] + scale * sum_{t: ids[t] = v} dout[t, :].
//
// The gradient is the product of the transposed one-entry-per-row matrix with
// dout.  Its row structure is made on the device by sorting the tokens by id:
// keys (id << 32 | position) are unique, so any correct sort of them is the
// stable order, and the sums below have a fixed order.
#include <algorithm>

#include "spmm_internal.h"
#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

// ---- lookup -----------------------------------------------------------------

constexpr int EMBED_THREADS = 256;
constexpr int EMBED_BATCH = 4;       // accesses in flight per thread

// A block takes `block_rows` rows; its threads walk the rows' accesses in
// order (nv accesses of W elements per row, then the next row), so narrow
// rows share a warp and the stores of neighbouring threads are contiguous.
// The bound is HBM: one table row read and one written per token.
template <typename T, int W>
__global__ __launch_bounds__(EMBED_THREADS) void embed_rows(EmbedParams p, int nv,
                                                            int block_rows) {
    const T* table = static_cast<const T*>(p.table);
    T* out = static_cast<T*>(p.out);
    const int64_t row0 = (int64_t)blockIdx.x * block_rows;
    const int rows = (int)min((int64_t)block_rows, p.tokens - row0);
    const int step_r = EMBED_THREADS / nv, step_c = EMBED_THREADS % nv;
    int r = threadIdx.x / nv, c = threadIdx.x % nv;
    while (r < rows) {
        Vec<T, W> v[EMBED_BATCH];
        int64_t to[EMBED_BATCH];
        bool valid[EMBED_BATCH];
#pragma unroll
        for (int u = 0; u < EMBED_BATCH; ++u) {
            to[u] = -1;
            if (r < rows) {
                const int64_t row = row0 + r;
                const int id = p.ids[row];
                to[u] = row * p.ld_out + (int64_t)c * W;
                valid[u] = id >= 0 && id < p.vocab;
                if (valid[u])
                    v[u] = load_vec<Cache::KEEP, T, W>(table + id * p.ld_table + (int64_t)c * W);
            }
            r += step_r;
            c += step_c;
            if (c >= nv) {
                c -= nv;
                ++r;
            }
        }
#pragma unroll
        for (int u = 0; u < EMBED_BATCH; ++u) {
            if (to[u] < 0) continue;
            float f[W];
            unpack(v[u], f);
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = valid[u] ? p.scale * f[i] : 0.0f;
            store_vec<Cache::STREAM, T, W>(out + to[u], f);
        }
    }
}

template <typename T, int W>
cudaError_t launch_embed(const EmbedParams& p, int num_sms, cudaStream_t st) {
    const int nv = (int)(p.dim / W);
    // about 8 accesses per thread and block; fewer rows per block while that
    // would leave SMs without a block
    int64_t rows = std::max<int64_t>(1, EMBED_THREADS * 8 / nv);
    rows = std::max<int64_t>(1, std::min<int64_t>(rows, p.tokens / (4 * num_sms)));
    const int64_t blocks = (p.tokens + rows - 1) / rows;
    embed_rows<T, W><<<(unsigned)blocks, EMBED_THREADS, 0, st>>>(p, nv, (int)rows);
    return cudaGetLastError();
}

// ---- gradient: sort ------------------------------------------------------------

constexpr int SORT_TILE = 512;       // keys sorted by one block, one per thread
constexpr int MERGE_WAYS = 16;       // sorted runs merged per round
constexpr unsigned NO_ID = 0xffffffffu;

// Sorts each tile of SORT_TILE tokens with a bitonic network, one 64-bit key per
// thread: exchanges within a warp are shuffles (35 of the 45 steps), the others
// go through shared memory.  Small tiles, so that the SMs share the work: the
// whole of 65,536 tokens takes 128 blocks.  Ids outside [0, vocab) get the
// largest key and end up behind every row.  Also zeroes the sums' arrival counters.
__global__ __launch_bounds__(SORT_TILE) void sort_tiles(const int* ids, int tokens, int64_t vocab,
                                                        uint64_t* keys, int* arrived,
                                                        int64_t counters) {
    __shared__ uint64_t s[2][SORT_TILE];
    allow_successor();
    const int t = threadIdx.x;
    const int64_t at = (int64_t)blockIdx.x * SORT_TILE + t;
    uint64_t key = ~0ull;
    if (at < tokens) {
        const int id = ids[at];
        key = (uint64_t)(id >= 0 && id < vocab ? (unsigned)id : NO_ID) << 32 | (unsigned)at;
    }
    for (int64_t i = at; i < counters; i += (int64_t)gridDim.x * SORT_TILE) arrived[i] = 0;
    const int n = (int)min((int64_t)SORT_TILE, tokens - (int64_t)blockIdx.x * SORT_TILE);
    int turn = 0;
    // past the tile's keys there are only largest ones: a shorter network does
    for (int k = 2; k < 2 * n; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            uint64_t other;
            if (j >= 32) {
                // two buffers in turn: one barrier per exchange keeps them apart
                s[turn][t] = key;
                __syncthreads();
                other = s[turn][t ^ j];
                turn ^= 1;
            } else {
                other = __shfl_xor_sync(0xffffffffu, key, j);
            }
            const bool up = (t & k) == 0, low = (t & j) == 0;
            key = (up == low) == (key < other) ? key : other;
        }
    }
    if (at < tokens) keys[at] = key;
}

// Number of keys below `key` in a[0..n).
__device__ __forceinline__ int count_below(const uint64_t* a, int n, uint64_t key) {
    int lo = 0, len = n;
    while (len > 0) {
        const int half = len >> 1;
        if (a[lo + half] < key) {
            lo += half + 1;
            len -= half + 1;
        } else {
            len = half;
        }
    }
    return lo;
}

// Merges groups of MERGE_WAYS sorted runs of `run` keys (a power of two): keys
// are unique, so each key's place is the count of smaller keys over the group's
// runs.  The searches of all runs take their steps together, MERGE_WAYS loads
// at a time: a step costs one latency, not one for each run (65,536 keys:
// 35 us per round with one search after the other).
__global__ __launch_bounds__(256) void merge_runs(const uint64_t* in, uint64_t* out, int tokens,
                                                  int64_t run) {
    allow_successor();
    wait_for_predecessor();
    const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (g >= tokens) return;
    const uint64_t key = in[g];
    const int64_t first = g / (run * MERGE_WAYS) * (run * MERGE_WAYS);
    int64_t below[MERGE_WAYS];       // per run: start + keys known to be smaller
#pragma unroll
    for (int q = 0; q < MERGE_WAYS; ++q) below[q] = first + q * run;
    for (int64_t half = run >> 1; half > 0; half >>= 1) {
        uint64_t got[MERGE_WAYS];
#pragma unroll
        for (int q = 0; q < MERGE_WAYS; ++q) {
            const int64_t at = below[q] + half - 1;
            got[q] = at < tokens ? in[at] : ~0ull;
        }
#pragma unroll
        for (int q = 0; q < MERGE_WAYS; ++q)
            if (got[q] < key) below[q] += half;
    }
    // one candidate is left in each run
    int64_t place = first;
#pragma unroll
    for (int q = 0; q < MERGE_WAYS; ++q) {
        const int64_t at = below[q];
        place += at - (first + q * run) + (at < tokens && in[at] < key);
    }
    out[place] = key;
}

// ---- gradient: sums --------------------------------------------------------------

// The sorted tokens are cut into pieces of equal length; a warp sums one piece
// over one panel of columns, reading each token's row segment once.  A run of
// one id that lies within the piece is complete and goes to its table row; a
// run that crosses the piece's bounds leaves a partial sum, and the last of the
// run's pieces to arrive adds the run's partials in piece order.
constexpr int PANEL = 256;           // columns per warp: 512 bytes of a 16-bit row
constexpr int PIECE_MAX = 256;
constexpr int64_t SUM_WARPS = 16384;

// Tokens per piece: as many as leave about SUM_WARPS warps of work (three to four
// times what the SMs hold at once), so that few runs are cut; one where there is
// less, because a warp's tokens wait for one another.  It depends on the call's
// sizes only, so the order of every sum does too.
inline int64_t panels_of(int64_t dim) { return (dim + PANEL - 1) / PANEL; }
inline int piece_of(int64_t tokens, int64_t dim) {
    int piece = 1;
    while (piece < PIECE_MAX && tokens * panels_of(dim) / piece > SUM_WARPS) piece *= 2;
    return piece;
}
inline int64_t padded(int64_t dim) { return (dim + 7) / 8 * 8; }   // partial rows: 32 bytes

struct GradWork {
    const uint64_t* keys;            // sorted
    float* partials;                 // [pieces][2][padded dim]: run from before, run to the next
    int* arrived;                    // [pieces][panels], zeroed by sort_tiles
    int64_t dim_padded;
    int piece;
    int panels;
    int64_t sum_items;               // pieces * panels warps sum; the rest fill
    int fill_rows;                   // table rows per filling warp
};

// Number of keys below `key`, by the whole warp: 32 probes per step.
__device__ __forceinline__ int warp_count_below(const uint64_t* a, int n, uint64_t key, int lane) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo) / 32 + 1;
        const int64_t at = lo + (int64_t)lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && a[at] < key);
        const int k = __popc(below);
        if (k == 0) return lo;
        hi = (int)min((int64_t)hi, lo + (int64_t)k * step);
        lo += (k - 1) * step + 1;
    }
    return lo;
}

// W elements per access, V accesses per lane and row segment: W * V * 32 == PANEL.
template <typename T, typename G, int W, int V, int BATCH>
struct GradSum {
    static_assert(W * V * 32 == PANEL);
    const EmbedGradParams& p;
    const GradWork& k;
    int lane;
    int64_t col;                     // the panel's first column
    float acc[V][W];

    __device__ bool inside(int v) const { return col + (v * 32 + lane) * W < p.dim; }
    __device__ void clear() {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < W; ++i) acc[v][i] = 0.0f;
    }
    // dtable[row] = beta * dtable[row] + scale * acc
    __device__ void finish(unsigned row) {
        G* to = static_cast<G*>(p.dtable) + (int64_t)row * p.ld_dtable + col + lane * W;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!inside(v)) continue;
            float f[W];
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = p.scale * acc[v][i];
            if (p.beta != 0.0f) {
                float old[W];
                unpack(load_vec<Cache::STREAM, G, W>(to + v * 32 * W), old);
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] += p.beta * old[i];
            }
            store_vec<Cache::STREAM, G, W>(to + v * 32 * W, f);
        }
    }
    __device__ float* partial(int64_t slot) const {
        return k.partials + slot * k.dim_padded + col + lane * W;
    }
    // Keep the sum of a run that crosses the piece's bounds.
    __device__ void leave_partial(int64_t piece, bool from_before) {
        float* to = partial(2 * piece + (from_before ? 0 : 1));
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (inside(v)) store_vec<Cache::KEEP, float, W>(to + v * 32 * W, acc[v]);
    }
    // This piece's part of the run of `id` is kept: the last piece to come here
    // adds the parts in piece order.
    __device__ void join(unsigned id, int panel) {
        const int n = (int)p.tokens;
        const int a = warp_count_below(k.keys, n, (uint64_t)id << 32, lane);
        const int b = warp_count_below(k.keys, n, (uint64_t)(id + 1) << 32, lane);
        const int64_t first = a / k.piece, last = (b - 1) / k.piece;
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = atomicAdd(k.arrived + first * k.panels + panel, 1);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before != last - first) return;
        __threadfence();
        clear();
        for (int64_t q = first; q <= last; q += 4) {
            float got[4][V][W];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        got[u][v][i] = q + u <= last && inside(v)
                                           ? __ldcg(partial(2 * (q + u) + (q + u == first ? 1 : 0)) +
                                                    v * 32 * W + i)
                                           : 0.0f;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < W; ++i) acc[v][i] += got[u][v][i];
        }
        finish(id);
    }

    __device__ void sum(int64_t piece, int panel) {
        const T* dout = static_cast<const T*>(p.dout) + col + lane * W;
        const int s0 = (int)(piece * k.piece);
        const int s1 = (int)min((int64_t)s0 + k.piece, p.tokens);
        unsigned run = (unsigned)(k.keys[s0] >> 32);            // the id being summed
        if (run == NO_ID) return;
        bool from_before = s0 > 0 && (unsigned)(k.keys[s0 - 1] >> 32) == run;
        unsigned head = NO_ID;                                  // a run from before that ended
        clear();
        for (int base = s0; base < s1; base += 32) {
            const uint64_t mine = base + lane < s1 ? k.keys[base + lane] : ~0ull;
            const unsigned id_l = (unsigned)(mine >> 32), pos_l = (unsigned)mine;
            const int live = __popc(__ballot_sync(0xffffffffu, id_l != NO_ID));  // a prefix
            for (int j = 0; j < live; j += BATCH) {
                Vec<T, W> x[BATCH][V];
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int64_t row = __shfl_sync(0xffffffffu, pos_l, (j + u) & 31);
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (j + u < live && inside(v))
                            x[u][v] = load_vec<Cache::STREAM, T, W>(dout + row * p.ld_dout +
                                                                    v * 32 * W);
                }
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const unsigned id = __shfl_sync(0xffffffffu, id_l, (j + u) & 31);
                    if (j + u >= live) break;
                    if (id != run) {                            // the run before ends here
                        if (from_before) {
                            leave_partial(piece, true);
                            head = run;
                            from_before = false;
                        } else {
                            finish(run);
                        }
                        clear();
                        run = id;
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float f[W];
                        unpack(x[u][v], f);
#pragma unroll
                        for (int i = 0; i < W; ++i) acc[v][i] += f[i];
                    }
                }
            }
            if (live < 32) break;
        }
        const bool goes_on = s1 < p.tokens && (unsigned)(k.keys[s1] >> 32) == run;
        const bool crosses = from_before || goes_on;
        if (crosses) leave_partial(piece, from_before);
        else finish(run);
        if (head != NO_ID) join(head, panel);
        if (crosses) join(run, panel);
    }
};

// Rows without a token: beta * dtable, zeros for beta == 0.
template <typename G, int W>
__device__ void fill_rows(const EmbedGradParams& p, const GradWork& k, int64_t item, int lane) {
    const int64_t v0 = item * k.fill_rows;
    const int rows = (int)min((int64_t)k.fill_rows, p.vocab - v0);
    const int n = (int)p.tokens;
    const unsigned all = rows == 32 ? ~0u : (1u << rows) - 1;
    // where the first of these rows would be, and 32 keys from there: enough unless
    // its tokens are many, and then the other rows look for themselves
    const int at = warp_count_below(k.keys, n, (uint64_t)v0 << 32, lane);
    const uint64_t key = at + lane < n ? k.keys[at + lane] : ~0ull;
    const int64_t row = (int64_t)(key >> 32) - v0;
    unsigned present = __reduce_or_sync(0xffffffffu, row < rows ? 1u << row : 0u);
    if (__shfl_sync(0xffffffffu, row, 31) < rows) {
        bool here = false;
        if (lane < rows) {
            const int i = count_below(k.keys, n, (uint64_t)(v0 + lane) << 32);
            here = i < n && (int64_t)(k.keys[i] >> 32) == v0 + lane;
        }
        present = __ballot_sync(0xffffffffu, here);
    }
    const unsigned todo = all & ~present;
    for (int r = 0; r < rows; ++r) {
        if (!(todo >> r & 1)) continue;
        G* to = static_cast<G*>(p.dtable) + (v0 + r) * p.ld_dtable;
        for (int64_t c = lane * W; c < p.dim; c += 32 * W) {
            float f[W];
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = 0.0f;
            if (p.beta != 0.0f) {
                unpack(load_vec<Cache::STREAM, G, W>(to + c), f);
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] *= p.beta;
            }
            store_vec<Cache::STREAM, G, W>(to + c, f);
        }
    }
}

template <typename T, typename G, int W, int V, int BATCH>
__global__ __launch_bounds__(256) void grad_sums(EmbedGradParams p, GradWork k) {
    wait_for_predecessor();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item < k.sum_items) {
        const int panel = (int)(item % k.panels);
        GradSum<T, G, W, V, BATCH> s{p, k, lane, (int64_t)panel * PANEL};
        s.sum(item / k.panels, panel);
    } else {
        const int64_t fill = item - k.sum_items;
        if (fill * k.fill_rows < p.vocab) fill_rows<G, W>(p, k, fill, lane);
    }
}

struct GradLayout {
    size_t keys, other, arrived, partials, total;
};
GradLayout grad_layout(int64_t tokens, int64_t dim) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const int piece = piece_of(tokens, dim);
    const size_t pieces = (size_t)((tokens + piece - 1) / piece);
    GradLayout l{};
    l.other = up((size_t)tokens * 8);
    l.arrived = l.other + up((size_t)tokens * 8);
    l.partials = l.arrived + up(pieces * (size_t)panels_of(dim) * sizeof(int));
    l.total = l.partials + up(pieces * 2 * (size_t)padded(dim) * sizeof(float));
    return l;
}

}  // namespace

cudaError_t launch_embedding(spmm_type_t type, const EmbedParams& p, int num_sms,
                             cudaStream_t st) {
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        constexpr int W = 16 / sizeof(T);
        const bool wide = p.dim % W == 0 && rows_aligned16(p.out, p.ld_out, sizeof(T)) &&
                          (p.vocab == 0 || rows_aligned16(p.table, p.ld_table, sizeof(T)));
        return wide ? launch_embed<T, W>(p, num_sms, st) : launch_embed<T, 1>(p, num_sms, st);
    });
}

size_t embed_grad_scratch(int64_t tokens, int64_t dim) { return grad_layout(tokens, dim).total; }

// Pieces get longer as the work grows, so a smaller call may need more: what
// covers every call.  pieces <= min(tokens, SUM_WARPS / panels + 1), or
// tokens / PIECE_MAX + 1 once the pieces are longest; padded(dim) <= PANEL * panels.
size_t embed_grad_scratch_upto(int64_t tokens, int64_t dim) {
    const size_t wide = (size_t)padded(dim), most = (size_t)tokens / PIECE_MAX + 1;
    const size_t rows = std::max(
        std::min((size_t)tokens * wide, (size_t)SUM_WARPS * PANEL + wide), most * wide);
    const size_t counters = std::max((size_t)SUM_WARPS + panels_of(dim), most * panels_of(dim));
    return (size_t)tokens * 16 + counters * sizeof(int) + rows * 2 * sizeof(float) + 4 * 256;
}

cudaError_t launch_embedding_grad(spmm_type_t type, spmm_type_t grad_type,
                                  const EmbedGradParams& p, char* scratch, int num_sms,
                                  cudaStream_t st) {
    (void)num_sms;
    const GradLayout l = grad_layout(p.tokens, p.dim);
    uint64_t* keys = reinterpret_cast<uint64_t*>(scratch);
    uint64_t* other = reinterpret_cast<uint64_t*>(scratch + l.other);
    GradWork k{};
    k.arrived = reinterpret_cast<int*>(scratch + l.arrived);
    k.partials = reinterpret_cast<float*>(scratch + l.partials);
    k.dim_padded = padded(p.dim);
    k.piece = piece_of(p.tokens, p.dim);
    k.panels = (int)panels_of(p.dim);
    k.sum_items = (p.tokens + k.piece - 1) / k.piece * k.panels;
    // a filling warp writes about 32 KB when no row of its share has a token
    const int64_t row_bytes = p.dim * lm_elem_size(grad_type);
    k.fill_rows = (int)std::min<int64_t>(32, std::max<int64_t>(1, 32768 / row_bytes));
    const int64_t fill_items =
        p.beta == 1.0f ? 0 : (p.vocab + k.fill_rows - 1) / k.fill_rows;
    if (p.tokens > 0) {
        const int tiles = (int)((p.tokens + SORT_TILE - 1) / SORT_TILE);
        sort_tiles<<<tiles, SORT_TILE, 0, st>>>(p.ids, (int)p.tokens, p.vocab, keys, k.arrived,
                                                k.sum_items);
        cudaError_t e = cudaGetLastError();
        for (int64_t run = SORT_TILE; e == cudaSuccess && run < p.tokens; run *= MERGE_WAYS) {
            e = launch_chained(merge_runs, dim3((unsigned)((p.tokens + 255) / 256)), dim3(256), 0,
                               st, true, (const uint64_t*)keys, other, (int)p.tokens, run);
            std::swap(keys, other);
        }
        if (e != cudaSuccess) return e;
    }
    k.keys = keys;
    const int64_t blocks = (k.sum_items + fill_items + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    const bool same = type == grad_type;
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        constexpr int W = 16 / sizeof(T);
        auto run = [&](auto kernel) {
            return launch_chained(kernel, dim3((unsigned)blocks), dim3(256), 0, st, p.tokens > 0,
                                  p, k);
        };
        const bool wide = p.dim % W == 0 &&
                          rows_aligned16(p.dtable, p.ld_dtable, lm_elem_size(grad_type)) &&
                          (p.tokens == 0 || rows_aligned16(p.dout, p.ld_dout, sizeof(T)));
        if (same)
            return wide ? run(grad_sums<T, T, W, PANEL / 32 / W, W>)
                        : run(grad_sums<T, T, 1, PANEL / 32, 4>);
        return wide ? run(grad_sums<T, float, W, PANEL / 32 / W, W>)
                    : run(grad_sums<T, float, 1, PANEL / 32, 4>);
    });
}

}  // namespace spmm
