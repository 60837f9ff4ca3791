// Embedding lookup out[t, :] = scale * table[ids[t], :] and its gradient
// dtable[v, :] = beta * dtable[v, :] + scale * sum_{t: ids[t] = v} dout[t, :].
//
// The gradient is the product of the transposed one-entry-per-row matrix with
// dout.  Its row structure is made on the device by sorting the tokens by id:
// keys (id << 32 | position) are unique, so any correct sort of them is the
// stable order, and the sums below have a fixed order.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "spmm_internal.h"
#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

// ---- lookup -----------------------------------------------------------------

constexpr int EMBED_THREADS = 256;
constexpr int EMBED_BATCH = 4;       // accesses in flight per thread

// The elements of an access times scale; padding: zeros, by its bits rather than element
// by element.
template <typename T, int W>
__device__ __forceinline__ void scaled(Vec<T, W> got, int id, const EmbedParams& p, float (&f)[W]) {
    const bool valid = id >= 0 && id < p.vocab;
    const uint32_t keep = valid ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < Vec<T, W>::WORDS; ++i) got.w[i] &= keep;
    const float scale = valid ? p.scale : 0.0f;
    const uint64_t scale2 = pair(scale, scale);
    unpack(got, f);
#pragma unroll
    for (int i = 0; i < W; i += 2) halves(mul2(pair(f[i], f[i + 1]), scale2), f[i], f[i + 1]);
}

// A block takes `block_rows` rows; its threads walk the rows' accesses in
// order (nv accesses of 16 bytes per row, then the next row), so narrow
// rows share a warp and the stores of neighbouring threads are contiguous.
// The bound is HBM: one table row read and one written per token.  100,003
// Zipf-distributed tokens of 4096 bf16: 172 us, 6.1 TB/s of distinct rows read and rows
// written (90% of the copy rate; 241 us before a batch's accesses were free of branches
// and kept packed).
template <typename T>
__global__ __launch_bounds__(EMBED_THREADS) void embed_rows(EmbedParams p, int nv,
                                                            int block_rows) {
    constexpr int W = 16 / (int)sizeof(T);
    const T* table = static_cast<const T*>(p.table);
    const int64_t row0 = (int64_t)blockIdx.x * block_rows;
    const int* ids = p.ids + row0;
    T* out = static_cast<T*>(p.out) + row0 * p.ld_out;
    const int rows = (int)min((int64_t)block_rows, p.tokens - row0);
    const int step_r = EMBED_THREADS / nv, step_c = EMBED_THREADS % nv;
    int r = threadIdx.x / nv, c = threadIdx.x % nv;
    while (r < rows) {
        // ids, then rows, each for the whole batch and none behind a branch (past the
        // block's rows and for padding some row is read in vain), so that all are
        // on their way together
        int id[EMBED_BATCH], row[EMBED_BATCH], col[EMBED_BATCH];
        Vec<T, W> v[EMBED_BATCH];
#pragma unroll
        for (int u = 0; u < EMBED_BATCH; ++u) {
            row[u] = r;
            col[u] = c * W;
            id[u] = ids[min(r, rows - 1)];
            r += step_r;
            c += step_c;
            if (c >= nv) {
                c -= nv;
                ++r;
            }
        }
        if (p.vocab > 0) {
#pragma unroll
            for (int u = 0; u < EMBED_BATCH; ++u) {
                const bool valid = id[u] >= 0 && id[u] < p.vocab;
                v[u] = load_vec<Cache::KEEP, T, W>(table + (valid ? id[u] : 0) * p.ld_table +
                                                   col[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < EMBED_BATCH; ++u) {
            if (row[u] >= rows) continue;
            float f[W];
            scaled(v[u], id[u], p, f);
            store_vec<Cache::STREAM, T, W>(out + row[u] * p.ld_out + col[u], f);
        }
    }
}

// Any width and alignment: accesses are those of out's aligned words, and the table is
// read from wherever their elements lie, as the two aligned words around them.  What
// places a row (its id, its first word, the shift between the two) is found once and
// serves COLS accesses of each of its lanes (a power of two of them, a warp's where it has as
// many accesses), or one where a thread takes ROWS rows: EMBED_BATCH in flight either way.
// Where lanes of a warp have one row its shift is theirs, and the words it takes are chosen by
// a branch.  A warp goes through its row part by part, because the parts share sectors, which
// have to be written together; only few rows are spread over blockIdx.y.  100,000 x 2001
// bf16 take 92 us (79% of the copy rate), 115 with the parts over the grid, 111 with four
// rows per warp and 140 with accesses that place themselves one by one as above.
template <typename T, int ROWS>
__global__ __launch_bounds__(EMBED_THREADS, 4) void embed_shifted(EmbedParams p, int lanes_log,
                                                                  int parts, int used) {
    constexpr int W = 16 / (int)sizeof(T), COLS = EMBED_BATCH / ROWS;
    const T* table = static_cast<const T*>(p.table);
    const int lane = threadIdx.x & ((1 << lanes_log) - 1);
    const int64_t row0 =
        (((int64_t)blockIdx.x * EMBED_THREADS + threadIdx.x) >> lanes_log) * ROWS;
    if (row0 >= p.tokens) return;
    const int dim = (int)p.dim;
    const int64_t elements = (p.vocab - 1) * p.ld_table + p.dim;
    int id[ROWS], lead[ROWS], nv[ROWS];
    int64_t at[ROWS];
    T* to[ROWS];
    bool clear = true;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) id[r] = p.ids[min(row0 + r, p.tokens - 1)];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        to[r] = static_cast<T*>(p.out) + min(row0 + r, p.tokens - 1) * p.ld_out;
        lead[r] = lead_of(to[r], 16);
        nv[r] = (dim + lead[r] + W - 1) / W;
        const bool valid = id[r] >= 0 && id[r] < p.vocab;
        // padding: some row away from the table's ends is read in vain
        at[r] = (valid ? id[r] : p.vocab / 2) * p.ld_table;
        // an access begins at most W - 1 elements before the row and at most at its last,
        // and its aligned words reach from less than W before it to less than 2 W behind
        clear &= at[r] >= 2 * W && at[r] + dim + 2 * W <= elements;
    }
    for (int part = blockIdx.y; part < parts; part += gridDim.y) {
        const int first = part * used * 32 + lane;              // its accesses: 32 apart
        Vec<T, W> v[ROWS][COLS];
        if (clear) {
            // all at once; past the row its last one again
            Unaligned<T> far[ROWS][COLS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int u = 0; u < COLS; ++u)
                    far[r][u].load(
                        table + at[r] +
                        (min(first + (u < used ? u * 32 : 0), nv[r] - 1) * W - lead[r]));
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if constexpr (ROWS <= 2) {
                    auto take = [&](auto word) {
#pragma unroll
                        for (int u = 0; u < COLS; ++u)
                            v[r][u] = far[r][u].template from_word<decltype(word)::value>();
                    };
                    switch (far[r][0].shift / 4) {
                        case 0: take(std::integral_constant<int, 0>{}); break;
                        case 1: take(std::integral_constant<int, 1>{}); break;
                        case 2: take(std::integral_constant<int, 2>{}); break;
                        default: take(std::integral_constant<int, 3>{});
                    }
                } else {
                    v[r][0] = far[r][0].get();
                }
            }
        } else if (p.vocab > 0) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int u = 0; u < COLS; ++u)
                    v[r][u] = load_some<T, W>(table + at[r], (first + u * 32) * W - lead[r], dim);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (row0 + r >= p.tokens) break;
#pragma unroll
            for (int u = 0; u < COLS; ++u) {
                if (u >= used) break;
                float f[W];
                scaled(v[r][u], id[r], p, f);
                store_some<T, W>(to[r], (first + u * 32) * W - lead[r], dim, f);
            }
        }
    }
}

template <typename T>
cudaError_t launch_embed(const EmbedParams& p, bool whole, int num_sms, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);
    if (whole) {
        // about 8 accesses per thread and block; fewer rows per block while that
        // would leave SMs without a block
        const int nv = (int)(p.dim / W);
        int64_t rows = std::max<int64_t>(1, EMBED_THREADS * 8 / nv);
        rows = std::max<int64_t>(1, std::min<int64_t>(rows, p.tokens / (4 * num_sms)));
        const unsigned blocks = (unsigned)((p.tokens + rows - 1) / rows);
        return launch(embed_rows<T>, blocks, EMBED_THREADS, 0, st, p, nv, (int)rows);
    }
    // a row between boundaries covers up to W - 1 elements more
    const int64_t nv = (p.dim + 2 * (W - 1)) / W;
    int lanes_log = 0;
    while (lanes_log < 5 && (1 << lanes_log) < nv) ++lanes_log;
    const int lane_accesses = (int)((nv + 31) / 32);
    const int rows = lane_accesses == 1 ? 4 : lane_accesses == 2 ? 2 : 1;
    const int parts = (lane_accesses + EMBED_BATCH / rows - 1) / (EMBED_BATCH / rows);
    const int used = (lane_accesses + parts - 1) / parts;
    const int64_t block_rows = (int64_t)(EMBED_THREADS >> lanes_log) * rows;
    const int64_t blocks = (p.tokens + block_rows - 1) / block_rows;
    const dim3 grid((unsigned)blocks, (unsigned)std::min<int64_t>(
                                          parts, std::max<int64_t>(1, 4 * num_sms / blocks)));
    auto run = [&](auto kernel) {
        return launch(kernel, grid, EMBED_THREADS, 0, st, p, lanes_log, parts, used);
    };
    return rows == 4   ? run(embed_shifted<T, 4>)
           : rows == 2 ? run(embed_shifted<T, 2>) : run(embed_shifted<T, 1>);
}

// ---- gradient: sort ------------------------------------------------------------

constexpr int SORT_TILE = 512;       // keys sorted by one block, one per thread
constexpr int MERGE_WAYS = 16;       // sorted runs merged per round, at most
// From so many keys on the searches cost more than the launches they save, and fours
// merged round by round have the fewest: 300,000 tokens of 64 columns take 134 us, with 16
// runs to a round 167 and with 8 168; 65,536 tokens the same either way.
constexpr unsigned MERGE_MANY = 32768;
constexpr unsigned NO_ID = 0xfffffffdu;  // of padding tokens
constexpr unsigned REST = 0xfffffffeu;   // behind them, what fills the last tile

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
    uint64_t key = (uint64_t)REST << 32;
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
    keys[at] = key;
    if (at == 0) keys[(int64_t)gridDim.x * SORT_TILE] = ~0ull;
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

// Merges groups of WAYS sorted runs of `run` keys (a power of two): each key's place
// is the count of smaller keys over the group's runs.  An earlier run holds earlier
// tokens, so of equal ids those of earlier runs count, and the ids alone decide.
// A block takes 32 consecutive keys, a warp of it one of the runs: its lanes search
// for neighbouring keys, so their probes share memory words, and a search is one chain
// of loads with many others beside it: 8192 keys 5 us (one thread per key with WAYS
// chains: 25 us, its loads waiting for one another).  Behind the `total` keys (whole
// tiles) lies a largest one, which ends every search that would go further.  The keys are
// read through ordinary loads: the kernel may start while its predecessor writes them, so
// they are not constant for its lifetime.
template <int WAYS>
__global__ __launch_bounds__(32 * WAYS) void merge_runs(const uint64_t* in, uint64_t* out,
                                                        unsigned total, unsigned run) {
    __shared__ unsigned count[WAYS][32];
    allow_successor();
    wait_for_predecessor();
    const unsigned lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const unsigned g = blockIdx.x * 32 + lane;
    if (g == 0 && q == 0) out[total] = ~0ull;
    const uint64_t key = in[g];
    const unsigned* ids = reinterpret_cast<const unsigned*>(in) + 1;     // of key i at 2 i
    // total <= 2^30 and run < total: no sum of these reaches 2^32 before it is cut at total
    const uint64_t group = (uint64_t)run * WAYS;
    const unsigned first = (unsigned)(g / group * group);
    const unsigned own = (g - first) / run;
    const unsigned start = (unsigned)min(first + (uint64_t)q * run, (uint64_t)total);
    unsigned below = start;
    if (q == own) {
        below = g;
    } else {
        const unsigned bound = (unsigned)(key >> 32) + (q < own);
        for (unsigned half = run >> 1; half > 0; half >>= 1)
            below += ids[2 * min(below + half - 1, total)] < bound ? half : 0;
        below += ids[2 * min(below, total)] < bound;            // one candidate is left
    }
    count[q][lane] = below - start;
    __syncthreads();
    if (q > 0) return;
    unsigned place = first;
#pragma unroll
    for (int i = 0; i < WAYS; ++i) place += count[i][lane];
    out[place] = key;
}

// ---- gradient: sums --------------------------------------------------------------

// The sorted tokens are cut into pieces of equal length; a warp sums one piece
// over one panel of columns, reading each token's row segment once.  A run of
// one id that lies within the piece is complete and goes to its table row; a
// run that crosses the piece's bounds leaves a partial sum.  Of each JOIN pieces
// (by number) the last one to arrive adds the run's partials in piece order, and
// the last of those sums to arrive adds them in order: a token that makes up a
// tenth of 300,000 has near a thousand pieces.  Warps behind those of the sums write the
// rows without a token.  The bound is HBM: 65,536 tokens of 4096 bf16 into a table of
// 131,072 binary32 rows take 407 us with the sort, 6.5 TB/s of what must move (97% of
// the copy rate).  80 registers for three blocks per SM (some spill in the joins): 414 us
// with 99 and two, and where rows are added to instead of written 294 us against 252.
constexpr int PANEL = 256;           // columns per warp: 512 bytes of a 16-bit row
constexpr int PIECE_MAX = 128;
constexpr int64_t SUM_WARPS = 4096;
constexpr int JOIN = 32;             // pieces of a run joined at once
constexpr int COUNTERS = 3;          // per piece and panel

// Tokens per piece: as many as leave about SUM_WARPS warps of work (about what the SMs
// hold at once), so that few runs are cut; one where there is less, because a warp's
// tokens wait for one another.  8192 tokens of 2048 bf16 take 41 us with 4096 warps, 45
// with 8192 and 43 with 2048; 1224 tokens of 6263 f16 added to their rows 34, 39 and 28,
// but 20,000 of 2001 bf16 73, 74 and 97.  No piece is longer than PIECE_MAX: 65,536
// tokens of 4096 bf16 added to binary32 rows take 251 us with 128 and 272 with 256.  It
// depends on the call's sizes only, so the order of every sum does too.
inline int64_t panels_of(int64_t dim) { return (dim + PANEL - 1) / PANEL; }
inline int piece_log_of(int64_t tokens, int64_t dim) {
    int log = 0;
    while ((1 << log) < PIECE_MAX && (tokens * panels_of(dim) >> log) > SUM_WARPS) ++log;
    return log;
}
inline int64_t pieces_of(int64_t tokens, int piece_log) {
    return (tokens + (1 << piece_log) - 1) >> piece_log;
}
// A partial row: whole accesses of 32 bytes, one more for rows between boundaries.
inline int64_t padded(int64_t dim) { return (dim + 7) / 8 * 8 + 8; }

struct GradWork {
    const uint64_t* keys;            // sorted
    float* partials;                 // [pieces][2][padded dim]: run from before, run to the next
    int* arrived;                    // [COUNTERS][pieces][panels], zeroed by sort_tiles
    int64_t dim_padded;
    int piece_log;                   // tokens per piece: a power of two
    int pieces;
    int panels;
    int64_t sum_items;               // pieces * panels warps sum; the rest fill
    int fill_rows;                   // table rows per filling warp
};

// Number of keys below each of `key`, by the whole warp: 32 probes per key and step.
template <int N>
__device__ __forceinline__ void warp_count_below(const uint64_t* a, int n, const uint64_t (&key)[N],
                                                 int (&count)[N], int lane) {
    int lo[N], hi[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        lo[i] = 0;
        hi[i] = n;
    }
    bool open = n > 0;
    while (open) {
        uint64_t got[N];
        int step[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            step[i] = (hi[i] - lo[i]) / 32 + 1;
            got[i] = a[min((int64_t)lo[i] + (int64_t)lane * step[i], (int64_t)n - 1)];
        }
        open = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool is = (int64_t)lo[i] + (int64_t)lane * step[i] < hi[i];
            const int k = __popc(__ballot_sync(0xffffffffu, is & (got[i] < key[i])));
            if (k == 0) {
                hi[i] = lo[i];
            } else {
                hi[i] = (int)min((int64_t)hi[i], lo[i] + (int64_t)k * step[i]);
                lo[i] += (k - 1) * step[i] + 1;
            }
            open |= lo[i] < hi[i];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) count[i] = lo[i];
}

// W elements per access, V accesses per lane and row segment: W * V * 32 == PANEL.
// EDGES: any width and alignment: accesses are those of the table row's aligned words
// (its first begins `lead` columns before it), and dout is read from wherever their
// elements lie.
template <typename T, typename G, int W, int V, int BATCH, bool EDGES>
struct GradSum {
    static_assert(W * V * 32 == PANEL);
    const EmbedGradParams& p;
    const GradWork& k;
    int lane;
    int col;                         // the panel's first column
    int dim;
    int lead;                        // of the row being summed
    float acc[V][W];

    __device__ G* row_of(unsigned id) const {
        return static_cast<G*>(p.dtable) + (int64_t)id * p.ld_dtable;
    }
    __device__ int lead_for(unsigned id) const { return EDGES ? lead_of(row_of(id), 16) : 0; }
    __device__ int column(int v, int lead) const { return col + (v * 32 + lane) * W - lead; }
    __device__ void begin(unsigned id) {
        lead = lead_for(id);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < W; ++i) acc[v][i] = 0.0f;
    }
    // dtable[row] = beta * dtable[row] + scale * acc
    __device__ void finish(unsigned id) {
        G* to = row_of(id);
        Vec<G, W> old[V];
        if (p.beta != 0.0f)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // past the row column 0 is read in vain: an access behind a branch would
                // keep the others waiting
                const int c = column(v, lead);
                if constexpr (EDGES)
                    old[v] = c >= 0 && c + W <= dim ? load_vec<Cache::STREAM, G, W>(to + c)
                                                    : load_some<G, W>(to, c, dim);
                else
                    old[v] = load_vec<Cache::STREAM, G, W>(to + (c < dim ? c : 0));
            }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f[W];
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = p.scale * acc[v][i];
            if (p.beta != 0.0f) {
                float o[W];
                unpack(old[v], o);
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] += p.beta * o[i];
            }
            const int c = column(v, lead);
            if (EDGES) store_some<G, W>(to, c, dim, f);
            else if (c < dim) store_vec<Cache::STREAM, G, W>(to + c, f);
        }
    }
    // partial rows begin with the lead
    __device__ float* partial(int64_t slot) const { return k.partials + slot * k.dim_padded; }
    __device__ bool inside(int v) const { return column(v, lead) < dim; }
    // Keep the sum of a run that crosses the piece's bounds.
    __device__ void leave_partial(int piece, bool from_before) {
        float* to = partial(2 * (int64_t)piece + (from_before ? 0 : 1));
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (inside(v)) store_vec<Cache::KEEP, float, W>(to + column(v, 0), acc[v]);
    }
    // Whether this warp is the last of `all` to come to a counter; what the others wrote
    // before is visible then: one lane's count releases what its warp wrote and acquires
    // what the warps counted before it did (a fence of every lane on both sides costs more).
    __device__ bool last_of(int64_t counter, int panel, int64_t all) const {
        unsigned before = 0;
        __syncwarp();
        if (lane == 0)
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                         : "=r"(before)
                         : "l"(k.arrived + counter * k.panels + panel)
                         : "memory");
        __syncwarp();
        return __shfl_sync(0xffffffffu, before, 0) == all - 1;
    }
    // Adds the partials of every `stride`-th piece from `from` to `to`; of the run's first
    // piece `first` it is the second one.
    __device__ void add_partials(int from, int to, int stride, int first) {
        constexpr int MANY = 32 / (V * W);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < W; ++i) acc[v][i] = 0.0f;
        for (int q = from; q <= to; q += MANY * stride) {
            float got[MANY][V][W];
#pragma unroll
            for (int u = 0; u < MANY; ++u) {
                const int piece = q + u * stride <= to ? q + u * stride : q;
                const float* part = partial(2 * (int64_t)piece + (piece == first));
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        got[u][v][i] = __ldcg(part + (inside(v) ? column(v, 0) : 0) + i);
            }
#pragma unroll
            for (int u = 0; u < MANY; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        acc[v][i] += q + u * stride <= to ? got[u][v][i] : 0.0f;
        }
    }
    // The first and the last piece of the run of `id`, which goes through `piece`'s bounds.
    __device__ void run_pieces(int piece, unsigned id, int& first, int& last) const {
        // The pieces' own first keys tell how far the run goes on, the keys before them
        // whether it came from before: 32 of each at once.
        const int behind = piece + 1 + lane, before = piece - lane;
        const unsigned at = (unsigned)min(behind, k.pieces - 1) << k.piece_log;
        const unsigned from = (unsigned)max(before, 1) << k.piece_log;
        const bool goes_on = (unsigned)(k.keys[at] >> 32) == id && behind < k.pieces;
        const bool came = (unsigned)(k.keys[min((int64_t)from, p.tokens) - 1] >> 32) == id && before > 0;
        const unsigned on = __ballot_sync(0xffffffffu, goes_on);
        const unsigned back = __ballot_sync(0xffffffffu, came);
        if ((on != ~0u) & (back != ~0u)) {
            first = piece - (__ffs(~back) - 1);
            last = piece + (__ffs(~on) - 1);
            return;
        }
        const uint64_t bounds[2] = {(uint64_t)id << 32, (uint64_t)(id + 1) << 32};
        int place[2];
        warp_count_below(k.keys, (int)p.tokens, bounds, place, lane);
        first = place[0] >> k.piece_log;
        last = (place[1] - 1) >> k.piece_log;
    }
    // This piece's part of the run of `id` is kept: the last to come here joins the parts.
    __device__ void join(int piece, unsigned id, int panel) {
        int first, last;
        run_pieces(piece, id, first, last);
        const int from = max(first, piece / JOIN * JOIN);
        const int to = min(last, piece / JOIN * JOIN + JOIN - 1);
        const int64_t pieces = k.pieces;
        // a piece begins one run and may continue another: two counters
        if (!last_of((from == first ? pieces : 0) + from, panel, to - from + 1)) return;
        lead = lead_for(id);
        add_partials(from, to, 1, first);
        if (first / JOIN != last / JOIN) {
            float* sum = partial(2 * (int64_t)from + (from == first));
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (inside(v)) store_vec<Cache::KEEP, float, W>(sum + column(v, 0), acc[v]);
            if (!last_of(2 * pieces + first, panel, last / JOIN - first / JOIN + 1)) return;
            // the first group's sum is at `first`, the others' at their first pieces
            add_partials((first / JOIN + 1) * JOIN, last, JOIN, first);
            const float* part = partial(2 * (int64_t)first + 1);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    acc[v][i] = __ldcg(part + (inside(v) ? column(v, 0) : 0) + i) + acc[v][i];
        }
        finish(id);
    }

    __device__ void sum(int piece, int panel) {
        const T* dout = static_cast<const T*>(p.dout);
        const int64_t elements = (p.tokens - 1) * p.ld_dout + p.dim;
        const int s0 = piece << k.piece_log;
        const int s1 = (int)min((int64_t)s0 + (1 << k.piece_log), p.tokens);
        // the first keys, the one before and the one behind (which is there always), all
        // on their way together
        uint64_t mine = k.keys[min(s0 + lane, s1 - 1)];
        const uint64_t key_before = k.keys[max(s0 - 1, 0)], key_behind = k.keys[s1];
        unsigned run = (unsigned)(__shfl_sync(0xffffffffu, mine, 0) >> 32);   // the id being summed
        if (run == NO_ID) return;
        bool from_before = s0 > 0 && (unsigned)(key_before >> 32) == run;
        unsigned head = NO_ID;                                  // a run from before that ended
        begin(run);
        for (int base = s0; base < s1; base += 32) {
            if (base > s0) mine = k.keys[min(base + lane, s1 - 1)];
            const unsigned pos_l = (unsigned)mine;
            const unsigned id_l = base + lane < s1 ? (unsigned)(mine >> 32) : NO_ID;
            const int live = __popc(__ballot_sync(0xffffffffu, id_l != NO_ID));  // a prefix
            for (int j = 0; j < live; j += BATCH) {
                // all of a batch's rows at once; past the live ones and past the row some
                // element is read in vain
                using Read = std::conditional_t<EDGES, Unaligned<T>, Vec<T, W>>;
                Read x[BATCH][V];
                int64_t row[BATCH];
                int leads[BATCH];
                bool clear = true;
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int from = min(j + u, live - 1);
                    row[u] = __shfl_sync(0xffffffffu, pos_l, from) * p.ld_dout;
                    if constexpr (EDGES) {
                        leads[u] = lead_for(__shfl_sync(0xffffffffu, id_l, from));
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            clear &= clear_of_ends<W>(row[u] + min(column(v, leads[u]), dim - 1),
                                                      elements);
                    }
                }
                if constexpr (EDGES) {
                    if (clear) {
#pragma unroll
                        for (int u = 0; u < BATCH; ++u)
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                x[u][v].load(dout + row[u] + min(column(v, leads[u]), dim - 1));
                    } else {
#pragma unroll
                        for (int u = 0; u < BATCH; ++u)
#pragma unroll
                            for (int v = 0; v < V; ++v) {
                                x[u][v].a = load_some<T, W>(dout + row[u], column(v, leads[u]), dim);
                                x[u][v].b = x[u][v].a;
                                x[u][v].shift = 0;
                            }
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < BATCH; ++u)
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            x[u][v] = load_vec<Cache::STREAM, T, W>(
                                dout + row[u] + (column(v, 0) < dim ? column(v, 0) : 0));
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
                        begin(id);
                        run = id;
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float f[W];
                        if constexpr (EDGES) unpack(x[u][v].get(), f);
                        else unpack(x[u][v], f);
#pragma unroll
                        for (int i = 0; i < W; ++i) acc[v][i] += f[i];
                    }
                }
            }
            if (live < 32) break;
        }
        const bool goes_on = s1 < p.tokens && (unsigned)(key_behind >> 32) == run;
        const bool crosses = from_before || goes_on;
        if (crosses) leave_partial(piece, from_before);
        else finish(run);
        if (head != NO_ID) join(piece, head, panel);
        if (crosses) join(piece, run, panel);
    }
};

// Rows without a token: beta * dtable, zeros for beta == 0.
template <typename G, bool EDGES>
__device__ void fill_rows(const EmbedGradParams& p, const GradWork& k, int64_t item, int lane) {
    const int64_t v0 = item * k.fill_rows;
    const int rows = (int)min((int64_t)k.fill_rows, p.vocab - v0);
    const int n = (int)p.tokens;
    const unsigned all = rows == 32 ? ~0u : (1u << rows) - 1;
    // where the first of these rows would be, and 32 keys from there: enough unless
    // its tokens are many, and then the other rows look for themselves
    const uint64_t bound[1] = {(uint64_t)v0 << 32};
    int found[1];
    warp_count_below(k.keys, n, bound, found, lane);
    const int at = found[0];
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
        constexpr int W = 16 / (int)sizeof(G);
        G* to = static_cast<G*>(p.dtable) + (v0 + r) * p.ld_dtable;
        const int dim = (int)p.dim;
        for (int c = lane * W - (EDGES ? lead_of(to, 16) : 0); c < dim; c += 32 * W) {
            float f[W];
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = 0.0f;
            if (p.beta != 0.0f) {
                unpack(!EDGES || (c >= 0 && c + W <= dim) ? load_vec<Cache::STREAM, G, W>(to + c)
                                                          : load_some<G, W>(to, c, dim), f);
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] *= p.beta;
            }
            if (EDGES) store_some<G, W>(to, c, dim, f);
            else store_vec<Cache::STREAM, G, W>(to + c, f);
        }
    }
}

template <typename T, typename G, bool EDGES>
__global__ __launch_bounds__(256, 3) void grad_sums(EmbedGradParams p, GradWork k) {
    constexpr int W = 16 / (int)sizeof(T), V = PANEL / 32 / W;
    constexpr int BATCH = EDGES ? 4 / V : 8 / V;     // 8 words in flight per lane
    wait_for_predecessor();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item < k.sum_items) {
        // a division of 32 bits where it will do
        const int piece = (int)(item <= UINT_MAX ? (unsigned)item / (unsigned)k.panels
                                                 : item / k.panels);
        const int panel = (int)(item - (int64_t)piece * k.panels);
        GradSum<T, G, W, V, BATCH, EDGES> s{p, k, lane, panel * PANEL, (int)p.dim};
        s.sum(piece, panel);
    } else {
        const int64_t fill = item - k.sum_items;
        if (fill * k.fill_rows < p.vocab) fill_rows<G, EDGES>(p, k, fill, lane);
    }
}

// Whole tiles and the key behind them.
size_t key_bytes(int64_t tokens) {
    return (size_t)((tokens + SORT_TILE - 1) / SORT_TILE * SORT_TILE + 1) * sizeof(uint64_t);
}

struct GradLayout {
    size_t keys, other, arrived, partials, total;
};
GradLayout grad_layout(int64_t tokens, int64_t dim) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t pieces = (size_t)pieces_of(tokens, piece_log_of(tokens, dim));
    GradLayout l{};
    l.other = up(key_bytes(tokens));
    l.arrived = l.other + up(key_bytes(tokens));
    l.partials = l.arrived + up(pieces * (size_t)(panels_of(dim) + 1) * COUNTERS * sizeof(int));
    l.total = l.partials + up(pieces * 2 * (size_t)padded(dim) * sizeof(float));
    return l;
}

}  // namespace

cudaError_t launch_embedding(spmm_type_t type, const EmbedParams& p, int num_sms,
                             cudaStream_t st) {
    const bool whole = p.dim * lm_elem_size(type) % 16 == 0 &&
                       rows_aligned16(p.out, p.ld_out, lm_elem_size(type)) &&
                       (p.vocab == 0 || rows_aligned16(p.table, p.ld_table, lm_elem_size(type)));
    return with_type(type,
                     [&](auto t) { return launch_embed<decltype(t)>(p, whole, num_sms, st); });
}

size_t embed_grad_scratch(int64_t tokens, int64_t dim) { return grad_layout(tokens, dim).total; }

// Pieces get longer as the work grows, so a smaller call may need more: what
// covers every call.  pieces <= min(tokens, SUM_WARPS / panels + 1), or
// tokens / PIECE_MAX + 1 once the pieces are longest; padded(dim) <= PANEL * panels + 8.
size_t embed_grad_scratch_upto(int64_t tokens, int64_t dim) {
    const size_t wide = (size_t)padded(dim), most = (size_t)tokens / PIECE_MAX + 1;
    const size_t rows = std::max(
        std::min((size_t)tokens * wide, (size_t)SUM_WARPS * (PANEL + 8) + wide), most * wide);
    const size_t panels = (size_t)panels_of(dim) + 1;
    const size_t counters = std::max(2 * (size_t)SUM_WARPS + panels, most * panels);
    return 2 * key_bytes(tokens) + counters * COUNTERS * sizeof(int) +
           rows * 2 * sizeof(float) + 4 * 256;
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
    k.piece_log = piece_log_of(p.tokens, p.dim);
    k.pieces = (int)pieces_of(p.tokens, k.piece_log);
    const int W = 16 / lm_elem_size(type);
    const bool whole = p.dim % W == 0 &&
                       rows_aligned16(p.dtable, p.ld_dtable, lm_elem_size(grad_type)) &&
                       (p.tokens == 0 || rows_aligned16(p.dout, p.ld_dout, lm_elem_size(type)));
    // a row between boundaries covers up to W - 1 columns more
    k.panels = (int)panels_of(p.dim + (whole ? 0 : W - 1));
    k.sum_items = (int64_t)k.pieces * k.panels;
    // a filling warp writes about 32 KB when no row of its share has a token
    const int64_t row_bytes = p.dim * lm_elem_size(grad_type);
    k.fill_rows = (int)std::min<int64_t>(32, std::max<int64_t>(1, 32768 / row_bytes));
    const int64_t fill_items =
        p.beta == 1.0f ? 0 : (p.vocab + k.fill_rows - 1) / k.fill_rows;
    if (p.tokens > 0) {
        const int tiles = (int)((p.tokens + SORT_TILE - 1) / SORT_TILE);
        cudaError_t e = launch(sort_tiles, tiles, SORT_TILE, 0, st, p.ids, (int)p.tokens, p.vocab,
                               keys, k.arrived, k.sum_items * COUNTERS);
        const unsigned total = (unsigned)tiles * SORT_TILE;
        for (int64_t run = SORT_TILE; e == cudaSuccess && run < total;) {
            const int64_t runs = (total + run - 1) / run;
            const int ways = runs <= 4 || total > MERGE_MANY ? 4 : runs <= 8 ? 8 : MERGE_WAYS;
            auto kernel = ways == 4 ? merge_runs<4> : ways == 8 ? merge_runs<8> : merge_runs<16>;
            e = launch_chained(kernel, dim3(total / 32), dim3(32 * ways), 0, st, true,
                               (const uint64_t*)keys, other, total, (unsigned)run);
            std::swap(keys, other);
            run *= ways;
        }
        if (e != cudaSuccess) return e;
    }
    k.keys = keys;
    const int64_t blocks = (k.sum_items + fill_items + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    const bool same = type == grad_type;
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        auto run = [&](auto kernel) {
            return launch_chained(kernel, dim3((unsigned)blocks), dim3(256), 0, st, p.tokens > 0,
                                  p, k);
        };
        if (same) return whole ? run(grad_sums<T, T, false>) : run(grad_sums<T, T, true>);
        return whole ? run(grad_sums<T, float, false>) : run(grad_sums<T, float, true>);
    });
}

}  // namespace spmm
