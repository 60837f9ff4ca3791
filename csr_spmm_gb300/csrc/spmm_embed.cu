// Embedding lookup out[t, :] = scale * table[ids[t], :] and its gradient
// dtable[v, :] = beta * dtable[v, :] + scale * sum_{t: ids[t] = v} dout[t, :].
//
// The gradient is the product of the transposed one-entry-per-row matrix with
// dout.  Its row structure is made on the device by sorting the tokens by id:
// keys (id << 32 | position) are unique, so any correct sort of them is the
// stable order, and the sums below have a fixed order.
#include <algorithm>

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
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = valid[u] ? p.scale * to_f32(v[u].v[i]) : 0.0f;
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

constexpr int SORT_TILE = 4096;      // keys sorted by one block in shared memory
constexpr int SORT_THREADS = 1024;
constexpr int MERGE_WAYS = 16;       // sorted runs merged per round
constexpr unsigned NO_ID = 0xffffffffu;

// Sorts each tile of SORT_TILE tokens: a bitonic network on the 64-bit keys
// in shared memory.  Ids outside [0, vocab) get the largest key and end up
// behind every row.  Pairs at distance <= 32 stay within one warp's 64 keys,
// so those steps need no block barrier.
__global__ __launch_bounds__(SORT_THREADS) void sort_tiles(const int* ids, int tokens,
                                                           int64_t vocab, uint64_t* keys) {
    __shared__ uint64_t s[SORT_TILE];
    const int t0 = blockIdx.x * SORT_TILE;
    const int n = min(SORT_TILE, tokens - t0);
    int np = 64;
    while (np < n) np <<= 1;
    for (int i = threadIdx.x; i < np; i += SORT_THREADS) {
        uint64_t key = ~0ull;
        if (i < n) {
            const int id = ids[t0 + i];
            key = (uint64_t)(id >= 0 && id < vocab ? (unsigned)id : NO_ID) << 32 |
                  (unsigned)(t0 + i);
        }
        s[i] = key;
    }
    bool wide = true;                // the last step crossed warps
    for (int k = 2; k <= np; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            if (wide || j > 32) __syncthreads();
            else __syncwarp();
            wide = j > 32;
            for (int i = threadIdx.x; i < np / 2; i += SORT_THREADS) {
                const int a = 2 * i - (i & (j - 1));
                const int b = a + j;
                const uint64_t x = s[a], y = s[b];
                if ((x > y) == ((a & k) == 0)) {
                    s[a] = y;
                    s[b] = x;
                }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += SORT_THREADS) keys[t0 + i] = s[i];
}

// Number of keys below `key` in a[0..n), by halving steps of a fixed count.
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

// Merges groups of MERGE_WAYS sorted runs of `run` keys: each key's place is
// its own index plus the count of smaller keys in the other runs.
__global__ __launch_bounds__(256) void merge_runs(const uint64_t* in, uint64_t* out, int tokens,
                                                  int64_t run) {
    const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (g >= tokens) return;
    const uint64_t key = in[g];
    const int64_t own = g / run;
    const int64_t first = own / MERGE_WAYS * MERGE_WAYS;
    int64_t place = first * run + (g - own * run);
    for (int64_t q = first; q < first + MERGE_WAYS; ++q) {
        const int64_t start = q * run;
        if (start >= tokens) break;
        if (q != own)
            place += count_below(in + start, (int)min(run, tokens - start), key);
    }
    out[place] = key;
}

// ---- gradient: sums --------------------------------------------------------------

// One warp per table row.
template <typename T, typename G>
__global__ __launch_bounds__(256) void grad_rows(EmbedGradParams p, const uint64_t* keys) {
    const int lane = threadIdx.x & 31;
    const T* dout = static_cast<const T*>(p.dout);
    G* dtable = static_cast<G*>(p.dtable);
    const int64_t warps = (int64_t)gridDim.x * 8;
    for (int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); v < p.vocab; v += warps) {
        const int a = count_below(keys, (int)p.tokens, (uint64_t)v << 32);
        const int b = count_below(keys, (int)p.tokens, (uint64_t)(v + 1) << 32);
        if (a == b && p.beta == 1.0f) continue;
        for (int64_t c = lane; c < p.dim; c += 32) {
            float sum = 0.0f;
            for (int i = a; i < b; ++i)
                sum += to_f32(dout[(int64_t)(unsigned)keys[i] * p.ld_dout + c]);
            sum *= p.scale;
            G* at = dtable + v * p.ld_dtable + c;
            if (p.beta != 0.0f) sum += p.beta * to_f32(*at);
            *at = from_f32<G>(sum);
        }
    }
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

size_t embed_grad_scratch(int64_t tokens, int64_t dim) {
    (void)dim;
    return (size_t)tokens * 16;
}

cudaError_t launch_embedding_grad(spmm_type_t type, spmm_type_t grad_type,
                                  const EmbedGradParams& p, char* scratch, int num_sms,
                                  cudaStream_t st) {
    uint64_t* keys = reinterpret_cast<uint64_t*>(scratch);
    uint64_t* other = keys + p.tokens;
    if (p.tokens > 0) {
        const int tiles = (int)((p.tokens + SORT_TILE - 1) / SORT_TILE);
        sort_tiles<<<tiles, SORT_THREADS, 0, st>>>(p.ids, (int)p.tokens, p.vocab, keys);
        for (int64_t run = SORT_TILE; run < p.tokens; run *= MERGE_WAYS) {
            merge_runs<<<(unsigned)((p.tokens + 255) / 256), 256, 0, st>>>(keys, other,
                                                                         (int)p.tokens, run);
            std::swap(keys, other);
        }
    }
    const unsigned blocks = (unsigned)std::min<int64_t>((p.vocab + 7) / 8, num_sms * 8);
    const bool same = type == grad_type;
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        if (same) grad_rows<T, T><<<blocks, 256, 0, st>>>(p, keys);
        else grad_rows<T, float><<<blocks, 256, 0, st>>>(p, keys);
        return cudaGetLastError();
    });
}

}  // namespace spmm
