// Layer norm y = (x - mean) * rstd * weight + bias over the rows of a matrix,
// and its gradients with respect to x, weight and bias.
//
// Mean and deviations are binary32 sums.  A warp sums the differences d of its n_w elements to a
// number b, and their squares, in one pass.  b is an element of its own; where their mean turns
// out to be over 4 of their deviations from it, so that the squares would lose digits, they
// are taken again from b + sum d / n_w.  With q an element of the row, e_w = b - q + sum d / n_w
// and e = sum n_w e_w / n,
//   mean = q + e
//   sum (x - mean)^2 = sum_w [sum d^2 - (sum d)^2 / n_w + n_w (e_w - e)^2]
// so no digits are lost to a mean far from zero, and a row that hardly varies has the mean that
// it would have near zero, rounded once.  (A mean summed from the elements as they are gave
// a row of 7 times 1000 deviations of 6e-5, and y = -0.02 instead of 0.)
//
// The kernels read rows in aligned accesses wherever a row starts:
// accesses are counted from the 16-byte boundary at or before the row's start, and
// elements outside the row are left out.  A thread's rows lie a fixed stride apart
// that keeps them at the same distance from such a boundary, so its columns,
// and what it holds for them in registers, are the same for all of its rows.
#include <algorithm>

#include "spmm_internal.h"
#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

constexpr unsigned ALL = 0xffffffffu;

// ---- shared pieces ----------------------------------------------------------------

// How a row lies on threads: `warps` warps of 32 lanes, or `lanes` < 32 lanes of one warp.
struct Layout {
    int lanes;
    int warps;
    int rows;                // rows of a block
    int threads() const { return lanes * warps; }
};

__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    if (lanes == 32) return warp_sum(x);
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(ALL, x, o);
    return x;
}
// Two of them at once: the exchanges of one wait beside the other's.
__device__ __forceinline__ void lanes_sum(float& x, float& y, int lanes) {
    if (lanes == 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x += __shfl_xor_sync(ALL, x, o);
            y += __shfl_xor_sync(ALL, y, o);
        }
    } else {
        for (int o = lanes >> 1; o > 0; o >>= 1) {
            x += __shfl_xor_sync(ALL, x, o);
            y += __shfl_xor_sync(ALL, y, o);
        }
    }
}
// Barrier of one row's warps (barrier 0 is the block's own).
__device__ __forceinline__ void row_barrier(int row, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "r"(threads) : "memory");
}

// Parameters of columns [c, c + W), `none` where there are none.
template <typename P, int W>
__device__ __forceinline__ Vec<P, W> load_params(const void* p, int c, int dim, float none) {
    if (!p) {
        Vec<P, W> r;
        if constexpr (W == 1) {
            r.w = from_f32<P>(none);
        } else {
            const float f[2] = {none, none};
#pragma unroll
            for (int i = 0; i < Vec<P, W>::WORDS; ++i) {
                if constexpr (sizeof(P) == 4) r.w[i] = __float_as_uint(none);
                else r.w[i] = pack_word(f, P{});
            }
        }
        return r;
    }
    const P* from = static_cast<const P*>(p);
    if (W > 1 && c >= 0 && c + W <= dim && reinterpret_cast<uintptr_t>(from + c) % 16 == 0)
        return load_vec<Cache::KEEP, P, W>(from + c);
    return load_some<P, W>(from, c, dim);
}

// The same, whole and aligned.
template <typename P, int W>
__device__ __forceinline__ void vec_params(const void* p, int c, float none, float (&f)[W]) {
    if (p) {
        unpack(load_vec<Cache::KEEP, P, W>(static_cast<const P*>(p) + c), f);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = none;
    }
}

// A matrix's rows read in aligned accesses: one that reaches over the row's ends is
// still a whole one where memory of the matrix lies there (another row, or the gap
// between two), and is taken element by element at the matrix's own ends.
template <typename T, int W>
struct Rows {
    const T* base;
    int64_t ld;
    const T* end;            // of the matrix
    int dim;
    __device__ Rows(const void* p, int64_t ld, int64_t rows, int64_t dim)
        : base(static_cast<const T*>(p)), ld(ld), end(base + (rows - 1) * ld + dim), dim((int)dim) {}
    __device__ const T* row(int64_t r) const { return base + r * ld; }
    // whether an access to row r may reach over the matrix's ends
    __device__ bool at_ends(int64_t r, int64_t rows) const { return r < W || r >= rows - W; }
    __device__ bool inside(const T* row, int c) const {
        return (c >= 0 && c + W <= dim) || (row + c >= base && row + c + W <= end);
    }
    __device__ Vec<T, W> load(const T* row, int c) const {
        return inside(row, c) ? load_vec<Cache::STREAM, T, W>(row + c) : load_some<T, W>(row, c, dim);
    }
    __device__ void copy(Vec<T, W>* to, const T* row, int c) const {
        if (inside(row, c)) copy_async<T, W>(to, row + c);
        else *to = load_some<T, W>(row, c, dim);
    }
};
// The bits of an access's elements that belong to the row.
template <typename T, int W>
__device__ __forceinline__ Vec<T, W> mask_of(int c, int dim) {
    Vec<T, W> r;
#pragma unroll
    for (int i = 0; i < Vec<T, W>::WORDS; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (c + i >= 0 && c + i < dim) {
            if constexpr (sizeof(T) == 4) r.w[i] = 0xffffffffu;
            else r.w[i / 2] |= 0xffffu << ((i & 1) * 16);
        }
    return r;
}
template <typename T, int W>
__device__ __forceinline__ Vec<T, W> masked(Vec<T, W> v, uint32_t all) {
#pragma unroll
    for (int i = 0; i < Vec<T, W>::WORDS; ++i) v.w[i] &= all;
    return v;
}
template <typename T, int W>
__device__ __forceinline__ Vec<T, W> masked(Vec<T, W> v, const Vec<T, W>& mask, uint32_t all) {
#pragma unroll
    for (int i = 0; i < Vec<T, W>::WORDS; ++i) v.w[i] &= mask.w[i] & all;
    return v;
}
template <int W>
__device__ __forceinline__ void clear_outside(int c, int dim, float (&f)[W]) {
    if (c >= 0 && c + W <= dim) return;
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (c + i < 0 || c + i >= dim) f[i] = 0.0f;
}
// ---- forward ------------------------------------------------------------------------

// How a row meets its threads' accesses: ALL: every lane's are whole and in the row, and
// there are a weight and a bias; WHOLE: whole, some lanes have fewer; EDGES: any width,
// any start.
enum class Fit { ALL, WHOLE, EDGES };

// A row in registers, K accesses of W elements per lane: read once, one exchange
// between its warps.  The bound is HBM (read x, write y) as long as an element costs
// few instructions: 65,521 f16 rows of 8192 took 476 us at 27 per element and take 363 at 17,
// two elements at a time and, but for the second look, without a branch (5.9 TB/s, 87% of the
// copy rate; 40,000 binary32 rows of 2048: 101 us, 95%; 60,000 x 2001 bf16 110 us, 64%).  A
// second look at one of the eight warps' parts of every row (an outlier at its first element)
// makes 424 us of 367 (calls back to back).  Rows with edges walk the matrix with a
// fixed grid and keep the parameters in shared memory in binary32, (weight, bias)
// of column c at [c mod W][c / W]: wherever a row starts, a warp reads neighbours.
// The others have a block of threads each and read the parameters from L1.  (Measured and
// dropped: a fixed grid with the next row on its way to shared memory, 386 us; 48
// registers for 1280 threads per SM, 457 us, it spills.)
template <typename T, typename P, int W, int K, Fit FIT>
__global__ __launch_bounds__(1024) void norm_rows(NormParams p, Layout l, int64_t stride,
                                                  int pitch) {
    constexpr bool EDGES = FIT == Fit::EDGES;
    __shared__ float4 slots[2][32];
    extern __shared__ __align__(16) float2 params[];     // [W][pitch]
    const int threads = l.lanes * l.warps;
    const int in_block = threadIdx.x / threads, tid = threadIdx.x % threads;
    const int lane = threadIdx.x & 31;
    const Rows<T, W> x(p.x, p.ldx, p.rows, p.dim);
    const int dim = (int)p.dim;
    const int step = threads * W;                // columns from one access to the next
    int64_t r = (int64_t)blockIdx.x * l.rows + in_block;
    int64_t first = r - lane / l.lanes;          // the warp's first row: all lanes stay together
    if constexpr (EDGES) {
        for (int c = threadIdx.x; c < dim; c += blockDim.x) {
            params[(c % W) * pitch + c / W] =
                make_float2(p.weight ? to_f32(static_cast<const P*>(p.weight)[c]) : 1.0f,
                            p.bias ? to_f32(static_cast<const P*>(p.bias)[c]) : 0.0f);
        }
        __syncthreads();
    }
    // the rows' first accesses begin `lead` columns before them; element i of access j is
    // column j W + i - lead
    const int lead = EDGES ? lead_of(x.row(r), W * (int)sizeof(T)) : 0;
    int param_at[EDGES ? W : 1];
#pragma unroll
    for (int i = 0; i < (EDGES ? W : 0); ++i) {
        const int e = i - lead + W;              // > 0
        param_at[i] = e % W * pitch + e / W - 1 + tid;
    }
    const float per_dim = 1.0f / (float)dim;
    // the warp's elements of a row
    float count = (float)(l.lanes * W * K);
    if constexpr (FIT != Fit::ALL) {
        int own = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = tid * W - lead + k * step;
            if (c < dim) own += EDGES ? min(c + W, dim) - max(c, 0) : W;
        }
        count = lanes_sum((float)own, l.lanes);
    }
    const float per_count = count > 0.0f ? __fdividef(1.0f, count) : 0.0f;
    int turn = 0;
    for (; first < p.rows; first += stride, r += stride) {
        const T* row = x.row(r);
        const int c0 = tid * W - lead;
        const bool live = FIT == Fit::ALL || r < p.rows;
        Vec<T, W> held[K];
        auto in = [&](int k) { return FIT == Fit::ALL || (live && c0 + k * step < dim); };
        if (EDGES && x.at_ends(r, p.rows)) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in(k)) held[k] = x.load(row, c0 + k * step);   // at_ends: !live too
        } else {
            // past the row its last access is read in vain: one behind a branch would keep
            // the others waiting
            const T* from = live ? row : x.base;
            const int last = (dim - 1 + lead) / W * W - lead;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = c0 + k * step;
                held[k] = load_vec<Cache::STREAM, T, W>(from + (FIT == Fit::ALL ? c : min(c, last)));
            }
        }
        // what is not in the row counts as 0
        if constexpr (FIT == Fit::WHOLE)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < Vec<T, W>::WORDS; ++i) held[k].w[i] = in(k) ? held[k].w[i] : 0;
        // b and q, 0 where they are infinite or NaN.  q is the middle one of three, so that a few
        // columns of large values do not put it far from the mean, whose rounding would be that
        // of the distance; b too in rows with edges, where a second look costs more (with a
        // first column far from the others 60,000 x 2001 bf16 would take 181 us), but not in the
        // others, whose lanes would have to ask twice more (65,521 x 8192 f16 377 us).
        auto finite = [](float v) { return fabsf(v) < INFINITY ? v : 0.0f; };
        auto middle = [&](const T* of) {
            const float u = to_f32(of[0]), v = to_f32(of[dim / 2]), w = to_f32(of[dim - 1]);
            return finite(fmaxf(fminf(u, v), fminf(fmaxf(u, v), w)));
        };
        float base, pivot;
        if constexpr (EDGES) {
            base = pivot = middle(live ? row : x.base);
        } else {
            float f[W];
            unpack(held[0], f);
            base = pivot = finite(__shfl_sync(ALL, f[0], lane & ~(l.lanes - 1)));
            if (l.warps > 1) pivot = middle(row);
        }
        uint64_t d1 = pair(0.0f, 0.0f), d2 = d1;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (EDGES && !in(k)) continue;
            float f[W];
            unpack(held[k], f);
            const float from = FIT == Fit::ALL || in(k) ? base : 0.0f;
            if (EDGES) {
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] -= base;
                clear_outside(c0 + k * step, dim, f);
            }
            const uint64_t k2 = pair(-from, -from);
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                uint64_t d = pair(f[i], f[i + 1]);
                if (!EDGES) d = add2(d, k2);
                d1 = add2(d1, d);
                d2 = fma2(d, d, d2);
            }
        }
        float deviations, squares, lo, hi;
        halves(d1, lo, hi);
        deviations = lo + hi;
        halves(d2, lo, hi);
        squares = lo + hi;
        lanes_sum(deviations, squares, l.lanes);
        float off = deviations * per_count;
        const bool far = deviations * off > 0.94f * squares;
        if (__any_sync(ALL, far)) {
            // From memory again (y, which may be x, is written behind the exchange below, or by
            // these lanes): a second use of `held` here would cost every row registers.
            const float better = base + off;
            float again = 0.0f, squares_again = 0.0f;
#pragma unroll 1
            for (int k = 0; k < K; ++k) {
                const int c = c0 + k * step;
                if (!in(k)) continue;
                auto add = [&](float v) {
                    again += v - better;
                    squares_again = fmaf(v - better, v - better, squares_again);
                };
                if constexpr (EDGES) {
#pragma unroll 1
                    for (int e = max(c, 0); e < min(c + W, dim); ++e) add(to_f32(row[e]));
                } else {
                    float f[W];
                    unpack(load_vec<Cache::KEEP, T, W>(row + c), f);
#pragma unroll
                    for (int i = 0; i < W; ++i) add(f[i]);
                }
            }
            lanes_sum(again, squares_again, l.lanes);
            if (far) {
                base = better;
                if (l.warps == 1) pivot = better;
                deviations = again;
                off = again * per_count;
                squares = squares_again;
            }
        }
        // what is left is at least 6% of them; squares beyond binary32 stay so (rstd 0), unless there
        // is an infinite element (NaN)
        squares = fmaf(squares < INFINITY ? -deviations : 0.0f, off, squares);
        off += base - pivot;
        if (l.warps > 1) {
            // two sets of slots in turn: one barrier per row keeps them apart
            float4* s = slots[turn] + in_block * l.warps;
            turn ^= 1;
            if (lane == 0) s[tid >> 5] = make_float4(off * count, off, squares, count);
            row_barrier(in_block, threads);
            if (l.warps >= 8) {
                // a lane for each warp's part: 10 shuffles instead of 7 instructions for each
                // (18,000 x 16,384 bf16, 16 warps: 230 us, 254 with the loop below)
                const float4 v = lane < l.warps ? s[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                off = warp_sum(v.x) * per_dim;
                squares = warp_sum(fmaf(v.w * (v.y - off), v.y - off, v.z));
            } else {
                off = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < l.warps) off += s[i].x;
                off *= per_dim;
                squares = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < l.warps) squares += s[i].z + s[i].w * (s[i].y - off) * (s[i].y - off);
            }
        }
        if (!live) continue;                     // narrow rows: a warp holds several
        const float mean = pivot + off;
        const float rstd = rsqrtf(squares * per_dim + p.eps);
        T* y = static_cast<T*>(p.y) + r * p.ldy;
        const uint64_t r2 = pair(rstd, rstd), m2 = pair(-mean, -mean);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = c0 + k * step;
            if (!in(k)) continue;
            float f[W], w[W], b[W];
            unpack(held[k], f);
            if constexpr (EDGES) {
                // outside the row whatever lies there
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float2 wb = params[param_at[i] + k * threads];
                    w[i] = wb.x;
                    b[i] = wb.y;
                }
            } else if constexpr (FIT == Fit::ALL) {
                unpack(load_vec<Cache::KEEP, P, W>(static_cast<const P*>(p.weight) + c), w);
                unpack(load_vec<Cache::KEEP, P, W>(static_cast<const P*>(p.bias) + c), b);
            } else {
                vec_params<P, W>(p.weight, c, 1.0f, w);
                vec_params<P, W>(p.bias, c, 0.0f, b);
            }
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                const uint64_t d = mul2(add2(pair(f[i], f[i + 1]), m2), r2);
                halves(fma2(d, pair(w[i], w[i + 1]), pair(b[i], b[i + 1])), f[i], f[i + 1]);
            }
            if (EDGES) store_some<T, W>(y, c, dim, f);
            else store_vec<Cache::STREAM, T, W>(y + c, f);
        }
        if (tid == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

constexpr int ANY_THREADS = 256;

// Sum over the block (every thread gets it); `s` holds one float per warp.
__device__ __forceinline__ float block_sum(float x, float* s) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < ANY_THREADS / 32; ++i) t += s[i];
    return t;
}
template <typename P>
__device__ __forceinline__ float param(const void* p, int64_t i, float none) {
    return p ? to_f32(static_cast<const P*>(p)[i]) : none;
}

// Rows too wide for registers, or x and y that lie differently against 16-byte
// boundaries: a block per row, element by element, the row read again for each pass.
template <typename T, typename P>
__global__ __launch_bounds__(ANY_THREADS) void norm_any(NormParams p) {
    __shared__ float s[ANY_THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        T* y = static_cast<T*>(p.y) + r * p.ldy;
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < p.dim; c += ANY_THREADS) sum += to_f32(x[c]);
        float mean = block_sum(sum, s) / (float)p.dim;
        auto variance = [&] {
            float squares = 0.0f;
            for (int64_t c = threadIdx.x; c < p.dim; c += ANY_THREADS) {
                const float d = to_f32(x[c]) - mean;
                squares += d * d;
            }
            return block_sum(squares, s) / (float)p.dim;
        };
        float var = variance();
        if (var <= mean * mean * 0x1p-10f && mean != 0.0f) {
            // a row that hardly varies would show the mean's rounding: the mean of the
            // deviations corrects it
            sum = 0.0f;
            for (int64_t c = threadIdx.x; c < p.dim; c += ANY_THREADS) sum += to_f32(x[c]) - mean;
            mean += block_sum(sum, s) / (float)p.dim;
            var = variance();
        }
        const float rstd = rsqrtf(var + p.eps);
        for (int64_t c = threadIdx.x; c < p.dim; c += ANY_THREADS)
            y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * param<P>(p.weight, c, 1.0f) +
                               param<P>(p.bias, c, 0.0f));
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// ---- gradient -----------------------------------------------------------------------

constexpr int GRAD_THREADS = 512;    // a row's threads, at most; up to 128 registers each
constexpr int GRAD_COLUMNS = GRAD_THREADS * 16;
// Stages of the ring: what GRAD_THREADS threads can have of the 227 KB, four at most.
template <typename T>
constexpr int GRAD_STAGES = sizeof(T) == 4 ? 3 : 4;

// Elements outside the row are masked (EDGES: bit by bit; WHOLE: an access at a time), not
// branched around: a branch per access kept the others waiting
// (32,768 x 4096 bf16 with branches: 219 us).
//
// dx, and this group's share of dweight and dbias, in one pass over dy and x: a row's
// threads walk the rows with a fixed stride, the rows ahead on their way to shared
// memory (each lane's accesses in slots of its own), and keep their columns' sums of
// dy * xhat and dy in registers to the end.  GIVEN: rows of more than GRAD_COLUMNS
// columns, in tiles of as many (blockIdx.y); the row's two means come from
// grad_means and nothing is exchanged.  The bound is HBM (read dy and x, write dx):
// 32,768 rows of 4096 bf16 138 us with the join, 5.8 TB/s (86% of the copy rate), 30,000
// binary32 rows of 4096 239 us (91%).  128 registers hold the sums, which leaves 16 warps
// per SM; 64 or 80 registers spill and take 220 us or more.
// part: [slices, or blocks of narrow rows][2][dim].
template <typename T, typename P, int W, int K, Fit FIT, bool GIVEN>
__global__ __launch_bounds__(GRAD_THREADS) void norm_grad_rows(NormGradParams p, Layout l,
                                                               int slices) {
    constexpr int STAGES = GRAD_STAGES<T>;
    constexpr bool EDGES = FIT == Fit::EDGES;
    __shared__ float2 slots[2][32];
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    Vec<T, W>* ring = reinterpret_cast<Vec<T, W>*>(ring_bytes) + threadIdx.x;
    const int threads = l.lanes * l.warps;
    const int in_block = threadIdx.x / threads, tid = threadIdx.x % threads;
    const int lane = threadIdx.x & 31;
    const Rows<T, W> x(p.x, p.ldx, p.rows, p.dim), dy(p.dy, p.ld_dy, p.rows, p.dim);
    const int dim = (int)p.dim;
    const int slice = blockIdx.x * l.rows + in_block;
    int64_t r = slice, first = r - lane / l.lanes;
    // the tile's accesses follow the ones of the tiles before, so none is in two tiles
    const int c0 = tid * W - (EDGES ? lead_of(x.row(r), W * (int)sizeof(T)) : 0) +
                   (GIVEN ? (int)blockIdx.y * GRAD_COLUMNS : 0);
    const int step = threads * W;
    auto in = [&](int k) { return FIT == Fit::ALL || c0 + k * step < dim; };
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.rows) {
            const T* xr = x.row(row);
            const T* dyr = dy.row(row);
            Vec<T, W>* to = ring + stage * 2 * K * blockDim.x;
            if (EDGES && x.at_ends(row, p.rows)) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!in(k)) continue;
                    x.copy(to + k * blockDim.x, xr, c0 + k * step);
                    dy.copy(to + (K + k) * blockDim.x, dyr, c0 + k * step);
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!in(k)) continue;
                    copy_async<T, W>(to + k * blockDim.x, xr + c0 + k * step);
                    copy_async<T, W>(to + (K + k) * blockDim.x, dyr + c0 + k * step);
                }
            }
        }
        copies_issued();
    };
    // the masks follow the ring
    Vec<T, W>* mask = ring + STAGES * 2 * K * blockDim.x;
    if (EDGES)
#pragma unroll
        for (int k = 0; k < K; ++k) mask[k * blockDim.x] = mask_of<T, W>(c0 + k * step, dim);
    // slices beyond the grid's last row group have no rows (slice >= slices)
    const int64_t rows = slice - lane / l.lanes < slices ? p.rows : 0;
    if (rows > 0)
        for (int i = 0; i < STAGES - 1; ++i) fetch(r + (int64_t)i * slices, i);
    Vec<P, W> w[K];
    uint64_t dw[K][W / 2], db[K][W / 2];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) dw[k][i] = db[k][i] = pair(0.0f, 0.0f);
        w[k] = load_params<P, W>(p.weight, c0 + k * step, dim, 1.0f);
    }
    const float per_dim = 1.0f / (float)dim;
    int turn = 0, stage = 0;
    // the next row's statistics are on their way during this one's sums
    float next_mean = 0.0f, next_rstd = 0.0f;
    float2 next_ab{};
    auto statistics = [&](int64_t row) {
        if (row >= rows || slice >= slices) return;
        next_mean = p.mean[row];
        next_rstd = p.rstd[row];
        if (GIVEN) next_ab = reinterpret_cast<const float2*>(p.means)[row];
    };
    statistics(r);
    for (; first < rows; first += slices, r += slices) {
        const bool live = FIT == Fit::ALL || (r < rows && slice < slices);
        const float mean = next_mean, rstd = next_rstd;
        const float2 ab = next_ab;
        statistics(r + slices);
        copies_wait<STAGES - 2>();
        uint64_t a2 = pair(0.0f, 0.0f), b2 = a2;
        const uint64_t m2 = pair(-mean, -mean), r2 = pair(rstd, rstd);
        // xhat, dy and dy * weight of access k.  Rows with edges take them from the ring for
        // each of two passes: beside the masks there is no room to keep them.
        auto take = [&](int k, uint64_t (&xh)[W / 2], uint64_t (&d)[W / 2], uint64_t (&g)[W / 2]) {
            float xf[W], gf[W], wf[W];
            const Vec<T, W>* from = ring + (stage * 2 * K + k) * blockDim.x;
            if constexpr (EDGES) {
                const uint32_t all = live ? ~0u : 0u;
                unpack(masked(*from, mask[k * blockDim.x], all), xf);
                unpack(masked(from[K * blockDim.x], mask[k * blockDim.x], all), gf);
            } else if constexpr (FIT == Fit::WHOLE) {
                const uint32_t all = live && in(k) ? ~0u : 0u;
                unpack(masked(*from, all), xf);
                unpack(masked(from[K * blockDim.x], all), gf);
            } else {
                unpack(*from, xf);
                unpack(from[K * blockDim.x], gf);
            }
            unpack(w[k], wf);
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                d[i] = pair(gf[2 * i], gf[2 * i + 1]);
                xh[i] = mul2(add2(pair(xf[2 * i], xf[2 * i + 1]), m2), r2);
                g[i] = mul2(d[i], pair(wf[2 * i], wf[2 * i + 1]));
            }
        };
        uint64_t kept[EDGES ? 1 : 2][EDGES ? 1 : K][W / 2];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint64_t xh[W / 2], d[W / 2], g[W / 2];
            take(k, xh, d, g);
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                if constexpr (!EDGES) {
                    kept[0][k][i] = xh[i];
                    kept[1][k][i] = g[i];
                }
                dw[k][i] = fma2(d[i], xh[i], dw[k][i]);
                db[k][i] = add2(db[k][i], d[i]);
                if (!GIVEN) {
                    a2 = add2(a2, g[i]);
                    b2 = fma2(g[i], xh[i], b2);
                }
            }
        }
        // to the stage of the row before
        fetch(r + (int64_t)(STAGES - 1) * slices, stage == 0 ? STAGES - 1 : stage - 1);
        float a, b;
        if constexpr (GIVEN) {
            a = ab.x;
            b = ab.y;
        } else {
            float lo, hi;
            halves(a2, lo, hi);
            a = lo + hi;
            halves(b2, lo, hi);
            b = lo + hi;
            lanes_sum(a, b, FIT == Fit::ALL ? 32 : l.lanes);
            if (l.warps > 1) {
                // two sets of slots in turn: one barrier per row keeps them apart
                float2* s = slots[turn] + in_block * l.warps;
                turn ^= 1;
                if (lane == 0) s[tid >> 5] = make_float2(a, b);
                row_barrier(in_block, threads);
                a = b = 0.0f;
#pragma unroll 8
                for (int i = 0; i < l.warps; ++i) {
                    a += s[i].x;
                    b += s[i].y;
                }
            }
            a *= per_dim;
            b *= per_dim;
        }
        T* dx = static_cast<T*>(p.dx) + r * p.ld_dx;
        const uint64_t na = pair(-a, -a), nb = pair(-b, -b);
        if (live)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = c0 + k * step;
                uint64_t xh[W / 2], d[W / 2], g[W / 2];
                if constexpr (EDGES) {
                    take(k, xh, d, g);
                } else {
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        xh[i] = kept[0][k][i];
                        g[i] = kept[1][k][i];
                    }
                }
                if (!in(k)) continue;
                float f[W];
#pragma unroll
                for (int i = 0; i < W / 2; ++i)
                    halves(mul2(r2, fma2(nb, xh[i], add2(g[i], na))), f[2 * i], f[2 * i + 1]);
                if (EDGES) store_some<T, W>(dx, c, dim, f);
                else store_vec<Cache::STREAM, T, W>(dx + c, f);
            }
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    allow_successor();
    if (!p.part) return;
    // one part per row group; narrow rows, many to a block, are first added up there: over
    // the warp's lanes where they have the same columns, then one after the other in
    // shared memory
    const bool narrow = l.lanes < 32;
    bool mine = slice < slices;
    if (narrow && __all_sync(ALL, c0 == (lane & (l.lanes - 1)) * W)) {
        for (int o = l.lanes; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    dw[k][i] = add2(dw[k][i], __shfl_xor_sync(ALL, dw[k][i], o));
                    db[k][i] = add2(db[k][i], __shfl_xor_sync(ALL, db[k][i], o));
                }
        mine = lane < l.lanes;
    }
    float* part = p.part + (int64_t)(narrow ? blockIdx.x : slice) * 2 * p.dim;
    if (narrow) {
        copies_wait<0>();
        __syncthreads();
        part = reinterpret_cast<float*>(ring_bytes);
        for (int i = threadIdx.x; i < 2 * dim; i += blockDim.x) part[i] = 0.0f;
    }
    for (int group = 0; group < (narrow ? l.rows : 1); ++group) {
        if (narrow) {
            if (!__syncthreads_or(group == in_block && mine)) continue;
            if (group != in_block) continue;
        }
        if (!mine) continue;
        float sums[2][K][W];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                halves(dw[k][i], sums[0][k][2 * i], sums[0][k][2 * i + 1]);
                halves(db[k][i], sums[1][k][2 * i], sums[1][k][2 * i + 1]);
            }
        if (narrow)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const int c = c0 + k * step + i;
                    if (c < 0 || c >= dim) continue;
                    sums[0][k][i] += part[c];
                    sums[1][k][i] += part[dim + c];
                }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int c = c0 + k * step + i;
                if (c < 0 || c >= dim) continue;
                part[c] = sums[0][k][i];
                part[dim + c] = sums[1][k][i];
            }
    }
    if (narrow) {
        __syncthreads();
        float* to = p.part + (int64_t)blockIdx.x * 2 * p.dim;
        for (int i = threadIdx.x; i < 2 * dim; i += blockDim.x) to[i] = part[i];
    }
}

// The two means of each row: a block per row.  W == 1 where x and dy lie differently
// against 16-byte boundaries.  Wide rows read dy and x twice so: 18,000 of 16,384 bf16
// take 482 us, 5 passes over memory where 3 are needed (261 us).
template <typename T, typename P, int W>
__global__ __launch_bounds__(ANY_THREADS) void grad_means(NormGradParams p) {
    __shared__ float s[ANY_THREADS / 32];
    const Rows<T, W> x(p.x, p.ldx, p.rows, p.dim), dy(p.dy, p.ld_dy, p.rows, p.dim);
    const int dim = (int)p.dim;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* xr = x.row(r);
        const T* dyr = dy.row(r);
        const int lead = W > 1 ? lead_of(xr, W * (int)sizeof(T)) : 0;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float a = 0.0f, b = 0.0f;
        for (int c = threadIdx.x * W - lead; c < dim; c += 2 * ANY_THREADS * W) {
            Vec<T, W> xv[2], dyv[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = c + u * ANY_THREADS * W;
                const bool whole = at >= 0 && at + W <= dim;
                xv[u] = whole ? load_vec<Cache::KEEP, T, W>(xr + at) : load_some<T, W>(xr, at, dim);
                dyv[u] = whole ? load_vec<Cache::KEEP, T, W>(dyr + at)
                               : load_some<T, W>(dyr, at, dim);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float xf[W], gf[W], wf[W];
                unpack(xv[u], xf);
                unpack(dyv[u], gf);
                unpack(load_params<P, W>(p.weight, c + u * ANY_THREADS * W, dim, 1.0f), wf);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float g = gf[i] * wf[i];   // 0 outside the row
                    a += g;
                    b = fmaf(g, (xf[i] - mean) * rstd, b);
                }
            }
        }
        a = block_sum(a, s) / (float)dim;
        b = block_sum(b, s) / (float)dim;
        if (threadIdx.x == 0) reinterpret_cast<float2*>(p.means)[r] = make_float2(a, b);
    }
}

// Where x, dy and dx lie differently against 16-byte boundaries: element by element,
// a thread per column and slice of the rows, the row's means from grad_means.
constexpr int64_t SLICE_ROWS = 256, SLICES = 32768;      // rows at least, slices at most
int64_t slice_rows(int64_t rows) { return std::max(SLICE_ROWS, (rows + SLICES - 1) / SLICES); }
int64_t slices_any(int64_t rows) { return (rows + slice_rows(rows) - 1) / slice_rows(rows); }
template <typename T, typename P>
__global__ __launch_bounds__(ANY_THREADS) void norm_grad_any(NormGradParams p, int64_t slice) {
    const int64_t c = (int64_t)blockIdx.x * ANY_THREADS + threadIdx.x;
    if (c >= p.dim) return;
    const float w = param<P>(p.weight, c, 1.0f);
    float dw = 0.0f, db = 0.0f;
    const int64_t r0 = (int64_t)blockIdx.y * slice;
    const int64_t r1 = min(r0 + slice, p.rows);
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        const float g = to_f32(static_cast<const T*>(p.dy)[r * p.ld_dy + c]);
        const float x = to_f32(static_cast<const T*>(p.x)[r * p.ldx + c]);
        const float rstd = p.rstd[r];
        const float xhat = (x - p.mean[r]) * rstd;
        const float2 ab = reinterpret_cast<const float2*>(p.means)[r];
        dw += g * xhat;
        db += g;
        static_cast<T*>(p.dx)[r * p.ld_dx + c] =
            from_f32<T>(rstd * (g * w - ab.x - xhat * ab.y));
    }
    if (!p.part) return;
    p.part[(int64_t)blockIdx.y * 2 * p.dim + c] = dw;
    p.part[((int64_t)blockIdx.y * 2 + 1) * p.dim + c] = db;
}

// dweight and dbias from the slices' partial sums: a block takes 32 columns, each
// of its warps every JOIN_WARPS-th slice in order, then the warps' sums are added
// in order.  As many warps as a block may have: the sums are short, and what
// counts is how many loads wait together (608 slices of 4096 columns: 6 us).
constexpr int JOIN_WARPS = 32;
template <typename P>
__global__ __launch_bounds__(32 * JOIN_WARPS) void norm_dw_join(NormGradParams p, int slices) {
    __shared__ float s[JOIN_WARPS][32];
    wait_for_predecessor();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int which = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    P* out = static_cast<P*>(which ? p.dbias : p.dweight);
    if (!out) return;
    float t = 0.0f;
    if (c < p.dim) {
        const float* part = p.part + which * p.dim + c;
#pragma unroll 8
        for (int k = w; k < slices; k += JOIN_WARPS) t += part[(int64_t)k * 2 * p.dim];
    }
    s[w][lane] = t;
    __syncthreads();
    if (w > 0 || c >= p.dim) return;
#pragma unroll
    for (int i = 1; i < JOIN_WARPS; ++i) t += s[i][lane];
    out[c] = from_f32<P>(t);
}

// ---- launch -----------------------------------------------------------------------------

// The layout of rows of `columns` columns, K accesses of W elements per lane, in
// blocks of at least `least` threads.  Rows with edges take a power of two of warps
// (9635 x 1500 bf16, gradient: 38 us with 4, 48 with 3), others as many as they need
// (4071 x 2368 f16: 27 us with 5, 32 with 8).
Layout layout_of(int64_t columns, int W, int K, int least, bool whole) {
    const int64_t lanes = (columns + (int64_t)W * K - 1) / ((int64_t)W * K);
    Layout l{1, 1, 1};
    while (l.lanes < 32 && l.lanes < lanes) l.lanes *= 2;
    if (whole) l.warps = (int)std::max<int64_t>(1, (lanes + 31) / 32);
    else while ((int64_t)l.lanes * l.warps < lanes) l.warps *= 2;
    l.rows = std::max(1, least / l.threads());
    return l;
}

// A row of `dim` columns covers up to W - 1 more where it starts between boundaries.
bool off_boundary(const void* p, int64_t ld, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 != 0 || ld * (int64_t)es % 16 != 0;
}
// Each row of one at the same distance from a 16-byte boundary as in the other.
bool alike(const void* a, int64_t lda, const void* b, int64_t ldb, size_t es) {
    return (reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b)) % 16 == 0 &&
           (lda - ldb) * (int64_t)es % 16 == 0;
}
// Blocks of `rows` rows for a grid of at most `most`; a grid that does not cover the rows
// at once keeps its stride a multiple of W rows.
int64_t blocks_of(int64_t total, int rows, int64_t most, int W) {
    const int64_t blocks = (total + rows - 1) / rows;
    if (blocks <= most) return blocks;
    return rows % W == 0 ? most : std::max<int64_t>(W, most / W * W);
}

// Dynamic shared memory that needs no leave, and the most that a launch here asks for: the
// parameters of the widest row with edges, and the ring of the most threads with its masks.
constexpr size_t SHARED_FREE = 32768;
constexpr int EDGES_COLUMNS = 16384;
template <int W>
constexpr size_t NORM_SHARED = (size_t)W * (EDGES_COLUMNS / W + 3) * sizeof(float2);
template <typename T>
constexpr size_t ring_size(int threads, int K) {
    return ((size_t)GRAD_STAGES<T> * 2 + 1) * K * threads * 16;
}

template <typename T, typename P, int W, int K, bool WHOLE>
cudaError_t norm_launch(const NormParams& p, int64_t columns, int num_sms, cudaStream_t st) {
    const Layout l = layout_of(columns, W, K, 256, WHOLE);
    const int threads = l.threads() * l.rows;
    int64_t blocks = (p.rows + l.rows - 1) / l.rows;
    int pitch = 0;
    auto kernel = norm_rows<T, P, W, K, WHOLE ? Fit::WHOLE : Fit::EDGES>;
    if constexpr (!WHOLE) {
        blocks = blocks_of(p.rows, l.rows, (int64_t)num_sms * std::max(1, 1024 / threads), W);
        pitch = ((int)(p.dim / W) + 2) | 1;
    } else if (p.dim == (int64_t)l.threads() * W * K && p.rows % l.rows == 0 && p.weight &&
               p.bias) {
        kernel = norm_rows<T, P, W, K, Fit::ALL>;
    }
    const size_t shared = (size_t)W * pitch * sizeof(float2);
    if (shared > SHARED_FREE) {
        const cudaError_t e = allow_shared(kernel, NORM_SHARED<W>);
        if (e != cudaSuccess) return e;
    }
    return launch(kernel, (unsigned)blocks, threads, shared, st, p, l, blocks * l.rows, pitch);
}

// Row groups (slices) of the gradient's grid at 512 threads per SM.
int64_t slices_most(int num_sms, const Layout& l) {
    return (int64_t)num_sms * l.rows * std::max(1, GRAD_THREADS / (l.threads() * l.rows));
}

template <typename T, typename P, bool GIVEN>
cudaError_t norm_grad_launch(const NormGradParams& p, int64_t columns, int num_sms,
                             cudaStream_t st, int* parts) {
    constexpr int W = 16 / (int)sizeof(T), K = 16 / W;
    const bool whole = columns == p.dim && p.dim % W == 0;
    const Layout l = layout_of(std::min<int64_t>(columns, GRAD_COLUMNS), W, K, 128, whole);
    const int64_t blocks = blocks_of(p.rows, l.rows, slices_most(num_sms, l) / l.rows, W);
    const int slices = (int)std::min<int64_t>(p.rows, blocks * l.rows);
    *parts = l.lanes < 32 ? (int)blocks : slices;
    const int threads = l.threads() * l.rows;
    const unsigned tiles = GIVEN ? (unsigned)((columns + GRAD_COLUMNS - 1) / GRAD_COLUMNS) : 1;
    // the ring, and masks for rows with edges
    const size_t shared = ring_size<T>(threads, K);
    auto kernel = norm_grad_rows<T, P, W, K, Fit::EDGES, GIVEN>;
    if (whole && l.lanes == 32 && p.dim == (int64_t)tiles * l.threads() * W * K)
        kernel = norm_grad_rows<T, P, W, K, Fit::ALL, GIVEN>;
    else if (whole)
        kernel = norm_grad_rows<T, P, W, K, Fit::WHOLE, GIVEN>;
    if (shared > SHARED_FREE) {
        const cudaError_t e = allow_shared(kernel, ring_size<T>(GRAD_THREADS, K));
        if (e != cudaSuccess) return e;
    }
    return launch(kernel, dim3((unsigned)blocks, tiles), threads, shared, st, p, l, slices);
}

template <typename F>
cudaError_t with_types(spmm_type_t type, spmm_type_t param_type, F&& f) {
    return with_type(type, [&](auto t) {
        return type == param_type ? f(t, t) : f(t, float{});
    });
}

}  // namespace

cudaError_t launch_layer_norm(spmm_type_t type, spmm_type_t param_type, const NormParams& p,
                              int num_sms, cudaStream_t st) {
    return with_types(type, param_type, [&](auto t, auto pt) {
        using T = decltype(t);
        using P = decltype(pt);
        constexpr int W = 16 / (int)sizeof(T);
        if (alike(p.x, p.ldx, p.y, p.ldy, sizeof(T))) {
            const bool whole = !off_boundary(p.x, p.ldx, sizeof(T)) && p.dim % W == 0 &&
                               !(p.weight && reinterpret_cast<uintptr_t>(p.weight) % 16) &&
                               !(p.bias && reinterpret_cast<uintptr_t>(p.bias) % 16);
            const int64_t columns = p.dim + W - 1;
            // Few rows leave SMs idle: then the most threads per row give the shortest
            // call; many rows take 64 bytes per lane.  Beside binary32 parameters 16-bit
            // rows are read four elements at a time, so that a warp's parameters, too,
            // are read from consecutive 16-byte words.
            const bool few = p.rows <= 2 * num_sms;
            constexpr int V = sizeof(P) > sizeof(T) ? 4 : W;
            if (whole) {
                if (few && p.dim <= 1024 * V)
                    return norm_launch<T, P, V, 1, true>(p, p.dim, num_sms, st);
                if (p.dim <= 4096 * W)
                    return norm_launch<T, P, V, 4 * W / V, true>(p, p.dim, num_sms, st);
            } else {
                if (few && columns <= 1024 * W)
                    return norm_launch<T, P, W, 1, false>(p, columns, num_sms, st);
                // the parameters take 8 bytes of shared memory per column
                if (columns <= EDGES_COLUMNS) return norm_launch<T, P, W, 4, false>(p, columns, num_sms, st);
            }
        }
        const unsigned blocks = (unsigned)std::min<int64_t>(p.rows, num_sms * 8);
        return launch(norm_any<T, P>, blocks, ANY_THREADS, 0, st, p);
    });
}

size_t norm_grad_scratch(int64_t rows, int64_t dim, int num_sms) {
    // a row group per warp at most; and the rows' means
    const int64_t slices =
        std::max(std::min((rows + SLICE_ROWS - 1) / SLICE_ROWS, SLICES),
                 std::min<int64_t>(rows, (int64_t)num_sms * (GRAD_THREADS / 32)));
    return ((size_t)slices * 2 * (size_t)dim + (size_t)rows * 2) * sizeof(float);
}

cudaError_t launch_layer_norm_grad(spmm_type_t type, spmm_type_t param_type,
                                   const NormGradParams& given, int num_sms, cudaStream_t st) {
    return with_types(type, param_type, [&](auto t, auto pt) {
        using T = decltype(t);
        using P = decltype(pt);
        constexpr int W = 16 / (int)sizeof(T);
        NormGradParams p = given;
        const bool sums = p.dweight || p.dbias;
        p.means = p.part;
        p.part = sums ? p.means + 2 * p.rows : nullptr;
        int slices = 0;
        cudaError_t e = cudaSuccess;
        if (p.rows > 0) {
            const int64_t columns = p.dim + (off_boundary(p.x, p.ldx, sizeof(T)) ? W - 1 : 0);
            const bool same = alike(p.x, p.ldx, p.dy, p.ld_dy, sizeof(T)) &&
                              alike(p.x, p.ldx, p.dx, p.ld_dx, sizeof(T));
            if (same && columns <= GRAD_COLUMNS) {
                e = norm_grad_launch<T, P, false>(p, columns, num_sms, st, &slices);
            } else {
                const unsigned blocks = (unsigned)std::min<int64_t>(p.rows, num_sms * 8);
                auto means = alike(p.x, p.ldx, p.dy, p.ld_dy, sizeof(T)) ? grad_means<T, P, W>
                                                                         : grad_means<T, P, 1>;
                e = launch(means, blocks, ANY_THREADS, 0, st, p);
                if (e != cudaSuccess) return e;
                if (same) {
                    e = norm_grad_launch<T, P, true>(p, columns, num_sms, st, &slices);
                } else {
                    slices = (int)slices_any(p.rows);
                    const dim3 grid((unsigned)((p.dim + ANY_THREADS - 1) / ANY_THREADS),
                                    (unsigned)slices);
                    e = launch(norm_grad_any<T, P>, grid, ANY_THREADS, 0, st, p,
                               slice_rows(p.rows));
                }
            }
        }
        if (e != cudaSuccess || !sums) return e;
        return launch_chained(norm_dw_join<P>, dim3((unsigned)((p.dim + 31) / 32), 2),
                              dim3(32 * JOIN_WARPS), 0, st, p.rows > 0, p, slices);
    });
}

}  // namespace spmm
