// Layer norm y = (x - mean) * rstd * weight + bias over the rows of a matrix,
// and its gradients with respect to x, weight and bias.
//
// Mean and deviations are binary32 sums; the deviations are taken from the
// row's own mean in a second pass over the row, so no digits are lost to a
// mean far from zero.
#include <algorithm>

#include "spmm_internal.h"
#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

constexpr int NORM_THREADS = 256;
constexpr int NORM_GRAD_THREADS = 512;   // the gradient's block: up to 128 registers a thread

// Sum over the block (every thread gets it); `s` holds one float per warp.
template <int THREADS>
__device__ __forceinline__ float block_sum(float x, float* s) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += s[i];
    return t;
}

template <typename P>
__device__ __forceinline__ float param(const void* p, int64_t i, float none) {
    return p ? to_f32(static_cast<const P*>(p)[i]) : none;
}

// W parameters from column c, or the value `none` where there are none.
template <typename P, int W>
__device__ __forceinline__ void params(const void* p, int64_t c, float none, float (&f)[W]) {
    if (p) {
        unpack(load_vec<Cache::KEEP, P, W>(static_cast<const P*>(p) + c), f);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = none;
    }
}

// Barrier of one row's warps (barrier 0 is the block's own).
__device__ __forceinline__ void row_barrier(int row, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "r"(threads) : "memory");
}

// Sum over a row's `warps` warps, in warp order; `s` has a slot for each.
__device__ __forceinline__ float row_sum(float x, float* s, int row, int warps) {
    x = warp_sum(x);
    if (warps == 1) return x;
    if ((threadIdx.x & 31) == 0) s[(threadIdx.x >> 5) % warps] = x;
    row_barrier(row, warps * 32);
    float t = 0.0f;
    for (int i = 0; i < warps; ++i) t += s[i];
    return t;
}

// The row in registers: `warps` warps hold it in K accesses of W elements per
// lane, so x is read once and the second pass over it costs no memory.  Several
// narrow rows share a block.  With STAGES > 0 the row's warps walk the rows with
// a fixed stride and keep STAGES - 1 rows ahead on their way to shared memory,
// each lane's accesses in slots of its own.  The bound is HBM (read x, write y).
template <typename T, typename P, int W, int K, int STAGES>
__global__ __launch_bounds__(1024) void norm_rows(NormParams p, int warps, int nvec,
                                                  int64_t stride) {
    __shared__ float s[2][32];
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    const int threads = warps * 32;
    const int in_block = threadIdx.x / threads, tid = threadIdx.x % threads;
    const T* xs = static_cast<const T*>(p.x);
    int64_t r = (int64_t)blockIdx.x * (blockDim.x / threads) + in_block;
    Vec<T, W>* ring = reinterpret_cast<Vec<T, W>*>(ring_bytes) + threadIdx.x;
    auto copy = [&](int64_t row, int stage) {
        if constexpr (STAGES > 0) {
            if (row < p.rows)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k * threads + tid < nvec)
                        copy_async<T, W>(ring + (stage * K + k) * blockDim.x,
                                         xs + row * p.ldx + (int64_t)(k * threads + tid) * W);
            copies_issued();
        }
    };
    for (int i = 0; i < STAGES - 1; ++i) copy(r + i * stride, i);
    int stage = 0;
    for (; r < p.rows; r += stride) {
        Vec<T, W> held[K];
        if constexpr (STAGES > 0) {
            copies_wait<(STAGES > 1 ? STAGES - 2 : 0)>();
#pragma unroll
            for (int k = 0; k < K; ++k) held[k] = ring[(stage * K + k) * blockDim.x];
            copy(r + (STAGES - 1) * stride, stage == 0 ? STAGES - 1 : stage - 1);
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k * threads + tid < nvec)
                    held[k] = load_vec<Cache::STREAM, T, W>(xs + r * p.ldx +
                                                            (int64_t)(k * threads + tid) * W);
        }
        // one access per lane is the case of few rows, where latency counts: the
        // parameters are on their way during the sums
        float w0[W], b0[W];
        if constexpr (K == 1)
            if (tid < nvec) {
                params<P, W>(p.weight, tid * W, 1.0f, w0);
                params<P, W>(p.bias, tid * W, 0.0f, b0);
            }
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * threads + tid < nvec) {
                float f[W];
                unpack(held[k], f);
#pragma unroll
                for (int i = 0; i < W; ++i) sum += f[i];
            }
        float* slot = s[0] + in_block * warps;
        const float mean = row_sum(sum, slot, in_block, warps) / (float)p.dim;
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * threads + tid < nvec) {
                float f[W];
                unpack(held[k], f);
#pragma unroll
                for (int i = 0; i < W; ++i) sum += (f[i] - mean) * (f[i] - mean);
            }
        slot = s[1] + in_block * warps;
        const float var = row_sum(sum, slot, in_block, warps) / (float)p.dim;
        const float rstd = 1.0f / sqrtf(var + p.eps);
        T* y = static_cast<T*>(p.y) + r * p.ldy;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = k * threads + tid;
            if (at >= nvec) continue;
            float f[W], w[W], b[W];
            unpack(held[k], f);
            if constexpr (K > 1) {
                params<P, W>(p.weight, at * W, 1.0f, w);
                params<P, W>(p.bias, at * W, 0.0f, b);
            }
#pragma unroll
            for (int i = 0; i < W; ++i)
                f[i] = (f[i] - mean) * rstd * (K == 1 ? w0[i] : w[i]) + (K == 1 ? b0[i] : b[i]);
            store_vec<Cache::STREAM, T, W>(y + (int64_t)at * W, f);
        }
        if (tid == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// Any width and alignment: a block per row, the row read again for each pass.
template <typename T, typename P>
__global__ __launch_bounds__(NORM_THREADS) void norm_any(NormParams p) {
    __shared__ float s[NORM_THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        T* y = static_cast<T*>(p.y) + r * p.ldy;
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < p.dim; c += NORM_THREADS) sum += to_f32(x[c]);
        const float mean = block_sum<NORM_THREADS>(sum, s) / (float)p.dim;
        sum = 0.0f;
        for (int64_t c = threadIdx.x; c < p.dim; c += NORM_THREADS) {
            const float d = to_f32(x[c]) - mean;
            sum += d * d;
        }
        const float var = block_sum<NORM_THREADS>(sum, s) / (float)p.dim;
        const float rstd = 1.0f / sqrtf(var + p.eps);
        for (int64_t c = threadIdx.x; c < p.dim; c += NORM_THREADS)
            y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * param<P>(p.weight, c, 1.0f) +
                               param<P>(p.bias, c, 0.0f));
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// dx, and this block's share of dweight and dbias, in one pass over dy and x: a
// row's `warps` warps hold it in registers, walk the rows with a fixed stride, and keep their
// columns' sums of dy * xhat and dy in registers to the end.  The rows ahead are
// on their way to shared memory, each lane's accesses in slots of its own
// (single 16-bit elements cannot be copied so: the next row waits in registers).
// The bound is HBM (read dy and x, write dx).  part: [slices][2][dim].
// Stages of the ring: what 512 threads can have of the 227 KB, four at most.
template <typename T, int W, int K>
constexpr int GRAD_STAGES = sizeof(T) * W * K > 32 ? 3 : 4;
template <typename T, typename P, int W, int K>
__global__ __launch_bounds__(NORM_GRAD_THREADS) void norm_grad_rows(NormGradParams p, int warps,
                                                                    int nvec, int slices) {
    __shared__ float s[2][2][32];
    const int threads = warps * 32;
    const int in_block = threadIdx.x / threads, tid = threadIdx.x % threads;
    const int slice = blockIdx.x * (blockDim.x / threads) + in_block;
    if (slice >= slices) return;
    const T* xs = static_cast<const T*>(p.x);
    const T* dys = static_cast<const T*>(p.dy);
    const bool sums = p.dweight || p.dbias;
    // 16 elements a lane leave no registers for the weights in binary32 (W = 4) and
    // for single accesses (W = 1): those read them again for each row, from L1
    constexpr bool HOLD = W * K < 16 || W == 8;
    constexpr bool RING = can_copy_async<T, W>;
    constexpr int STAGES = GRAD_STAGES<T, W, K>;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    Vec<T, W>* ring = reinterpret_cast<Vec<T, W>*>(ring_bytes) + threadIdx.x;
    Vec<T, W> x[K], dy[K];
    float weight[HOLD ? K : 1][W], dw[K][W], db[K][W];
    // sends for row r: to a stage of the ring, or to the registers
    auto fetch = [&](int64_t r, int stage) {
        if (r < p.rows)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = k * threads + tid;
                if (at >= nvec) continue;
                const T* xr = xs + r * p.ldx + (int64_t)at * W;
                const T* dyr = dys + r * p.ld_dy + (int64_t)at * W;
                if constexpr (RING) {
                    copy_async<T, W>(ring + (stage * 2 * K + k) * blockDim.x, xr);
                    copy_async<T, W>(ring + (stage * 2 * K + K + k) * blockDim.x, dyr);
                } else {
                    x[k] = load_vec<Cache::STREAM, T, W>(xr);
                    dy[k] = load_vec<Cache::STREAM, T, W>(dyr);
                }
            }
        if constexpr (RING) copies_issued();
    };
    if constexpr (RING)
        for (int i = 0; i < STAGES - 1; ++i) fetch(slice + (int64_t)i * slices, i);
    else
        fetch(slice, 0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int i = 0; i < W; ++i) dw[k][i] = db[k][i] = 0.0f;
        if (HOLD && k * threads + tid < nvec)
            params<P, W>(p.weight, (int64_t)(k * threads + tid) * W, 1.0f, weight[HOLD ? k : 0]);
    }
    int turn = 0, stage = 0;
    for (int64_t r = slice; r < p.rows; r += slices) {
        if constexpr (RING) {
            copies_wait<STAGES - 2>();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                x[k] = ring[(stage * 2 * K + k) * blockDim.x];
                dy[k] = ring[(stage * 2 * K + K + k) * blockDim.x];
            }
            fetch(r + (int64_t)(STAGES - 1) * slices, stage == 0 ? STAGES - 1 : stage - 1);
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
        const float mean = p.mean[r], rstd = p.rstd[r];
        float xh[K][W], g[K][W];
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * threads + tid < nvec) {
                unpack(x[k], xh[k]);
                unpack(dy[k], g[k]);
                float (&wk)[W] = weight[HOLD ? k : 0];
                if (!HOLD) params<P, W>(p.weight, (int64_t)(k * threads + tid) * W, 1.0f, wk);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    xh[k][i] = (xh[k][i] - mean) * rstd;
                    dw[k][i] += g[k][i] * xh[k][i];
                    db[k][i] += g[k][i];
                    g[k][i] *= wk[i];
                    a += g[k][i];
                    b += g[k][i] * xh[k][i];
                }
            }
        if constexpr (!RING) fetch(r + slices, 0);
        a = warp_sum(a);
        b = warp_sum(b);
        if (warps > 1) {
            // two sets of slots in turn: one barrier per row keeps them apart
            float* sa = s[turn][0] + in_block * warps;
            float* sb = s[turn][1] + in_block * warps;
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) {
                sa[tid >> 5] = a;
                sb[tid >> 5] = b;
            }
            row_barrier(in_block, threads);
            a = b = 0.0f;
            for (int i = 0; i < warps; ++i) {
                a += sa[i];
                b += sb[i];
            }
        }
        a /= (float)p.dim;
        b /= (float)p.dim;
        T* dx = static_cast<T*>(p.dx) + r * p.ld_dx;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = k * threads + tid;
            if (at >= nvec) continue;
#pragma unroll
            for (int i = 0; i < W; ++i) g[k][i] = rstd * (g[k][i] - a - xh[k][i] * b);
            store_vec<Cache::STREAM, T, W>(dx + (int64_t)at * W, g[k]);
        }
    }
    allow_successor();
    if (!sums) return;
    float* part = p.part + (int64_t)slice * 2 * p.dim;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int at = k * threads + tid;
        if (at >= nvec) continue;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            part[(int64_t)at * W + i] = dw[k][i];
            part[p.dim + (int64_t)at * W + i] = db[k][i];
        }
    }
}

// Any width and alignment: dx, a block per row.
template <typename T, typename P>
__global__ __launch_bounds__(NORM_THREADS) void norm_dx_any(NormGradParams p) {
    __shared__ float s[NORM_THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        const T* dy = static_cast<const T*>(p.dy) + r * p.ld_dy;
        T* dx = static_cast<T*>(p.dx) + r * p.ld_dx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float a = 0.0f, b = 0.0f;
        for (int64_t c = threadIdx.x; c < p.dim; c += NORM_THREADS) {
            const float g = to_f32(dy[c]) * param<P>(p.weight, c, 1.0f);
            a += g;
            b += g * ((to_f32(x[c]) - mean) * rstd);
        }
        a = block_sum<NORM_THREADS>(a, s) / (float)p.dim;
        b = block_sum<NORM_THREADS>(b, s) / (float)p.dim;
        for (int64_t c = threadIdx.x; c < p.dim; c += NORM_THREADS) {
            const float g = to_f32(dy[c]) * param<P>(p.weight, c, 1.0f);
            dx[c] = from_f32<T>(rstd * (g - a - (to_f32(x[c]) - mean) * rstd * b));
        }
    }
}

// Column sums of dy * xhat and dy over a slice of the rows: a warp per row of
// 32 columns, blocks (column tile, slice).  part: [slices][2][dim].
constexpr int SLICE_ROWS = 256;
template <typename T>
__global__ __launch_bounds__(256) void norm_dw_any(NormGradParams p) {
    __shared__ float s[2][8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const int64_t r0 = (int64_t)blockIdx.y * SLICE_ROWS;
    const int64_t r1 = min(r0 + SLICE_ROWS, p.rows);
    float dw = 0.0f, db = 0.0f;
    if (c < p.dim) {
        for (int64_t r = r0 + w; r < r1; r += 8) {
            const float g = to_f32(static_cast<const T*>(p.dy)[r * p.ld_dy + c]);
            const float x = to_f32(static_cast<const T*>(p.x)[r * p.ldx + c]);
            dw += g * ((x - p.mean[r]) * p.rstd[r]);
            db += g;
        }
    }
    s[0][w][lane] = dw;
    s[1][w][lane] = db;
    __syncthreads();
    if (w < 2 && c < p.dim) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[w][i][lane];
        p.part[((int64_t)blockIdx.y * 2 + w) * p.dim + c] = t;
    }
}

// dweight and dbias from the slices' partial sums: a block takes 32 columns, each
// of its warps every JOIN_WARPS-th slice in order, then the warps' sums are added
// in order.  As many warps as a block may have: the sums are short, and what
// counts is how many loads wait together.
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

int64_t slices_any(int64_t rows) { return (rows + SLICE_ROWS - 1) / SLICE_ROWS; }

// Warps that hold a row of nvec accesses, K per lane.
int warps_for(int64_t nvec, int K) {
    int warps = 1;
    while ((int64_t)warps * 32 * K < nvec) warps *= 2;
    return warps;
}

// Slices of the register kernel's grid: one row at a time each, as many as the
// SMs hold (`sm_warps` warps each, by the kernel's registers).
int64_t slices_rows(int64_t rows, int warps, int num_sms, int sm_warps) {
    return std::min<int64_t>(rows, (int64_t)num_sms * sm_warps / warps);
}
constexpr int SM_WARPS_MOST = 32;    // 64 registers a thread: up to 4 elements per lane

template <typename... KArgs>
cudaError_t allow_shared(void (*kernel)(KArgs...), size_t bytes) {
    return bytes <= 32768 ? cudaSuccess
                          : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)bytes);
}

template <typename T, typename P, int W, int K, int STAGES>
cudaError_t norm_launch(const NormParams& p, int num_sms, cudaStream_t st) {
    const int nvec = (int)(p.dim / W);
    const int warps = warps_for(nvec, K);
    const int rows = std::max(1, 8 / warps);          // at least 256 threads
    int64_t blocks = (p.rows + rows - 1) / rows;
    // with a ring: as many blocks as the SMs hold at 64 registers a thread
    if (STAGES > 0) blocks = std::min<int64_t>(blocks, (int64_t)num_sms * (32 / (rows * warps)));
    const size_t shared = (size_t)STAGES * K * rows * warps * 32 * sizeof(Vec<T, W>);
    auto kernel = norm_rows<T, P, W, K, STAGES>;
    cudaError_t e = allow_shared(kernel, shared);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, rows * warps * 32, shared, st>>>(p, warps, nvec, blocks * rows);
    return cudaGetLastError();
}

template <typename T, typename P, int W, int K>
cudaError_t norm_grad_launch(const NormGradParams& p, int num_sms, cudaStream_t st, int* slices) {
    const int nvec = (int)(p.dim / W);
    const int warps = warps_for(nvec, K);
    const int rows = std::max(1, 4 / warps);          // at least 128 threads
    constexpr int SM_WARPS = W * K <= 4 ? SM_WARPS_MOST : SM_WARPS_MOST / 2;
    *slices = (int)slices_rows(p.rows, warps, num_sms, SM_WARPS);
    const size_t shared = can_copy_async<T, W>
                              ? (size_t)GRAD_STAGES<T, W, K> * 2 * K * rows * warps * 32 * sizeof(Vec<T, W>)
                              : 0;
    auto kernel = norm_grad_rows<T, P, W, K>;
    cudaError_t e = allow_shared(kernel, shared);
    if (e != cudaSuccess) return e;
    kernel<<<(*slices + rows - 1) / rows, rows * warps * 32, shared, st>>>(p, warps, nvec,
                                                                          *slices);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(spmm_type_t type, spmm_type_t param_type, const NormParams& p,
                              int num_sms, cudaStream_t st) {
    auto typed = [&](auto t, auto pt) {
        using T = decltype(t);
        using P = decltype(pt);
        constexpr int W = 16 / sizeof(T);
        const bool wide = p.dim % W == 0 && rows_aligned16(p.x, p.ldx, sizeof(T)) &&
                          rows_aligned16(p.y, p.ldy, sizeof(T)) &&
                          (!p.weight || rows_aligned16(p.weight, 0, 1)) &&
                          (!p.bias || rows_aligned16(p.bias, 0, 1));
        // A row takes at most 1024 threads.  Few rows leave SMs idle: then the
        // most threads per row (one access each) give the shortest call; many
        // rows take four accesses per lane, fewer barriers per byte.
        if (wide) {
            const int64_t nvec = p.dim / W;
            if (nvec <= 1024 && (p.rows <= 2 * num_sms || nvec <= 32))
                return norm_launch<T, P, W, 1, 0>(p, num_sms, st);
            if (nvec <= 4096) return norm_launch<T, P, W, 4, 3>(p, num_sms, st);
        } else {
            if (p.dim <= 4096) return norm_launch<T, P, 1, 4, 0>(p, num_sms, st);
            if (p.dim <= 16384) return norm_launch<T, P, 1, 16, 0>(p, num_sms, st);
        }
        const unsigned blocks = (unsigned)std::min<int64_t>(p.rows, num_sms * 8);
        norm_any<T, P><<<blocks, NORM_THREADS, 0, st>>>(p);
        return cudaGetLastError();
    };
    return with_type(type, [&](auto t) {
        return type == param_type ? typed(t, t) : typed(t, float{});
    });
}

size_t norm_grad_scratch(int64_t rows, int64_t dim, int num_sms) {
    const int64_t slices = std::max(slices_any(rows), slices_rows(rows, 1, num_sms, SM_WARPS_MOST));
    return (size_t)slices * 2 * (size_t)dim * sizeof(float);
}

cudaError_t launch_layer_norm_grad(spmm_type_t type, spmm_type_t param_type,
                                   const NormGradParams& p, int num_sms, cudaStream_t st) {
    auto typed = [&](auto t, auto pt) {
        using T = decltype(t);
        using P = decltype(pt);
        constexpr int W = 16 / sizeof(T);
        constexpr int K = 16 / W;                     // 16 elements of the row per lane
        const bool sums = p.dweight || p.dbias;
        int slices = 0;
        cudaError_t e = cudaSuccess;
        if (p.rows > 0) {
            const bool wide = p.dim % W == 0 && rows_aligned16(p.x, p.ldx, sizeof(T)) &&
                              rows_aligned16(p.dy, p.ld_dy, sizeof(T)) &&
                              rows_aligned16(p.dx, p.ld_dx, sizeof(T)) &&
                              (!p.weight || rows_aligned16(p.weight, 0, 1));
            if (wide && p.dim <= NORM_GRAD_THREADS * 16) {
                e = norm_grad_launch<T, P, W, K>(p, num_sms, st, &slices);
            } else if (p.dim <= NORM_GRAD_THREADS * 4) {
                e = norm_grad_launch<T, P, 1, 4>(p, num_sms, st, &slices);
            } else if (p.dim <= NORM_GRAD_THREADS * 8) {
                e = norm_grad_launch<T, P, 1, 8>(p, num_sms, st, &slices);
            } else if (p.dim <= NORM_GRAD_THREADS * 16) {
                e = norm_grad_launch<T, P, 1, 16>(p, num_sms, st, &slices);
            } else {
                // the sums first: dx may be dy
                slices = (int)slices_any(p.rows);
                if (sums) {
                    const dim3 grid((unsigned)((p.dim + 31) / 32), (unsigned)slices);
                    norm_dw_any<T><<<grid, 256, 0, st>>>(p);
                }
                const unsigned blocks = (unsigned)std::min<int64_t>(p.rows, num_sms * 8);
                norm_dx_any<T, P><<<blocks, NORM_THREADS, 0, st>>>(p);
                e = cudaGetLastError();
            }
        }
        if (e != cudaSuccess || !sums) return e;
        return launch_chained(norm_dw_join<P>, dim3((unsigned)((p.dim + 31) / 32), 2),
                              dim3(32 * JOIN_WARPS), 0, st, p.rows > 0, p, slices);
    };
    return with_type(type, [&](auto t) {
        return type == param_type ? typed(t, t) : typed(t, float{});
    });
}

}  // namespace spmm
