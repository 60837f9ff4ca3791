// Layer norm y = (x - mean) * rstd * weight + bias over the rows of a matrix,
// and its gradients with respect to x, weight and bias.
//
// Mean and deviations are binary32 sums; the deviations are taken from the
// row's own mean in a second pass over the row, so no digits are lost to a
// mean far from zero.
#include <algorithm>

#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

constexpr int NORM_THREADS = 256;

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

// dweight and dbias from the slices' partial sums, added in slice order.
template <typename P>
__global__ __launch_bounds__(256) void norm_dw_join(NormGradParams p, int slices) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * p.dim) return;
    const int which = i >= p.dim;
    const int64_t c = i - which * p.dim;
    P* out = static_cast<P*>(which ? p.dbias : p.dweight);
    if (!out) return;
    float t = 0.0f;
    for (int k = 0; k < slices; ++k) t += p.part[((int64_t)k * 2 + which) * p.dim + c];
    out[c] = from_f32<P>(t);
}

int64_t slices_of(int64_t rows) { return (rows + SLICE_ROWS - 1) / SLICE_ROWS; }

}  // namespace

cudaError_t launch_layer_norm(spmm_type_t type, spmm_type_t param_type, const NormParams& p,
                              int num_sms, cudaStream_t st) {
    const unsigned blocks = (unsigned)std::min<int64_t>(p.rows, num_sms * 8);
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        if (type == param_type) norm_any<T, T><<<blocks, NORM_THREADS, 0, st>>>(p);
        else norm_any<T, float><<<blocks, NORM_THREADS, 0, st>>>(p);
        return cudaGetLastError();
    });
}

size_t norm_grad_scratch(int64_t rows, int64_t dim, int num_sms) {
    (void)num_sms;
    return (size_t)slices_of(rows) * 2 * (size_t)dim * sizeof(float);
}

cudaError_t launch_layer_norm_grad(spmm_type_t type, spmm_type_t param_type,
                                   const NormGradParams& p, int num_sms, cudaStream_t st) {
    const unsigned blocks = (unsigned)std::min<int64_t>(p.rows, num_sms * 8);
    const int slices = (int)slices_of(p.rows);
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        if (p.dweight || p.dbias) {
            const dim3 grid((unsigned)((p.dim + 31) / 32), (unsigned)slices);
            if (slices > 0) norm_dw_any<T><<<grid, 256, 0, st>>>(p);
            const unsigned jb = (unsigned)((2 * p.dim + 255) / 256);
            if (type == param_type) norm_dw_join<T><<<jb, 256, 0, st>>>(p, slices);
            else norm_dw_join<float><<<jb, 256, 0, st>>>(p, slices);
        }
        // after the sums: dx may be dy
        if (p.rows > 0) {
            if (type == param_type) norm_dx_any<T, T><<<blocks, NORM_THREADS, 0, st>>>(p);
            else norm_dx_any<T, float><<<blocks, NORM_THREADS, 0, st>>>(p);
        }
        return cudaGetLastError();
    });
}

}  // namespace spmm
