// Device helpers of the language-model operators: element types, 16-byte and
// single-element accesses, and warp reductions.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "spmm_lm.h"

namespace spmm {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// W consecutive elements, moved with one access.
template <typename T, int W>
struct alignas(sizeof(T) * W) Vec {
    T v[W];
};

// How a load treats the caches: KEEP for what is read again, STREAM for what
// is read once.
enum class Cache { KEEP, STREAM };

template <Cache C, typename T, int W>
__device__ __forceinline__ Vec<T, W> load_vec(const T* p) {
    Vec<T, W> r;
    if constexpr (sizeof(T) * W == 16) {
        const int4 u = C == Cache::STREAM ? __ldcs(reinterpret_cast<const int4*>(p))
                                          : *reinterpret_cast<const int4*>(p);
        r = *reinterpret_cast<const Vec<T, W>*>(&u);
    } else {
        static_assert(W == 1);
        r.v[0] = C == Cache::STREAM ? __ldcs(p) : *p;
    }
    return r;
}

// Store W floats rounded to T.  W * sizeof(T) is 16 or 32 bytes (one or two
// accesses), or one element.
template <Cache C, typename T, int W>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[W]) {
    Vec<T, W> r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i] = from_f32<T>(f[i]);
    if constexpr (W > 1) {
        static_assert(sizeof(T) * W % 16 == 0);
        const int4* u = reinterpret_cast<const int4*>(&r);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) * W / 16); ++i) {
            if (C == Cache::STREAM) __stcs(reinterpret_cast<int4*>(p) + i, u[i]);
            else reinterpret_cast<int4*>(p)[i] = u[i];
        }
    } else {
        if (C == Cache::STREAM) __stcs(p, r.v[0]);
        else *p = r.v[0];
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Host: base and rows 16-byte aligned.
inline bool rows_aligned16(const void* p, int64_t ld, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * (int64_t)es) % 16 == 0;
}

// Calls f with a value of the C++ type of `t`.
template <typename F>
inline cudaError_t with_type(spmm_type_t t, F&& f) {
    switch (t) {
        case SPMM_F32: return f(float{});
        case SPMM_F16: return f(__half{});
        default: return f(__nv_bfloat16{});
    }
}

}  // namespace spmm
