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

// W consecutive elements as they lie in memory: W > 1 in 32-bit words, so that
// 16-bit elements stay packed in registers until they are used.
template <typename T, int W>
struct alignas(sizeof(T) * W % 16 == 0 ? 16 : sizeof(T) * W) Vec {
    static constexpr int WORDS = (int)sizeof(T) * W / 4;
    uint32_t w[WORDS];
};
template <typename T>
struct Vec<T, 1> {
    T w;
};

__device__ __forceinline__ void unpack_word(uint32_t w, float* f, __nv_bfloat16) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_word(uint32_t w, float* f, __half) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
    f[0] = x.x;
    f[1] = x.y;
}
__device__ __forceinline__ uint32_t pack_word(const float* f, __nv_bfloat16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t pack_word(const float* f, __half) {
    const __half2 x = __floats2half2_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// The elements of a Vec in binary32.
template <typename T, int W>
__device__ __forceinline__ void unpack(const Vec<T, W>& r, float (&f)[W]) {
    if constexpr (W == 1) {
        f[0] = to_f32(r.w);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) unpack_word(r.w[i], f + 2 * i, T{});
    }
}

// How a load treats the caches: KEEP for what is read again, STREAM for what
// is read once.
enum class Cache { KEEP, STREAM };

// W consecutive elements: 16-byte accesses (one of 8 bytes for four 16-bit elements)
// when W > 1, one element otherwise.
template <Cache C, typename T, int W>
__device__ __forceinline__ Vec<T, W> load_vec(const T* p) {
    Vec<T, W> r;
    if constexpr (sizeof(T) * W == 8) {
        const uint2* from = reinterpret_cast<const uint2*>(p);
        const uint2 u = C == Cache::STREAM ? __ldcs(from) : *from;
        r.w[0] = u.x;
        r.w[1] = u.y;
    } else if constexpr (W > 1) {
        static_assert(sizeof(T) * W % 16 == 0);
        const uint4* from = reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int i = 0; i < Vec<T, W>::WORDS / 4; ++i) {
            const uint4 u = C == Cache::STREAM ? __ldcs(from + i) : from[i];
            r.w[4 * i] = u.x;
            r.w[4 * i + 1] = u.y;
            r.w[4 * i + 2] = u.z;
            r.w[4 * i + 3] = u.w;
        }
    } else {
        r.w = C == Cache::STREAM ? __ldcs(p) : *p;
    }
    return r;
}

// Store W floats rounded to T, with the same accesses.
template <Cache C, typename T, int W>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[W]) {
    if constexpr (W > 1) {
        static_assert(sizeof(T) * W % 16 == 0 || sizeof(T) * W == 8);
        uint32_t w[Vec<T, W>::WORDS];
#pragma unroll
        for (int i = 0; i < Vec<T, W>::WORDS; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
            else w[i] = pack_word(f + 2 * i, T{});
        }
        if constexpr (sizeof(T) * W == 8) {
            const uint2 u = make_uint2(w[0], w[1]);
            if (C == Cache::STREAM) __stcs(reinterpret_cast<uint2*>(p), u);
            else *reinterpret_cast<uint2*>(p) = u;
        }
        uint4* to = reinterpret_cast<uint4*>(p);
#pragma unroll
        for (int i = 0; i < Vec<T, W>::WORDS / 4; ++i) {
            const uint4 u = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            if (C == Cache::STREAM) __stcs(to + i, u);
            else to[i] = u;
        }
    } else {
        const T v = from_f32<T>(f[0]);
        if (C == Cache::STREAM) __stcs(p, v);
        else *p = v;
    }
}

// 16 bytes of elements from any element address: the two aligned words they lie in
// (one, when aligned), and the bytes of the first that come before them.
template <typename T>
struct Unaligned {
    static constexpr int W = 16 / (int)sizeof(T);
    Vec<T, W> a, b;
    unsigned shift;

    __device__ __forceinline__ void load(const T* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        shift = at % 16;
        const T* from = reinterpret_cast<const T*>(at - shift);
        a = load_vec<Cache::KEEP, T, W>(from);
        b = load_vec<Cache::KEEP, T, W>(from + (shift ? W : 0));
    }
    __device__ __forceinline__ Vec<T, W> get() const {
        const uint32_t w[8] = {a.w[0], a.w[1], a.w[2], a.w[3], b.w[0], b.w[1], b.w[2], b.w[3]};
        uint32_t t[6], u[5];
#pragma unroll
        for (int i = 0; i < 6; ++i) t[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = shift & 4 ? t[i + 1] : t[i];
        Vec<T, W> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = __funnelshift_r(u[i], u[i + 1], (shift & 2) * 8);
        return r;
    }
    // The same where the shift is known to begin in word F of the first.
    template <int F>
    __device__ __forceinline__ Vec<T, W> from_word() const {
        const uint32_t w[8] = {a.w[0], a.w[1], a.w[2], a.w[3], b.w[0], b.w[1], b.w[2], b.w[3]};
        Vec<T, W> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = __funnelshift_r(w[F + i], w[F + i + 1], (shift & 2) * 8);
        return r;
    }
};
// A matrix whose rows are read so: whether W elements from element `at` of the matrix
// (rows and gaps) can be, i.e. no aligned word of theirs reaches over its ends.
template <int W>
__device__ __forceinline__ bool clear_of_ends(int64_t at, int64_t elements) {
    return at >= W && at + 2 * W <= elements;
}

// Elements [c, c + W) of a row of `dim`, those outside it 0, one by one.
template <typename T, int W>
__device__ __forceinline__ Vec<T, W> load_some(const T* row, int c, int dim) {
    Vec<T, W> r;
    if constexpr (W == 1) {
        r.w = c >= 0 && c < dim ? row[c] : from_f32<T>(0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < Vec<T, W>::WORDS; ++i) r.w[i] = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (c + i < 0 || c + i >= dim) continue;
            if constexpr (sizeof(T) == 4)
                r.w[i] = reinterpret_cast<const uint32_t*>(row)[c + i];
            else
                r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[c + i]
                              << ((i & 1) * 16);
        }
    }
    return r;
}
// Stores W elements to [c, c + W) of a row of `dim`, a whole access at once (it must be
// aligned either way), those of another that lie in the row one by one or, of 16 bits, in pairs.
template <typename T, int W>
__device__ __forceinline__ void store_some(T* row, int c, int dim, const float (&f)[W]) {
    if (c >= 0 && c + W <= dim) {
        store_vec<Cache::STREAM, T, W>(row + c, f);
        return;
    }
    if constexpr (sizeof(T) == 2 && W > 1) {
        // words with both elements in the row at once
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const bool low = (unsigned)(c + i) < (unsigned)dim;
            const bool high = (unsigned)(c + i + 1) < (unsigned)dim;
            if (low & high) *reinterpret_cast<uint32_t*>(row + c + i) = pack_word(f + i, T{});
            else if (low) row[c + i] = from_f32<T>(f[i]);
            else if (high) row[c + i + 1] = from_f32<T>(f[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if ((unsigned)(c + i) < (unsigned)dim) row[c + i] = from_f32<T>(f[i]);
    }
}
// Columns before the row's start that its first aligned access of `bytes` covers.
template <typename T>
__device__ __forceinline__ int lead_of(const T* row, int bytes) {
    return (int)(reinterpret_cast<uintptr_t>(row) % bytes / sizeof(T));
}

// Asynchronous copies of a 16-byte Vec into the issuing thread's own slot of shared
// memory: no registers wait for them, and since no other thread reads the slot,
// no barrier is needed either.
template <typename T, int W>
__device__ __forceinline__ void copy_async(Vec<T, W>* to, const T* from) {
    static_assert(sizeof(T) * W == 16);
    const unsigned a = (unsigned)__cvta_generic_to_shared(to);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_issued() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most N later groups of copies are outstanding.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two binary32 operations in one instruction (sm_100 and later); each half is
// rounded as the single operation would be, but for a mul2 whose product an add2 takes:
// the two become one fma2 (measured), where a product has to be rounded first use
// __fmul_rn.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void halves(uint64_t r, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
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
