// Token log probabilities: per row of logits the log-sum-exp, the log
// probability of a given token, the entropy and the top alternatives; and the
// logits' gradient.
#include <algorithm>

#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

constexpr int LP_THREADS = 256;

// A number that orders logits by value, then by lowest index: 0 for what is
// never an alternative (-inf and NaN).  -0 counts as 0.
__device__ __forceinline__ uint64_t rank_key(float x, unsigned index) {
    if (!(x > -INFINITY)) return 0;
    const unsigned u = __float_as_uint(x + 0.0f);
    const unsigned order = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)order << 32 | (0xffffffffu - index);
}

__device__ __forceinline__ float block_sum(float x, float* s) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < LP_THREADS / 32; ++i) t += s[i];
    return t;
}

__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int i = 0; i < LP_THREADS / 32; ++i) t = max(t, s[i]);
    return t;
}

// One block per row, the row read again for each step.
template <typename T>
__global__ __launch_bounds__(LP_THREADS) void logprob_rows(LogprobParams p) {
    __shared__ float sf[LP_THREADS / 32];
    __shared__ uint64_t sk[LP_THREADS / 32];
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.logits) + r * p.ld;
    const int n = (int)p.vocab;
    uint64_t best = 0;
    for (int c = threadIdx.x; c < n; c += LP_THREADS) best = max(best, rank_key(to_f32(x[c]), c));
    best = block_max(best, sk);
    const float m = best ? to_f32(x[0xffffffffu - (unsigned)best]) : 0.0f;
    // sums of e = exp(alpha (x - m)) and of e * alpha (x - m); a masked logit adds nothing
    float sum = 0.0f, weighted = 0.0f;
    for (int c = threadIdx.x; c < n; c += LP_THREADS) {
        const float v = to_f32(x[c]);
        if (v == -INFINITY) continue;
        const float t = p.alpha * (v - m);
        const float e = expf(t);
        sum += e;
        if (e != 0.0f) weighted += e * t;
    }
    sum = block_sum(sum, sf);
    weighted = block_sum(weighted, sf);
    const float log_sum = logf(sum);                    // -inf for a row without a logit
    const float lse = p.alpha * m + log_sum;
    if (threadIdx.x == 0) {
        if (p.lse) p.lse[r] = lse;
        if (p.entropy) p.entropy[r] = sum == 0.0f ? 0.0f : log_sum - weighted / sum;
        if (p.targets) {
            const int t = p.targets[r];
            float v = 0.0f;
            if (t >= 0 && t < n) v = sum == 0.0f ? -INFINITY : p.alpha * to_f32(x[t]) - lse;
            p.logprob[r] = v;
        }
    }
    for (int k = 0; k < p.top_k; ++k) {
        if (threadIdx.x == 0) {
            const int i = best ? (int)(0xffffffffu - (unsigned)best) : -1;
            p.top_index[r * p.top_k + k] = i;
            p.top_logprob[r * p.top_k + k] = sum != sum ? NAN
                                             : i < 0    ? -INFINITY
                                                        : p.alpha * to_f32(x[i]) - lse;
        }
        uint64_t next = 0;
        for (int c = threadIdx.x; c < n; c += LP_THREADS) {
            const uint64_t key = rank_key(to_f32(x[c]), c);
            if (key < best) next = max(next, key);
        }
        best = block_max(next, sk);
    }
}

// One block per row.
template <typename T>
__global__ __launch_bounds__(LP_THREADS) void logprob_grad_rows(LogprobGradParams p) {
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.logits) + r * p.ld;
    T* dx = static_cast<T*>(p.dlogits) + r * p.ld_out;
    const float lse = p.lse[r];
    const int target = p.targets ? p.targets[r] : -1;
    const bool has = target >= 0 && target < p.vocab;
    const float up = has ? p.dlogprob[r] : 0.0f;
    const float de = p.dentropy ? p.dentropy[r] : 0.0f;
    const float ent = p.dentropy ? p.entropy[r] : 0.0f;
    for (int64_t c = threadIdx.x; c < p.vocab; c += LP_THREADS) {
        float d = 0.0f;
        if (lse != -INFINITY) {
            const float q = fmaf(p.alpha, to_f32(x[c]), -lse);
            const float e = expf(q);
            d = (c == target ? up : 0.0f) - up * e;
            if (e != 0.0f) d -= de * e * (q + ent);
        }
        dx[c] = from_f32<T>(p.alpha * d);
    }
}

}  // namespace

cudaError_t launch_token_logprob(spmm_type_t type, const LogprobParams& p, int num_sms,
                                 cudaStream_t st) {
    (void)num_sms;
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        logprob_rows<T><<<(unsigned)p.rows, LP_THREADS, 0, st>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_token_logprob_grad(spmm_type_t type, const LogprobGradParams& p, int num_sms,
                                      cudaStream_t st) {
    (void)num_sms;
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        logprob_grad_rows<T><<<(unsigned)p.rows, LP_THREADS, 0, st>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace spmm
