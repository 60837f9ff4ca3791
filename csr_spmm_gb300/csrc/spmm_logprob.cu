// Token log probabilities: per row of logits the log-sum-exp, the log
// probability of a given token, the entropy and the top alternatives; and the
// logits' gradient.
//
// With z = alpha x and any base b, in units of log 2 (c = alpha log2 e):
//   t = c x - b,  S = sum 2^t,  U = sum 2^t t
//   lse = (b + log2 S) ln 2,  entropy = (log2 S - U / S) ln 2
// so one pass over the row is enough: b follows the running maximum, and a
// change from b to b' scales S by 2^(b - b') and U to 2^(b - b') (U + (b - b') S).
#include <algorithm>
#include <cooperative_groups.h>

#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned ALL = 0xffffffffu;
constexpr float LN2 = 0.6931471805599453f;
constexpr float LOG2E = 1.4426950408889634f;

// ---- small pieces ---------------------------------------------------------------

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger one; NaN when either is.
__device__ __forceinline__ float max_nan(float x, float y) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
    return m;
}
// Largest over the warp, NaNs left out.
__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

// A whole number that orders logits by value (-0 counts as 0): 0 for what is
// never an alternative, -inf and NaN.
__device__ __forceinline__ unsigned order_of(float x) {
    if (!(x > -INFINITY)) return 0;
    const unsigned u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned order) {
    return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}
// Orders alternatives: by value, then by lowest index.
__device__ __forceinline__ uint64_t rank_key(unsigned order, unsigned index) {
    return (uint64_t)order << 32 | (0xffffffffu - index);
}

// ---- a row as 16-byte accesses -----------------------------------------------------

// A row need not start on a 16-byte boundary: accesses are counted from the
// boundary before it, `off` elements earlier, and those that reach outside the
// row are taken element by element, with -inf for what is outside.
template <typename T>
struct Row {
    static constexpr int W = 16 / (int)sizeof(T);
    const T* from;                   // the boundary: element i of the row is from[off + i]
    int off;
    int64_t end;                     // off + columns

    __device__ Row(const T* x, int64_t n) {
        off = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
        from = x - off;
        end = off + n;
    }
    __device__ bool whole(int64_t j) const { return j * W >= off && (j + 1) * W <= end; }
    __device__ Vec<T, W> edge(int64_t j) const {
        Vec<T, W> r;
        constexpr unsigned none = sizeof(T) == 4 ? 0xff800000u
                                  : std::is_same_v<T, __half> ? 0xfc00u : 0xff80u;
#pragma unroll
        for (int i = 0; i < Vec<T, W>::WORDS; ++i) r.w[i] = sizeof(T) == 4 ? none : none * 0x10001u;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t at = j * W + i;
            if (at < off || at >= end) continue;
            if constexpr (sizeof(T) == 4) {
                r.w[i] = __float_as_uint(from[at]);
            } else {
                const unsigned short b = reinterpret_cast<const unsigned short*>(from)[at];
                const unsigned shift = (i & 1) * 16;
                r.w[i / 2] = (r.w[i / 2] & ~(0xffffu << shift)) | (unsigned)b << shift;
            }
        }
        return r;
    }
    template <Cache C>
    __device__ Vec<T, W> load(int64_t j) const {
        return whole(j) ? load_vec<C, T, W>(from + j * W) : edge(j);
    }
};

// Largest of an access's elements, NaNs left out.
template <typename T, int W>
__device__ __forceinline__ float vec_max(const Vec<T, W>& v) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.w[0]), __uint_as_float(v.w[1])),
                     fmaxf(__uint_as_float(v.w[2]), __uint_as_float(v.w[3])));
    } else if constexpr (std::is_same_v<T, __half>) {
        const __half2* h = reinterpret_cast<const __half2*>(v.w);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(v.w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

// ---- forward --------------------------------------------------------------------------

constexpr int LP_WARPS = 8;                     // at most
constexpr int UNITS = 4;                        // accesses in flight per lane
constexpr int GROUPS = 32 * LP_WARPS;           // groups of the selection, at most
constexpr int CANDIDATES = SPMM_TOP_MAX * SPMM_TOP_MAX;

// Sums of a part of a row.  The base is c * max(m, -lim), rounded: every use must see
// the same number, so the product may not become part of a fused multiply-add.
struct Sums {
    float m, s, u;
};
__device__ __forceinline__ float base_of(float m, float c, float lim) {
    return __fmul_rn(fmaxf(m, -lim), c);
}
__device__ __forceinline__ void add(Sums& a, const Sums& b, float c, float lim) {
    const float m = fmaxf(a.m, b.m);
    const float base = base_of(m, c, lim);
    const float da = base_of(a.m, c, lim) - base, db = base_of(b.m, c, lim) - base;
    const float ea = exp2_approx(da), eb = exp2_approx(db);
    // a part without weight (e == 0) may be any distance away
    a.u = ea * (a.u + (ea > 0.0f ? da : 0.0f) * a.s) + eb * (b.u + (eb > 0.0f ? db : 0.0f) * b.s);
    a.s = ea * a.s + eb * b.s;
    a.m = m;
}

struct RowShared {
    Sums sums[LP_WARPS];
    Sums total;                                 // this block's part of the row
    uint64_t best[SPMM_TOP_MAX];                // its alternatives, largest first (0: none)
    unsigned group_max[GROUPS];                 // order_of each group's largest logit
    int chosen[SPMM_TOP_MAX];                   // the groups that hold the alternatives
    int chosen_count;
    int count;
    uint64_t list[CANDIDATES];
};

// The alternatives of this block's part of the row, into sh.best.
//
// The part's accesses fall into groups of 2^shift, contiguous and in index order,
// at most one group per thread.  Take the k groups whose largest logits rank highest (equal
// ones by lowest group): every alternative lies in one of them, since an
// element of another group is beaten by the largest of each of the k.  The
// smallest of the k maxima, tau, is a lower bound of the alternatives' values.
// So a second look at k groups (in L2) is enough: collect what lies above tau,
// and of each group's elements equal to tau the first k, then rank that short
// list.  Only a row with more than CANDIDATES such elements takes k rounds of
// the largest one left.
template <typename T>
__device__ void choose(RowShared& sh, const Row<T>& row, int64_t unit0, int64_t units, int shift,
                       int k) {
    constexpr int W = Row<T>::W;
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    const unsigned mine = sh.group_max[tid];
    // tau: the largest order that at least k groups reach (0: fewer than k have any)
    unsigned tau = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const unsigned next = tau | 1u << bit;
        if (__syncthreads_count(mine >= next) >= k) tau = next;
    }
    if (tid < k) sh.best[tid] = 0;
    if (tid == 0) {
        sh.chosen_count = 0;
        sh.count = 0;
    }
    __syncthreads();
    // groups above tau, then those equal to tau from the lowest; for tau == 0 all that have any
    if (mine > tau) sh.chosen[atomicAdd(&sh.chosen_count, 1)] = tid;
    __syncthreads();
    if (tau > 0 && tid < 32) {
        int have = sh.chosen_count;
        for (int g = lane; have < k && g - lane < (int)blockDim.x; g += 32) {
            const unsigned equal = __ballot_sync(ALL, sh.group_max[g] == tau);
            const int at = have + __popc(equal & ((1u << lane) - 1));
            if ((equal >> lane & 1) && at < k) sh.chosen[at] = g;
            have += __popc(equal);
        }
        if (lane == 0) sh.chosen_count = min(have, k);
    }
    __syncthreads();
    const int chosen = sh.chosen_count;
    const unsigned least = max(tau, 1u);
    // 32 lanes, or 2^shift where that is less, per group; its elements in index order
    const int width = min(32, 1 << shift), together = 32 / width;
    const int64_t j_end = (unit0 + units) * 32;
    const int steps = shift > 5 ? 1 << (shift - 5) : 1;
    for (int q0 = (tid >> 5) * together; q0 < chosen; q0 += warps * together) {
        const int q = q0 + lane / width;
        int64_t j = unit0 * 32 + (lane & (width - 1));
        j = q < chosen ? j + ((int64_t)sh.chosen[q] << shift) : j_end;
        int equal_seen = 0;
        for (int step = 0; step < steps; ++step, j += 32) {
            unsigned order[W];
            int equal = 0;
            bool any = false;
            if (j < j_end) {
                float f[W];
                unpack(row.template load<Cache::KEEP>(j), f);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    order[i] = order_of(f[i]);
                    any |= order[i] >= least;
                    equal += order[i] == least;
                }
            }
            if (!__any_sync(ALL, any)) continue;
            int before = equal;                 // equal ones in the group's lower lanes
            for (int o = 1; o < width; o <<= 1) {
                const int up = __shfl_up_sync(ALL, before, o, width);
                if ((lane & (width - 1)) >= o) before += up;
            }
            const int all = __shfl_sync(ALL, before, width - 1, width);
            before += equal_seen - equal;
            equal_seen += all;
            if (!any) continue;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (order[i] < least) continue;
                if (order[i] == least && before++ >= k) continue;
                const int at = atomicAdd(&sh.count, 1);
                if (at < CANDIDATES)
                    sh.list[at] = rank_key(order[i], (unsigned)(j * W + i - row.off));
            }
        }
    }
    __syncthreads();
    const int n = sh.count;
    if (n <= CANDIDATES) {
        // keys are unique: each one's place is the count of larger ones
        for (int a = tid; a < n; a += blockDim.x) {
            const uint64_t key = sh.list[a];
            int place = 0;
            for (int b = 0; b < n; ++b) place += sh.list[b] > key;
            if (place < k) sh.best[place] = key;
        }
    } else {
        uint64_t last = ~0ull;
        for (int round = 0; round < k; ++round) {
            uint64_t best = 0;
            for (int q = tid >> 5; q < chosen; q += warps) {
                const int64_t j0 = unit0 * 32 + ((int64_t)sh.chosen[q] << shift);
                const int64_t j1 = min(j0 + ((int64_t)1 << shift), j_end);
                for (int64_t j = j0 + lane; j < j1; j += 32) {
                    float f[W];
                    unpack(row.template load<Cache::KEEP>(j), f);
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const unsigned order = order_of(f[i]);
                        const uint64_t key = rank_key(order, (unsigned)(j * W + i - row.off));
                        if (order > 0 && key < last && key > best) best = key;
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(ALL, best, o));
            __syncthreads();                    // the list is free: its entries are not used here
            if (lane == 0) sh.list[tid >> 5] = best;
            __syncthreads();
            for (int w = 0; w < warps; ++w) best = max(best, sh.list[w]);
            last = best;
            if (tid == 0) sh.best[round] = best;
            if (best == 0) break;
        }
    }
    __syncthreads();
}

// A block (SPLIT: one of a cluster's blocks, each with an equal share of the
// units) per row.  Each warp takes UNITS accesses of 32 lanes at a time, its own
// running maximum as the base; the groups' maxima for the alternatives come
// from the same registers.  The bound is HBM (the row once).
template <typename T, bool TOP, bool SPLIT>
__global__ __launch_bounds__(32 * LP_WARPS, 4) void logprob_rows(LogprobParams p, int split,
                                                                 int shift) {
    constexpr int W = Row<T>::W;
    __shared__ RowShared sh;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, warps = blockDim.x >> 5;
    const int64_t r = SPLIT ? blockIdx.x / split : blockIdx.x;
    const int part = SPLIT ? blockIdx.x % split : 0;
    const T* x = static_cast<const T*>(p.logits) + r * p.ld;
    const Row<T> row(x, p.vocab);
    const int64_t all_units = (row.end + 32 * W - 1) / (32 * W);
    const int64_t share = SPLIT ? (all_units + split - 1) / split : all_units;
    const int64_t unit0 = part * share;
    const int64_t units = max((int64_t)0, min(share, all_units - unit0));
    const float c = p.alpha * LOG2E;
    const float lim = fminf(1e30f, 1e36f / c);      // |m| up to here: c m is far from overflow

    if (TOP) {
        sh.group_max[tid] = 0;
        __syncthreads();
    }
    Sums a{-INFINITY, 0.0f, 0.0f};
    float base = base_of(a.m, c, lim);
    for (int64_t t = (int64_t)w * UNITS; t < units; t += warps * UNITS) {
        Vec<T, W> v[UNITS];
        const int64_t j0 = (unit0 + t) * 32 + lane;
        if (t + UNITS <= units && row.whole(j0 - lane) && row.whole(j0 - lane + 32 * UNITS - 1)) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                v[i] = load_vec<TOP ? Cache::KEEP : Cache::STREAM, T, W>(row.from + (j0 + 32 * i) * W);
        } else {
            // past this part's units the accesses are taken from past the row: empty
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                v[i] = row.template load<Cache::KEEP>(
                    t + i < units ? j0 + 32 * i : (all_units + i) * 32 + lane);
        }
        float m = -INFINITY;
        if (TOP && shift >= 5) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const float um = warp_max(vec_max(v[i]));
                m = fmaxf(m, um);
                if (lane == 0 && t + i < units) {
                    unsigned* g = sh.group_max + ((t + i) >> (shift - 5));
                    if (shift == 5) *g = order_of(um);
                    else atomicMax(g, order_of(um));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                float gm = vec_max(v[i]);
                if (TOP && t + i < units) {     // groups narrower than a unit
                    for (int o = 1; o < 1 << shift; o <<= 1)
                        gm = fmaxf(gm, __shfl_xor_sync(ALL, gm, o));
                    if ((lane & ((1 << shift) - 1)) == 0)
                        sh.group_max[((t + i) * 32 + lane) >> shift] = order_of(gm);
                }
                m = fmaxf(m, gm);
            }
            m = warp_max(m);
        }
        if (m > a.m) {
            const float next = base_of(m, c, lim), d = base - next, e = exp2_approx(d);
            a.u = e * (a.u + (e > 0.0f ? d : 0.0f) * a.s);
            a.s *= e;
            a.m = m;
            base = next;
        }
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            float f[W];
            unpack(v[i], f);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                // far below the base 2^t is 0, and 0 * t must be 0 too; NaN stays NaN
                const float d = max_nan(fmaf(f[e], c, -base), -200.0f);
                const float q = exp2_approx(d);
                a.s += q;
                a.u = fmaf(q, d, a.u);
            }
        }
    }
    a.s = warp_sum(a.s);
    a.u = warp_sum(a.u);
    if (lane == 0) sh.sums[w] = a;
    __syncthreads();
    if (tid == 0) {
        a = sh.sums[0];
        for (int i = 1; i < warps; ++i) add(a, sh.sums[i], c, lim);
        sh.total = a;
    }
    if (TOP) choose(sh, row, unit0, units, shift, p.top_k);
    __syncthreads();
    a = sh.total;
    if constexpr (SPLIT) {
        // the first block joins the parts in order
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (part == 0) {
            for (int i = 1; i < split; ++i) add(a, cluster.map_shared_rank(&sh, i)->total, c, lim);
            if (TOP) {
                const int n = split * p.top_k;      // at most one key per thread
                uint64_t key = 0;
                if (tid < n) key = cluster.map_shared_rank(&sh, tid / p.top_k)->best[tid % p.top_k];
                __syncthreads();
                if (tid < n) sh.list[tid] = key;
                if (tid < p.top_k) sh.best[tid] = 0;
                __syncthreads();
                if (key != 0) {
                    int place = 0;
                    for (int i = 0; i < n; ++i) place += sh.list[i] > key;
                    if (place < p.top_k) sh.best[place] = key;
                }
                __syncthreads();
            }
        }
        cluster.sync();
        if (part != 0) return;
    }
    if (a.m > lim || (a.m < -lim && a.m > -INFINITY)) {
        // a maximum that the base cannot follow (the type's lowest value throughout, +inf):
        // the sums again, from the differences to it
        a.s = a.u = 0.0f;
        for (int64_t i = tid; i < p.vocab; i += blockDim.x) {
            const float v = to_f32(x[i]);
            const float d = max_nan((v - a.m) * c, -200.0f);
            const float q = exp2_approx(d);
            a.s += q;
            a.u = fmaf(q, d, a.u);
        }
        a.s = warp_sum(a.s);
        a.u = warp_sum(a.u);
        __syncthreads();
        if (lane == 0) sh.sums[w] = a;
        __syncthreads();
        a.s = a.u = 0.0f;
        for (int i = 0; i < warps; ++i) {
            a.s += sh.sums[i].s;
            a.u += sh.sums[i].u;
        }
        base = a.m * c;
    } else {
        base = base_of(a.m, c, lim);
    }
    // alpha m carries the bulk; the rest is what the base's rounding left of c m, and log2 S
    const bool none = a.s == 0.0f;                  // nothing unmasked (NaN is not 0)
    const float log_s = log2f(a.s);
    const float left = a.m > lim || a.m < -lim ? 0.0f : fmaf(-a.m, c, base);
    const float lse = none ? -INFINITY
                      : a.m == -INFINITY ? NAN      // NaNs alone
                                         : fmaf(p.alpha, a.m, LN2 * (log_s + left));
    if (tid == 0) {
        if (p.lse) p.lse[r] = lse;
        if (p.entropy) p.entropy[r] = none ? 0.0f : LN2 * (log_s - a.u / a.s);
        if (p.targets) {
            const int t = p.targets[r];
            float v = 0.0f;
            if (t >= 0 && t < p.vocab) v = none ? -INFINITY : fmaf(p.alpha, to_f32(x[t]), -lse);
            p.logprob[r] = v;
        }
    }
    if (TOP && tid < p.top_k) {
        const uint64_t key = sh.best[tid];
        const int64_t at = r * p.top_k + tid;
        p.top_index[at] = key ? (int)(0xffffffffu - (unsigned)key) : -1;
        p.top_logprob[at] = lse != lse ? NAN
                            : key ? fmaf(p.alpha, value_of((unsigned)(key >> 32)), -lse)
                                  : -INFINITY;
    }
}

template <typename T>
cudaError_t launch_forward(const LogprobParams& p, int num_sms, cudaStream_t st) {
    constexpr int UNIT = 32 * Row<T>::W;
    const int64_t units = (p.vocab + Row<T>::W + UNIT - 2) / UNIT;     // at most, by alignment
    // Few rows: several blocks share a row, as long as each has 8 units per warp.
    int split = 1;
    while (split < 8 && p.rows * split * 2 <= 2 * num_sms && units >= 64 * split) split *= 2;
    int64_t share = (units + split - 1) / split;
    // A warp per 8 units, so that narrow rows leave room for other rows' blocks.
    int warps = LP_WARPS;
    while (warps > 1 && share < 8 * warps / 2 && split == 1) warps /= 2;
    int shift = 0;
    while ((share * 32 + (1LL << shift) - 1) >> shift > 32 * warps) ++shift;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * split));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    auto kernel = p.top_k > 0
                      ? (split > 1 ? logprob_rows<T, true, true> : logprob_rows<T, true, false>)
                      : (split > 1 ? logprob_rows<T, false, true> : logprob_rows<T, false, false>);
    return cudaLaunchKernelEx(&cfg, kernel, p, split, shift);
}

// ---- gradient ---------------------------------------------------------------------------

constexpr int LG_THREADS = 256;
constexpr int LG_BATCH = 4;          // accesses in flight per thread

// dx = p * (-(up + de * entropy) - de * q) (+ up at the target), with alpha in up
// and de, q = alpha x - lse and p = exp(q).  Blocks (row, columns); W == 1 where
// logits and dlogits lie differently against 16-byte boundaries.  The bound is HBM
// (read x, write dx).
template <typename T, int W>
__global__ __launch_bounds__(LG_THREADS) void logprob_grad_rows(LogprobGradParams p) {
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.logits) + r * p.ld;
    T* dx = static_cast<T*>(p.dlogits) + r * p.ld_out;
    const Row<T> row(x, p.vocab);
    const int off = W > 1 ? row.off : 0;
    dx -= off;
    const int64_t end = off + p.vocab;
    const int64_t nvec = (end + W - 1) / W;
    const int step = blockDim.x;
    const float lse = p.lse[r];
    const int target = p.targets ? p.targets[r] : -1;
    const bool has = target >= 0 && target < p.vocab;
    const float up = has ? p.alpha * p.dlogprob[r] : 0.0f;
    const float de = p.dentropy ? p.alpha * p.dentropy[r] : 0.0f;
    const float k = p.dentropy ? -fmaf(de, p.entropy[r], up) : -up;
    const int64_t at_target = has ? (int64_t)target + off : -1;
    for (int64_t j0 = (int64_t)blockIdx.y * step * LG_BATCH + threadIdx.x; j0 < nvec;
         j0 += (int64_t)gridDim.y * step * LG_BATCH) {
        float f[LG_BATCH][W];
#pragma unroll
        for (int b = 0; b < LG_BATCH; ++b) {
            const int64_t j = j0 + (int64_t)b * step;
            if (j >= nvec) continue;
            if constexpr (W > 1) unpack(row.template load<Cache::STREAM>(j), f[b]);
            else f[b][0] = to_f32(x[j]);
        }
#pragma unroll
        for (int b = 0; b < LG_BATCH; ++b) {
            const int64_t j = j0 + (int64_t)b * step;
            if (j >= nvec) continue;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                // masked: p is 0, and 0 times the rest must be 0 too; NaN stays NaN
                const float q = max_nan(fmaf(p.alpha, f[b][i], -lse), -200.0f);
                const float e = exp2_approx(q * LOG2E);
                f[b][i] = lse == -INFINITY ? 0.0f : e * fmaf(-de, q, k);
            }
            if (at_target >= j * W && at_target < (j + 1) * W && lse != -INFINITY)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (j * W + i == at_target) f[b][i] += up;
            if (W == 1 || row.whole(j)) {
                store_vec<Cache::STREAM, T, W>(dx + j * W, f[b]);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (j * W + i >= off && j * W + i < end)
                        dx[j * W + i] = from_f32<T>(f[b][i]);
            }
        }
    }
}

template <typename T, int W>
cudaError_t launch_grad(const LogprobGradParams& p, cudaStream_t st) {
    const int64_t nvec = (p.vocab + 2 * (W - 1)) / W;                  // at most, by alignment
    int threads = LG_THREADS;
    while (threads > 64 && nvec <= threads / 2 * LG_BATCH) threads /= 2;
    const int64_t pieces = (nvec + threads * LG_BATCH - 1) / (threads * LG_BATCH);
    const dim3 grid((unsigned)p.rows, (unsigned)std::min<int64_t>(pieces, 65535));
    logprob_grad_rows<T, W><<<grid, threads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprob(spmm_type_t type, const LogprobParams& p, int num_sms,
                                 cudaStream_t st) {
    return with_type(type, [&](auto t) { return launch_forward<decltype(t)>(p, num_sms, st); });
}

cudaError_t launch_token_logprob_grad(spmm_type_t type, const LogprobGradParams& p, int num_sms,
                                      cudaStream_t st) {
    (void)num_sms;
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        const uintptr_t a = reinterpret_cast<uintptr_t>(p.logits);
        const uintptr_t b = reinterpret_cast<uintptr_t>(p.dlogits);
        // every row the same distance from a 16-byte boundary in both
        const bool alike = a % 16 == b % 16 && (p.ld - p.ld_out) * (int64_t)sizeof(T) % 16 == 0;
        return alike ? launch_grad<T, 16 / (int)sizeof(T)>(p, st) : launch_grad<T, 1>(p, st);
    });
}

}  // namespace spmm
