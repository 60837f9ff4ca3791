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

#include "spmm_internal.h"
#include "spmm_lm_device.cuh"

namespace spmm {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned ALL = 0xffffffffu;
constexpr float LN2 = 0.6931471805599453f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LARGEST = 3.402823466e38f;

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

// Largest elements of accesses, NaNs left out, packed as the elements are; and
// the accesses' elements kept from falling below `low` (NaN stays NaN).
template <typename T>
struct Largest {
    using Pair = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    Pair m, low;

    __device__ explicit Largest(float least) : m(both(-INFINITY)), low(both(least)) {}
    __device__ static Pair both(float x) {
        if constexpr (std::is_same_v<T, __half>) return __float2half2_rn(x);
        else return __float2bfloat162_rn(x);
    }
    __device__ void see(const Vec<T, 8>& v) {
        const Pair* x = reinterpret_cast<const Pair*>(v.w);
        m = __hmax2(m, __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3])));
    }
    __device__ float value() const { return fmaxf(__low2float(m), __high2float(m)); }
    __device__ void floor(const Vec<T, 8>& v, float (&f)[8]) const {
        Vec<T, 8> r;
        const Pair* x = reinterpret_cast<const Pair*>(v.w);
        Pair* y = reinterpret_cast<Pair*>(r.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __hmax2_nan(x[i], low);
        unpack(r, f);
    }
};
template <>
struct Largest<float> {
    float m, low;

    __device__ explicit Largest(float least) : m(-INFINITY), low(least) {}
    __device__ void see(const Vec<float, 4>& v) {
        float f[4];
        unpack(v, f);
        m = fmaxf(m, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
    }
    __device__ float value() const { return m; }
    __device__ void floor(const Vec<float, 4>& v, float (&f)[4]) const {
        unpack(v, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = max_nan(f[i], low);
    }
};

// ---- forward --------------------------------------------------------------------------

constexpr int LP_WARPS = 8;                     // at most
constexpr int UNITS = 4;                        // accesses in flight per lane
constexpr int CANDIDATES = SPMM_TOP_MAX * SPMM_TOP_MAX;

// Sums of a part of a row.  The base is c * max(m, low), rounded: every use must see
// the same number, so the product may not become part of a fused multiply-add.
struct Sums {
    float m, s, u;
};
__device__ __forceinline__ float base_of(float m, float c, float low) {
    return __fmul_rn(fmaxf(m, low), c);
}
// A part's sums from its own base to the one `d` above it (d <= 0).
__device__ __forceinline__ void rebase(float& s, float& u, float d) {
    const float e = exp2_approx(d);
    u = e * fmaf(fmaxf(d, -200.0f), s, u);      // no weight is left long before -200
    s *= e;
}
// The warp's lanes' sums, each from its own base, to the base of their maximum.
__device__ __forceinline__ Sums join(Sums a, float c, float low) {
    const float m = warp_max(a.m);
    rebase(a.s, a.u, base_of(a.m, c, low) - base_of(m, c, low));
    return {m, warp_sum(a.s), warp_sum(a.u)};
}

// From here on a logit's and lse's last places (1/8) count beside the logarithms that tell them
// apart.  z = alpha x is a binary32 number there, like lse: the places that it has lost would
// otherwise show in z - lse (equal logits of 1e37 would differ from their lse by 1e29).  Below,
// alpha x joins a sum in one rounding, which is closer to the exact one.
constexpr float LARGE = 1048576.0f;
// Log probability of a logit.  One that alpha takes below binary32's range is masked, whatever
// lse would make of it.
__device__ __forceinline__ float log_p(float alpha, float x, float lse) {
    const float z = __fmul_rn(alpha, x);
    return fabsf(z) < LARGE ? fmaf(alpha, x, -lse) : z - lse;
}

struct RowShared {
    Sums sums[LP_WARPS];
    Sums total;                                 // this block's part of the row
    uint64_t best[SPMM_TOP_MAX];                // its alternatives, largest first (0: none)
    unsigned short chosen[32 * LP_WARPS * UNITS];   // groups that hold the alternatives
    int chosen_count;
    int count;
    unsigned bound[LP_WARPS];                   // a number that some of the warp's lanes reach
    uint64_t list[CANDIDATES];
};

// How a block's threads share its part of a row: units of 32 accesses, each warp
// UNITS at a time.  The i-th accesses of thread t's turns are group t * UNITS + i.
struct Part {
    int64_t unit0, units;
    int warps;
    __device__ int64_t turns() const { return (units + (int64_t)warps * UNITS - 1) / (warps * UNITS); }
    // the q-th access of group g (past the end of the part: -1)
    __device__ int64_t access(int g, int64_t q) const {
        const int64_t unit = (q * warps + g / (32 * UNITS)) * UNITS + g % UNITS;
        return unit < units ? (unit0 + unit) * 32 + g / UNITS % 32 : -1;
    }
};

// Adds the elements of order >= least among the accesses of the chosen groups to
// the list of candidates.  The block's threads share those accesses, four at a time.
template <typename T>
__device__ void collect(RowShared& sh, const Row<T>& row, const Part& part, int chosen,
                        unsigned least) {
    constexpr int W = Row<T>::W;
    // in values: NaN and -inf compare false, and what is no number's order means all
    const float from = least > 0x00800000u ? value_of(least) : -LARGEST;
    const int own = (int)part.turns();              // accesses of a group, at most
    const int all = chosen * own;
    for (int i0 = threadIdx.x; i0 < all; i0 += 4 * blockDim.x) {
        Vec<T, W> v[4];
        int64_t j[4];
        bool all_whole = true;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = i0 + b * blockDim.x;
            j[b] = i < all ? part.access(sh.chosen[i / own], i % own) : -1;
            all_whole &= j[b] < 0 || row.whole(j[b]);
        }
        // an access behind a branch would keep the others waiting: those past the end are
        // read in vain
        if (all_whole && row.whole(1)) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                v[b] = load_vec<Cache::KEEP, T, W>(row.from + (j[b] < 0 ? 1 : j[b]) * W);
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (j[b] >= 0) v[b] = row.template load<Cache::KEEP>(j[b]);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (j[b] < 0) continue;
            Largest<T> top(0.0f);
            top.see(v[b]);
            if (!(top.value() >= from)) continue;
            float f[W];
            unpack(v[b], f);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (!(f[i] >= from)) continue;
                const int at = atomicAdd(&sh.count, 1);
                if (at < CANDIDATES)
                    sh.list[at] = rank_key(order_of(f[i]), (unsigned)(j[b] * W + i - row.off));
            }
        }
    }
}

// The `many`-th largest of the lanes' values (0: that many have none).
__device__ __forceinline__ unsigned warp_nth(unsigned x, int many, int lane) {
    unsigned m = 0;
    for (int i = 0; i < many; ++i) {
        m = __reduce_max_sync(ALL, x);
        if (lane == __ffs(__ballot_sync(ALL, x == m)) - 1) x = 0;
    }
    return m;
}

// A number that at least k threads' values reach (0: fewer have any), bit by bit from
// what is known of it, `bit` the next to look at.  ENOUGH: until exactly k reach it, else
// to the end: the k-th largest itself.
template <bool ENOUGH>
__device__ __forceinline__ unsigned block_nth(unsigned x, int k, unsigned tau, int bit) {
    int reach = 0;
    for (; bit >= 0 && !(ENOUGH && reach == k); --bit) {
        const unsigned next = tau | 1u << bit;
        const int n = __syncthreads_count(x >= next);
        if (n < k) continue;
        tau = next;
        reach = n;
    }
    return tau;
}

// The alternatives of this block's part of the row, into sh.best.
//
// group[i] is the order of the largest logit of this thread's i-th group, `mine` the
// largest of them.  A number tau that the largest logits of k threads reach is a lower
// bound of the k-th largest logit, and every logit that reaches it belongs to a group
// whose largest does.  So a second look (in L2) at those groups, few of the block's
// 1024, gives a short list that holds the alternatives; its entries are ranked by
// counting.  tau is searched until exactly k threads reach it.  QUICK: it is the least
// of the warps' n-th largest, n their share of k (sh.bound, before the call's barrier):
// fewer barriers for some more groups, which pays where a call is short (8 rows of 131,072
// bf16: 7.7 us, 8.6 without) and costs where it is not (4099 rows of 50,001: 154, 146
// without).
// When more than CANDIDATES logits reach tau, it is raised to the k-th largest of the
// threads' largest, which nearly all of them must equal then: the list is made of those
// above tau, and the first equal ones in index order.
template <typename T, bool QUICK>
__device__ void choose(RowShared& sh, const Row<T>& row, const Part& part,
                       const unsigned (&group)[UNITS], unsigned mine, int k) {
    constexpr int W = Row<T>::W;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    unsigned tau;
    if constexpr (QUICK) {
        tau = sh.bound[0];
        for (int i = 1; i < part.warps; ++i) tau = min(tau, sh.bound[i]);
        // a warp without enough logits (past the row's end, masked) says nothing of the others
        if (tau == 0) tau = block_nth<true>(mine, k, 0, 31);
    } else {
        // from the bits that all threads' values have in common
        const unsigned wmax = __reduce_max_sync(ALL, mine), wmin = __reduce_min_sync(ALL, mine);
        if (lane == 0) sh.list[w] = (uint64_t)wmax << 32 | wmin;
        __syncthreads();
        unsigned most = wmax, fewest = wmin;
        for (int i = 0; i < part.warps; ++i) {
            most = max(most, (unsigned)(sh.list[i] >> 32));
            fewest = min(fewest, (unsigned)sh.list[i]);
        }
        const int bit = most == fewest ? -1 : 31 - __clz(most ^ fewest);
        tau = bit < 0 ? most : bit == 31 ? 0 : most >> (bit + 1) << (bit + 1);
        tau = block_nth<true>(mine, k, tau, bit);
        __syncthreads();                            // the list is free again
    }
    const unsigned least = max(tau, 1u);
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
        if (group[i] >= least)
            sh.chosen[atomicAdd(&sh.chosen_count, 1)] = (unsigned short)(tid * UNITS + i);
    __syncthreads();
    const int chosen = sh.chosen_count;
    collect(sh, row, part, chosen, least);
    __syncthreads();
    if (sh.count > CANDIDATES) {
        tau = block_nth<false>(mine, k, 0, 31);
        __syncthreads();
        if (tid == 0) sh.count = 0;
        __syncthreads();
        collect(sh, row, part, chosen, max(tau, 1u) + 1);
        __syncthreads();
        const int above = sh.count;
        __syncthreads();
        if (above > CANDIDATES) {
            // many far above the others, all in a few threads' hands: k rounds of the
            // largest one left
            const int own = (int)part.turns();
            uint64_t last = ~0ull;
            for (int round = 0; round < k; ++round) {
                uint64_t best = 0;
                for (int g = w; g < chosen; g += part.warps)
                    for (int q = lane; q < own; q += 32) {
                        const int64_t j = part.access(sh.chosen[g], q);
                        if (j < 0) continue;
                        float f[W];
                        unpack(row.template load<Cache::KEEP>(j), f);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const unsigned order = order_of(f[i]);
                            const uint64_t key =
                                rank_key(order, (unsigned)(j * W + i - row.off));
                            if (order > 0 && key < last && key > best) best = key;
                        }
                    }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(ALL, best, o));
                if (lane == 0) sh.list[w] = best;
                __syncthreads();
                for (int i = 0; i < part.warps; ++i) best = max(best, sh.list[i]);
                __syncthreads();
                last = best;
                if (tid == 0) sh.best[round] = best;
            }
            __syncthreads();
            return;
        }
        if (w == 0 && tau > 0) {
            // the equal ones, in index order until there are enough
            int have = above;
            for (int64_t u = 0; u < part.units && have < k; ++u) {
                const int64_t j = (part.unit0 + u) * 32 + lane;
                float f[W];
                unpack(row.template load<Cache::KEEP>(j), f);
                int equal = 0;
#pragma unroll
                for (int i = 0; i < W; ++i) equal += order_of(f[i]) == tau;
                int at = equal;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(ALL, at, o);
                    if (lane >= o) at += up;
                }
                const int all = __shfl_sync(ALL, at, 31);
                at += have - equal;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (order_of(f[i]) == tau) {
                        if (at < k) sh.list[at] = rank_key(tau, (unsigned)(j * W + i - row.off));
                        ++at;
                    }
                have += all;
            }
            if (lane == 0) sh.count = max(above, min(have, k));
        }
        __syncthreads();
    }
    // keys are unique: each one's place is the count of larger ones
    const int n = sh.count;
    for (int a = tid; a < n; a += blockDim.x) {
        const uint64_t key = sh.list[a];
        int place = 0;
#pragma unroll 4
        for (int b = 0; b < n; ++b) place += sh.list[b] > key;
        if (place < k) sh.best[place] = key;
    }
}

// A block (SPLIT: one of a cluster's blocks, each with an equal share of the
// units) per row.  Each lane takes UNITS accesses at a time and keeps its own
// running maximum, base and sums, so the loop has no exchange between lanes; the
// same maxima serve the choice of the alternatives.  The bound is HBM (the row
// once) while an element costs under about 9 instructions: 16-bit maxima and the floor
// are taken two at a time before unpacking, products and sums two at a time after.
// 8192 rows of 131,072 bf16: 308 us without alternatives (the copy rate), 372 us with 20
// (85%): between a row's last access and the next row's first the block ranks, and the
// SM's other blocks are not enough to fill that time.  8 rows with 8: 7.7 us in clusters
// of 8 blocks.
template <typename T, bool TOP, bool SPLIT>
__global__ __launch_bounds__(32 * LP_WARPS, 4) void logprob_rows(LogprobParams p, int split) {
    constexpr int W = Row<T>::W;
    __shared__ RowShared sh;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, warps = blockDim.x >> 5;
    const int64_t r = SPLIT ? blockIdx.x / split : blockIdx.x;
    const int rank = SPLIT ? blockIdx.x % split : 0;
    const T* x = static_cast<const T*>(p.logits) + r * p.ld;
    const Row<T> row(x, p.vocab);
    const int64_t all_units = (row.end + 32 * W - 1) / (32 * W);
    const int64_t share = SPLIT ? (all_units + split - 1) / split : all_units;
    Part part{rank * share, 0, warps};
    part.units = max((int64_t)0, min(share, all_units - part.unit0));
    const float c = fminf(p.alpha * LOG2E, LARGEST);
    // the target's logit, wanted at the end
    const int target = tid == 0 && p.targets ? p.targets[r] : -1;
    const bool has_target = target >= 0 && target < p.vocab;
    const float target_logit = has_target ? to_f32(x[target]) : 0.0f;
    // logits up to here: c x is rounded by less than 1/16, so that a difference of two
    // equal ones, one of them rounded, stays small
    const float lim = fminf(1e30f, 1e6f / c);

    // Masked logits, and all that are lower, count as `low`, far below the base: 2^t is
    // 0 there and 0 * t is 0.  (Lanes that see nothing else count them in full, but
    // lose them on the way to the row's base.)
    const float low =
        to_f32(from_f32<T>(std::is_same_v<T, __half> ? fmaxf(-lim, -65504.0f) : -lim));
    Largest<T> top[UNITS] = {Largest<T>(low), Largest<T>(low), Largest<T>(low), Largest<T>(low)};
    static_assert(UNITS == 4);
    Sums a{-INFINITY, 0.0f, 0.0f};
    float base = base_of(a.m, c, low);
    uint64_t s2 = pair(0.0f, 0.0f), u2 = s2;
    const uint64_t c2 = pair(c, c);
    for (int64_t t = (int64_t)w * UNITS; t < part.units; t += warps * UNITS) {
        Vec<T, W> v[UNITS];
        const int64_t j0 = (part.unit0 + t) * 32 + lane;
        if (t + UNITS <= part.units && row.whole(j0 - lane) &&
            row.whole(j0 - lane + 32 * UNITS - 1)) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                v[i] = load_vec<TOP ? Cache::KEEP : Cache::STREAM, T, W>(row.from + (j0 + 32 * i) * W);
        } else {
            // past this part's units the accesses are taken from past the row: empty
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                v[i] = row.template load<Cache::KEEP>(
                    t + i < part.units ? j0 + 32 * i : (all_units + i) * 32 + lane);
        }
#pragma unroll
        for (int i = 0; i < UNITS; ++i) top[TOP ? i : 0].see(v[i]);
        float m = top[0].value();
        if (TOP)
#pragma unroll
            for (int i = 1; i < UNITS; ++i) m = fmaxf(m, top[i].value());
        if (m > a.m) {
            const float next = base_of(m, c, low);
            float s0, s1, u0, u1;
            halves(s2, s0, s1);
            halves(u2, u0, u1);
            rebase(s0, u0, base - next);
            rebase(s1, u1, base - next);
            s2 = pair(s0, s1);
            u2 = pair(u0, u1);
            a.m = m;
            base = next;
        }
        const uint64_t b2 = pair(-base, -base);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            float f[W];
            top[0].floor(v[i], f);
#pragma unroll
            for (int e = 0; e < W; e += 2) {
                const uint64_t d2 = fma2(pair(f[e], f[e + 1]), c2, b2);
                float d0, d1;
                halves(d2, d0, d1);
                const uint64_t q2 = pair(exp2_approx(d0), exp2_approx(d1));
                s2 = add2(s2, q2);
                u2 = fma2(q2, d2, u2);
            }
        }
    }
    {
        float s0, s1, u0, u1;
        halves(s2, s0, s1);
        halves(u2, u0, u1);
        a.s = s0 + s1;
        a.u = u0 + u1;
    }
    a = join(a, c, low);
    if (lane == 0) sh.sums[w] = a;
    unsigned group[UNITS], mine = 0;
    if constexpr (TOP) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            group[i] = order_of(top[i].value());
            mine = max(mine, group[i]);
        }
        if constexpr (SPLIT) {
            const unsigned bound = warp_nth(mine, (p.top_k + warps - 1) / warps, lane);
            if (lane == 0) sh.bound[w] = bound;
        }
        if (tid < p.top_k) sh.best[tid] = 0;
        if (tid == 0) sh.chosen_count = sh.count = 0;
    }
    __syncthreads();
    if (w == 0) {
        a = join(lane < warps ? sh.sums[lane] : Sums{-INFINITY, 0.0f, 0.0f}, c, low);
        if (lane == 0) sh.total = a;
    }
    if constexpr (TOP) choose<T, SPLIT>(sh, row, part, group, mine, p.top_k);
    __syncthreads();
    a = sh.total;
    if constexpr (SPLIT) {
        // the first block joins the parts
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (rank == 0) {
            a = join(lane < split ? cluster.map_shared_rank(&sh, lane)->total
                                  : Sums{-INFINITY, 0.0f, 0.0f}, c, low);
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
        if (rank != 0) return;
    }
    const bool far =
        a.m > lim || (a.m > -INFINITY && ((a.m - low) * c < 200.0f || c == LARGEST));
    if (far) {
        // a maximum that the base cannot follow (+inf, huge values) or that is not far above
        // `low` (the type's lowest value throughout), or a c that was cut (alpha over 2.3e38):
        // the sums again, from the differences to it
        a.s = a.u = 0.0f;
        for (int64_t i = tid; i < p.vocab; i += blockDim.x) {
            const float v = to_f32(x[i]);
            const float d = max_nan((v - a.m) * p.alpha * LOG2E, -200.0f);
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
    }
    // alpha m carries the bulk; the rest is what the base's rounding left of c m, and log2 S.
    // A maximum that alpha takes beyond binary32 counts as infinite: below, the row has
    // nothing unmasked; above, it is NaN, as a row of NaNs alone (m = -inf) is.
    const float z = __fmul_rn(p.alpha, a.m);
    const bool none = z == -INFINITY && a.s == a.s;      // and no NaN
    const bool nan = !none && !(fabsf(z) < INFINITY);
    const float log_s = log2f(a.s);
    const float left = far ? 0.0f : fmaf(-a.m, c, base_of(a.m, c, low));
    const float above = LN2 * (log_s + left);
    const float lse = none               ? -INFINITY
                      : nan              ? NAN
                      : fabsf(z) < LARGE ? fmaf(p.alpha, a.m, above)
                                         : z + above;
    if (tid == 0) {
        if (p.lse) p.lse[r] = lse;
        if (p.entropy) p.entropy[r] = none ? 0.0f : nan ? NAN : LN2 * (log_s - a.u / a.s);
        if (p.targets)
            p.logprob[r] = !has_target ? 0.0f : none ? -INFINITY : log_p(p.alpha, target_logit, lse);
    }
    if (TOP && tid < p.top_k) {
        const uint64_t key = sh.best[tid];
        const float logit = value_of((unsigned)(key >> 32));
        const bool there = key && __fmul_rn(p.alpha, logit) > -INFINITY;
        const int64_t at = r * p.top_k + tid;
        p.top_index[at] = there ? (int)(0xffffffffu - (unsigned)key) : -1;
        p.top_logprob[at] = lse != lse ? NAN : there ? log_p(p.alpha, logit, lse) : -INFINITY;
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
    // Enough units per warp to carry a row's fixed cost (eight turns; two when the SMs are
    // not full and the shortest call is wanted): fewer warps leave room for other rows.
    // 4096 rows of 50,001 bf16: 95 us with 8 warps, 82 with 4; 16,384 rows of 1500 f32:
    // 50 us with 2 warps, 39 with 1.
    int warps = LP_WARPS;
    const int64_t least = p.rows >= 4 * num_sms ? 8 * UNITS : 2 * UNITS;
    // the choice wants twice as many lanes as alternatives, and all it can get for few rows
    const int most = p.rows >= 4 * num_sms ? (2 * p.top_k + 31) / 32 : p.top_k > 0 ? LP_WARPS : 1;
    while (warps > most && warps > 1 && share < least * warps && split == 1) warps /= 2;
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
    return own_error(cudaLaunchKernelEx(&cfg, kernel, p, split));
}

// ---- gradient ---------------------------------------------------------------------------

constexpr int LG_THREADS = 256;
constexpr int LG_BATCH = 4;          // accesses in flight per thread

// The columns c, c + stride, ... of a row whose lse is LARGE.  Seldom, and not inlined: a second
// form of the loop below would take its registers (8192 x 131,072 bf16 712 us, 683 with a
// choice at each element).
template <typename T>
__device__ __noinline__ void grad_one_by_one(const T* x, T* dx, int64_t vocab, int64_t c,
                                             int64_t stride, float alpha, float lse, float de,
                                             float k, int target, float up) {
    for (; c < vocab; c += stride) {
        const float q = max_nan(__fmul_rn(alpha, to_f32(x[c])) - lse, -200.0f);
        const float d = exp2_approx(q * LOG2E) * fmaf(-de, q, k);
        dx[c] = from_f32<T>(c == target ? d + up : d);
    }
}

// dx = p * (-(up + de * entropy) - de * q) (+ up at the target), with alpha in up
// and de, q = z - lse (z = alpha x, a binary32 number where lse is LARGE) and
// p = exp(q).  A row takes `pieces` consecutive blocks, so that blocks in flight
// together work on neighbouring memory; W == 1 where logits and dlogits lie
// differently against 16-byte boundaries.  The bound is HBM (read x, write dx): 8192 rows of 131,072 bf16 645 us, 6.7 TB/s (98% of
// the copy rate; 986 us when each access was unpacked before the next was sent).
template <typename T, int W>
__global__ __launch_bounds__(LG_THREADS) void logprob_grad_rows(LogprobGradParams p, int pieces) {
    const int64_t r = blockIdx.x / pieces;
    const int piece = blockIdx.x % pieces;
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
    const bool empty = lse == -INFINITY;
    if (fabsf(lse) >= LARGE && !empty) {
        grad_one_by_one(x, dx + off, p.vocab, (int64_t)piece * step + threadIdx.x,
                        (int64_t)pieces * step, p.alpha, lse, de, k, has ? target : -1, up);
        return;
    }
    for (int64_t j0 = (int64_t)piece * step * LG_BATCH + threadIdx.x; j0 < nvec;
         j0 += (int64_t)pieces * step * LG_BATCH) {
        Vec<T, W> v[LG_BATCH];       // packed until all are on their way
#pragma unroll
        for (int b = 0; b < LG_BATCH; ++b) {
            const int64_t j = j0 + (int64_t)b * step;
            if (j >= nvec) continue;
            if constexpr (W > 1) v[b] = row.template load<Cache::STREAM>(j);
            else v[b].w = x[j];
        }
#pragma unroll
        for (int b = 0; b < LG_BATCH; ++b) {
            const int64_t j = j0 + (int64_t)b * step;
            if (j >= nvec) continue;
            float f[W];
            unpack(v[b], f);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                // masked: p is 0, and 0 times the rest must be 0 too; NaN stays NaN
                const float q = max_nan(fmaf(p.alpha, f[i], -lse), -200.0f);
                f[i] = exp2_approx(q * LOG2E) * fmaf(-de, q, k);
            }
            const int64_t hit = at_target - j * W;
            if (hit >= 0 && hit < W)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i == hit) f[i] += up;
            if (empty)
#pragma unroll
                for (int i = 0; i < W; ++i) f[i] = 0.0f;
            if (W == 1 || row.whole(j)) {
                store_vec<Cache::STREAM, T, W>(dx + j * W, f);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (j * W + i >= off && j * W + i < end)
                        dx[j * W + i] = from_f32<T>(f[i]);
            }
        }
    }
}

template <typename T, int W>
cudaError_t launch_grad(const LogprobGradParams& p, cudaStream_t st) {
    const int64_t nvec = (p.vocab + 2 * (W - 1)) / W;                  // at most, by alignment
    int threads = LG_THREADS;
    while (threads > 64 && nvec <= threads / 2 * LG_BATCH) threads /= 2;
    const int64_t whole = (nvec + threads * LG_BATCH - 1) / (threads * LG_BATCH);
    const int pieces = (int)std::max<int64_t>(1, std::min<int64_t>(whole, 0x7fffffff / p.rows));
    return launch(logprob_grad_rows<T, W>, (unsigned)(p.rows * pieces), threads, 0, st, p, pieces);
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
