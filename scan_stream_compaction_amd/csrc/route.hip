// The router of a mixture of experts: the experts of each token and their
// weights from a row of logits, how evenly the tokens fall on the experts, and
// the gradient. HIP kernels for MI355X (gfx950) and their part of the C ABI in
// include/ssc.h.
//
//   p = softmax(logits[t]),  ids = the `per` largest, weights = p[ids] (/ their sum)
//   counts[e] = assignments of expert e,  share[e] = mean of p[t, e] over the n live tokens
//   loss = E * sum over e of counts[e] / (per n) * share[e]
//   dlogits = p * (g - <p, g>),  g[e] = dloss * E * counts[e] / (per n) / n + dweights of e
//
// A row is held by G lanes of a wavefront (8 to 64), N logits each, so that
// one instruction serves 64 / G tokens and a sum over the row is three to six
// steps across lanes. The row is read once and stays in registers.
//
// Few tokens are bound by the launch: 16 of 8 of 128 bf16 2.6 us. Many by
// instructions and by HBM: 65,536 tokens, 8 of 128 fp32 with the balance, 17.7 us
// and 4.3 for the join (34 MB read, 4 written: 7 us at a copy's 5.15 TB/s; 5.9 M
// vector instructions, 1440 a wavefront for its 16 rows: 9.6 us at 2.4 GHz).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssc.h"
#include "ssc_device.h"
#include "ssc_host.h"

namespace ssc {
namespace {

constexpr int kRouteBlock = 256;
constexpr int64_t kExpertsMax = 1024;
constexpr int64_t kPerMax = 64;
constexpr int kIndexBits = 10;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1u;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2), may_alias));

// Which logits of a row a lane holds: chunks of kC consecutive ones, a group's
// chunks side by side, so that its lanes read consecutive addresses. Chunks of
// 16 bytes that the row ends in start early, so that every load is whole and
// none waits behind a branch; what they share with the chunk before is not
// theirs.
template <class T, int G, int N>
struct Held {
    static constexpr int kC = N < 16 / static_cast<int>(sizeof(T)) ? N : 16 / static_cast<int>(sizeof(T));
    static constexpr int kChunks = N / kC;
    static constexpr bool kWide = kC * sizeof(T) == 16;  // of rows of at least that many logits
    typedef T V __attribute__((ext_vector_type(kC)));
    struct Narrow {
        T e[kC];
    };
    using Raw = std::conditional_t<kWide, u32x4, Narrow>;
    int n, sub, start[kChunks];

    __device__ __forceinline__ Held(int sub, int n) : n(n), sub(sub) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) start[c] = kWide && at(c) > n - kC ? n - kC : at(c);
    }
    __device__ __forceinline__ int at(int c) const { return (c * G + sub) * kC; }
    // the expert of logit j, and whether it is this lane's
    __device__ __forceinline__ int index(int j) const { return start[j / kC] + j % kC; }
    __device__ __forceinline__ bool own(int j) const {
        const int i = index(j);
        return kWide ? i >= at(j / kC) : i < n;
    }
    // every lane's chunk lies inside the row (the same in all lanes)
    __device__ __forceinline__ bool whole(int c) const { return (c + 1) * G * kC <= n; }

    __device__ __forceinline__ void fetch(const T *row, Raw (&raw)[kChunks]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if constexpr (kWide) {
                raw[c] = *reinterpret_cast<const u32x4_any *>(row + start[c]);
            } else {
#pragma unroll
                for (int e = 0; e < kC; ++e) raw[c].e[e] = row[start[c] + e < n ? start[c] + e : n - 1];
            }
        }
    }
    // a logit that is no number, or not this lane's, is as one of -infinity, and -0 as 0
    __device__ __forceinline__ void unpack(const Raw (&raw)[kChunks], float (&x)[N]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if constexpr (kWide) {
                const V v = __builtin_bit_cast(V, raw[c]);
#pragma unroll
                for (int e = 0; e < kC; ++e) x[c * kC + e] = static_cast<float>(v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < kC; ++e) x[c * kC + e] = static_cast<float>(raw[c].e[e]);
            }
            if (!whole(c)) {
#pragma unroll
                for (int j = c * kC; j < (c + 1) * kC; ++j) x[j] = own(j) ? x[j] : -__builtin_inff();
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = fmaxf(x[j] + 0.0f, -__builtin_inff());
    }
    __device__ __forceinline__ void store(T *row, const float (&x)[N]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (kWide && start[c] == at(c)) {
                V v;
#pragma unroll
                for (int e = 0; e < kC; ++e) v[e] = static_cast<T>(x[c * kC + e]);
                if constexpr (kWide) *reinterpret_cast<u32x4_any *>(row + start[c]) = __builtin_bit_cast(u32x4, v);
            } else {
#pragma unroll
                for (int j = c * kC; j < (c + 1) * kC; ++j)
                    if (own(j)) row[index(j)] = static_cast<T>(x[j]);
            }
        }
    }
};

// The value of another lane of the group: xor by 1 and 2 inside four lanes, the
// mirrored lane of 8 and 16 (the other half, once the halves are uniform), and
// of 32 and 64 by a shuffle.
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
    if constexpr (STEP == 1) return dpp_move<0xB1, 0xf>(v);
    if constexpr (STEP == 2) return dpp_move<0x4E, 0xf>(v);
    if constexpr (STEP == 4) return dpp_move<0x141, 0xf>(v);
    if constexpr (STEP == 8) return dpp_move<0x140, 0xf>(v);
    return static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), STEP));
}
template <int STEP>
__device__ __forceinline__ int32_t partner(int32_t v) {
    return static_cast<int32_t>(partner<STEP>(static_cast<uint32_t>(v)));
}
template <int STEP>
__device__ __forceinline__ float partner(float v) {
    return __uint_as_float(partner<STEP>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double partner(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    const uint64_t hi = partner<STEP>(static_cast<uint32_t>(b >> 32)), lo = partner<STEP>(static_cast<uint32_t>(b));
    return __longlong_as_double(static_cast<long long>(hi << 32 | lo));
}
template <int G, class V, class F>
__device__ __forceinline__ V over_group(V v, F f) {
    v = f(v, partner<1>(v));
    v = f(v, partner<2>(v));
    v = f(v, partner<4>(v));
    if constexpr (G > 8) v = f(v, partner<8>(v));
    if constexpr (G > 16) v = f(v, partner<16>(v));
    if constexpr (G > 32) v = f(v, partner<32>(v));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    return over_group<G>(v, [](float a, float b) { return a + b; });
}
// Sum over the groups of a wavefront, lane by lane.
template <int G>
__device__ __forceinline__ float over_groups(float v) {
    if constexpr (G <= 8) v += __uint_as_float(dpp_move<0x128, 0xf>(__float_as_uint(v)));  // 8 lanes on in each 16
    if constexpr (G <= 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (G <= 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
    return over_group<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// A logit (no NaN, no -0) and its expert in one number that is largest for the
// largest logit, the lowest expert of equal ones. A 16-bit logit's fp32 bits end in
// 13 zeros or more, which take the index; as signed integers, those of negative
// ones inverted but for the sign, they are in order.
template <class T>
struct Key {
    using K = int32_t;
    static constexpr uint32_t kInf = 0x7f800000u;
    __device__ static __forceinline__ uint32_t ordered(uint32_t b) {
        return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) & 0x7fffffffu);
    }
    __device__ static __forceinline__ K make(float x, int index) {
        return static_cast<K>((ordered(__float_as_uint(x)) & ~kIndexMask) | (kIndexMask - static_cast<uint32_t>(index)));
    }
    __device__ static __forceinline__ K none() { return INT32_MIN; }
    __device__ static __forceinline__ K larger(K a, K b) { return a > b ? a : b; }
    __device__ static __forceinline__ K smaller(K a, K b) { return a > b ? b : a; }
    // above those of -infinity, which end in other bits than 0
    __device__ static __forceinline__ bool expert(K k) { return k >= static_cast<K>(0x80800000u); }
    __device__ static __forceinline__ int index(K k) {
        return static_cast<int>(kIndexMask - (static_cast<uint32_t>(k) & kIndexMask));
    }
    __device__ static __forceinline__ float value(K k) {
        return __uint_as_float(ordered(static_cast<uint32_t>(k)) & ~kIndexMask);
    }
};
// An fp32 logit is the high half of a double, which orders such halves as floats
// (none reaches the exponent of NaN: that of infinity is 0x7f8 of 0x7ff), with the
// index behind it, inverted where the sign inverts the order. Maxima are one
// instruction.
template <>
struct Key<float> {
    using K = double;
    __device__ static __forceinline__ uint32_t high(K k) {
        return static_cast<uint32_t>(static_cast<uint64_t>(__double_as_longlong(k)) >> 32);
    }
    __device__ static __forceinline__ uint32_t low(K k) {
        return static_cast<uint32_t>(static_cast<uint64_t>(__double_as_longlong(k)));
    }
    __device__ static __forceinline__ K of(uint32_t hi, uint32_t lo) {
        return __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(hi) << 32 | lo));
    }
    __device__ static __forceinline__ K make(float x, int index) {
        const uint32_t b = __float_as_uint(x);
        return of(b, ~static_cast<uint32_t>(index) ^ static_cast<uint32_t>(static_cast<int32_t>(b) >> 31));
    }
    __device__ static __forceinline__ K none() { return of(0xff800000u, ~0u); }
    // no key is NaN, so the instructions are used as they are
    __device__ static __forceinline__ K larger(K a, K b) {
        K r;
        asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    __device__ static __forceinline__ K smaller(K a, K b) {
        K r;
        asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    __device__ static __forceinline__ bool expert(K k) { return high(k) != 0xff800000u; }
    __device__ static __forceinline__ int index(K k) {
        return static_cast<int>(~(low(k) ^ static_cast<uint32_t>(static_cast<int32_t>(high(k)) >> 31)));
    }
    __device__ static __forceinline__ float value(K k) { return __uint_as_float(high(k)); }
};

// a where mask is 0, b where it is all ones (a choice by a condition between
// two elements of an array becomes an index into it, and that sixteen selects)
__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t a, uint32_t b) { return a ^ ((a ^ b) & mask); }
__device__ __forceinline__ int32_t pick(uint32_t mask, int32_t a, int32_t b) {
    return static_cast<int32_t>(pick(mask, static_cast<uint32_t>(a), static_cast<uint32_t>(b)));
}
__device__ __forceinline__ double pick(uint32_t mask, double a, double b) {
    const uint64_t x = static_cast<uint64_t>(__double_as_longlong(a)), y = static_cast<uint64_t>(__double_as_longlong(b));
    const uint32_t lo = pick(mask, static_cast<uint32_t>(x), static_cast<uint32_t>(y));
    const uint32_t hi = pick(mask, static_cast<uint32_t>(x >> 32), static_cast<uint32_t>(y >> 32));
    return __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(hi) << 32 | lo));
}

template <class Q>
__device__ __forceinline__ void exchange(typename Q::K &a, typename Q::K &b) {
    const auto big = Q::larger(a, b);
    b = Q::smaller(a, b);
    a = big;
}

// Of two runs of TOP keys, largest first, the larger half, again in order.
template <class Q, int TOP, class F>
__device__ __forceinline__ void merge_keys(typename Q::K *k, F other) {
#pragma unroll
    for (int i = 0; i < TOP / 2; ++i) {
        const auto a = Q::larger(k[i], other(TOP - 1 - i)), b = Q::larger(k[TOP - 1 - i], other(i));
        k[i] = a;
        k[TOP - 1 - i] = b;
    }
#pragma unroll
    for (int h = TOP / 2; h >= 1; h /= 2) {
#pragma unroll
        for (int i = 0; i < TOP; ++i)
            if ((i & h) == 0) exchange<Q>(k[i], k[i + h]);
    }
}

// The TOP largest keys of a lane's N, largest first, in its first places: runs
// of TOP sorted by merging of odd and even places, and merged (8 of 16: 2 x 19
// exchanges, 8 maxima and 12 exchanges).
template <class Q, int N, int TOP>
__device__ __forceinline__ void sort_keys(typename Q::K (&k)[N]) {
#pragma unroll
    for (int run = 0; run < N; run += TOP) {
#pragma unroll
        for (int p = 1; p < TOP; p *= 2) {
#pragma unroll
            for (int h = p; h >= 1; h /= 2) {
#pragma unroll
                for (int j = h % p; j + h < TOP; j += 2 * h) {
#pragma unroll
                    for (int i = 0; i < h; ++i) {
                        const int a = j + i, b = j + i + h;
                        if (b < TOP && a / (2 * p) == b / (2 * p)) exchange<Q>(k[run + a], k[run + b]);
                    }
                }
            }
        }
        if (run > 0) merge_keys<Q, TOP>(k, [&](int i) { return k[run + i]; });
    }
}

// The TOP largest of the group's, largest first, in every lane of it.
template <class Q, int G, int TOP, int STEP = 1>
__device__ __forceinline__ void merge_group(typename Q::K *k) {
    if constexpr (STEP < G) {
        typename Q::K other[TOP];
#pragma unroll
        for (int i = 0; i < TOP; ++i) other[i] = partner<STEP>(k[i]);
        merge_keys<Q, TOP>(k, [&](int i) { return other[i]; });
        merge_group<Q, G, TOP, 2 * STEP>(k);
    }
}

// A row of logits as exponentials of their distance from the largest: 2^((x -
// top) log2(e)), off by 2.3 |x - top| half steps of fp32 for the difference,
// the product and the constant, and by 2 for the exponential. Beside a logit of
// +infinity no other counts. A row without experts has none (sum 0).
template <int G, int N>
struct Softmax {
    float top, sum, inv;
    bool lift;

    __device__ __forceinline__ float lifted(float x) const {
        return lift ? (x == __builtin_inff() ? 0.0f : -__builtin_inff()) : x;
    }
    // x as lifted: the largest is finite, and -infinity gives 0
    __device__ __forceinline__ float weight(float x) const {
        return __builtin_amdgcn_exp2f((x - top) * 1.44269504088896340736f);
    }
    __device__ __forceinline__ void make(float (&x)[N], float (&e)[N]) {
        float m = x[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = fmaxf(m, x[j]);
        top = fmaxf(group_max<G>(m), -0x1.fffffep127f);
        lift = top == __builtin_inff();
        if (__builtin_expect(ballot(lift) != 0, 0)) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = lifted(x[j]);
            if (lift) top = 0.0f;
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            e[j] = weight(x[j]);
            s += e[j];
        }
        sum = group_sum<G>(s);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
};

struct RouteArgs {
    const void *logits;
    int64_t stride, tokens;
    const uint8_t *live;
    int experts, per;
    bool normalize;
    int32_t *ids;
    float *weights;
    // scratch of the balance: each workgroup's sums of p and assignments, its live
    // tokens behind them; and how many workgroups of the join are done
    float *part_share;
    int32_t *part_count;
    double *part_loss;
    uint32_t *done;
    // the results, where one workgroup has all of the tokens
    int32_t *counts;
    float *share, *loss;
};

// With the balance a workgroup adds up its tokens' softmax, so it is larger and
// there are fewer: as many threads as the registers of N logits allow.
template <int N, bool BALANCE>
constexpr int kThreads = !BALANCE ? kRouteBlock : (N > 16 ? 512 : 1024);

// MERGE: up to TOP are chosen, 4 or 8, and the lanes' runs of them are merged
// (48 instructions a step for 8 of fp32); otherwise TOP = N, and each is found by a
// maximum over the heads of the lanes' runs, and taken off its run (32 and more).
// 65,536 tokens without the balance, fp32 and bf16: 8 of 256 18.0 and 15.9 us, 16 of 256
// 43.5 and 23.1, 10 of 512 66.5 and 36.8 (139 MB of fp32: 27 at a copy's rate).
template <class T, int G, int N, int TOP, bool MERGE, bool BALANCE>
__global__ __launch_bounds__((kThreads<N, BALANCE>)) void route_kernel(RouteArgs a) {
    using H = Held<T, G, N>;
    using Q = Key<T>;
    using K = typename Q::K;
    constexpr int kBlock = kThreads<N, BALANCE>;
    constexpr int kTokens = kBlock / G;  // of a workgroup at a time
    constexpr int kHalf = kBlock / kWave / 2;
    __shared__ uint32_t s_count[BALANCE ? G * N + 1 : 1];
    __shared__ float s_share[BALANCE ? kHalf : 1][BALANCE ? G * N : 1];
    const int lane = lane_id();
    const int sub = lane & (G - 1);
    const H held(sub, a.experts);
    float share[N];
    if constexpr (BALANCE) {
        for (int e = threadIdx.x; e <= G * N; e += kBlock) s_count[e] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) share[j] = 0.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.counts == nullptr) *a.done = 0;
    }
    // a row's loads are on their way while the one before it is worked on, where
    // the registers hold both
    constexpr bool kAhead = MERGE || !BALANCE;
    typename H::Raw raw[H::kChunks];
    bool live;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kTokens;
    const auto fetch = [&](int64_t t) {
        const int64_t row = t < a.tokens ? t : a.tokens - 1;
        held.fetch(static_cast<const T *>(a.logits) + row * a.stride, raw);
        live = t < a.tokens && (a.live == nullptr || a.live[row] != 0);
    };
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * kTokens;
    if (kAhead && begin < a.tokens) fetch(begin + threadIdx.x / G);
    for (int64_t base = begin; base < a.tokens; base += step) {
        const int64_t t = base + threadIdx.x / G;
        const bool inside = t < a.tokens;
        float x[N], p[N];
        if (!kAhead) fetch(t);
        held.unpack(raw, x);
        if (__builtin_expect(ballot(!live) != 0, 0)) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = live ? x[j] : -__builtin_inff();
        }
        if (kAhead && base + step < a.tokens) fetch(t + step);
        Softmax<G, N> sm;
        sm.make(x, p);
        if constexpr (BALANCE) {
#pragma unroll
            for (int j = 0; j < N; ++j) share[j] = __builtin_fmaf(p[j], sm.inv, share[j]);
            if (sub == 0 && sm.sum > 0.0f)
                __hip_atomic_fetch_add(&s_count[G * N], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        K key[N];
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = Q::make(x[j], held.index(j));
        sort_keys<Q, N, TOP>(key);
        // G places a round, one to a lane; exponentials wait for their sum where
        // they will be read again: in a register, or in the weights if there are more
        float e = 0.0f, chosen = 0.0f;
        const auto take = [&](K place, int r, int most) {
            const bool expert = Q::expert(place);
            const int id = expert ? Q::index(place) : -1;
            e = expert ? sm.weight(Q::value(place)) : 0.0f;
            chosen += e;
            if (inside && sub < most) {
                a.ids[t * a.per + r + sub] = id;
                if (a.per > G) a.weights[t * a.per + r + sub] = e;
                if (BALANCE && id >= 0)
                    __hip_atomic_fetch_add(&s_count[id], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            }
        };
        if constexpr (MERGE) {
            merge_group<Q, G, TOP>(key);
            K place = Q::none();
#pragma unroll
            for (int i = 0; i < TOP; ++i) place = pick(sub == i && i < a.per ? ~0u : 0u, place, key[i]);
            take(place, 0, a.per);
        } else {
            for (int r = 0; r < a.per; r += G) {
                const int most = a.per - r < G ? a.per - r : G;
                K place = Q::none();
                for (int k = 0; k < most; ++k) {
                    const K best = over_group<G>(key[0], Q::larger);
                    const uint32_t mine = best == key[0] ? ~0u : 0u;
#pragma unroll
                    for (int j = 0; j + 1 < N; ++j) key[j] = pick(mine, key[j], key[j + 1]);
                    key[N - 1] = pick(mine, key[N - 1], Q::none());
                    place = pick(sub == k ? ~0u : 0u, place, best);
                }
                take(place, r, most);
            }
        }
        float inv = sm.inv;
        if (a.normalize) {
            chosen = group_sum<G>(chosen);
            inv = chosen > 0.0f ? 1.0f / chosen : 0.0f;
        }
        if (inside) {
            float *w = a.weights + t * a.per;
            if (a.per <= G) {
                if (sub < a.per) w[sub] = e * inv;
            } else {
                for (int k = sub; k < a.per; k += G) w[k] *= inv;
            }
        }
    }
    if constexpr (BALANCE) {
        const int w = static_cast<int>(uniform(threadIdx.x / kWave));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            share[j] = over_groups<G>(share[j]);
            if (w >= kHalf && lane < G && held.own(j)) s_share[w - kHalf][held.index(j)] = share[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (w < kHalf && lane < G && held.own(j)) s_share[w][held.index(j)] += share[j];
        __syncthreads();
        if (a.counts != nullptr) {
            __shared__ double s_loss[kBlock / kWave];
            const uint32_t n = s_count[G * N];
            double sum = 0.0;
            for (int i = threadIdx.x; i < a.experts; i += kBlock) {
                double p = 0.0;
#pragma unroll
                for (int v = 0; v < kHalf; ++v) p += static_cast<double>(s_share[v][i]);
                p = n > 0 ? p / n : 0.0;
                a.share[i] = static_cast<float>(p);
                a.counts[i] = static_cast<int32_t>(s_count[i]);
                sum += p * s_count[i];
            }
#pragma unroll
            for (int off = 1; off < kWave; off *= 2) sum += __shfl_xor(sum, off);
            if (lane == 0) s_loss[w] = sum;
            __syncthreads();
            if (threadIdx.x == 0) {
                a.counts[a.experts] = static_cast<int32_t>(n);
                for (int v = 1; v < kBlock / kWave; ++v) sum += s_loss[v];
                *a.loss = static_cast<float>(n > 0 ? sum * a.experts / (static_cast<double>(n) * a.per) : 0.0);
            }
            return;
        }
        float *to = a.part_share + static_cast<int64_t>(blockIdx.x) * a.experts;
        int32_t *count = a.part_count + static_cast<int64_t>(blockIdx.x) * (a.experts + 1);
        for (int i = threadIdx.x; i < a.experts; i += kBlock) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < kHalf; ++v) s += s_share[v][i];
            to[i] = s;
            count[i] = static_cast<int32_t>(s_count[i]);
        }
        if (threadIdx.x == 0) count[a.experts] = static_cast<int32_t>(s_count[G * N]);
    }
}

// The workgroups' sums joined, in fp64: 16 experts to a workgroup, 64 threads
// to an expert. The workgroup that is done last adds the loss. 256 workgroups of
// 128 experts: 4.3 us, all of it latency (1 MB read).
constexpr int kJoinBlock = 1024;
constexpr int kJoinCols = 16;
constexpr int kJoinRows = kJoinBlock / kJoinCols;
constexpr int kJoinWaves = kJoinBlock / kWave;

__global__ __launch_bounds__(kJoinBlock) void route_join_kernel(RouteArgs a, int blocks, int32_t *__restrict__ counts,
                                                                float *__restrict__ share, float *__restrict__ loss) {
    __shared__ double s_p[kJoinWaves][kJoinCols];
    __shared__ int32_t s_c[kJoinWaves][kJoinCols];
    __shared__ int32_t s_live[kJoinWaves];
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int col = lane % kJoinCols;
    const int e = static_cast<int>(blockIdx.x) * kJoinCols + col;
    const int at = e < a.experts ? e : a.experts - 1;
    double p = 0.0;
    int32_t c = 0, n = 0;
#pragma unroll 4
    for (int b = static_cast<int>(threadIdx.x) / kJoinCols; b < blocks; b += kJoinRows) {
        p += static_cast<double>(a.part_share[static_cast<int64_t>(b) * a.experts + at]);
        c += a.part_count[static_cast<int64_t>(b) * (a.experts + 1) + at];
        n += a.part_count[static_cast<int64_t>(b) * (a.experts + 1) + a.experts];
    }
#pragma unroll
    for (int off = kJoinCols; off < kWave; off *= 2) {
        p += __shfl_xor(p, off);
        c += __shfl_xor(c, off);
        n += __shfl_xor(n, off);
    }
    if (lane < kJoinCols) {
        s_p[w][col] = p;
        s_c[w][col] = c;
        s_live[w] = n;
    }
    __syncthreads();
    if (w > 0) return;
    p = 0.0;
    c = 0;
    n = 0;
#pragma unroll
    for (int v = 0; v < kJoinWaves; ++v) {
        p += s_p[v][col];
        c += s_c[v][col];
        n += s_live[v];
    }
    p = n > 0 ? p / n : 0.0;
    if (lane < kJoinCols && e < a.experts) {
        share[e] = static_cast<float>(p);
        counts[e] = c;
    }
    double s = e < a.experts ? p * c : 0.0;
#pragma unroll
    for (int off = 1; off < kJoinCols; off *= 2) s += __shfl_xor(s, off);
    uint32_t before = 0;
    if (lane == 0) {
        if (blockIdx.x == 0) counts[a.experts] = n;
        __hip_atomic_store(a.part_loss + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // acknowledged before the workgroup counts as done
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        before = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (uniform(before) != gridDim.x - 1) return;
    // up to 64 workgroups, a lane each, added in one order
    s = lane < static_cast<int>(gridDim.x)
            ? __hip_atomic_load(a.part_loss + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
            : 0.0;
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) s += __shfl_xor(s, off);
    if (lane == 0) *loss = static_cast<float>(n > 0 ? s * a.experts / (static_cast<double>(n) * a.per) : 0.0);
}
static_assert(kExpertsMax / kJoinCols <= kWave, "a lane a workgroup");

// The gradient. What a chosen expert adds is computed by the lane that holds
// its place among the chosen and handed to the lane that holds its logit
// through LDS; an id that a row names twice counts twice. 65,536 tokens, 6 of 160
// bf16: 14.9 us, 25 MB read and 21 written (8.8 us at a copy's rate); with the
// prologue's loads behind one another and no row on its way ahead 26.9.
struct RouteGradArgs {
    const void *logits;
    int64_t stride, tokens;
    const uint8_t *live;
    const int32_t *ids;
    int experts, per;
    bool normalize;
    const float *dweights;
    const int32_t *counts;
    const float *dloss;
    void *dlogits;
};

template <class T, int G, int N>
__global__ __launch_bounds__(kRouteBlock) void route_grad_kernel(RouteGradArgs a) {
    using H = Held<T, G, N>;
    constexpr int kTokens = kRouteBlock / G;
    __shared__ float s_add[kRouteBlock * N];
    const int lane = lane_id();
    const int sub = lane & (G - 1);
    float *add = s_add + (threadIdx.x / G) * (G * N);  // of this token
    const H held(sub, a.experts);
    float even[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        even[j] = 0.0f;
        add[sub + j * G] = 0.0f;
    }
    if (a.counts != nullptr) {
        const int64_t n = a.counts[a.experts];
        const float each = static_cast<float>(
            n > 0 ? static_cast<double>(*a.dloss) * a.experts / (static_cast<double>(n) * n * a.per) : 0.0);
        int32_t c[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            c[j] = a.counts[H::kWide || held.index(j) < a.experts ? held.index(j) : a.experts - 1];
#pragma unroll
        for (int j = 0; j < N; ++j) even[j] = each * static_cast<float>(c[j]);
    }
    wave_lds_order();
    // this lane's place of a round of G among the chosen
    struct Chosen {
        int id;
        float d, x;
    };
    // A row's loads, and those of its first G chosen, are on their way while the
    // one before it is worked on; none waits behind a branch: what is not wanted
    // is read all the same.
    typename H::Raw raw[H::kChunks];
    int next_id = -1;
    float next_d = 0.0f;
    bool next_live;
    const auto fetch = [&](int64_t t) {
        const int64_t in = t < a.tokens ? t : a.tokens - 1;
        if (a.dweights != nullptr) {
            const int64_t at = in * a.per + (sub < a.per ? sub : a.per - 1);
            next_id = a.ids[at];
            next_d = a.dweights[at];
        }
        held.fetch(static_cast<const T *>(a.logits) + in * a.stride, raw);
        next_live = t < a.tokens && (a.live == nullptr || a.live[in] != 0);
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * kTokens;
    fetch(static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / G);
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTokens; base < a.tokens; base += step) {
        const int64_t t = base + threadIdx.x / G;
        const bool inside = t < a.tokens;
        const bool live = next_live;
        const T *row = static_cast<const T *>(a.logits) + (inside ? t : a.tokens - 1) * a.stride;
        Chosen first{-1, 0.0f, -__builtin_inff()};
        if (sub < a.per && next_id >= 0 && next_id < a.experts && live) first = {next_id, next_d, 0.0f};
        // in a cache by now
        const float first_x = static_cast<float>(row[first.id >= 0 ? first.id : 0]);
        const auto chosen = [&](int k) -> Chosen {
            if (!live || k >= a.per || a.dweights == nullptr) return {-1, 0.0f, -__builtin_inff()};
            const int id = a.ids[t * a.per + k];
            const float d = a.dweights[t * a.per + k];
            if (id < 0 || id >= a.experts) return {-1, 0.0f, -__builtin_inff()};
            return {id, d, fmaxf(static_cast<float>(row[id]), -__builtin_inff())};
        };
        float x[N], p[N];
        held.unpack(raw, x);
        if (__builtin_expect(ballot(!live) != 0, 0)) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = live ? x[j] : -__builtin_inff();
        }
        if (base + step < a.tokens) fetch(t + step);
        Softmax<G, N> sm;
        sm.make(x, p);
        if (first.id >= 0) first.x = fmaxf(first_x, -__builtin_inff());  // NaN as -infinity
        const float y = sm.weight(sm.lifted(first.x));
        float w = y, wd = y > 0.0f ? y * first.d : 0.0f;
        for (int k = G + sub; k - sub < a.per; k += G) {
            const Chosen c = chosen(k);
            const float z = sm.weight(sm.lifted(c.x));
            w += z;
            wd += z > 0.0f ? z * c.d : 0.0f;
        }
        w = group_sum<G>(w);
        wd = group_sum<G>(wd);
        const float inv = a.normalize ? (w > 0.0f ? 1.0f / w : 0.0f) : sm.inv;
        const float mean = wd * inv, less = a.normalize ? mean : 0.0f;
        const auto hand = [&](const Chosen &c, float z) {
            if (z > 0.0f)
                __hip_atomic_fetch_add(&add[c.id], z * inv * (c.d - less), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
        };
        hand(first, y);
        for (int k = G + sub; k - sub < a.per; k += G) {
            const Chosen c = chosen(k);
            hand(c, sm.weight(sm.lifted(c.x)));
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            p[j] *= sm.inv;
            s = __builtin_fmaf(p[j], even[j], s);
        }
        s = group_sum<G>(s);
        if (!a.normalize) s += mean;
        wave_lds_order();
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = __builtin_fmaf(p[j], even[j] - s, add[held.index(j)]);
        if (__builtin_expect(ballot(!(sm.sum > 0.0f)) != 0, 0)) {
#pragma unroll
            for (int j = 0; j < N; ++j) p[j] = sm.sum > 0.0f ? p[j] : 0.0f;
        }
        wave_lds_order();
        if (first.id >= 0) add[first.id] = 0.0f;
        for (int k = G + sub; k < a.per; k += G) {
            const Chosen c = chosen(k);
            if (c.id >= 0) add[c.id] = 0.0f;
        }
        wave_lds_order();
        if (inside) held.store(static_cast<T *>(a.dlogits) + t * a.experts, p);
    }
}

// ============================================================ host side ---
// Calls f with the lanes of a row and the logits of a lane: as few lanes as
// hold it with 16 each, or 24. 65,536 tokens, 8 lanes of 24 against 16 of 16, us:
//               without balance   with it     gradient
//   160 fp32        13.2 18.3     22.1 26.9   18.8 18.7
//   160 bf16        11.0 16.0     21.0 25.3   13.8 15.3
//   192 fp32        12.9 17.3     22.7 27.2   24.3 23.3
//   192 bf16        11.1 16.0     21.2 25.3   15.5 16.1
// For 257 to 384 experts, and 513 to 768, it was not tried.
template <class F>
int with_row(int64_t experts, F f) {
    using std::integral_constant;
    if (experts <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (experts <= 16) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    if (experts <= 32) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    if (experts <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (experts <= 128) return f(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    if (experts <= 192) return f(integral_constant<int, 8>{}, integral_constant<int, 24>{});
    if (experts <= 256) return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    if (experts <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

// Tokens of a workgroup at a time, with the balance.
int64_t balance_tokens(int64_t experts) {
    return experts <= 128 ? 128 : (experts <= 192 ? 64 : (experts <= 256 ? 64 : (experts <= 512 ? 32 : 16)));
}

// Workgroups of a pass with the balance: one alone for up to four rows of a lane,
// which needs no join (90 tokens of 53 experts 16.3 us a call, 20.7 with one), else
// one a compute unit, and more where a lane would add over 64 rows, one after
// another in fp32.
constexpr int64_t kAlone = 4;

struct RoutePlan {
    int64_t blocks;
    size_t share, count, loss, bytes;  // offsets into the scratch
};

RoutePlan route_plan(int64_t tokens, int64_t experts) {
    RoutePlan p{};
    const int64_t each = balance_tokens(experts);
    const int64_t all = (tokens + each - 1) / each;
    p.blocks = all <= kAlone ? 1 : (all < 256 ? all : 256);
    if (p.blocks < (all + 63) / 64) p.blocks = (all + 63) / 64;
    if (p.blocks == 1) return p;
    p.loss = 16;
    p.share = p.loss + 8 * ((experts + kJoinCols - 1) / kJoinCols);
    p.count = p.share + static_cast<size_t>(p.blocks) * experts * 4;
    p.bytes = p.count + static_cast<size_t>(p.blocks) * (experts + 1) * 4;
    return p;
}

int check_route(int dtype, int64_t tokens, int64_t experts, int64_t stride, int64_t per) {
    if (!dtype_ok(dtype) || tokens < 0 || experts < 1 || per < 1 || per > experts || stride < experts)
        return SSC_ERR_ARG;
    if (tokens > INT32_MAX || experts > kExpertsMax || per > kPerMax || tokens * per > INT32_MAX ||
        stride > (int64_t{1} << 30))
        return SSC_ERR_SIZE;
    return SSC_OK;
}

size_t strided_bytes(int64_t rows, int64_t stride, int64_t width, int dtype) {
    return rows > 0 ? (static_cast<size_t>(rows - 1) * stride + width) * elem_bytes(dtype) : 0;
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

size_t ssc_route_scratch_bytes(int64_t tokens, int64_t experts) {
    return tokens < 0 || tokens > INT32_MAX || experts < 1 || experts > kExpertsMax ? 0
                                                                                   : route_plan(tokens, experts).bytes;
}

int ssc_route_rows(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t stride,
                   const uint8_t *live, int64_t per, int normalize, int32_t *ids, float *weights, int32_t *counts,
                   float *share, float *loss, void *scratch, size_t scratch_bytes, void *stream) {
    SSC_TRY(check_route(dtype, tokens, experts, stride, per));
    if (tokens > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return SSC_ERR_ARG;
    const bool balance = counts != nullptr;
    if ((share != nullptr) != balance || (loss != nullptr) != balance) return SSC_ERR_ARG;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(counts, 4) ||
        !aligned(share, 4) || !aligned(loss, 4))
        return SSC_ERR_ARG;
    const RoutePlan p = route_plan(tokens, experts);
    const size_t need = balance ? p.bytes : 0;
    if (need > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < need)) return SSC_ERR_SCRATCH;
    const size_t slots = static_cast<size_t>(tokens) * per * 4;
    const Span written[] = {{ids, slots},
                            {weights, slots},
                            {counts, (static_cast<size_t>(experts) + 1) * 4},
                            {share, static_cast<size_t>(experts) * 4},
                            {loss, 4},
                            {scratch, need}};
    const Span read[] = {{logits, strided_bytes(tokens, stride, experts, dtype)}, {live, static_cast<size_t>(tokens)}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &w : written)
        for (const Span &r : read)
            if (overlap(w.p, w.bytes, r.p, r.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (tokens == 0 && !balance) return SSC_OK;
    RouteArgs a{};
    a.logits = logits;
    a.stride = stride;
    a.tokens = tokens;
    a.live = live;
    a.experts = static_cast<int>(experts);
    a.per = static_cast<int>(per);
    a.normalize = normalize != 0;
    a.ids = ids;
    a.weights = weights;
    if (balance && p.blocks == 1) {
        a.counts = counts;
        a.share = share;
        a.loss = loss;
    } else if (balance) {
        char *at = static_cast<char *>(scratch);
        a.done = reinterpret_cast<uint32_t *>(at);
        a.part_loss = reinterpret_cast<double *>(at + p.loss);
        a.part_share = reinterpret_cast<float *>(at + p.share);
        a.part_count = reinterpret_cast<int32_t *>(at + p.count);
    }
    SSC_TRY(with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return with_row(experts, [&](auto g, auto n) {
            constexpr int G = decltype(g)::value, N = decltype(n)::value;
            const auto launch = [&](auto top, auto merge) {
                constexpr int TOP = decltype(top)::value;
                constexpr bool M = decltype(merge)::value;
                const int64_t all = (tokens + kRouteBlock / G - 1) / (kRouteBlock / G);
                if (balance)
                    hipLaunchKernelGGL((route_kernel<T, G, N, TOP, M, true>), dim3(static_cast<unsigned>(p.blocks)),
                                       dim3((kThreads<N, true>)), 0, s, a);
                else
                    hipLaunchKernelGGL((route_kernel<T, G, N, TOP, M, false>),
                                       dim3(static_cast<unsigned>(all < 8192 ? all : 8192)),
                                       dim3((kThreads<N, false>)), 0, s, a);
                return launched();
            };
            if constexpr (N >= 8) {
                if (per <= 4) return launch(std::integral_constant<int, 4>{}, std::true_type{});
                if (per <= 8) return launch(std::integral_constant<int, 8>{}, std::true_type{});
            }
            return launch(std::integral_constant<int, N>{}, std::false_type{});
        });
    }));
    if (!balance || p.blocks == 1) return SSC_OK;
    hipLaunchKernelGGL(route_join_kernel, dim3(static_cast<unsigned>((experts + kJoinCols - 1) / kJoinCols)),
                       dim3(kJoinBlock), 0, s, a, static_cast<int>(p.blocks), counts, share, loss);
    return launched();
}

int ssc_route_rows_grad(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t stride,
                        const uint8_t *live, const int32_t *ids, int64_t per, int normalize, const float *dweights,
                        const int32_t *counts, const float *dloss, void *dlogits, void *stream) {
    SSC_TRY(check_route(dtype, tokens, experts, stride, per));
    if (tokens > 0 && (logits == nullptr || dlogits == nullptr || (dweights != nullptr && ids == nullptr)))
        return SSC_ERR_ARG;
    if ((counts != nullptr) != (dloss != nullptr)) return SSC_ERR_ARG;
    const size_t es = elem_bytes(dtype);
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(ids, 4) || !aligned(dweights, 4) ||
        !aligned(counts, 4) || !aligned(dloss, 4))
        return SSC_ERR_ARG;
    const size_t slots = static_cast<size_t>(tokens) * per * 4, out = static_cast<size_t>(tokens) * experts * es;
    const Span read[] = {{logits, strided_bytes(tokens, stride, experts, dtype)},
                         {live, static_cast<size_t>(tokens)},
                         {ids, slots},
                         {dweights, slots},
                         {counts, (static_cast<size_t>(experts) + 1) * 4},
                         {dloss, 4}};
    for (const Span &r : read)
        if (overlap(dlogits, out, r.p, r.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (tokens == 0) return SSC_OK;
    RouteGradArgs a{};
    a.logits = logits;
    a.stride = stride;
    a.tokens = tokens;
    a.live = live;
    a.ids = ids;
    a.experts = static_cast<int>(experts);
    a.per = static_cast<int>(per);
    a.normalize = normalize != 0;
    a.dweights = dweights;
    a.counts = counts;
    a.dloss = dloss;
    a.dlogits = dlogits;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return with_row(experts, [&](auto g, auto n) {
            constexpr int G = decltype(g)::value, N = decltype(n)::value;
            const int64_t all = (tokens + kRouteBlock / G - 1) / (kRouteBlock / G);
            hipLaunchKernelGGL((route_grad_kernel<T, G, N>), dim3(static_cast<unsigned>(all < 1024 ? all : 1024)),
                               dim3(kRouteBlock), 0, static_cast<hipStream_t>(stream), a);
            return launched();
        });
    });
}

}  // extern "C"
