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
// chunks side by side, so that its lanes read consecutive addresses.
template <class T, int G, int N>
struct Held {
    static constexpr int kC = N < 16 / static_cast<int>(sizeof(T)) ? N : 16 / static_cast<int>(sizeof(T));
    __device__ static __forceinline__ int at(int sub, int j) { return ((j / kC) * G + sub) * kC + j % kC; }

    // a logit that is no number is as one of -infinity
    __device__ static __forceinline__ void load(const T *row, int sub, int n, float (&x)[N]) {
#pragma unroll
        for (int c = 0; c < N / kC; ++c) {
            const int i = at(sub, c * kC);
            if (kC * sizeof(T) == 16 && i + kC <= n) {
                typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
                const u32x4 r = *reinterpret_cast<const u32x4_any *>(row + i);
                const V v = __builtin_bit_cast(V, r);
#pragma unroll
                for (int e = 0; e < kC; ++e) x[c * kC + e] = static_cast<float>(v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < kC; ++e)
                    x[c * kC + e] = i + e < n ? static_cast<float>(row[i + e]) : -__builtin_inff();
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = fmaxf(x[j], -__builtin_inff());
    }
    __device__ static __forceinline__ void store(T *row, int sub, int n, const float (&x)[N]) {
#pragma unroll
        for (int c = 0; c < N / kC; ++c) {
            const int i = at(sub, c * kC);
            if (kC * sizeof(T) == 16 && i + kC <= n) {
                typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
                V v;
#pragma unroll
                for (int e = 0; e < kC; ++e) v[e] = static_cast<T>(x[c * kC + e]);
                *reinterpret_cast<u32x4_any *>(row + i) = __builtin_bit_cast(u32x4, v);
            } else {
#pragma unroll
                for (int e = 0; e < kC; ++e)
                    if (i + e < n) row[i + e] = static_cast<T>(x[c * kC + e]);
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
template <int G>
__device__ __forceinline__ float group_max(float v) {
    return over_group<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// A logit and its expert in one number that is largest for the largest logit,
// the lowest expert of equal ones; a key of value 0 is no expert. 16-bit logits
// fit with their index into 32 bits, fp32 ones into the fraction of a double
// (2^52 above them keeps it normal), whose maximum is one instruction.
template <class T>
struct Key {
    using K = uint32_t;
    __device__ static __forceinline__ K make(float x, int index) {
        const uint32_t b = __float_as_uint(x + 0.0f) >> 16;
        uint32_t k;
        if constexpr (std::is_same_v<T, _Float16>) {
            const uint32_t h = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x + 0.0f));
            k = h & 0x8000u ? ~h & 0xffffu : h | 0x8000u;
        } else {
            k = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
        }
        return x > -__builtin_inff() ? k << kIndexBits | (kIndexMask - static_cast<uint32_t>(index)) : 0u;
    }
    __device__ static __forceinline__ K none() { return 0u; }
    __device__ static __forceinline__ K larger(K a, K b) { return a > b ? a : b; }
    __device__ static __forceinline__ K smaller(K a, K b) { return a > b ? b : a; }
    __device__ static __forceinline__ bool expert(K k) { return k > kIndexMask; }
    __device__ static __forceinline__ int index(K k) { return static_cast<int>(kIndexMask - (k & kIndexMask)); }
    __device__ static __forceinline__ float value(K k) {
        const uint32_t o = k >> kIndexBits, b = o & 0x8000u ? o & 0x7fffu : ~o & 0xffffu;
        if constexpr (std::is_same_v<T, _Float16>)
            return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
        else
            return __uint_as_float(b << 16);
    }
};
template <>
struct Key<float> {
    using K = double;
    static constexpr uint64_t kBase = 0x4330000000000000ull;
    __device__ static __forceinline__ uint64_t bits(K k) { return static_cast<uint64_t>(__double_as_longlong(k)); }
    __device__ static __forceinline__ K make(float x, int index) {
        const uint32_t b = __float_as_uint(x + 0.0f);
        const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
        const uint64_t k = static_cast<uint64_t>(o) << kIndexBits | (kIndexMask - static_cast<uint32_t>(index));
        return __longlong_as_double(static_cast<long long>(x > -__builtin_inff() ? kBase | k : kBase));
    }
    __device__ static __forceinline__ K none() { return 0x1p52; }
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
    __device__ static __forceinline__ bool expert(K k) { return bits(k) - kBase > kIndexMask; }
    __device__ static __forceinline__ int index(K k) {
        return static_cast<int>(kIndexMask - (static_cast<uint32_t>(bits(k)) & kIndexMask));
    }
    __device__ static __forceinline__ float value(K k) {
        const uint32_t o = static_cast<uint32_t>((bits(k) - kBase) >> kIndexBits);
        return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
    }
};

// a where mask is 0, b where it is all ones (a choice by a condition between
// two elements of an array becomes an index into it, and that sixteen selects)
__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t a, uint32_t b) { return a ^ ((a ^ b) & mask); }
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

// The TOP largest keys of a lane's N, largest first, in its first places: by
// merging of odd and even places (63 exchanges for 16), for 8 of more in runs of
// 8, of two of which the larger half is kept and put in order (19 an run, 8
// maxima and 12 a merge: 108 instructions for 8 of 16 against 126).
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
        if (run == 0) continue;
#pragma unroll
        for (int i = 0; i < TOP; ++i) k[i] = Q::larger(k[i], k[run + TOP - 1 - i]);
#pragma unroll
        for (int h = TOP / 2; h >= 1; h /= 2) {
#pragma unroll
            for (int i = 0; i < TOP; ++i)
                if ((i & h) == 0) exchange<Q>(k[i], k[i + h]);
        }
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
};

// With the balance a workgroup adds up its tokens' softmax, so it is larger and
// there are fewer: as many threads as the registers of N logits allow.
template <int N, bool BALANCE>
constexpr int kThreads = !BALANCE ? kRouteBlock : (N > 16 ? 512 : 1024);

// TOP: of the lane's logits, how many may be chosen (8 where `per` is no more).
template <class T, int G, int N, int TOP, bool BALANCE>
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
    float share[N];
    if constexpr (BALANCE) {
        for (int e = threadIdx.x; e <= G * N; e += kBlock) s_count[e] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) share[j] = 0.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    }
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTokens; base < a.tokens;
         base += static_cast<int64_t>(gridDim.x) * kTokens) {
        const int64_t t = base + threadIdx.x / G;
        const bool inside = t < a.tokens;
        const bool live = inside && (a.live == nullptr || a.live[t] != 0);
        float x[N], p[N];
        H::load(static_cast<const T *>(a.logits) + (live ? t : 0) * a.stride, sub, live ? a.experts : 0, x);
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
        for (int j = 0; j < N; ++j) key[j] = Q::make(x[j], H::at(sub, j));
        sort_keys<Q, N, TOP>(key);
        // G places a round, one to a lane; exponentials wait for their sum where
        // they will be read again: in a register, or in the weights if there are more
        float e = 0.0f, chosen = 0.0f;
        for (int r = 0; r < a.per; r += G) {
            const int most = a.per - r < G ? a.per - r : G;
            K place = Q::none();
            for (int k = 0; k < most; ++k) {
                const K best = over_group<G>(key[0], Q::larger);
                const uint32_t mine = best == key[0] ? ~0u : 0u;
#pragma unroll
                for (int j = 0; j + 1 < TOP; ++j) key[j] = pick(mine, key[j], key[j + 1]);
                key[TOP - 1] = pick(mine, key[TOP - 1], Q::none());
                place = pick(sub == k ? ~0u : 0u, place, best);
            }
            const float v = Q::value(place);
            const bool expert = Q::expert(place);
            const int id = expert ? Q::index(place) : -1;
            e = expert ? sm.weight(v) : 0.0f;
            chosen += e;
            if (inside && sub < most) {
                a.ids[t * a.per + r + sub] = id;
                if (a.per > G) a.weights[t * a.per + r + sub] = e;
                if (BALANCE && id >= 0)
                    __hip_atomic_fetch_add(&s_count[id], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
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
#pragma unroll
            for (int off = G; off < kWave; off *= 2) share[j] += __shfl_xor(share[j], off);
            if (w >= kHalf && lane < G) s_share[w - kHalf][H::at(sub, j)] = share[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (w < kHalf && lane < G) s_share[w][H::at(sub, j)] += share[j];
        __syncthreads();
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

// The workgroups' sums joined: 16 experts to a workgroup, sixteen threads to an
// expert, in fp64. The workgroup that is done last adds the loss.
constexpr int kJoinCols = 16;
constexpr int kJoinRows = kRouteBlock / kJoinCols;
constexpr int kJoinWaves = kRouteBlock / kWave;

__global__ __launch_bounds__(kRouteBlock) void route_join_kernel(RouteArgs a, int blocks, int32_t *__restrict__ counts,
                                                                float *__restrict__ share, float *__restrict__ loss) {
    __shared__ double s_p[kJoinRows][kJoinCols + 1];
    __shared__ int32_t s_c[kJoinRows][kJoinCols + 1];
    __shared__ int32_t s_live[kJoinWaves];
    __shared__ double s_loss[kJoinCols];
    __shared__ uint32_t s_last;
    const int col = threadIdx.x % kJoinCols, row = threadIdx.x / kJoinCols;
    const int e = blockIdx.x * kJoinCols + col;
    int32_t n = 0;
    for (int b = threadIdx.x; b < blocks; b += kRouteBlock)
        n += a.part_count[static_cast<int64_t>(b) * (a.experts + 1) + a.experts];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off);
    if (lane_id() == 0) s_live[threadIdx.x / kWave] = n;
    double p = 0.0;
    int32_t c = 0;
    if (e < a.experts) {
#pragma unroll 8
        for (int b = row; b < blocks; b += kJoinRows) {
            p += static_cast<double>(a.part_share[static_cast<int64_t>(b) * a.experts + e]);
            c += a.part_count[static_cast<int64_t>(b) * (a.experts + 1) + e];
        }
    }
    s_p[row][col] = p;
    s_c[row][col] = c;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kJoinWaves; ++w) n += s_live[w];
    if (row == 0) {
        p = 0.0;
        c = 0;
        for (int r = 0; r < kJoinRows; ++r) {
            p += s_p[r][col];
            c += s_c[r][col];
        }
        p = n > 0 ? p / n : 0.0;
        if (e < a.experts) {
            share[e] = static_cast<float>(p);
            counts[e] = c;
        }
        s_loss[col] = e < a.experts ? p * c : 0.0;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < kJoinCols; ++i) s += s_loss[i];
        __hip_atomic_store(a.part_loss + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) counts[a.experts] = n;
    __syncthreads();
    if (s_last == gridDim.x - 1 && threadIdx.x == 0) {
        double s = 0.0;
        for (uint32_t b = 0; b < gridDim.x; ++b)
            s += __hip_atomic_load(a.part_loss + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *loss = static_cast<float>(n > 0 ? s * a.experts / (static_cast<double>(n) * a.per) : 0.0);
    }
}

// The gradient. What a chosen expert adds is computed by the lane that holds
// its place among the chosen and handed to the lane that holds its logit
// through LDS; an id that a row names twice counts twice.
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
    float even[N];
    const int64_t n = a.counts != nullptr ? a.counts[a.experts] : 0;
    const double each = n > 0 ? static_cast<double>(*a.dloss) * a.experts / (static_cast<double>(n) * n * a.per) : 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = H::at(sub, j);
        even[j] = n > 0 && e < a.experts ? static_cast<float>(each * a.counts[e]) : 0.0f;
        add[sub + j * G] = 0.0f;
    }
    wave_lds_order();
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTokens; base < a.tokens;
         base += static_cast<int64_t>(gridDim.x) * kTokens) {
        const int64_t t = base + threadIdx.x / G;
        const bool inside = t < a.tokens;
        const bool live = inside && (a.live == nullptr || a.live[t] != 0);
        const T *row = static_cast<const T *>(a.logits) + (live ? t : 0) * a.stride;
        // this lane's place of a round of G among the chosen
        struct Chosen {
            int id;
            float d, x;
        };
        const auto chosen = [&](int k) -> Chosen {
            if (!live || k >= a.per || a.dweights == nullptr) return {-1, 0.0f, -__builtin_inff()};
            const int id = a.ids[t * a.per + k];
            const float d = a.dweights[t * a.per + k];
            if (id < 0 || id >= a.experts) return {-1, 0.0f, -__builtin_inff()};
            return {id, d, fmaxf(static_cast<float>(row[id]), -__builtin_inff())};  // NaN as -infinity
        };
        const Chosen first = chosen(sub);
        float x[N], p[N];
        H::load(row, sub, live ? a.experts : 0, x);
        Softmax<G, N> sm;
        sm.make(x, p);
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
        for (int j = 0; j < N; ++j)
            p[j] = sm.sum > 0.0f ? __builtin_fmaf(p[j], even[j] - s, add[H::at(sub, j)]) : 0.0f;
        wave_lds_order();
        if (first.id >= 0) add[first.id] = 0.0f;
        for (int k = G + sub; k < a.per; k += G) {
            const Chosen c = chosen(k);
            if (c.id >= 0) add[c.id] = 0.0f;
        }
        wave_lds_order();
        if (inside) H::store(static_cast<T *>(a.dlogits) + t * a.experts, sub, a.experts, p);
    }
}

// ============================================================ host side ---
// Calls f with the lanes of a row and the logits of a lane: as few lanes as
// hold it with 16 each, or 24.
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

// Workgroups of a pass with the balance: one a compute unit, and more where a
// lane would add over 64 rows, one after another in fp32.
struct RoutePlan {
    int64_t blocks;
    size_t share, count, loss, bytes;  // offsets into the scratch
};

RoutePlan route_plan(int64_t tokens, int64_t experts) {
    RoutePlan p{};
    const int64_t each = balance_tokens(experts);
    const int64_t all = (tokens + each - 1) / each;
    p.blocks = all < 1 ? 1 : (all < 256 ? all : 256);
    if (p.blocks < (all + 63) / 64) p.blocks = (all + 63) / 64;
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
    if (balance) {
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
            const auto launch = [&](auto top) {
                constexpr int TOP = decltype(top)::value;
                const int64_t all = (tokens + kRouteBlock / G - 1) / (kRouteBlock / G);
                if (balance)
                    hipLaunchKernelGGL((route_kernel<T, G, N, TOP, true>), dim3(static_cast<unsigned>(p.blocks)),
                                       dim3((kThreads<N, true>)), 0, s, a);
                else
                    hipLaunchKernelGGL((route_kernel<T, G, N, TOP, false>),
                                       dim3(static_cast<unsigned>(all < 8192 ? all : 8192)),
                                       dim3((kThreads<N, false>)), 0, s, a);
                return launched();
            };
            if (N > 8 && per <= 8) return launch(std::integral_constant<int, (N > 8 ? 8 : N)>{});
            return launch(std::integral_constant<int, N>{});
        });
    }));
    if (!balance) return SSC_OK;
    hipLaunchKernelGGL(route_join_kernel, dim3(static_cast<unsigned>((experts + kJoinCols - 1) / kJoinCols)),
                       dim3(kRouteBlock), 0, s, a, static_cast<int>(p.blocks), counts, share, loss);
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
            hipLaunchKernelGGL((route_grad_kernel<T, G, N>), dim3(static_cast<unsigned>(all < 2048 ? all : 2048)),
                               dim3(kRouteBlock), 0, static_cast<hipStream_t>(stream), a);
            return launched();
        });
    });
}

}  // extern "C"
