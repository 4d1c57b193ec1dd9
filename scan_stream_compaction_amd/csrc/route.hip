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
constexpr int kRouteWaves = kRouteBlock / kWave;
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

// The N keys of a lane, largest first, by merging of odd and even places
// (63 exchanges for 16).
template <class Q, int N>
__device__ __forceinline__ void sort_keys(typename Q::K (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2) {
#pragma unroll
        for (int h = p; h >= 1; h /= 2) {
#pragma unroll
            for (int j = h % p; j + h < N; j += 2 * h) {
#pragma unroll
                for (int i = 0; i < h; ++i) {
                    const int a = j + i, b = j + i + h;
                    if (b < N && a / (2 * p) == b / (2 * p)) {
                        const auto big = Q::larger(k[a], k[b]);
                        k[b] = Q::smaller(k[a], k[b]);
                        k[a] = big;
                    }
                }
            }
        }
    }
}

// exp(d) for d <= 0, by 2^(d log2(e)) with what the product's rounding loses put
// back to first order; below -200 it is 0.
__device__ __forceinline__ float exp_of(float d) {
    constexpr float kHi = 1.44269504088896340736f;
    constexpr float kLo = static_cast<float>(1.44269504088896340736 - static_cast<double>(kHi));
    d = fmaxf(d, -200.0f);
    const float a = d * kHi;
    const float r = __builtin_fmaf(d, kLo, __builtin_fmaf(d, kHi, -a));
    const float e = __builtin_amdgcn_exp2f(a);
    return __builtin_fmaf(e, r * 0.69314718055994530942f, e);
}

// A row of logits as exponentials of their distance from the largest. Beside one
// of +infinity no other counts. A row without experts has none (sum 0).
template <int G, int N>
struct Softmax {
    float top, sum, inv;
    bool lift;

    __device__ __forceinline__ float lifted(float x) const {
        return lift ? (x == __builtin_inff() ? 0.0f : -__builtin_inff()) : x;
    }
    __device__ __forceinline__ float weight(float x) const {
        const float y = lifted(x);
        return y > -__builtin_inff() ? exp_of(y - top) : 0.0f;
    }
    __device__ __forceinline__ void make(const float (&x)[N], float (&e)[N]) {
        float m = x[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = fmaxf(m, x[j]);
        top = group_max<G>(m);
        lift = top == __builtin_inff();
        if (lift) top = 0.0f;
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

template <class T, int G, int N, bool BALANCE>
__global__ __launch_bounds__(kRouteBlock) void route_kernel(RouteArgs a) {
    using H = Held<T, G, N>;
    using Q = Key<T>;
    using K = typename Q::K;
    constexpr int kTokens = kRouteBlock / G;       // of a workgroup at a time
    constexpr int kRounds = N < 64 / G ? N : 64 / G;  // of G places among the chosen
    __shared__ uint32_t s_count[BALANCE ? G * N + 1 : 1];
    __shared__ float s_share[BALANCE ? kRouteWaves : 1][BALANCE ? G * N : 1];
    const int lane = lane_id();
    const int sub = lane & (G - 1);
    float share[N];
    if constexpr (BALANCE) {
        for (int e = threadIdx.x; e <= G * N; e += kRouteBlock) s_count[e] = 0;
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
        sort_keys<Q, N>(key);
        float e[kRounds], chosen = 0.0f;
        int id[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            e[r] = 0.0f;
            id[r] = -1;
            const int most = a.per - r * G < G ? a.per - r * G : G;
            for (int k = 0; k < most; ++k) {
                const K best = over_group<G>(key[0], Q::larger);
                const bool mine = best == key[0];
#pragma unroll
                for (int j = 0; j + 1 < N; ++j) key[j] = mine ? key[j + 1] : key[j];
                if (mine) key[N - 1] = Q::make(-__builtin_inff(), 0);
                if (sub == k && Q::expert(best)) {
                    const float w = sm.weight(Q::value(best));
                    if (sm.lifted(Q::value(best)) > -__builtin_inff()) {
                        id[r] = Q::index(best);
                        e[r] = w;
                    }
                }
            }
            chosen += e[r];
        }
        float inv = sm.inv;
        if (a.normalize) {
            chosen = group_sum<G>(chosen);
            inv = chosen > 0.0f ? 1.0f / chosen : 0.0f;
        }
        if (inside) {
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                const int k = r * G + sub;
                if (k < a.per) {
                    a.ids[t * a.per + k] = id[r];
                    a.weights[t * a.per + k] = e[r] * inv;
                    if (BALANCE && id[r] >= 0)
                        __hip_atomic_fetch_add(&s_count[id[r]], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                }
            }
        }
    }
    if constexpr (BALANCE) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
#pragma unroll
            for (int off = G; off < kWave; off *= 2) share[j] += __shfl_xor(share[j], off);
            if (lane < G) s_share[threadIdx.x / kWave][H::at(sub, j)] = share[j];
        }
        __syncthreads();
        float *to = a.part_share + static_cast<int64_t>(blockIdx.x) * a.experts;
        int32_t *count = a.part_count + static_cast<int64_t>(blockIdx.x) * (a.experts + 1);
        for (int i = threadIdx.x; i < a.experts; i += kRouteBlock) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kRouteWaves; ++w) s += s_share[w][i];
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

__global__ __launch_bounds__(kRouteBlock) void route_join_kernel(RouteArgs a, int blocks, int32_t *__restrict__ counts,
                                                                float *__restrict__ share, float *__restrict__ loss) {
    __shared__ double s_p[kJoinRows][kJoinCols + 1];
    __shared__ int32_t s_c[kJoinRows][kJoinCols + 1];
    __shared__ int32_t s_live[kRouteWaves];
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
    for (int w = 0; w < kRouteWaves; ++w) n += s_live[w];
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
    constexpr int kRounds = N < 64 / G ? N : 64 / G;
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
        int id[kRounds];
        float d[kRounds], y[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int k = r * G + sub;
            const bool has = live && k < a.per && a.dweights != nullptr;
            id[r] = has ? a.ids[t * a.per + k] : -1;
            if (id[r] >= a.experts || id[r] < 0) id[r] = -1;
            d[r] = id[r] >= 0 ? a.dweights[t * a.per + k] : 0.0f;
            y[r] = id[r] >= 0 ? fmaxf(static_cast<float>(row[id[r]]), -__builtin_inff()) : -__builtin_inff();
        }
        float x[N], p[N];
        H::load(row, sub, live ? a.experts : 0, x);
        Softmax<G, N> sm;
        sm.make(x, p);
        float w = 0.0f, wd = 0.0f;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            y[r] = sm.weight(y[r]);
            w += y[r];
            wd += y[r] > 0.0f ? y[r] * d[r] : 0.0f;
        }
        w = group_sum<G>(w);
        wd = group_sum<G>(wd);
        const float inv = a.normalize ? (w > 0.0f ? 1.0f / w : 0.0f) : sm.inv;
        const float mean = wd * inv;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (y[r] > 0.0f)
                __hip_atomic_fetch_add(&add[id[r]], y[r] * inv * (a.normalize ? d[r] - mean : d[r]), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
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
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (id[r] >= 0) add[id[r]] = 0.0f;
        wave_lds_order();
        if (inside) H::store(static_cast<T *>(a.dlogits) + t * a.experts, sub, a.experts, p);
    }
}

// ============================================================ host side ---
// Calls f with the lanes of a row and the logits of a lane: as few lanes as
// hold it with 16 each.
template <class F>
int with_row(int64_t experts, F f) {
    const auto of = [&](auto g, auto n) { return f(g, n); };
    using std::integral_constant;
    if (experts <= 8) return of(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (experts <= 16) return of(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    if (experts <= 32) return of(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    if (experts <= 64) return of(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (experts <= 128) return of(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    if (experts <= 256) return of(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    if (experts <= 512) return of(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    return of(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

int lanes_of(int64_t experts) {
    return experts <= 128 ? 8 : experts <= 256 ? 16 : experts <= 512 ? 32 : 64;
}

// Workgroups of a pass with the balance: two a compute unit, and more where a
// lane would add over 64 rows, one after another in fp32.
struct RoutePlan {
    int64_t blocks;
    size_t share, count, loss, bytes;  // offsets into the scratch
};

RoutePlan route_plan(int64_t tokens, int64_t experts) {
    RoutePlan p{};
    const int64_t each = kRouteBlock / lanes_of(experts);
    const int64_t all = (tokens + each - 1) / each;
    p.blocks = all < 1 ? 1 : (all < 512 ? all : 512);
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
            const int64_t all = (tokens + kRouteBlock / G - 1) / (kRouteBlock / G);
            if (balance)
                hipLaunchKernelGGL((route_kernel<T, G, N, true>), dim3(static_cast<unsigned>(p.blocks)),
                                   dim3(kRouteBlock), 0, s, a);
            else
                hipLaunchKernelGGL((route_kernel<T, G, N, false>), dim3(static_cast<unsigned>(all < 8192 ? all : 8192)),
                                   dim3(kRouteBlock), 0, s, a);
            return launched();
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
