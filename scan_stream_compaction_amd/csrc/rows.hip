// Rows moved by a key, for the token path of a language model: the stable
// many-way partition of keys (token or expert ids) and the operators that
// carry rows of features with it. HIP kernels for MI355X (gfx950) and their
// part of the C ABI in include/ssc.h.
//
//   group_by_key      ranks[i] = offsets[key] + equal keys before i
//   embed_rows        out[i] = scale * table[ids[i]]
//   embed_rows_grad   grad[v] = scale * sum of dout[i] over ids[i] = v
//   dispatch_rows     out[ranks[t, k]] = x[t]
//   combine_rows      out[t] = sum over k of w[t, k] * y[ranks[t, k]]
//   combine_rows_grad dy[ranks[t, k]] = w[t, k] * dout[t],
//                     dw[t, k] = <dout[t], y[ranks[t, k]]>
//
// Rows hold fp32, bf16 or fp16 elements. Sums run in fp32, in an order fixed
// by the sizes and the ranks alone, and are rounded to the output's type once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssc.h"
#include "ssc_device.h"
#include "ssc_host.h"

namespace ssc {
namespace {

// =============================================== stable partition by key ---
// An LSD sort of (key, position) by digits of at most 9 bits: `groups`
// values and one more for keys outside [0, groups), which sort last and are
// given no place. Up to 511 groups take a single pass. Each pass ranks keys
// in input order: a wavefront takes 64 consecutive keys at a time, and a
// ballot per digit bit gives each lane the mask of the lanes that hold its
// digit; its rank is the wavefront's running count of that digit plus the
// matching lanes below it.
constexpr int kGroupBlock = 1024;
constexpr int kGroupWaves = kGroupBlock / kWave;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kGroupSmall = 16 * kGroupBlock;   // keys one workgroup sorts alone
constexpr int kGroupItems = 8;                  // keys per thread and step of the tiled form
constexpr int kGroupStep = kGroupItems * kGroupBlock;
constexpr int kGroupTiles = 256;                // most workgroups of a tiled pass

template <class K>
__device__ __forceinline__ uint32_t key_of(K k, uint32_t groups) {
    return k >= 0 && static_cast<uint64_t>(k) < groups ? static_cast<uint32_t>(k) : groups;
}

// Rank of each lane's digit among the keys this wavefront has seen, in
// order; cnt holds the wavefront's counts.
__device__ __forceinline__ uint32_t digit_rank(uint32_t d, bool valid, int bits, uint32_t *cnt) {
    uint64_t m = ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const uint64_t bb = ballot(valid && ((d >> b) & 1u));
        m &= ((d >> b) & 1u) ? bb : ~bb;
    }
    const uint32_t below = mbcnt64(m);
    const uint32_t same = static_cast<uint32_t>(__builtin_popcountll(m));
    uint32_t run = 0;
    if (valid) {
        run = cnt[d];
        if (below + 1u == same) cnt[d] = run + same;
    }
    return run + below;
}

// Exclusive prefix of v over the workgroup's threads.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t *s_wave) {
    const uint32_t incl = wave_inclusive_scan<SumU32>(v);
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    if (lane == kWave - 1) s_wave[w] = incl;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += s_wave[i];
    __syncthreads();
    return before + incl - v;
}

// The wavefronts' counts of a tile, cnt[w][d], become the counts of earlier
// wavefronts; returns the tile's count of digit threadIdx.x (0 beyond the digits).
__device__ __forceinline__ uint32_t counts_before(uint32_t (*cnt)[kDigits], uint32_t digits) {
    uint32_t total = 0;
    if (threadIdx.x < digits) {
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            const uint32_t c = cnt[w][threadIdx.x];
            cnt[w][threadIdx.x] = total;
            total += c;
        }
    }
    return total;
}

// offsets[v] for every v whose first sorted position lies in [s0, s1), with
// position n standing for the group after the last: the position s with key
// k after key p starts groups p + 1 .. k. Long gaps between present keys are
// filled by the whole workgroup.
struct GapList {
    uint32_t count;
    uint32_t lo[kGroupBlock], hi[kGroupBlock], at[kGroupBlock];
};
constexpr uint32_t kGapLong = 32;

template <class F>
__device__ __forceinline__ void fill_offsets(F key, uint32_t s0, uint32_t s1, uint32_t n, uint32_t groups,
                                             int32_t *__restrict__ offsets, GapList &gaps) {
    for (uint32_t base = s0; base < s1; base += kGroupBlock) {
        if (threadIdx.x == 0) gaps.count = 0;
        __syncthreads();
        const uint32_t s = base + threadIdx.x;
        if (s < s1) {
            const uint32_t lo = s == 0 ? 0u : key(s - 1) + 1u;
            const uint32_t end = (s < n ? key(s) : groups) + 1u;  // keys stop at groups <= INT32_MAX
            if (lo < end) {
                if (end - lo <= kGapLong) {
                    for (uint32_t v = lo; v < end; ++v) offsets[v] = static_cast<int32_t>(s);
                } else {
                    const uint32_t e = __hip_atomic_fetch_add(&gaps.count, 1u, __ATOMIC_RELAXED,
                                                              __HIP_MEMORY_SCOPE_WORKGROUP);
                    gaps.lo[e] = lo;
                    gaps.hi[e] = end;
                    gaps.at[e] = s;
                }
            }
        }
        __syncthreads();
        for (uint32_t e = 0; e < gaps.count; ++e)
            for (uint32_t v = gaps.lo[e] + threadIdx.x; v < gaps.hi[e]; v += kGroupBlock)
                offsets[v] = static_cast<int32_t>(gaps.at[e]);
        __syncthreads();
    }
}

// Up to 16,384 keys: one workgroup holds (key, position) in registers and
// exchanges them through LDS between passes.
template <class K, int ITEMS>
__global__ __launch_bounds__(kGroupBlock) void group_small_kernel(
    const K *__restrict__ keys, uint32_t n, uint32_t groups, int passes, int bits,
    int32_t *__restrict__ order, int32_t *__restrict__ ranks, int32_t *__restrict__ offsets) {
    __shared__ uint32_t s_key[ITEMS * kGroupBlock];
    __shared__ uint16_t s_pos[ITEMS * kGroupBlock];
    __shared__ uint32_t s_cnt[kGroupWaves][kDigits];
    __shared__ uint32_t s_start[kDigits];
    __shared__ uint32_t s_wave[kGroupWaves];
    __shared__ GapList s_gaps;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t digits = 1u << bits;
    const uint32_t first = static_cast<uint32_t>(w) * kWave * ITEMS + lane;
    uint32_t key[ITEMS], pos[ITEMS], rk[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = first + j * kWave;
        pos[j] = i;
        key[j] = i < n ? key_of(keys[i], groups) : 0u;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        for (uint32_t d = threadIdx.x; d < digits * kGroupWaves; d += kGroupBlock)
            s_cnt[d >> bits][d & (digits - 1)] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
            rk[j] = digit_rank((key[j] >> shift) & (digits - 1), first + j * kWave < n, bits, s_cnt[w]);
        __syncthreads();
        const uint32_t total = counts_before(s_cnt, digits);
        const uint32_t start = block_exclusive(total, s_wave);
        if (threadIdx.x < digits) s_start[threadIdx.x] = start;
        __syncthreads();
        const bool last = p == passes - 1;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            if (first + j * kWave >= n) continue;
            const uint32_t d = (key[j] >> shift) & (digits - 1);
            const uint32_t at = s_start[d] + s_cnt[w][d] + rk[j];
            s_key[at] = key[j];
            if (!last) {
                s_pos[at] = static_cast<uint16_t>(pos[j]);
            } else {
                const bool kept = key[j] < groups;
                if (order != nullptr && kept) order[at] = static_cast<int32_t>(pos[j]);
                if (ranks != nullptr) ranks[pos[j]] = kept ? static_cast<int32_t>(at) : -1;
            }
        }
        __syncthreads();
        if (!last) {
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                const uint32_t i = first + j * kWave;
                if (i < n) {
                    key[j] = s_key[i];
                    pos[j] = s_pos[i];
                }
            }
        }
    }
    if (passes == 1) {  // the digit starts are the offsets
        if (threadIdx.x <= groups) offsets[threadIdx.x] = static_cast<int32_t>(s_start[threadIdx.x]);
    } else {
        fill_offsets([&](uint32_t s) { return s_key[s]; }, 0, n + 1, n, groups, offsets, s_gaps);
    }
}

// The tiled form: a pass is a counting launch and a scattering launch, each
// of up to 256 workgroups that take one span of the keys in steps of 8192.
// table[t][d] = keys of span t with digit d.
template <class K>
__device__ __forceinline__ uint32_t pass_key(const K *keys, const uint32_t *sorted, uint32_t i, uint32_t groups) {
    return sorted != nullptr ? sorted[i] : key_of(keys[i], groups);
}

template <class K>
__global__ __launch_bounds__(kGroupBlock) void group_count_kernel(
    const K *__restrict__ keys, const uint32_t *__restrict__ sorted, uint32_t n, uint32_t span,
    uint32_t groups, int shift, int bits, uint32_t *__restrict__ table) {
    __shared__ uint32_t s_cnt[kDigits];
    const uint32_t digits = 1u << bits;
    if (threadIdx.x < digits) s_cnt[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * span;
    const uint32_t end = n - begin < span ? n : begin + span;
    for (uint32_t i = begin + threadIdx.x; i < end; i += kGroupBlock) {
        const uint32_t d = (pass_key(keys, sorted, i, groups) >> shift) & (digits - 1);
        __hip_atomic_fetch_add(&s_cnt[d], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    if (threadIdx.x < digits) table[blockIdx.x * digits + threadIdx.x] = s_cnt[threadIdx.x];
}

template <class K>
__global__ __launch_bounds__(kGroupBlock) void group_scatter_kernel(
    const K *__restrict__ keys, const uint32_t *__restrict__ sorted, const uint32_t *__restrict__ positions,
    uint32_t n, uint32_t span, uint32_t groups, int shift, int bits, const uint32_t *__restrict__ table,
    uint32_t *__restrict__ sorted_out, uint32_t *__restrict__ positions_out,
    int32_t *__restrict__ order, int32_t *__restrict__ ranks, int32_t *__restrict__ offsets) {
    __shared__ uint32_t s_cnt[kGroupWaves][kDigits];
    __shared__ uint32_t s_part[2][2][kDigits];
    __shared__ uint32_t s_base[kDigits];
    __shared__ uint32_t s_wave[kGroupWaves];
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t digits = 1u << bits;
    // where this span's first key of each digit goes: the keys of smaller
    // digits, then those of the same digit in earlier spans; each half of
    // the workgroup sums half of the table
    {
        const uint32_t d = threadIdx.x % kDigits, half = threadIdx.x / kDigits;
        uint32_t before = 0, all = 0;
        if (d < digits) {
#pragma unroll 8
            for (uint32_t t = half; t < gridDim.x; t += 2) {
                const uint32_t c = table[t * digits + d];
                all += c;
                before += t < blockIdx.x ? c : 0u;
            }
        }
        s_part[half][0][d] = before;
        s_part[half][1][d] = all;
    }
    __syncthreads();
    uint32_t total = 0, base = 0;
    if (threadIdx.x < digits) {
        total = s_part[0][1][threadIdx.x] + s_part[1][1][threadIdx.x];
        base = s_part[0][0][threadIdx.x] + s_part[1][0][threadIdx.x];
    }
    const uint32_t start = block_exclusive(total, s_wave);
    if (threadIdx.x < digits) {
        s_base[threadIdx.x] = start + base;
        if (offsets != nullptr && blockIdx.x == 0 && threadIdx.x <= groups)
            offsets[threadIdx.x] = static_cast<int32_t>(start);
    }
    const uint32_t begin = blockIdx.x * span;
    const uint32_t end = n - begin < span ? n : begin + span;
    for (uint32_t step = begin; step < end; step += kGroupStep) {
        for (uint32_t d = threadIdx.x; d < digits * kGroupWaves; d += kGroupBlock)
            s_cnt[d >> bits][d & (digits - 1)] = 0;
        const uint32_t first = step + static_cast<uint32_t>(w) * kWave * kGroupItems + lane;
        uint32_t key[kGroupItems], rk[kGroupItems];
#pragma unroll
        for (int j = 0; j < kGroupItems; ++j) {
            const uint32_t i = first + j * kWave;
            key[j] = i < end ? pass_key(keys, sorted, i, groups) : 0u;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kGroupItems; ++j)
            rk[j] = digit_rank((key[j] >> shift) & (digits - 1), first + j * kWave < end, bits, s_cnt[w]);
        __syncthreads();
        const uint32_t count = counts_before(s_cnt, digits);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kGroupItems; ++j) {
            const uint32_t i = first + j * kWave;
            if (i >= end) continue;
            const uint32_t d = (key[j] >> shift) & (digits - 1);
            const uint32_t at = s_base[d] + s_cnt[w][d] + rk[j];
            if (at >= n) continue;  // only a table changed under the call
            const uint32_t pos = positions != nullptr ? positions[i] : i;
            if (sorted_out != nullptr) sorted_out[at] = key[j];
            if (positions_out != nullptr) {
                positions_out[at] = pos;
            } else {
                const bool kept = key[j] < groups;
                if (order != nullptr && kept) order[at] = static_cast<int32_t>(pos);
                if (ranks != nullptr) ranks[pos] = kept ? static_cast<int32_t>(at) : -1;
            }
        }
        __syncthreads();
        if (threadIdx.x < digits) s_base[threadIdx.x] += count;
    }
}

__global__ __launch_bounds__(kGroupBlock) void group_offsets_kernel(const uint32_t *__restrict__ sorted,
                                                                   uint32_t n, uint32_t groups,
                                                                   int32_t *__restrict__ offsets) {
    __shared__ GapList s_gaps;
    const uint32_t s0 = blockIdx.x * kGroupBlock;
    const uint32_t s1 = n + 1 - s0 < kGroupBlock ? n + 1 : s0 + kGroupBlock;
    fill_offsets([&](uint32_t s) { return sorted[s]; }, s0, s1, n, groups, offsets, s_gaps);
}

__global__ __launch_bounds__(256) void fill_zero_kernel(uint32_t *__restrict__ p, int64_t words) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < words; i += gridDim.x * 256ll) p[i] = 0;
}

// ============================================================== rows ---
// A chunk is what one lane moves at a time: 16 bytes, or one element where
// the row is shorter than that. The last chunk of a row whose width is no
// multiple of the chunk starts early, so that it is whole; `skip` of its
// elements belong to the chunk before it and are computed twice. Rows need
// no alignment beyond their element's: gfx950 takes unaligned 16-byte
// global accesses.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <class T, bool VEC>
struct Chunk {
    static constexpr int kN = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    float f[kN];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < kN; ++e) f[e] = 0.0f;
    }
    __device__ __forceinline__ void load(const T *p) {
        typedef T V __attribute__((ext_vector_type(kN)));
        if constexpr (VEC) {
            const u32x4 r = *reinterpret_cast<const u32x4_any *>(p);
            const V v = __builtin_bit_cast(V, r);
#pragma unroll
            for (int e = 0; e < kN; ++e) f[e] = static_cast<float>(v[e]);
        } else {
            f[0] = static_cast<float>(*p);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        typedef T V __attribute__((ext_vector_type(kN)));
        if constexpr (VEC) {
            V v;
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = static_cast<T>(f[e]);
            *reinterpret_cast<u32x4_any *>(p) = __builtin_bit_cast(u32x4, v);
        } else {
            *p = static_cast<T>(f[0]);
        }
    }
};

// N fp32 values to and from consecutive elements of type G.
template <class G, int N>
__device__ __forceinline__ void load_values(const G *p, float *f) {
    constexpr bool VEC = sizeof(G) * N % 16 == 0;
    using C = Chunk<G, VEC>;
#pragma unroll
    for (int i = 0; i < N / C::kN; ++i) {
        C v;
        v.load(p + i * C::kN);
#pragma unroll
        for (int e = 0; e < C::kN; ++e) f[i * C::kN + e] = v.f[e];
    }
}
template <class G, int N>
__device__ __forceinline__ void store_values(G *p, const float *f) {
    constexpr bool VEC = sizeof(G) * N % 16 == 0;
    using C = Chunk<G, VEC>;
#pragma unroll
    for (int i = 0; i < N / C::kN; ++i) {
        C v;
#pragma unroll
        for (int e = 0; e < C::kN; ++e) v.f[e] = f[i * C::kN + e];
        v.store(p + i * C::kN);
    }
}

// Which row and which of its chunks a thread works on: 2^lg threads to a
// row, the column blocks in gridDim.y.
struct RowMap {
    int lg;          // log2 of the threads of a row (0 .. 8)
    int chunks;      // chunks of a row
    int width;       // elements of a row
};
constexpr int kRowBlock = 256;

__device__ __forceinline__ int64_t row_of(const RowMap &m) {
    const uint32_t sub = threadIdx.x >> m.lg;
    return (static_cast<int64_t>(blockIdx.x) << (8 - m.lg)) + (m.lg >= 6 ? uniform(sub) : sub);
}
__device__ __forceinline__ int col_of(const RowMap &m) {
    return static_cast<int>((blockIdx.y << m.lg) + (threadIdx.x & ((1u << m.lg) - 1u)));
}
__device__ __forceinline__ int col_step(const RowMap &m) { return static_cast<int>(gridDim.y << m.lg); }

template <int N>
__device__ __forceinline__ int chunk_start(int c, int width) {
    const int at = c * N;
    return at + N <= width ? at : width - N;
}

template <class T, bool VEC, class I>
__global__ __launch_bounds__(kRowBlock) void embed_kernel(const T *__restrict__ table, int64_t vocab,
                                                          const I *__restrict__ ids, int64_t n, float scale,
                                                          T *__restrict__ out, RowMap m) {
    using C = Chunk<T, VEC>;
    const int64_t row = row_of(m);
    if (row >= n) return;
    const int64_t id = ids[row];
    const bool inside = id >= 0 && id < vocab;
    const T *src = table + (inside ? id : 0) * m.width;
    T *dst = out + row * m.width;
    for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
        const int at = chunk_start<C::kN>(c, m.width);
        C x;
        x.zero();
        if (inside) x.load(src + at);
#pragma unroll
        for (int e = 0; e < C::kN; ++e) x.f[e] *= scale;
        x.store(dst + at);
    }
}

template <class T, bool VEC>
__global__ __launch_bounds__(kRowBlock) void dispatch_kernel(const T *__restrict__ x, int64_t tokens, int per,
                                                             const int32_t *__restrict__ ranks, int64_t rows,
                                                             T *__restrict__ out, RowMap m) {
    using C = Chunk<T, VEC>;
    const int64_t t = row_of(m);
    if (t >= tokens) return;
    const T *src = x + t * m.width;
    const int32_t *rk = ranks + t * per;
    for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
        const int at = chunk_start<C::kN>(c, m.width);
        C v;
        v.load(src + at);
        for (int k = 0; k < per; ++k) {
            const int64_t r = rk[k];
            if (r >= 0 && r < rows) v.store(out + r * m.width + at);
        }
    }
}

template <class T, bool VEC, bool WEIGHTED>
__global__ __launch_bounds__(kRowBlock) void combine_kernel(const T *__restrict__ y, int64_t rows,
                                                            const int32_t *__restrict__ ranks,
                                                            const float *__restrict__ weights, int64_t tokens,
                                                            int per, T *__restrict__ out, RowMap m) {
    using C = Chunk<T, VEC>;
    const int64_t t = row_of(m);
    if (t >= tokens) return;
    const int32_t *rk = ranks + t * per;
    const float *wt = weights + t * per;
    for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
        const int at = chunk_start<C::kN>(c, m.width);
        C acc;
        acc.zero();
#pragma unroll 4
        for (int k = 0; k < per; ++k) {
            const int64_t r = rk[k];
            const bool ok = r >= 0 && r < rows;
            const float w = WEIGHTED ? wt[k] : 1.0f;
            if (ok) {
                C v;
                v.load(y + r * m.width + at);
#pragma unroll
                for (int e = 0; e < C::kN; ++e) acc.f[e] = __builtin_fmaf(w, v.f[e], acc.f[e]);
            }
        }
        acc.store(out + t * m.width + at);
    }
}

// Sum over the 2^lg threads of a row, in thread 0 of the row.
__device__ __forceinline__ float row_sum(float v, int lg, float *s_wave) {
    for (int off = 1 << (lg < 6 ? lg : 6); off > 1; off >>= 1) v += __shfl_xor(v, off >> 1);
    if (lg <= 6) return v;
    const int w = static_cast<int>(threadIdx.x / kWave);
    __syncthreads();
    if (lane_id() == 0) s_wave[w] = v;
    __syncthreads();
    const int waves = 1 << (lg - 6), w0 = w & ~(waves - 1);
    float t = 0.0f;
    for (int i = 0; i < waves; ++i) t += s_wave[w0 + i];
    return t;
}

// One token's dout row meets its `per` rows of y: each chunk of dout is read
// once for up to kGradPer of them.
constexpr int kGradPer = 8;

template <class T, bool VEC>
__global__ __launch_bounds__(kRowBlock) void combine_grad_kernel(
    const T *__restrict__ dout, const T *__restrict__ y, int64_t rows, const int32_t *__restrict__ ranks,
    const float *__restrict__ weights, int64_t tokens, int per, T *__restrict__ dy,
    float *__restrict__ dweights, RowMap m) {
    using C = Chunk<T, VEC>;
    __shared__ float s_wave[kRowBlock / kWave];
    const int64_t row = row_of(m);
    const bool live = row < tokens;       // threads of no row still meet the barriers
    const int64_t t = live ? row : tokens - 1;
    const int32_t *rk = ranks + t * per;
    const float *wt = weights + t * per;
    const T *src = dout + t * m.width;
    for (int k0 = 0; k0 < per; k0 += kGradPer) {
        float dot[kGradPer];
#pragma unroll
        for (int j = 0; j < kGradPer; ++j) dot[j] = 0.0f;
        if (live) {
            for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
                const int at = chunk_start<C::kN>(c, m.width);
                const int skip = c * C::kN - at;
                C d;
                d.load(src + at);
#pragma unroll
                for (int j = 0; j < kGradPer; ++j) {
                    if (k0 + j >= per) continue;
                    const int64_t r = rk[k0 + j];
                    if (r < 0 || r >= rows) continue;
                    const float w = wt[k0 + j];
                    C v, g;
                    v.load(y + r * m.width + at);
#pragma unroll
                    for (int e = 0; e < C::kN; ++e) {
                        g.f[e] = w * d.f[e];
                        dot[j] = __builtin_fmaf(e >= skip ? d.f[e] : 0.0f, e >= skip ? v.f[e] : 0.0f, dot[j]);
                    }
                    g.store(dy + r * m.width + at);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kGradPer; ++j) {
            if (k0 + j >= per) break;  // the same in every thread
            const float s = row_sum(dot[j], m.lg, s_wave);
            if (live && (threadIdx.x & ((1u << m.lg) - 1u)) == 0) dweights[t * per + k0 + j] = s;
        }
    }
}

// ------------------------------------------- gradient of the embedding ---
// The tokens of a vocabulary row are consecutive in `order`. A row with few
// tokens is summed by the threads that write it. For the frequent ones,
// sums over aligned blocks of 16, 256 and 4096 sorted positions that hold
// one id only are made first (a launch a level), and a row then adds the
// largest blocks that fit into its range, at most 30 of a level: the work
// per row stays even when one id takes the whole batch, with no atomics, in
// an order that the offsets fix.
constexpr int kSumLevels = 3;
constexpr int kSumLg = 4;  // 16 positions to a block, 16 blocks to a block of the next level

struct BlockSums {
    float *level[kSumLevels];  // [n / 16^(l + 1)][width]
    int levels;
};

// ids of the block's first and last position are the same
template <class I>
__device__ __forceinline__ bool one_id(const I *ids, const int32_t *order, int64_t lo, int64_t hi, uint32_t n,
                                       int64_t vocab) {
    const uint32_t i0 = static_cast<uint32_t>(order[lo]), i1 = static_cast<uint32_t>(order[hi]);
    if (i0 >= n || i1 >= n) return false;
    const int64_t a = ids[i0], b = ids[i1];
    return a == b && a >= 0 && a < vocab;
}

template <class T, bool VEC, class I>
__global__ __launch_bounds__(kRowBlock) void grad_blocks_kernel(
    const T *__restrict__ dout, const I *__restrict__ ids, const int32_t *__restrict__ order,
    const int32_t *__restrict__ offsets, uint32_t n, int64_t vocab, int level, BlockSums sums, RowMap m) {
    using C = Chunk<T, VEC>;
    const int lg = kSumLg * (level + 1);
    const int64_t block = row_of(m);
    const int64_t lo = block << lg, hi = lo + (int64_t{1} << lg) - 1;
    const int64_t kept = offsets[vocab] < static_cast<int64_t>(n) ? offsets[vocab] : n;
    if (hi >= kept || !one_id(ids, order, lo, hi, n, vocab)) return;
    float *dst = sums.level[level] + block * m.width;
    for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
        const int at = chunk_start<C::kN>(c, m.width);
        float acc[C::kN];
#pragma unroll
        for (int e = 0; e < C::kN; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int j = 0; j < (1 << kSumLg); ++j) {
            if (level == 0) {
                const uint32_t i = static_cast<uint32_t>(order[lo + j]);
                if (i >= n) continue;
                C v;
                v.load(dout + static_cast<int64_t>(i) * m.width + at);
#pragma unroll
                for (int e = 0; e < C::kN; ++e) acc[e] += v.f[e];
            } else {
                float p[C::kN];
                load_values<float, C::kN>(sums.level[level - 1] + ((block << kSumLg) + j) * m.width + at, p);
#pragma unroll
                for (int e = 0; e < C::kN; ++e) acc[e] += p[e];
            }
        }
        store_values<float, C::kN>(dst + at, acc);
    }
}

template <class T, bool VEC, class G>
__global__ __launch_bounds__(kRowBlock) void embed_grad_kernel(
    const T *__restrict__ dout, const int32_t *__restrict__ order, const int32_t *__restrict__ offsets,
    uint32_t n, int64_t vocab, float scale, int accumulate, BlockSums sums, G *__restrict__ grad, RowMap m) {
    using C = Chunk<T, VEC>;
    constexpr int N = C::kN;
    const int64_t v = row_of(m);
    if (v >= vocab) return;
    const uint32_t a = static_cast<uint32_t>(offsets[v]);
    uint32_t b = static_cast<uint32_t>(offsets[v + 1]);
    if (b > n) b = n;
    if (accumulate && a >= b) return;
    G *dst = grad + v * m.width;
    for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
        const int at = chunk_start<N>(c, m.width);
        const int skip = c * N - at;
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        for (uint32_t s = a; s < b;) {
            // the largest block that starts here and ends inside, and the
            // run of its level up to the next larger block
            int l = 0;
            while (l < sums.levels && (s & ((1u << (kSumLg * (l + 1))) - 1u)) == 0 &&
                   b - s >= (1u << (kSumLg * (l + 1))))
                ++l;
            const int lg = kSumLg * l;
            uint32_t count = (b - s) >> lg;
            if (l < sums.levels) {
                const uint32_t left = (1u << kSumLg) - ((s >> lg) & ((1u << kSumLg) - 1u));
                count = count < left ? count : left;
            }
            if (l == 0) {
#pragma unroll 4
                for (uint32_t j = 0; j < count; ++j) {
                    const uint32_t i = static_cast<uint32_t>(order[s + j]);
                    if (i >= n) continue;
                    C x;
                    x.load(dout + static_cast<int64_t>(i) * m.width + at);
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] += x.f[e];
                }
            } else {
                const float *p = sums.level[l - 1] + static_cast<int64_t>(s >> lg) * m.width + at;
#pragma unroll 4
                for (uint32_t j = 0; j < count; ++j) {
                    float x[N];
                    load_values<float, N>(p + static_cast<int64_t>(j) * m.width, x);
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] += x[e];
                }
            }
            s += count << lg;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= scale;
        if (skip == 0) {
            if (accumulate) {
                float old[N];
                load_values<G, N>(dst + at, old);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += old[e];
            }
            store_values<G, N>(dst + at, acc);
        } else {  // elements that another lane owns are not added to twice
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (e < skip) continue;
                dst[at + e] = static_cast<G>(accumulate ? static_cast<float>(dst[at + e]) + acc[e] : acc[e]);
            }
        }
    }
}

// ============================================================ host side ---
int bits_of(uint64_t v) { return v == 0 ? 1 : 64 - __builtin_clzll(v); }

struct GroupPlan {
    int bits, passes;
    uint32_t tiles, span;
    size_t table_bytes, bytes;
};

GroupPlan group_plan(int64_t n, int64_t groups) {
    GroupPlan p{};
    const int all = bits_of(static_cast<uint64_t>(groups));  // values 0 .. groups
    p.passes = (all + kDigitBits - 1) / kDigitBits;
    p.bits = (all + p.passes - 1) / p.passes;
    if (n <= kGroupSmall) return p;
    int64_t tiles = (n + kGroupStep - 1) / kGroupStep;
    if (tiles > kGroupTiles) tiles = kGroupTiles;
    int64_t span = (n + tiles - 1) / tiles;
    span = (span + kGroupBlock - 1) / kGroupBlock * kGroupBlock;
    p.span = static_cast<uint32_t>(span);
    p.tiles = static_cast<uint32_t>((n + span - 1) / span);
    p.table_bytes = (static_cast<size_t>(p.tiles) << p.bits) * 4;
    p.bytes = p.table_bytes;
    // (key, position) between passes; the last pass leaves its sorted keys
    if (p.passes > 1) p.bytes += static_cast<size_t>(n) * 4 * (p.passes > 2 ? 4 : 3);
    return p;
}

bool group_sizes_ok(int64_t n, int64_t groups) {
    return n >= 0 && n <= INT32_MAX && groups >= 1 && groups <= INT32_MAX - 1;
}

template <class K>
int launch_small(const K *keys, uint32_t n, uint32_t groups, const GroupPlan &p, int32_t *order, int32_t *ranks,
                 int32_t *offsets, hipStream_t s) {
    const dim3 one(1), block(kGroupBlock);
    if (n <= kGroupBlock)
        hipLaunchKernelGGL((group_small_kernel<K, 1>), one, block, 0, s, keys, n, groups, p.passes, p.bits, order,
                           ranks, offsets);
    else if (n <= 4 * kGroupBlock)
        hipLaunchKernelGGL((group_small_kernel<K, 4>), one, block, 0, s, keys, n, groups, p.passes, p.bits, order,
                           ranks, offsets);
    else
        hipLaunchKernelGGL((group_small_kernel<K, 16>), one, block, 0, s, keys, n, groups, p.passes, p.bits, order,
                           ranks, offsets);
    return launched();
}

template <class K>
int group_impl(const K *keys, int64_t n, int64_t groups, int32_t *order, int32_t *ranks, int32_t *offsets,
               void *scratch, size_t scratch_bytes, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (n < 0 || groups < 1) return SSC_ERR_ARG;
    if (!group_sizes_ok(n, groups)) return SSC_ERR_SIZE;
    if (offsets == nullptr || (n > 0 && keys == nullptr)) return SSC_ERR_ARG;
    if (!aligned(keys, sizeof(K)) || !aligned(order, 4) || !aligned(ranks, 4) || !aligned(offsets, 4))
        return SSC_ERR_ARG;
    const GroupPlan p = group_plan(n, groups);
    const size_t bytes = static_cast<size_t>(n) * 4;
    if (p.bytes > 0 && (scratch == nullptr || !aligned(scratch, 8) || scratch_bytes < p.bytes))
        return SSC_ERR_SCRATCH;
    const Span arrays[] = {{keys, static_cast<size_t>(n) * sizeof(K)},
                           {order, bytes},
                           {ranks, bytes},
                           {offsets, (static_cast<size_t>(groups) + 1) * 4},
                           {scratch, p.bytes}};
    if (spans_overlap(arrays)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (n == 0) {
        const int64_t words = groups + 1;
        const int64_t blocks = (words + 255) / 256;
        hipLaunchKernelGGL(fill_zero_kernel, dim3(static_cast<unsigned>(blocks < 1024 ? blocks : 1024)), dim3(256),
                           0, s, reinterpret_cast<uint32_t *>(offsets), words);
        return launched();
    }
    const uint32_t un = static_cast<uint32_t>(n), ug = static_cast<uint32_t>(groups);
    if (n <= kGroupSmall) return launch_small(keys, un, ug, p, order, ranks, offsets, s);
    uint32_t *table = static_cast<uint32_t *>(scratch);
    uint32_t *buf[2][2];  // keys and positions of the two sides
    uint32_t *at = table + p.table_bytes / 4;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j, at += n) buf[i][j] = at;
    const uint32_t *sorted = nullptr, *positions = nullptr;
    const dim3 grid(p.tiles), block(kGroupBlock);
    for (int q = 0; q < p.passes; ++q) {
        const bool last = q == p.passes - 1;
        hipLaunchKernelGGL((group_count_kernel<K>), grid, block, 0, s, keys, sorted, un, p.span, ug, q * p.bits,
                           p.bits, table);
        SSC_TRY(launched());
        hipLaunchKernelGGL((group_scatter_kernel<K>), grid, block, 0, s, keys, sorted, positions, un, p.span, ug,
                           q * p.bits, p.bits, static_cast<const uint32_t *>(table),
                           p.passes == 1 ? nullptr : buf[q & 1][0], last ? nullptr : buf[q & 1][1],
                           last ? order : nullptr, last ? ranks : nullptr, p.passes == 1 ? offsets : nullptr);
        SSC_TRY(launched());
        sorted = buf[q & 1][0];
        positions = buf[q & 1][1];
    }
    if (p.passes > 1) {
        hipLaunchKernelGGL(group_offsets_kernel, dim3(un / kGroupBlock + 1), block, 0, s, sorted, un, ug, offsets);
        return launched();
    }
    return SSC_OK;
}

size_t elem_bytes(int dtype) { return dtype == SSC_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == SSC_F32 || dtype == SSC_BF16 || dtype == SSC_F16; }

// Calls f with the element type of dtype and whether a row holds a 16-byte chunk.
template <class F>
int with_type(int dtype, int64_t width, F f) {
    const bool vec = width * static_cast<int64_t>(elem_bytes(dtype)) >= 16;
    switch (dtype) {
    case SSC_F32: return vec ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
    case SSC_BF16: return vec ? f(__bf16{}, std::true_type{}) : f(__bf16{}, std::false_type{});
    default: return vec ? f(_Float16{}, std::true_type{}) : f(_Float16{}, std::false_type{});
    }
}

// A wavefront to a row, or the few threads that a short row needs; where the
// rows are too few to fill the chip (fewer than two workgroups a compute
// unit), more threads to a row, and columns over several workgroups (split).
struct RowLaunch {
    RowMap map;
    dim3 grid;
};

RowLaunch row_launch(int64_t rows, int64_t width, int per_chunk, bool split) {
    RowLaunch r{};
    r.map.width = static_cast<int>(width);
    r.map.chunks = static_cast<int>((width + per_chunk - 1) / per_chunk);
    const int64_t enough = 512;
    int lg = 0;
    while (lg < 6 && (1 << lg) < r.map.chunks) ++lg;
    while (lg < 8 && (1 << lg) < r.map.chunks && (rows >> (8 - lg)) < enough) ++lg;
    r.map.lg = lg;
    const int64_t blocks = (rows + (256 >> lg) - 1) >> (8 - lg);
    int64_t cols = 1;
    const int64_t most = (r.map.chunks + (1 << lg) - 1) >> lg;
    while (split && cols < most && cols < 64 && blocks * cols < enough) ++cols;
    r.grid = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(cols));
    return r;
}

// Element type and width of a row; byte extents of INT32_MAX rows then fit
// into 63 bits.
int check_rows(int dtype, int64_t width) {
    if (!dtype_ok(dtype) || width < 1) return SSC_ERR_ARG;
    return width > (1 << 28) ? SSC_ERR_SIZE : SSC_OK;
}

template <class I>
int embed_impl(const void *table, int dtype, int64_t vocab, int64_t width, const I *ids, int64_t n, float scale,
               void *out, void *stream) {
    SSC_TRY(check_rows(dtype, width));
    if (n < 0 || vocab < 0) return SSC_ERR_ARG;
    if (n > INT32_MAX || vocab > INT32_MAX) return SSC_ERR_SIZE;
    if (n > 0 && (ids == nullptr || out == nullptr || (vocab > 0 && table == nullptr))) return SSC_ERR_ARG;
    const size_t es = elem_bytes(dtype);
    if (!aligned(table, es) || !aligned(out, es) || !aligned(ids, sizeof(I))) return SSC_ERR_ARG;
    const Span arrays[] = {{out, static_cast<size_t>(n) * width * es},
                           {table, static_cast<size_t>(vocab) * width * es},
                           {ids, static_cast<size_t>(n) * sizeof(I)}};
    for (int i = 1; i < 3; ++i)
        if (overlap(arrays[0].p, arrays[0].bytes, arrays[i].p, arrays[i].bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (n == 0) return SSC_OK;
    return with_type(dtype, width, [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr bool V = decltype(vec)::value;
        const RowLaunch r = row_launch(n, width, Chunk<T, V>::kN, true);
        hipLaunchKernelGGL((embed_kernel<T, V, I>), r.grid, dim3(kRowBlock), 0, static_cast<hipStream_t>(stream),
                           static_cast<const T *>(table), vocab, ids, n, scale, static_cast<T *>(out), r.map);
        return launched();
    });
}

int sum_levels(int64_t n) {
    int l = 0;
    while (l < kSumLevels && n >> (kSumLg * (l + 2)) > 0) ++l;
    return l;
}

size_t grad_scratch(int64_t n, int64_t width) {
    size_t rows = 0;
    for (int l = 0; l < sum_levels(n); ++l) rows += static_cast<size_t>(n >> (kSumLg * (l + 1)));
    return rows * static_cast<size_t>(width) * sizeof(float);
}

template <class I>
int embed_grad_impl(const void *dout, int dtype, int64_t n, int64_t width, const I *ids, const int32_t *order,
                    const int32_t *offsets, int64_t vocab, float scale, void *grad, int grad_dtype, int accumulate,
                    void *scratch, size_t scratch_bytes, void *stream) {
    SSC_TRY(check_rows(dtype, width));
    if (!dtype_ok(grad_dtype) || (grad_dtype != dtype && grad_dtype != SSC_F32)) return SSC_ERR_ARG;
    if (n < 0 || vocab < 1) return SSC_ERR_ARG;
    if (n > INT32_MAX || vocab > INT32_MAX - 1) return SSC_ERR_SIZE;
    if (offsets == nullptr || grad == nullptr ||
        (n > 0 && (dout == nullptr || ids == nullptr || order == nullptr)))
        return SSC_ERR_ARG;
    const size_t es = elem_bytes(dtype), gs = elem_bytes(grad_dtype);
    if (!aligned(dout, es) || !aligned(grad, gs) || !aligned(ids, sizeof(I)) || !aligned(order, 4) ||
        !aligned(offsets, 4))
        return SSC_ERR_ARG;
    const size_t need = grad_scratch(n, width);
    if (need > 0 && (scratch == nullptr || !aligned(scratch, 8) || scratch_bytes < need)) return SSC_ERR_SCRATCH;
    const Span written[] = {{grad, static_cast<size_t>(vocab) * width * gs}, {scratch, need}};
    const Span read[] = {{dout, static_cast<size_t>(n) * width * es},
                         {ids, static_cast<size_t>(n) * sizeof(I)},
                         {order, static_cast<size_t>(n) * 4},
                         {offsets, (static_cast<size_t>(vocab) + 1) * 4}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &w : written)
        for (const Span &r : read)
            if (overlap(w.p, w.bytes, r.p, r.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint32_t un = static_cast<uint32_t>(n);
    return with_type(dtype, width, [&](auto t, auto vec) -> int {
        using T = decltype(t);
        constexpr bool V = decltype(vec)::value;
        BlockSums sums{};
        sums.levels = sum_levels(n);
        float *at = static_cast<float *>(scratch);
        for (int l = 0; l < sums.levels; ++l) {
            const int64_t blocks = n >> (kSumLg * (l + 1));
            sums.level[l] = at;
            at += blocks * width;
        }
        for (int l = 0; l < sums.levels; ++l) {
            const RowLaunch r = row_launch(n >> (kSumLg * (l + 1)), width, Chunk<T, V>::kN, true);
            hipLaunchKernelGGL((grad_blocks_kernel<T, V, I>), r.grid, dim3(kRowBlock), 0, s,
                               static_cast<const T *>(dout), ids, order, offsets, un, vocab, l, sums, r.map);
            SSC_TRY(launched());
        }
        const RowLaunch r = row_launch(vocab, width, Chunk<T, V>::kN, true);
        if (grad_dtype == dtype)
            hipLaunchKernelGGL((embed_grad_kernel<T, V, T>), r.grid, dim3(kRowBlock), 0, s,
                               static_cast<const T *>(dout), order, offsets, un, vocab, scale, accumulate, sums,
                               static_cast<T *>(grad), r.map);
        else
            hipLaunchKernelGGL((embed_grad_kernel<T, V, float>), r.grid, dim3(kRowBlock), 0, s,
                               static_cast<const T *>(dout), order, offsets, un, vocab, scale, accumulate, sums,
                               static_cast<float *>(grad), r.map);
        return launched();
    });
}

// The sizes that the routed calls share: tokens x per slots, rows of y.
int check_routed(int dtype, int64_t tokens, int64_t per, int64_t width, int64_t rows) {
    SSC_TRY(check_rows(dtype, width));
    if (tokens < 0 || per < 1 || rows < 0) return SSC_ERR_ARG;
    if (tokens > INT32_MAX || per > INT32_MAX || tokens * per > INT32_MAX || rows > INT32_MAX) return SSC_ERR_SIZE;
    return SSC_OK;
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

size_t ssc_group_scratch_bytes(int64_t n, int64_t groups) {
    return group_sizes_ok(n, groups) ? group_plan(n, groups).bytes : 0;
}

int ssc_group_by_key_i32(const int32_t *keys, int64_t n, int64_t groups, int32_t *order, int32_t *ranks,
                         int32_t *offsets, void *scratch, size_t scratch_bytes, void *stream) {
    return group_impl(keys, n, groups, order, ranks, offsets, scratch, scratch_bytes, stream);
}

int ssc_group_by_key_i64(const int64_t *keys, int64_t n, int64_t groups, int32_t *order, int32_t *ranks,
                         int32_t *offsets, void *scratch, size_t scratch_bytes, void *stream) {
    return group_impl(keys, n, groups, order, ranks, offsets, scratch, scratch_bytes, stream);
}

int ssc_embed_rows_i32(const void *table, int dtype, int64_t vocab, int64_t width, const int32_t *ids, int64_t n,
                       float scale, void *out, void *stream) {
    return embed_impl(table, dtype, vocab, width, ids, n, scale, out, stream);
}

int ssc_embed_rows_i64(const void *table, int dtype, int64_t vocab, int64_t width, const int64_t *ids, int64_t n,
                       float scale, void *out, void *stream) {
    return embed_impl(table, dtype, vocab, width, ids, n, scale, out, stream);
}

size_t ssc_embed_grad_scratch_bytes(int64_t n, int64_t width) {
    return n < 0 || n > INT32_MAX || width < 1 ? 0 : grad_scratch(n, width);
}

int ssc_embed_rows_grad_i32(const void *dout, int dtype, int64_t n, int64_t width, const int32_t *ids,
                            const int32_t *order, const int32_t *offsets, int64_t vocab, float scale, void *grad,
                            int grad_dtype, int accumulate, void *scratch, size_t scratch_bytes, void *stream) {
    return embed_grad_impl(dout, dtype, n, width, ids, order, offsets, vocab, scale, grad, grad_dtype, accumulate,
                           scratch, scratch_bytes, stream);
}

int ssc_embed_rows_grad_i64(const void *dout, int dtype, int64_t n, int64_t width, const int64_t *ids,
                            const int32_t *order, const int32_t *offsets, int64_t vocab, float scale, void *grad,
                            int grad_dtype, int accumulate, void *scratch, size_t scratch_bytes, void *stream) {
    return embed_grad_impl(dout, dtype, n, width, ids, order, offsets, vocab, scale, grad, grad_dtype, accumulate,
                           scratch, scratch_bytes, stream);
}

int ssc_dispatch_rows(const void *x, int dtype, int64_t tokens, int64_t per, int64_t width, const int32_t *ranks,
                      int64_t rows, void *out, void *stream) {
    SSC_TRY(check_routed(dtype, tokens, per, width, rows));
    const size_t es = elem_bytes(dtype);
    if (tokens > 0 && (x == nullptr || ranks == nullptr || (rows > 0 && out == nullptr))) return SSC_ERR_ARG;
    if (!aligned(x, es) || !aligned(out, es) || !aligned(ranks, 4)) return SSC_ERR_ARG;
    const size_t out_bytes = static_cast<size_t>(rows) * width * es;
    if (overlap(out, out_bytes, x, static_cast<size_t>(tokens) * width * es) ||
        overlap(out, out_bytes, ranks, static_cast<size_t>(tokens) * per * 4))
        return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (tokens == 0 || rows == 0) return SSC_OK;
    return with_type(dtype, width, [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr bool V = decltype(vec)::value;
        const RowLaunch r = row_launch(tokens, width, Chunk<T, V>::kN, true);
        hipLaunchKernelGGL((dispatch_kernel<T, V>), r.grid, dim3(kRowBlock), 0, static_cast<hipStream_t>(stream),
                           static_cast<const T *>(x), tokens, static_cast<int>(per), ranks, rows,
                           static_cast<T *>(out), r.map);
        return launched();
    });
}

int ssc_combine_rows(const void *y, int dtype, int64_t rows, int64_t width, const int32_t *ranks,
                     const float *weights, int64_t tokens, int64_t per, void *out, void *stream) {
    SSC_TRY(check_routed(dtype, tokens, per, width, rows));
    const size_t es = elem_bytes(dtype);
    if (tokens > 0 && (out == nullptr || ranks == nullptr || (rows > 0 && y == nullptr))) return SSC_ERR_ARG;
    if (!aligned(y, es) || !aligned(out, es) || !aligned(ranks, 4) || !aligned(weights, 4)) return SSC_ERR_ARG;
    const size_t out_bytes = static_cast<size_t>(tokens) * width * es, slot_bytes = static_cast<size_t>(tokens) * per * 4;
    if (overlap(out, out_bytes, y, static_cast<size_t>(rows) * width * es) ||
        overlap(out, out_bytes, ranks, slot_bytes) || overlap(out, out_bytes, weights, slot_bytes))
        return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (tokens == 0) return SSC_OK;
    return with_type(dtype, width, [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr bool V = decltype(vec)::value;
        const RowLaunch r = row_launch(tokens, width, Chunk<T, V>::kN, true);
        if (weights != nullptr)
            hipLaunchKernelGGL((combine_kernel<T, V, true>), r.grid, dim3(kRowBlock), 0,
                               static_cast<hipStream_t>(stream), static_cast<const T *>(y), rows, ranks, weights,
                               tokens, static_cast<int>(per), static_cast<T *>(out), r.map);
        else
            hipLaunchKernelGGL((combine_kernel<T, V, false>), r.grid, dim3(kRowBlock), 0,
                               static_cast<hipStream_t>(stream), static_cast<const T *>(y), rows, ranks, weights,
                               tokens, static_cast<int>(per), static_cast<T *>(out), r.map);
        return launched();
    });
}

int ssc_combine_rows_grad(const void *dout, const void *y, int dtype, int64_t rows, int64_t width,
                          const int32_t *ranks, const float *weights, int64_t tokens, int64_t per, void *dy,
                          float *dweights, void *stream) {
    SSC_TRY(check_routed(dtype, tokens, per, width, rows));
    const size_t es = elem_bytes(dtype);
    if (tokens > 0 && (dout == nullptr || ranks == nullptr || weights == nullptr || dweights == nullptr ||
                       (rows > 0 && (y == nullptr || dy == nullptr))))
        return SSC_ERR_ARG;
    if (!aligned(dout, es) || !aligned(y, es) || !aligned(dy, es) || !aligned(ranks, 4) || !aligned(weights, 4) ||
        !aligned(dweights, 4))
        return SSC_ERR_ARG;
    const size_t row_bytes = static_cast<size_t>(rows) * width * es, slot_bytes = static_cast<size_t>(tokens) * per * 4;
    const Span written[] = {{dy, row_bytes}, {dweights, slot_bytes}};
    const Span read[] = {{dout, static_cast<size_t>(tokens) * width * es},
                         {y, row_bytes},
                         {ranks, slot_bytes},
                         {weights, slot_bytes}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &w : written)
        for (const Span &r : read)
            if (overlap(w.p, w.bytes, r.p, r.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (tokens == 0) return SSC_OK;
    return with_type(dtype, width, [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr bool V = decltype(vec)::value;
        const RowLaunch r = row_launch(tokens, width, Chunk<T, V>::kN, false);
        hipLaunchKernelGGL((combine_grad_kernel<T, V>), r.grid, dim3(kRowBlock), 0, static_cast<hipStream_t>(stream),
                           static_cast<const T *>(dout), static_cast<const T *>(y), rows, ranks, weights, tokens,
                           static_cast<int>(per), static_cast<T *>(dy), dweights, r.map);
        return launched();
    });
}

}  // extern "C"
