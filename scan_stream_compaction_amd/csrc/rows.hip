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
#include "ssc_sets.h"

namespace ssc {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
constexpr int kGroupSmall = 8 * kGroupBlock;    // keys one workgroup sorts alone
constexpr int kGroupFew = 4096;                 // groups whose offsets it then finds itself
constexpr int kGroupTiles = 256;                // most workgroups of a tiled pass

template <class K>
__device__ __forceinline__ uint32_t key_of(K k, uint32_t groups) {
    return k >= 0 && static_cast<uint64_t>(k) < groups ? static_cast<uint32_t>(k) : groups;
}

// Ranks of ITEMS consecutive sets of 64 keys among the keys
// this wavefront has seen, in order; cnt holds the wavefront's counts. The
// lanes' masks do not depend on one another and come first; the counts then
// follow key order.
template <int ITEMS>
__device__ __forceinline__ void digit_ranks(const uint32_t (&d)[ITEMS], const bool (&valid)[ITEMS], int bits,
                                            uint32_t *cnt, uint32_t (&rk)[ITEMS]) {
    uint32_t lo[ITEMS], hi[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint64_t all = ballot(valid[j]);
        lo[j] = static_cast<uint32_t>(all);
        hi[j] = static_cast<uint32_t>(all >> 32);
    }
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        if (b >= bits) continue;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t bit = static_cast<uint32_t>(static_cast<int32_t>(d[j] << (31 - b)) >> 31);  // 0 or all ones
            const uint64_t bb = ballot(bit != 0);
            lo[j] &= ~(static_cast<uint32_t>(bb) ^ bit);
            hi[j] &= ~(static_cast<uint32_t>(bb >> 32) ^ bit);
        }
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t below = __builtin_amdgcn_mbcnt_hi(hi[j], __builtin_amdgcn_mbcnt_lo(lo[j], 0u));
        const uint32_t same = static_cast<uint32_t>(__builtin_popcount(lo[j]) + __builtin_popcount(hi[j]));
        // every lane reads its digit's count before the last lane of the digit
        // raises it, and the next set's lanes read after that
        const uint32_t run = valid[j] ? cnt[d[j]] : 0u;
        wave_lds_order();
        if (valid[j] && below + 1u == same) cnt[d[j]] = run + same;
        wave_lds_order();
        rk[j] = run + below;
    }
}

// Exclusive prefix of v over the workgroup's threads.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t *s_wave) {
    const uint32_t incl = wave_inclusive_scan<SumU32>(v);
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    if (lane == kWave - 1) s_wave[w] = incl;
    __syncthreads();
    const uint32_t totals = wave_inclusive_scan<SumU32>(lane < kGroupWaves ? s_wave[lane] : 0u);
    const uint32_t before =
        w == 0 ? 0u : static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(totals), w - 1));
    return before + incl - v;
}

// The wavefronts' counts of a tile, cnt[w][d], become the counts of earlier
// wavefronts; returns the tile's count of digit threadIdx.x (0 beyond the digits).
__device__ __forceinline__ uint32_t counts_before(uint32_t (*cnt)[kDigits], uint32_t digits) {
    uint32_t total = 0;
    if (threadIdx.x < digits) {
        uint32_t c[kGroupWaves];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) c[w] = cnt[w][threadIdx.x];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            cnt[w][threadIdx.x] = total;
            total += c[w];
        }
    }
    return total;
}

// Number of sorted keys below v, known to lie in [lo, hi].
__device__ __forceinline__ uint32_t keys_below(const uint32_t *sorted, uint32_t lo, uint32_t hi, uint32_t v) {
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        if (sorted[mid] < v)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Up to 8192 keys: one workgroup holds (key, position) in registers and
// exchanges them through LDS between passes. Bound by the instructions of its
// ranks (half of a pass) and the latency of its LDS steps: 128 keys of 128
// groups 2.7 us, 5000 keys in two passes 9.5 (11.4 with the number of sets
// known at run time only). One launch beats the tiled form's two (four) up to
// here: 8000 keys of 64 groups 10.4 us a call against 15.3, of 10,007 groups 23
// against 27.
template <class K, int ITEMS>
__global__ __launch_bounds__(kGroupBlock) void group_small_kernel(
    const K *__restrict__ keys, uint32_t n, uint32_t groups, int passes, int bits,
    int32_t *__restrict__ order, int32_t *__restrict__ ranks, int32_t *__restrict__ offsets,
    uint32_t *__restrict__ sorted_out) {
    __shared__ uint32_t s_key[ITEMS * kGroupBlock];
    __shared__ uint16_t s_pos[ITEMS * kGroupBlock];
    __shared__ uint32_t s_cnt[kGroupWaves][kDigits];
    __shared__ uint32_t s_start[kDigits];
    __shared__ uint32_t s_wave[kGroupWaves];
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t digits = 1u << bits;
    const uint32_t first = static_cast<uint32_t>(w * kWave * ITEMS + lane);
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
        uint32_t dig[ITEMS];
        bool valid[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            dig[j] = (key[j] >> shift) & (digits - 1);
            valid[j] = first + j * kWave < n;
        }
        digit_ranks<ITEMS>(dig, valid, bits, s_cnt[w], rk);
        __syncthreads();
        const uint32_t total = counts_before(s_cnt, digits);
        const uint32_t start = block_exclusive(total, s_wave);
        if (threadIdx.x < digits) s_start[threadIdx.x] = start;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            if (!valid[j]) continue;
            const uint32_t at = s_start[dig[j]] + s_cnt[w][dig[j]] + rk[j];
            s_key[at] = key[j];
            s_pos[at] = static_cast<uint16_t>(pos[j]);
        }
        __syncthreads();
        if (p < passes - 1) {
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                const uint32_t i = first + j * kWave;
                if (valid[j]) {
                    key[j] = s_key[i];
                    pos[j] = s_pos[i];
                }
            }
        }
    }
    // the outputs leave from LDS in order
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = threadIdx.x + j * kGroupBlock;
        if (i < n) {
            key[j] = s_key[i];
            pos[j] = s_pos[i];
            if (sorted_out != nullptr) sorted_out[i] = key[j];
            if (order != nullptr && key[j] < groups) order[i] = static_cast<int32_t>(pos[j]);
        }
    }
    if (passes == 1) {  // the digit starts are the offsets
        if (threadIdx.x <= groups) offsets[threadIdx.x] = static_cast<int32_t>(s_start[threadIdx.x]);
    } else if (sorted_out == nullptr) {  // 0.9 us for each 1024 groups, against a launch of 4 us for any number
        for (uint32_t v = threadIdx.x; v <= groups; v += kGroupBlock)
            offsets[v] = static_cast<int32_t>(keys_below(s_key, 0, n, v));
    }
    if (ranks != nullptr) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t i = threadIdx.x + j * kGroupBlock;
            if (i < n) s_key[pos[j]] = key[j] < groups ? i : ~0u;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t i = threadIdx.x + j * kGroupBlock;
            if (i < n) ranks[i] = static_cast<int32_t>(s_key[i]);
        }
    }
}

// The tiled form: a pass is a counting launch and a scattering launch, each
// of up to 256 workgroups that take one span of the keys in steps.
// table[t][d] = keys of span t with digit d. Spans are as short as 256 of them
// allow (1024 keys at least), for these launches are bound by latency: 65,536
// keys by 9 bits in 64 spans count in 3.5 us and scatter in 8.8, in 8 spans of
// 8192 scatter in 19.5. The scattering workgroups each sum the whole table
// (128 KiB here, in the caches) instead of a third launch doing so.
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

template <class K, int ITEMS>
__global__ __launch_bounds__(kGroupBlock) void group_scatter_kernel(
    const K *__restrict__ keys, const uint32_t *__restrict__ sorted, const uint32_t *__restrict__ positions,
    uint32_t n, uint32_t span, uint32_t groups, int shift, int bits, const uint32_t *__restrict__ table,
    uint32_t *__restrict__ sorted_out, uint32_t *__restrict__ positions_out,
    int32_t *__restrict__ order, int32_t *__restrict__ ranks, int32_t *__restrict__ offsets) {
    __shared__ uint32_t s_cnt[kGroupWaves][kDigits];
    __shared__ __attribute__((aligned(16))) uint32_t s_part[2][4 * kGroupBlock];
    __shared__ uint32_t s_base[kDigits];
    __shared__ uint32_t s_wave[kGroupWaves];
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t digits = 1u << bits;
    const uint32_t begin = blockIdx.x * span;
    const uint32_t end = n - begin < span ? n : begin + span;
    // a step's keys: the first step's are on their way while the table is read
    uint32_t first = begin + static_cast<uint32_t>(w) * kWave * ITEMS + lane;
    uint32_t key[ITEMS], pos[ITEMS];
    const auto load = [&]() {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t i = first + j * kWave;
            key[j] = i < end ? pass_key(keys, sorted, i, groups) : 0u;
            pos[j] = positions != nullptr && i < end ? positions[i] : i;
        }
    };
    load();
    // where this span's first key of each digit goes: the keys of smaller
    // digits, then those of the same digit in earlier spans; a thread sums
    // four digits over every parts-th row of the table
    {
        const uint32_t d = (4 * threadIdx.x) & (digits - 1), parts = (4 * kGroupBlock) >> bits;
        u32x4 before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
#pragma unroll 8
        for (uint32_t t = (4 * threadIdx.x) >> bits; t < gridDim.x; t += parts) {
            const u32x4 c = *reinterpret_cast<const u32x4 *>(table + t * digits + d);
            all += c;
            before += t < blockIdx.x ? c : u32x4{0, 0, 0, 0};
        }
        *reinterpret_cast<u32x4 *>(&s_part[0][4 * threadIdx.x]) = before;
        *reinterpret_cast<u32x4 *>(&s_part[1][4 * threadIdx.x]) = all;
    }
    __syncthreads();
    uint32_t total = 0, base = 0;
    if (threadIdx.x < digits) {
        for (uint32_t i = threadIdx.x; i < 4 * kGroupBlock; i += digits) {
            base += s_part[0][i];
            total += s_part[1][i];
        }
    }
    const uint32_t start = block_exclusive(total, s_wave);
    if (threadIdx.x < digits) {
        s_base[threadIdx.x] = start + base;
        if (offsets != nullptr && blockIdx.x == 0 && threadIdx.x <= groups)
            offsets[threadIdx.x] = static_cast<int32_t>(start);
    }
    for (uint32_t step = begin; step < end; step += ITEMS * kGroupBlock) {
        if (step != begin) {
            first += ITEMS * kGroupBlock;
            load();
        }
        for (uint32_t d = threadIdx.x; d < digits * kGroupWaves; d += kGroupBlock)
            s_cnt[d >> bits][d & (digits - 1)] = 0;
        __syncthreads();
        uint32_t dig[ITEMS], rk[ITEMS];
        bool valid[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            dig[j] = (key[j] >> shift) & (digits - 1);
            valid[j] = first + j * kWave < end;
        }
        digit_ranks<ITEMS>(dig, valid, bits, s_cnt[w], rk);
        __syncthreads();
        const uint32_t count = counts_before(s_cnt, digits);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            if (!valid[j]) continue;
            const uint32_t at = s_base[dig[j]] + s_cnt[w][dig[j]] + rk[j];
            if (at >= n) continue;  // only a table changed under the call
            if (sorted_out != nullptr) sorted_out[at] = key[j];
            if (positions_out != nullptr) {
                positions_out[at] = pos[j];
            } else {
                const bool kept = key[j] < groups;
                if (order != nullptr && kept) order[at] = static_cast<int32_t>(pos[j]);
                if (ranks != nullptr) ranks[pos[j]] = kept ? static_cast<int32_t>(at) : -1;
            }
        }
        __syncthreads();
        if (threadIdx.x < digits) s_base[threadIdx.x] += count;
    }
}

// offsets[v] = number of sorted keys below v, by bisection: first among up
// to 4096 keys at even distances, in LDS, then between two of them.
constexpr uint32_t kSamples = 4096;

__global__ __launch_bounds__(kGroupBlock) void group_offsets_kernel(const uint32_t *__restrict__ sorted,
                                                                   uint32_t n, uint32_t groups,
                                                                   int32_t *__restrict__ offsets) {
    __shared__ uint32_t s_key[kSamples];
    const uint32_t stride = (n + kSamples - 1) / kSamples;
    const uint32_t samples = n / stride;  // the last of each whole stride
    for (uint32_t i = threadIdx.x; i < samples; i += kGroupBlock) s_key[i] = sorted[(i + 1) * stride - 1];
    __syncthreads();
    const uint32_t v = blockIdx.x * kGroupBlock + threadIdx.x;
    if (v > groups) return;
    const uint32_t s = keys_below(s_key, 0, samples, v);  // strides that end below v
    offsets[v] = static_cast<int32_t>(keys_below(sorted, s * stride, s < samples ? (s + 1) * stride - 1 : n, v));
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

template <class T, bool VEC>
struct Chunk {
    static constexpr int kN = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    typedef T V __attribute__((ext_vector_type(kN)));
    using Raw = std::conditional_t<VEC, u32x4, T>;

    __device__ static __forceinline__ Raw load(const T *p) {
        if constexpr (VEC)
            return *reinterpret_cast<const u32x4_any *>(p);
        else
            return *p;
    }
    // what a call reads or writes once goes past the caches
    __device__ static __forceinline__ Raw load_stream(const T *p) {
        if constexpr (VEC)
            return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
        else
            return *p;
    }
    __device__ static __forceinline__ void store_stream(T *p, Raw r) {
        if constexpr (VEC)
            __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any *>(p));
        else
            *p = r;
    }
    __device__ static __forceinline__ Raw none() {
        if constexpr (VEC)
            return u32x4{0, 0, 0, 0};
        else
            return static_cast<T>(0.0f);
    }
    __device__ static __forceinline__ void unpack(Raw r, float *f) {
        if constexpr (VEC) {
            const V v = __builtin_bit_cast(V, r);
#pragma unroll
            for (int e = 0; e < kN; ++e) f[e] = static_cast<float>(v[e]);
        } else {
            f[0] = static_cast<float>(r);
        }
    }
    __device__ static __forceinline__ Raw pack(const float *f) {
        if constexpr (VEC) {
            V v;
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = static_cast<T>(f[e]);
            return __builtin_bit_cast(u32x4, v);
        } else {
            return static_cast<T>(f[0]);
        }
    }
};

// N fp32 values to and from consecutive elements of type G.
template <class G, int N>
__device__ __forceinline__ void load_values(const G *p, float *f) {
    using C = Chunk<G, sizeof(G) * N % 16 == 0>;
#pragma unroll
    for (int i = 0; i < N / C::kN; ++i) C::unpack(C::load(p + i * C::kN), f + i * C::kN);
}
template <class G, int N>
__device__ __forceinline__ void store_values(G *p, const float *f) {
    using C = Chunk<G, sizeof(G) * N % 16 == 0>;
#pragma unroll
    for (int i = 0; i < N / C::kN; ++i) C::store_stream(p + i * C::kN, C::pack(f + i * C::kN));
}

// Which row and which of its chunks a thread works on: 2^lg threads to a
// row, the column blocks in gridDim.y, further rows in gridDim.z (a
// dimension of a launch holds at most 2^32 - 1 threads). WAVE: whole
// wavefronts to a row (lg >= 6), whose ids, ranks and weights then come through
// scalar loads. CH: chunks that a thread has in flight at a time.
struct RowMap {
    int lg;          // log2 of the threads of a row (0 .. 8)
    int chunks;      // chunks of a row
    int width;       // elements of a row
};
constexpr int kRowBlock = 256;

template <bool WAVE>
__device__ __forceinline__ int64_t row_of(const RowMap &m) {
    const uint32_t sub = threadIdx.x >> m.lg;
    const int64_t block = static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x;
    return (block << (8 - m.lg)) + (WAVE ? uniform(sub) : sub);
}
__device__ __forceinline__ int col_of(const RowMap &m) {
    return static_cast<int>((blockIdx.y << m.lg) + (threadIdx.x & ((1u << m.lg) - 1u)));
}
__device__ __forceinline__ int col_step(const RowMap &m) { return static_cast<int>(gridDim.y << m.lg); }

// Where chunk c starts; one past the last stands for the last, which a
// thread may read again but does not write.
template <int N>
__device__ __forceinline__ int chunk_start(int c, const RowMap &m) {
    const int at = (c < m.chunks ? c : m.chunks - 1) * N;
    return at + N <= m.width ? at : m.width - N;
}

// Bound by HBM: 32,768 rows of 4096 bf16 in 61.3 us, 433 MB of traffic with
// what several XCDs read of the same row.
template <class T, bool VEC, bool WAVE, int CH, class I>
__global__ __launch_bounds__(kRowBlock) void embed_kernel(const T *__restrict__ table, int64_t vocab,
                                                          const I *__restrict__ ids, int64_t n, float scale,
                                                          T *__restrict__ out, RowMap m) {
    using C = Chunk<T, VEC>;
    const int64_t row = row_of<WAVE>(m);
    if (row >= n) return;
    const int64_t id = ids[row];
    const bool inside = id >= 0 && id < vocab;
    const T *src = table + (inside ? id : 0) * m.width;
    T *dst = out + row * m.width;
    const int step = col_step(m);
    for (int c0 = col_of(m); c0 < m.chunks; c0 += CH * step) {
        typename C::Raw r[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) r[j] = inside ? C::load(src + chunk_start<C::kN>(c0 + j * step, m)) : C::none();
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float f[C::kN];
            C::unpack(r[j], f);
#pragma unroll
            for (int e = 0; e < C::kN; ++e) f[e] = inside ? f[e] * scale : 0.0f;
            if (c0 + j * step < m.chunks) C::store_stream(dst + chunk_start<C::kN>(c0 + j * step, m), C::pack(f));
        }
    }
}

// By tokens, not by slots: a token's row is read once and stored `per` times.
// Bound by HBM writes: 16,384 tokens x 8 rows of 2048 bf16 in 97 us, 6.1 TB/s.
template <class T, bool VEC, bool WAVE, int CH>
__global__ __launch_bounds__(kRowBlock) void dispatch_kernel(const T *__restrict__ x, int64_t tokens, int per,
                                                             const int32_t *__restrict__ ranks, int64_t rows,
                                                             T *__restrict__ out, RowMap m) {
    using C = Chunk<T, VEC>;
    const int64_t t = row_of<WAVE>(m);
    if (t >= tokens) return;
    const T *src = x + t * m.width;
    const int32_t *rk = ranks + t * per;
    const int step = col_step(m);
    for (int c0 = col_of(m); c0 < m.chunks; c0 += CH * step) {
        typename C::Raw r[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) r[j] = C::load(src + chunk_start<C::kN>(c0 + j * step, m));
        for (int k = 0; k < per; ++k) {
            const int64_t slot = rk[k];
            if (slot < 0 || slot >= rows) continue;
            T *dst = out + slot * m.width;
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (c0 + j * step < m.chunks) C::store_stream(dst + chunk_start<C::kN>(c0 + j * step, m), r[j]);
        }
    }
}

// The rows of K assignments are in flight together, with two chunks of each
// where a thread has more than one: whole rows then go by at a time (8192
// tokens x 8 rows of 4096 bf16: 107 us with 8 rows of one chunk, 103 with 4 of
// two). An assignment without a row loads row 0 and adds nothing.
template <class T, bool VEC, bool WAVE, int CH, bool WEIGHTED>
__global__ __launch_bounds__(kRowBlock) void combine_kernel(const T *__restrict__ y, int64_t rows,
                                                            const int32_t *__restrict__ ranks,
                                                            const float *__restrict__ weights, int64_t tokens,
                                                            int per, T *__restrict__ out, RowMap m) {
    using C = Chunk<T, VEC>;
    constexpr int K = CH == 1 ? 8 : 4;
    const int64_t t = row_of<WAVE>(m);
    if (t >= tokens) return;
    const int32_t *rk = ranks + t * per;
    const float *wt = weights + t * per;
    const int step = col_step(m);
    for (int c0 = col_of(m); c0 < m.chunks; c0 += CH * step) {
        float acc[CH][C::kN];
#pragma unroll
        for (int q = 0; q < CH; ++q) {
#pragma unroll
            for (int e = 0; e < C::kN; ++e) acc[q][e] = 0.0f;
        }
        for (Sets<K> k(rows > 0 ? per : 0); k.more(); k.next()) {
            typename C::Raw r[K][CH];
            float w[K];
            bool ok[K];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (!k.has(j)) continue;
                const int64_t slot = rk[k.at(j)];
                ok[j] = slot >= 0 && slot < rows;
                w[j] = WEIGHTED ? wt[k.at(j)] : 1.0f;
                const T *src = y + (ok[j] ? slot : 0) * m.width;
#pragma unroll
                for (int q = 0; q < CH; ++q) r[j][q] = C::load_stream(src + chunk_start<C::kN>(c0 + q * step, m));
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (!k.has(j) || !ok[j]) continue;
#pragma unroll
                for (int q = 0; q < CH; ++q) {
                    float v[C::kN];
                    C::unpack(r[j][q], v);
#pragma unroll
                    for (int e = 0; e < C::kN; ++e) acc[q][e] = __builtin_fmaf(w[j], v[e], acc[q][e]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < CH; ++q)
            if (c0 + q * step < m.chunks)
                C::store_stream(out + t * m.width + chunk_start<C::kN>(c0 + q * step, m), C::pack(acc[q]));
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

// One token's dout row meets its `per` rows of y, K at a time (8192 tokens x
// 8 rows of 4096 bf16: 222 us with 8 rows of one chunk, 216 with 4 of two
// chunks, 213 with 2).
template <class T, bool VEC, bool WAVE, int CH>
__global__ __launch_bounds__(kRowBlock) void combine_grad_kernel(
    const T *__restrict__ dout, const T *__restrict__ y, int64_t rows, const int32_t *__restrict__ ranks,
    const float *__restrict__ weights, int64_t tokens, int per, T *__restrict__ dy,
    float *__restrict__ dweights, RowMap m) {
    using C = Chunk<T, VEC>;
    constexpr int N = C::kN, K = CH == 1 ? 8 : 2;
    __shared__ float s_wave[kRowBlock / kWave];
    const int64_t row = row_of<WAVE>(m);
    const bool live = row < tokens && rows > 0;  // the other threads still meet the barriers
    const int64_t t = row < tokens ? row : tokens - 1;
    const int32_t *rk = ranks + t * per;
    const float *wt = weights + t * per;
    const T *src = dout + t * m.width;
    const int step = col_step(m);
    for (Sets<K> k(per); k.more(); k.next()) {
        float dot[K];
#pragma unroll
        for (int j = 0; j < K; ++j) dot[j] = 0.0f;
        if (live) {
            for (int c0 = col_of(m); c0 < m.chunks; c0 += CH * step) {
                typename C::Raw dr[CH], r[K][CH];
#pragma unroll
                for (int q = 0; q < CH; ++q) dr[q] = C::load(src + chunk_start<N>(c0 + q * step, m));
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (!k.has(j)) continue;
                    const int64_t slot = rk[k.at(j)];
                    const T *from = y + (slot >= 0 && slot < rows ? slot : 0) * m.width;
#pragma unroll
                    for (int q = 0; q < CH; ++q) r[j][q] = C::load_stream(from + chunk_start<N>(c0 + q * step, m));
                }
#pragma unroll
                for (int q = 0; q < CH; ++q) {
                    const int c = c0 + q * step;
                    if (c >= m.chunks) continue;
                    const int at = chunk_start<N>(c, m);
                    const int skip = c * N - at;  // elements that the chunk before counts
                    float d[N], own[N];
                    C::unpack(dr[q], d);
#pragma unroll
                    for (int e = 0; e < N; ++e) own[e] = e >= skip ? d[e] : 0.0f;
#pragma unroll
                    for (int j = 0; j < K; ++j) {
                        if (!k.has(j)) continue;
                        const int64_t slot = rk[k.at(j)];
                        if (slot < 0 || slot >= rows) continue;
                        const float w = wt[k.at(j)];
                        float v[N], g[N];
                        C::unpack(r[j][q], v);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            g[e] = w * d[e];
                            dot[j] = __builtin_fmaf(own[e], e >= skip ? v[e] : 0.0f, dot[j]);
                        }
                        C::store_stream(dy + slot * m.width + at, C::pack(g));
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (!k.has(j)) continue;  // the same in every thread
            const float s = row_sum(dot[j], m.lg, s_wave);
            if (row < tokens && (threadIdx.x & ((1u << m.lg) - 1u)) == 0) dweights[t * per + k.at(j)] = s;
        }
    }
}

// ------------------------------------------- gradient of the embedding ---
// The tokens of a vocabulary row are consecutive in `order`. A row with few
// tokens is summed by the threads that write it. For the frequent ones,
// sums over aligned blocks of 16, 256 and 4096 sorted positions that hold
// one id only are made first (a launch a level), and a row then adds the
// largest blocks that fit into its range: at most 30 single tokens, 30 blocks
// of each level below the largest one made, and of the largest what the range
// holds, 1023 at most up to 262,143 tokens and then n / 4096 (1,220 for one id
// over 5M tokens, one after another). No atomics, and an order that the
// offsets fix. Bound by HBM: 65,536 tokens over 131,072 rows of 2048 bf16,
// frequencies falling as 1/rank, in 24 us of block sums and 121 us of rows
// (707 MB; writing zeros alone takes 78).
constexpr int kSumLevels = 3;
constexpr int kSumLg = 4;  // 16 positions to a block, 16 blocks to a block of the next level
constexpr int kSumRows = 1 << kSumLg;

struct BlockSums {
    float *level[kSumLevels];  // [n / 16^(l + 1)][width]
    int levels;
};

// The sorted positions that hold tokens of the vocabulary. A block's sum is
// read only where a row's range holds all of it, and made where it may be: the
// two kernels agree on which blocks end before this.
__device__ __forceinline__ uint32_t sorted_tokens(const int32_t *offsets, int64_t vocab, uint32_t n) {
    const uint32_t kept = static_cast<uint32_t>(offsets[vocab]);
    return kept < n ? kept : n;
}

// Whether the block's first and last position hold the same id, as far as
// they hold one: a position outside [0, n) adds nothing to the sum, but leaves
// open whose block it is.
template <class I>
__device__ __forceinline__ bool one_id(const I *ids, const int32_t *order, int64_t lo, int64_t hi, uint32_t n,
                                       int64_t vocab) {
    const uint32_t i0 = static_cast<uint32_t>(order[lo]), i1 = static_cast<uint32_t>(order[hi]);
    if (i0 >= n || i1 >= n) return true;
    const int64_t a = ids[i0], b = ids[i1];
    return a == b && a >= 0 && a < vocab;
}

template <class T, bool VEC, bool WAVE, class I>
__global__ __launch_bounds__(kRowBlock) void grad_blocks_kernel(
    const T *__restrict__ dout, const I *__restrict__ ids, const int32_t *__restrict__ order,
    const int32_t *__restrict__ offsets, uint32_t n, int64_t vocab, int level, BlockSums sums, RowMap m) {
    using C = Chunk<T, VEC>;
    constexpr int N = C::kN;
    const int lg = kSumLg * (level + 1);
    const int64_t block = row_of<WAVE>(m);
    const int64_t lo = block << lg, hi = lo + (int64_t{1} << lg) - 1;
    if (hi >= sorted_tokens(offsets, vocab, n) || !one_id(ids, order, lo, hi, n, vocab)) return;
    float *dst = sums.level[level] + block * m.width;
    for (int c = col_of(m); c < m.chunks; c += col_step(m)) {
        const int at = chunk_start<N>(c, m);
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        if (level == 0) {
            typename C::Raw r[kSumRows];
            bool ok[kSumRows];
#pragma unroll
            for (int j = 0; j < kSumRows; ++j) {
                const uint32_t i = static_cast<uint32_t>(order[lo + j]);
                ok[j] = i < n;
                r[j] = C::load_stream(dout + static_cast<int64_t>(ok[j] ? i : 0) * m.width + at);
            }
#pragma unroll
            for (int j = 0; j < kSumRows; ++j) {
                float v[N];
                C::unpack(r[j], v);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += ok[j] ? v[e] : 0.0f;
            }
        } else {
            const float *p = sums.level[level - 1] + (block << kSumLg) * m.width + at;
#pragma unroll 4
            for (int j = 0; j < kSumRows; ++j) {
                float v[N];
                load_values<float, N>(p + static_cast<int64_t>(j) * m.width, v);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += v[e];
            }
        }
        store_values<float, N>(dst + at, acc);
    }
}

template <class T, bool VEC, bool WAVE, int CH, class G>
__global__ __launch_bounds__(kRowBlock) void embed_grad_kernel(
    const T *__restrict__ dout, const int32_t *__restrict__ order, const int32_t *__restrict__ offsets,
    uint32_t n, int64_t vocab, float scale, int accumulate, BlockSums sums, G *__restrict__ grad, RowMap m) {
    using C = Chunk<T, VEC>;
    constexpr int N = C::kN;
    const int64_t v = row_of<WAVE>(m);
    if (v >= vocab) return;
    const uint32_t a = static_cast<uint32_t>(offsets[v]);
    uint32_t b = static_cast<uint32_t>(offsets[v + 1]);
    const uint32_t kept = sorted_tokens(offsets, vocab, n);
    if (b > kept) b = kept;
    if (accumulate && a >= b) return;
    G *dst = grad + v * m.width;
    const int step = col_step(m);
    for (int c0 = col_of(m); c0 < m.chunks; c0 += CH * step) {
        int at[CH];
        float acc[CH][N];
#pragma unroll
        for (int q = 0; q < CH; ++q) {
            at[q] = chunk_start<N>(c0 + q * step, m);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[q][e] = 0.0f;
        }
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
                const uint32_t left = kSumRows - ((s >> lg) & (kSumRows - 1u));
                count = count < left ? count : left;
            }
            // kRows rows in flight, then the rest one by one
            const auto add_rows = [&](uint32_t first, auto rows) {
                constexpr uint32_t R = decltype(rows)::value;
                typename C::Raw r[R][CH];
                bool ok[R];
#pragma unroll
                for (uint32_t j = 0; j < R; ++j) {
                    const uint32_t i = static_cast<uint32_t>(order[first + j]);
                    ok[j] = i < n;
                    const T *src = dout + static_cast<int64_t>(ok[j] ? i : 0) * m.width;
#pragma unroll
                    for (int q = 0; q < CH; ++q) r[j][q] = C::load_stream(src + at[q]);
                }
#pragma unroll
                for (uint32_t j = 0; j < R; ++j) {
                    if (!ok[j]) continue;
#pragma unroll
                    for (int q = 0; q < CH; ++q) {
                        float x[N];
                        C::unpack(r[j][q], x);
#pragma unroll
                        for (int e = 0; e < N; ++e) acc[q][e] += x[e];
                    }
                }
            };
            const auto add_sums = [&](const float *p, auto rows) {
                constexpr uint32_t R = decltype(rows)::value;
                float x[R][CH][N];
#pragma unroll
                for (uint32_t j = 0; j < R; ++j) {
#pragma unroll
                    for (int q = 0; q < CH; ++q) load_values<float, N>(p + static_cast<int64_t>(j) * m.width + at[q], x[j][q]);
                }
#pragma unroll
                for (uint32_t j = 0; j < R; ++j) {
#pragma unroll
                    for (int q = 0; q < CH; ++q) {
#pragma unroll
                        for (int e = 0; e < N; ++e) acc[q][e] += x[j][q][e];
                    }
                }
            };
            constexpr uint32_t kRows = CH == 1 ? 4 : 2;
            using Many = std::integral_constant<uint32_t, kRows>;
            using One = std::integral_constant<uint32_t, 1>;
            uint32_t j = 0;
            if (l == 0) {
                for (; j + kRows <= count; j += kRows) add_rows(s + j, Many{});
                for (; j < count; ++j) add_rows(s + j, One{});
            } else {
                const float *p = sums.level[l - 1] + static_cast<int64_t>(s >> lg) * m.width;
                for (; j + kRows <= count; j += kRows) add_sums(p + static_cast<int64_t>(j) * m.width, Many{});
                for (; j < count; ++j) add_sums(p + static_cast<int64_t>(j) * m.width, One{});
            }
            s += count << lg;
        }
#pragma unroll
        for (int q = 0; q < CH; ++q) {
            const int c = c0 + q * step;
            if (c >= m.chunks) continue;
            const int skip = c * N - at[q];
#pragma unroll
            for (int e = 0; e < N; ++e) acc[q][e] *= scale;
            if (!accumulate) {
                store_values<G, N>(dst + at[q], acc[q]);
            } else if (skip == 0) {
                float old[N];
                load_values<G, N>(dst + at[q], old);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[q][e] += old[e];
                store_values<G, N>(dst + at[q], acc[q]);
            } else {  // elements that another lane owns are not added to twice
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    G *p = dst + at[q] + e;
                    if (e >= skip) *p = static_cast<G>(static_cast<float>(*p) + acc[q][e]);
                }
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
    if (p.bits < 2) p.bits = 2;  // the table is read four digits at a time
    if (n <= kGroupSmall) {
        // the sorted keys, for a launch that finds the offsets of many groups
        p.bytes = p.passes > 1 && groups > kGroupFew ? static_cast<size_t>(n) * 4 : 0;
        return p;
    }
    int64_t tiles = (n + kGroupBlock - 1) / kGroupBlock;
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

int launch_offsets(const uint32_t *sorted, uint32_t n, uint32_t groups, int32_t *offsets, hipStream_t s) {
    hipLaunchKernelGGL(group_offsets_kernel, dim3(groups / kGroupBlock + 1), dim3(kGroupBlock), 0, s, sorted, n,
                       groups, offsets);
    return launched();
}

template <class K>
int launch_small(const K *keys, uint32_t n, uint32_t groups, const GroupPlan &p, int32_t *order, int32_t *ranks,
                 int32_t *offsets, uint32_t *sorted, hipStream_t s) {
    const auto launch = [&](auto items) {
        hipLaunchKernelGGL((group_small_kernel<K, decltype(items)::value>), dim3(1), dim3(kGroupBlock), 0, s, keys, n,
                           groups, p.passes, p.bits, order, ranks, offsets, sorted);
        return launched();
    };
    // as few keys to a wavefront as all sixteen leave it, known to the compiler
    switch ((n + kGroupBlock - 1) / kGroupBlock) {
    case 1: SSC_TRY(launch(std::integral_constant<int, 1>{})); break;
    case 2: SSC_TRY(launch(std::integral_constant<int, 2>{})); break;
    case 3: SSC_TRY(launch(std::integral_constant<int, 3>{})); break;
    case 4: SSC_TRY(launch(std::integral_constant<int, 4>{})); break;
    case 5: SSC_TRY(launch(std::integral_constant<int, 5>{})); break;
    case 6: SSC_TRY(launch(std::integral_constant<int, 6>{})); break;
    case 7: SSC_TRY(launch(std::integral_constant<int, 7>{})); break;
    default: SSC_TRY(launch(std::integral_constant<int, 8>{})); break;
    }
    return sorted != nullptr ? launch_offsets(sorted, n, groups, offsets, s) : SSC_OK;
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
    if (p.bytes > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < p.bytes))
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
    if (n <= kGroupSmall)
        return launch_small(keys, un, ug, p, order, ranks, offsets,
                            p.bytes > 0 ? static_cast<uint32_t *>(scratch) : nullptr, s);
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
        const auto scatter = [&](auto items) {
            hipLaunchKernelGGL((group_scatter_kernel<K, decltype(items)::value>), grid, block, 0, s, keys, sorted,
                               positions, un, p.span, ug, q * p.bits, p.bits, static_cast<const uint32_t *>(table),
                               p.passes == 1 ? nullptr : buf[q & 1][0], last ? nullptr : buf[q & 1][1],
                               last ? order : nullptr, last ? ranks : nullptr, p.passes == 1 ? offsets : nullptr);
            return launched();
        };
        SSC_TRY(p.span >= 4 * kGroupBlock ? scatter(std::integral_constant<int, 4>{})
                                          : scatter(std::integral_constant<int, 1>{}));
        sorted = buf[q & 1][0];
        positions = buf[q & 1][1];
    }
    return p.passes > 1 ? launch_offsets(sorted, un, ug, offsets, s) : SSC_OK;
}

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

// Up to a workgroup to a row (a wavefront to a row, with four or eight chunks
// to a thread, was slower: embed 63.6 us against 61.3, combine's gradient 271
// against 222, dispatch 101 against 97.7). Up to 256 chunks a row gets a
// thread a chunk, or half the threads with two chunks each, all of a row's
// loads in flight: where the chunks fill at most `halve` eighths of the
// threads. Rows of bf16, one chunk against two, us a call; 40,000 ids drawn
// evenly, or falling as 1/rank as in text:
//   chunks                               65           138          192          256
//   threads                           128   64     256   128    256   128    256   128
//   embed, table of 60,000, even     17.0  14.8   28.9  28.7   36.3  37.9   51.5  48.6
//     as in text                     16.3  11.2   25.6  21.2   28.5  27.1   38.2  35.9
//   combine's gradient, 20,000 x 2   31.5  24.6   60.3  46.3   64.8  54.5   74.3  70.7
//   combine, 10,000 x 2               8.2   6.3   13.3  11.7   15.4  15.8   20.4  20.6
//     40,000 x 6                     53.1  52.5    110   109    150   148    200   198
//   dispatch                         26.0  27.8   50.9  55.8
//   embed's gradient, text, 16,384   27.6  32.2   35.4  39.2   43.7  48.8   53.4  59.1
//     32,768                         29.6  33.5   44.5  46.2   52.3  53.2   63.6  65.8
//     60,000                         36.9  38.3   59.2  58.5   70.0  68.0   82.8  81.0
//     90,000                         45.8  42.1   73.6  73.0   86.8  84.0    102   102
//     even, 60,000                   36.4  31.9   57.6  56.1   61.4  61.0   75.4  74.4
// so embed and combine's gradient always; combine up to 5/8 (160 chunks 14.2
// against 12.8, from 182 on within 3% either way); dispatch never; embed's
// gradient from tables of 65,536 rows on, below which the long run of a frequent
// id, two chunks to a thread, counts for more than what evenly drawn ids gain.
// Where the rows are too few to fill the chip (fewer than two workgroups a
// compute unit), columns go over several workgroups (split).
struct RowLaunch {
    RowMap map;
    dim3 grid;
    bool wave;   // whole wavefronts to a row
    int deep;    // chunks to a thread, as 1, 2 or 4
};

RowLaunch row_launch(int64_t rows, int64_t width, int per_chunk, bool split, int halve) {
    RowLaunch r{};
    r.map.width = static_cast<int>(width);
    r.map.chunks = static_cast<int>((width + per_chunk - 1) / per_chunk);
    const int64_t enough = 512;
    int lg = 0;
    while (lg < 8 && (1 << lg) < r.map.chunks) ++lg;
    if (lg > 6 && r.map.chunks <= halve << (lg - 3)) --lg;
    r.map.lg = lg;
    const int64_t blocks = (rows + (256 >> lg) - 1) >> (8 - lg);
    int64_t cols = 1;
    const int64_t parts = (r.map.chunks + (1 << lg) - 1) >> lg;
    while (split && cols < parts && cols < 64 && blocks * cols < enough) ++cols;
    constexpr int64_t kMostBlocks = int64_t{1} << 22;
    const int64_t x = blocks < kMostBlocks ? blocks : kMostBlocks;
    r.grid = dim3(static_cast<unsigned>(x), static_cast<unsigned>(cols), static_cast<unsigned>((blocks + x - 1) / x));
    r.wave = lg >= 6;
    const int64_t each = (parts + cols - 1) / cols;
    r.deep = !r.wave || each == 1 ? 1 : (each == 2 ? 2 : 4);
    return r;
}

// Calls f with the launch's WAVE and its chunks in flight.
template <class F>
int with_shape(const RowLaunch &r, F f) {
    if (r.deep == 4) return f(std::true_type{}, std::integral_constant<int, 4>{});
    if (r.deep == 2) return f(std::true_type{}, std::integral_constant<int, 2>{});
    if (r.wave) return f(std::true_type{}, std::integral_constant<int, 1>{});
    return f(std::false_type{}, std::integral_constant<int, 1>{});
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
        const RowLaunch r = row_launch(n, width, Chunk<T, V>::kN, true, 8);
        return with_shape(r, [&](auto wave, auto ch) {
            hipLaunchKernelGGL((embed_kernel<T, V, decltype(wave)::value, decltype(ch)::value, I>), r.grid,
                               dim3(kRowBlock), 0, static_cast<hipStream_t>(stream), static_cast<const T *>(table),
                               vocab, ids, n, scale, static_cast<T *>(out), r.map);
            return launched();
        });
    });
}

// A level is made where the batch holds at least 16 of its blocks, the third
// where it holds 64: a launch more for every batch, against at most 1023
// blocks of 256 that a row with nearly all of the tokens has to add. Rows of
// 1024 bf16, a table of 32,000, us without the third level and with it:
//   tokens                    70,000   131,072   262,143
//   ids drawn evenly          40  41   62   64   117  119
//   a tenth of them one id    47  49   77   73   129  123
//   all one id               122  56  212   83   430  162
int sum_levels(int64_t n) {
    int l = 0;
    while (l < kSumLevels && n >> (kSumLg * (l + 2) + (l == 2 ? 2 : 0)) > 0) ++l;
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
    if (need > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < need)) return SSC_ERR_SCRATCH;
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
            const RowLaunch r = row_launch(n >> (kSumLg * (l + 1)), width, Chunk<T, V>::kN, true, 0);
            if (r.wave)
                hipLaunchKernelGGL((grad_blocks_kernel<T, V, true, I>), r.grid, dim3(kRowBlock), 0, s,
                                   static_cast<const T *>(dout), ids, order, offsets, un, vocab, l, sums, r.map);
            else
                hipLaunchKernelGGL((grad_blocks_kernel<T, V, false, I>), r.grid, dim3(kRowBlock), 0, s,
                                   static_cast<const T *>(dout), ids, order, offsets, un, vocab, l, sums, r.map);
            SSC_TRY(launched());
        }
        const RowLaunch r = row_launch(vocab, width, Chunk<T, V>::kN, true, vocab >= 65536 ? 8 : 0);
        const auto launch = [&](auto *g) {
            using G = std::remove_pointer_t<decltype(g)>;
            return with_shape(r, [&](auto wave, auto ch) {
                hipLaunchKernelGGL((embed_grad_kernel<T, V, decltype(wave)::value, decltype(ch)::value, G>), r.grid,
                                   dim3(kRowBlock), 0, s, static_cast<const T *>(dout), order, offsets, un, vocab,
                                   scale, accumulate, sums, g, r.map);
                return launched();
            });
        };
        return grad_dtype == dtype ? launch(static_cast<T *>(grad)) : launch(static_cast<float *>(grad));
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
        const RowLaunch r = row_launch(tokens, width, Chunk<T, V>::kN, true, 0);
        return with_shape(r, [&](auto wave, auto ch) {
            hipLaunchKernelGGL((dispatch_kernel<T, V, decltype(wave)::value, decltype(ch)::value>), r.grid,
                               dim3(kRowBlock), 0, static_cast<hipStream_t>(stream), static_cast<const T *>(x),
                               tokens, static_cast<int>(per), ranks, rows, static_cast<T *>(out), r.map);
            return launched();
        });
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
        const RowLaunch r = row_launch(tokens, width, Chunk<T, V>::kN, true, 5);
        const auto launch = [&](auto weighted) {
            return with_shape(r, [&](auto wave, auto ch) {
                constexpr int kCh = decltype(ch)::value > 1 ? 2 : 1;
                hipLaunchKernelGGL((combine_kernel<T, V, decltype(wave)::value, kCh, decltype(weighted)::value>), r.grid,
                                   dim3(kRowBlock), 0, static_cast<hipStream_t>(stream), static_cast<const T *>(y),
                                   rows, ranks, weights, tokens, static_cast<int>(per), static_cast<T *>(out), r.map);
                return launched();
            });
        };
        return weights != nullptr ? launch(std::true_type{}) : launch(std::false_type{});
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
        const RowLaunch r = row_launch(tokens, width, Chunk<T, V>::kN, false, 8);
        return with_shape(r, [&](auto wave, auto ch) {
            constexpr int kCh = decltype(ch)::value > 1 ? 2 : 1;
            hipLaunchKernelGGL((combine_grad_kernel<T, V, decltype(wave)::value, kCh>), r.grid, dim3(kRowBlock), 0,
                               static_cast<hipStream_t>(stream), static_cast<const T *>(dout),
                               static_cast<const T *>(y), rows, ranks, weights, tokens, static_cast<int>(per),
                               static_cast<T *>(dy), dweights, r.map);
            return launched();
        });
    });
}

}  // extern "C"
