// A cache of keys and values cut to the rows that were attended to most: HIP
// kernels for MI355X (gfx950) and their part of the C ABI in include/ssc.h.
//
//   accumulate_weights  scores[b, h, i] = decay * scores + sum of the attention weights that position i got
//   evict_rows          kept[b, h, :] = the positions that stay, increasing: a selection, then a compaction
//   move_rows           out[b, h, s] = cache[b, h, kept[b, h, s]], in place or to another cache
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssc.h"
#include "ssc_device.h"
#include "ssc_host.h"

namespace ssc {
namespace {

// ---------------------------------------------------- weights added up ---
// A lane holds 16 bytes of columns of the weights and adds up its rows (the
// queries of the heads that share a cache head), eight in flight; the
// wavefronts of a workgroup take every WAVES-th row and are joined in LDS.
struct AccumulateArgs {
    float *scores;
    int64_t score_batch, score_head;
    const void *weights;
    int64_t weight_batch, weight_head, weight_query;
    const int32_t *lengths;
    int heads, capacity, group, queries, length;
    int64_t fresh;
    float decay;
};

template <class T, int WAVES>
__global__ __launch_bounds__(WAVES *kWave) void accumulate_kernel(AccumulateArgs a) {
    constexpr int kN = 16 / static_cast<int>(sizeof(T));
    constexpr int kFlight = 8;
    typedef T V __attribute__((ext_vector_type(kN)));
    typedef uint32_t Raw __attribute__((ext_vector_type(4)));
    typedef uint32_t RawAny __attribute__((ext_vector_type(4), aligned(2), may_alias));
    __shared__ float s_sum[WAVES > 1 ? WAVES - 1 : 1][WAVES > 1 ? kWave * kN : 1];
    const int64_t bh = blockIdx.y;
    const int64_t b = bh / a.heads, h = bh % a.heads;
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int lane = lane_id();
    int64_t len = a.length;
    if (a.lengths != nullptr) len = a.lengths[b];
    if (len > a.length) len = a.length;
    const int64_t block_first = static_cast<int64_t>(blockIdx.x) * kWave * kN;
    if (block_first >= len) return;
    const int64_t first = block_first + lane * kN;
    const T *from = static_cast<const T *>(a.weights) + b * a.weight_batch + h * a.group * a.weight_head + first;
    const bool whole = first + kN <= a.length;
    float sum[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) sum[e] = 0.0f;
    const uint32_t rows = static_cast<uint32_t>(a.group) * static_cast<uint32_t>(a.queries);
    const uint32_t queries = static_cast<uint32_t>(a.queries);
    // a weight that is no number (of a query whose mask left nothing) adds nothing
    const auto add = [&](const V &v) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float x = static_cast<float>(v[e]);
            sum[e] += x == x ? x : 0.0f;
        }
    };
    const auto row = [&](uint32_t r) { return from + (r / queries) * a.weight_head + (r % queries) * a.weight_query; };
    if (whole) {
        uint32_t r = w;
        for (; r + (kFlight - 1) * WAVES < rows; r += kFlight * WAVES) {
            Raw raw[kFlight];
#pragma unroll
            for (int j = 0; j < kFlight; ++j)
                raw[j] = __builtin_nontemporal_load(reinterpret_cast<const RawAny *>(row(r + j * WAVES)));
#pragma unroll
            for (int j = 0; j < kFlight; ++j) add(__builtin_bit_cast(V, raw[j]));
        }
        for (; r < rows; r += WAVES) {
            const Raw raw = __builtin_nontemporal_load(reinterpret_cast<const RawAny *>(row(r)));
            add(__builtin_bit_cast(V, raw));
        }
    } else if (first < a.length) {
        for (uint32_t r = w; r < rows; r += WAVES) {
            const T *p = row(r);
            V v;
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = first + e < a.length ? p[e] : static_cast<T>(0.0f);
            add(v);
        }
    }
    if constexpr (WAVES > 1) {
        if (w > 0) {
#pragma unroll
            for (int e = 0; e < kN; ++e) s_sum[w - 1][e * kWave + lane] = sum[e];
        }
        __syncthreads();
        if (w > 0) return;
        for (int v = 0; v < WAVES - 1; ++v) {
#pragma unroll
            for (int e = 0; e < kN; ++e) sum[e] += s_sum[v][e * kWave + lane];
        }
    }
    float *to = a.scores + b * a.score_batch + h * a.score_head + first;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        const int64_t i = first + e;
        if (i >= len) continue;
        const float old = i < len - a.fresh ? to[e] * a.decay : 0.0f;
        to[e] = old + sum[e];
    }
}

// ------------------------------------------------------- which rows stay ---
// A workgroup a row. The threshold is the `need`-th largest score, found by
// its leading 11, 11 and 10 bits: counts by digit in LDS, a scan from the
// largest digit down, then the digit's own members by the next one. What lies
// above it stays, and of the scores equal to it the first ones. Wavefronts hold
// consecutive positions, 64 at a time, so that a ballot ranks them.
constexpr int kEvictBlock = 1024;
constexpr int kEvictWaves = kEvictBlock / kWave;
constexpr int kEvictBins = 2048;

struct EvictArgs {
    const float *scores;
    int64_t score_batch, score_head;
    const int32_t *lengths;
    int heads;
    uint32_t capacity, keep, first, recent;
    int32_t *kept, *counts;
};

// The score as an integer of the same order; NaN as the lowest, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return x == x ? k : 0u;
}

struct EvictShared {
    uint32_t hist[kEvictBins];
    uint32_t wave[kEvictWaves];
    uint32_t wave_equal[kEvictWaves];
    uint32_t digit, above, inside;
};

// ITEMS: scores of a lane, held in registers; 0: read again each time.
template <int ITEMS>
__global__ __launch_bounds__(kEvictBlock) void evict_kernel(EvictArgs a) {
    __shared__ EvictShared sh;
    const int64_t bh = blockIdx.x;
    const int64_t b = bh / a.heads, h = bh % a.heads;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    int32_t *kept = a.kept + bh * a.keep;
    uint32_t len = a.capacity;
    if (a.lengths != nullptr) {
        const int32_t l = a.lengths[b];
        len = l < 0 ? 0u : (static_cast<uint32_t>(l) < a.capacity ? static_cast<uint32_t>(l) : a.capacity);
    }
    if (len <= a.keep) {  // all stay
        for (uint32_t s = threadIdx.x; s < a.keep; s += kEvictBlock) kept[s] = s < len ? static_cast<int32_t>(s) : -1;
        if (threadIdx.x == 0) a.counts[bh] = static_cast<int32_t>(len);
        return;
    }
    const float *scores = a.scores + b * a.score_batch + h * a.score_head;
    const uint32_t begin = a.first, end = len - a.recent;  // those between stay by their score
    uint32_t need = a.keep - a.first - a.recent;
    const uint32_t sets = ITEMS > 0 ? ITEMS : (len + kEvictBlock - 1) / kEvictBlock;
    const uint32_t base = static_cast<uint32_t>(w) * sets * kWave;
    uint32_t held[ITEMS > 0 ? ITEMS : 1];
    if constexpr (ITEMS > 0) {
        float x[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t i = base + j * kWave + lane;
            x[j] = i >= begin && i < end ? scores[i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) held[j] = score_key(x[j]);
    }
    // f(position, key, whether the score decides) for this lane's positions
    const auto each = [&](auto f) {
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                const uint32_t i = base + j * kWave + lane;
                f(i, held[j], i >= begin && i < end);
            }
        } else {
            for (uint32_t j = 0; j < sets; ++j) {
                const uint32_t i = base + j * kWave + lane;
                const bool open = i >= begin && i < end;
                f(i, open ? score_key(scores[i]) : 0u, open);
            }
        }
    };
    // scores from `low` on stay if all of a digit does; else those above, and
    // `need` of those equal to it
    uint32_t low = 0, fixed = 0;  // the digits found, and their bits
    bool all = need == 0;
    if (need == 0) low = 0xffffffffu;  // no score's
    for (int pass = 0; pass < 3 && !all; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const uint32_t bins = pass == 2 ? 1024u : 2048u;
        for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) sh.hist[i] = 0;
        __syncthreads();
        each([&](uint32_t, uint32_t k, bool open) {
            if (open && (k & fixed) == low)
                __hip_atomic_fetch_add(&sh.hist[(k >> shift) & (bins - 1u)], 1u, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
        });
        __syncthreads();
        // two bins a thread, the largest first
        const uint32_t top = kEvictBins - 1u - 2u * threadIdx.x;
        const uint32_t c0 = sh.hist[top], c1 = sh.hist[top - 1u];
        const uint32_t incl = wave_inclusive_scan<SumU32>(c0 + c1);
        if (lane == kWave - 1) sh.wave[w] = incl;
        __syncthreads();
        uint32_t above = incl - c0 - c1;
        for (int v = 0; v < w; ++v) above += sh.wave[v];
        if (above < need && need <= above + c0) {
            sh.digit = top;
            sh.above = above;
            sh.inside = c0;
        } else if (above + c0 < need && need <= above + c0 + c1) {
            sh.digit = top - 1u;
            sh.above = above + c0;
            sh.inside = c1;
        }
        __syncthreads();
        low |= sh.digit << shift;
        fixed |= (bins - 1u) << shift;
        need -= sh.above;
        all = need == sh.inside;
    }
    const auto better = [&](uint32_t k) { return all ? k >= low : k > low; };
    // the wavefront's share: those that stay in any case, and those equal
    uint32_t sure = 0, equal = 0;
    each([&](uint32_t i, uint32_t k, bool open) {
        const bool yes = i < begin || (i >= end && i < len) || (open && better(k));
        const bool same = open && !all && k == low;
        sure += static_cast<uint32_t>(__builtin_popcountll(ballot(yes)));
        equal += static_cast<uint32_t>(__builtin_popcountll(ballot(same)));
    });
    if (lane == 0) {
        sh.wave[w] = sure;
        sh.wave_equal[w] = equal;
    }
    __syncthreads();
    uint32_t at = 0, equals = 0;
    for (int v = 0; v < w; ++v) {
        at += sh.wave[v];
        equals += sh.wave_equal[v];
    }
    at += equals < need ? equals : need;
    each([&](uint32_t i, uint32_t k, bool open) {
        bool yes = i < begin || (i >= end && i < len) || (open && better(k));
        const bool same = open && !all && k == low;
        const uint64_t sames = ballot(same);
        yes = yes || (same && equals + mbcnt64(sames) < need);
        equals += static_cast<uint32_t>(__builtin_popcountll(sames));
        const uint64_t yeses = ballot(yes);
        const uint32_t slot = at + mbcnt64(yeses);
        if (yes && slot < a.keep) kept[slot] = static_cast<int32_t>(i);
        at += static_cast<uint32_t>(__builtin_popcountll(yeses));
    });
    if (threadIdx.x == 0) a.counts[bh] = static_cast<int32_t>(a.keep);
}

// ------------------------------------------------------------ rows moved ---
// Rows are bytes here. A lane moves 16 of them, or an element where the row is
// shorter; the last 16 of a row that is no multiple start early and share some
// with the ones before.
//
// In place a workgroup takes the rows of a head in order, a set at a time: kept
// positions increase, so a set's rows lie at or past its own slots, and a set is
// stored once all of it has been read. What later sets read is not written by
// then. Workgroups that share a head's columns do not share bytes.
struct MoveArgs {
    const char *from;
    char *to;
    int64_t from_batch, from_head, from_row;  // strides in bytes
    int64_t to_batch, to_head, to_row;
    const int32_t *kept;
    int heads, capacity, keep;
    int row_bytes, chunks;
    int lg;      // log2 of the lanes of a row
    int cols;    // chunks of a row that a workgroup moves
};

template <int BYTES>
struct Piece {
    using V = std::conditional_t<BYTES == 1, uint8_t,
                                 std::conditional_t<BYTES == 2, uint16_t,
                                                    std::conditional_t<BYTES == 4, uint32_t, uint64_t>>>;
    typedef V Any __attribute__((aligned(1), may_alias));
    __device__ static __forceinline__ V load(const char *p) { return *reinterpret_cast<const Any *>(p); }
    __device__ static __forceinline__ V load_stream(const char *p) { return load(p); }
    __device__ static __forceinline__ void store(char *p, V v) { *reinterpret_cast<Any *>(p) = v; }
    __device__ static __forceinline__ void store_stream(char *p, V v) { store(p, v); }
};
template <>
struct Piece<16> {
    typedef uint32_t V __attribute__((ext_vector_type(4)));
    typedef uint32_t Any __attribute__((ext_vector_type(4), aligned(1), may_alias));
    __device__ static __forceinline__ V load(const char *p) { return *reinterpret_cast<const Any *>(p); }
    __device__ static __forceinline__ V load_stream(const char *p) {
        return __builtin_nontemporal_load(reinterpret_cast<const Any *>(p));
    }
    __device__ static __forceinline__ void store(char *p, V v) { *reinterpret_cast<Any *>(p) = v; }
    __device__ static __forceinline__ void store_stream(char *p, V v) {
        __builtin_nontemporal_store(v, reinterpret_cast<Any *>(p));
    }
};

constexpr int kMoveBlock = 256;
constexpr int kMoveFlight = 4;

template <int BYTES>
__device__ __forceinline__ int piece_at(const MoveArgs &a, int c) {
    const int at = c * BYTES;
    return at + BYTES <= a.row_bytes ? at : a.row_bytes - BYTES;
}

template <int BYTES>
__global__ __launch_bounds__(kMoveBlock) void move_kernel(MoveArgs a) {
    using P = Piece<BYTES>;
    const int64_t bh = blockIdx.y;
    const int64_t b = bh / a.heads, h = bh % a.heads;
    const char *from = a.from + b * a.from_batch + h * a.from_head;
    char *to = a.to + b * a.to_batch + h * a.to_head;
    const int32_t *kept = a.kept + bh * a.keep;
    const int rows = kMoveBlock >> a.lg;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows * kMoveFlight + (threadIdx.x >> a.lg);
    int64_t pos[kMoveFlight];
#pragma unroll
    for (int j = 0; j < kMoveFlight; ++j) {
        const int64_t s = first + j * rows;
        pos[j] = s < a.keep ? kept[s] : -1;
        if (pos[j] >= a.capacity) pos[j] = -1;
    }
    for (int c = static_cast<int>(threadIdx.x) & ((1 << a.lg) - 1); c < a.chunks; c += 1 << a.lg) {
        const int at = piece_at<BYTES>(a, c);
        typename P::V v[kMoveFlight];
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j)
            if (pos[j] >= 0) v[j] = P::load_stream(from + pos[j] * a.from_row + at);
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j)
            if (pos[j] >= 0) P::store_stream(to + (first + j * rows) * a.to_row + at, v[j]);
    }
}

constexpr int kPlaceBlock = 1024;

template <int BYTES>
__global__ __launch_bounds__(kPlaceBlock) void move_in_place_kernel(MoveArgs a) {
    using P = Piece<BYTES>;
    const int64_t bh = blockIdx.y;
    const int64_t b = bh / a.heads, h = bh % a.heads;
    char *rows_at = a.to + b * a.to_batch + h * a.to_head;
    const int32_t *kept = a.kept + bh * a.keep;
    const int rows = kPlaceBlock >> a.lg;
    const int lane_col = static_cast<int>(threadIdx.x) & ((1 << a.lg) - 1);
    const int c0 = static_cast<int>(blockIdx.x) * a.cols, c1 = c0 + a.cols < a.chunks ? c0 + a.cols : a.chunks;
    for (int64_t set = 0; set < a.keep; set += rows * kMoveFlight) {
        int64_t pos[kMoveFlight];
        const int64_t first = set + (threadIdx.x >> a.lg);
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j) {
            const int64_t s = first + j * rows;
            pos[j] = s < a.keep ? kept[s] : -1;
            // a row that stays where it is needs no move; one that lies before its slot is none of evict_rows
            if (pos[j] >= a.capacity || pos[j] <= s) pos[j] = -1;
        }
        for (int base = c0; base < c1; base += 1 << a.lg) {
            const int c = base + lane_col;
            const int at = piece_at<BYTES>(a, c < c1 ? c : c0);
            typename P::V v[kMoveFlight];
#pragma unroll
            for (int j = 0; j < kMoveFlight; ++j)
                if (pos[j] >= 0 && c < c1) v[j] = P::load(rows_at + pos[j] * a.to_row + at);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kMoveFlight; ++j)
                if (pos[j] >= 0 && c < c1) P::store(rows_at + (first + j * rows) * a.to_row + at, v[j]);
        }
    }
}

// ============================================================ host side ---
int check_cache(int64_t batch, int64_t heads, int64_t capacity) {
    if (batch < 0 || heads < 1 || capacity < 1) return SSC_ERR_ARG;
    if (batch > INT32_MAX || heads > INT32_MAX || capacity > INT32_MAX - 4096 || batch * heads > 65535)
        return SSC_ERR_SIZE;
    return SSC_OK;
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

int ssc_accumulate_weights(float *scores, int64_t batch, int64_t heads, int64_t capacity, int64_t score_batch,
                           int64_t score_head, const void *weights, int dtype, int64_t group, int64_t queries,
                           int64_t length, int64_t weight_batch, int64_t weight_head, int64_t weight_query,
                           const int32_t *lengths, int64_t fresh, float decay, void *stream) {
    SSC_TRY(check_cache(batch, heads, capacity));
    if (!dtype_ok(dtype) || group < 1 || queries < 0 || length < 0 || length > capacity || fresh < 0) return SSC_ERR_ARG;
    if (group > INT32_MAX || queries > INT32_MAX || group * queries > (int64_t{1} << 30) || heads * group > INT32_MAX)
        return SSC_ERR_SIZE;
    const View<3> s{{batch, heads, capacity}, {score_batch, score_head, 1}};
    const View<4> w{{batch, heads * group, queries, length}, {weight_batch, weight_head, weight_query, 1}};
    if (!s.strides_ok() || !w.strides_ok() || !s.distinct()) return SSC_ERR_ARG;
    if (batch > 0 && (scores == nullptr || (w.extent() > 0 && weights == nullptr))) return SSC_ERR_ARG;
    if (!aligned(scores, 4) || !aligned(weights, elem_bytes(dtype)) || !aligned(lengths, 4)) return SSC_ERR_ARG;
    const size_t out = static_cast<size_t>(s.extent()) * 4;
    if (overlap(scores, out, weights, static_cast<size_t>(w.extent()) * elem_bytes(dtype)) ||
        overlap(scores, out, lengths, static_cast<size_t>(batch) * 4))
        return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (batch == 0 || length == 0) return SSC_OK;
    AccumulateArgs a{};
    a.scores = scores;
    a.score_batch = score_batch;
    a.score_head = score_head;
    a.weights = weights;
    a.weight_batch = weight_batch;
    a.weight_head = weight_head;
    a.weight_query = weight_query;
    a.lengths = lengths;
    a.heads = static_cast<int>(heads);
    a.capacity = static_cast<int>(capacity);
    a.group = static_cast<int>(group);
    a.queries = static_cast<int>(queries > 0 ? queries : 1);
    if (queries == 0) a.group = 0;  // no rows
    a.length = static_cast<int>(length);
    a.fresh = fresh;
    a.decay = decay;
    dim3 grid(1, static_cast<unsigned>(batch * heads));
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t cols = kWave * 16 / static_cast<int64_t>(sizeof(T));
        grid.x = static_cast<unsigned>((length + cols - 1) / cols);
        const auto launch = [&](auto waves) {
            constexpr int W = decltype(waves)::value;
            hipLaunchKernelGGL((accumulate_kernel<T, W>), grid, dim3(W * kWave), 0, static_cast<hipStream_t>(stream),
                               a);
            return launched();
        };
        const int64_t rows = group * queries;
        if (rows <= 16) return launch(std::integral_constant<int, 1>{});
        if (rows <= 64) return launch(std::integral_constant<int, 4>{});
        return launch(std::integral_constant<int, 8>{});
    });
}

int ssc_evict_rows(const float *scores, int64_t batch, int64_t heads, int64_t capacity, int64_t score_batch,
                   int64_t score_head, const int32_t *lengths, int64_t keep, int64_t first, int64_t recent,
                   int32_t *kept, int32_t *counts, void *stream) {
    SSC_TRY(check_cache(batch, heads, capacity));
    if (keep < 1 || keep > capacity || first < 0 || recent < 0 || first > keep || recent > keep - first)
        return SSC_ERR_ARG;
    const View<3> s{{batch, heads, capacity}, {score_batch, score_head, 1}};
    if (!s.strides_ok()) return SSC_ERR_ARG;
    if (batch > 0 && (scores == nullptr || kept == nullptr || counts == nullptr)) return SSC_ERR_ARG;
    if (!aligned(scores, 4) || !aligned(lengths, 4) || !aligned(kept, 4) || !aligned(counts, 4)) return SSC_ERR_ARG;
    const size_t rows = static_cast<size_t>(batch) * heads;
    const Span written[] = {{kept, rows * keep * 4}, {counts, rows * 4}};
    const Span read[] = {{scores, static_cast<size_t>(s.extent()) * 4}, {lengths, static_cast<size_t>(batch) * 4}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &x : written)
        for (const Span &y : read)
            if (overlap(x.p, x.bytes, y.p, y.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (batch == 0) return SSC_OK;
    EvictArgs a{};
    a.scores = scores;
    a.score_batch = score_batch;
    a.score_head = score_head;
    a.lengths = lengths;
    a.heads = static_cast<int>(heads);
    a.capacity = static_cast<uint32_t>(capacity);
    a.keep = static_cast<uint32_t>(keep);
    a.first = static_cast<uint32_t>(first);
    a.recent = static_cast<uint32_t>(recent);
    a.kept = kept;
    a.counts = counts;
    const auto launch = [&](auto items) {
        hipLaunchKernelGGL((evict_kernel<decltype(items)::value>), dim3(static_cast<unsigned>(rows)), dim3(kEvictBlock),
                           0, static_cast<hipStream_t>(stream), a);
        return launched();
    };
    if (capacity <= 4 * kEvictBlock) return launch(std::integral_constant<int, 4>{});
    if (capacity <= 8 * kEvictBlock) return launch(std::integral_constant<int, 8>{});
    if (capacity <= 32 * kEvictBlock) return launch(std::integral_constant<int, 32>{});
    return launch(std::integral_constant<int, 0>{});
}

int ssc_move_rows(const void *cache, int elem_bytes, int64_t batch, int64_t heads, int64_t capacity, int64_t width,
                  int64_t cache_batch, int64_t cache_head, int64_t cache_row, const int32_t *kept, int64_t keep,
                  void *out, int64_t out_batch, int64_t out_head, int64_t out_row, void *stream) {
    SSC_TRY(check_cache(batch, heads, capacity));
    if ((elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4 && elem_bytes != 8) || width < 1 || keep < 1 ||
        keep > capacity)
        return SSC_ERR_ARG;
    if (width > (1 << 24)) return SSC_ERR_SIZE;
    const View<4> c{{batch, heads, capacity, width}, {cache_batch, cache_head, cache_row, 1}};
    const View<4> o{{batch, heads, keep, width}, {out_batch, out_head, out_row, 1}};
    if (!c.strides_ok() || !o.strides_ok() || !o.distinct()) return SSC_ERR_ARG;
    if (batch > 0 && (cache == nullptr || kept == nullptr || out == nullptr)) return SSC_ERR_ARG;
    const size_t es = static_cast<size_t>(elem_bytes);
    if (!aligned(cache, es) || !aligned(out, es) || !aligned(kept, 4)) return SSC_ERR_ARG;
    const size_t cache_bytes = static_cast<size_t>(c.extent()) * es, out_bytes = static_cast<size_t>(o.extent()) * es;
    // in place: the same rows, told by their address and strides
    const bool place = cache == out && (batch <= 1 || cache_batch == out_batch) &&
                       (heads <= 1 || cache_head == out_head) && cache_row == out_row;
    if (place && !c.distinct()) return SSC_ERR_ARG;
    if ((!place && overlap(out, out_bytes, cache, cache_bytes)) ||
        overlap(out, place ? cache_bytes : out_bytes, kept, static_cast<size_t>(batch) * heads * keep * 4))
        return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (batch == 0) return SSC_OK;
    MoveArgs a{};
    a.from = static_cast<const char *>(cache);
    a.to = static_cast<char *>(out);
    a.from_batch = cache_batch * elem_bytes;
    a.from_head = cache_head * elem_bytes;
    a.from_row = cache_row * elem_bytes;
    a.to_batch = out_batch * elem_bytes;
    a.to_head = out_head * elem_bytes;
    a.to_row = out_row * elem_bytes;
    a.kept = kept;
    a.heads = static_cast<int>(heads);
    a.capacity = static_cast<int>(capacity);
    a.keep = static_cast<int>(keep);
    a.row_bytes = static_cast<int>(width * elem_bytes);
    // pieces that overlap must all be read before one is stored
    const bool shared = place && a.row_bytes % 16 != 0 && a.row_bytes > 16 << 8;
    const int bytes = a.row_bytes >= 16 && !shared ? 16 : elem_bytes;
    a.chunks = (a.row_bytes + bytes - 1) / bytes;
    a.cols = a.chunks;
    while (a.lg < 8 && (1 << a.lg) < a.chunks) ++a.lg;
    dim3 grid(1, static_cast<unsigned>(batch * heads));
    if (place) {
        // few heads: their columns over several workgroups, where no two of
        // these share bytes of a row
        int parts = 1;
        while (a.row_bytes % bytes == 0 && batch * heads * parts < 256 && a.chunks / (parts * 2) >= 4 &&
               a.chunks % (parts * 2) == 0)
            parts *= 2;
        a.cols = a.chunks / parts;
        a.lg = 0;
        while (a.lg < 8 && (1 << a.lg) < a.cols) ++a.lg;
        grid.x = static_cast<unsigned>(parts);
    } else {
        const int64_t rows = static_cast<int64_t>(kMoveBlock >> a.lg) * kMoveFlight;
        grid.x = static_cast<unsigned>((keep + rows - 1) / rows);
    }
    const auto launch = [&](auto piece) {
        constexpr int B = decltype(piece)::value;
        if (place)
            hipLaunchKernelGGL((move_in_place_kernel<B>), grid, dim3(kPlaceBlock), 0, static_cast<hipStream_t>(stream),
                               a);
        else
            hipLaunchKernelGGL((move_kernel<B>), grid, dim3(kMoveBlock), 0, static_cast<hipStream_t>(stream), a);
        return launched();
    };
    switch (bytes) {
    case 1: return launch(std::integral_constant<int, 1>{});
    case 2: return launch(std::integral_constant<int, 2>{});
    case 4: return launch(std::integral_constant<int, 4>{});
    case 8: return launch(std::integral_constant<int, 8>{});
    default: return launch(std::integral_constant<int, 16>{});
    }
}

}  // extern "C"
