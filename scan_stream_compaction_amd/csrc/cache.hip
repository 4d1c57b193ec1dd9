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
// queries of the heads that share a cache head), sixteen in flight; the
// wavefronts of a workgroup take every WAVES-th row and are joined in LDS.
struct AccumulateArgs {
    float *scores;
    int64_t score_batch, score_head;
    const void *weights;
    int64_t weight_batch, weight_group, weight_head, weight_query;  // group: of the heads of a cache head
    const int32_t *lengths;
    int length;
    uint32_t group, queries;
    int64_t fresh;
    float decay;
};

// EVEN: the rows of a cache head lie evenly apart (queries of one head)
template <class T, int WAVES, bool EVEN>
__global__ __launch_bounds__(WAVES *kWave) void accumulate_kernel(AccumulateArgs a) {
    constexpr int kN = 16 / static_cast<int>(sizeof(T));
    constexpr int kFlight = 16;
    typedef T V __attribute__((ext_vector_type(kN)));
    typedef uint32_t Raw __attribute__((ext_vector_type(4)));
    typedef uint32_t RawAny __attribute__((ext_vector_type(4), aligned(2), may_alias));
    typedef float Score __attribute__((ext_vector_type(4)));
    typedef float ScoreAny __attribute__((ext_vector_type(4), aligned(4), may_alias));
    __shared__ float s_sum[WAVES > 1 ? WAVES - 1 : 1][WAVES > 1 ? kWave * kN : 1];
    const int64_t h = blockIdx.y, b = blockIdx.z;
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int lane = lane_id();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kWave * kN + lane * kN;
    const T *from = static_cast<const T *>(a.weights) + b * a.weight_batch + h * a.weight_group + first;
    float *to = a.scores + b * a.score_batch + h * a.score_head + first;
    int64_t len = a.length;
    if (a.lengths != nullptr) {
        const int64_t l = a.lengths[b];
        len = l < len ? l : len;
    }
    if (first - lane * kN >= len) return;
    const bool whole = first + kN <= a.length;
    // the earlier scores are on their way while the weights are read
    const int64_t old = len - a.fresh;  // positions with an earlier score
    Score before[kN / 4];
    const bool vector = first + kN <= len && first + kN <= old && w == 0;
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
        before[i] = Score{0.0f, 0.0f, 0.0f, 0.0f};
        if (vector) before[i] = *reinterpret_cast<const ScoreAny *>(to + 4 * i);
    }
    float sum[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) sum[e] = 0.0f;
    const uint32_t rows = a.group * a.queries;
    // a weight that is no number (of a query whose mask left nothing) adds nothing
    const auto add = [&](const V &v) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float x = static_cast<float>(v[e]);
            sum[e] += x == x ? x : 0.0f;
        }
    };
    const auto row = [&](uint32_t r) {
        if constexpr (EVEN) return from + r * a.weight_query;
        return from + (r / a.queries) * a.weight_head + (r % a.queries) * a.weight_query;
    };
    if (whole) {
        uint32_t r = w;
        const auto some = [&](auto count) {
            constexpr int C = decltype(count)::value;
            Raw raw[C];
#pragma unroll
            for (int j = 0; j < C; ++j)
                raw[j] = __builtin_nontemporal_load(reinterpret_cast<const RawAny *>(row(r + j * WAVES)));
#pragma unroll
            for (int j = 0; j < C; ++j) add(__builtin_bit_cast(V, raw[j]));
            r += C * WAVES;
        };
        while (r + (kFlight - 1) * WAVES < rows) some(std::integral_constant<int, kFlight>{});
        if (r + 7 * WAVES < rows) some(std::integral_constant<int, 8>{});
        if (r + 3 * WAVES < rows) some(std::integral_constant<int, 4>{});
        while (r < rows) some(std::integral_constant<int, 1>{});
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
    if (vector) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) {
            Score s;
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = __builtin_fmaf(before[i][e], a.decay, sum[4 * i + e]);
            *reinterpret_cast<ScoreAny *>(to + 4 * i) = s;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const int64_t i = first + e;
            if (i < len) to[e] = i < old ? __builtin_fmaf(to[e], a.decay, sum[e]) : sum[e];
        }
    }
}

// ------------------------------------------------------- which rows stay ---
// The threshold is the `need`-th largest score, found by its leading 11, 11 and
// 10 bits: counts by digit in LDS, a scan from the largest digit down, then the
// digit's own members by the next one. What lies above it stays, and of the
// scores equal to it the first ones. Wavefronts hold consecutive positions, 64
// at a time, so that ballots rank them.
//
// Up to 32,768 positions a workgroup does all of a head, its scores in
// registers. Longer heads, and those of a few that leave the chip empty, go over
// several workgroups (splits) and four launches: a count by each digit, which
// first joins the splits' counts of the one before, and the output.
constexpr int kEvictBlock = 1024;
constexpr int kEvictWaves = kEvictBlock / kWave;
constexpr int kEvictBins = 2048;
constexpr int kEvictPasses = 3;
constexpr int kEvictHeld = 32 * kEvictBlock;  // positions of a head that one workgroup holds

// What is known of the threshold: its leading digits, and how many of the
// scores that share them stay. `all`: every one.
struct Threshold {
    uint32_t low, fixed, need, all;
};

struct EvictArgs {
    const float *scores;
    int64_t score_batch, score_head;
    const int32_t *lengths;
    int heads;
    uint32_t capacity, keep, first, recent;
    int32_t *kept, *counts;
    // of the splits
    uint32_t splits, span;  // and positions of one, a multiple of kEvictTile
    Threshold *found;       // [rows][passes]
    uint32_t *before;       // [rows][splits] scores of earlier splits that stay, as far as known
    uint32_t *hist;         // [2][rows][splits][bins] of this pass and the one before
};

__device__ __forceinline__ int digit_shift(int pass) { return pass == 0 ? 21 : (pass == 1 ? 10 : 0); }
__device__ __forceinline__ uint32_t digit_bins(int pass) { return pass == 2 ? 1024u : 2048u; }

// A head of the cache: its positions in use, and those that a score decides on.
struct Head {
    const float *scores;
    int32_t *kept;
    uint32_t len, begin, end;

    __device__ __forceinline__ Head(const EvictArgs &a, int64_t h, int64_t b) {
        scores = a.scores + b * a.score_batch + h * a.score_head;
        kept = a.kept + (b * a.heads + h) * a.keep;
        len = a.capacity;
        if (a.lengths != nullptr) {
            const int32_t l = a.lengths[b];
            len = l < 0 ? 0u : (static_cast<uint32_t>(l) < a.capacity ? static_cast<uint32_t>(l) : a.capacity);
        }
        begin = a.first;
        end = len - a.recent;  // used where len > keep
    }
    // up to `keep` positions: all stay; by `stride` threads
    __device__ __forceinline__ void keep_all(const EvictArgs &a, int32_t *count, uint32_t thread, uint32_t stride) const {
        for (uint32_t s = thread; s < a.keep; s += stride) kept[s] = s < len ? static_cast<int32_t>(s) : -1;
        if (thread == 0) *count = static_cast<int32_t>(len);
    }
    // The scores at base, base + 64, ... as integers of the same order. Positions
    // that stay in any case are above all, NaN is below all scores, -0 as 0, and
    // positions at or past `to` are below that.
    template <int ITEMS>
    __device__ __forceinline__ void load(uint32_t base, uint32_t to, uint32_t (&key)[ITEMS]) const {
        float x[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t i = base + j * kWave;
            x[j] = scores[i < len ? i : len - 1u];
        }
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t i = base + j * kWave;
            const uint32_t b = __float_as_uint(x[j] + 0.0f);
            uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
            k = x[j] == x[j] ? k : 1u;
            k = i - begin < end - begin ? k : ~0u;
            key[j] = i < to ? k : 0u;
        }
    }
};

struct EvictShared {
    uint32_t hist[kEvictBins];
    uint32_t wave[kEvictWaves];
    uint32_t wave_equal[kEvictWaves];
    uint32_t digit, above, inside, before;
};

// Counts a wavefront's digits, where they count. Many scores may be equal (0
// above all): the lanes that share the first one's digit are counted by one add.
__device__ __forceinline__ void count_digit(uint32_t *hist, uint32_t d, bool counts) {
    const uint64_t active = ballot(counts);
    if (active == 0) return;
    const int leader = __builtin_ctzll(active);
    const uint32_t common = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(d), leader));
    const bool same = d == common;
    const uint32_t many = static_cast<uint32_t>(__builtin_popcountll(ballot(same) & active));
    const bool leads = lane_id() == leader;
    if ((counts && !same) || leads)
        __hip_atomic_fetch_add(&hist[d], leads ? many : 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

template <int ITEMS>
__device__ __forceinline__ void count_digits(uint32_t *hist, const uint32_t (&key)[ITEMS], const Threshold &t, int pass) {
    if (pass == 0) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) count_digit(hist, key[j] >> 21, true);
    } else {
        const uint32_t bins = digit_bins(pass);
        const int shift = digit_shift(pass);
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) count_digit(hist, (key[j] >> shift) & (bins - 1u), (key[j] & t.fixed) == t.low);
    }
}

// The digit that the need-th largest falls into; c0 and c1 are the counts of this
// thread's bins, 2047 - 2 * thread and the one below. Every thread meets it.
__device__ __forceinline__ void find_digit(EvictShared &sh, uint32_t c0, uint32_t c1, int pass, Threshold &t) {
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t top = kEvictBins - 1u - 2u * threadIdx.x;
    const uint32_t incl = wave_inclusive_scan<SumU32>(c0 + c1);
    if (lane_id() == kWave - 1) sh.wave[w] = incl;
    __syncthreads();
    const uint32_t totals = wave_inclusive_scan<SumU32>(lane_id() < kEvictWaves ? sh.wave[lane_id()] : 0u);
    const uint32_t earlier =
        w == 0 ? 0u : static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(totals), w - 1));
    const uint32_t above = earlier + incl - c0 - c1;
    if (above < t.need && t.need <= above + c0) {
        sh.digit = top;
        sh.above = above;
        sh.inside = c0;
    } else if (above + c0 < t.need && t.need <= above + c0 + c1) {
        sh.digit = top - 1u;
        sh.above = above + c0;
        sh.inside = c1;
    }
    __syncthreads();
    t.low |= sh.digit << digit_shift(pass);
    t.fixed |= (digit_bins(pass) - 1u) << digit_shift(pass);
    t.need -= sh.above;
    t.all = t.need == sh.inside;
}

// This wavefront's keys that stay, by item: those better than the threshold, and
// those equal to it where not all of them stay.
template <int ITEMS>
struct Staying {
    bool sure[ITEMS], equal[ITEMS];
    uint32_t sures, equals;

    __device__ __forceinline__ Staying(const uint32_t (&key)[ITEMS], const Threshold &t) : sures(0), equals(0) {
        const uint32_t from = t.all ? t.low : t.low + 1u;  // no threshold that others are equal to is the largest
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            sure[j] = key[j] >= from;
            equal[j] = key[j] == t.low && !t.all;
            sures += static_cast<uint32_t>(__builtin_popcountll(ballot(sure[j])));
            equals += static_cast<uint32_t>(__builtin_popcountll(ballot(equal[j])));
        }
    }
    // their positions, base + 64 j, from slot `at` on; of the equal ones, of which
    // `run` came before, the first `need` of all
    __device__ __forceinline__ void emit(const EvictArgs &a, const Head &head, uint32_t base, uint32_t at, uint32_t run,
                                         uint32_t need) const {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint64_t same = ballot(equal[j]);
            bool yes = sure[j];
            if (same != 0) {
                yes = yes || (equal[j] && run + mbcnt64(same) < need);
                run += static_cast<uint32_t>(__builtin_popcountll(same));
            }
            const uint64_t all = ballot(yes);
            const uint32_t slot = at + mbcnt64(all);
            if (yes && slot < a.keep) head.kept[slot] = static_cast<int32_t>(base + j * kWave);
            at += static_cast<uint32_t>(__builtin_popcountll(all));
        }
    }
};

// Sums over the wavefronts of what their lane 0 put into LDS: of those before
// wavefront w, and of all.
__device__ __forceinline__ uint32_t waves_before(const uint32_t *values, int w, uint32_t &all) {
    const uint32_t v = wave_inclusive_scan<SumU32>(lane_id() < kEvictWaves ? values[lane_id()] : 0u);
    all = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), kEvictWaves - 1));
    return w == 0 ? 0u : static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), w - 1));
}

__device__ __forceinline__ uint32_t least(uint32_t x, uint32_t y) { return x < y ? x : y; }

template <int ITEMS>
__global__ __launch_bounds__(kEvictBlock) void evict_kernel(EvictArgs a) {
    __shared__ EvictShared sh;
    const Head head(a, blockIdx.x, blockIdx.y);
    int32_t *count = a.counts + static_cast<int64_t>(blockIdx.y) * a.heads + blockIdx.x;
    if (head.len <= a.keep) {
        head.keep_all(a, count, threadIdx.x, kEvictBlock);
        return;
    }
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t base = static_cast<uint32_t>(w) * ITEMS * kWave + lane_id();
    uint32_t key[ITEMS];
    head.load(base, head.len, key);
    Threshold t{0u, 0u, a.keep, 0u};
    for (int pass = 0; pass < kEvictPasses && !t.all; ++pass) {
        for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) sh.hist[i] = 0;
        __syncthreads();
        count_digits(sh.hist, key, t, pass);
        __syncthreads();
        const uint32_t top = kEvictBins - 1u - 2u * threadIdx.x;
        find_digit(sh, sh.hist[top], sh.hist[top - 1u], pass, t);
    }
    const Staying<ITEMS> stay(key, t);
    __syncthreads();
    if (lane_id() == 0) {
        sh.wave[w] = stay.sures;
        sh.wave_equal[w] = stay.equals;
    }
    __syncthreads();
    uint32_t all;
    const uint32_t run = waves_before(sh.wave_equal, w, all);
    stay.emit(a, head, base, waves_before(sh.wave, w, all) + least(run, t.need), run, t.need);
    if (threadIdx.x == 0) *count = static_cast<int32_t>(a.keep);
}

// ---- by several workgroups ----
constexpr int kEvictItems = 8;
constexpr uint32_t kEvictTile = kEvictItems * kEvictBlock;

// The counts of pass - 1 joined over the splits: the digit, and how many scores of
// earlier splits stay for it (`equals`: of those that share the digits found, where
// not all of them do).
__device__ __forceinline__ void join_splits(const EvictArgs &a, EvictShared &sh, int64_t bh, int64_t rows, int pass,
                                            Threshold &t, uint32_t &before, uint32_t &equals) {
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t top = kEvictBins - 1u - 2u * threadIdx.x;
    const uint32_t *hist = a.hist + ((((pass - 1) & 1) * rows + bh) * a.splits) * kEvictBins;
    uint32_t c0 = 0, c1 = 0, b0 = 0, b1 = 0;
#pragma unroll 16
    for (uint32_t s = 0; s < a.splits; ++s) {
        const uint2 c = *reinterpret_cast<const uint2 *>(hist + static_cast<int64_t>(s) * kEvictBins + top - 1u);
        c0 += c.y;
        c1 += c.x;
        b0 += s < blockIdx.z ? c.y : 0u;
        b1 += s < blockIdx.z ? c.x : 0u;
    }
    find_digit(sh, c0, c1, pass - 1, t);
    const uint32_t d = sh.digit;
    const uint32_t mine = (top > d ? b0 : 0u) + (top - 1u > d ? b1 : 0u);
    const uint32_t sum = wave_inclusive_scan<SumU32>(mine);
    if (lane_id() == kWave - 1) sh.wave_equal[w] = sum;
    if (top == d) sh.before = b0;
    if (top - 1u == d) sh.before = b1;
    __syncthreads();
    uint32_t all;
    waves_before(sh.wave_equal, 0, all);
    before += all;
    equals = t.all ? 0u : sh.before;
    if (t.all) before += sh.before;
    __syncthreads();
}

// pass 0 .. 2: counts by a digit; 3: the output
template <bool LAST>
__global__ __launch_bounds__(kEvictBlock) void evict_split_kernel(EvictArgs a, int pass) {
    __shared__ EvictShared sh;
    const uint32_t split = blockIdx.z;
    const int64_t bh = static_cast<int64_t>(blockIdx.y) * a.heads + blockIdx.x;
    const int64_t rows = static_cast<int64_t>(gridDim.x) * gridDim.y;
    const Head head(a, blockIdx.x, blockIdx.y);
    if (head.len <= a.keep) {
        if (LAST) head.keep_all(a, a.counts + bh, split * kEvictBlock + threadIdx.x, a.splits * kEvictBlock);
        return;
    }
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t from = split * a.span;
    const uint32_t to = head.len - least(from, head.len) < a.span ? head.len : from + a.span;
    // the first tile's scores are on their way while the splits' counts are joined
    const uint32_t mine = static_cast<uint32_t>(w) * kEvictItems * kWave + lane_id();
    uint32_t key[kEvictItems];
    head.load(from + mine, to, key);
    Threshold t{0u, 0u, a.keep, 0u};
    uint32_t before = 0, equals = 0;
    if (pass > 0) {
        if (pass > 1) {
            t = a.found[bh * kEvictPasses + pass - 2];
            before = a.before[bh * a.splits + split];
        }
        if (!t.all) join_splits(a, sh, bh, rows, pass, t, before, equals);
        if (!LAST && threadIdx.x == 0) {
            if (split == 0) a.found[bh * kEvictPasses + pass - 1] = t;
            a.before[bh * a.splits + split] = before;
        }
    }
    if constexpr (!LAST) {
        if (t.all) return;
        for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) sh.hist[i] = 0;
        __syncthreads();
        for (uint32_t tile = from; tile < to; tile += kEvictTile) {
            if (tile != from) head.load(tile + mine, to, key);
            count_digits(sh.hist, key, t, pass);
        }
        __syncthreads();
        uint32_t *hist = a.hist + (((pass & 1) * rows + bh) * a.splits + split) * kEvictBins;
        for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) hist[i] = sh.hist[i];
    } else {
        for (uint32_t tile = from; tile < to; tile += kEvictTile) {
            if (tile != from) head.load(tile + mine, to, key);
            const Staying<kEvictItems> stay(key, t);
            if (lane_id() == 0) {
                sh.wave[w] = stay.sures;
                sh.wave_equal[w] = stay.equals;
            }
            __syncthreads();
            uint32_t all_sures, all_equals;
            const uint32_t run = equals + waves_before(sh.wave_equal, w, all_equals);
            stay.emit(a, head, tile + mine, before + waves_before(sh.wave, w, all_sures) + least(run, t.need), run, t.need);
            before += all_sures;
            equals += all_equals;
            __syncthreads();
        }
        if (split == 0 && threadIdx.x == 0) a.counts[bh] = static_cast<int32_t>(a.keep);
    }
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
    const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.heads + h;
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
    const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.heads + h;
    char *rows_at = a.to + b * a.to_batch + h * a.to_head;
    const int32_t *kept = a.kept + bh * a.keep;
    const int rows = kPlaceBlock >> a.lg;
    const int lane_col = static_cast<int>(threadIdx.x) & ((1 << a.lg) - 1);
    const int c0 = static_cast<int>(blockIdx.x) * a.cols, c1 = c0 + a.cols < a.chunks ? c0 + a.cols : a.chunks;
    const int64_t step = static_cast<int64_t>(rows) * kMoveFlight;
    // a slot's position, -1 for none: one that stays where it is needs no move, one
    // that lies before its slot is none of evict_rows
    int32_t pos[kMoveFlight], next[kMoveFlight];
    const auto positions = [&](int64_t set, int32_t(&p)[kMoveFlight]) {
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j) {
            const int64_t s = set + (threadIdx.x >> a.lg) + j * rows;
            const int32_t k = kept[s < a.keep ? s : a.keep - 1];
            p[j] = s < a.keep && k < a.capacity && k > s ? k : -1;
        }
    };
    typename P::V v[kMoveFlight];
    const auto load = [&](int base, const int32_t(&p)[kMoveFlight]) {
        const int c = base + lane_col;
        const int at = piece_at<BYTES>(a, c < c1 ? c : c0);
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j)
            if (p[j] >= 0 && c < c1) v[j] = P::load_stream(rows_at + static_cast<int64_t>(p[j]) * a.to_row + at);
    };
    positions(0, pos);
    load(c0, pos);
    for (int64_t set = 0; set < a.keep; set += step) {
        if (set + step < a.keep) positions(set + step, next);
        for (int base = c0; base < c1; base += 1 << a.lg) {
            __syncthreads();  // all of this set's pieces have been read
            const int c = base + lane_col;
            const int at = piece_at<BYTES>(a, c < c1 ? c : c0);
            const int64_t first = set + (threadIdx.x >> a.lg);
#pragma unroll
            for (int j = 0; j < kMoveFlight; ++j)
                if (pos[j] >= 0 && c < c1) P::store_stream(rows_at + (first + j * rows) * a.to_row + at, v[j]);
            // the next pieces are on their way while these are stored
            if (base + (1 << a.lg) < c1)
                load(base + (1 << a.lg), pos);
            else if (set + step < a.keep)
                load(c0, next);
        }
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j) pos[j] = next[j];
    }
}

// ============================================================ host side ---
int check_cache(int64_t batch, int64_t heads, int64_t capacity) {
    if (batch < 0 || heads < 1 || capacity < 1) return SSC_ERR_ARG;
    if (batch > INT32_MAX || heads > INT32_MAX || capacity > INT32_MAX - 4096 || batch * heads > 65535)
        return SSC_ERR_SIZE;
    return SSC_OK;
}

// Splits of a head: of 8192 positions where that gives up to 512 workgroups,
// else of 32,768, and longer ones where there would be over 64 of a head.
struct EvictPlan {
    uint32_t splits, span;
    size_t found, before, bytes;  // offsets into the scratch
};

EvictPlan evict_plan(int64_t rows, int64_t capacity) {
    EvictPlan p{};
    p.splits = 1;
    const int64_t tiles = (capacity + kEvictTile - 1) / kEvictTile;
    const bool few = rows * tiles <= 512 && capacity > 2 * kEvictTile;
    if (rows < 1 || (capacity <= kEvictHeld && !few)) return p;
    int64_t each = few ? 1 : kEvictHeld / kEvictTile;
    if (each < (tiles + 63) / 64) each = (tiles + 63) / 64;
    p.splits = static_cast<uint32_t>((tiles + each - 1) / each);
    p.span = static_cast<uint32_t>(each * kEvictTile);
    const size_t all = static_cast<size_t>(rows) * p.splits;
    p.found = 2 * all * kEvictBins * 4;
    p.before = p.found + static_cast<size_t>(rows) * kEvictPasses * sizeof(Threshold);
    p.bytes = p.before + all * 4;
    return p;
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

size_t ssc_evict_scratch_bytes(int64_t batch, int64_t heads, int64_t capacity) {
    if (check_cache(batch, heads, capacity) != SSC_OK) return 0;
    return evict_plan(batch * heads, capacity).bytes;
}

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
    a.weight_group = group * weight_head;
    a.weight_head = weight_head;
    a.weight_query = weight_query;
    a.lengths = lengths;
    a.length = static_cast<int>(length);
    a.group = static_cast<uint32_t>(group);
    a.queries = static_cast<uint32_t>(queries);
    a.fresh = fresh < length ? fresh : length;
    a.decay = decay;
    // one query a head, or all of a head's before the next head's: rows evenly apart
    if (queries == 1) a.weight_query = weight_head;
    const bool even = group == 1 || queries <= 1 || weight_head == queries * weight_query;
    const int64_t rows = group * queries;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t cols = kWave * 16 / static_cast<int64_t>(sizeof(T));
        const dim3 grid(static_cast<unsigned>((length + cols - 1) / cols), static_cast<unsigned>(heads),
                        static_cast<unsigned>(batch));
        const auto launch = [&](auto waves) {
            constexpr int W = decltype(waves)::value;
            if (even)
                hipLaunchKernelGGL((accumulate_kernel<T, W, true>), grid, dim3(W * kWave), 0,
                                   static_cast<hipStream_t>(stream), a);
            else
                hipLaunchKernelGGL((accumulate_kernel<T, W, false>), grid, dim3(W * kWave), 0,
                                   static_cast<hipStream_t>(stream), a);
            return launched();
        };
        if (rows <= 16) return launch(std::integral_constant<int, 1>{});
        if (rows <= 64) return launch(std::integral_constant<int, 4>{});
        return launch(std::integral_constant<int, 8>{});
    });
}

int ssc_evict_rows(const float *scores, int64_t batch, int64_t heads, int64_t capacity, int64_t score_batch,
                   int64_t score_head, const int32_t *lengths, int64_t keep, int64_t first, int64_t recent,
                   int32_t *kept, int32_t *counts, void *scratch, size_t scratch_bytes, void *stream) {
    SSC_TRY(check_cache(batch, heads, capacity));
    if (keep < 1 || keep > capacity || first < 0 || recent < 0 || first > keep || recent > keep - first)
        return SSC_ERR_ARG;
    const View<3> view{{batch, heads, capacity}, {score_batch, score_head, 1}};
    if (!view.strides_ok()) return SSC_ERR_ARG;
    if (batch > 0 && (scores == nullptr || kept == nullptr || counts == nullptr)) return SSC_ERR_ARG;
    if (!aligned(scores, 4) || !aligned(lengths, 4) || !aligned(kept, 4) || !aligned(counts, 4)) return SSC_ERR_ARG;
    const size_t rows = static_cast<size_t>(batch) * heads;
    const EvictPlan p = evict_plan(batch * heads, capacity);
    if (p.bytes > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < p.bytes)) return SSC_ERR_SCRATCH;
    const Span written[] = {{kept, rows * keep * 4}, {counts, rows * 4}, {scratch, p.bytes}};
    const Span read[] = {{scores, static_cast<size_t>(view.extent()) * 4}, {lengths, static_cast<size_t>(batch) * 4}};
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
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.splits > 1) {
        char *at = static_cast<char *>(scratch);
        a.splits = p.splits;
        a.span = p.span;
        a.hist = reinterpret_cast<uint32_t *>(at);
        a.found = reinterpret_cast<Threshold *>(at + p.found);
        a.before = reinterpret_cast<uint32_t *>(at + p.before);
        const dim3 grid(static_cast<unsigned>(heads), static_cast<unsigned>(batch), p.splits);
        for (int pass = 0; pass < kEvictPasses; ++pass) {
            hipLaunchKernelGGL((evict_split_kernel<false>), grid, dim3(kEvictBlock), 0, s, a, pass);
            SSC_TRY(launched());
        }
        hipLaunchKernelGGL((evict_split_kernel<true>), grid, dim3(kEvictBlock), 0, s, a, kEvictPasses);
        return launched();
    }
    const auto launch = [&](auto items) {
        hipLaunchKernelGGL((evict_kernel<decltype(items)::value>),
                           dim3(static_cast<unsigned>(heads), static_cast<unsigned>(batch)), dim3(kEvictBlock), 0, s, a);
        return launched();
    };
    if (capacity <= 4 * kEvictBlock) return launch(std::integral_constant<int, 4>{});
    if (capacity <= 8 * kEvictBlock) return launch(std::integral_constant<int, 8>{});
    if (capacity <= 16 * kEvictBlock) return launch(std::integral_constant<int, 16>{});
    return launch(std::integral_constant<int, 32>{});
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
    dim3 grid(1, static_cast<unsigned>(heads), static_cast<unsigned>(batch));
    if (place) {
        // few heads: their columns over several workgroups, where no two of
        // these share bytes of a row
        int parts = 1;
        while (a.row_bytes % bytes == 0 && batch * heads * parts < 512 && a.chunks / (parts * 2) >= 4 &&
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
