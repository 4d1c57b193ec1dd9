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
//
// Only the sixteen (or the last fifteen) are added up in fp32; what a wavefront of
// more has is held in fp64 and rounded once, so that a sum is off by 25 half steps
// of the magnitudes' at most (15, one rounding, 7 over the wavefronts, one over the
// parts, one for the earlier score), for any number of rows: 262,144 rows of one
// weight, in one chain a wavefront, were off by up to 3000.
//
// Rows that start anywhere are read by aligned loads and shifted into place in
// registers: a lane's piece ends in the next lane's load, so the last lane only
// reads. The loads stay inside the 16 bytes that hold a row's first and last
// element. 4 x 8 heads, 128 rows of 10,007 fp16: 18.9 us so, 23.7 by 16-byte loads
// from any address; of 10,240, where every row starts at such bytes: 16.5 without
// the shift, 19.5 with it.
//
// Bound by HBM: those 10,240 at 5.2 TB/s, 10,007 at 4.5; 32 x 8 heads of 8192, 4
// rows of bf16, 6.5 us (34 MB, 5.2 TB/s).
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
    // few long columns: the rows in `splits` parts, their sums in scratch
    uint32_t splits, col_blocks;
    float *part;  // [splits][batch][heads][length]
};

// Lanes of a wavefront that hold columns; SHIFT: rows that do not all start at a
// multiple of 16 bytes.
template <bool SHIFT>
constexpr int kColumnLanes = SHIFT ? kWave - 1 : kWave;

// Workgroups of up to this many wavefronts have up to sixteen rows for each.
constexpr int kFewWaves = 4;

// EVEN: the rows of a cache head lie evenly apart (queries of one head)
template <class T, int WAVES, bool EVEN, bool SHIFT>
__global__ __launch_bounds__(WAVES *kWave) void accumulate_kernel(AccumulateArgs a) {
    constexpr int kN = 16 / static_cast<int>(sizeof(T));
    constexpr int kFlight = 16;
    typedef T V __attribute__((ext_vector_type(kN)));
    typedef uint32_t Raw __attribute__((ext_vector_type(4)));
    typedef float Score __attribute__((ext_vector_type(4)));
    typedef float ScoreAny __attribute__((ext_vector_type(4), aligned(4), may_alias));
    __shared__ float s_sum[WAVES > 1 ? WAVES - 1 : 1][WAVES > 1 ? kWave * kN : 1];
    const int64_t h = blockIdx.y, b = blockIdx.z;
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int lane = lane_id();
    const uint32_t split = blockIdx.x / a.col_blocks;
    const int64_t block_first = static_cast<int64_t>(blockIdx.x - split * a.col_blocks) * (kColumnLanes<SHIFT> * kN);
    const int64_t first = block_first + lane * kN;
    float *to = a.scores + b * a.score_batch + h * a.score_head + first;
    int64_t len = a.length;
    if (a.lengths != nullptr) {
        const int64_t l = a.lengths[b];
        len = l < len ? l : len;
    }
    if (block_first >= len) return;
    // the earlier scores are on their way while the weights are read
    const int64_t old = len - a.fresh;  // positions with an earlier score
    Score before[kN / 4];
    const bool mine = w == 0 && lane < kColumnLanes<SHIFT>;
    const bool vector = first + kN <= len && first + kN <= old && mine && a.splits == 1;
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) before[i] = Score{0.0f, 0.0f, 0.0f, 0.0f};
    if (vector) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) before[i] = *reinterpret_cast<const ScoreAny *>(to + 4 * i);
    }
    float sum[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) sum[e] = 0.0f;
    const uint32_t all = a.group * a.queries, share = (all + a.splits - 1) / a.splits;
    const uint32_t begin = split * share < all ? split * share : all;  // the last parts may be empty
    const uint32_t rows = all - begin < share ? all : begin + share;
    // the row at the workgroup's first column, the same in all lanes
    const T *from = static_cast<const T *>(a.weights) + b * a.weight_batch + h * a.weight_group + block_first;
    const auto row = [&](uint32_t r) {
        if constexpr (EVEN) return from + r * a.weight_query;
        return from + (r / a.queries) * a.weight_head + (r % a.queries) * a.weight_query;
    };
    // bytes of a row's first load before that column
    const auto skip_of = [](const T *p) {
        return SHIFT ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u : 0u;
    };
    const uint64_t left = static_cast<uint64_t>(a.length - block_first) * sizeof(T) - 1;  // to the row's last byte
    const uint32_t last = left < 65536 ? static_cast<uint32_t>(left) : 65536u;
    const auto load = [&](const T *p) {
        const uint32_t skip = skip_of(p), most = (last + skip) & ~15u, at = 16u * lane;
        return __builtin_nontemporal_load(
            reinterpret_cast<const Raw *>(reinterpret_cast<const char *>(p) - skip + (at < most ? at : most)));
    };
    // a weight that is no number (of a query whose mask left nothing) adds nothing
    const auto add = [&](Raw raw, uint32_t skip) {
        if (skip != 0) {  // the same in all lanes
            const uint32_t two = skip & 8u ? ~0u : 0u, one = skip & 4u ? ~0u : 0u;
            const auto pick = [](uint32_t mask, uint32_t x, uint32_t y) { return (x & ~mask) | (y & mask); };
            const uint32_t x0 = raw[0], x1 = raw[1], x2 = raw[2], x3 = raw[3];
            const uint32_t x4 = dpp_move<0x130, 0xf>(x0), x5 = dpp_move<0x130, 0xf>(x1);  // of the next lane
            const uint32_t x6 = dpp_move<0x130, 0xf>(x2), x7 = dpp_move<0x130, 0xf>(x3);
            const uint32_t y0 = pick(two, x0, x2), y1 = pick(two, x1, x3), y2 = pick(two, x2, x4);
            const uint32_t y3 = pick(two, x3, x5), y4 = pick(two, x4, x6), y5 = pick(two, x5, x7);
            const uint32_t z0 = pick(one, y0, y1), z1 = pick(one, y1, y2), z2 = pick(one, y2, y3);
            const uint32_t z3 = pick(one, y3, y4), z4 = pick(one, y4, y5);
            raw = Raw{__builtin_amdgcn_alignbyte(z1, z0, skip & 3u), __builtin_amdgcn_alignbyte(z2, z1, skip & 3u),
                      __builtin_amdgcn_alignbyte(z3, z2, skip & 3u), __builtin_amdgcn_alignbyte(z4, z3, skip & 3u)};
        }
        const V v = __builtin_bit_cast(V, raw);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float y = static_cast<float>(v[e]);
            sum[e] += y == y ? y : 0.0f;
        }
    };
    double total[WAVES > kFewWaves ? kN : 1];  // of the wavefront's rows before those in `sum`
#pragma unroll
    for (double &t : total) t = 0.0;
    uint32_t r = begin + w;
    const auto some = [&](auto count) {
        constexpr int C = decltype(count)::value;
        Raw raw[C];
#pragma unroll
        for (int j = 0; j < C; ++j) raw[j] = load(row(r + j * WAVES));
        __builtin_amdgcn_sched_barrier(0);  // all of them first: left alone, one waits for another
#pragma unroll
        for (int j = 0; j < C; ++j) add(raw[j], skip_of(row(r + j * WAVES)));
        r += C * WAVES;
    };
    while (r + (kFlight - 1) * WAVES < rows) {
        some(std::integral_constant<int, kFlight>{});
        if constexpr (WAVES > kFewWaves) {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                total[e] += static_cast<double>(sum[e]);
                sum[e] = 0.0f;
            }
        }
    }
    if (r + 7 * WAVES < rows) some(std::integral_constant<int, 8>{});
    if (r + 3 * WAVES < rows) some(std::integral_constant<int, 4>{});
    while (r < rows) some(std::integral_constant<int, 1>{});
    if constexpr (WAVES > kFewWaves) {
#pragma unroll
        for (int e = 0; e < kN; ++e) sum[e] = static_cast<float>(total[e] + static_cast<double>(sum[e]));
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
    if (a.splits > 1) {
        float *part = a.part + ((static_cast<int64_t>(split) * gridDim.z + b) * gridDim.y + h) * a.length + first;
#pragma unroll
        for (int e = 0; e < kN; ++e)
            if (mine && first + e < len) part[e] = sum[e];
    } else if (vector) {
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
            if (mine && i < len) to[e] = i < old ? __builtin_fmaf(to[e], a.decay, sum[e]) : sum[e];
        }
    }
}

// The parts' sums joined, in their order, in fp64.
__global__ __launch_bounds__(256) void accumulate_join_kernel(AccumulateArgs a) {
    const int64_t h = blockIdx.y, b = blockIdx.z;
    int64_t len = a.length;
    if (a.lengths != nullptr) {
        const int64_t l = a.lengths[b];
        len = l < len ? l : len;
    }
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= len) return;
    float *to = a.scores + b * a.score_batch + h * a.score_head + i;
    const float old = i < len - a.fresh ? *to : 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.z) * gridDim.y * a.length;
    const float *part = a.part + (b * gridDim.y + h) * a.length + i;
    double all = 0.0;
#pragma unroll 8
    for (uint32_t s = 0; s < a.splits; ++s) all += static_cast<double>(part[s * step]);
    const float sum = static_cast<float>(all);
    *to = i < len - a.fresh ? __builtin_fmaf(old, a.decay, sum) : sum;
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
// several workgroups (splits) and three launches: counts by the first digit;
// these joined, counts by the second and a list of the scores that share the
// first; those joined, the third digit from the lists, and the output.
//
// Bound by latency, of the steps of a workgroup or of three launches: 256 heads of
// 8192 cut to 4096 9.6 us (10 MB moved, 2 us at a copy's rate), 8 of 131,072 cut to
// 16,384 4.5 + 7.9 + 9.1 us traced and 16 to 20 a call, as their lengths fall; by one
// workgroup a head 168.
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
    Threshold *found;       // [rows] by the first digit
    uint32_t *before;       // [rows][splits] scores of earlier splits that stay for it
    uint32_t *hist;         // [2][rows][splits][bins] of the first two digits
    uint32_t *listed;       // [rows][splits] scores that share the first digit,
    uint32_t *list;         // [rows][splits][span] and they, in no order
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

// How many scores of earlier splits stay for the digit that was found: those of
// larger ones, and its own if all of it does. Otherwise `equals` is the number
// of its own. b0 and b1 are the earlier splits' counts of this thread's bins.
__device__ __forceinline__ void count_before(EvictShared &sh, uint32_t top, uint32_t b0, uint32_t b1,
                                             const Threshold &t, uint32_t &before, uint32_t &equals) {
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
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

// The splits' counts of a pass joined.
__device__ __forceinline__ void join_splits(const EvictArgs &a, EvictShared &sh, int64_t bh, int64_t rows, int pass,
                                            Threshold &t, uint32_t &before, uint32_t &equals) {
    const uint32_t top = kEvictBins - 1u - 2u * threadIdx.x;
    const uint32_t *hist = a.hist + ((pass * rows + bh) * a.splits) * kEvictBins;
    uint32_t c0 = 0, c1 = 0, b0 = 0, b1 = 0;
#pragma unroll 16
    for (uint32_t s = 0; s < a.splits; ++s) {
        const uint2 c = *reinterpret_cast<const uint2 *>(hist + static_cast<int64_t>(s) * kEvictBins + top - 1u);
        c0 += c.y;
        c1 += c.x;
        b0 += s < blockIdx.z ? c.y : 0u;
        b1 += s < blockIdx.z ? c.x : 0u;
    }
    find_digit(sh, c0, c1, pass, t);
    count_before(sh, top, b0, b1, t, before, equals);
}

// The third digit from the lists of the scores that share the first, of which a
// wavefront reads every 16th split's.
__device__ __forceinline__ void join_lists(const EvictArgs &a, EvictShared &sh, uint32_t *before_hist, int64_t bh,
                                           Threshold &t, uint32_t &before, uint32_t &equals) {
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) {
        sh.hist[i] = 0;
        before_hist[i] = 0;
    }
    __syncthreads();
    for (uint32_t s = w; s < a.splits; s += kEvictWaves) {
        const uint32_t n = least(a.listed[bh * a.splits + s], a.span);
        const uint32_t *list = a.list + (bh * a.splits + s) * a.span;
        for (uint32_t i = 0; i < n; i += 4 * kWave) {
            uint32_t k[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) k[j] = list[least(i + j * kWave + lane, n - 1u)];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const bool counts = i + j * kWave + lane < n && (k[j] & t.fixed) == t.low;
                count_digit(sh.hist, k[j] & 1023u, counts);
                if (s < blockIdx.z) count_digit(before_hist, k[j] & 1023u, counts);
            }
        }
    }
    __syncthreads();
    const uint32_t top = kEvictBins - 1u - 2u * threadIdx.x;
    const uint32_t b0 = before_hist[top], b1 = before_hist[top - 1u];
    find_digit(sh, sh.hist[top], sh.hist[top - 1u], 2, t);
    count_before(sh, top, b0, b1, t, before, equals);
}

enum EvictStep { kFirstDigit, kSecondDigit, kOutput };

template <EvictStep STEP>
__global__ __launch_bounds__(kEvictBlock) void evict_split_kernel(EvictArgs a) {
    __shared__ EvictShared sh;
    __shared__ uint32_t s_more[STEP == kOutput ? kEvictBins : 1];
    const uint32_t split = blockIdx.z;
    const int64_t bh = static_cast<int64_t>(blockIdx.y) * a.heads + blockIdx.x;
    const int64_t rows = static_cast<int64_t>(gridDim.x) * gridDim.y;
    const Head head(a, blockIdx.x, blockIdx.y);
    if (head.len <= a.keep) {
        if (STEP == kOutput) head.keep_all(a, a.counts + bh, split * kEvictBlock + threadIdx.x, a.splits * kEvictBlock);
        return;
    }
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t from = split * a.span;
    const uint32_t to = head.len - least(from, head.len) < a.span ? head.len : from + a.span;
    // the first tile's scores are on their way while the splits' counts are joined
    const uint32_t mine = static_cast<uint32_t>(w) * kEvictItems * kWave + lane;
    uint32_t key[kEvictItems];
    head.load(from + mine, to, key);
    Threshold t{0u, 0u, a.keep, 0u};
    uint32_t before = 0, equals = 0;
    if constexpr (STEP == kSecondDigit) {
        join_splits(a, sh, bh, rows, 0, t, before, equals);
        if (threadIdx.x == 0) {
            if (split == 0) a.found[bh] = t;
            a.before[bh * a.splits + split] = before;
            sh.before = 0;  // scores listed so far
        }
        if (t.all) return;
    }
    if constexpr (STEP == kOutput) {
        t = a.found[bh];
        before = a.before[bh * a.splits + split];
        if (!t.all) join_splits(a, sh, bh, rows, 1, t, before, equals);
        if (!t.all) join_lists(a, sh, s_more, bh, t, before, equals);
    }
    if constexpr (STEP != kOutput) {
        constexpr int kPass = STEP == kFirstDigit ? 0 : 1;
        for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) sh.hist[i] = 0;
        __syncthreads();
        uint32_t *list = a.list + (bh * a.splits + split) * a.span;
        for (uint32_t tile = from; tile < to; tile += kEvictTile) {
            if (tile != from) head.load(tile + mine, to, key);
            count_digits(sh.hist, key, t, kPass);
            if constexpr (STEP == kSecondDigit) {
                uint32_t many = 0;
#pragma unroll
                for (int j = 0; j < kEvictItems; ++j)
                    many += static_cast<uint32_t>(__builtin_popcountll(ballot((key[j] & t.fixed) == t.low)));
                uint32_t at = 0;
                if (lane == 0 && many > 0)
                    at = __hip_atomic_fetch_add(&sh.before, many, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                at = uniform(at);
#pragma unroll
                for (int j = 0; j < kEvictItems; ++j) {
                    const bool shares = (key[j] & t.fixed) == t.low;
                    const uint64_t shared = ballot(shares);
                    const uint32_t slot = at + mbcnt64(shared);
                    if (shares && slot < a.span) list[slot] = key[j];
                    at += static_cast<uint32_t>(__builtin_popcountll(shared));
                }
            }
        }
        __syncthreads();
        uint32_t *hist = a.hist + ((kPass * rows + bh) * a.splits + split) * kEvictBins;
        for (uint32_t i = threadIdx.x; i < kEvictBins; i += kEvictBlock) hist[i] = sh.hist[i];
        if (STEP == kSecondDigit && threadIdx.x == 0) a.listed[bh * a.splits + split] = sh.before;
    } else {
        for (uint32_t tile = from; tile < to; tile += kEvictTile) {
            if (tile != from) head.load(tile + mine, to, key);
            const Staying<kEvictItems> stay(key, t);
            if (lane == 0) {
                sh.wave[w] = stay.sures;
                sh.wave_equal[w] = stay.equals;
            }
            __syncthreads();
            uint32_t all_sures, all_equals;
            const uint32_t run = equals + waves_before(sh.wave_equal, w, all_equals);
            stay.emit(a, head, tile + mine, before + waves_before(sh.wave, w, all_sures) + least(run, t.need), run,
                      t.need);
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
//
// Bound by HBM: 256 heads, 4096 rows of 256 bytes in place 102 us, 541 MB at 5.3
// TB/s, a copy's rate. Small moves by the launch: 15 heads, 509 rows of 130 bytes to
// another cache 3.8 us.
struct MoveArgs {
    const char *from;
    char *to;
    int64_t from_batch, from_head, from_row;  // strides in bytes
    int64_t to_batch, to_head, to_row;
    const int32_t *kept;
    int heads, capacity, keep;
    int row_bytes, chunks;
    int moved;   // 0: every row that is kept; in place, those that lie past their slot: to scratch (1),
                 // or from there (2), where row s is slot s's
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
    // no load waits behind a branch: a slot without a row reads row 0
    int32_t k[kMoveFlight];
#pragma unroll
    for (int j = 0; j < kMoveFlight; ++j) {
        const int64_t s = first + j * rows;
        k[j] = kept[s < a.keep ? s : a.keep - 1];
    }
    bool moves[kMoveFlight];
    const char *src[kMoveFlight];
#pragma unroll
    for (int j = 0; j < kMoveFlight; ++j) {
        const int64_t s = first + j * rows;
        moves[j] = s < a.keep && k[j] >= 0 && k[j] < a.capacity && (a.moved == 0 || k[j] > s);
        src[j] = from + (moves[j] ? (a.moved == 2 ? s : k[j]) : 0) * a.from_row;
    }
    for (int c = static_cast<int>(threadIdx.x) & ((1 << a.lg) - 1); c < a.chunks; c += 1 << a.lg) {
        const int at = piece_at<BYTES>(a, c);
        typename P::V v[kMoveFlight];
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j) v[j] = P::load_stream(src[j] + at);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kMoveFlight; ++j)
            if (moves[j]) P::store_stream(to + (first + j * rows) * a.to_row + at, v[j]);
    }
}

constexpr int kPlaceBlock = 1024;
constexpr int kPlaceFlight = 4;  // pieces of a lane at a time

template <int BYTES>
__global__ __launch_bounds__(kPlaceBlock) void move_in_place_kernel(MoveArgs a) {
    using P = Piece<BYTES>;
    // the columns of a head last: where the heads are a multiple of 8 they share an XCD
    const int64_t h = blockIdx.x, b = blockIdx.y, bh = b * a.heads + h;
    char *rows_at = a.to + b * a.to_batch + h * a.to_head;
    const int32_t *kept = a.kept + bh * a.keep;
    const int rows = kPlaceBlock >> a.lg;
    const int lane_col = static_cast<int>(threadIdx.x) & ((1 << a.lg) - 1);
    const int c0 = static_cast<int>(blockIdx.z) * a.cols, c1 = c0 + a.cols < a.chunks ? c0 + a.cols : a.chunks;
    const int64_t step = static_cast<int64_t>(rows) * kPlaceFlight;
    // a slot's position, -1 for none: one that stays where it is needs no move, one
    // that lies before its slot is none of evict_rows
    int32_t pos[kPlaceFlight], next[kPlaceFlight];
    const auto positions = [&](int64_t set, int32_t(&p)[kPlaceFlight]) {
        int32_t k[kPlaceFlight];
#pragma unroll
        for (int j = 0; j < kPlaceFlight; ++j) {
            const int64_t s = set + (threadIdx.x >> a.lg) + j * rows;
            k[j] = kept[s < a.keep ? s : a.keep - 1];
        }
#pragma unroll
        for (int j = 0; j < kPlaceFlight; ++j) {
            const int64_t s = set + (threadIdx.x >> a.lg) + j * rows;
            p[j] = s < a.keep && k[j] < a.capacity && k[j] > s ? k[j] : -1;
        }
    };
    // no load waits behind a branch: a slot without a row reads row 0
    typename P::V v[kPlaceFlight];
    const auto load = [&](int base, const int32_t(&p)[kPlaceFlight]) {
        const int c = base + lane_col;
        const int at = piece_at<BYTES>(a, c < c1 ? c : c0);
#pragma unroll
        for (int j = 0; j < kPlaceFlight; ++j)
            v[j] = P::load_stream(rows_at + static_cast<int64_t>(p[j] >= 0 ? p[j] : 0) * a.to_row + at);
    };
    positions(0, pos);
    load(c0, pos);
    for (int64_t set = 0; set < a.keep; set += step) {
        if (set + step < a.keep) positions(set + step, next);
        for (int base = c0; base < c1; base += 1 << a.lg) {
            // All of this set's pieces have been read: the barrier alone does not wait for
            // loads under way, and other wavefronts store where they read.
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            const int c = base + lane_col;
            const int at = piece_at<BYTES>(a, c < c1 ? c : c0);
            const int64_t first = set + (threadIdx.x >> a.lg);
#pragma unroll
            for (int j = 0; j < kPlaceFlight; ++j)
                if (pos[j] >= 0 && c < c1) P::store_stream(rows_at + (first + j * rows) * a.to_row + at, v[j]);
            // the next pieces are on their way while these are stored
            if (base + (1 << a.lg) < c1)
                load(base + (1 << a.lg), pos);
            else if (set + step < a.keep)
                load(c0, next);
        }
#pragma unroll
        for (int j = 0; j < kPlaceFlight; ++j) pos[j] = next[j];
    }
}

// ============================================================ host side ---
int check_cache(int64_t batch, int64_t heads, int64_t capacity) {
    if (batch < 0 || heads < 1 || capacity < 1) return SSC_ERR_ARG;
    if (batch > INT32_MAX || heads > INT32_MAX || capacity > INT32_MAX - 4096 || batch * heads > 65535)
        return SSC_ERR_SIZE;
    return SSC_OK;
}

// Where the wavefronts are few (under 2048) and have over 16 rows each, the rows in
// parts, up to 4096 wavefronts in all. Two heads of 4 sequences, 456 rows of 1390
// fp16: 39 us a call in one part, 11.5 in four (traced 8.7 and 3.6 for the join).
struct AccumulatePlan {
    uint32_t splits;
    size_t bytes;
};

AccumulatePlan accumulate_plan(int64_t heads, int64_t rows, int64_t length, int dtype) {
    AccumulatePlan p{};
    const int64_t cols = kColumnLanes<true> * 16 / static_cast<int64_t>(elem_bytes(dtype));
    p.splits = 1;
    const int64_t waves = heads * ((length + cols - 1) / cols) * 8;
    if (waves > 0 && waves < 2048 && rows > 128) {
        const int64_t wanted = (4096 + waves - 1) / waves, most = (rows + 127) / 128;
        p.splits = static_cast<uint32_t>(wanted < most ? wanted : most);
        p.bytes = static_cast<size_t>(p.splits) * heads * length * 4;
    }
    return p;
}

// A move in place: directly, few heads with their columns over several
// workgroups (no two of these share bytes of a row, nor less than 64 bytes), or
// by way of scratch. A workgroup's set of rows takes 4.5 us one after another; the
// scratch doubles the traffic but has no such order. Rows moved, direct against
// scratch, us, and the rows read and written once at a copy's rate:
//   2 heads x 20,000 of 128 bytes   84  9.5   2.0    4 heads x 2500 of 1024 bytes   19   13   4.0
//   8 x 20,000 of 256               88   35    16    8 x 1024 of 256               5.6  9.8   0.8
//   22 x 4382 of 192                25   18   7.2    48 x 4695 of 256               36   46    22
//   32 x 2048 of 130                32   14   3.3    256 x 4096 of 256             102  188   104
// 8 x 20,000 of 256, traced: 17.2 us to scratch and 17.2 back, each 41 MB read and 41 written.
struct MovePlan {
    int piece, cols;
    size_t bytes;
};

MovePlan move_plan(int64_t heads, int64_t keep, int64_t row_bytes, int elem) {
    MovePlan p{};
    // pieces that overlap must all be read before one is stored
    const bool overlap = row_bytes % 16 != 0 && row_bytes > 16 << 8;
    p.piece = row_bytes >= 16 && !overlap ? 16 : elem;
    const int64_t chunks = (row_bytes + p.piece - 1) / p.piece;
    int64_t parts = 1;
    if (row_bytes % p.piece == 0 && heads > 0) {
        const int64_t most = chunks * p.piece / 64;
        parts = 512 / heads;
        parts = parts < most ? parts : most;
        parts = parts < 1 ? 1 : parts;
    }
    p.cols = static_cast<int>((chunks + parts - 1) / parts);
    int lg = 0;
    while (lg < 8 && (1 << lg) < p.cols) ++lg;
    const int64_t set = (kPlaceBlock >> lg) * kPlaceFlight;
    const double sets = static_cast<double>((keep + set - 1) / set) * ((p.cols + (1 << lg) - 1) >> lg);
    const double bytes = static_cast<double>(heads) * static_cast<double>(keep) * static_cast<double>(row_bytes);
    if (4.5 * sets > 6.0 + 4.0 * bytes / 6.3e6) p.bytes = static_cast<size_t>(heads) * keep * row_bytes;
    return p;
}

// Splits of a head: of 8192 positions where that gives up to 512 workgroups,
// else of 32,768, and longer ones where there would be over 64 of a head. us a call,
// one workgroup a head against splits of 8192 (of 16,384):
//   8 x 20,000     18.0  16.1      128 x 20,000    19.8  28.4      320 x 20,000     37  53 (47)
//   64 x 20,000    19.5  18.3      128 x 32,768    22.2  33.7      320 x 32,768     42  73 (63)
// (the border is right for longer heads; the 128 would take the other side), and splits
// of 8192 against 32,768:
//   8 x 65,536     18.3  33.0      64 x 65,536     36.1  38.0      320 x 65,536    170  111
//   8 x 131,072    20.3  34.3      80 x 65,536     47.2  38.6      320 x 131,072   348  186
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
    p.before = p.found + static_cast<size_t>(rows) * sizeof(Threshold);
    p.bytes = p.before + 2 * all * 4 + all * p.span * 4;
    return p;
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

size_t ssc_accumulate_scratch_bytes(int64_t batch, int64_t heads, int64_t group, int64_t queries, int64_t length,
                                    int dtype) {
    if (check_cache(batch, heads, 1) != SSC_OK || !dtype_ok(dtype) || group < 1 || queries < 0 || length < 0 ||
        length > INT32_MAX || group > INT32_MAX || queries > INT32_MAX)
        return 0;
    return accumulate_plan(batch * heads, group * queries, length, dtype).bytes;
}

size_t ssc_move_scratch_bytes(int elem_bytes, int64_t batch, int64_t heads, int64_t keep, int64_t width) {
    if (check_cache(batch, heads, 1) != SSC_OK || batch < 1 || keep < 1 || keep > INT32_MAX || width < 1 ||
        width > (1 << 24) || elem_bytes < 1 || elem_bytes > 8)
        return 0;
    return move_plan(batch * heads, keep, width * elem_bytes, elem_bytes).bytes;
}

size_t ssc_evict_scratch_bytes(int64_t batch, int64_t heads, int64_t capacity) {
    if (check_cache(batch, heads, capacity) != SSC_OK) return 0;
    return evict_plan(batch * heads, capacity).bytes;
}

int ssc_accumulate_weights(float *scores, int64_t batch, int64_t heads, int64_t capacity, int64_t score_batch,
                           int64_t score_head, const void *weights, int dtype, int64_t group, int64_t queries,
                           int64_t length, int64_t weight_batch, int64_t weight_head, int64_t weight_query,
                           const int32_t *lengths, int64_t fresh, float decay, void *scratch, size_t scratch_bytes,
                           void *stream) {
    SSC_TRY(check_cache(batch, heads, capacity));
    if (!dtype_ok(dtype) || group < 1 || queries < 0 || length < 0 || length > capacity || fresh < 0) return SSC_ERR_ARG;
    if (group > INT32_MAX || queries > INT32_MAX || group * queries > (int64_t{1} << 30) || heads * group > INT32_MAX)
        return SSC_ERR_SIZE;
    const View<3> s{{batch, heads, capacity}, {score_batch, score_head, 1}};
    const View<4> w{{batch, heads * group, queries, length}, {weight_batch, weight_head, weight_query, 1}};
    if (!s.strides_ok() || !w.strides_ok() || !s.distinct()) return SSC_ERR_ARG;
    if (batch > 0 && (scores == nullptr || (w.extent() > 0 && weights == nullptr))) return SSC_ERR_ARG;
    if (!aligned(scores, 4) || !aligned(weights, elem_bytes(dtype)) || !aligned(lengths, 4)) return SSC_ERR_ARG;
    const AccumulatePlan p = accumulate_plan(batch * heads, group * queries, length, dtype);
    if (p.bytes > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < p.bytes)) return SSC_ERR_SCRATCH;
    const Span written[] = {{scores, static_cast<size_t>(s.extent()) * 4}, {scratch, p.bytes}};
    const Span read[] = {{weights, static_cast<size_t>(w.extent()) * elem_bytes(dtype)},
                         {lengths, static_cast<size_t>(batch) * 4}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &x : written)
        for (const Span &y : read)
            if (overlap(x.p, x.bytes, y.p, y.bytes)) return SSC_ERR_ALIAS;
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
    a.splits = p.splits;
    a.part = static_cast<float *>(scratch);
    const int64_t es = static_cast<int64_t>(elem_bytes(dtype));
    const bool shift = !aligned(weights, 16) || (batch > 1 && weight_batch * es % 16 != 0) ||
                       (heads * group > 1 && weight_head * es % 16 != 0) || (queries > 1 && weight_query * es % 16 != 0);
    const int64_t cols = (shift ? kColumnLanes<true> : kColumnLanes<false>)*16 / es;
    a.col_blocks = static_cast<uint32_t>((length + cols - 1) / cols);
    SSC_TRY(with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const dim3 grid(p.splits * a.col_blocks, static_cast<unsigned>(heads), static_cast<unsigned>(batch));
        const auto launch = [&](auto waves, auto e, auto sh) {
            constexpr int W = decltype(waves)::value;
            hipLaunchKernelGGL((accumulate_kernel<T, W, decltype(e)::value, decltype(sh)::value>), grid,
                               dim3(W * kWave), 0, static_cast<hipStream_t>(stream), a);
            return launched();
        };
        const auto shaped = [&](auto waves) {
            if (even)
                return shift ? launch(waves, std::true_type{}, std::true_type{})
                             : launch(waves, std::true_type{}, std::false_type{});
            return shift ? launch(waves, std::false_type{}, std::true_type{})
                         : launch(waves, std::false_type{}, std::false_type{});
        };
        if (rows <= 16) return shaped(std::integral_constant<int, 1>{});
        if (rows <= 16 * kFewWaves) return shaped(std::integral_constant<int, kFewWaves>{});
        return shaped(std::integral_constant<int, 8>{});
    }));
    if (p.splits == 1) return SSC_OK;
    hipLaunchKernelGGL(accumulate_join_kernel,
                       dim3(static_cast<unsigned>((length + 255) / 256), static_cast<unsigned>(heads),
                            static_cast<unsigned>(batch)),
                       dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return launched();
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
        a.listed = a.before + rows * p.splits;
        a.list = a.listed + rows * p.splits;
        const dim3 grid(static_cast<unsigned>(heads), static_cast<unsigned>(batch), p.splits);
        hipLaunchKernelGGL((evict_split_kernel<kFirstDigit>), grid, dim3(kEvictBlock), 0, s, a);
        SSC_TRY(launched());
        hipLaunchKernelGGL((evict_split_kernel<kSecondDigit>), grid, dim3(kEvictBlock), 0, s, a);
        SSC_TRY(launched());
        hipLaunchKernelGGL((evict_split_kernel<kOutput>), grid, dim3(kEvictBlock), 0, s, a);
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
                  void *out, int64_t out_batch, int64_t out_head, int64_t out_row, void *scratch, size_t scratch_bytes,
                  void *stream) {
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
    const MovePlan p = move_plan(batch * heads, keep, width * elem_bytes, elem_bytes);
    const size_t need = place ? p.bytes : 0;
    if (need > 0) {
        if (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < need) return SSC_ERR_SCRATCH;
        if (overlap(scratch, need, out, cache_bytes) ||
            overlap(scratch, need, kept, static_cast<size_t>(batch) * heads * keep * 4))
            return SSC_ERR_ALIAS;
    }
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
    const bool direct = place && need == 0;
    const int bytes = direct ? p.piece : (a.row_bytes >= 16 ? 16 : elem_bytes);
    a.chunks = (a.row_bytes + bytes - 1) / bytes;
    a.cols = direct ? p.cols : a.chunks;
    while (a.lg < 8 && (1 << a.lg) < a.cols) ++a.lg;
    const int64_t rows = static_cast<int64_t>(kMoveBlock >> a.lg) * kMoveFlight;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const auto launch = [&](auto piece) {
        constexpr int B = decltype(piece)::value;
        if (direct) {
            const dim3 grid(static_cast<unsigned>(heads), static_cast<unsigned>(batch),
                            static_cast<unsigned>((a.chunks + a.cols - 1) / a.cols));
            hipLaunchKernelGGL((move_in_place_kernel<B>), grid, dim3(kPlaceBlock), 0, s, a);
            return launched();
        }
        const dim3 grid(static_cast<unsigned>((keep + rows - 1) / rows), static_cast<unsigned>(heads),
                        static_cast<unsigned>(batch));
        if (!place) {
            hipLaunchKernelGGL((move_kernel<B>), grid, dim3(kMoveBlock), 0, s, a);
            return launched();
        }
        MoveArgs m = a;  // to scratch, and back into place
        m.moved = 1;
        m.to = static_cast<char *>(scratch);
        m.to_row = a.row_bytes;
        m.to_head = keep * m.to_row;
        m.to_batch = heads * m.to_head;
        hipLaunchKernelGGL((move_kernel<B>), grid, dim3(kMoveBlock), 0, s, m);
        SSC_TRY(launched());
        m.moved = 2;
        m.from = m.to;
        m.from_row = m.to_row;
        m.from_head = m.to_head;
        m.from_batch = m.to_batch;
        m.to = a.to;
        m.to_row = a.to_row;
        m.to_head = a.to_head;
        m.to_batch = a.to_batch;
        hipLaunchKernelGGL((move_kernel<B>), grid, dim3(kMoveBlock), 0, s, m);
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
