// The next token of a row of logits, from a given random number, under
// temperature, top-k, top-p and min-p: HIP kernels for MI355X (gfx950) and
// their part of the C ABI in include/ssc.h.
//
// Every filter keeps a prefix of the row in the order (logit descending,
// index ascending). No row is sorted: a histogram over 2048 bins of distance
// from the row's maximum shows which bin a filter's border falls into, the few
// logits of that bin are collected (a compaction) and sorted alone, and
// everything in better bins is kept without a look at its order. The token is
// the first index at which the running kept weight exceeds u times its sum:
// a selection by a scan, over the sums of parts of the row, then inside one
// part.
//
// Weights exp((x - max) / T) are computed in fp64 and held as integers with
// 62 - bits(vocab) fractional bits (at most 50): integer sums do not depend
// on their order, so rows may be split and added with atomics, and a call
// repeats bit for bit.
//
// Launches, each over parts of rows except the last: maxima; histograms (only
// where a filter is given; a row's last workgroup finds the border bins); sums
// of the better bins with the border bins' logits collected; border and token.
// 256 rows of 131,072 bf16 under mixed settings take 12 + 32 + 28 + 11 us, the
// first bound by HBM, the second by exponentials and 64-bit LDS adds in the rows
// that top_p alone cuts (256 such rows 43 us, 256 of top_k 23) and the latency of
// its steps, the third by exponentials, the last by latency; one such row of
// fp32 takes 3.0 + 7.6 + 4.4 + 7.6 us, latency throughout: as one compute unit
// runs a row's histogram end and its token, an instruction of every wavefront
// counts there, and a load that waits for another counts twice.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssc.h"
#include "ssc_device.h"
#include "ssc_host.h"

namespace ssc {
namespace {

constexpr int kPartLg = 12;
constexpr int kPart = 1 << kPartLg;   // logits of a part
constexpr int kPartBlock = 256;
constexpr int kPartItems = kPart / kPartBlock;
constexpr int kHistPart = 8192;       // fewest logits of a workgroup of a row's histogram
constexpr int kHistMost = 32768;      // and most, where the row is split
constexpr int kHistBlock = 512;
constexpr int kBins = 2048;
constexpr int kTokenBlock = 1024;
constexpr int kList = 4096;           // collected logits a row has room for
constexpr int kListTopK = kList / 2;  // up to this top_k, all its logits are collected
constexpr int64_t kVocabMax = int64_t{1} << 22;
constexpr int kPartsMax = static_cast<int>(kVocabMax / kPart);
static_assert(kPartsMax <= kTokenBlock, "a part to a thread");
constexpr uint32_t kNoCut = 0xffffffffu;

// What is known of a row's border. Bins are numbered from the maximum down:
// those below `lo` are kept, those in [lo, hi] and `extra` are collected.
struct RowState {
    uint64_t mass;        // weight of the bins below lo ...
    uint64_t extra_mass;  // ... and below extra
    uint64_t total;       // of the row, where top_p alone cuts it; else 0
    double rate;          // log2(e) / temperature, divided once
    uint32_t count, extra_count;  // their logits
    int32_t lo, hi, extra;        // extra: top_k's border bin, where top_p's lies before it (-1: none)
    uint32_t listed;      // logits collected so far (may pass kList: the list is then not used)
    uint32_t done;        // workgroups of the row that have added their histogram
};

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int vocab, parts, bits;  // bits: fractional bits of a weight
    int splits;              // workgroups of a row's histogram
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens, *kept;
    float *logprobs;
    // scratch
    float2 *part_range;      // [rows][parts] largest and smallest token logit
    uint64_t *part_mass;     // [rows][parts]
    uint32_t *part_count;    // [rows][parts]
    RowState *state;         // [rows]
    uint64_t *hist_mass;     // [rows][kBins], where a filter is given
    uint32_t *hist_count;    // [rows][kBins]
    uint64_t *list;          // [rows][kList]
};

// The logit as an integer of the same order; 0 for NaN and -infinity, which
// are no token. -0 counts as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return x > -__builtin_inff() ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// A row's filters, with what is out of range put in its place.
struct Filters {
    float t;        // temperature; 0: the first of the order alone
    float top_p;    // 2: off
    int32_t top_k;  // 0: off
    float min_p, u;

    // u stands in for a setting that is not given, so that no load waits
    // behind a branch and all are in flight together
    __device__ __forceinline__ Filters(const SampleArgs &a, int row) {
        const auto at = [&](const void *p) {
            return reinterpret_cast<const uint32_t *>(p != nullptr ? p : a.u)[row];
        };
        const uint32_t bits_t = at(a.temperature), bits_k = at(a.top_k), bits_p = at(a.top_p), bits_m = at(a.min_p),
                       bits_u = at(a.u);
        t = a.temperature != nullptr ? __uint_as_float(bits_t) : 1.0f;
        min_p = a.min_p != nullptr ? __uint_as_float(bits_m) : 0.0f;
        u = __uint_as_float(bits_u);
        const bool greedy = !(t > 0.0f);
        if (greedy) t = 0.0f;
        const int32_t k = a.top_k != nullptr ? static_cast<int32_t>(bits_k) : 0;
        // no weight reaches a min_p above 1: the first of the order alone
        top_k = greedy || min_p > 1.0f ? 1 : (k < 1 || k >= a.vocab ? 0 : k);
        const float p = a.top_p != nullptr ? __uint_as_float(bits_p) : 2.0f;
        top_p = greedy || !(p < 1.0f) ? 2.0f : p;
        if (top_p <= 0.0f) top_k = 1;
        if (top_k == 1) top_p = 2.0f;
    }
    __device__ __forceinline__ bool nucleus() const { return top_p < 1.0f; }
    // one logit needs no histogram, all of them neither
    __device__ __forceinline__ bool searched() const { return top_k > 1 || nucleus(); }
    // a small top_k is resolved among its collected logits alone
    __device__ __forceinline__ bool small_k() const { return top_k > 1 && top_k <= kListTopK; }
};

// s * g + c with the constant in scalar registers: the compiler's own choice
// for a polynomial, a multiply-add onto a copy of each constant, takes two more
// instructions a step.
__device__ __forceinline__ double fma_const(double s, double g, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(s), "v"(g), "s"(c));
    return d;
}

// Weights and bins of a row. A row with a logit of +infinity has no other
// tokens: with `lift`, +infinity is read as 0 and everything else as -infinity.
struct Scale {
    double max, rate, min_w;  // rate: log2(e) / T; min_w at the weights' scale
    float top, width;         // the maximum; bins per unit of distance from it
    int bits;
    bool lift;

    __device__ __forceinline__ Scale(const SampleArgs &a, const Filters &f, double rate, float2 range) : rate(rate) {
        lift = range.x == __builtin_inff();
        top = lift ? 0.0f : range.x;
        max = static_cast<double>(top);
        const float t = f.t > 0.0f ? f.t : 1.0f;
        bits = a.bits;
        min_w = ldexp(f.min_p > 0.0f ? static_cast<double>(f.min_p) : 0.0, bits);
        // the bins span the row, or as far down as weights matter
        const float span = lift ? 0.0f : fminf(fminf(top - range.y, 64.0f * t), 0x1.fffffep127f);
        width = span > 0.0f ? fminf((kBins - 1) / span, 0x1p100f) : 0.0f;
    }
    // A token's logit on the axis of the bins: bin b is [b, b + 1), the last
    // without an end; a larger logit never lies further.
    __device__ __forceinline__ float place(float x) const { return (top - x) * width; }
    __device__ __forceinline__ int bin(float x) const {
        return static_cast<int>(fminf(place(x), static_cast<float>(kBins - 1)));
    }
    // exp((x - max) / T) * 2^bits, by 2^y = 2^round(y) * 2^(y - round(y)), the
    // second factor by its Taylor series in fp64, ln(2)^k / k!: terms up to
    // the 11th leave 8.7e-15 of it at most (y - n = -1/2), and rate, the product
    // and the steps some 2^-53 of y and of it more, together under 2^-46 of the
    // largest weight: up to ten of the integers' own steps at 50 bits, half a
    // step at 45 and none at 0, the largest. 0 for -infinity and NaN.
    __device__ __forceinline__ double scaled(float x) const {
        constexpr double L1 = 0.69314718055994530942, L2 = L1 * L1, L4 = L2 * L2, L8 = L4 * L4;
        const double y = fmax((static_cast<double>(x) - max) * rate, -1000.0);
        const double n = __builtin_rint(y);
        const double r = y - n;
        double s = fma_const(r, L8 * L2 * L1 / 39916800, L8 * L2 / 3628800);
        s = fma_const(s, r, L8 * L1 / 362880);
        s = fma_const(s, r, L8 / 40320);
        s = fma_const(s, r, L4 * L2 * L1 / 5040);
        s = fma_const(s, r, L4 * L2 / 720);
        s = fma_const(s, r, L4 * L1 / 120);
        s = fma_const(s, r, L4 / 24);
        s = fma_const(s, r, L2 * L1 / 6);
        s = fma_const(s, r, L2 / 2);
        s = fma_const(s, r, L1);
        s = __builtin_fma(s, r, 1.0);
        return ldexp(s, static_cast<int>(n) + bits);
    }
    // Rounded to an integer: adding 2^52 leaves it in the low bits, under the
    // bits of 2^52 itself. A sum of n such takes those off once.
    __device__ __forceinline__ static uint64_t raised(double w) {
        return static_cast<uint64_t>(__double_as_longlong(w + 0x1p52));
    }
    static constexpr uint64_t kRaise = 0x4330000000000000ull;
    __device__ __forceinline__ static uint64_t fixed(double w) { return raised(w) - kRaise; }
    __device__ __forceinline__ uint64_t weight(float x) const { return fixed(scaled(x)); }
    // whether min_p keeps it
    __device__ __forceinline__ bool large(double w, float x) const { return w >= min_w || x == top; }
};

// Neither NaN nor -infinity.
__device__ __forceinline__ bool is_token(float x) { return x >= -0x1.fffffep127f; }

// 16 bytes of logits from any element address.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Logits [i, i + kN) of a row of n; those past the end become -infinity.
template <class T>
struct Logits {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    float x[kN];
    __device__ __forceinline__ void load(const T *row, int i, int n) {
        typedef T V __attribute__((ext_vector_type(kN)));
        if (i + kN <= n) {
            const u32x4 r = *reinterpret_cast<const u32x4_any *>(row + i);
            const V v = __builtin_bit_cast(V, r);
#pragma unroll
            for (int e = 0; e < kN; ++e) x[e] = static_cast<float>(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) x[e] = i + e < n ? static_cast<float>(row[i + e]) : -__builtin_inff();
        }
    }
    __device__ __forceinline__ void lift(bool lift) {
        if (lift) {
#pragma unroll
            for (int e = 0; e < kN; ++e) x[e] = x[e] == __builtin_inff() ? 0.0f : -__builtin_inff();
        }
    }
    __device__ __forceinline__ void load(const T *row, int i, int n, const Scale &sc) {
        load(row, i, n);
        lift(sc.lift);
    }
};

template <class T>
__device__ __forceinline__ const T *row_at(const SampleArgs &a, int row) {
    return static_cast<const T *>(a.logits) + static_cast<int64_t>(row) * a.stride;
}

// Across a wavefront, all of whose lanes are active, by DPP as
// wave_inclusive_scan does it: shuffles through LDS took four times as long.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint64_t dpp_move64(uint64_t v) {
    return static_cast<uint64_t>(dpp_move<CTRL, ROW_MASK>(static_cast<uint32_t>(v >> 32))) << 32 |
           dpp_move<CTRL, ROW_MASK>(static_cast<uint32_t>(v));
}
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
    v += dpp_move64<0x111, 0xf>(v);
    v += dpp_move64<0x112, 0xf>(v);
    v += dpp_move64<0x114, 0xf>(v);
    v += dpp_move64<0x118, 0xf>(v);
    v += dpp_move64<0x142, 0xa>(v);
    v += dpp_move64<0x143, 0xc>(v);
    return v;
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), kWave - 1));
}
__device__ __forceinline__ uint64_t last_lane64(uint64_t v) {
    return static_cast<uint64_t>(last_lane(static_cast<uint32_t>(v >> 32))) << 32 | last_lane(static_cast<uint32_t>(v));
}
__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) { return last_lane64(wave_scan64(v)); }
__device__ __forceinline__ uint32_t wave_sum32(uint32_t v) { return last_lane(wave_inclusive_scan<SumU32>(v)); }
// Of a workgroup's wavefront totals (up to 16, in LDS): the sum of those before
// wavefront w, and of all. A lane a total, for a loop over them would be read
// by every wavefront, one after another (1 us with sixteen).
template <int WAVES>
__device__ __forceinline__ uint64_t sum_before64(const unsigned long long *totals, int w, uint64_t &all) {
    const int lane = lane_id();
    uint64_t v = lane < WAVES ? totals[lane] : 0;
    v += dpp_move64<0x111, 0xf>(v);
    v += dpp_move64<0x112, 0xf>(v);
    v += dpp_move64<0x114, 0xf>(v);
    v += dpp_move64<0x118, 0xf>(v);
    const auto at = [&](int l) {
        return static_cast<uint64_t>(static_cast<uint32_t>(
                   __builtin_amdgcn_readlane(static_cast<int>(v >> 32), l))) << 32 |
               static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l));
    };
    all = at(WAVES - 1);
    return w == 0 ? 0 : at(w - 1);
}
template <int WAVES>
__device__ __forceinline__ uint32_t sum_before32(const uint32_t *totals, int w, uint32_t &all) {
    const int lane = lane_id();
    const uint32_t v = wave_inclusive_scan<SumU32>(lane < WAVES ? totals[lane] : 0u);
    all = last_lane(v);
    return w == 0 ? 0 : static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), w - 1));
}
// a lane without a source keeps its own
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float2 range_step(float2 r) {
    const auto from = [](float v) {
        const int own = __float_as_int(v);
        return __int_as_float(__builtin_amdgcn_update_dpp(own, own, CTRL, ROW_MASK, 0xf, false));
    };
    return {fmaxf(r.x, from(r.x)), fminf(r.y, from(r.y))};
}
__device__ __forceinline__ float2 wave_range(float2 r) {
    r = range_step<0x111, 0xf>(r);
    r = range_step<0x112, 0xf>(r);
    r = range_step<0x114, 0xf>(r);
    r = range_step<0x118, 0xf>(r);
    r = range_step<0x142, 0xa>(r);
    r = range_step<0x143, 0xc>(r);
    return {__uint_as_float(last_lane(__float_as_uint(r.x))), __uint_as_float(last_lane(__float_as_uint(r.y)))};
}

// Largest and smallest token logit of a row, by every wavefront for itself;
// -infinity as the largest: no token.
__device__ __forceinline__ float2 row_range(const SampleArgs &a, int row) {
    float2 r = {-__builtin_inff(), __builtin_inff()};
    for (int p = lane_id(); p < a.parts; p += kWave) {
        const float2 v = a.part_range[static_cast<int64_t>(row) * a.parts + p];
        r.x = fmaxf(r.x, v.x);
        r.y = fminf(r.y, v.y);
    }
    return wave_range(r);
}

// ---- range of each part; clears the rows' histograms and sets their state ----
template <class T>
__global__ __launch_bounds__(kPartBlock) void sample_max_kernel(SampleArgs a) {
    __shared__ float2 s_range[kPartBlock / kWave];
    const int row = blockIdx.y;
    const T *x = row_at<T>(a, row);
    using L = Logits<T>;
    const Filters f(a, row);
    if (a.splits > 1 && f.searched()) {
        for (int b = static_cast<int>(blockIdx.x * kPartBlock + threadIdx.x); b < kBins; b += gridDim.x * kPartBlock) {
            a.hist_mass[static_cast<int64_t>(row) * kBins + b] = 0;
            a.hist_count[static_cast<int64_t>(row) * kBins + b] = 0;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        RowState s{};
        s.extra = -1;
        s.rate = 1.4426950408889634 / (f.t > 0.0f ? static_cast<double>(f.t) : 1.0);
        if (f.top_k == 1) {  // the first of the order is in bin 0
            s.lo = s.hi = 0;
        } else {             // everything is kept, unless the histogram says otherwise
            s.lo = kBins;
            s.hi = kBins - 1;
        }
        a.state[row] = s;
    }
    for (int part = blockIdx.x; part < a.parts; part += gridDim.x) {
        float2 r = {-__builtin_inff(), __builtin_inff()};
        L v[kPartItems / L::kN];
#pragma unroll
        for (int j = 0; j < kPartItems / L::kN; ++j)
            v[j].load(x, part * kPart + (j * kPartBlock + static_cast<int>(threadIdx.x)) * L::kN, a.vocab);
#pragma unroll
        for (int j = 0; j < kPartItems / L::kN; ++j) {
#pragma unroll
            for (int e = 0; e < L::kN; ++e) {
                // NaN gives way in both; x * 0 is one for the infinities
                r.x = fmaxf(r.x, v[j].x[e]);
                r.y = fminf(r.y, __builtin_fmaf(v[j].x[e], 0.0f, v[j].x[e]));
            }
        }
        r = wave_range(r);
        __syncthreads();
        if (lane_id() == 0) s_range[threadIdx.x / kWave] = r;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kPartBlock / kWave; ++w) {
                r.x = fmaxf(r.x, s_range[w].x);
                r.y = fminf(r.y, s_range[w].y);
            }
            a.part_range[static_cast<int64_t>(row) * a.parts + part] = r;
        }
    }
}

// ---- counts and weights by bin, and the border bins ----
// The last 64, one a lane, take what needs no place: masked logits are many,
// and a wavefront's adds to one bin go one after another.
struct Hist {
    unsigned long long mass[kBins + kWave];
    uint32_t count[kBins + kWave];
};

__device__ __forceinline__ void hist_count(Hist &h, int bin) {
    __hip_atomic_fetch_add(&h.count[bin], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void hist_mass(Hist &h, int bin, uint64_t w) {
    __hip_atomic_fetch_add(&h.mass[bin], static_cast<unsigned long long>(w), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_WORKGROUP);
}

// Where a running sum over the bins reaches a goal.
struct Found {
    int bin;                    // -1: nowhere
    uint32_t before, count;     // keys in earlier bins, in this one
    uint64_t before_mass, mass;
};

template <int BLOCK>
struct FindShared {
    unsigned long long wave_mass[BLOCK / kWave];
    uint32_t wave_count[BLOCK / kWave];
    Found found[3];
};

// The first bin at whose end the count reaches `need` (found[0]) and the
// first at whose end the mass reaches target (found[1], found[2]), from
// `before` and `before_mass` at the first bin on. REVERSED: from the last bin down.
template <int BLOCK, bool REVERSED>
__device__ __forceinline__ void find_bins(const Hist &h, FindShared<BLOCK> &sh, uint32_t need, double target1,
                                          double target2, uint32_t before, uint64_t before_mass) {
    constexpr int kEach = kBins / BLOCK;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    uint32_t c[kEach], cs = 0;
    uint64_t m[kEach], ms = 0;
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
        const int b = static_cast<int>(threadIdx.x) * kEach + s;
        c[s] = h.count[REVERSED ? kBins - 1 - b : b];
        m[s] = h.mass[REVERSED ? kBins - 1 - b : b];
        cs += c[s];
        ms += m[s];
    }
    const uint32_t ci = wave_inclusive_scan<SumU32>(cs);
    const uint64_t mi = wave_scan64(ms);
    if (lane == kWave - 1) {
        sh.wave_count[w] = ci;
        sh.wave_mass[w] = mi;
    }
    if (threadIdx.x < 3) sh.found[threadIdx.x].bin = -1;
    __syncthreads();
    uint32_t cr = before + ci - cs;
    uint64_t mr = before_mass + mi - ms;
    constexpr int kWaves = BLOCK / kWave;
    uint32_t all_count;
    uint64_t all_mass;
    cr += sum_before32<kWaves>(sh.wave_count, w, all_count);
    mr += sum_before64<kWaves>(sh.wave_mass, w, all_mass);
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
        const int b = static_cast<int>(threadIdx.x) * kEach + s;
        const Found f{REVERSED ? kBins - 1 - b : b, cr, c[s], mr, m[s]};
        const double m0 = static_cast<double>(mr), m1 = static_cast<double>(mr + m[s]);
        // one bin only meets each of these
        if (cr < need && cr + c[s] >= need) sh.found[0] = f;
        if (m0 < target1 && m1 >= target1) sh.found[1] = f;
        if (m0 < target2 && m1 >= target2) sh.found[2] = f;
        cr += c[s];
        mr += m[s];
    }
    __syncthreads();
}

template <class T>
__global__ __launch_bounds__(kHistBlock) void sample_hist_kernel(SampleArgs a) {
    __shared__ Hist h;
    __shared__ FindShared<kHistBlock> sh;
    __shared__ bool s_last;
    const int row = blockIdx.y;
    const Filters f(a, row);
    if (!f.searched()) return;
    const Scale sc(a, f, a.state[row].rate, row_range(a, row));
    for (int b = threadIdx.x; b < kBins; b += kHistBlock) {
        h.mass[b] = 0;
        h.count[b] = 0;
    }
    __syncthreads();
    const T *x = row_at<T>(a, row);
    using L = Logits<T>;
    const bool counts = f.top_k > 0, masses = f.nucleus() && !f.small_k();
    const auto each = [&](auto counted, auto weighed) {
        constexpr int kStep = kHistBlock * L::kN, kDeep = 2;
        const int nowhere = kBins + lane_id();
        uint32_t deepest = 0;
        for (int i0 = (blockIdx.x * kHistBlock + static_cast<int>(threadIdx.x)) * L::kN; i0 < a.vocab;
             i0 += kDeep * a.splits * kStep) {
            L v[kDeep];
#pragma unroll
            for (int j = 0; j < kDeep; ++j) v[j].load(x, i0 + j * a.splits * kStep, a.vocab, sc);
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
#pragma unroll
                for (int e = 0; e < L::kN; ++e) {
                    const float xe = v[j].x[e];
                    const int b = is_token(xe) ? sc.bin(xe) : nowhere;
                    if (decltype(counted)::value) {  // the last bin's in a register
                        const bool last = b == kBins - 1;
                        deepest += last ? 1u : 0u;
                        hist_count(h, last ? nowhere : b);
                    }
                    if (decltype(weighed)::value) {
                        const uint64_t w = sc.weight(xe);
                        hist_mass(h, w != 0 ? b : nowhere, w);
                    }
                }
            }
        }
        if (decltype(counted)::value) {
            deepest = wave_sum32(deepest);
            if (lane_id() == 0 && deepest != 0)
                __hip_atomic_fetch_add(&h.count[kBins - 1], deepest, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    };
    if (counts && masses)
        each(std::true_type{}, std::true_type{});
    else if (counts)
        each(std::true_type{}, std::false_type{});
    else
        each(std::false_type{}, std::true_type{});
    __syncthreads();
    if (a.splits > 1) {
        unsigned long long *gm =
            reinterpret_cast<unsigned long long *>(a.hist_mass) + static_cast<int64_t>(row) * kBins;
        uint32_t *gc = a.hist_count + static_cast<int64_t>(row) * kBins;
        for (int b = threadIdx.x; b < kBins; b += kHistBlock) {
            if (counts && h.count[b] != 0)
                __hip_atomic_fetch_add(gc + b, h.count[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (masses && h.mass[b] != 0)
                __hip_atomic_fetch_add(gm + b, h.mass[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        // The workgroup that adds last finds the border bins. Everything it
        // reads was written by agent-scope atomics, which take effect beyond
        // the XCDs' own L2 caches: once each wavefront has waited for its own
        // to be acknowledged, agent-scope loads see them, and no cache has to
        // be written back (with release fences instead, 256 rows of 131,072
        // logits in 16 workgroups each took 641 us against 47).
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
            s_last = __hip_atomic_fetch_add(&a.state[row].done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                     gridDim.x - 1;
        __syncthreads();
        if (!s_last) return;
        // all loads in flight before the first is used: one after another
        // they took 2 us
        constexpr int kEach = kBins / kHistBlock;
        uint32_t c[kEach];
        unsigned long long m[kEach];
#pragma unroll
        for (int s = 0; s < kEach; ++s) {
            const int b = s * kHistBlock + static_cast<int>(threadIdx.x);
            c[s] = counts ? __hip_atomic_load(gc + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
            m[s] = masses ? __hip_atomic_load(gm + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
        }
#pragma unroll
        for (int s = 0; s < kEach; ++s) {
            const int b = s * kHistBlock + static_cast<int>(threadIdx.x);
            h.count[b] = c[s];
            h.mass[b] = m[s];
        }
        __syncthreads();
    }
    uint32_t n = 0;
    uint64_t total = 0;
    for (int b = threadIdx.x; b < kBins; b += kHistBlock) {
        n += h.count[b];
        total += h.mass[b];
    }
    n = wave_sum32(n);
    total = wave_sum64(total);
    if (lane_id() == 0) {
        sh.wave_count[threadIdx.x / kWave] = n;
        sh.wave_mass[threadIdx.x / kWave] = total;
    }
    __syncthreads();
    sum_before32<kHistBlock / kWave>(sh.wave_count, 0, n);
    sum_before64<kHistBlock / kWave>(sh.wave_mass, 0, total);
    __syncthreads();
    RowState *s = a.state + row;
    const uint32_t k = static_cast<uint32_t>(f.top_k);
    const double p = static_cast<double>(f.top_p);
    if (f.small_k()) {
        // all of the first top_k are collected (all there are, if fewer)
        find_bins<kHistBlock, false>(h, sh, k < n ? k : n, -1.0, -1.0, 0, 0);
        if (threadIdx.x == 0) {
            s->lo = 0;
            s->hi = sh.found[0].bin;
        }
    } else if (f.top_k > 0 && k < n) {
        find_bins<kHistBlock, false>(h, sh, k, -1.0, -1.0, 0, 0);
        const Found fk = sh.found[0];
        __syncthreads();
        if (!f.nucleus()) {
            if (threadIdx.x == 0) {
                s->lo = s->hi = fk.bin;
                s->count = fk.before;
            }
            return;
        }
        // top_p's border lies between those that the least and the most
        // weight of the first top_k would give
        const double low = p * static_cast<double>(fk.before_mass),
                     high = p * static_cast<double>(fk.before_mass + fk.mass);
        find_bins<kHistBlock, false>(h, sh, 0, low, high, 0, 0);
        if (threadIdx.x == 0) {
            const Found fl = sh.found[1], fh = sh.found[2];
            s->lo = fl.bin < 0 ? 0 : fl.bin;
            s->hi = fh.bin < 0 ? fk.bin : fh.bin;
            s->mass = fl.bin < 0 ? 0 : fl.before_mass;
            s->count = fl.bin < 0 ? 0 : fl.before;
            if (fk.bin > s->hi) {
                s->extra = fk.bin;
                s->extra_mass = fk.before_mass;
                s->extra_count = fk.before;
            }
        }
    } else if (f.nucleus()) {
        find_bins<kHistBlock, false>(h, sh, 0, p * static_cast<double>(total), -1.0, 0, 0);
        if (threadIdx.x == 0 && sh.found[1].bin >= 0) {
            s->lo = s->hi = sh.found[1].bin;
            s->mass = sh.found[1].before_mass;
            s->total = total;
        }
    }
}

// ---- kept weight of the better bins by part, and the logits of the border bins ----
// An entry of the list orders as the row does, from the largest down.
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int i) {
    return static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(i);
}

template <class T>
__global__ __launch_bounds__(kPartBlock) void sample_sum_kernel(SampleArgs a) {
    constexpr int kWaves = kPartBlock / kWave;
    __shared__ float s_x[kWaves][kPart / kWaves];
    __shared__ uint16_t s_i[kWaves][kPart / kWaves];
    __shared__ unsigned long long s_mass[kWaves];
    __shared__ uint32_t s_count[kWaves];
    const int row = blockIdx.y;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const T *x = row_at<T>(a, row);
    using L = Logits<T>;
    constexpr int kEach = kPartItems / L::kN;
    const Filters f(a, row);
    const Scale sc(a, f, a.state[row].rate, row_range(a, row));
    RowState *st = a.state + row;
    const int lo = st->lo, hi = st->hi, extra = st->extra;
    // No logit below `least` is kept or collected: those that are lie above
    // top - (deepest + 1) / width but for some roundings, which the added 2
    // covers; rounding the difference to fp32 keeps its order among logits.
    const int deepest = extra > hi ? extra : hi;
    constexpr float kLowest = -0x1.fffffep127f;
    const float least = lo >= kBins || deepest >= kBins - 1 || sc.width == 0.0f
                            ? kLowest
                            : fmaxf(sc.top - (static_cast<float>(deepest) + 2.0f) / sc.width, kLowest);
    for (int part = blockIdx.x; part < a.parts; part += gridDim.x) {
        L v[kEach];
        const int first = part * kPart + static_cast<int>(threadIdx.x) * L::kN;
#pragma unroll
        for (int j = 0; j < kEach; ++j) v[j].load(x, first + j * kPartBlock * L::kN, a.vocab, sc);
        uint64_t mass = 0;
        uint32_t count = 0;  // of the wavefront
        if (lo >= kBins) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
#pragma unroll
                for (int e = 0; e < L::kN; ++e) {
                    const float xe = v[j].x[e];
                    const double we = sc.scaled(xe);
                    const uint64_t keep = ballot(sc.large(we, xe)) & ballot(is_token(xe));
                    count += static_cast<uint32_t>(__builtin_popcountll(keep));
                    mass += (keep >> lane) & 1 ? Scale::fixed(we) : 0;
                }
            }
        } else {
            // what may be kept or collected is packed first, so that the rest
            // of the work runs on full wavefronts
            uint32_t packed = 0;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
#pragma unroll
                for (int e = 0; e < L::kN; ++e) {
                    const float xe = v[j].x[e];
                    const bool near = xe >= least;
                    const uint64_t mask = ballot(near);
                    if (mask == 0) continue;
                    if (near) {
                        const uint32_t at = packed + mbcnt64(mask);
                        s_x[w][at] = xe;
                        s_i[w][at] = static_cast<uint16_t>((j * kPartBlock + static_cast<int>(threadIdx.x)) * L::kN + e);
                    }
                    packed += static_cast<uint32_t>(__builtin_popcountll(mask));
                }
            }
            wave_lds_order();  // written by one lane, read by another
            // places in [0, kept) are kept, those in [kept, end) and [far, far_end)
            // collected; the last bin's end is a NaN, which nothing reaches
            const float kept = static_cast<float>(lo);
            const float end = hi >= kBins - 1 ? __builtin_nanf("") : static_cast<float>(hi + 1);
            const float far = extra < 0 ? __builtin_nanf("") : static_cast<float>(extra);
            const float far_end = extra >= kBins - 1 ? __builtin_nanf("") : far + 1.0f;
            for (uint32_t i0 = 0; i0 < packed; i0 += kWave) {
                const uint32_t i = i0 + lane;
                const bool here = i < packed;
                const float xe = here ? s_x[w][i] : -__builtin_inff();
                const float pl = sc.place(xe);
                if (lo > 0) {
                    const double we = sc.scaled(xe);
                    const bool keep = here && pl < kept && sc.large(we, xe);
                    mass += keep ? Scale::fixed(we) : 0;
                    count += static_cast<uint32_t>(__builtin_popcountll(ballot(keep)));
                }
                const bool list = here && ((pl >= kept && !(pl >= end)) || (pl >= far && !(pl >= far_end)));
                const uint64_t mask = ballot(list);
                if (mask != 0) {
                    uint32_t at = 0;
                    if (lane == 0)
                        at = __hip_atomic_fetch_add(&st->listed, static_cast<uint32_t>(__builtin_popcountll(mask)),
                                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    at = uniform(at) + mbcnt64(mask);
                    if (list && at < kList)
                        a.list[static_cast<int64_t>(row) * kList + at] = entry_of(key_of(xe), part * kPart + s_i[w][i]);
                }
            }
        }
        mass = wave_sum64(mass);
        __syncthreads();
        if (lane == 0) {
            s_mass[w] = mass;
            s_count[w] = count;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kWaves; ++i) {
                mass += s_mass[i];
                count += s_count[i];
            }
            a.part_mass[static_cast<int64_t>(row) * a.parts + part] = mass;
            a.part_count[static_cast<int64_t>(row) * a.parts + part] = count;
        }
    }
}

// ---- border and token ----
// A kept logit's weight; 0 and not counted for the others.
struct Border {
    uint32_t key, cut;  // smallest kept key, last index at which it is kept
    __device__ __forceinline__ uint64_t weight(const Scale &sc, float x, int i, bool &kept) const {
        const uint32_t k = key_of(x);
        kept = false;
        if (k == 0 || k < key || (k == key && static_cast<uint32_t>(i) > cut)) return 0;
        const double w = sc.scaled(x);
        kept = sc.large(w, x);
        return kept ? Scale::fixed(w) : 0;
    }
};

struct TokenShared {
    union {
        struct {
            __attribute__((aligned(16))) unsigned long long entry[kList];
        } list;
        Hist h;
    };
    FindShared<kTokenBlock> find;
    unsigned long long mass[kPartsMax];
    unsigned long long at_skip, at_end, goal, total;
    uint32_t count, cut;
    Border border;
    int part;
};

// The slow way, for a row whose border bins hold more logits than the list
// (equal or nearly equal logits in numbers): the border key digit by digit.
template <class T>
__device__ __forceinline__ void refine(const SampleArgs &a, const T *x, const Scale &sc, TokenShared &sh,
                                       bool weigh, uint32_t prefix, int shift, int width) {
    for (int b = threadIdx.x; b < kBins; b += kTokenBlock) {
        sh.h.mass[b] = 0;
        sh.h.count[b] = 0;
    }
    __syncthreads();
    using L = Logits<T>;
    for (int i = static_cast<int>(threadIdx.x) * L::kN; i < a.vocab; i += kTokenBlock * L::kN) {
        L v;
        v.load(x, i, a.vocab, sc);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) {
            const uint32_t k = key_of(v.x[e]);
            const bool mine = k != 0 && (shift + width >= 32 || k >> (shift + width) == prefix);
            const uint64_t all = ballot(mine);
            if (all == 0) continue;
            // the logits equal to the first lane's go in one add: this way is
            // taken for rows with many of the same
            const uint32_t k0 = static_cast<uint32_t>(
                __builtin_amdgcn_readlane(static_cast<int>(k), __builtin_ctzll(all)));
            const uint64_t same = ballot(mine && k == k0);
            const bool first = lane_id() == __builtin_ctzll(all);
            if (!mine || (k == k0 && !first)) continue;
            const uint32_t n = first ? static_cast<uint32_t>(__builtin_popcountll(same)) : 1u;
            const int b = static_cast<int>((k >> shift) & ((1u << width) - 1u));
            __hip_atomic_fetch_add(&sh.h.count[b], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            if (weigh) hist_mass(sh.h, b, n * sc.weight(v.x[e]));
        }
    }
    __syncthreads();
}

// The key at which the count reaches `need`, or the mass `target` (bin: the
// key; -1 where neither is reached).
template <class T>
__device__ __forceinline__ Found border_key(const SampleArgs &a, const T *x, const Scale &sc, TokenShared &sh,
                                            bool weigh, uint32_t need, double target) {
    const int which = need > 0 ? 0 : 1;
    uint32_t key = 0, before = 0;
    uint64_t before_mass = 0;
    Found f{};
    for (int level = 0; level < (sizeof(T) == 2 ? 2 : 3); ++level) {
        const int shift = level == 0 ? 21 : (level == 1 ? 10 : 0), width = level == 2 ? 10 : 11;
        refine(a, x, sc, sh, weigh, key, shift, width);
        find_bins<kTokenBlock, true>(sh.h, sh.find, need, target, -1.0, before, before_mass);
        f = sh.find.found[which];
        __syncthreads();
        if (f.bin < 0) return f;
        key = key << width | static_cast<uint32_t>(f.bin);
        before = f.before;
        before_mass = f.before_mass;
    }
    if (sizeof(T) == 2) key = key << 10 | ((key >> 21) != 0 ? 0u : 0x3ffu);  // the sign gives the rest
    f.bin = static_cast<int>(key);
    return f;
}

// The index of the `need`-th logit, in index order, with this key.
template <class T>
__device__ __forceinline__ uint32_t tie_index(const SampleArgs &a, const T *x, const Scale &sc, TokenShared &sh,
                                              uint32_t key, uint32_t need) {
    using L = Logits<T>;
    constexpr int kWaves = kTokenBlock / kWave;
    constexpr int kStep = kWave * L::kN;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int steps = (a.vocab + kStep - 1) / kStep;
    const int each = (steps + kWaves - 1) / kWaves;
    const int first = w * each, last = first + each < steps ? first + each : steps;
    uint32_t count = 0;
    for (int s = first; s < last; ++s) {
        L v;
        v.load(x, s * kStep + lane * L::kN, a.vocab, sc);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) count += key_of(v.x[e]) == key ? 1u : 0u;
    }
    count = wave_sum32(count);
    if (threadIdx.x == 0) sh.cut = kNoCut;
    if (lane == 0) sh.find.wave_count[w] = count;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += sh.find.wave_count[i];
    if (before < need && before + count >= need) {  // this wavefront holds it
        for (int s = first; s < last; ++s) {
            const int i = s * kStep + lane * L::kN;
            L v;
            v.load(x, i, a.vocab, sc);
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < L::kN; ++e) mine += key_of(v.x[e]) == key ? 1u : 0u;
            const uint32_t incl = wave_inclusive_scan<SumU32>(mine);
            uint32_t c = before + incl - mine;
            if (c < need && c + mine >= need) {
#pragma unroll
                for (int e = 0; e < L::kN; ++e) {
                    if (key_of(v.x[e]) == key && ++c == need) sh.cut = static_cast<uint32_t>(i + e);
                }
            }
            before += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(incl), kWave - 1));
            if (before >= need) break;
        }
    }
    __syncthreads();
    const uint32_t cut = sh.cut;
    __syncthreads();
    return cut;
}

template <class T>
__device__ __forceinline__ Border slow_border(const SampleArgs &a, const T *x, const Filters &f, const Scale &sc,
                                              TokenShared &sh) {
    Border out{1u, kNoCut};
    uint32_t ties = 0, have = 0;
    double all = -1.0;  // weight that top_k leaves
    if (f.top_k == 1) {
        out.key = key_of(sc.top);
        out.cut = tie_index(a, x, sc, sh, out.key, 1);
        return out;
    }
    if (f.top_k > 0) {
        const Found k = border_key(a, x, sc, sh, f.nucleus(), static_cast<uint32_t>(f.top_k), -1.0);
        if (k.bin != -1) {
            out.key = static_cast<uint32_t>(k.bin);
            ties = static_cast<uint32_t>(f.top_k) - k.before;
            have = k.count;
            all = static_cast<double>(k.before_mass + ties * sc.weight(value_of(out.key)));
        }
    }
    if (f.nucleus()) {
        if (all < 0.0) {  // all of the row's
            refine(a, x, sc, sh, true, 0, 21, 11);
            uint64_t m = 0;
            for (int b = threadIdx.x; b < kBins; b += kTokenBlock) m += sh.h.mass[b];
            m = wave_sum64(m);
            if (lane_id() == 0) sh.find.wave_mass[threadIdx.x / kWave] = m;
            __syncthreads();
            m = 0;
            for (int i = 0; i < kTokenBlock / kWave; ++i) m += sh.find.wave_mass[i];
            __syncthreads();
            all = static_cast<double>(m);
        }
        const double target = static_cast<double>(f.top_p) * all;
        const Found p = border_key(a, x, sc, sh, true, 0, target);
        if (p.bin != -1) {
            // ties j = 0, 1, ... are kept while before_mass + j * weight < target
            const uint32_t key = static_cast<uint32_t>(p.bin);
            const uint64_t wt = sc.weight(value_of(key));
            uint32_t j = p.count;
            if (wt != 0) {
                const double q = (target - static_cast<double>(p.before_mass)) / static_cast<double>(wt);
                j = q < static_cast<double>(p.count) ? static_cast<uint32_t>(q) : p.count;
                while (j > 0 && static_cast<double>(p.before_mass + (j - 1) * wt) >= target) --j;
                while (j < p.count && static_cast<double>(p.before_mass + j * wt) < target) ++j;
            }
            if (key != out.key || j < ties || ties == 0) {
                out.key = key;
                ties = j;
                have = p.count;
            }
        }
    }
    if (ties < have) out.cut = tie_index(a, x, sc, sh, out.key, ties);
    return out;
}

// Entries [0, n) of e from the largest down into out, for n2 <= 512: each
// entry's place is the number of larger ones, counted by kTokenBlock / n2
// threads together, two entries a read (n2 is a power of two of 32 at least, e
// filled up with 0).
__device__ __forceinline__ void rank_list(const unsigned long long *e, unsigned long long *out, int n, int n2) {
    typedef unsigned long long Pair __attribute__((ext_vector_type(2)));
    const Pair *pairs = reinterpret_cast<const Pair *>(e);
    const int lg = __builtin_ctz(kTokenBlock / n2);
    const int i = static_cast<int>(threadIdx.x) >> lg, part = static_cast<int>(threadIdx.x) & ((1 << lg) - 1);
    const unsigned long long mine = e[i];
    uint32_t place = 0;
#pragma unroll 4
    for (int j = part; j < (n + 1) / 2; j += 1 << lg) {
        const Pair v = pairs[j];
        place += (v[0] > mine ? 1u : 0u) + (v[1] > mine ? 1u : 0u);
    }
    for (int off = 1 << lg; off > 1; off >>= 1) place += __shfl_xor(place, off >> 1);
    if (part == 0 && i < n) out[place] = mine;
    __syncthreads();
}

// Sorts n2 entries (a power of two, 4 at least) from the largest down: bitonic
// merges, two distances d and d / 2 at a time on four entries in registers.
// A wavefront's entries are 256 of its own while d is at most 128, so only
// the longer distances need the workgroup's barriers.
__device__ __forceinline__ void order_pair(unsigned long long &u, unsigned long long &v, bool down) {
    if ((u < v) == down) {
        const unsigned long long x = u;
        u = v;
        v = x;
    }
}
__device__ __forceinline__ void sort_list(unsigned long long *e, int n2) {
    const int quads = n2 / 4;
    for (int size = 2; size <= n2; size <<= 1) {
        int d = size >> 1;
        // an odd number of distances: the first alone
        const bool odd = (__builtin_ctz(static_cast<unsigned>(size)) & 1) != 0;
        for (bool single = odd; d > 0; d >>= single ? 1 : 2, single = false) {
            const int h = single ? d : d >> 1;
            for (int t = threadIdx.x; t < quads; t += kTokenBlock) {
                if (single) {  // pairs 2t and 2t + 1 of the distance
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int p = 2 * t + s, i = 2 * p - (p & (d - 1));
                        unsigned long long u = e[i], v = e[i + d];
                        order_pair(u, v, (i & size) == 0);
                        e[i] = u;
                        e[i + d] = v;
                    }
                } else {
                    const int i = 4 * t - 3 * (t & (h - 1));
                    const bool down = (i & size) == 0;
                    unsigned long long q0 = e[i], q1 = e[i + h], q2 = e[i + d], q3 = e[i + d + h];
                    order_pair(q0, q2, down);
                    order_pair(q1, q3, down);
                    order_pair(q0, q1, down);
                    order_pair(q2, q3, down);
                    e[i] = q0;
                    e[i + h] = q1;
                    e[i + d] = q2;
                    e[i + d + h] = q3;
                }
            }
            // the next step's first distance
            const int left = single ? d >> 1 : d >> 2;
            const int next = left > 0 ? left : size;
            if (d > 2 * kWave || next > 2 * kWave || (left == 0 && size == n2)) {
                __syncthreads();
            } else {
                wave_lds_order();
            }
        }
    }
}

template <class T>
__global__ __launch_bounds__(kTokenBlock) void sample_token_kernel(SampleArgs a) {
    __shared__ TokenShared sh;
    constexpr int kWaves = kTokenBlock / kWave;
    const int row = blockIdx.x;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int64_t base = static_cast<int64_t>(row) * a.parts;
    // all first loads before anything waits for one; a part to a thread
    const RowState st = a.state[row];
    const bool has_part = static_cast<int>(threadIdx.x) < a.parts;
    const uint64_t part_mass = has_part ? a.part_mass[base + threadIdx.x] : 0;
    uint32_t count = has_part ? a.part_count[base + threadIdx.x] : 0;
    const uint64_t *list = a.list + static_cast<int64_t>(row) * kList;
    const uint64_t first_entry = list[threadIdx.x];  // used where it has been written
    const Filters f(a, row);
    const float2 range = row_range(a, row);
    if (range.x == -__builtin_inff()) {
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.kept != nullptr) a.kept[row] = 0;
            if (a.logprobs != nullptr) a.logprobs[row] = -__builtin_inff();
        }
        return;
    }
    const Scale sc(a, f, st.rate, range);
    const T *x = row_at<T>(a, row);
    Border border{1u, kNoCut};
    if (has_part) sh.mass[threadIdx.x] = part_mass;
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    if (st.listed > kList) {
        border = slow_border(a, x, f, sc, sh);
        // the parts' sums again, with the border known
        count = 0;
        for (int p = w; p < a.parts; p += kWaves) {
            using L = Logits<T>;
            uint64_t mass = 0;
            for (int i = p * kPart + lane * L::kN; i < a.vocab && i < (p + 1) * kPart; i += kWave * L::kN) {
                L v;
                v.load(x, i, a.vocab, sc);
#pragma unroll
                for (int e = 0; e < L::kN; ++e) {
                    bool kept;
                    mass += border.weight(sc, v.x[e], i + e, kept);
                    count += kept ? 1u : 0u;
                }
            }
            mass = wave_sum64(mass);
            if (lane == 0) sh.mass[p] = mass;
        }
        __syncthreads();
    } else if (st.lo < kBins) {
        // the collected logits in order; those of [lo, hi] come first
        const int n = static_cast<int>(st.listed);
        int n2 = 32;
        while (n2 < n) n2 <<= 1;
        unsigned long long *sorted = sh.list.entry;
        sorted[threadIdx.x] = static_cast<int>(threadIdx.x) < n ? first_entry : 0ull;
        for (int i = threadIdx.x + kTokenBlock; i < n2; i += kTokenBlock) sorted[i] = i < n ? list[i] : 0ull;
        __syncthreads();
        if (n2 <= 512) {  // by the squares of n: 200 entries 1.2 us against 6 by merges, 512 as long
            sorted += kList / 2;
            rank_list(sh.list.entry, sorted, n, n2);
        } else {
            sort_list(sorted, n2);
        }
        // each thread's consecutive entries, their weights and the running
        // sum; n1 of all entries lie in [lo, hi], the rest in the extra bin
        constexpr int kEach = kList / kTokenBlock;
        const int each = n <= kTokenBlock ? 1 : kEach;
        unsigned long long entry[kEach];
        uint64_t we[kEach], ms = 0;
        double full[kEach];
        uint32_t mine = 0;
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const int i = static_cast<int>(threadIdx.x) * each + q;
            entry[q] = 0;
            full[q] = 0.0;
            we[q] = 0;
            if (q < each && i < n) {
                entry[q] = sorted[i];
                const float xe = value_of(static_cast<uint32_t>(entry[q] >> 32));
                full[q] = sc.scaled(xe);
                we[q] = Scale::fixed(full[q]);
                ms += we[q];
                mine += sc.bin(xe) <= st.hi ? 1u : 0u;
            }
        }
        // wavefronts without entries leave the work to the others
        const bool busy = w * kWave * each < n;
        uint64_t mi = 0;
        if (busy) {
            mi = wave_scan64(ms);
            mine = wave_sum32(mine);
        }
        if (lane == kWave - 1) {
            sh.find.wave_mass[w] = mi;
            sh.find.wave_count[w] = mine;
        }
        __syncthreads();
        uint64_t run = mi - ms, all_mass;
        uint32_t n1;
        run += sum_before64<kWaves>(sh.find.wave_mass, w, all_mass);
        sum_before32<kWaves>(sh.find.wave_count, 0, n1);
        // nk: the entries of [lo, hi] that top_k leaves; the first top_k end
        // before entry `end`, and their weight is `from` and that of the
        // entries from `skip` on
        uint32_t nk = n1, skip = 0, end = n1;
        uint64_t from = st.mass;
        if (f.top_k > 0 && st.total == 0) {
            if (st.extra >= 0) {
                const uint32_t more = static_cast<uint32_t>(f.top_k) - st.extra_count;
                skip = n1;
                end = n1 + more < static_cast<uint32_t>(n) ? n1 + more : static_cast<uint32_t>(n);
                from = st.extra_mass;
            } else {
                const uint32_t more = static_cast<uint32_t>(f.top_k) - st.count;
                nk = more < n1 ? more : n1;
                end = nk;
            }
        }
        // running sums at skip and end, by the threads that hold the entries before them
        if (busy) {
            uint64_t at = run;
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const uint32_t i = threadIdx.x * each + q + 1;
                at += we[q];
                if (q < each && i == skip) sh.at_skip = at;
                if (q < each && i == end) sh.at_end = at;
            }
        }
        if (threadIdx.x == 0) {
            if (skip == 0) sh.at_skip = 0;
            if (end == 0) sh.at_end = 0;
            sh.border = Border{n > 0 ? static_cast<uint32_t>(sorted[0] >> 32) + 1u : 1u, kNoCut};  // nothing of the list
        }
        __syncthreads();
        const uint64_t all = st.total != 0 ? st.total : from + (sh.at_end - sh.at_skip);
        const double target = f.nucleus() ? static_cast<double>(f.top_p) * static_cast<double>(all) : __builtin_inf();
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            if (!busy || q >= each) continue;
            const uint32_t i = threadIdx.x * each + q;
            const bool keep = i < nk && static_cast<double>(st.mass + run) < target;
            run += we[q];
            if (!keep) continue;
            const uint32_t index = ~static_cast<uint32_t>(entry[q]);
            if (sc.large(full[q], value_of(static_cast<uint32_t>(entry[q] >> 32)))) {
                __hip_atomic_fetch_add(&sh.mass[index >> kPartLg], static_cast<unsigned long long>(we[q]),
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                ++count;
            }
            // the last kept entry is the border
            if (!(i + 1 < nk && static_cast<double>(st.mass + run) < target))
                sh.border = Border{static_cast<uint32_t>(entry[q] >> 32), index};
        }
        __syncthreads();
        border = sh.border;
    }
    // the part in which the running weight passes the goal
    if (ballot(count != 0) != 0) {
        count = wave_sum32(count);
        if (lane == 0) __hip_atomic_fetch_add(&sh.count, count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    if (w == 0) {
        uint64_t total = 0;
        for (int p = lane; p < a.parts; p += kWave) total += sh.mass[p];
        total = wave_sum64(total);
        float u = f.u > 0.0f ? f.u : 0.0f;
        u = u < 0x1.fffffep-1f ? u : 0x1.fffffep-1f;
        const uint64_t goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
        uint64_t before = 0;
        for (int p0 = 0; p0 < a.parts; p0 += kWave) {
            const uint64_t m = p0 + lane < a.parts ? sh.mass[p0 + lane] : 0;
            const uint64_t incl = wave_scan64(m);
            const uint64_t hit = ballot(before + incl > goal);
            if (hit != 0) {
                const int l = __builtin_ctzll(hit);
                if (lane == l) {
                    sh.part = p0 + l;
                    sh.goal = goal - (before + incl - m);  // what is left to pass in the part
                    sh.total = total;
                }
                break;
            }
            before += last_lane64(incl);
        }
        if (lane == 0 && a.kept != nullptr) a.kept[row] = static_cast<int32_t>(sh.count);
    }
    __syncthreads();
    // each thread takes consecutive logits of the part
    constexpr int kEach = kPart / kTokenBlock;
    const uint64_t goal = sh.goal;
    const int first = sh.part * kPart + static_cast<int>(threadIdx.x) * kEach;
    float v[kEach];
    uint64_t we[kEach], ms = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        bool kept;
        v[e] = first + e < a.vocab ? static_cast<float>(x[first + e]) : -__builtin_inff();
        if (sc.lift) v[e] = v[e] == __builtin_inff() ? 0.0f : -__builtin_inff();
        we[e] = border.weight(sc, v[e], first + e, kept);
        ms += we[e];
    }
    const uint64_t incl = wave_scan64(ms);
    if (lane == kWave - 1) sh.find.wave_mass[w] = incl;
    __syncthreads();
    uint64_t all_mass;
    const uint64_t before = sum_before64<kWaves>(sh.find.wave_mass, w, all_mass);
    uint64_t run = before + incl - ms;
    if (run <= goal && run + ms > goal) {
        int at = -1;
        float chosen = 0.0f;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            run += we[e];
            if (at < 0 && run > goal) {
                at = first + e;
                chosen = v[e];
            }
        }
        a.tokens[row] = at;
        if (a.logprobs != nullptr) {
            const double z = (static_cast<double>(chosen) - sc.max) * (sc.rate / 1.4426950408889634);
            a.logprobs[row] = static_cast<float>(z - log(ldexp(static_cast<double>(sh.total), -sc.bits)));
        }
    }
}

// ============================================================ host side ---
struct SamplePlan {
    int64_t parts;
    size_t list, hist_mass, part_mass, part_range, state, hist_count, part_count, bytes;  // offsets
};

bool sample_sizes_ok(int64_t rows, int64_t vocab) {
    // rows are a grid's second dimension
    return rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= kVocabMax;
}

SamplePlan sample_plan(int64_t rows, int64_t vocab) {
    SamplePlan p{};
    p.parts = (vocab + kPart - 1) / kPart;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 15) & ~size_t{15};
        return here;
    };
    const size_t r = static_cast<size_t>(rows), g = static_cast<size_t>(p.parts);
    p.list = take(r * kList * 8);
    p.hist_mass = take(r * kBins * 8);
    p.hist_count = take(r * kBins * 4);
    p.part_mass = take(r * g * 8);
    p.part_range = take(r * g * 8);
    p.part_count = take(r * g * 4);
    p.state = take(r * sizeof(RowState));
    p.bytes = at;
    return p;
}

template <class T>
int sample_launch(const SampleArgs &a, int64_t rows, bool searched, hipStream_t s) {
    const unsigned r = static_cast<unsigned>(rows);
    // up to 4096 workgroups, each with several parts of a row where there are
    // more (sums of 256 rows of 131,072: 2048, 4096, 8192 workgroups 35, 30, 32 us)
    const int64_t each = (static_cast<int64_t>(a.parts) * rows + 4095) / 4096;
    const dim3 parts(static_cast<unsigned>((a.parts + each - 1) / each), r);
    hipLaunchKernelGGL((sample_max_kernel<T>), parts, dim3(kPartBlock), 0, s, a);
    SSC_TRY(launched());
    if (searched) {
        hipLaunchKernelGGL((sample_hist_kernel<T>), dim3(a.splits, r), dim3(kHistBlock), 0, s, a);
        SSC_TRY(launched());
    }
    hipLaunchKernelGGL((sample_sum_kernel<T>), parts, dim3(kPartBlock), 0, s, a);
    SSC_TRY(launched());
    hipLaunchKernelGGL((sample_token_kernel<T>), dim3(r), dim3(kTokenBlock), 0, s, a);
    return launched();
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

size_t ssc_sample_scratch_bytes(int64_t rows, int64_t vocab) {
    return sample_sizes_ok(rows, vocab) ? sample_plan(rows, vocab).bytes : 0;
}

int ssc_sample_rows(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride, const float *u,
                    const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                    int32_t *tokens, int32_t *kept, float *logprobs, void *scratch, size_t scratch_bytes,
                    void *stream) {
    if (dtype != SSC_F32 && dtype != SSC_BF16 && dtype != SSC_F16) return SSC_ERR_ARG;
    if (rows < 0 || vocab < 1 || stride < vocab) return SSC_ERR_ARG;
    if (!sample_sizes_ok(rows, vocab) || stride > (int64_t{1} << 40)) return SSC_ERR_SIZE;
    if (rows > 0 && (logits == nullptr || u == nullptr || tokens == nullptr)) return SSC_ERR_ARG;
    const size_t es = dtype == SSC_F32 ? 4 : 2;
    if (!aligned(logits, es) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(kept, 4) ||
        !aligned(logprobs, 4))
        return SSC_ERR_ARG;
    const SamplePlan p = sample_plan(rows, vocab);
    if (p.bytes > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < p.bytes))
        return SSC_ERR_SCRATCH;
    const size_t each = static_cast<size_t>(rows) * 4;
    const Span written[] = {{tokens, each}, {kept, each}, {logprobs, each}, {scratch, p.bytes}};
    const size_t extent = rows > 0 ? (static_cast<size_t>(rows - 1) * stride + vocab) * es : 0;
    const Span read[] = {{logits, extent}, {u, each}, {temperature, each}, {top_k, each}, {top_p, each}, {min_p, each}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &w : written)
        for (const Span &r : read)
            if (overlap(w.p, w.bytes, r.p, r.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (rows == 0) return SSC_OK;
    SampleArgs a{};
    a.logits = logits;
    a.stride = stride;
    a.vocab = static_cast<int>(vocab);
    a.parts = static_cast<int>(p.parts);
    int len = 0;
    while (vocab >> len) ++len;
    a.bits = 62 - len < 50 ? 62 - len : 50;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.kept = kept;
    a.logprobs = logprobs;
    char *base = static_cast<char *>(scratch);
    a.part_range = reinterpret_cast<float2 *>(base + p.part_range);
    a.part_mass = reinterpret_cast<uint64_t *>(base + p.part_mass);
    a.part_count = reinterpret_cast<uint32_t *>(base + p.part_count);
    a.state = reinterpret_cast<RowState *>(base + p.state);
    a.list = reinterpret_cast<uint64_t *>(base + p.list);
    // A histogram only where a row may ask for one. A workgroup adds its 2048
    // bins to the row's by atomics, so a split costs as much as some thousand
    // logits: rows are split until there are two workgroups to a compute unit
    // or parts are of 8192 logits, and into parts of at most 32,768 in any
    // case, since rows differ in work. bf16, top_k of 50, top_p of 0.9, us:
    //   part                1 x 131,072   64 x 131,072   256 x 131,072   1 x 4,194,304
    //   4096                7.7, 9.2      21.1, 34.6     75, 119         33, 38
    //   8192                7.7, 9.2      15.3, 23.2     41, 65          21, 25
    //   16,384              8.5, 11.2     11.9, 18.0     28, 49          17, 21
    //   32,768              9.1, 14.7     11.0, 18.8     23, 44          16, 22
    const bool searched = top_k != nullptr || top_p != nullptr;
    a.splits = 1;
    if (searched) {
        const int64_t most = (vocab + kHistPart - 1) / kHistPart;
        while (a.splits < most && (a.splits * rows < 512 || vocab > int64_t{kHistMost} * a.splits)) ++a.splits;
        a.hist_mass = reinterpret_cast<uint64_t *>(base + p.hist_mass);
        a.hist_count = reinterpret_cast<uint32_t *>(base + p.hist_count);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case SSC_F32: return sample_launch<float>(a, rows, searched, s);
    case SSC_BF16: return sample_launch<__bf16>(a, rows, searched, s);
    default: return sample_launch<_Float16>(a, rows, searched, s);
    }
}

}  // extern "C"
