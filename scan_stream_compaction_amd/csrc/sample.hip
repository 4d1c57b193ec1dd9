// The next token of a row of logits, from a given random number, under
// temperature, top-k, top-p and min-p: HIP kernels for MI355X (gfx950) and
// their part of the C ABI in include/ssc.h.
//
// Every filter keeps a prefix of the row in the order (logit descending,
// index ascending), so the kept set is {key > t} and the ties {key = t} up to
// an index, with `key` the logit's bits as an ordered integer. No row is
// sorted: the border t is found digit by digit in histograms of the keys
// (11 bits each: two steps for 16-bit logits, three for fp32) that hold each
// bin's count and weight, which is also what makes it exact. The token is then
// the first index at which the running kept weight exceeds u times its sum:
// a selection by a scan, over the sums of parts of the row and then inside
// one part.
//
// Weights exp((x - max) / T) are computed in fp64 and held as integers with
// 62 - bits(vocab) fractional bits (at most 50): integer sums do not depend
// on their order, so rows may be split and added with atomics, and a call
// repeats bit for bit.
//
// Launches: row maxima; histograms; borders; kept weight of each part; token.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssc.h"
#include "ssc_device.h"
#include "ssc_host.h"

namespace ssc {
namespace {

constexpr int kPart = 4096;           // logits of a part
constexpr int kPartBlock = 256;
constexpr int kPartItems = kPart / kPartBlock;
constexpr int kHistPart = 16384;      // logits a workgroup adds to its row's histogram
constexpr int kHistBlock = 512;
constexpr int kBins = 2048;
constexpr int kBorderBlock = 1024;
constexpr uint32_t kNoCut = 0xffffffffu;

// What the border search of a row leaves for the later launches.
struct RowState {
    uint32_t border;  // smallest kept key
    uint32_t cut;     // last index at which that key is kept
};

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int vocab, parts, bits;  // bits: fractional bits of a weight
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens, *kept;
    float *logprobs;
    // scratch, per row: part maxima (keys), part sums, histogram, state
    uint32_t *part_max;      // [rows][parts]
    uint64_t *part_mass;     // [rows][parts]
    uint32_t *part_count;    // [rows][parts]
    uint64_t *hist_mass;     // [rows][kBins]
    uint32_t *hist_count;    // [rows][kBins]
    RowState *state;         // [rows]
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

// A row's settings, with what is out of range put in its place.
struct Settings {
    double inv_t, max, scale, min_w;
    float top_p;   // 2: off
    int32_t top_k;  // 0: off
    bool max_inf;

    __device__ __forceinline__ Settings(const SampleArgs &a, int row, uint32_t max_key) {
        const float t = a.temperature != nullptr ? a.temperature[row] : 1.0f;
        const bool greedy = !(t > 0.0f);
        inv_t = greedy ? 1.0 : 1.0 / static_cast<double>(t);
        const float m = value_of(max_key);
        max_inf = m == __builtin_inff();
        max = max_inf ? 0.0 : static_cast<double>(m);
        scale = static_cast<double>(uint64_t{1} << a.bits);
        const float mp = a.min_p != nullptr ? a.min_p[row] : 0.0f;
        min_w = mp > 1.0f ? 1.0 : (mp > 0.0f ? static_cast<double>(mp) : 0.0);
        const int32_t k = a.top_k != nullptr ? a.top_k[row] : 0;
        top_k = greedy ? 1 : (k < 1 || k >= a.vocab ? 0 : k);
        const float p = a.top_p != nullptr ? a.top_p[row] : 2.0f;
        top_p = greedy || !(p < 1.0f) ? 2.0f : p;
        if (top_p <= 0.0f) {
            top_p = 2.0f;
            top_k = 1;
        }
    }
    // exp((x - max) / T) of a logit that is a token
    __device__ __forceinline__ double weight(float x) const {
        if (max_inf) return x == __builtin_inff() ? 1.0 : 0.0;
        return exp((static_cast<double>(x) - max) * inv_t);
    }
    // ... as an integer: adding 2^52 leaves the rounded value in the low bits
    __device__ __forceinline__ uint64_t fixed(double w) const {
        return static_cast<uint64_t>(__double_as_longlong(__builtin_fma(w, scale, 0x1p52))) & ((uint64_t{1} << 52) - 1);
    }
};

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
};

template <class T>
__device__ __forceinline__ const T *row_at(const SampleArgs &a, int row) {
    return static_cast<const T *>(a.logits) + static_cast<int64_t>(row) * a.stride;
}

__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(static_cast<unsigned long long>(v), off);
    return v;
}
__device__ __forceinline__ uint32_t wave_max32(uint32_t v) {
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o = __shfl_xor(v, off);
        v = v > o ? v : o;
    }
    return v;
}
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
    const int lane = lane_id();
    for (int off = 1; off < kWave; off <<= 1) {
        const uint64_t o = __shfl_up(static_cast<unsigned long long>(v), off);
        v += lane >= off ? o : 0;
    }
    return v;
}

// The row's largest key, by every wavefront for itself.
__device__ __forceinline__ uint32_t row_max(const SampleArgs &a, int row) {
    uint32_t m = 0;
    for (int p = lane_id(); p < a.parts; p += kWave) {
        const uint32_t v = a.part_max[static_cast<int64_t>(row) * a.parts + p];
        m = m > v ? m : v;
    }
    return uniform(wave_max32(m));
}

// ---- largest key of each part; clears the rows' histograms ----
template <class T>
__global__ __launch_bounds__(kPartBlock) void sample_max_kernel(SampleArgs a) {
    __shared__ uint32_t s_max[kPartBlock / kWave];
    const int row = blockIdx.y, part = blockIdx.x;
    const T *x = row_at<T>(a, row);
    using L = Logits<T>;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPartItems / L::kN; ++j) {
        const int i = part * kPart + (j * kPartBlock + static_cast<int>(threadIdx.x)) * L::kN;
        if (i >= a.vocab) continue;
        L v;
        v.load(x, i, a.vocab);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) {
            const uint32_t k = key_of(v.x[e]);
            m = m > k ? m : k;
        }
    }
    m = wave_max32(m);
    if (lane_id() == 0) s_max[threadIdx.x / kWave] = m;
    if (a.hist_count != nullptr) {
        for (int b = part * kPartBlock + static_cast<int>(threadIdx.x); b < kBins; b += a.parts * kPartBlock) {
            a.hist_mass[static_cast<int64_t>(row) * kBins + b] = 0;
            a.hist_count[static_cast<int64_t>(row) * kBins + b] = 0;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kPartBlock / kWave; ++w) m = m > s_max[w] ? m : s_max[w];
        a.part_max[static_cast<int64_t>(row) * a.parts + part] = m;
    }
}

// ---- counts and weights by the keys' top 11 bits ----
struct Hist {
    unsigned long long mass[kBins];
    uint32_t count[kBins];
};

__device__ __forceinline__ void hist_add(Hist &h, uint32_t bin, uint64_t w) {
    __hip_atomic_fetch_add(&h.count[bin], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    if (w != 0)
        __hip_atomic_fetch_add(&h.mass[bin], static_cast<unsigned long long>(w), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
}

template <class T>
__global__ __launch_bounds__(kHistBlock) void sample_hist_kernel(SampleArgs a) {
    __shared__ Hist h;
    const int row = blockIdx.y;
    const uint32_t max_key = row_max(a, row);
    const Settings st(a, row, max_key);
    // the largest logit alone needs no histogram
    if (max_key == 0 || st.top_k == 1 || (st.top_k == 0 && st.top_p > 1.0f)) return;
    for (int b = threadIdx.x; b < kBins; b += kHistBlock) {
        h.mass[b] = 0;
        h.count[b] = 0;
    }
    __syncthreads();
    const T *x = row_at<T>(a, row);
    using L = Logits<T>;
    const int begin = blockIdx.x * kHistPart;
    const int end = a.vocab - begin < kHistPart ? a.vocab : begin + kHistPart;
    for (int i = begin + static_cast<int>(threadIdx.x) * L::kN; i < end; i += kHistBlock * L::kN) {
        L v;
        v.load(x, i, a.vocab);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) {
            const uint32_t k = key_of(v.x[e]);
            if (k != 0) hist_add(h, k >> 21, st.fixed(st.weight(v.x[e])));
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kHistBlock) {
        if (h.count[b] == 0) continue;
        __hip_atomic_fetch_add(a.hist_count + static_cast<int64_t>(row) * kBins + b, h.count[b], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        if (h.mass[b] != 0)
            __hip_atomic_fetch_add(reinterpret_cast<unsigned long long *>(a.hist_mass) +
                                       static_cast<int64_t>(row) * kBins + b,
                                   h.mass[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// ---- the border of a row ----
struct Found {
    uint32_t bin, count;          // the border's bin, its keys
    uint32_t above;               // keys in larger bins
    unsigned long long above_mass, mass;
};

struct BorderShared {
    Hist h;
    unsigned long long wave_mass[kBorderBlock / kWave];
    uint32_t wave_count[kBorderBlock / kWave];
    Found found;
    uint32_t cut;
    unsigned long long total_mass;
};

// The bin, from the largest down, that holds the `need`-th key (by count) or
// in which the mass before a key reaches `target` (by mass); `before` and
// `before_mass` lie above all bins. The last bin with keys stands where none does.
__device__ __forceinline__ Found find_bin(BorderShared &sh, bool by_count, uint32_t need, double target,
                                          uint32_t before, uint64_t before_mass) {
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int b0 = kBins - 1 - 2 * static_cast<int>(threadIdx.x), b1 = b0 - 1;
    const uint32_t c0 = sh.h.count[b0], c1 = sh.h.count[b1];
    const uint64_t m0 = sh.h.mass[b0], m1 = sh.h.mass[b1];
    const uint32_t ci = wave_inclusive_scan<SumU32>(c0 + c1);
    const uint64_t mi = wave_scan64(m0 + m1);
    if (lane == kWave - 1) {
        sh.wave_count[w] = ci;
        sh.wave_mass[w] = mi;
    }
    __syncthreads();
    uint32_t c = before + ci - c0 - c1;
    uint64_t m = before_mass + mi - m0 - m1;
    for (int i = 0; i < w; ++i) {
        c += sh.wave_count[i];
        m += sh.wave_mass[i];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t cc = s == 0 ? c0 : c1;
        const uint64_t mm = s == 0 ? m0 : m1;
        // one bin only meets this: the first whose end reaches the goal
        const bool start = by_count ? c < need : static_cast<double>(m) < target;
        const bool stop = by_count ? c + cc >= need : static_cast<double>(m + mm) >= target;
        if (cc != 0 && start && stop) {
            sh.found.bin = static_cast<uint32_t>(s == 0 ? b0 : b1);
            sh.found.count = cc;
            sh.found.above = c;
            sh.found.above_mass = m;
            sh.found.mass = mm;
        }
        c += cc;
        m += mm;
    }
    __syncthreads();
    const Found f = sh.found;
    __syncthreads();
    return f;
}

// Histogram of the keys whose bits above `shift + width` equal `prefix`, by
// the `width` bits at `shift`.
template <class T>
__device__ __forceinline__ void refine(const SampleArgs &a, const T *x, const Settings &st, BorderShared &sh,
                                       uint32_t prefix, int shift, int width) {
    for (int b = threadIdx.x; b < kBins; b += kBorderBlock) {
        sh.h.mass[b] = 0;
        sh.h.count[b] = 0;
    }
    __syncthreads();
    using L = Logits<T>;
    for (int i = static_cast<int>(threadIdx.x) * L::kN; i < a.vocab; i += kBorderBlock * L::kN) {
        L v;
        v.load(x, i, a.vocab);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) {
            const uint32_t k = key_of(v.x[e]);
            if (k >> (shift + width) == prefix && k != 0)
                hist_add(sh.h, (k >> shift) & ((1u << width) - 1u), st.fixed(st.weight(v.x[e])));
        }
    }
    __syncthreads();
}

// The border key of one filter: where the `need`-th key, or the mass
// `target`, is reached.
template <class T>
__device__ __forceinline__ Found border_key(const SampleArgs &a, int row, const T *x, const Settings &st,
                                            BorderShared &sh, bool by_count, uint32_t need, double target) {
    for (int b = threadIdx.x; b < kBins; b += kBorderBlock) {
        sh.h.mass[b] = a.hist_mass[static_cast<int64_t>(row) * kBins + b];
        sh.h.count[b] = a.hist_count[static_cast<int64_t>(row) * kBins + b];
    }
    __syncthreads();
    Found f = find_bin(sh, by_count, need, target, 0, 0);
    uint32_t key = f.bin;
    refine(a, x, st, sh, key, 10, 11);
    f = find_bin(sh, by_count, need, target, f.above, f.above_mass);
    key = key << 11 | f.bin;
    if (sizeof(T) == 4) {
        refine(a, x, st, sh, key, 0, 10);
        f = find_bin(sh, by_count, need, target, f.above, f.above_mass);
        key = key << 10 | f.bin;
    } else {  // a 16-bit logit's low bits follow from its sign
        key = key << 10 | ((key >> 21) != 0 ? 0u : 0x3ffu);
    }
    f.bin = key;
    return f;
}

// The index of the `need`-th logit, in index order, with this key.
template <class T>
__device__ __forceinline__ uint32_t tie_index(const SampleArgs &a, const T *x, BorderShared &sh, uint32_t key,
                                              uint32_t need) {
    using L = Logits<T>;
    constexpr int kWaves = kBorderBlock / kWave;
    constexpr int kStep = kWave * L::kN;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int steps = (a.vocab + kStep - 1) / kStep;
    const int each = (steps + kWaves - 1) / kWaves;
    const int first = w * each, last = first + each < steps ? first + each : steps;
    uint32_t count = 0;
    for (int s = first; s < last; ++s) {
        L v;
        v.load(x, s * kStep + lane * L::kN, a.vocab);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) count += key_of(v.x[e]) == key ? 1u : 0u;
    }
    for (int off = 32; off > 0; off >>= 1) count += __shfl_xor(count, off);
    if (lane == 0) sh.wave_count[w] = count;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += sh.wave_count[i];
    if (before < need && before + count >= need) {  // this wavefront holds it
        for (int s = first; s < last; ++s) {
            const int i = s * kStep + lane * L::kN;
            L v;
            v.load(x, i, a.vocab);
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
    return sh.cut;
}

template <class T>
__global__ __launch_bounds__(kBorderBlock) void sample_border_kernel(SampleArgs a) {
    __shared__ BorderShared sh;
    const int row = blockIdx.x;
    const uint32_t max_key = row_max(a, row);
    const Settings st(a, row, max_key);
    RowState out{1u, kNoCut};  // every token
    const T *x = row_at<T>(a, row);
    if (threadIdx.x == 0) sh.cut = kNoCut;
    __syncthreads();
    if (max_key != 0 && st.top_k == 1) {
        out.border = max_key;
        out.cut = tie_index(a, x, sh, max_key, 1);
    } else if (max_key != 0 && (st.top_k > 0 || st.top_p <= 1.0f)) {
        uint64_t mass = 0;       // of the keys that top_k leaves
        uint32_t ties = 0, have = 0;
        if (st.top_k > 0) {
            // fewer tokens than top_k: all of them
            uint32_t n = 0;
            for (int b = threadIdx.x; b < kBins; b += kBorderBlock) {
                n += a.hist_count[static_cast<int64_t>(row) * kBins + b];
                mass += a.hist_mass[static_cast<int64_t>(row) * kBins + b];
            }
            for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off);
            mass = wave_sum64(mass);
            if (lane_id() == 0) {
                sh.wave_count[threadIdx.x / kWave] = n;
                sh.wave_mass[threadIdx.x / kWave] = mass;
            }
            __syncthreads();
            n = 0;
            mass = 0;
            for (int i = 0; i < kBorderBlock / kWave; ++i) {
                n += sh.wave_count[i];
                mass += sh.wave_mass[i];
            }
            __syncthreads();
            if (n > static_cast<uint32_t>(st.top_k)) {
                const Found f = border_key(a, row, x, st, sh, true, static_cast<uint32_t>(st.top_k), 0.0);
                out.border = f.bin;
                ties = static_cast<uint32_t>(st.top_k) - f.above;
                have = f.count;
                mass = f.above_mass + ties * st.fixed(st.weight(value_of(f.bin)));
            }
        } else {
            for (int b = threadIdx.x; b < kBins; b += kBorderBlock)
                mass += a.hist_mass[static_cast<int64_t>(row) * kBins + b];
            mass = wave_sum64(mass);
            if (lane_id() == 0) sh.wave_mass[threadIdx.x / kWave] = mass;
            __syncthreads();
            mass = 0;
            for (int i = 0; i < kBorderBlock / kWave; ++i) mass += sh.wave_mass[i];
            __syncthreads();
        }
        if (st.top_p <= 1.0f) {
            const double target = static_cast<double>(st.top_p) * static_cast<double>(mass);
            const Found f = border_key(a, row, x, st, sh, false, 0, target);
            // ties j = 0, 1, ... are kept while above_mass + j * weight < target
            const uint64_t wt = st.fixed(st.weight(value_of(f.bin)));
            uint32_t j = f.count;
            if (wt != 0) {
                const double q = (target - static_cast<double>(f.above_mass)) / static_cast<double>(wt);
                uint32_t g = q < static_cast<double>(f.count) ? static_cast<uint32_t>(q) : f.count;
                while (g > 0 && static_cast<double>(f.above_mass + (g - 1) * wt) >= target) --g;
                while (g < f.count && static_cast<double>(f.above_mass + g * wt) < target) ++g;
                j = g;
            }
            if (f.bin != out.border || j < ties || ties == 0) {
                out.border = f.bin;
                ties = j;
                have = f.count;
            }
        }
        if (ties < have) out.cut = tie_index(a, x, sh, out.border, ties);
    }
    if (threadIdx.x == 0) a.state[row] = out;
}

// ---- kept weight and count of each part ----
// A kept logit's weight as an integer; 0 and not counted for the others.
__device__ __forceinline__ uint64_t kept_weight(const Settings &st, const RowState &rs, uint32_t key, float x, int i,
                                                uint32_t max_key, bool &kept) {
    kept = false;
    if (key == 0 || key < rs.border || (key == rs.border && static_cast<uint32_t>(i) > rs.cut)) return 0;
    const double w = st.weight(x);
    kept = key == max_key || w >= st.min_w;
    return kept ? st.fixed(w) : 0;
}

template <class T>
__global__ __launch_bounds__(kPartBlock) void sample_sum_kernel(SampleArgs a) {
    __shared__ unsigned long long s_mass[kPartBlock / kWave];
    __shared__ uint32_t s_count[kPartBlock / kWave];
    const int row = blockIdx.y, part = blockIdx.x;
    const uint32_t max_key = row_max(a, row);
    const Settings st(a, row, max_key);
    const RowState rs = a.hist_count != nullptr ? a.state[row] : RowState{1u, kNoCut};
    const T *x = row_at<T>(a, row);
    using L = Logits<T>;
    uint64_t mass = 0;
    uint32_t count = 0;
#pragma unroll
    for (int j = 0; j < kPartItems / L::kN; ++j) {
        const int i = part * kPart + (j * kPartBlock + static_cast<int>(threadIdx.x)) * L::kN;
        if (i >= a.vocab) continue;
        L v;
        v.load(x, i, a.vocab);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) {
            bool kept;
            mass += kept_weight(st, rs, key_of(v.x[e]), v.x[e], i + e, max_key, kept);
            count += kept ? 1u : 0u;
        }
    }
    mass = wave_sum64(mass);
    for (int off = 32; off > 0; off >>= 1) count += __shfl_xor(count, off);
    if (lane_id() == 0) {
        s_mass[threadIdx.x / kWave] = mass;
        s_count[threadIdx.x / kWave] = count;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kPartBlock / kWave; ++w) {
            mass += s_mass[w];
            count += s_count[w];
        }
        a.part_mass[static_cast<int64_t>(row) * a.parts + part] = mass;
        a.part_count[static_cast<int64_t>(row) * a.parts + part] = count;
    }
}

// ---- the token ----
template <class T>
__global__ __launch_bounds__(kPartBlock) void sample_token_kernel(SampleArgs a) {
    __shared__ unsigned long long s_wave[kPartBlock / kWave];
    __shared__ int s_part;
    __shared__ unsigned long long s_before, s_total;
    const int row = blockIdx.x;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const uint32_t max_key = row_max(a, row);
    const Settings st(a, row, max_key);
    const RowState rs = a.hist_count != nullptr ? a.state[row] : RowState{1u, kNoCut};
    const int64_t base = static_cast<int64_t>(row) * a.parts;
    if (max_key == 0) {
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.kept != nullptr) a.kept[row] = 0;
            if (a.logprobs != nullptr) a.logprobs[row] = -__builtin_inff();
        }
        return;
    }
    if (w == 0) {  // the part in which the running weight passes the goal
        uint64_t total = 0;
        uint32_t count = 0;
        for (int p = lane; p < a.parts; p += kWave) {
            total += a.part_mass[base + p];
            count += a.part_count[base + p];
        }
        total = wave_sum64(total);
        for (int off = 32; off > 0; off >>= 1) count += __shfl_xor(count, off);
        float u = a.u[row];
        u = u > 0.0f ? u : 0.0f;
        u = u < 0x1.fffffep-1f ? u : 0x1.fffffep-1f;
        const uint64_t goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
        uint64_t before = 0;
        for (int p0 = 0; p0 < a.parts; p0 += kWave) {
            const uint64_t m = p0 + lane < a.parts ? a.part_mass[base + p0 + lane] : 0;
            const uint64_t incl = wave_scan64(m);
            const uint64_t hit = ballot(before + incl > goal);
            if (hit != 0) {
                const int l = __builtin_ctzll(hit);
                if (lane == l) {
                    s_part = p0 + l;
                    s_before = goal - (before + incl - m);  // what is left to pass in the part
                    s_total = total;
                }
                break;
            }
            before += __shfl(static_cast<unsigned long long>(incl), kWave - 1);
        }
        if (lane == 0 && a.kept != nullptr) a.kept[row] = static_cast<int32_t>(count);
    }
    __syncthreads();
    const uint64_t goal = s_before;
    const T *x = row_at<T>(a, row);
    // each thread takes consecutive logits of the part
    const int first = s_part * kPart + static_cast<int>(threadIdx.x) * kPartItems;
    float v[kPartItems];
    uint64_t mass = 0;
    using L = Logits<T>;
#pragma unroll
    for (int j = 0; j < kPartItems / L::kN; ++j) {
        L l;
        l.load(x, first + j * L::kN, a.vocab);
#pragma unroll
        for (int e = 0; e < L::kN; ++e) {
            const int i = j * L::kN + e;
            bool kept;
            v[i] = l.x[e];
            mass += kept_weight(st, rs, key_of(v[i]), v[i], first + i, max_key, kept);
        }
    }
    const uint64_t incl = wave_scan64(mass);
    if (lane == kWave - 1) s_wave[w] = incl;
    __syncthreads();
    uint64_t run = incl - mass;
    for (int i = 0; i < w; ++i) run += s_wave[i];
    if (run <= goal && run + mass > goal) {
        int at = -1;
        float chosen = 0.0f;
#pragma unroll
        for (int i = 0; i < kPartItems; ++i) {
            bool kept;
            run += kept_weight(st, rs, key_of(v[i]), v[i], first + i, max_key, kept);
            if (at < 0 && run > goal) {
                at = first + i;
                chosen = v[i];
            }
        }
        a.tokens[row] = at;
        if (a.logprobs != nullptr) {
            const double z = st.max_inf ? 0.0 : (static_cast<double>(chosen) - st.max) * st.inv_t;
            a.logprobs[row] = static_cast<float>(z - log(static_cast<double>(s_total) / st.scale));
        }
    }
}

// ============================================================ host side ---
constexpr int64_t kVocabMax = int64_t{1} << 22;

struct SamplePlan {
    int64_t parts;
    size_t hist_mass, part_mass, hist_count, part_max, part_count, state, bytes;  // offsets
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
    p.hist_mass = take(r * kBins * 8);
    p.part_mass = take(r * g * 8);
    p.hist_count = take(r * kBins * 4);
    p.part_max = take(r * g * 4);
    p.part_count = take(r * g * 4);
    p.state = take(r * sizeof(RowState));
    p.bytes = at;
    return p;
}

template <class T>
int sample_launch(const SampleArgs &a, int64_t rows, bool border, hipStream_t s) {
    const unsigned r = static_cast<unsigned>(rows);
    const dim3 parts(static_cast<unsigned>(a.parts), r);
    hipLaunchKernelGGL((sample_max_kernel<T>), parts, dim3(kPartBlock), 0, s, a);
    SSC_TRY(launched());
    if (border) {
        hipLaunchKernelGGL((sample_hist_kernel<T>), dim3((a.vocab + kHistPart - 1) / kHistPart, r), dim3(kHistBlock),
                           0, s, a);
        SSC_TRY(launched());
        hipLaunchKernelGGL((sample_border_kernel<T>), dim3(r), dim3(kBorderBlock), 0, s, a);
        SSC_TRY(launched());
    }
    hipLaunchKernelGGL((sample_sum_kernel<T>), parts, dim3(kPartBlock), 0, s, a);
    SSC_TRY(launched());
    hipLaunchKernelGGL((sample_token_kernel<T>), dim3(r), dim3(kPartBlock), 0, s, a);
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
    // temperatures may be 0, which keeps one token
    const bool border = temperature != nullptr || top_k != nullptr || top_p != nullptr;
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
    a.part_max = reinterpret_cast<uint32_t *>(base + p.part_max);
    a.part_mass = reinterpret_cast<uint64_t *>(base + p.part_mass);
    a.part_count = reinterpret_cast<uint32_t *>(base + p.part_count);
    a.state = reinterpret_cast<RowState *>(base + p.state);
    if (border) {
        a.hist_mass = reinterpret_cast<uint64_t *>(base + p.hist_mass);
        a.hist_count = reinterpret_cast<uint32_t *>(base + p.hist_count);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case SSC_F32: return sample_launch<float>(a, rows, border, s);
    case SSC_BF16: return sample_launch<__bf16>(a, rows, border, s);
    default: return sample_launch<_Float16>(a, rows, border, s);
    }
}

}  // extern "C"
