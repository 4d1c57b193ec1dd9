// Drafted tokens held against the probabilities of the model that they were
// drafted for, from given random numbers: HIP kernels for MI355X (gfx950) and
// their part of the C ABI in include/ssc.h.
//
// Draft i of a sequence stands while u_i * q_i(x_i) < p_i(x_i); after the a
// drafts that stand one token is drawn by the weights max(p_a - q_a, 0), after
// all of them by p_a: the first index at which their running sum exceeds
// u_last times their sum. The tokens then come as from p alone. Of the (drafts
// + 1) rows of a sequence one is read, beside 2 * drafts single values.
//
// Every wavefront finds a (a few dependent loads) and sums segments of 1024
// weights; then a workgroup a sequence finds the segment by a scan of the sums,
// and the token in it by reading it again: in one launch, or in two where few
// long rows would leave the chip empty. Sums are fp64, in an order that the sizes
// fix: a border of u that fp32 sums would miss once in some hundred rows (131,072
// borders, 1e-8 of the sum each) is met. For few rows bound
// by latency (one of 131,072 fp32, in two launches: 3.5 + 3.6 us). 192 of 131,072
// bf16 with 4 drafts: 21.4 us for 75 MB, 3.5 TB/s where a copy reaches 5.15: a row
// whose drafts all stand reads p alone, another p and q, and one workgroup has
// either; in two launches, with the segments spread evenly, 17.9 + 4.2.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssc.h"
#include "ssc_device.h"
#include "ssc_host.h"

namespace ssc {
namespace {

constexpr int kSeg = 1024;             // weights of a segment: 16 a lane
constexpr int kEach = kSeg / kWave;
constexpr int kSumBlock = 256;
constexpr int kSumWaves = kSumBlock / kWave;
constexpr int kDrawBlock = 256;
// The form in one launch, a row to a workgroup: for rows of up to 64 segments, and
// of up to 128 where there are enough to fill the chip. us a call (repeated by
// prepared), one launch against two, fp32:
//   rows of        32,768                     65,536                      131,072
//   1        12.6 16.7 ( 7.9  7.1)     12.5 16.7 (10.4  6.9)     15.5 16.7 (15.4  6.8)
//   64       12.6 16.7 ( 9.0  7.7)     12.7 16.7 (11.6  9.4)     19.0 16.4 (19.0 15.2)
//   192      12.5 16.8 (10.9 12.3)     17.3 18.4 (17.3 18.1)     27.2 28.9 (27.1 28.8)
// and by prepared alone, bf16 (the rows partly in the last-level cache), around the borders:
//   rows of      65,536       98,304      131,072      152,000      256,000
//   128       12.8 12.3    15.9 14.4    18.6 16.8    20.9 18.7    30.4 25.7
//   160       13.4 13.5    16.7 16.3    19.7 19.2    21.5 21.1    31.7 29.9
//   192       14.2 14.4    17.4 17.6    20.9 21.4    22.7 23.9    34.6 35.2
//   256       15.7 16.5    19.7 20.8    24.5 25.4    26.6 29.0    43.9 50.4
// so that from 192 rows on longer vocabularies would gain by one launch, too: they
// take two, for the sums of 128 segments that the form holds.
constexpr int kRowBlock = 1024;
constexpr int kRowSegs = 128;
constexpr int kRowMany = 160;
constexpr int64_t kVerifyVocabMax = int64_t{1} << 22;
constexpr int kSegsMax = static_cast<int>(kVerifyVocabMax / kSeg);

struct VerifyState {
    int32_t accepted, length;
};

struct VerifyArgs {
    const void *probs, *draft;  // draft null: a drafted token has probability 1
    int64_t row, place, draft_row, draft_place;  // strides
    const void *ids;
    const float *u;
    const int32_t *lengths;
    int drafts, vocab, segs;
    int32_t *tokens, *accepted;
    VerifyState *state;  // [rows]
    double *sums;        // [rows][segs]
};

// A random number outside [0, 1) as the nearest in it, NaN as 0.
__device__ __forceinline__ float unit(float u) { return fminf(fmaxf(u, 0.0f), 0x1.fffffep-1f); }

// How many drafts stand, by every wavefront for itself.
template <class T, class I>
__device__ __forceinline__ VerifyState drafts_that_stand(const VerifyArgs &a, int64_t b) {
    int length = a.drafts;
    if (a.lengths != nullptr) {
        const int l = a.lengths[b];
        length = l < 0 ? 0 : (l < a.drafts ? l : a.drafts);
    }
    for (int base = 0; base < length; base += kWave) {
        const int i = base + lane_id();
        bool falls = false;
        if (i < length) {
            const int64_t x = static_cast<const I *>(a.ids)[b * a.drafts + i];
            const bool token = x >= 0 && x < a.vocab;
            const int64_t at = token ? x : 0;
            const double p = static_cast<float>(static_cast<const T *>(a.probs)[b * a.row + i * a.place + at]);
            const double q = a.draft != nullptr ? static_cast<float>(static_cast<const T *>(
                                                      a.draft)[b * a.draft_row + i * a.draft_place + at])
                                                : 1.0f;
            const double u = unit(a.u[b * (a.drafts + 1) + i]);
            falls = !(token && u * q < p);
        }
        const uint64_t fallen = ballot(falls);
        if (fallen != 0) return {base + __builtin_ctzll(fallen), length};
    }
    return {length, length};
}

// The weights that the token is drawn by. Neither a value that is not above 0
// nor one that is not finite weighs anything.
template <class T>
struct Weights {
    const T *p, *q;  // q null: nothing taken away but `without`
    int n, without;

    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    typedef T V __attribute__((ext_vector_type(kN)));
    typedef uint32_t Raw __attribute__((ext_vector_type(4)));
    typedef uint32_t RawAny __attribute__((ext_vector_type(4), aligned(2), may_alias));

    template <class I>
    __device__ __forceinline__ Weights(const VerifyArgs &a, int64_t b, const VerifyState &s, const I *ids)
        : p(static_cast<const T *>(a.probs) + b * a.row + s.accepted * a.place), q(nullptr), n(a.vocab), without(-1) {
        if (s.accepted < s.length) {
            if (a.draft != nullptr)
                q = static_cast<const T *>(a.draft) + b * a.draft_row + s.accepted * a.draft_place;
            else {
                const int64_t x = ids[b * a.drafts + s.accepted];
                without = x >= 0 && x < n ? static_cast<int>(x) : -1;
            }
        }
    }
    __device__ static __forceinline__ double weight(double w) { return w > 0.0 && w < __builtin_inf() ? w : 0.0; }

    // kN values of each row, as they lie in memory
    struct Pair {
        Raw x, y;
    };
    // [i, i + kN), which the row holds all of
    __device__ __forceinline__ Pair fetch(int i) const {
        Pair r;
        r.x = *reinterpret_cast<const RawAny *>(p + i);
        r.y = q != nullptr ? static_cast<Raw>(*reinterpret_cast<const RawAny *>(q + i)) : Raw{0, 0, 0, 0};
        return r;
    }
    __device__ __forceinline__ void unpack(const Pair &r, int i, double (&w)[kN]) const {
        const V x = __builtin_bit_cast(V, r.x), y = __builtin_bit_cast(V, r.y);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const double a = static_cast<float>(x[e]), b = static_cast<float>(y[e]);
            w[e] = weight(a - b);
        }
        if (without >= 0) {
#pragma unroll
            for (int e = 0; e < kN; ++e) w[e] = i + e == without ? 0.0 : w[e];
        }
    }
    // weights [i, i + kN); past the end 0
    __device__ __forceinline__ void load(int i, double (&w)[kN]) const {
        if (i + kN <= n) {
            unpack(fetch(i), i, w);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                double v = 0.0;
                if (i + e < n && i + e != without) {
                    v = static_cast<float>(p[i + e]);
                    if (q != nullptr) v -= static_cast<double>(static_cast<float>(q[i + e]));
                }
                w[e] = weight(v);
            }
        }
    }
};

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_move_f64(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    const uint64_t hi = dpp_move<CTRL, ROW_MASK>(static_cast<uint32_t>(b >> 32));
    const uint64_t lo = dpp_move<CTRL, ROW_MASK>(static_cast<uint32_t>(b));
    return __longlong_as_double(static_cast<long long>(hi << 32 | lo));
}
// Inclusive scan over the wavefront, as wave_inclusive_scan (0 is its identity).
__device__ __forceinline__ double wave_scan_f64(double v) {
    v += dpp_move_f64<0x111, 0xf>(v);
    v += dpp_move_f64<0x112, 0xf>(v);
    v += dpp_move_f64<0x114, 0xf>(v);
    v += dpp_move_f64<0x118, 0xf>(v);
    v += dpp_move_f64<0x142, 0xa>(v);
    v += dpp_move_f64<0x143, 0xc>(v);
    return v;
}

// Sum of a segment's weights over the wavefront, in its last lane.
template <class T>
__device__ __forceinline__ double segment_sum(const Weights<T> &w, int seg) {
    constexpr int kN = Weights<T>::kN;
    double v[kEach / kN][kN], s = 0.0;
#pragma unroll
    for (int j = 0; j < kEach / kN; ++j) w.load(seg * kSeg + (j * kWave + lane_id()) * kN, v[j]);
#pragma unroll
    for (int j = 0; j < kEach / kN; ++j) {
#pragma unroll
        for (int e = 0; e < kN; ++e) s += v[j][e];
    }
    return wave_scan_f64(s);
}

// Sums of the segments first, first + step, ... into sums, by a wavefront. One
// that the row holds all of is on its way while the one before it is added up.
template <class T>
__device__ __forceinline__ void segment_sums(const VerifyArgs &a, const Weights<T> &w, int first, int step,
                                             double *sums) {
    using W = Weights<T>;
    constexpr int kN = W::kN, kParts = kEach / kN;
    const int lane = lane_id();
    const int whole = a.vocab / kSeg;
    typename W::Pair raw[kParts];
    const auto fetch = [&](int at) {
#pragma unroll
        for (int j = 0; j < kParts; ++j) raw[j] = w.fetch(at * kSeg + (j * kWave + lane) * kN);
    };
    int seg = first;
    if (seg < whole) fetch(seg);
    for (; seg < whole; seg += step) {
        typename W::Pair now[kParts];
#pragma unroll
        for (int j = 0; j < kParts; ++j) now[j] = raw[j];
        if (seg + step < whole) fetch(seg + step);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            double v[kN];
            w.unpack(now[j], seg * kSeg + (j * kWave + lane) * kN, v);
#pragma unroll
            for (int e = 0; e < kN; ++e) sum += v[e];
        }
        sum = wave_scan_f64(sum);
        if (lane == kWave - 1) sums[seg] = sum;
    }
    if (seg < a.segs) {  // the last, in part
        const double sum = segment_sum(w, seg);
        if (lane == kWave - 1) sums[seg] = sum;
    }
}

template <class T, class I>
__global__ __launch_bounds__(kSumBlock) void verify_sum_kernel(VerifyArgs a) {
    const int64_t b = blockIdx.y;
    const VerifyState s = drafts_that_stand<T, I>(a, b);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.state[b] = s;
    const Weights<T> w(a, b, s, static_cast<const I *>(a.ids));
    segment_sums(a, w, static_cast<int>(blockIdx.x) * kSumWaves + static_cast<int>(uniform(threadIdx.x / kWave)),
                 static_cast<int>(gridDim.x) * kSumWaves, a.sums + b * a.segs);
}

// The token of a row from the sums of its segments, by a workgroup: where their
// running sum first exceeds the goal, then where that of the segment's weights
// does. What weighs nothing is no place. Writes the row's results.
template <int BLOCK>
struct DrawShared {
    double wave[BLOCK / kWave];
    int first[BLOCK / kWave];
};

template <int BLOCK, class T, class I>
__device__ __forceinline__ void draw(const VerifyArgs &a, int64_t b, const VerifyState &s, Weights<T> &weights,
                                     double *sums, DrawShared<BLOCK> &sh) {
    constexpr int kWaves = BLOCK / kWave;
    const int lane = lane_id();
    const int w = static_cast<int>(uniform(threadIdx.x / kWave));
    const double u = unit(a.u[b * (a.drafts + 1) + a.drafts]);
    // a thread runs over consecutive segments
    const int each = (a.segs + BLOCK - 1) / BLOCK;
    const int begin = static_cast<int>(threadIdx.x) * each;
    const int end = begin + each < a.segs ? begin + each : a.segs;
    double own, incl, before, total;
    const auto scan = [&]() {
        own = 0.0;
        for (int i = begin; i < end; ++i) own += sums[i];
        incl = wave_scan_f64(own);
        if (lane == kWave - 1) sh.wave[w] = incl;
        __syncthreads();
        before = 0.0;
        total = 0.0;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const double x = sh.wave[v];
            before += v < w ? x : 0.0;
            total += x;
        }
    };
    scan();
    if (!(total > 0.0) && s.accepted < s.length) {  // q covers p: the token is drawn by p itself
        weights.q = nullptr;
        weights.without = -1;
        __syncthreads();
        segment_sums(a, weights, w, kWaves, sums);
        __syncthreads();
        scan();
    }
    const double goal = u * total;
    // the first segment at whose end the running sum exceeds the goal, or the
    // last that weighs anything (where rounding leaves none)
    double run = before + incl - own;
    int seg = -1, last = -1;
    for (int i = begin; i < end; ++i) {
        const double v = sums[i];
        run += v;
        if (v > 0.0) last = i;
        if (seg < 0 && v > 0.0 && run > goal) seg = i;
    }
    {
        const uint64_t found = ballot(seg >= 0), any = ballot(last >= 0);
        int first = -1;
        if (found != 0)
            first = __builtin_amdgcn_readlane(seg, __builtin_ctzll(found));
        else if (any != 0)
            first = -2 - __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(any));
        if (lane == 0) sh.first[w] = first;
    }
    __syncthreads();
    int at = -1, fallback = -1;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
        const int f = sh.first[v];
        if (f >= 0 && at < 0) at = f;
        if (f < -1) fallback = -2 - f;
    }
    if (at < 0) at = fallback;
    int32_t token = -1;
    if (at >= 0) {
        // the sum before the segment, added up as the search did; the wavefronts'
        // totals have been read by now
        if (static_cast<int>(threadIdx.x) == at / each) {
            double base = before + incl - own;
            for (int i = begin; i < at; ++i) base += sums[i];
            sh.wave[0] = base;
        }
        __syncthreads();
        if (w == 0) {
            constexpr int kN = Weights<T>::kN;
            double v[kEach / kN][kN], sum = 0.0;
#pragma unroll
            for (int j = 0; j < kEach / kN; ++j) weights.load(at * kSeg + lane * kEach + j * kN, v[j]);
#pragma unroll
            for (int j = 0; j < kEach / kN; ++j) {
#pragma unroll
                for (int e = 0; e < kN; ++e) sum += v[j][e];
            }
            double r = sh.wave[0] + wave_scan_f64(sum) - sum;
            int first = -1, any = -1;
#pragma unroll
            for (int j = 0; j < kEach / kN; ++j) {
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    r += v[j][e];
                    const int i = at * kSeg + lane * kEach + j * kN + e;
                    if (v[j][e] > 0.0) any = i;
                    if (first < 0 && v[j][e] > 0.0 && r > goal) first = i;
                }
            }
            const uint64_t found = ballot(first >= 0), some = ballot(any >= 0);
            if (found != 0)
                token = __builtin_amdgcn_readlane(first, __builtin_ctzll(found));
            else if (some != 0)
                token = __builtin_amdgcn_readlane(any, 63 - __builtin_clzll(some));
        }
    }
    if (w == 0) {
        const I *ids = static_cast<const I *>(a.ids) + b * a.drafts;
        for (int i = lane; i <= a.drafts; i += kWave)
            a.tokens[b * (a.drafts + 1) + i] =
                i < s.accepted ? static_cast<int32_t>(ids[i]) : (i == s.accepted ? token : -1);
        if (lane == 0) a.accepted[b] = s.accepted;
    }
}

template <class T, class I>
__global__ __launch_bounds__(kDrawBlock) void verify_draw_kernel(VerifyArgs a) {
    __shared__ double s_sums[kSegsMax];
    __shared__ DrawShared<kDrawBlock> sh;
    const int64_t b = blockIdx.x;
    for (int i = threadIdx.x; i < a.segs; i += kDrawBlock) s_sums[i] = a.sums[b * a.segs + i];
    const VerifyState s = a.state[b];
    Weights<T> weights(a, b, s, static_cast<const I *>(a.ids));
    __syncthreads();
    draw<kDrawBlock, T, I>(a, b, s, weights, s_sums, sh);
}

// A row by one workgroup, in one launch.
template <class T, class I>
__global__ __launch_bounds__(kRowBlock) void verify_row_kernel(VerifyArgs a) {
    __shared__ double s_sums[kRowSegs];
    __shared__ DrawShared<kRowBlock> sh;
    const int64_t b = blockIdx.x;
    const VerifyState s = drafts_that_stand<T, I>(a, b);
    Weights<T> weights(a, b, s, static_cast<const I *>(a.ids));
    segment_sums(a, weights, static_cast<int>(uniform(threadIdx.x / kWave)), kRowBlock / kWave, s_sums);
    __syncthreads();
    draw<kRowBlock, T, I>(a, b, s, weights, s_sums, sh);
}

// ============================================================ host side ---
struct VerifyPlan {
    int segs;
    size_t sums, bytes;
};
VerifyPlan verify_plan(int64_t rows, int64_t vocab) {
    VerifyPlan p{};
    p.segs = static_cast<int>((vocab + kSeg - 1) / kSeg);
    if (p.segs <= kRowSegs / 2 || (p.segs <= kRowSegs && rows >= kRowMany)) return p;
    p.sums = (static_cast<size_t>(rows) * sizeof(VerifyState) + 15) / 16 * 16;
    p.bytes = p.sums + static_cast<size_t>(rows) * p.segs * sizeof(double);
    return p;
}
bool verify_sizes_ok(int64_t rows, int64_t vocab) {
    return rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= kVerifyVocabMax;
}

template <class I>
int verify_impl(const void *probs, int dtype, int64_t rows, int64_t drafts, int64_t vocab, int64_t row, int64_t place,
                const I *ids, const void *draft, int64_t draft_row, int64_t draft_place, const float *u,
                const int32_t *lengths, int32_t *tokens, int32_t *accepted, void *scratch, size_t scratch_bytes,
                void *stream) {
    if (!dtype_ok(dtype) || rows < 0 || drafts < 0 || vocab < 1) return SSC_ERR_ARG;
    if (!verify_sizes_ok(rows, vocab) || drafts > (1 << 20)) return SSC_ERR_SIZE;
    const View<3> p{{rows, drafts + 1, vocab}, {row, place, 1}};
    const View<3> q{{rows, draft != nullptr ? drafts : 0, vocab}, {draft_row, draft_place, 1}};
    if (!p.strides_ok() || (draft != nullptr && !q.strides_ok())) return SSC_ERR_ARG;
    if (rows > 0 && (probs == nullptr || u == nullptr || tokens == nullptr || accepted == nullptr ||
                     (drafts > 0 && ids == nullptr)))
        return SSC_ERR_ARG;
    const size_t es = elem_bytes(dtype);
    if (!aligned(probs, es) || !aligned(draft, es) || !aligned(ids, sizeof(I)) || !aligned(u, 4) ||
        !aligned(lengths, 4) || !aligned(tokens, 4) || !aligned(accepted, 4))
        return SSC_ERR_ARG;
    const VerifyPlan plan = verify_plan(rows, vocab);
    if (plan.bytes > 0 && (scratch == nullptr || !aligned(scratch, 16) || scratch_bytes < plan.bytes)) return SSC_ERR_SCRATCH;
    const size_t n = static_cast<size_t>(rows);
    const Span written[] = {{tokens, n * (drafts + 1) * 4}, {accepted, n * 4}, {scratch, plan.bytes}};
    const Span read[] = {{probs, static_cast<size_t>(p.extent()) * es},
                         {draft, static_cast<size_t>(q.extent()) * es},
                         {ids, n * drafts * sizeof(I)},
                         {u, n * (drafts + 1) * 4},
                         {lengths, n * 4}};
    if (spans_overlap(written)) return SSC_ERR_ALIAS;
    for (const Span &x : written)
        for (const Span &y : read)
            if (overlap(x.p, x.bytes, y.p, y.bytes)) return SSC_ERR_ALIAS;
    SSC_TRY(check_device());
    if (rows == 0) return SSC_OK;
    VerifyArgs a{};
    a.probs = probs;
    a.draft = draft;
    a.row = row;
    a.place = place;
    a.draft_row = draft_row;
    a.draft_place = draft_place;
    a.ids = ids;
    a.u = u;
    a.lengths = lengths;
    a.drafts = static_cast<int>(drafts);
    a.vocab = static_cast<int>(vocab);
    a.segs = plan.segs;
    a.tokens = tokens;
    a.accepted = accepted;
    a.state = static_cast<VerifyState *>(scratch);
    a.sums = reinterpret_cast<double *>(static_cast<char *>(scratch) + plan.sums);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (plan.bytes == 0)
        return with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            hipLaunchKernelGGL((verify_row_kernel<T, I>), dim3(static_cast<unsigned>(rows)), dim3(kRowBlock), 0, s, a);
            return launched();
        });
    // a segment to a wavefront, or several where there are more than the chip holds
    int64_t each = rows * plan.segs / 6144;
    each = each < 1 ? 1 : (each > 8 ? 8 : each);
    const int64_t blocks = (plan.segs + kSumWaves * each - 1) / (kSumWaves * each);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((verify_sum_kernel<T, I>), dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(rows)),
                           dim3(kSumBlock), 0, s, a);
        SSC_TRY(launched());
        hipLaunchKernelGGL((verify_draw_kernel<T, I>), dim3(static_cast<unsigned>(rows)), dim3(kDrawBlock), 0, s, a);
        return launched();
    });
}

}  // namespace
}  // namespace ssc

using namespace ssc;

extern "C" {

size_t ssc_verify_scratch_bytes(int64_t rows, int64_t vocab) {
    return rows > 0 && verify_sizes_ok(rows, vocab) ? verify_plan(rows, vocab).bytes : 0;
}

int ssc_verify_rows_i32(const void *probs, int dtype, int64_t rows, int64_t drafts, int64_t vocab, int64_t stride_row,
                        int64_t stride_place, const int32_t *drafted, const void *draft_probs, int64_t draft_stride_row,
                        int64_t draft_stride_place, const float *u, const int32_t *lengths, int32_t *tokens,
                        int32_t *accepted, void *scratch, size_t scratch_bytes, void *stream) {
    return verify_impl(probs, dtype, rows, drafts, vocab, stride_row, stride_place, drafted, draft_probs,
                       draft_stride_row, draft_stride_place, u, lengths, tokens, accepted, scratch, scratch_bytes,
                       stream);
}

int ssc_verify_rows_i64(const void *probs, int dtype, int64_t rows, int64_t drafts, int64_t vocab, int64_t stride_row,
                        int64_t stride_place, const int64_t *drafted, const void *draft_probs, int64_t draft_stride_row,
                        int64_t draft_stride_place, const float *u, const int32_t *lengths, int32_t *tokens,
                        int32_t *accepted, void *scratch, size_t scratch_bytes, void *stream) {
    return verify_impl(probs, dtype, rows, drafts, vocab, stride_row, stride_place, drafted, draft_probs,
                       draft_stride_row, draft_stride_place, u, lengths, tokens, accepted, scratch, scratch_bytes,
                       stream);
}

}  // extern "C"
