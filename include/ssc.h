/*
 * ssc.h -- single-pass scan, stream compaction and stable partition on
 * AMD Instinct MI355X (gfx950), as a C ABI.
 *
 * The method: evaluate a predicate on every element (a 0/1 flag), take the
 * exclusive scan of the flags, and scatter every survivor x[i] to
 * out[rank[i]]. Input order is kept, the survivor count is the top of the
 * scan, and a stable partition addresses its second half with i - rank[i]
 * from the same scan ("Day 33 compaction.cu", header comment and
 * scatterCompact / scatterPartition). The scan runs in one pass over the
 * input with per-tile descriptors and a decoupled look-back over earlier
 * tiles, tile numbers being taken from an atomic counter ("CUDA Handbook
 * ch. 13, Stream Compaction", Listings 13-17 and 13-18).
 *
 * Conventions shared by every call:
 *   - All array, count and scratch pointers are DEVICE pointers (hipMalloc
 *     or equivalent) owned by the caller. The library never allocates and
 *     never frees.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream); it
 *     must belong to the current device. Calls only enqueue work on it and
 *     never synchronise; counts and totals stay in device memory.
 *   - Scratch: a caller-provided device buffer of at least
 *     ssc_scratch_bytes(n) bytes, 8-byte aligned, ZERO-FILLED BEFORE ITS
 *     FIRST USE (ssc_scratch_init, or any memset to 0). The library keeps it
 *     ready for the next call by itself: no clearing between calls, so a
 *     call is a single kernel launch (two for a partition). Pass the same
 *     scratch_bytes every time a buffer is used. One scratch buffer must not
 *     serve two calls that may run at the same time (the calls race).
 *     Diagnostic: a look-back wait that gives up after its bounded spin
 *     (only possible on misuse, such as a scratch that was never zeroed or
 *     one shared by two calls in flight) sets a time-out flag in the
 *     scratch; ssc_scratch_timed_out reads it. Once set, the results of the
 *     calls made with that scratch are invalid and the flag stays set: the
 *     scratch must be re-initialised (ssc_scratch_init) before it is used
 *     again.
 *   - Element pointers must be 4-byte aligned. 16-byte aligned arrays take
 *     the 128-bit load/store path; other arrays take a 32-bit path with the
 *     same results.
 *   - Sizes: n is an element count, 0 <= n <= INT32_MAX (ranks and counts are
 *     int32). n == 0 writes 0 to `count` / `total` and returns SSC_OK; array
 *     pointers may then be NULL (count/total may not be, where required).
 *   - Errors: every call returns an ssc_status; arguments are checked before
 *     anything is enqueued, and on an argument error nothing is enqueued. A
 *     failed launch gives SSC_ERR_HIP (ssc_last_hip_error() has the code).
 *     The library never exits or aborts.
 *   - Only the elements out[0 .. count) of a compaction are written; the rest
 *     of `out` is left as it was.
 */
#ifndef SSC_H
#define SSC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ssc_status {
    SSC_OK = 0,
    SSC_ERR_ARG = 1,     /* null pointer, n < 0, bad predicate or predicate argument, misalignment */
    SSC_ERR_SIZE = 2,    /* n > INT32_MAX (the small-tile test build: n > 2^17 x 3840) */
    SSC_ERR_ALIAS = 3,   /* buffers overlap where they must not */
    SSC_ERR_SCRATCH = 4, /* scratch too small or not 8-byte aligned */
    SSC_ERR_HIP = 5,     /* a HIP call or kernel launch failed */
    SSC_ERR_DEVICE = 6   /* current device is not gfx950 with 64-wide wavefronts */
} ssc_status;

/* Predicate kinds. pa/pb are ignored where not listed.
 *   NONZERO    x != 0              zero removal ("Day 33 compaction.cu", markNonZero)
 *   ODD        (x & 1) == 1        ("CUDA Handbook ch. 13", Listing 13-17, isOdd)
 *   EVEN       (x & 1) == 0        ("Day 33 compaction.cu", markEven)
 *   BIT_SET    bit pa of x is 1    0 <= pa <= 31 (one split of an LSD radix sort,
 *   BIT_CLEAR  bit pa of x is 0      "CIS 565 Project 2: Stream Compaction")
 *   MOD_LT     r < pb where r is the non-negative residue of x modulo pa, pa >= 1
 * Bit tests use the two's-complement bits, so -3 is odd.
 * For fp32 arrays (the *_f32 calls; the compaction kernel of "CUDA Handbook
 * ch. 13" is a template over the element type), with thresholds a, b and
 * IEEE comparisons (every comparison with NaN is false, -0.0 == 0.0):
 *   F32_NONZERO  x != 0          (NaN is nonzero, -0.0 is zero)
 *   F32_GT       x > a
 *   F32_LT       x < a
 *   F32_IN       a <= x && x < b
 * The int32 calls take predicates 0..5 only and the fp32 calls 6..9. */
typedef enum ssc_pred {
    SSC_PRED_NONZERO = 0,
    SSC_PRED_ODD = 1,
    SSC_PRED_EVEN = 2,
    SSC_PRED_BIT_SET = 3,
    SSC_PRED_BIT_CLEAR = 4,
    SSC_PRED_MOD_LT = 5,
    SSC_PRED_F32_NONZERO = 6,
    SSC_PRED_F32_GT = 7,
    SSC_PRED_F32_LT = 8,
    SSC_PRED_F32_IN = 9
} ssc_pred;

/* Elements per tile: the share of the single pass behind one tile number
 * claimed from the atomic counter and one look-back descriptor (a workgroup
 * of the compaction kernel processes several tiles in turn). 30720; 3840 in
 * the library's small-tile test build (libssc_stress.so), which otherwise
 * has the same calls and results. */
int64_t ssc_tile_elems(void);

/* Scratch bytes needed by the scan, compaction, partition and counting calls
 * for n elements: a 512-byte header (tile counter and epoch, counting-pass
 * accumulators) plus 16 bytes of look-back descriptors per ssc_tile_elems()
 * elements (one 8-byte descriptor per tile; the fp32 scans use two, the
 * key-value and 64-bit compactions have tiles of half the size). */
size_t ssc_scratch_bytes(int64_t n);

/* Scratch bytes needed by ssc_radix_sort_u32 for n keys. */
size_t ssc_radix_sort_scratch_bytes(int64_t n);

/* Scratch bytes needed by ssc_radix_sort4_u32 for n keys: a scan scratch for
 * a 16 x ceil(n / 8192) table of per-tile digit counts, then the table. */
size_t ssc_radix_sort4_scratch_bytes(int64_t n);

/* Zero-fills a scratch buffer on `stream` (needed once, before first use,
 * and again after a time-out, see below). */
int ssc_scratch_init(void *scratch, size_t scratch_bytes, void *stream);

/* Stream-ordered check of a scratch buffer: writes 1 to *flag (a device
 * int32) if a look-back wait of a call made with this scratch gave up after
 * its bounded spin since the scratch was last initialised, else 0. A set
 * flag means those calls' results are invalid and the scratch needs
 * ssc_scratch_init before further use; it never comes from a correct call.
 * One tiny launch; flag must not lie inside the scratch. */
int ssc_scratch_timed_out(const void *scratch, size_t scratch_bytes, int32_t *flag, void *stream);

/* Exclusive scan of int32 values: out[0] = 0, out[i] = in[0] + ... + in[i-1],
 * with two's-complement wrap (sums taken modulo 2^32). `total` (nullable)
 * receives the sum of all n values. out == in is allowed (in place); any
 * other overlap of in/out/total is SSC_ERR_ALIAS.
 * Source: "Day 32 scan_2.cu" (scanExclusiveCpu) and the exclusive
 * convention of the "CIS 565 Project 2" transcript (0 13 50 ... for 13 37 15 ...). */
int ssc_exclusive_scan_i32(const int32_t *in, int32_t *out, int64_t n, int32_t *total,
                           void *scratch, size_t scratch_bytes, void *stream);

/* Exclusive scan of fp32 values. The prefix inside a tile (at most 30720
 * values) is summed in fp32 in a tiled order; the carries between tiles are
 * fp64, and each output is rounded to fp32 once from the fp64 sum of carry
 * and in-tile prefix, so the error does not grow with the number of tiles
 * (the double accumulation of "Day 32 scan_2.cu", scanExclusiveCpu, for the
 * part that spans tiles). Tested within 1e-6 relative of the exactly
 * accumulated prefix for non-negative values up to n = 2^27. Aliasing rules
 * as above. */
int ssc_exclusive_scan_f32(const float *in, float *out, int64_t n, float *total,
                           void *scratch, size_t scratch_bytes, void *stream);

/* Inclusive scan of int32 values: out[i] = in[0] + ... + in[i], with
 * two's-complement wrap; `total` (nullable) receives out[n-1] (0 for n = 0).
 * Aliasing rules as for the exclusive scan.
 * Source: "Day 31 scan.cu" (scanInclusiveCpu and the inclusive block scans;
 * here over the whole array, not restarted per tile). */
int ssc_inclusive_scan_i32(const int32_t *in, int32_t *out, int64_t n, int32_t *total,
                           void *scratch, size_t scratch_bytes, void *stream);

/* Inclusive scan of fp32 values, accumulated as the exclusive fp32 scan is;
 * same accuracy statement and aliasing rules. Source: "Day 31 scan.cu". */
int ssc_inclusive_scan_f32(const float *in, float *out, int64_t n, float *total,
                           void *scratch, size_t scratch_bytes, void *stream);

/* Order-preserving compaction: out[0 .. count) = the elements x with P(x)
 * true, in input order; *count = their number (the top of the scan of the
 * flags). `ranks` (nullable) receives the exclusive scan of the flags for
 * every i: the output slot of in[i] when it survives. No overlap between
 * in, out, count and ranks is allowed.
 * Source: "Day 33 compaction.cu" (compactCpu, scatterCompact) and
 * "CUDA Handbook ch. 13" (Listing 13-17: survivors scattered to
 * base + index within the tile; the last tile writes the total). */
int ssc_compact_i32(const int32_t *in, int32_t *out, int64_t n, int pred, int32_t pa,
                    int32_t pb, int32_t *count, int32_t *ranks, void *scratch,
                    size_t scratch_bytes, void *stream);

/* ssc_compact_i32 without a scratch argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc). Same arguments, results, errors and
 * kernels as ssc_compact_i32; nothing is allocated or freed: the scratch is a
 * library-owned device array of 1,119,232 bytes on each GPU (enough for every
 * n up to INT32_MAX; a larger scratch need would give SSC_ERR_SIZE), held
 * until the process ends. Its address is looked up and the array zero-filled
 * by one clearing kernel on `stream` at the first call on a device; later
 * calls reuse it as left by the previous call, which keeps it ready. All
 * calls on one GPU share that one array, so calls that may run at the same
 * time on one GPU (other streams, other host threads) race and give wrong
 * results: serialise them. */
int ssc_compact_i32_noalloc(const int32_t *in, int32_t *out, int64_t n, int pred, int32_t pa,
                            int32_t pb, int32_t *count, int32_t *ranks, void *stream);

/* ssc_compact_i32 for fp32 arrays with an fp32 predicate (6..9) and its
 * thresholds a, b; values move bit for bit (-0.0 and NaN payloads kept). */
int ssc_compact_f32(const float *in, float *out, int64_t n, int pred, float a, float b,
                    int32_t *count, int32_t *ranks, void *scratch, size_t scratch_bytes,
                    void *stream);

/* Selection (the index form of compaction): idx[0 .. count) = the
 * positions i, increasing, of the elements with P(in[i]) true; *count =
 * their number. idx[count .. n) is not written. Same single pass as
 * ssc_compact_i32, with each survivor's index scattered instead of its
 * value. No overlap between in, idx and count is allowed.
 * Source: "CUDA Handbook ch. 13, Stream Compaction" (the exclusive scan of
 * the flags gives each kept element its output position). */
int ssc_select_index_i32(const int32_t *in, int32_t *idx, int64_t n, int pred, int32_t pa,
                         int32_t pb, int32_t *count, void *scratch, size_t scratch_bytes,
                         void *stream);

/* ssc_select_index_i32 for fp32 arrays with an fp32 predicate (6..9). */
int ssc_select_index_f32(const float *in, int32_t *idx, int64_t n, int pred, float a, float b,
                         int32_t *count, void *scratch, size_t scratch_bytes, void *stream);

/* Stable partition: out[0 .. K) = the elements with P true, out[K .. n) =
 * the elements with P false, both in input order; *count = K. Kept x[i]
 * goes to out[rank[i]], rejected x[i] to out[K + i - rank[i]], where rank
 * is the exclusive scan of the flags. K is counted first by a reduction
 * pass over the input (written to *count), then one single pass scans and
 * scatters: two launches. No overlap between in, out and count is allowed.
 * Source: "Day 33 compaction.cu" (partitionCpu, scatterPartition). */
int ssc_partition_i32(const int32_t *in, int32_t *out, int64_t n, int pred, int32_t pa,
                      int32_t pb, int32_t *count, void *scratch, size_t scratch_bytes,
                      void *stream);

/* ssc_partition_i32 for fp32 arrays with an fp32 predicate (6..9). */
int ssc_partition_f32(const float *in, float *out, int64_t n, int pred, float a, float b,
                      int32_t *count, void *scratch, size_t scratch_bytes, void *stream);

/* Compaction by a caller's own predicate, given as one flag byte per
 * element: out[0 .. count) = the 32-bit elements in[i] (int32, fp32 or any
 * 4-byte type, moved bit for bit) whose flags[i] is nonzero, in input
 * order; *count = their number; out[count .. n) is not written. Same single
 * pass as ssc_compact_i32, the flags read in place of a predicate.
 * flags must be 4-byte aligned: the library reads it in 32-bit words,
 * including the whole word that holds flags[n - 1] (never past that word).
 * No overlap between in, flags, out and count is allowed.
 * Source: "Day 33 compaction.cu" (the predicate is the only part that
 * changes; everything after it reads an array of ones and zeros). */
int ssc_compact_flags_b32(const void *in, const uint8_t *flags, void *out, int64_t n,
                          int32_t *count, void *scratch, size_t scratch_bytes, void *stream);

/* Positions of the nonzero flag bytes: idx[0 .. count) = the i, increasing,
 * with flags[i] != 0; *count = their number (the flag-byte form of
 * ssc_select_index_i32; same alignment rule for flags). A 16-byte aligned
 * flag array is read in 128-bit words by a kernel with 61,440-flag tiles
 * (faster: each tile carries twice the bytes per look-back); it too
 * reads nothing past the 32-bit word that holds flags[n - 1]. No overlap
 * between flags, idx and count is allowed. Source: as ssc_compact_flags_b32. */
int ssc_select_flags(const uint8_t *flags, int32_t *idx, int64_t n, int32_t *count,
                     void *scratch, size_t scratch_bytes, void *stream);

/* Key-value compaction: the pairs (keys[i], vals[i]) whose key satisfies the
 * predicate (pred 0..5 with pa, pb as in ssc_compact_i32), in input order:
 * keys_out[0 .. count) and vals_out[0 .. count) hold the same positions;
 * *count = their number. Values are 4-byte words moved bit for bit. One
 * single pass over both arrays (1024 pairs per wavefront and tile). No
 * overlap between any two of keys, vals, keys_out, vals_out and count.
 * Source: the element-type template of "CUDA Handbook ch. 13, Stream
 * Compaction", with a value carried beside each kept key. */
int ssc_compact_kv_i32(const int32_t *keys, const void *vals, int32_t *keys_out, void *vals_out,
                       int64_t n, int pred, int32_t pa, int32_t pb, int32_t *count,
                       void *scratch, size_t scratch_bytes, void *stream);

/* ssc_compact_kv_i32 with fp32 keys and an fp32 predicate (6..9). */
int ssc_compact_kv_f32(const float *keys, const void *vals, float *keys_out, void *vals_out,
                       int64_t n, int pred, float a, float b, int32_t *count, void *scratch,
                       size_t scratch_bytes, void *stream);

/* Compaction of 64-bit elements (int64 or uint64 bits): out[0 .. count) =
 * the elements with P true in input order; *count = their number. P is
 * NONZERO, ODD, EVEN, BIT_SET or BIT_CLEAR on the 64 bits of the value, the
 * bit 0..63 given in `bit`; MOD_LT and the fp32 predicates give
 * SSC_ERR_ARG. in and out must be 8-byte aligned. One single pass (1024
 * elements per wavefront and tile). No overlap between in, out and count.
 * Source: "CUDA Handbook ch. 13, Stream Compaction" (Listing 13-17 is a
 * template over the element type; isOdd is x & 1). */
int ssc_compact_i64(const int64_t *in, int64_t *out, int64_t n, int pred, int32_t bit,
                    int32_t *count, void *scratch, size_t scratch_bytes, void *stream);

/* Selection over 64-bit elements: idx[0 .. count) = the positions i with
 * P(in[i]) true (predicates as ssc_compact_i64). No overlap between in, idx
 * and count. */
int ssc_select_index_i64(const int64_t *in, int32_t *idx, int64_t n, int pred, int32_t bit,
                         int32_t *count, void *scratch, size_t scratch_bytes, void *stream);

/* *count = number of elements with P true (a reduction of the flags; one
 * launch). Needs a scratch buffer of at least ssc_scratch_bytes(0) bytes. */
int ssc_count_if_i32(const int32_t *in, int64_t n, int pred, int32_t pa, int32_t pb,
                     int32_t *count, void *scratch, size_t scratch_bytes, void *stream);

/* Unordered compaction by atomic counter, kept only for comparison (it
 * needs no scratch: its counter is *count itself):
 * out[0 .. count) holds the same multiset as ssc_compact_i32's output, in
 * an order the hardware scheduler decides. variant 0: one atomicAdd per
 * 512-thread workgroup and 8192-element tile (its survivors keep tile
 * order inside the reserved range); variant 1: one atomicAdd per
 * survivor (the form of "Day 33 compaction.cu", compactAtomic). *count is
 * cleared and used as the counter. No overlap between in, out and count. */
int ssc_compact_atomic_i32(const int32_t *in, int32_t *out, int64_t n, int pred, int32_t pa,
                           int32_t pb, int32_t *count, int variant, void *stream);

/* LSD radix sort of uint32 keys as 32 chained stable 1-bit partitions,
 * pass b keeping keys whose bit b is clear first (bit 0 first), leaving
 * out[] ascending. One counting pass over the input gives the size of the
 * first half for every bit at once (a permutation does not change how many
 * keys have bit b clear). tmp is n words of caller workspace; in is not
 * modified. out == in is allowed; tmp must not overlap in or out.
 * Source: "CIS 565 Project 2: Stream Compaction" (radix sort built on the
 * compaction primitives, checked against std::sort). */
int ssc_radix_sort_u32(const uint32_t *in, uint32_t *out, uint32_t *tmp, int64_t n,
                       void *scratch, size_t scratch_bytes, void *stream);

/* LSD radix sort of uint32 keys with 4-bit digits: `passes` (1..8) stable
 * 16-way splits, pass p by digit (x >> 4p) & 15, so out[] ends stably sorted
 * by the low 4*passes bits of the keys (passes = 8: ascending). One 4-bit
 * split gives the same order as the four 1-bit splits of those bits in
 * ssc_radix_sort_u32, each a stable partition by a bit-test predicate. Each
 * pass: per-tile digit counts (tiles of 8192 keys), one exclusive scan of
 * the digit-major count table (the single-pass scan), then a stable scatter
 * in 16 contiguous runs per tile. tmp is n words of caller workspace; in is
 * not modified. out == in is allowed when passes is even; tmp must not
 * overlap in or out. passes outside 1..8 is SSC_ERR_ARG.
 * Source: "CIS 565 Project 2: Stream Compaction" (radix sort built on
 * split, LSD bit order); the digit width is this library's. */
int ssc_radix_sort4_u32(const uint32_t *in, uint32_t *out, uint32_t *tmp, int64_t n, int passes,
                        void *scratch, size_t scratch_bytes, void *stream);

/* Comparison only: the multi-launch structure of the pages, ported so that
 * the single pass can be measured against it on this hardware. A scan is a
 * tree of tile scans (8192-element tiles; each level writes its tiles'
 * exclusive prefixes and one sum per tile, and the next level scans the
 * sums) with the carries added back level by level: 3 launches up to
 * 8192^2 elements ("Day 32 scan_2.cu": tile scan, scan of the tile sums,
 * add the offsets). A compaction marks the flags into `ranks`, scans them
 * there with that tree and scatters the survivors to out[rank], recomputing
 * the predicate: 7 launches at 2^28 elements ("Day 33 compaction.cu": mark,
 * scan, scatter). `ranks` (required, n words) ends as the exclusive scan of
 * the flags. Results equal those of ssc_exclusive_scan_i32 and
 * ssc_compact_i32; scratch (16-byte aligned, ssc_multipass_scratch_bytes
 * bytes) holds the tile sums; no overlap of the arrays is allowed, except
 * in == out for the scan. */
size_t ssc_multipass_scratch_bytes(int64_t n);
int ssc_exclusive_scan_multipass_i32(const int32_t *in, int32_t *out, int64_t n, int32_t *total,
                                     void *scratch, size_t scratch_bytes, void *stream);
int ssc_compact_multipass_i32(const int32_t *in, int32_t *out, int64_t n, int pred, int32_t pa,
                              int32_t pb, int32_t *count, int32_t *ranks, void *scratch,
                              size_t scratch_bytes, void *stream);

/* Comparison only, the separate steps of that multi-launch compaction, so
 * that each can be timed alone ("Day 33 compaction.cu", markNonZero /
 * markEven and scatterCompact, and its table of where the time goes):
 * ssc_mark_i32 writes flags[i] = P(in[i]) (0 or 1) for every i;
 * ssc_scatter_i32 writes out[ranks[i]] = in[i] for every i with P(in[i])
 * (the predicate evaluated again, not read back) given the exclusive scan
 * of the flags in `ranks`, and *count = ranks[n-1] + P(in[n-1]). A rank
 * outside [0, n) is skipped. No overlap of the arrays is allowed. */
int ssc_mark_i32(const int32_t *in, int32_t *flags, int64_t n, int pred, int32_t pa, int32_t pb,
                 void *stream);
int ssc_scatter_i32(const int32_t *in, const int32_t *ranks, int32_t *out, int64_t n, int pred,
                    int32_t pa, int32_t pb, int32_t *count, void *stream);

/* out[i] = in[i] with 128-bit nontemporal loads and stores (32-bit ones when
 * either array is not 16-byte aligned), one 256-thread workgroup per 4096
 * elements: the bandwidth reference the single pass is compared with ("Day
 * 33 compaction.cu", copyInts; "Day 32 scan_2.cu", copyFloats). No overlap
 * allowed. */
int ssc_copy_i32(const int32_t *in, int32_t *out, int64_t n, void *stream);

/* ------------------------------------------------------------------------
 * Rows moved by a key, and the choice of the next token: the same work
 * (flags or keys, counts, scans, stable placement, selection) for the token
 * path of a language model. Element types of rows: */
typedef enum ssc_dtype {
    SSC_F32 = 0,
    SSC_BF16 = 1,
    SSC_F16 = 2
} ssc_dtype;
/* Conventions of these calls beside the shared ones above:
 *   - Rows are contiguous, `width` elements (1 <= width <= 2^28) of one
 *     type; arrays need the alignment of their element only.
 *   - Row, token and group counts are at most INT32_MAX (groups and vocab of
 *     the grouping and the gradient: INT32_MAX - 1); larger ones give
 *     SSC_ERR_SIZE.
 *   - Scratch is 16-byte aligned, needs no initialisation and keeps nothing
 *     between calls; one buffer must not serve two calls that may run at the same time. Where
 *     the size function returns 0 it may be NULL.
 *   - Ids, ranks and positions read from device memory are checked there: one
 *     out of its range moves nothing and adds nothing, and nothing outside the
 *     arrays is touched.
 *   - Inputs may overlap each other; an output must not overlap any other
 *     array of the call (SSC_ERR_ALIAS).
 *   - Sums are held in fp32 and rounded to the output's type once; their order
 *     depends on the sizes and the ranks only, so a call repeats bit for bit.
 */

/* Scratch bytes of a grouping of n keys (0 for up to 8192 keys of at most
 * 4096 groups). */
size_t ssc_group_scratch_bytes(int64_t n, int64_t groups);

/* Stable partition into `groups` groups: key k belongs to group k, and one
 * outside [0, groups) to none (give -1 for padding or a dropped assignment).
 *   offsets[g] = keys of groups below g, for g in [0, groups]; the last
 *                entry is the number of keys that belong to a group
 *   ranks[i]   = the slot of key i: offsets[keys[i]] + equal keys before i;
 *                -1 for a key of no group                        (nullable)
 *   order[s]   = the i with ranks[i] = s, for s < offsets[groups]; the
 *                entries past that are not written               (nullable)
 * The many-way form of ssc_partition_i32: one counting and one scattering
 * step per 9 bits of group number (a single launch for up to 8192 keys of at
 * most 4096 groups). */
int ssc_group_by_key_i32(const int32_t *keys, int64_t n, int64_t groups, int32_t *order,
                         int32_t *ranks, int32_t *offsets, void *scratch, size_t scratch_bytes,
                         void *stream);
int ssc_group_by_key_i64(const int64_t *keys, int64_t n, int64_t groups, int32_t *order,
                         int32_t *ranks, int32_t *offsets, void *scratch, size_t scratch_bytes,
                         void *stream);

/* Embedding lookup: out[i] = scale * table[ids[i]] for n ids, the table
 * holding `vocab` rows; an id outside [0, vocab) gives a row of zeros. */
int ssc_embed_rows_i32(const void *table, int dtype, int64_t vocab, int64_t width,
                       const int32_t *ids, int64_t n, float scale, void *out, void *stream);
int ssc_embed_rows_i64(const void *table, int dtype, int64_t vocab, int64_t width,
                       const int64_t *ids, int64_t n, float scale, void *out, void *stream);

/* Scratch bytes of the embedding's gradient: fp32 sums of blocks of 16, 256
 * and 4096 sorted tokens (0 for fewer than 256 tokens). */
size_t ssc_embed_grad_scratch_bytes(int64_t n, int64_t width);

/* Gradient of the lookup with respect to the table, by sorted tokens:
 * grad[v] = scale * (sum of dout[i] over all i with ids[i] = v), given the
 * grouping of these ids (`order` and `offsets` of ssc_group_by_key with groups
 * = vocab). accumulate = 0 writes every row of grad, zeros where no token
 * has the id; otherwise the sum is added to the row, and rows without tokens
 * are not touched. grad_dtype is dtype or SSC_F32. */
int ssc_embed_rows_grad_i32(const void *dout, int dtype, int64_t n, int64_t width,
                            const int32_t *ids, const int32_t *order, const int32_t *offsets,
                            int64_t vocab, float scale, void *grad, int grad_dtype, int accumulate,
                            void *scratch, size_t scratch_bytes, void *stream);
int ssc_embed_rows_grad_i64(const void *dout, int dtype, int64_t n, int64_t width,
                            const int64_t *ids, const int32_t *order, const int32_t *offsets,
                            int64_t vocab, float scale, void *grad, int grad_dtype, int accumulate,
                            void *scratch, size_t scratch_bytes, void *stream);

/* Rows to their groups: out[ranks[t, k]] = x[t] for t < tokens, k < per, with
 * ranks (tokens x per, distinct, as the grouping of the tokens' expert ids
 * gives them) below `rows`, the rows of out; rows that no rank names are not
 * written. Its gradient is ssc_combine_rows without weights. */
int ssc_dispatch_rows(const void *x, int dtype, int64_t tokens, int64_t per, int64_t width,
                      const int32_t *ranks, int64_t rows, void *out, void *stream);

/* Rows back from their groups: out[t] = sum over k of weights[t, k] *
 * y[ranks[t, k]] (weights nullable: all one). A rank outside [0, rows) adds
 * nothing; a token with no rank inside gets a row of zeros. */
int ssc_combine_rows(const void *y, int dtype, int64_t rows, int64_t width, const int32_t *ranks,
                     const float *weights, int64_t tokens, int64_t per, void *out, void *stream);

/* Gradients of ssc_combine_rows: dy[ranks[t, k]] = weights[t, k] * dout[t] and
 * dweights[t, k] = <dout[t], y[ranks[t, k]]> (0 for a rank outside); rows of dy
 * that no rank names are not written. One pass over dout and y. Ranks must be
 * distinct. */
int ssc_combine_rows_grad(const void *dout, const void *y, int dtype, int64_t rows, int64_t width,
                          const int32_t *ranks, const float *weights, int64_t tokens, int64_t per,
                          void *dy, float *dweights, void *stream);

/* Scratch bytes of ssc_sample_rows: about 56 KiB a row and 20 bytes for each
 * 4096 logits of it, whatever the filters. */
size_t ssc_sample_scratch_bytes(int64_t rows, int64_t vocab);

/* The next token of each row of logits (row r at logits + r * stride
 * elements, stride >= vocab), from a given random number u[r] in [0, 1). With
 * the row's tokens ordered by logit, largest first, equal ones by index, and
 * w_i = exp((logit_i - largest) / temperature), the kept tokens are
 *   the first top_k of the order (top_k < 1: all);
 *   of these, each one before which the weights sum to less than top_p times
 *     the sum over all of them (top_p >= 1: all);
 *   of these, those with w_i >= min_p;
 * and always the first of the order. tokens[r] is the first index, in index
 * order, at which the running sum of the kept weights exceeds u[r] times their
 * sum. A temperature that is not above 0 keeps the first of the order alone.
 * A logit of NaN or -infinity is no token, and beside one of +infinity no
 * other is (those of +infinity weigh the same). A row with no token gives
 * tokens[r] = -1, kept[r] = 0, logprobs[r] = -infinity. A u outside [0, 1) is
 * taken as the nearest end (NaN as 0), a top_p of NaN as 1, of 0 or less as one
 * that keeps the first only, a min_p of NaN as 0. No weight reaches a min_p
 * above 1, which so keeps the first only, too.
 * The settings are arrays of one value a row, each nullable: temperature 1,
 * no top_k, no top_p, no min_p. kept[r] (nullable) is the number of kept
 * tokens, logprobs[r] (nullable) the logarithm of the chosen weight over the
 * kept ones' sum. Weights are computed in fp64 and summed as fixed-point
 * integers, so that neither the order of a sum nor the split of a row changes
 * a result: of 62 - ceil(log2(vocab + 1)) fractional bits, at most 50, where
 * the largest weight is 1. Each is off by half the last bit and, by its fp64
 * exponential, by less than 2^-46 (the largest, and those equal to it, by
 * nothing), so a sum over the row by vocab times that at most, and a border of
 * top_p or u that lies as near a running sum may fall on either side of it:
 * 2^-28 of the largest weight for 131,072 logits, 2^-18 for 2^22, where
 * rounding all goes one way.
 * 1 <= vocab <= 2^22 and at most 65,535 rows. */
int ssc_sample_rows(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                    const float *u, const float *temperature, const int32_t *top_k,
                    const float *top_p, const float *min_p, int32_t *tokens, int32_t *kept,
                    float *logprobs, void *scratch, size_t scratch_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Before the grouping: the router of a mixture of experts. Conventions of the
 * row calls above; rows of logits may lie apart (row t at logits + t * stride
 * elements, stride >= experts). 1 <= experts <= 1024, 1 <= per <= experts and
 * per <= 64. */

/* Scratch bytes of ssc_route_rows with its balance (0 without, and for up to 64
 * tokens, up to 512 of fewer than 129 experts). */
size_t ssc_route_scratch_bytes(int64_t tokens, int64_t experts);

/* The experts of each token: ids[t, :] (tokens x per) are the experts of its
 * `per` largest logits, largest first, equal ones by index, and weights[t, :]
 * their shares of the softmax over the row, with `normalize` divided by their
 * sum. A logit of NaN or -infinity is no expert, and beside one of +infinity no
 * other is (those of +infinity weigh the same); places that a row has no expert
 * for get id -1 and weight 0. A token with live[t] == 0 (nullable: all live) has
 * no expert.
 * The balance (counts, share and loss, all three or none) over the n tokens with
 * an expert, p their softmax:
 *   counts[e]  = assignments of expert e, for e < experts; counts[experts] = n
 *   share[e]   = mean of p[t, e] over them (0 for n = 0)
 *   loss       = experts * sum over e of counts[e] / (per * n) * share[e]: 1 where
 *                tokens fall evenly (0 for n = 0)
 * What a workgroup adds up is fp32: up to 64 rows of a lane, then its lanes and
 * wavefronts, up to 8192 tokens of up to 128 experts; sums of workgroups are fp64.
 * What lies between rows that are apart counts as theirs: no output may lie there. */
int ssc_route_rows(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t stride,
                   const uint8_t *live, int64_t per, int normalize, int32_t *ids, float *weights,
                   int32_t *counts, float *share, float *loss, void *scratch, size_t scratch_bytes,
                   void *stream);

/* The gradient with respect to the logits (dlogits: tokens x experts of dtype,
 * contiguous) of <dweights, weights> + dloss * loss, given the ids that
 * ssc_route_rows gave. dweights (with ids) and dloss (one value in device memory,
 * with counts) are nullable, each for 0. counts may be those of several calls
 * added up, n among them: the loss is then that of all of them. As in the
 * forward pass, counts are constants. Ids outside [0, experts) add nothing, one
 * that a row names twice counts twice; rows of tokens that are not live or have no
 * expert are zeros. */
int ssc_route_rows_grad(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t stride,
                        const uint8_t *live, const int32_t *ids, int64_t per, int normalize,
                        const float *dweights, const int32_t *counts, const float *dloss,
                        void *dlogits, void *stream);

/* ------------------------------------------------------------------------
 * After the choice of tokens: drafts verified. */

/* Scratch bytes of ssc_verify_rows: about 8 for each 1024 tokens of the
 * vocabulary and row; 0 up to 65,536 tokens, and for 160 rows or more up to
 * 131,072. */
size_t ssc_verify_scratch_bytes(int64_t rows, int64_t vocab);

/* Drafted tokens held against the probabilities of the model that they were
 * drafted for. probs holds drafts + 1 rows of `vocab` probabilities for each of
 * `rows` sequences (row i of sequence b at probs + b * stride_row + i *
 * stride_place elements), draft_probs the `drafts` rows that the drafts were drawn
 * by, with strides of its own (nullable: drafted without chance, probability 1);
 * drafted is rows x drafts, u rows x (drafts + 1) of [0, 1). lengths[b] (nullable:
 * drafts) is the number of drafts of a sequence, held to [0, drafts].
 * Draft i stands if all before it do and u[b, i] * q_i(x_i) < p_i(x_i); a token
 * outside the vocabulary falls. With a the number that stand, one more token is
 * drawn by weights w: max(p_a - q_a, 0) where draft a fell (p_a without x_a if
 * draft_probs is NULL; p_a, where none of these is above 0), p_a where all stood. It
 * is the first index at which the running sum of w exceeds u[b, drafts] times
 * their sum. Then
 *   tokens[b, :]  = the a drafts, the drawn token, -1 for the rest (rows x (drafts + 1))
 *   accepted[b]   = a
 * Probabilities need not sum to 1; what is not above 0 or not finite weighs
 * nothing, and a sequence without weights draws -1. A u outside [0, 1) is taken as
 * the nearest in it (NaN as 0). Products, differences and sums are fp64, in an
 * order that the sizes fix: a border that lies within some 2^-50 of their sum may fall on
 * either side. 1 <= vocab <= 2^22, at most 65,535 rows and 2^20 drafts. */
int ssc_verify_rows_i32(const void *probs, int dtype, int64_t rows, int64_t drafts, int64_t vocab,
                        int64_t stride_row, int64_t stride_place, const int32_t *drafted,
                        const void *draft_probs, int64_t draft_stride_row, int64_t draft_stride_place,
                        const float *u, const int32_t *lengths, int32_t *tokens, int32_t *accepted,
                        void *scratch, size_t scratch_bytes, void *stream);
int ssc_verify_rows_i64(const void *probs, int dtype, int64_t rows, int64_t drafts, int64_t vocab,
                        int64_t stride_row, int64_t stride_place, const int64_t *drafted,
                        const void *draft_probs, int64_t draft_stride_row, int64_t draft_stride_place,
                        const float *u, const int32_t *lengths, int32_t *tokens, int32_t *accepted,
                        void *scratch, size_t scratch_bytes, void *stream);

/* ------------------------------------------------------------------------
 * A cache cut to the rows that were attended to most. Caches are batch x heads x
 * capacity (x width) with strides in elements for all but the last dimension,
 * which is contiguous; strides are not negative, and what a call writes does not
 * overlap itself. A view counts from its first element to its last where overlaps
 * are checked, the gaps between its rows with it. At most 65,535 batch * heads and
 * 2^31 - 4097 positions.
 * lengths[b] (nullable: all) is the number of positions in use, held to what there
 * is. */

/* Scratch bytes of ssc_accumulate_weights: sums of the parts that the rows (group *
 * queries) of a few short heads are added up in; 0 otherwise, and for up to 128 rows. */
size_t ssc_accumulate_scratch_bytes(int64_t batch, int64_t heads, int64_t group, int64_t queries,
                                    int64_t length, int dtype);

/* The attention weights that each cached position got, added up: for i <
 * min(length, lengths[b])
 *   scores[b, h, i] = decay * scores[b, h, i] + sum of weights[b, g, q, i]
 * over the heads g in [h * group, (h + 1) * group) and all queries. Of the last
 * `fresh` of these positions (new ones) the score is not read but taken as 0.
 * Positions past them are left as they were. A weight of NaN adds nothing. weights
 * is batch x (heads * group) x queries x length, length <= capacity. Each score is
 * within 26 half steps of fp32 (2^-24 of the sum of the magnitudes that it is made
 * of), for any number of rows (group * queries, up to 2^30). */
int ssc_accumulate_weights(float *scores, int64_t batch, int64_t heads, int64_t capacity,
                           int64_t score_stride_batch, int64_t score_stride_head, const void *weights,
                           int dtype, int64_t group, int64_t queries, int64_t length,
                           int64_t weight_stride_batch, int64_t weight_stride_head,
                           int64_t weight_stride_query, const int32_t *lengths, int64_t fresh,
                           float decay, void *scratch, size_t scratch_bytes, void *stream);

/* Scratch bytes of ssc_evict_rows (0 for up to 16,384 positions, and up to 32,768
 * of many heads): 4 for each position, and 16 KiB for each 8192 positions of a few
 * heads, or each 32,768 of many. */
size_t ssc_evict_scratch_bytes(int64_t batch, int64_t heads, int64_t capacity);

/* The positions that stay when every head is cut to `keep` rows: kept (batch x
 * heads x keep, contiguous) holds them increasing, -1 behind them, and counts
 * (batch x heads) their number. A sequence of up to `keep` positions keeps all; a
 * longer one its `first` first and `recent` last, and of the others those with the
 * largest scores, of equal ones the first (NaN is the lowest). first + recent <=
 * keep <= capacity, keep >= 1. The selection and compaction of
 * ssc_select_index_f32 with a threshold that is found. */
int ssc_evict_rows(const float *scores, int64_t batch, int64_t heads, int64_t capacity,
                   int64_t score_stride_batch, int64_t score_stride_head, const int32_t *lengths,
                   int64_t keep, int64_t first, int64_t recent, int32_t *kept, int32_t *counts,
                   void *scratch, size_t scratch_bytes, void *stream);

/* Scratch bytes of ssc_move_rows in place: those of all keep rows of every head,
 * where a few long heads go by way of it (as many bytes as the cache keeps); 0
 * otherwise, and for a move to another cache. */
size_t ssc_move_scratch_bytes(int elem_bytes, int64_t batch, int64_t heads, int64_t keep, int64_t width);

/* Rows of a cache moved together: out[b, h, s, :] = cache[b, h, kept[b, h, s], :]
 * for s < keep (1 to capacity), bit for bit, for elements of 1, 2, 4 or 8 bytes.
 * Slots whose position lies outside [0, capacity) are not written. out may be the
 * cache itself (the same address and strides): then positions that lie before their
 * slot, which ssc_evict_rows gives none of, are not moved. Any other overlap is an
 * error. */
int ssc_move_rows(const void *cache, int elem_bytes, int64_t batch, int64_t heads, int64_t capacity,
                  int64_t width, int64_t cache_stride_batch, int64_t cache_stride_head,
                  int64_t cache_stride_row, const int32_t *kept, int64_t keep, void *out,
                  int64_t out_stride_batch, int64_t out_stride_head, int64_t out_stride_row,
                  void *scratch, size_t scratch_bytes, void *stream);

/* Human-readable name of a status code (static storage). */
const char *ssc_status_str(int status);

/* The hipError_t of the last SSC_ERR_HIP on the calling thread (0 if none). */
int ssc_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SSC_H */
