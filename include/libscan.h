/*
 * libscan.h -- device-wide prefix scan and stream compaction for AMD MI355X (gfx950).
 *
 * C ABI: plain pointers and sizes, no C++ or framework types.  Unless marked
 * "host", every pointer is a device pointer (memory from hipMalloc or an
 * allocator built on it) on the device that is current when the call is made.
 *
 * Sources of the operations (page title and section):
 *   [Scan3]  geek-doc.cn, "并行前缀和 scan: Hillis-Steele、Blelloch 与 warp shuffle
 *            三种写法": section 一 (inclusive and exclusive scan, the total, and
 *            compaction by an exclusive scan of predicate flags), 四 (scans larger
 *            than one block), 五 (warp-level scan), pitfall list.
 *   [Blog2]  lpnh.cn/news/2866224, parallel scan overview: section 3.3 (a generic
 *            parallel_scan(in, out, n, op) over any associative operator), 4.1
 *            (compaction: flags, scan, scatter), 5.3 (work issued on streams),
 *            7.2 (segmented scans).
 *   [SIMT3]  pgsm.cn/news/414823, "SIMT数据依赖与并行前缀和：从原理到流压缩实战":
 *            section 4.2 (compaction writes the kept elements in order and a count
 *            computed on the device).
 *
 * Common rules for every entry point
 *   - Calls are asynchronous: work is enqueued on `stream` (a hipStream_t passed
 *     as void*; NULL = the null stream) and the call returns without waiting.
 *     Faults during execution surface at the caller's next synchronisation.
 *   - Arguments are validated on the host before anything is enqueued.  On a
 *     non-LS_OK status nothing has been enqueued and no output is written.
 *   - The caller owns every buffer.  The library allocates and frees nothing
 *     and never synchronises.
 *   - Element buffers must be 4-byte aligned.  16-byte alignment of `in` and
 *     `out` enables 128-bit loads and stores; other alignments are accepted and
 *     run a slower path.
 *   - Concurrent calls must use distinct workspaces; calls that share a
 *     workspace on different streams race.  So do calls that share one on the
 *     same stream, if several host threads enqueue them at the same time: some
 *     calls are several kernels, which must not stand between another call's.
 *
 * Workspaces
 *   The scans, segmented scans, compactions and the radix sort take a caller's
 *   device workspace of at least the size that the matching *_workspace_bytes
 *   query returns.  Inside a call, tiles hand their results on through tile
 *   status words in the workspace ([Scan3] 四: blocks passing their totals on
 *   through flags in global memory; [SIMT3] 5.1: flags published with fences).
 *   - Status workspaces, of the single-pass scans (scan_inclusive,
 *     scan_exclusive, scan_ex with a single-pass scheme), segmented scans and
 *     compactions: zero-filled once before first use, by ls_workspace_init (or
 *     any zero fill of the whole buffer; one that is only captured into a graph
 *     counts for that graph's calls alone).  Every call leaves the workspace ready
 *     for the next, so calls enqueue no clearing work of their own.  Between
 *     calls its contents must not change, and it must serve no other purpose: a
 *     status workspace used by a radix sort or a three-phase scan_ex, or written
 *     in any other way, must be initialised again.  Apart from that it may serve
 *     any sequence of these calls, of any sizes it is large enough for, up to
 *     2^26 calls: the words carry the call's epoch, compared modulo 2^26, so
 *     initialise it again before that many calls (the Python binding does so
 *     every 2^25).
 *   - The radix sort and the three-phase scan_ex schemes use their workspace as
 *     plain scratch: its contents on entry do not matter.  (For the sort's error
 *     word to be meaningful, initialise its workspace once.)
 *   - sample_tokens and the recurrence calls have workspaces of their own, zero-filled
 *     once, as their documentation says; experts_sort's is plain scratch.
 *   Each wait for another tile is bounded in time.  The single-pass scans
 *   (except the deterministic scheme) and the compactions take tiles by block
 *   index: a tile that has waited about a millisecond computes what it waited
 *   for from the input itself, and the result stays exact.  The deterministic
 *   scan, the segmented scans and the recurrence take tile ids in the order blocks
 *   start: a wait there gives up after about one second, the call's output is then
 *   incomplete, and the workspace records the fact; so does a call whose last
 *   tile waits more than about ten seconds for the other blocks to start.
 *   ls_workspace_check reports it.  In a correct run no wait lasts more than
 *   microseconds.
 */
#ifndef LIBSCAN_H
#define LIBSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LS_ABI_VERSION 5

/* Largest element count of the scans, segmented scans and the radix sort (tile ids
 * are 32 bits), and of the compaction family (its counts travel in 36 bits). */
#define LS_MAX_N (1LL << 40)
#define LS_COMPACT_MAX_N ((1LL << 36) - 1)

typedef enum ls_status {
    LS_OK = 0,
    LS_ERR_INVALID_ARG = 1, /* bad size, NULL, alignment, enum value, or overlap */
    LS_ERR_UNSUPPORTED = 2, /* an operator not defined for the element type (see ls_op); a recurrence of too many tiles */
    LS_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than the size query returned */
    LS_ERR_HIP = 4,         /* the HIP runtime reported an error when enqueuing */
    LS_ERR_INCOMPLETE = 5   /* ls_workspace_check: a call on the workspace gave up a wait */
} ls_status;

/* Element types.  All are 32 bits wide. */
typedef enum ls_dtype { LS_INT32 = 0, LS_UINT32 = 1, LS_FLOAT32 = 2 } ls_dtype;

/* Associative operators ([Scan3] 一 and 三; [Blog2] 3.3), combined as
 * op(earlier, later), left to right.
 *   LS_SUM     int32/uint32: addition modulo 2^32 (two's complement wrap);
 *              float32: IEEE addition; association order is the library's, so
 *              results may differ from a serial sum in the last bits ([Scan3]
 *              pitfall list).  The order depends only on n and the scheme, so
 *              they are the same bits on every run.
 *   LS_MAX     int32 signed, uint32 unsigned, float32 (a > b) ? a : b, which on a
 *              tie keeps the later element; bit-exact and run-to-run identical
 *              for data without NaN.  NaN inputs give unspecified results.
 *   LS_XOR     int32/uint32 bitwise; float32 -> LS_ERR_UNSUPPORTED.
 *   LS_MIN     as LS_MAX with (a < b) ? a : b (ties keep the later element).
 *   LS_AND, LS_OR  int32/uint32 bitwise ([Blog2] 3.3: logical AND/OR);
 *              float32 -> LS_ERR_UNSUPPORTED.
 *   LS_PROD    int32/uint32: multiplication modulo 2^32; float32: IEEE product
 *              (relative error up to about (i+1) * 2^-24 at element i, any
 *              association; [Blog2] 3.3).
 *   LS_AFFINE  uint32 only: element (a << 16) | b is the map v -> a*v + b mod
 *              2^16 (the 2x2 matrix [[a, b], [0, 1]]); the scan composes the maps,
 *              earlier applied first.  Not commutative, so it shows that results
 *              keep their left-right order ([Scan3] 三, matrix chain products).
 *              int32/float32 -> LS_ERR_UNSUPPORTED.
 * Identity (first exclusive cell, value for n = 0): 0 for sum, xor and or
 * (+0.0f for float32); INT32_MIN / 0u / -infinity for max; INT32_MAX /
 * 0xFFFFFFFF / +infinity for min; all ones for and; 1 (1.0f) for prod; the
 * identity map 0x00010000 for affine. */
typedef enum ls_op {
    LS_SUM = 0,
    LS_MAX = 1,
    LS_XOR = 2,
    LS_MIN = 3,
    LS_AND = 4,
    LS_OR = 5,
    LS_PROD = 6,
    LS_AFFINE = 7
} ls_op;

/* Compaction predicates: keep x when (x CMP threshold), compared in the element
 * type (signed, unsigned, or IEEE float with C semantics: NaN satisfies only NE). */
typedef enum ls_cmp { LS_LT = 0, LS_LE = 1, LS_GT = 2, LS_GE = 3, LS_EQ = 4, LS_NE = 5 } ls_cmp;

/* Device-wide schemes for scan_ex (the default entry points use the single pass).
 *   LS_SCHEME_SINGLE_PASS          one launch; each tile publishes its total, one
 *                                  resident wave turns the published totals into
 *                                  full prefixes in tile order, and each tile reads
 *                                  its predecessor's (the in-kernel hand-off through
 *                                  flags in global memory that [Scan3] 四 mentions;
 *                                  [SIMT3] 5.1).  Moves 2*n*4 bytes.
 *   LS_SCHEME_REDUCE_THEN_SCAN     tile totals, a scan of the totals, a seeded tile
 *                                  scan: three launches, 3*n*4 bytes ([Scan3] 四).
 *   LS_SCHEME_SCAN_THEN_PROPAGATE  tile scans with totals, a scan of the totals, an
 *                                  offset pass over the output: 4*n*4 bytes
 *                                  ([Scan3] 四, the three kernels as listed there).
 *   LS_SCHEME_SINGLE_PASS_DETERMINISTIC  the single pass with a fixed order of
 *                                  combination: tiles form groups of 64, the last
 *                                  tile of a group publishes a full prefix, and a
 *                                  tile combines it with its group's earlier totals
 *                                  in a fixed order.  Float sums and products are
 *                                  then the same bits on every run ([Scan3]
 *                                  pitfall list: a reproducible float result needs
 *                                  a fixed order).  Moves 2*n*4 bytes.
 * The three-phase schemes scan the tile totals recursively when they exceed one
 * tile, as [Scan3] 四 describes for very large arrays.  Their order of combination
 * depends only on n, so they too give the same bits on every run.  So does
 * LS_SCHEME_SINGLE_PASS: its resident wave combines the tile totals in groups of
 * 64 tiles aligned to tile 0, in an order fixed by the tile index. */
typedef enum ls_scheme {
    LS_SCHEME_SINGLE_PASS = 0,
    LS_SCHEME_REDUCE_THEN_SCAN = 1,
    LS_SCHEME_SCAN_THEN_PROPAGATE = 2,
    LS_SCHEME_SINGLE_PASS_DETERMINISTIC = 3
} ls_scheme;

/* Block-level scan used by batched_row_scan_ex for rows of more than 64 elements
 * (one block of 256 threads per row, 4 elements per thread per 1024-element chunk).
 *   LS_BLOCK_WAVE_DPP               64-lane DPP scans, wave totals through LDS, one
 *                                   barrier ([Scan3] 五, the two-level block scan)
 *   LS_BLOCK_HILLIS_STEELE          LDS Hillis-Steele, read / barrier / write /
 *                                   barrier per step ([Scan3] 二)
 *   LS_BLOCK_HILLIS_STEELE_DOUBLE   LDS Hillis-Steele with two buffers, one barrier
 *                                   per step ([Scan3] 二)
 *   LS_BLOCK_BLELLOCH               LDS up-sweep / down-sweep with padded indices
 *                                   ([Scan3] 三; [SIMT3] 5.4)
 * All four give identical results for integers and for max. */
typedef enum ls_block_scan {
    LS_BLOCK_WAVE_DPP = 0,
    LS_BLOCK_HILLIS_STEELE = 1,
    LS_BLOCK_HILLIS_STEELE_DOUBLE = 2,
    LS_BLOCK_BLELLOCH = 3
} ls_block_scan;

/* Returns LS_ABI_VERSION of the loaded library. */
int ls_abi_version(void);

/* A static, human-readable string for a status code (never NULL). */
const char *ls_status_string(ls_status s);

/* Zero-fills a workspace before its first use (or after ls_workspace_check
 * reported LS_ERR_INCOMPLETE): a fill kernel enqueued on `stream` (so the call
 * may be captured in a graph).
 *   ws        device workspace, 16-byte aligned.
 *   ws_bytes  its size: at least 256 and a multiple of 16.
 * Errors: LS_ERR_INVALID_ARG for NULL, misaligned or too small a workspace or a
 * size that is not a multiple of 16; LS_ERR_HIP when the launch fails. */
ls_status ls_workspace_init(void *ws, size_t ws_bytes, void *stream);

/* Reports whether a call on this workspace gave up a bounded wait since the
 * workspace was last initialised.  Unlike the other entry points this call
 * waits: it copies the workspace's error word to the host on `stream` and
 * synchronises the stream.
 *   flags (host, out, nullable): the error bits (1 = a wait gave up; 2 = a tile id
 *         beyond the call's tiles was handed out, i.e. the workspace was not
 *         initialised or calls sharing it overlapped).
 * Returns LS_OK when no bit is set, LS_ERR_INCOMPLETE when one is (the outputs of
 * the calls since the last initialisation may be incomplete; initialise the
 * workspace again before further use), LS_ERR_INVALID_ARG for a NULL or
 * misaligned ws, LS_ERR_HIP when the copy fails. */
ls_status ls_workspace_check(const void *ws, uint32_t *flags, void *stream);

/* Workspace size for scan_inclusive / scan_exclusive.
 *   bytes (host, out): size of the device workspace a call with these arguments
 *   needs (never 0).  Errors: LS_ERR_INVALID_ARG for n < 0, bytes == NULL or an
 *   unknown enum; LS_ERR_UNSUPPORTED for an operator not defined on t (see ls_op). */
ls_status ls_scan_workspace_bytes(int64_t n, ls_dtype t, ls_op op, size_t *bytes);

/* Inclusive scan: out[i] = in[0] (+) in[1] (+) ... (+) in[i].     [Scan3] 一
 * Exclusive scan: out[0] = identity, out[i] = in[0] (+) ... (+) in[i-1].
 *
 *   in, out   n elements of type t.  out == in (exact aliasing, in place) is
 *             allowed; any other overlap is LS_ERR_INVALID_ARG.
 *   n         element count, 0 <= n <= LS_MAX_N.  n == 0 writes only *total
 *             (= identity).
 *   t, op     element type and operator (see ls_op).
 *   total     nullable; receives one element: the reduction of all n inputs,
 *             i.e. the value that no exclusive cell holds ([Scan3] 一).
 *   ws        device workspace of ws_bytes >= ls_scan_workspace_bytes(...),
 *             16-byte aligned (else LS_ERR_INVALID_ARG), not overlapping any
 *             other argument, zero-filled before its first use (see
 *             "Workspaces" above).
 *   stream    hipStream_t as void*, or NULL.
 * One pass over the data: each element is read once and written once. */
ls_status scan_inclusive(const void *in, void *out, int64_t n, ls_dtype t, ls_op op, void *total,
                         void *ws, size_t ws_bytes, void *stream);
ls_status scan_exclusive(const void *in, void *out, int64_t n, ls_dtype t, ls_op op, void *total,
                         void *ws, size_t ws_bytes, void *stream);

/* Workspace size for scan_ex with the given scheme (rules as above). */
ls_status ls_scan_ex_workspace_bytes(int64_t n, ls_dtype t, ls_op op, ls_scheme scheme,
                                     size_t *bytes);

/* scan_inclusive / scan_exclusive with an explicit device-wide scheme.
 *   exclusive  nonzero: exclusive scan; zero: inclusive.
 *   scheme     see ls_scheme; an unknown value is LS_ERR_INVALID_ARG.
 *   ws         at least ls_scan_ex_workspace_bytes(n, t, op, scheme) bytes.
 * Other arguments, results and errors as for scan_inclusive. */
ls_status scan_ex(const void *in, void *out, int64_t n, ls_dtype t, ls_op op, int exclusive,
                  ls_scheme scheme, void *total, void *ws, size_t ws_bytes, void *stream);

/* Largest n that scan_noalloc accepts. */
#define LS_SCAN_NOALLOC_MAX_N 402653184LL

/* scan_inclusive / scan_exclusive for callers that cannot allocate device memory
 * at the point of the call: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  It takes no workspace: the library keeps a
 * fixed 8 MiB array in device memory per GPU (held until the process ends) and
 * uses it as the single-pass scan's workspace; the call itself allocates and frees
 * nothing.  The first call on a device looks the array up and enqueues its zero
 * fill on `stream` ahead of the scan; every 2^25-th call after that enqueues the
 * fill again (the array's status words compare epochs modulo 2^26).
 *   exclusive  nonzero: exclusive scan; zero: inclusive.
 *   n          0 <= n <= LS_SCAN_NOALLOC_MAX_N; a larger n returns
 *              LS_ERR_WORKSPACE and enqueues nothing.
 * Other arguments, results and errors as for scan_inclusive / scan_exclusive.
 * Every call on one GPU shares that GPU's array: calls whose execution may
 * overlap on one GPU (on different streams without an ordering between them, or
 * from several host threads) race and give wrong results.  Calls on one stream,
 * or ordered by events, are safe. */
ls_status scan_noalloc(const void *in, void *out, int64_t n, ls_dtype t, ls_op op, int exclusive,
                       void *total, void *stream);

/* Workspace size for compact_if (same rules as ls_scan_workspace_bytes). */
ls_status ls_compact_workspace_bytes(int64_t n, ls_dtype t, size_t *bytes);

/* Stable stream compaction ([Scan3] 一; [Blog2] 4.1; [SIMT3] 4.2):
 * every in[i] with (in[i] CMP threshold) is copied to out, in input order, and
 * the number kept is written to *count on the device.
 *
 *   in             n elements of type t.
 *   out            capacity n elements; must not overlap `in`.  Cells at index
 *                  >= *count are not written.
 *   n              0 <= n <= LS_COMPACT_MAX_N.
 *   count          device int64_t, written with the number of kept elements
 *                  (0 when n == 0).  Must not overlap in/out.
 *   threshold_bits the 32-bit pattern of the threshold in type t.
 *   ws, ws_bytes   as for the scans (ls_compact_workspace_bytes).
 * Uses no atomics on the data path; each element is read once and each kept
 * element written once. */
ls_status compact_if(const void *in, void *out, int64_t *count, int64_t n, ls_dtype t, ls_cmp cmp,
                     uint32_t threshold_bits, void *ws, size_t ws_bytes, void *stream);

/* Stable compaction by a flag array ([SIMT3] 4.1-4.2: the input comes with a
 * per-element validity mask; kept elements go to the front of the output in
 * order and the count is computed on the device).
 *   in, out   n 32-bit elements (any type; bits are copied); must not overlap.
 *   flags     n bytes, nonzero = keep; any alignment; must not overlap out.
 *   count     device int64_t, written with the number kept.
 *   ws        >= ls_compact_workspace_bytes(n, LS_UINT32, ...) bytes.
 * Cells of out at index >= *count are not written. */
ls_status compact_flags(const void *in, const uint8_t *flags, void *out, int64_t *count, int64_t n,
                        void *ws, size_t ws_bytes, void *stream);

/* Index selection: the positions i (uint32, ascending) of the elements that
 * compact_if would keep, i.e. the output index of the compaction's scatter
 * read the other way round ([Scan3] 一).  n < 2^32.  Other arguments as for
 * compact_if; out_indices holds n uint32 and must not overlap in. */
ls_status select_indices_if(const void *in, uint32_t *out_indices, int64_t *count, int64_t n,
                            ls_dtype t, ls_cmp cmp, uint32_t threshold_bits, void *ws,
                            size_t ws_bytes, void *stream);

/* The positions i (uint32, ascending) with flags[i] != 0.  n < 2^32. */
ls_status select_indices_flags(const uint8_t *flags, uint32_t *out_indices, int64_t *count,
                               int64_t n, void *ws, size_t ws_bytes, void *stream);

/* Row-wise scan of a rows x cols row-major, contiguous matrix: each row is
 * scanned on its own, with no carry between rows (the uniform-length case of a
 * segmented scan, [Blog2] 7.2).
 *
 *   in, out    rows*cols elements; out == in allowed, other overlap is not.
 *   rows, cols >= 0; either being 0 is a no-op returning LS_OK.
 *   exclusive  nonzero: exclusive scan per row, zero: inclusive.
 * Needs no workspace. */
ls_status batched_row_scan(const void *in, void *out, int64_t rows, int64_t cols, ls_dtype t,
                           ls_op op, int exclusive, void *stream);

/* batched_row_scan with an explicit block-level scan for the one-block-per-row
 * path (see ls_block_scan); with LS_BLOCK_WAVE_DPP it is batched_row_scan.  Other
 * kinds run rows of any length through that path.  An unknown kind is
 * LS_ERR_INVALID_ARG. */
ls_status batched_row_scan_ex(const void *in, void *out, int64_t rows, int64_t cols, ls_dtype t,
                              ls_op op, int exclusive, ls_block_scan block_scan, void *stream);

/* Workspace size for radix_sort (with_values: nonzero when values are sorted
 * along).  Errors: LS_ERR_INVALID_ARG for n < 0, n >= 2^32, bytes == NULL or an
 * unknown dtype. */
ls_status ls_radix_sort_workspace_bytes(int64_t n, ls_dtype t, int with_values, size_t *bytes);

/* Stable ascending radix sort of 32-bit keys, optionally carrying 32-bit values.
 * The pages' scan application ([Scan3] 一: each pass places keys by the scan of
 * a digit predicate, one group offset by the size of the others; [Blog2] 4.2:
 * per-digit histograms, their prefix sums, a reordering).
 *   keys_in, keys_out      n elements of type t.  keys_out == keys_in (in place)
 *                          is allowed; other overlap is LS_ERR_INVALID_ARG.
 *   values_in, values_out  both NULL (keys only) or both non-NULL: n 32-bit
 *                          values moved with their keys; values_out ==
 *                          values_in allowed.  One NULL and one not is
 *                          LS_ERR_INVALID_ARG.
 *   n                      0 <= n < 2^32.
 *   t                      key order: int32 signed, uint32 unsigned, float32
 *                          IEEE total order (-NaN < -inf < ... < -0 < +0 < ...
 *                          < +inf < +NaN, by bit pattern within NaNs).
 *   ws                     >= ls_radix_sort_workspace_bytes(n, t, values != NULL)
 *                          bytes, 16-byte aligned, overlapping no other buffer.
 * Equal keys keep their input order (the sort is stable), so the result,
 * values included, is unique.  Four passes of 8-bit digits; each reads the keys
 * twice and writes them once. */
ls_status radix_sort(const void *keys_in, void *keys_out, const void *values_in, void *values_out,
                     int64_t n, ls_dtype t, void *ws, size_t ws_bytes, void *stream);

/* Workspace size for segmented_scan / segmented_scan_offsets.  Errors as for
 * ls_scan_workspace_bytes. */
ls_status ls_segmented_workspace_bytes(int64_t n, ls_dtype t, ls_op op, size_t *bytes);

/* Segmented scan: the array is cut into consecutive segments and each segment is
 * scanned on its own, no value crossing a boundary ([Blog2] 7.2; the uniform
 * case is batched_row_scan).
 *   in, out    n elements; out == in allowed, other overlap is not.
 *   heads      n bytes; heads[i] != 0 marks the first element of a segment.
 *              Element 0 always starts one.  Any alignment.
 *   exclusive  nonzero: out[i] = identity where a segment starts, else the
 *              operator over the segment's elements before i; zero: inclusive.
 *   total      NULL or 1 element: the inclusive value of element n-1 (the last
 *              segment's reduction); the identity for n == 0.
 *   ws         >= ls_segmented_workspace_bytes(n, t, op) bytes, 16-byte aligned.
 * Operators, identities and float32 behaviour as for scan_inclusive (the same
 * bits on every run for the same input).  Errors: LS_ERR_INVALID_ARG for n <
 * 0, NULL or misaligned buffers with n > 0, overlap (heads or total with out,
 * ws with anything), unknown enums; LS_ERR_UNSUPPORTED and LS_ERR_WORKSPACE as
 * for scan_inclusive. */
ls_status segmented_scan(const void *in, void *out, int64_t n, ls_dtype t, ls_op op, int exclusive,
                         const uint8_t *heads, void *total, void *ws, size_t ws_bytes, void *stream);

/* Segmented scan with segments given as CSR offsets (the row-offset array of a
 * sparse matrix, one of scan's uses in [Scan3] 一): segment k is
 * [offsets[k], offsets[k+1]).
 *   offsets  nseg + 1 int64 (8-byte aligned), offsets[0] == 0, non-decreasing,
 *            offsets[nseg] == n; empty segments are allowed.  The kernel reads
 *            offsets[0 .. nseg-1]; offsets that break these rules give
 *            unspecified results but no access outside the buffers.
 *   nseg     >= 1 when n > 0.
 * Other arguments as for segmented_scan. */
ls_status segmented_scan_offsets(const void *in, void *out, int64_t n, ls_dtype t, ls_op op,
                                 int exclusive, const int64_t *offsets, int64_t nseg, void *total,
                                 void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * A decoding step: one token from each row of logits, and the books of a paged
 * cache (which pages a request holds, where its new tokens go).  The same common
 * rules hold: asynchronous on `stream`, arguments checked on the host before
 * anything is enqueued, kernels only (so calls can be captured in a graph), no
 * library call.  Results are the same bits on every run.
 * ------------------------------------------------------------------------- */

/* Element types of the logits. */
typedef enum ls_logits {
    LS_LOGITS_FLOAT32 = 0,
    LS_LOGITS_FLOAT16 = 1,
    LS_LOGITS_BFLOAT16 = 2
} ls_logits;

/* Workspace size for sample_tokens.  Errors: LS_ERR_INVALID_ARG for bytes == NULL,
 * rows or vocab outside [0, 2^31 - 1]. */
ls_status ls_sample_workspace_bytes(int64_t rows, int64_t vocab, size_t *bytes);

/* One token from each row, by given random numbers.  For a row x with largest
 * value M and temperature T > 0, token i has the weight w_i = exp((x_i - M) / T);
 * NaN counts as -infinity, and -infinity (a masked token) has no weight.  With the
 * tokens in order of x, largest first, equal ones by index:
 *   top_k  keeps the first k of the order (k <= 0: all);
 *   top_p  keeps of those each token whose weight before it is below p times
 *          their sum, and always the first (p <= 0 or NaN: only the first);
 *   min_p  keeps of those each token with w_i >= min(1, min_p) (<= 0 or NaN: all).
 * The token is the first index whose running sum of kept weights, in index order,
 * exceeds u times their sum Z.  Weights and sums are in 64 bits: a weight 2^-e is
 * right to a relative 2^-50 + e 2^-52 (below exp(-745) it is 0), a sum over a row to a
 * relative 2^-44 if vocab <= 2^17 or there are no cuts; a cut by value (top_p, or a
 * large top_k) of a longer row adds up to 2^-(61 - ceil(log2 vocab)), as bins of
 * weight hold 64 bits: 2^-43 for 2^18 tokens, 2^-37 for 2^24, 2^-30 for 2^31.
 *   logits       rows x vocab elements of type t; row r starts at element
 *                r * row_stride.  Any alignment to the element.
 *   rows, vocab  0 <= rows, vocab < 2^31; row_stride >= vocab when rows > 1, or 0
 *                (every row the same).
 *   uniforms     rows float32 in [0, 1).  1 and above take the last kept token whose
 *                weight is not 0, negative ones and NaN count as 0.
 *   temperature  rows float32.  T <= 0 or NaN: the lowest index of M, with
 *                log-probability 0; the cuts and the random number do not matter.
 *   top_k, top_p, min_p  rows int32 / float32 / float32 each, or NULL: no such cut.
 *   tokens       rows int64: the index, or -1 where no token is left (every logit
 *                -infinity or NaN, or vocab == 0).
 *   logprobs     rows float32 or NULL: ln(w / Z) of the token after the cuts;
 *                -infinity where no token is left.
 *   ws           >= ls_sample_workspace_bytes(rows, vocab) bytes, 16-byte aligned,
 *                zero-filled once by ls_workspace_init before its first use; each
 *                call leaves it ready for the next.  It serves sample_tokens only.
 * Outputs overlap no input and not each other (else LS_ERR_INVALID_ARG, as for
 * NULL, misaligned buffers, sizes and types outside the above). */
ls_status sample_tokens(const void *logits, int64_t rows, int64_t vocab, int64_t row_stride, ls_logits t,
                        const float *uniforms, const float *temperature, const int32_t *top_k,
                        const float *top_p, const float *min_p, int64_t *tokens, float *logprobs, void *ws,
                        size_t ws_bytes, void *stream);

/* Pages for the tokens that each request is about to add.  A request of len tokens
 * holds the ceil(len / page_size) pages at the front of its row of the table; with
 * new_len more it needs ceil((len + new_len) / page_size).  Requests are served in
 * order, each its missing pages from the end of the free list (the last free page
 * goes to the first missing column).  A request that needs more columns than the
 * table has gets nothing and is passed over; from the first request that the free
 * list cannot serve in full, only requests that miss no page are granted.
 *   lens, new_lens  requests int32 each; negative ones count as 0.  A request
 *                   whose len + new_len passes 2^31 - 1 gets nothing.
 *   tables          requests x columns int32, row r at element r * table_stride;
 *                   only the granted missing columns are written.
 *   free_pages      free_capacity int32, of which the first *free_count are free
 *                   (*free_count is taken as at least 0 and at most free_capacity).
 *   page_size       1 .. 2^31 - 1 tokens.
 *   count_out       device int64_t: free pages left.  Not free_count itself:
 *                   blocks that start late still read that.
 *   granted         requests bytes: 1 where the request has its pages, else 0.
 * No workspace.  Errors: LS_ERR_INVALID_ARG for negative or too large sizes
 * (requests, columns < 2^31; table_stride >= columns when requests > 1), NULL or
 * misaligned buffers, and outputs that overlap any other buffer. */
ls_status pages_append(const int32_t *lens, const int32_t *new_lens, int64_t requests, int32_t *tables,
                       int64_t columns, int64_t table_stride, const int32_t *free_pages, int64_t free_capacity,
                       const int64_t *free_count, int64_t page_size, int64_t *count_out, uint8_t *granted,
                       void *stream);

/* Where the new tokens of this step go in the cache.  Token j of the step, in order
 * of the requests and of their positions, belongs to request r with
 * offsets[r] <= j < offsets[r + 1], has position lens[r] + j - offsets[r] and slot
 * table[r][position / page_size] * page_size + position % page_size, or -1 where
 * the table has no such column or a negative page there.
 *   n          room in the outputs; tokens past it are left out, and entries past
 *              the last token get slot -1, position 0, request -1.
 *   slots      n int64; positions, request_ids: n int32.
 *   offsets    requests + 1 int64: the running sum of new_lens from 0.
 * Other arguments and errors as for pages_append; len + new_len of each request is
 * at most 2^31 - 1 (a token past that gets slot -1 and no defined position). */
ls_status slot_map(const int32_t *lens, const int32_t *new_lens, int64_t requests, const int32_t *tables,
                   int64_t columns, int64_t table_stride, int64_t page_size, int64_t n, int64_t *slots,
                   int32_t *positions, int32_t *request_ids, int64_t *offsets, void *stream);

/* The pages of finished requests go back on the free list: for each request with
 * finished[r] != 0, in order, the first min(ceil(lens[r] / page_size), columns)
 * entries of its table row are written behind the *free_count free pages.  Pages
 * past free_capacity are counted and not written.
 *   count_out  device int64_t: *free_count plus the pages of the finished
 *              requests.  Not free_count itself.
 * Other arguments and errors as for pages_append. */
ls_status pages_release(const int32_t *lens, const uint8_t *finished, int64_t requests, const int32_t *tables,
                        int64_t columns, int64_t table_stride, int32_t *free_pages, int64_t free_capacity,
                        const int64_t *free_count, int64_t page_size, int64_t *count_out, void *stream);

/* ---------------------------------------------------------------------------
 * A layer's scans: a gated linear recurrence over the tokens of each sequence, and
 * tokens to the rows of their experts and back, each with its gradients.  The common
 * rules hold: asynchronous on `stream`, arguments checked on the host before anything is
 * enqueued, kernels only (so calls can be captured in a graph), no library call.
 * Elements are float32, float16 or bfloat16 (ls_logits); states, sums and products are
 * in float32, and each output is rounded once.  Results are the same bits on every run.
 * ------------------------------------------------------------------------- */

/* What a gate value g means: the decay a, and what token x puts in.
 *   LS_GATE_DECAY    a = g,                 h = a h + x
 *   LS_GATE_LOG      a = exp(g),            h = a h + x
 *   LS_GATE_SIGMOID  a = 1 / (1 + exp(-g)), h = a h + (1 - a) x */
typedef enum ls_gating { LS_GATE_DECAY = 0, LS_GATE_LOG = 1, LS_GATE_SIGMOID = 2 } ls_gating;

/* Most channels of a row in the calls below. */
#define LS_MAX_CHANNELS (1LL << 23)
/* A recurrence keeps its value in front of every 64th row, for its gradients. */
#define LS_RECURRENCE_PERIOD 64

/* Rows of the array of carries: ceil(rows / LS_RECURRENCE_PERIOD), of each sequence, or once
 * where the rows are packed (packed != 0).  Errors: LS_ERR_INVALID_ARG for sizes outside
 * gated_recurrence's, or carry_rows == NULL. */
ls_status ls_recurrence_carry_rows(int64_t sequences, int64_t rows, int packed, int64_t *carry_rows);

/* Workspace size for gated_recurrence and gated_recurrence_backward of these sizes; 0 where
 * they need none.  Errors: LS_ERR_INVALID_ARG for sizes outside gated_recurrence's, an
 * unknown type or bytes == NULL. */
ls_status ls_recurrence_workspace_bytes(int64_t sequences, int64_t rows, int64_t channels, int packed, ls_logits t,
                                        size_t *bytes);

/* h_t = a_t h_{t-1} + b_t for the tokens t of each sequence, channel by channel, with a and b
 * from the gate and x as ls_gating says, and h_0 the sequence's state.
 *   x, gate, out   elements of type t.  Channel c of token r of sequence s is element
 *                  s * sequence_stride + r * row_stride + c.  Inputs may overlap each other and
 *                  themselves (stride 0: the same row for all); the output's rows lie apart,
 *                  sequence after sequence or token after token.
 *   offsets        NULL: each of `sequences` sequences has `rows` tokens.  Else sequences + 1
 *                  int64 on the device: sequence s is the rows offsets[s] .. offsets[s + 1] - 1
 *                  of one matrix of `rows` rows (sequence strides are not used), offsets[0] == 0,
 *                  none below the one before it, the last at most `rows`; sequences may be
 *                  empty.  Rows behind the last sequence are not written.  Offsets that break these
 *                  rules give unspecified results but no access outside the buffers.
 *   state          sequences x channels float32, row s at element s * state_stride, or NULL: zeros.
 *   state_out      the same with state_out_stride: h after each sequence's last token, not
 *                  rounded; the state itself for a sequence without tokens.  It may be `state`
 *                  (same pointer and stride), and else overlaps nothing.
 *   carries        NULL, or ls_recurrence_carry_rows x channels float32, for
 *                  gated_recurrence_backward.
 *   sequences, rows, channels   0 <= sequences, rows < 2^31; 0 <= channels <= LS_MAX_CHANNELS.
 *   ws             >= ls_recurrence_workspace_bytes bytes, 16-byte aligned, zero-filled once by
 *                  ls_workspace_init before its first use; each call leaves it ready for the next.
 *                  It serves the two recurrence calls only.  May be NULL where the size is 0.
 * A call whose sequences are cut into 2^23 or more tiles (64 tokens or more by 64 channels or more each; only rows
 * of few channels come to that) is refused with LS_ERR_UNSUPPORTED, whatever its workspace.
 * A tile waits for the ones in front of it.  A wait that lasts 1 s, which no correct run does, gives up: the outputs
 * are then incomplete, ls_workspace_check reports it, and the workspace has to be initialised again.
 * Decays of magnitude up to 1 are meant; larger ones work while the products of the decays of
 * any run of tokens stay within float32.  A sequence's infinities and NaN stay its own.
 * Errors: LS_ERR_INVALID_ARG (sizes, strides, NULL, alignment to the element, overlap, enums),
 * LS_ERR_WORKSPACE, LS_ERR_UNSUPPORTED. */
ls_status gated_recurrence(const void *x, int64_t x_sequence_stride, int64_t x_row_stride, const void *gate,
                           int64_t gate_sequence_stride, int64_t gate_row_stride, void *out,
                           int64_t out_sequence_stride, int64_t out_row_stride, const float *state,
                           int64_t state_stride, float *state_out, int64_t state_out_stride, float *carries,
                           const int64_t *offsets, int64_t sequences, int64_t rows, int64_t channels, ls_logits t,
                           ls_gating gating, void *ws, size_t ws_bytes, void *stream);

/* The gradients of gated_recurrence: from dout, that of out, and dstate_out, that of state_out
 * (NULL: zeros), those of x, gate and state.  x, gate, state, offsets, sizes, type and gating
 * are the forward call's, carries what it wrote.  dx and dgate have the type t, dstate is
 * float32; rows behind the last sequence are not written.  No output overlaps any other
 * buffer.  h is made again from x and gate in float32. */
ls_status gated_recurrence_backward(const void *dout, int64_t dout_sequence_stride, int64_t dout_row_stride,
                                    const void *x, int64_t x_sequence_stride, int64_t x_row_stride, const void *gate,
                                    int64_t gate_sequence_stride, int64_t gate_row_stride, const float *carries,
                                    const float *state, int64_t state_stride, const float *dstate_out,
                                    int64_t dstate_out_stride, void *dx, int64_t dx_sequence_stride,
                                    int64_t dx_row_stride, void *dgate, int64_t dgate_sequence_stride,
                                    int64_t dgate_row_stride, float *dstate, int64_t dstate_stride,
                                    const int64_t *offsets, int64_t sequences, int64_t rows, int64_t channels,
                                    ls_logits t, ls_gating gating, void *ws, size_t ws_bytes, void *stream);

#define LS_MAX_EXPERTS 1024

/* Workspace size for experts_sort.  Errors: LS_ERR_INVALID_ARG for sizes outside
 * experts_sort's or bytes == NULL. */
ls_status ls_experts_workspace_bytes(int64_t pairs, int64_t num_experts, size_t *bytes);

/* A stable sort of (token, expert) pairs by expert.
 *   experts      pairs int32 or int64 (id_bits 32 or 64): the expert of each pair, pair
 *                token * top + choice.  A number outside [0, num_experts) sends its pair nowhere.
 *   offsets      num_experts + 1 int64: expert e has the rows offsets[e] .. offsets[e + 1] - 1.
 *   order        pairs int32: the pair of each row, -1 behind the last row.
 *   places       pairs int32: the row of each pair, or -1.
 *   pairs, num_experts   0 <= pairs < 2^31; 1 <= num_experts <= LS_MAX_EXPERTS.
 *   ws           >= ls_experts_workspace_bytes bytes, 16-byte aligned; plain scratch.
 * Errors: LS_ERR_INVALID_ARG (sizes, NULL, alignment, outputs that overlap anything),
 * LS_ERR_WORKSPACE. */
ls_status experts_sort(const void *experts, int id_bits, int64_t pairs, int64_t num_experts, int64_t *offsets,
                       int32_t *order, int32_t *places, void *ws, size_t ws_bytes, void *stream);

/* Tokens to the rows of their pairs: rows[places[token * top + j]] = x[token].
 *   x            tokens x channels elements of type t, row r at element r * x_stride.
 *   places       tokens * top int32, as experts_sort gives them: different rows for different
 *                pairs.  A place outside [0, num_rows) takes part in nothing.
 *   rows         num_rows x channels, at rows_stride; rows that no place names are not written.
 *   sizes        0 <= tokens, top, num_rows, tokens * top < 2^31; channels <= LS_MAX_CHANNELS.
 * Its gradient is experts_combine without weights.  Errors: LS_ERR_INVALID_ARG. */
ls_status experts_gather(const void *x, int64_t x_stride, const int32_t *places, void *rows, int64_t rows_stride,
                         int64_t tokens, int64_t top, int64_t num_rows, int64_t channels, ls_logits t, void *stream);

/* The rows of each token's pairs, weighted and added up in the order of its pairs:
 * out[token] = sum over j of weights[token * top + j] * rows[places[token * top + j]]; zeros for
 * a token without a row.
 *   weights      tokens * top elements of type weight_type, or NULL: ones.  The weight of a
 *                pair without a row takes no part.
 * Other arguments as for experts_gather.  Without weights, its gradient is experts_gather. */
ls_status experts_combine(const void *rows, int64_t rows_stride, const int32_t *places, const void *weights,
                          ls_logits weight_type, void *out, int64_t out_stride, int64_t tokens, int64_t top,
                          int64_t num_rows, int64_t channels, ls_logits t, void *stream);

/* The gradients of experts_combine with weights: drows[place] = weight * dout[token], and
 * dweights[pair] = the product of dout[token] and rows[place] summed over the channels, 0 for a pair
 * without a row.  drows has the type t, its rows that no place names are not written; dweights
 * has the type weight_type. */
ls_status experts_combine_backward(const void *dout, int64_t dout_stride, const void *rows, int64_t rows_stride,
                                   const int32_t *places, const void *weights, ls_logits weight_type, void *drows,
                                   int64_t drows_stride, void *dweights, int64_t tokens, int64_t top, int64_t num_rows,
                                   int64_t channels, ls_logits t, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSCAN_H */
