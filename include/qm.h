/*
 * qm.h — C ABI of libqm: the GGML Q4_0 x f32 quantized matmul, the Q4_0
 * dequant, the Q8_0 dequant and quantize, a 4-bit key/value cache with its
 * attention, and the norm, routing and expert products of a decoder's layer, as
 * hand-written CUDA kernels for sm_103a (GB300).
 *
 * Operations (defined in "fuel-vulkan-kernels — quantized (GGML) kernel
 * contracts", fuel-dispatch 0.20.71, kernel-contracts/vulkan/quantized.fkc.md):
 *
 *   Q4_0 block: 18 bytes for 32 elements.  Bytes 0-1: the scale d, IEEE
 *   binary16, little-endian.  Bytes 2-17: 16 quant bytes; element j (0..15) is
 *   the low nibble of quant byte j and element j+16 its high nibble.  Element
 *   value = (nibble - 8) * d, nibble unsigned 0..15   (section "dequant_q4_0").
 *
 *   Matmul: C[m][n] = sum over k of A[m][k] * W[n][k], A f32 row-major [M][K],
 *   W a row-major [N][K/32] stream of Q4_0 blocks (row n holds blocks
 *   n*K/32 .. n*K/32 + K/32 - 1), C f32 row-major [M][N], K a multiple of 32
 *   (sections "qmatvec_q4_0" and "matmul_q4_0_tiled").  M = 1..8 runs the
 *   decode-regime GEMV kernels, M >= 9 the prefill GEMM.  The sum is taken in
 *   f32 in an order of the kernel's choosing; results agree with the exact
 *   sum to |error| <= 1e-5 * sum_k |A[m][k] * W[n][k]| + 1e-7 per element.
 *   The same call on the same inputs gives bitwise the same C (no atomics).
 *
 * Conventions for every entry point:
 *   - Pointers are device memory owned by the caller (cudaMalloc'd, managed,
 *     or mapped host memory with a device address).  Work is enqueued on
 *     `stream` (a cudaStream_t passed as void*; NULL means the legacy default
 *     stream) on the current device, and results are visible once that
 *     stream has been synchronized; no entry point but qm_device_status
 *     synchronizes.  Calls are thread-safe.
 *   - Memory: no entry point allocates device memory, and none writes
 *     anything but its outputs (and, for qm_matmul_q4_0_noalloc, its fixed
 *     scratch array).  The prefill GEMM splits A into bf16 pieces inside the
 *     kernel.  Where a GEMM or GEMV splits K over S CTAs (too few output tiles
 *     or rows to fill the SMs), S is 2, 4 or 8 and the S CTAs form a
 *     thread-block cluster that adds the partial sums in its shared memory;
 *     where those clusters would not all be resident at once, K is not split.
 *     The first call on a device sets kernel attributes and queries the
 *     device (host-side state only); after it, calls on any stream, including
 *     one being captured into a CUDA graph, enqueue kernels and nothing else.
 *   - Launch: the fast kernels are launched with programmatic dependent
 *     launch, so one may start its prologue while the previous kernel on the
 *     stream finishes; it reads and writes memory only after that kernel has
 *     completed, so stream order is kept exactly as for ordinary launches.
 *   - Operands are contiguous; no strides, offsets or broadcasts (but the rows
 *     that the key/value cache's and the layer's entry points take may be strided).
 *   - Arguments are checked on the host before anything is enqueued; a
 *     failed check returns a negative status and leaves memory untouched.
 *   - An output never aliases an input: overlapping byte ranges are rejected.
 *     (qm_kv_evict_q4_0 names its exceptions.)
 */
#ifndef QM_H
#define QM_H

#include <stdint.h>

#if defined(__GNUC__)
#define QM_API __attribute__((visibility("default")))
#else
#define QM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define QM_OK 0
#define QM_ERR_NULL (-1)        /* a required pointer is NULL                    */
#define QM_ERR_SHAPE (-2)       /* negative size, K % 32 != 0, or a size whose
                                   byte count does not fit in int64              */
#define QM_ERR_ALIGN (-3)       /* wq not 2-byte aligned, or A/C/out not 4-byte  */
#define QM_ERR_ALIAS (-4)       /* an output overlaps an input                   */
#define QM_ERR_CUDA (-5)        /* a CUDA call or kernel launch failed           */
#define QM_ERR_TIMEOUT (-6)     /* a kernel gave up a bounded wait (see
                                   qm_device_status)                             */
#define QM_ERR_UNSUPPORTED (-7) /* the forced algorithm cannot run this shape    */
#define QM_ERR_POINTER (-8)     /* a pointer is not device memory of the current
                                   device                                        */
#define QM_ERR_TOO_LARGE (-9)   /* beyond the fixed scratch of
                                   qm_matmul_q4_0_noalloc (M > 8)               */
#define QM_ERR_RANGE (-10)      /* a page number, length, row offset or expert in
                                   device memory was out of range (see
                                   qm_device_status)                             */
#define QM_ERR_WORKSPACE (-11)  /* the workspace is smaller than
                                   qm_attn_workspace_exact (or
                                   qm_experts_workspace) says                    */

/* Element types of keys, values, queries and attention outputs. */
#define QM_F32 0
#define QM_BF16 1

/* Bytes at the start of qm_attn_q4_0's workspace that are zero between calls. */
#define QM_ATTN_WORKSPACE_ZEROED 4096

/* Algorithms for qm_matmul_q4_0_algo. */
#define QM_ALGO_AUTO 0      /* what qm_matmul_q4_0 picks: GEMV_PK for M <= 2 and
                               N <= 1024, GEMV for M <= 8, otherwise GEMM_TC
                               where it applies, else GEMM_SIMT              */
#define QM_ALGO_GEMV 1      /* decode-regime GEMV on tensor cores (mma.sync, bf16
                               pieces, f32 sums); M 1..8                         */
#define QM_ALGO_GEMM_SIMT 2 /* prefill GEMM on FP32 FMA; any M >= 1              */
#define QM_ALGO_GEMV_SIMT 3 /* decode-regime GEMV on FP32 FMA; M 1..8             */
#define QM_ALGO_GEMM_TC 4   /* prefill GEMM on tcgen05 tensor cores (split bf16);
                               needs K % 256 == 0 and 16-byte aligned A and wq  */
#define QM_ALGO_GEMV_PK 5   /* decode-regime GEMV on packed FP32 FMA
                               (fma.rn.f32x2), one weight row per lane; M 1..2 */

/* Library version: major * 10000 + minor * 100 + patch. */
QM_API int qm_version(void);

/* A static, human-readable string for a status code. */
QM_API const char* qm_status_string(int status);

/*
 * qm_dequant_q4_0 — section "dequant_q4_0": out[32*b + j] = (q_j(b) - 8) * d(b)
 * for every block b < n_blocks and j < 32.
 *   wq       : n_blocks * 18 bytes of Q4_0 blocks, 2-byte aligned (16-byte
 *              aligned takes the fast path).
 *   n_blocks : number of blocks, >= 0.  0 enqueues nothing.
 *   out      : n_blocks * 32 floats, 4-byte aligned (16-byte aligned takes the
 *              fast path); must not overlap wq.
 * Exact: the product of an integer in [-8, 7] and a binary16 scale is
 * representable in f32, so the result is bit-identical to the definition,
 * including the sign of zero (q = 8 with d < 0 gives -0.0), infinities
 * (q != 8 with d = +-inf) and NaN (q = 8 with d infinite, or d NaN).
 * Returns QM_OK or a negative status.
 */
QM_API int qm_dequant_q4_0(const void* wq, int64_t n_blocks, float* out, void* stream);

/*
 * qm_dequant_q8_0 — section "dequant_q8_0": out[32*b + j] = qs_j(b) * d(b)
 * for every block b < n_blocks and j < 32.  A Q8_0 block is 34 bytes: the
 * scale d (IEEE binary16, little-endian) in bytes 0-1, then 32 signed 8-bit
 * quants qs_0 .. qs_31.
 *   wq       : n_blocks * 34 bytes, any alignment (16-byte aligned, with a
 *              16-byte aligned out, takes the fast path).
 *   n_blocks : number of blocks, >= 0.  0 enqueues nothing.
 *   out      : n_blocks * 32 floats, 4-byte aligned; must not overlap wq.
 * Exact: an 8-bit integer times a binary16 scale is representable in f32, so
 * the result is bit-identical to the definition, including the sign of zero,
 * infinities and NaN.  Returns QM_OK or a negative status.
 */
QM_API int qm_dequant_q8_0(const void* wq, int64_t n_blocks, float* out, void* stream);

/*
 * qm_quantize_q8_0 — section "quantize_q8_0": each block of 32 consecutive
 * elements of x becomes one 34-byte Q8_0 block with d = max|x| / 127 and
 * qs = round(x / d).  Where the section is silent this library takes:
 *   - f32 arithmetic; d = max|x| / 127 and each x / d are single correctly
 *     rounded f32 divisions; NaN elements do not raise the max;
 *   - the stored scale is d narrowed to binary16, round to nearest even
 *     (values from 65520 up become infinity);
 *   - round() takes halfway cases away from zero; qs is clamped to
 *     [-127, 127] (this binds only when d is an f32 subnormal);
 *   - qs = 0 where d is 0 or x / d is NaN.
 *   x          : n_elements floats, 4-byte aligned (16-byte aligned, with a
 *                16-byte aligned out, takes the fast path).
 *   n_elements : >= 0 and a multiple of 32, else QM_ERR_SHAPE.  0 enqueues
 *                nothing.
 *   out        : n_elements / 32 * 34 bytes, any alignment; must not overlap x.
 * Deterministic: every block depends only on its own 32 inputs.
 * Returns QM_OK or a negative status.
 */
QM_API int qm_quantize_q8_0(const float* x, int64_t n_elements, void* out, void* stream);

/*
 * qm_matmul_q4_0 — C = A x dequant(W)^T (see the header comment).
 *   A  : M*K floats, row-major [M][K], 4-byte aligned.
 *   wq : N*(K/32) Q4_0 blocks = N*K*9/16 bytes, row-major [N][K/32], 2-byte
 *        aligned.  Rows are 16-byte aligned, and the fastest GEMV path is
 *        taken, when wq is 16-byte aligned and K % 256 == 0.
 *   C  : M*N floats, row-major [M][N], 4-byte aligned; must overlap neither A
 *        nor wq.  Every element of C is written.
 *   M, N, K : M, N >= 0; K >= 0 with K % 32 == 0.
 * M == 0 or N == 0 enqueues nothing.  K == 0 sets C to +0.0 (the empty sum).
 * Returns QM_OK or a negative status.
 */
QM_API int qm_matmul_q4_0(const float* A, const void* wq, float* C, int64_t M,
                   int64_t N, int64_t K, void* stream);

/*
 * qm_matmul_q4_0_algo — qm_matmul_q4_0 with the algorithm forced (QM_ALGO_*),
 * for tests and benchmarks.  Returns QM_ERR_UNSUPPORTED when the algorithm
 * cannot run the shape (a GEMV with M > 8), QM_ERR_SHAPE for an unknown
 * algorithm number.
 */
QM_API int qm_matmul_q4_0_algo(const float* A, const void* wq, float* C, int64_t M,
                        int64_t N, int64_t K, int algo, void* stream);

/*
 * qm_device_status — synchronizes `stream` and reads the library's device
 * error word for the current device.  Kernels that wait on asynchronous
 * copies give up after a bounded number of polls, set this word and return
 * early (their output is then incomplete); the key/value cache's kernels set
 * it where a page number, a length or a row offset in device memory is out of
 * range, and skip the access.  Returns QM_OK if the word is clear,
 * QM_ERR_TIMEOUT if a wait gave up, QM_ERR_RANGE if only such a number was out
 * of range, QM_ERR_CUDA if the synchronize or the read failed.  With clear != 0 the word is reset after reading.
 */
QM_API int qm_device_status(void* stream, int clear);

/*
 * qm_selftest_wait_timeout — exercises the failure path of the bounded waits
 * without faulting or hanging anything.  No counterpart on the kernel-contract
 * pages; it exists so that tests can check, on a real GPU, that a wait which
 * runs out is reported and that the context stays usable.  Enqueues on
 * `stream` one kernel in which a single thread waits on an mbarrier that
 * nothing completes, giving up after 65536 polls; it then sets the device
 * error word and returns.  The next qm_device_status on the stream returns
 * QM_ERR_TIMEOUT (and, with clear != 0, resets the word, after which
 * qm_device_status returns QM_OK again).  No memory is read or written but the
 * error word.  Returns QM_OK, or QM_ERR_CUDA if the launch failed.
 */
QM_API int qm_selftest_wait_timeout(void* stream);

/*
 * qm_matmul_q4_0_noalloc — the decode-regime product C = A x dequant(W)^T for
 * M = 1..8, for callers that cannot call cudaMalloc.  No counterpart on the
 * kernel-contract pages: it exists for code that must not allocate device
 * memory at call time, such as a custom allocator or memory-pool callback,
 * a process running under a hard device-memory cap, or a runtime that owns
 * all device memory.  It meets the partial sums of a split K in a fixed array
 * compiled into the library (qm_matmul_q4_0 adds them up inside thread-block
 * clusters instead, and allocates nothing either), and allocates nothing,
 * ever.
 *   Arguments, layouts, alignment and aliasing rules: as qm_matmul_q4_0.
 *   Limit: M <= 8 (the GEMV regime); M > 8 returns QM_ERR_TOO_LARGE.  The
 *   array holds 1 MB of partial sums and 4096 row-group counters; when a
 *   shape's split would not fit, the kernel splits K less (down to not at
 *   all), so every N and K within the other limits is accepted.
 *   Memory: every GPU that loads the library holds the array (about 1 MB)
 *   until the process exits.
 *   Set-up: the first call on each device looks up the array's device
 *   address (cudaGetSymbolAddress) with that device current, and looks it up
 *   again when the device's current context has changed (after
 *   cudaDeviceReset); make that first call, and the first call after a reset,
 *   before any stream capture.
 *   Sharing: all calls use the same array, which keeps the last call's
 *   contents; a call clears the counters it needs before its kernel runs.
 *   Calls that overlap on the GPU (different streams, or concurrent graph
 *   launches) race on the array and may produce wrong results: order them.
 * Returns QM_OK or a negative status.
 */
QM_API int qm_matmul_q4_0_noalloc(const float* A, const void* wq, float* C, int64_t M,
                                  int64_t N, int64_t K, void* stream);

/*
 * qm_matmul_q4_0_q8act — the decode-regime product with the activations
 * quantized to Q8_0 first: C = A' x dequant(W)^T, A' = dequant_q8_0(
 * quantize_q8_0(A)) row by row (the GEMV fused with a preceding activation
 * quantization, the "act-quant fusion" item of "vulkan: shader and sequencing
 * efficiency backlog"; quantize_q8_0 with the readings of qm_quantize_q8_0).
 * A is read as f32 and quantized on chip; nothing but C is written.  Each
 * block of 32 then factors exactly into integers (d_a d_w (sum q qs - 8 sum
 * qs)), so the product runs on integer dot products, with one f32 rounding per
 * block; results agree with the exact product of A' and W to |error| <= 1e-5 *
 * sum_k |A'[m][k] * W[n][k]| + 1e-7, and infinities and NaN (a scale past
 * binary16's range) by class.  It is NOT the product with A: quantization
 * moves each activation by up to about half its block's step, max|x| / 254.
 *   A, wq, C, M, N, K, stream, alignment and aliasing: as qm_matmul_q4_0.
 *   M = 1..8 (M > 8 returns QM_ERR_TOO_LARGE); K % 256 == 0 with 16-byte
 *   aligned A and wq takes the staged kernel, other shapes a generic one.
 * Returns QM_OK or a negative status.
 */
QM_API int qm_matmul_q4_0_q8act(const float* A, const void* wq, float* C, int64_t M, int64_t N,
                                int64_t K, void* stream);

/*
 * qm_gemv_q4_0_list — a list of decode-regime products C_p = A_p x
 * dequant(W_p)^T (sections "qmatvec_q4_0" and "matmul_q4_0_tiled"; the
 * GEMV's cost is streaming the weight blocks once), all with the same M, in
 * one persistent launch where the shapes allow it: a decode step's chain of
 * projections without a fixed launch price per projection.
 *   problems : host array of `count` descriptors (read before the call
 *              returns).  Each problem follows the rules of qm_matmul_q4_0
 *              (operands, layouts, alignment, no output overlapping its own
 *              inputs).  wait_for is -1, or an index j below the problem's own:
 *              the problem's A is read only after problems 0..j have written
 *              their C (this is how a problem consumes an earlier one's
 *              output).  reserved must be 0.
 *   count    : >= 0.  M : >= 0, the rows of every A and C.
 *   counters : device memory of `count` uint32 (4-byte aligned, overlapping
 *              no operand) that the launch uses to count finished problems;
 *              it is cleared on `stream` before each launch that needs it.
 *              May be NULL: dependencies are then honoured by ending the
 *              launch before every problem that waits on one inside it.
 * Results are those of calling qm_matmul_q4_0 on the problems in list order.
 * Problems that neither wait on one another nor share memory may run in any
 * order; so no output may overlap another problem's weights, and an output
 * that overlaps another problem's activations or output (or whose
 * activations another problem's output overlaps) needs the later of the two
 * to wait for the earlier (QM_ERR_ALIAS otherwise).  The persistent kernel
 * takes M = 1, K % 2048 == 0, K <= 14336 and 16-byte aligned A and wq; other
 * problems run one by one through qm_matmul_q4_0's kernels, in list order on
 * the same stream.  Deterministic, like qm_matmul_q4_0.
 * Returns QM_OK or a negative status (nothing is enqueued when a check fails).
 */
typedef struct qm_gemv_problem {
    const float* A;   /* [M][K] f32, row-major                         */
    const void* wq;   /* [N][K/32] Q4_0 blocks                          */
    float* C;         /* [M][N] f32, row-major                          */
    int64_t N;
    int64_t K;
    int32_t wait_for; /* -1, or read A after problems 0..wait_for       */
    int32_t reserved; /* 0                                              */
} qm_gemv_problem;

QM_API int qm_gemv_q4_0_list(const qm_gemv_problem* problems, int64_t count, int64_t M,
                             uint32_t* counters, void* stream);

/*
 * qm_gemv_q4_0_q8act_list — qm_gemv_q4_0_list for the act-quant product of
 * qm_matmul_q4_0_q8act: every problem computes C_p = dequant_q8_0(
 * quantize_q8_0(A_p)) x dequant(W_p)^T, each activation vector quantized on
 * chip, in one persistent launch where the shapes allow it (M = 1, K % 2048
 * == 0, K <= 14336, 16-byte aligned A and wq); other problems run through
 * qm_matmul_q4_0_q8act in list order.  Arguments, ordering (wait_for,
 * counters), aliasing rules and errors: as qm_gemv_q4_0_list; M > 8 returns
 * QM_ERR_TOO_LARGE.  Precision: as qm_matmul_q4_0_q8act.
 */
QM_API int qm_gemv_q4_0_q8act_list(const qm_gemv_problem* problems, int64_t count, int64_t M,
                                   uint32_t* counters, void* stream);

/*
 * qm_gemm_plan — the work items the prefill GEMM on tensor cores
 * (QM_ALGO_GEMM_TC) takes for (M, N, K) on a device with sm_count SMs on
 * which fit2, fit4 and fit8 thread-block clusters of 2, 4 and 8 of its CTAs
 * can be resident at once.  Host only: touches no device and enqueues nothing;
 * meant for tests and tuning.
 *   out: 8 int64 values {tile width (112, 128 or 256), n-tiles, tiles, whole-tile
 *        items, s_rem K ranges of each later tile, 1 if the later tiles are
 *        split into 128-column halves instead, items (= CTAs), 1 if the K
 *        ranges add up through a cluster}.
 *   M, N >= 1, K a positive multiple of 256 (the shapes QM_ALGO_GEMM_TC takes).
 * Returns QM_OK, QM_ERR_NULL or QM_ERR_SHAPE.
 */
QM_API int qm_gemm_plan(int64_t M, int64_t N, int64_t K, int sm_count, int fit2, int fit4, int fit8,
                        int64_t* out);

/*
 * qm_gemv_plan — the launch plan the decode GEMV (QM_ALGO_GEMV, packed = 0;
 * QM_ALGO_GEMV_PK, packed = 1) takes for (M, N, K) on a device with sm_count
 * SMs and smem_optin bytes of opt-in shared memory per CTA.  With noalloc = 0
 * the plan of qm_matmul_q4_0, which adds a split K up through thread-block
 * clusters of 2, 4 or 8 CTAs, fit2, fit4 and fit8 of which can be resident
 * at once on that device; with noalloc = 1 the plan of
 * qm_matmul_q4_0_noalloc, whose split K meets in its fixed scratch array
 * (the fit counts are then ignored).  Host only: touches no device and
 * enqueues nothing; meant for tests and tuning.
 *   out: 13 int64 values {RG row groups, U units of 256 k, S K ranges, rps row
 *        groups per row block, c units per stage, hs warps per tile, rbpc row
 *        blocks per CTA, nu_max units in the largest K range, stages, grid
 *        CTAs, dynamic shared memory bytes, W consumer warps, 1 if the K
 *        ranges add up through a cluster}.
 *   M 1..8 (1..2 when packed), N >= 1, K a positive multiple of 256, fit
 *   counts >= 0.
 * Returns QM_OK, QM_ERR_NULL, QM_ERR_SHAPE, or QM_ERR_UNSUPPORTED when no
 * plan fits (the library then runs the generic GEMV).
 */
QM_API int qm_gemv_plan(int64_t M, int64_t N, int64_t K, int packed, int sm_count, int smem_optin,
                        int fit2, int fit4, int fit8, int noalloc, int64_t* out);

/* ------------------------------------------------------------------------
 * A 4-bit key/value cache: append, read back, attend, evict.  No counterpart
 * on the kernel-contract pages, which stop at the products: this is what a
 * decoder built on them keeps between its steps.  Keys and values are held as
 * Q4_0 values, (nibble - 8) * d with one binary16 scale d for each 32 elements
 * along the head dimension, in pages.
 *
 * Layout.  A cell holds 16 tokens of one kv head, 9 * head_dim bytes:
 * [head_dim / 32 blocks][16 tokens][16 quant bytes], then the scales
 * [16 tokens][head_dim / 32] in binary16.  The 16 quant bytes of a block are
 * those of a Q4_0 block (element j the low nibble of byte j, element j + 16 its
 * high nibble).  A page is page_tokens / 16 cells of one kv head in token
 * order; a pool is [n_pages][n_kv_heads] pages, one pool for keys and one for
 * values, same page numbers.  Token t of sequence b lives in page
 * page_table[b * table_stride + t / page_tokens].  Sequences may share pages
 * that a call only reads; one that it writes (qm_kv_append_q4_0, the `to` of
 * qm_kv_evict_q4_0) has a single place in the table.
 *
 * Rows of a call.  lengths[b] counts the tokens of sequence b including the
 * call's own; the call's rows of sequence b are its last ones, rows
 * q_starts[b] .. q_starts[b + 1] - 1 of the tensors (a device array of
 * n_seqs + 1; NULL gives every sequence n_tokens / n_seqs rows).  So a step
 * raises lengths, appends, then attends.  Rows that no sequence has are not
 * touched.
 *
 * What the host cannot see (page numbers, lengths, offsets) the kernels check:
 * a token whose page is missing or out of range, a length outside 0 .. max_len
 * or an offset outside the rows sets the device error word (QM_ERR_RANGE from
 * qm_device_status); the access is skipped and the outputs of that sequence
 * are unspecified.  Entries of page_table past a sequence's length are not
 * read.
 * ------------------------------------------------------------------------ */
typedef struct qm_kv_cache {
    void* k_pages;             /* n_pages * n_kv_heads pages, 16-byte aligned     */
    void* v_pages;             /* likewise                                        */
    const int32_t* page_table; /* device, [n_seqs][table_stride]                  */
    int32_t* lengths;          /* device, [n_seqs]                                */
    int64_t n_pages;
    int64_t table_stride;      /* page table entries per sequence                 */
    int64_t max_len;           /* no length is above it; <= table_stride *
                                  page_tokens and <= 2^30                         */
    int32_t n_seqs;            /* 0 .. 65535                                      */
    int32_t n_kv_heads;        /* 1 .. 32767                                      */
    int32_t head_dim;          /* a multiple of 32, 32 .. 256                     */
    int32_t page_tokens;       /* a power of two, 16 .. 65536                     */
    int32_t reserved;          /* 0                                               */
} qm_kv_cache;

/*
 * qm_kv_append_q4_0 — quantizes the call's rows of k and v into their places.
 *   k, v : [n_tokens][n_kv_heads][head_dim] of `dtype`, rows k_stride and
 *          v_stride elements apart (multiples of 4; so slices of a joint
 *          projection can be passed), 16-byte aligned (8-byte for QM_BF16).
 * Each block of 32 takes m, its first element of largest magnitude, d = m / -8
 * and r = 1 / d (each one correctly rounded f32 division), quants min(15,
 * floor(x r + 8.5)) (product and sum rounded to f32), and keeps d narrowed to
 * binary16, round to nearest even.  NaN elements do not raise the maximum and
 * become 8 (the value 0), as do all of a block whose m is 0; a magnitude past
 * 8 * 65504 makes d infinite.  Deterministic.  lengths is not changed.
 * Returns QM_OK or a negative status.
 */
QM_API int qm_kv_append_q4_0(const qm_kv_cache* cache, const void* k, const void* v, int dtype,
                             int64_t n_tokens, int64_t k_stride, int64_t v_stride,
                             const int32_t* q_starts, void* stream);

/*
 * qm_kv_read_q4_0 — the inverse: the values of the call's rows (the last ones
 * of each sequence) as f32, contiguous [n_tokens][n_kv_heads][head_dim],
 * 16-byte aligned.  Exact, as qm_dequant_q4_0.
 */
QM_API int qm_kv_read_q4_0(const qm_kv_cache* cache, float* k, float* v, int64_t n_tokens,
                           const int32_t* q_starts, void* stream);

/*
 * qm_attn_q4_0 — causal attention of the call's rows over the cache, grouped
 * query heads: query head h reads kv head h / (n_heads / n_kv_heads).
 *   s_j   = scale * q . k_j, for every token j that the row sees,
 *   out   = sum_j p_j v_j with p = softmax(s), lse = log sum_j exp(s_j).
 * A row at position p (0-based) of its sequence sees token j when j <= p and,
 * with window > 0, also j > p - window or j < sinks: a sliding window and a few
 * first tokens that stay visible.  A row that sees no token (its sequence is
 * shorter than its rows) gets out = +0 and lse = -infinity.
 *   q, out   : [n_tokens][n_heads][head_dim] of `dtype`, rows q_stride and
 *              out_stride elements apart (multiples of 4), 16-byte aligned
 *              (8-byte for QM_BF16).
 *   lse      : NULL, or [n_tokens][n_heads] f32, natural logarithm.
 *   weights  : NULL, or [n_seqs][n_kv_heads][weights_stride] f32 (weights_stride
 *              >= max_len): each token's accumulated attention weight;
 *              weights[b][h][j] += the sum of p_j over the sequence's rows and
 *              the query heads that read kv head h.  What qm_kv_evict_q4_0
 *              ranks by.
 *   max_q    : no sequence has more rows than this in the call (ignored
 *              without q_starts; 0 counts as 1).  The kernels and their grids
 *              are chosen by it: where it is far above the rows that there are
 *              (n_tokens for a batch of single tokens), a call takes a kernel
 *              for many rows and a grid of mostly idle blocks.
 *   workspace: qm_attn_workspace bytes, 16-byte aligned, its first
 *              QM_ATTN_WORKSPACE_ZEROED bytes zeroed once before its first use;
 *              every call leaves it fit for the next one, of this cache or
 *              another.  Calls that may run at the same time need a workspace
 *              each, and so do calls that threads make at the same time, on one
 *              stream too (a call may be several kernels).  One that a CUDA graph
 *              uses lives as long as the graph.
 * Precision: scores, statistics and sums in f32; products to about 2^-21 of
 * each |q_i k_i| and |p_j v_j| for QM_F32 (2^-17 of a |p_j v_j| that is 2^-18 of
 * the largest of the tokens around it, and less); for QM_BF16, where the output
 * keeps 8 bits, the probabilities and values of its sum may be rounded to 11
 * bits, probabilities below 2^-24 of the row's largest to 9 (lse and weights are
 * those of a QM_F32 call on the same queries).  Tokens that a row does not see
 * do not reach it, whatever their bytes hold.  A token that a row sees and
 * whose scales are not finite makes at least those entries of the row
 * non-finite that the formula does.  The same call on the same inputs gives
 * bitwise the same results (no atomics on floating values).
 * Returns QM_OK or a negative status.
 */
typedef struct qm_attn_args {
    const void* q;
    void* out;
    float* lse;
    float* weights;
    const int32_t* q_starts;
    void* workspace;
    int64_t workspace_bytes;
    int64_t n_tokens;
    int64_t max_q;
    int64_t q_stride;
    int64_t out_stride;
    int64_t weights_stride;
    int64_t window; /* 0: none */
    int64_t sinks;
    int64_t n_heads; /* a multiple of n_kv_heads; n_tokens * n_heads < 2^31 */
    float scale;
    int32_t dtype;    /* QM_F32 or QM_BF16 */
    int32_t reserved; /* 0 */
} qm_attn_args;

QM_API int qm_attn_q4_0(const qm_kv_cache* cache, const qm_attn_args* args, void* stream);

/*
 * qm_attn_workspace — bytes of workspace that qm_attn_q4_0 needs for any call
 * of at most these sizes (weights != 0: with or without accumulated weights).
 * Calls of few rows take another kernel than those of many, and may need more:
 * with weights, up to 24 rows and query heads of a kv head (256 in small
 * batches) keep 4 * max_len bytes for each until the call is over.
 * qm_attn_workspace_exact — the bytes for a call of exactly these sizes, with
 * weights as given: what the call itself asks for.
 * Host only.  Return the bytes (0: none is needed) or a negative status.
 */
QM_API int64_t qm_attn_workspace(const qm_kv_cache* cache, int64_t n_heads, int64_t n_tokens,
                                 int64_t max_q, int weights);
QM_API int64_t qm_attn_workspace_exact(const qm_kv_cache* cache, int64_t n_heads, int64_t n_tokens,
                                       int64_t max_q, int weights);

/*
 * qm_kv_evict_q4_0 — cuts every (sequence, kv head) of `from` back to `budget`
 * tokens and writes them, in order, to the first places of `to`.  A sequence
 * of length L <= budget keeps all its tokens.  Of a longer one stay its first
 * `sinks` tokens, its last `recent` ones (sinks + recent <= budget), and of
 * those between, the ones with the largest weights; of equal weights the
 * lowest positions; NaN ranks below every number and -0 equals +0.
 *   weights     : [n_seqs][n_kv_heads][weights_stride] f32.
 *   kept        : [n_seqs][n_kv_heads][budget] int32, the kept positions in
 *                 ascending order, then -1.
 *   weights_out : [n_seqs][n_kv_heads][out_stride] f32 (out_stride >= budget):
 *                 the kept tokens' weights, then 0 up to budget.  May be
 *                 `weights` itself (with the same stride).
 *   to->lengths is set to min(L, budget).  `to` is another cache (it may share
 *   pools, on other pages, and have pages of another size), or `from` itself:
 *   then the cache is cut back in place.  from->lengths may be to->lengths.
 * Cells are moved byte for byte; a kept token's position becomes its place.
 * Returns QM_OK or a negative status.
 */
QM_API int qm_kv_evict_q4_0(const qm_kv_cache* from, const qm_kv_cache* to, const float* weights,
                            int64_t weights_stride, int64_t budget, int64_t sinks, int64_t recent,
                            int32_t* kept, float* weights_out, int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------
 * What stands between a decoder's attention and its next one: the norm that
 * adds the residual, the choice of each token's experts, and the experts'
 * products.  No counterpart on the kernel-contract pages.  Rows may be strided
 * (strides in elements).
 * ------------------------------------------------------------------------ */

/*
 * qm_add_rmsnorm — for every row, in f32:
 *   s = x + residual (x without one),
 *   y = s / sqrt(mean(s^2) + eps) * (weight_offset + weight).
 * Written are, where wanted: s and y, each rounded once to `dtype`, and the Q8_0
 * blocks of y as qm_quantize_q8_0 makes them of f32 rows (not of rounded ones).
 *   x, residual, out, sum : [n_rows][width] of `dtype`, aligned to an element.
 *              residual, out and sum may be NULL; sum may be x or residual
 *              itself (same stride).
 *   weight   : [width] f32, or NULL for none (y = s / sqrt(..)).
 *   q8       : NULL, or n_rows * width / 32 blocks of 34 bytes, 2-byte aligned;
 *              needs width % 32 == 0.
 *   width    : 1 .. 2^20.  Rows of 8 elements' multiples, 16-byte aligned, take
 *              the fast path.
 * A row whose squares leave f32's range at either end, or that holds infinities
 * or NaN, gives what f32 arithmetic makes of the formula.  Deterministic.
 * Returns QM_OK or a negative status.
 */
typedef struct qm_rmsnorm_args {
    const void* x;
    const void* residual;
    const float* weight;
    void* out;
    void* sum;
    void* q8;
    int64_t n_rows;
    int64_t width;
    int64_t x_stride;
    int64_t residual_stride;
    int64_t out_stride;
    int64_t sum_stride;
    float eps;           /* >= 0 */
    float weight_offset; /* 0, or 1 for weights held as their distance from 1 */
    int32_t dtype;       /* QM_F32 or QM_BF16 */
    int32_t reserved;    /* 0 */
} qm_rmsnorm_args;

QM_API int qm_add_rmsnorm(const qm_rmsnorm_args* args, void* stream);

/*
 * qm_route_experts — each token's experts and their weights.  Of a token's logits
 * l: scores s = softmax(l) or 1 / (1 + exp(-l)); choices c = s + bias.  With
 * n_groups > 1 the experts are in n_groups equal ranges; a group counts as much
 * as its group_top (1 or 2) largest choices together, and the experts of all
 * but the top_groups largest groups are out.  ids get the top_k experts of the
 * largest choices, largest first; weights their scores (without the bias),
 * divided by their sum with `renormalize` (0 where that is 0; sums below 2^-26 are
 * taken again in f64, so that small scores keep their bits), times `scale`.
 * Equal choices, and equal groups, go to the lower index; without a bias the
 * experts' order is that of the logits.  Choices that lie so close that f32
 * could turn them around are compared in f64.
 *   logits : [n_tokens] rows of n_experts of `dtype`, aligned to an element.
 *   bias   : [n_experts] f32, or NULL.
 *   ids, weights : [n_tokens][top_k] int32 and f32, contiguous.
 *   n_experts 1 .. 1024, a multiple of n_groups; n_groups 1 .. 64; top_k 1 .. 32,
 *   at most the experts of top_groups groups.
 * A logit of -infinity has the score 0 (a row of nothing else, weights 0).  NaN
 * ranks below every number.  With softmax, a row with NaN or +infinity has NaN
 * weights.  The ids are experts, each at most once, whatever the logits hold.
 * Deterministic.  Returns QM_OK or a negative status.
 */
#define QM_SCORE_SOFTMAX 0
#define QM_SCORE_SIGMOID 1

typedef struct qm_route_args {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t n_tokens;
    int64_t logits_stride;
    int32_t n_experts;
    int32_t top_k;
    int32_t n_groups;
    int32_t top_groups;
    int32_t group_top;   /* 1 or 2 */
    int32_t scoring;     /* QM_SCORE_* */
    int32_t renormalize; /* 0 or 1 */
    float scale;
    int32_t dtype;       /* QM_F32 or QM_BF16 */
    int32_t reserved;    /* 0 */
} qm_route_args;

QM_API int qm_route_experts(const qm_route_args* args, void* stream);

/*
 * qm_experts_q4_0 — the feed-forward block of a decoder with experts:
 *   out[t] = sum_j weights[t][j] * W_down[e] (act(W_gate[e] x[t]) * (W_up[e] x[t])),
 * e = ids[t][j]; without w_gate, W_down[e] act(W_up[e] x[t]).  One expert with
 * top_k = 1 and ids of 0 is an ordinary feed-forward block.
 * The experts (qm_experts): Q4_0 block streams, each 16-byte aligned,
 *   w_gate, w_up : [n_experts] matrices of `inner` rows of hidden / 32 blocks,
 *   w_down       : [n_experts] matrices of `hidden` rows of inner / 32 blocks,
 *   *_stride     : bytes from one expert's matrix to the next (a multiple of 16,
 *                  so gate and up may be halves of one tensor).
 * The call:
 *   x, out    : [n_tokens][hidden] of `dtype`, rows x_stride and out_stride
 *               elements apart (multiples of 4), 16-byte aligned (8-byte for
 *               QM_BF16).  out may not be x.
 *   ids       : [n_tokens][top_k] int32.  A negative id is no expert (a row of
 *               padding, an expert that is elsewhere): nothing is added, and a
 *               token without experts gets 0.  The same expert twice counts
 *               twice.  An id from n_experts up sets the device error word
 *               (QM_ERR_RANGE from qm_device_status) and counts as none.
 *   weights   : [n_tokens][top_k] f32.
 *   workspace : qm_experts_workspace bytes, 16-byte aligned; its contents do not
 *               matter before or after a call.  Calls that may run at the same
 *               time need a workspace each, and so do calls that threads make at
 *               the same time, on one stream too (a call is several kernels, and
 *               another's may come between them).  One that a CUDA graph uses
 *               lives as long as the graph.
 * Precision: sums in f32, the inner activations in f32; for QM_F32 products to
 * about 2^-21 of |x_k w_k|, and 2^-38 of the row's largest |x| times |w_k|; for
 * QM_BF16 weights rounded to 11 bits, and inner activations to 11 bits (or 2^-38
 * of the row's largest).  Sums that come out infinite or NaN are taken again,
 * element by element in f32, from x (the inner activations) and the blocks.
 * Deterministic: the same call gives bitwise the same result.
 * Returns QM_OK or a negative status.
 */
#define QM_ACT_NONE 0
#define QM_ACT_SILU 1 /* a / (1 + exp(-a)) */
#define QM_ACT_GELU 2 /* a / 2 * (1 + tanh(sqrt(2 / pi) (a + 0.044715 a^3))) */

typedef struct qm_experts {
    const void* w_gate; /* or NULL */
    const void* w_up;
    const void* w_down;
    int64_t gate_stride; /* bytes, below 2^40 */
    int64_t up_stride;
    int64_t down_stride;
    int64_t hidden; /* a multiple of 32, 32 .. 65536 */
    int64_t inner;  /* likewise */
    int32_t n_experts;  /* 1 .. 1024 */
    int32_t activation; /* QM_ACT_* */
    int32_t reserved[2]; /* 0 */
} qm_experts;

typedef struct qm_experts_args {
    const void* x;
    void* out;
    const int32_t* ids;
    const float* weights;
    void* workspace;
    int64_t workspace_bytes;
    int64_t n_tokens;
    int64_t x_stride;
    int64_t out_stride;
    int32_t top_k;    /* 1 .. 1024; n_tokens * top_k < 2^24 */
    int32_t dtype;    /* QM_F32 or QM_BF16 */
    int32_t reserved[2]; /* 0 */
} qm_experts_args;

QM_API int qm_experts_q4_0(const qm_experts* experts, const qm_experts_args* args, void* stream);

/*
 * qm_experts_workspace — bytes of workspace that qm_experts_q4_0 needs for any
 * call of at most n_tokens tokens and top_k experts each, of either type.
 * Host only.  Returns the bytes or a negative status.
 */
QM_API int64_t qm_experts_workspace(const qm_experts* experts, int64_t n_tokens, int32_t top_k);

/*
 * qm_launch_count — the number of kernels this library has enqueued in this
 * process (all devices, all threads), for accounting in benchmarks.
 */
QM_API uint64_t qm_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* QM_H */
