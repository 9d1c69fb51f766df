/*
 * qmv.h -- C ABI of the weight-only mixed-bit packed matvec library (GB300,
 * sm_103a).
 *
 * y = W . x for weights stored as packed low-bit codes with fp16 scales,
 * fp16 activations and fp32 accumulation, with an optional residual-add +
 * RMSNorm folded into the matvec.  The method follows these pages:
 *   [A19]  "Gemma4 raw-Metal loop on A19 -- findings + the remaining (parked)
 *          levers", section "What moved the needle": int2 codes, 16 per 32-bit
 *          word, exact products, fp32 sums in code order; q/k/v and gate/up
 *          fused into single dispatches; residual-add + RMSNorm folded into
 *          the next matvec's prologue; int8 weights loaded as vectors.
 *   [PLAY] "raw-metal-loop-playbook", prefill-regimes table: chunks of M
 *          tokens read the weights once per M tokens; M = 8/16 tiles keep each
 *          output scalar's K-dot in the M = 1 order; M = 64/128 tiles use the
 *          matrix units and change the order.
 *
 * Conventions (all entry points):
 *   - Every pointer named d_* or described as "device" is a CUDA device
 *     pointer owned by the caller.  The library allocates no device memory:
 *     the scratch some calls need (the tensor-core tiles' split-K partial
 *     tiles, the fused prologue's normalised activations for M >= 2) is a
 *     caller-provided workspace whose size qmv_workspace_bytes() gives.
 *   - fp16 values are IEEE binary16 bit patterns (uint16_t / __half).
 *   - Matrices are row-major with no padding.  Activations are M x K (row m is
 *     column m of the matvec, i.e. token m); outputs are M x N.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous on it; nothing synchronises.
 *   - Every call returns a qmv_status.  Arguments are validated on the host;
 *     no call aborts, throws across the ABI or traps on the device.  A failed
 *     launch returns QMV_ERR_CUDA and qmv_last_cuda_error() gives the raw
 *     cudaError_t (thread-local).
 *   - Packs are immutable after qmv_pack_weights, so concurrent calls that
 *     share a pack are safe.
 *
 * Packed layout (the bit order is a reading: the pages give only "16 codes
 * per word"): row n of codes is K*bits/32 little-endian uint32 words; code k
 * sits in word floor(k*bits/32) at bit offset bits*(k mod (32/bits)); the
 * field holds u = v + 2^(bits-1) for the signed code v, so int2 fields
 * 0,1,2,3 decode to -2,-1,0,1.  Scales are fp16 [N][K/group].
 *
 * Accumulation order (QMV_EXACT, every CUDA-core path, any M): for
 * each output scalar, each block of 32 consecutive codes is summed serially
 * in k in fp32 (products are exact); with group 32 the block sum is
 * multiplied by its scale (rounded) and added to the accumulator (rounded),
 * blocks in order; with one scale per row (group == K) the block sums are
 * added serially and the total is multiplied by the scale once.  This is the
 * oracle's order, so QMV_EXACT results are bit-identical to it, and every
 * column of an M-tile is bit-identical to the M = 1 result.
 *
 * QMV_FAST (CUDA-core paths): the same blocks, scales and fold, with the code offset
 * taken out of the per-code work: each block is summed as sum(y*u) over the
 * unsigned fields u (even and odd words in two serial chains, then added)
 * minus 2^(bits-1) times the block's activation sum formed in the same
 * order.  Results are within max |y - ref| <= 1e-3*(1+|ref|) of the oracle
 * (in practice a few fp32 ulps of the block sums), a block of zero codes
 * gives exactly 0, and every column of an M-tile is still bit-identical to
 * the QMV_FAST M = 1 result.  Shapes outside the M = 1 pipeline (K not a
 * multiple of 256) keep the exact order in both modes.
 */
#ifndef QMV_H
#define QMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define QMV_API __attribute__((visibility("default")))
#else
#define QMV_API
#endif

typedef struct qmv_pack qmv_pack;   /* opaque host descriptor; owns no device memory */
typedef struct qmv_chain qmv_chain; /* opaque host descriptor of a matvec chain */
typedef struct qmv_w4pack qmv_w4pack; /* opaque host descriptor of 4-bit weights with zero points */

typedef enum {
    QMV_OK = 0,
    QMV_ERR_INVALID_ARG = -1,   /* null pointer, bad enum value, M out of range */
    QMV_ERR_UNSUPPORTED = -2,   /* valid but not implemented (e.g. a tile shape) */
    QMV_ERR_ALIGNMENT = -3,     /* a pointer is not aligned as documented */
    QMV_ERR_SHAPE = -4,         /* N/K/bits/group disagree with the pack or layout rules */
    QMV_ERR_CUDA = -5,          /* a CUDA runtime call or launch failed */
    QMV_ERR_TIMEOUT = -6,       /* a bounded device-side wait ran out */
    QMV_ERR_WORKSPACE = -7      /* the call needs a larger workspace (qmv_workspace_bytes) */
} qmv_status;

/* element types; QMV_BF16 is taken by the verification-step calls (the
 * qmv_w4_*, qmv_block_norm, qmv_softmax and qmv_verify_draft entry points) and the
 * decode-step calls after them */
typedef enum { QMV_F32 = 0, QMV_F16 = 1, QMV_BF16 = 2 } qmv_dtype;
typedef enum { QMV_FAST = 0, QMV_EXACT = 1 } qmv_mode;    /* accumulation mode */

/*
 * qmv_create_pack -- describe a packed weight matrix.  [A19] int2 item:
 * 16 codes per word; int4 and int8 use the same offset-binary rule.
 *   N, K   output and input features; K*bits/8 must be a multiple of 16
 *          (K % 64 == 0 for int2, K % 32 == 0 for int4 and int8).
 *   bits   2, 4 or 8.
 *   group  32 (one fp16 scale per 32 consecutive k of a row) or K (one
 *          scale per row).
 *   codes_bytes, scales_bytes  (out, nullable) bytes the caller must allocate
 *          for the packed codes (N*K*bits/8) and the scales (N*(K/group)*2).
 * Errors: QMV_ERR_INVALID_ARG (out is NULL, bits/group not allowed),
 * QMV_ERR_SHAPE (N < 1, K not allowed).  Host only; touches no device.
 */
QMV_API int qmv_create_pack(qmv_pack **out, int N, int K, int bits, int group,
                    size_t *codes_bytes, size_t *scales_bytes);

/*
 * qmv_pack_weights -- pack signed codes on the device and bind the pack to
 * the caller's buffers.  [A19] int2 item (16 codes per 32-bit word).
 *   d_codes_in   device int8 [N][K], signed codes in [-2^(bits-1), 2^(bits-1)-1].
 *                A code out of range is masked to its low `bits` bits.
 *   d_scales_in  device fp16 [N][K/group].
 *   d_codes      device, codes_bytes, 16-byte aligned: receives the words.
 *   d_scales     device, scales_bytes, 16-byte aligned: receives a copy of
 *                the scales.
 * The pack keeps d_codes/d_scales; they must outlive every later call that
 * uses the pack.  Errors: INVALID_ARG (NULL), ALIGNMENT, CUDA.
 */
QMV_API int qmv_pack_weights(qmv_pack *p, const int8_t *d_codes_in, const uint16_t *d_scales_in,
                     void *d_codes, void *d_scales, void *stream);

/*
 * qmv_workspace_bytes -- device scratch bytes that a call of qmv_gemv /
 * qmv_chunk_gemm (fused = 0) or qmv_fused_rmsnorm_gemv (fused = 1) with this
 * pack, M, y_dtype and mode needs in its d_workspace:
 *   - M = 1, or K not a multiple of 256: 0.
 *   - M > 32, QMV_FAST, int2, fused = 0 (the tensor-core tiles): fp32
 *     split-K partial tiles when the chosen split needs more than the output
 *     itself, else 0.
 *   - every other M >= 2 (the CUDA-core M-column tiles): the activation
 *     tables, built once per call: per 512 codes, 8960 bytes per 4 columns
 *     (ceil(M/4) * ceil(K/512) * 8960), or 17408 per 8 columns where the
 *     library takes 8-column tiles (M >= 5), fused or not.
 * The size depends only on these arguments and the device's SM count, so one
 * workspace serves every later call with them.  Host only; 0 for invalid
 * arguments.
 */
QMV_API size_t qmv_workspace_bytes(const qmv_pack *p, int M, int y_dtype, int mode, int fused);

/*
 * qmv_gemv -- y = x . W^T for M columns: y[m][n] = sum_g (sum_{k in g}
 * x[m][k] * v[n][k]) * s[n][g] in the order stated at the top of this file.
 * [A19] int2 item (exact products, fp32 in code order); [PLAY] K-order-fixed
 * row for M <= 16 and matrix-unit row for M >= 64.
 *   M            1 .. 4096.  Every M runs the CUDA-core kernels (QMV_EXACT
 *                bit-exact, QMV_FAST within tolerance, each column equal to
 *                the M = 1 result), except M > 32 with QMV_FAST and int2
 *                weights, which runs tcgen05 tensor-core tiles (fp32
 *                accumulate, hardware order, within tolerance).  With K a
 *                multiple of 256 the M >= 2 CUDA-core tiles take all M
 *                columns in one launch; otherwise 32 columns per launch.
 *   N, K, bits, group  must equal the pack's (QMV_ERR_SHAPE otherwise).
 *   x            device fp16 [M][K], 16-byte aligned.
 *   y            device [M][N] of y_dtype (fp32, or fp16 = RNE of the fp32
 *                result), 4-byte aligned.
 *   mode         QMV_FAST or QMV_EXACT.
 *   d_workspace, workspace_bytes  caller scratch, 256-byte aligned, at least
 *                qmv_workspace_bytes(p, M, y_dtype, mode, 0) bytes (may be
 *                NULL, 0 when that is 0).  Its contents on entry do not
 *                matter; calls that share a workspace must not overlap.
 * Errors: INVALID_ARG, SHAPE, ALIGNMENT, UNSUPPORTED, WORKSPACE, CUDA.
 */
QMV_API int qmv_gemv(const qmv_pack *p, int M, int N, int K, int bits, int group,
             const void *x, void *y, int y_dtype, int mode, void *d_workspace,
             size_t workspace_bytes, void *stream);

/*
 * qmv_fused_rmsnorm_gemv -- residual add + RMSNorm folded into the matvec
 * prologue ([A19] dispatch-count fusion item).  For each column m:
 *   h = fp16(x + residual); ss = sum of h*h (serial in blocks of 32, then
 *   serial over blocks); inv = 1/sqrt(ss/K + eps) (IEEE fp32 ops);
 *   y16 = fp16((h * inv) * gamma); then y = matvec(y16) as qmv_gemv.
 *   x, residual  device fp16 [M][K]; gamma device fp16 [K]; 16-byte aligned.
 *   h_out        nullable device fp16 [M][K]: receives h (the next residual).
 *   M            1 .. 4096; every column runs the CUDA-core kernels (the
 *                fused prologue never takes the tensor-core tiles), each
 *                column equal to the M = 1 result.
 *   d_workspace, workspace_bytes  as qmv_gemv, sized by
 *                qmv_workspace_bytes(p, M, y_dtype, mode, 1).
 * Errors: as qmv_gemv.
 */
QMV_API int qmv_fused_rmsnorm_gemv(const qmv_pack *p, int M, const void *x, const void *residual,
                           const void *gamma, float eps, void *h_out, void *y,
                           int y_dtype, int mode, void *d_workspace, size_t workspace_bytes,
                           void *stream);

/*
 * qmv_chunk_gemm -- a prefill chunk of M tokens against one pack ([PLAY]
 * prefill-regimes table): the same computation as qmv_gemv with the pack's
 * own N, K, bits and group.  M = 4, 8, 16 (and any M <= 32, or any M in
 * QMV_EXACT, or int4/int8) use the K-order-fixed CUDA-core tiles; M = 64,
 * 128 (any M > 32) in QMV_FAST with int2 weights use tcgen05 tensor-core
 * tiles.  d_workspace, workspace_bytes as qmv_gemv.
 */
QMV_API int qmv_chunk_gemm(const qmv_pack *p, int M, const void *x, void *y, int y_dtype,
                   int mode, void *d_workspace, size_t workspace_bytes, void *stream);

/*
 * qmv_gemv_argmax -- the lm_head matvec with the greedy-token step fused into
 * its epilogue ([A19] "The parked levers" table, argmax stage1+2 merge row:
 * one dispatch, first-max tie-break): y = matvec(x) for M = 1 as qmv_gemv
 * (or, with residual != NULL, as qmv_fused_rmsnorm_gemv with gamma, eps and
 * h_out), then the index of the largest fp32 result -- the lowest index among
 * equal maxima; values compare as numbers (-0 equals +0); NaN never wins.
 *   y            nullable: device [N] of y_dtype receives the logits; NULL
 *                skips the store.
 *   d_index      device int32: receives the index (-1 if every value is NaN).
 *   d_value      nullable device fp32: receives the maximum (its value;
 *                a maximum of -0 reads +0).
 *   d_workspace  device, qmv_argmax_workspace_bytes() bytes, 8-byte aligned,
 *                all zero before the first call; every completed call leaves
 *                it zero.  Calls sharing a workspace must not overlap.
 * The index is exact against the oracle in QMV_EXACT mode.  Needs
 * K % 256 == 0 (the M = 1 pipeline); QMV_ERR_UNSUPPORTED otherwise.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA.
 */
QMV_API size_t qmv_argmax_workspace_bytes(void);
QMV_API int qmv_gemv_argmax(const qmv_pack *p, const void *x, const void *residual,
                            const void *gamma, float eps, void *h_out, void *y, int y_dtype,
                            int mode, int *d_index, float *d_value, void *d_workspace,
                            void *stream);

/*
 * qmv_gemv_gather -- the expert-gather matvec of a mixture-of-experts decode
 * step, with no gathered copy of the weights ([PLAY] ranked-targets table,
 * MoE row: a zero-materialization expert-gather matvec): the pack holds E = N / rows_per_expert experts
 * of rows_per_expert rows each, stacked; for the n_selected expert ids in
 * d_expert_ids, y[j*rows_per_expert + r] = (row r of expert ids[j]) . x, for
 * M = 1, computed exactly as qmv_gemv computes those rows (the row groups of
 * the selected experts are fetched by index inside the kernel).
 *   rows_per_expert  divides N.
 *   d_expert_ids     device int32 [n_selected], 1 <= n_selected <= 256; may be
 *                    written by the kernel launched just before (it is read
 *                    after that kernel completes).  An id outside [0, E)
 *                    yields zero outputs for its rows and sets the device
 *                    error word (8).
 *   x  device fp16 [K];  y  device [n_selected * rows_per_expert] of y_dtype.
 * Needs K % 256 == 0 (the M = 1 pipeline).
 * Errors: INVALID_ARG, SHAPE, ALIGNMENT, UNSUPPORTED, CUDA.
 */
QMV_API int qmv_gemv_gather(const qmv_pack *p, int rows_per_expert, const int *d_expert_ids,
                            int n_selected, const void *x, void *y, int y_dtype, int mode,
                            void *stream);

/*
 * qmv_unpack_codes -- decode the packed words back to signed int8 codes
 * [N][K] with the same decode routine the matvec kernels use (a check of
 * that routine; not on the hot path).  d_codes_out: device int8, N*K bytes.
 */
QMV_API int qmv_unpack_codes(const qmv_pack *p, int8_t *d_codes_out, void *stream);

/* qmv_pack_info -- read back a pack's shape (any out pointer may be NULL). */
QMV_API int qmv_pack_info(const qmv_pack *p, int *N, int *K, int *bits, int *group);

/*
 * Saving and reloading packed weights.  A saved pack is its 64-byte header
 * followed by the bytes of d_codes and of d_scales exactly as
 * qmv_pack_weights wrote them (the caller copies them; the library does no
 * file or host I/O).  Header, little-endian:
 *   bytes  0..7   magic "QMVPACK" and a zero byte
 *   bytes  8..11  uint32 layout version (QMV_PACK_VERSION: the packed-word
 *                 layout of qmv_pack_weights; any other version is refused)
 *   bytes 12..15  uint32 header size (64)
 *   bytes 16..31  int32 N, K, bits, group
 *   bytes 32..47  uint64 codes_bytes, scales_bytes
 *   bytes 48..63  zero
 */
#define QMV_PACK_HEADER_BYTES 64
#define QMV_PACK_VERSION 1

/* qmv_pack_header -- write the header of pack p to header_out (64 bytes,
 * host memory).  Errors: INVALID_ARG (p not a pack, header_out NULL).
 * Host only. */
QMV_API int qmv_pack_header(const qmv_pack *p, void *header_out);

/* qmv_create_pack_from_header -- check a saved header and describe its pack,
 * as qmv_create_pack would (codes_bytes, scales_bytes nullable).
 * Errors: INVALID_ARG (NULL, wrong magic or header size, nonzero reserved
 * bytes, bits/group not allowed), UNSUPPORTED (another layout version),
 * SHAPE (shape not allowed, or byte counts that disagree with it).  Host only. */
QMV_API int qmv_create_pack_from_header(qmv_pack **out, const void *header,
                                        size_t *codes_bytes, size_t *scales_bytes);

/* qmv_bind_packed -- bind device buffers that already hold packed words and
 * scales (the output of qmv_pack_weights for this shape, e.g. reloaded from a
 * saved pack), without packing.  d_codes, d_scales: device, 16-byte aligned,
 * codes_bytes and scales_bytes long; the pack keeps them, as with
 * qmv_pack_weights.  Errors: INVALID_ARG (NULL), ALIGNMENT.  Host only. */
QMV_API int qmv_bind_packed(qmv_pack *p, void *d_codes, void *d_scales);

/* qmv_destroy_pack -- free the host descriptor (never the device buffers). */
QMV_API int qmv_destroy_pack(qmv_pack *p);

/*
 * qmv_set_pdl -- programmatic dependent launch of the M = 1 matvec kernels
 * for the calling thread (default off).  When on, a matvec launched right
 * after another kernel in the same stream may start while that kernel is
 * still running: it begins streaming its packed weights at once and waits
 * for the previous kernel to complete (griddepcontrol.wait) before it reads
 * x / residual / gamma or writes any output.  This hides launch latency
 * between the dependent matvecs of a decode layer ([A19] "What moved the
 * needle", dispatch-count item: the per-dispatch tax between kernels).
 * Requirement: the packed weights of a matvec must not be written by the
 * kernel launched just before it in the stream (pack once, then run), nor by the
 * kernel before a run of M = 1 matvecs or M-column tiles launched with this on,
 * since those let the next one start before they have waited themselves.
 * Works under stream capture (CUDA graphs).  Always returns QMV_OK.
 * (The verification-step calls below always let their launch overlap the end of
 * the kernel before, and wait for it before they touch memory and before they let
 * the next one start; with this on, qmv_w4_gemv also begins to stream its weights
 * before that wait, under the same requirement.)
 */
QMV_API int qmv_set_pdl(int enable);

/* qmv_status_string -- static text for a status code. */
QMV_API const char *qmv_status_string(int status);

/* qmv_last_cuda_error -- the raw cudaError_t behind the calling thread's
 * last QMV_ERR_CUDA (0 if none). */
QMV_API int qmv_last_cuda_error(void);

/*
 * qmv_device_error -- the device error word of the current device: 0, or
 * the code of the first bounded device-side wait that ran out (a kernel that
 * hits one stops, lets its own copies land and returns; its outputs are then
 * incomplete).  Synchronises with the device (reads a device symbol).
 *   out    receives the word.  clear: non-zero resets it to 0.
 * Errors: INVALID_ARG (out NULL), CUDA.
 */
QMV_API int qmv_device_error(int *out, int clear);

/*
 * Chains: a sequence of M = 1 matvecs (plain or with the fused residual-add +
 * RMSNorm prologue) run by one persistent launch -- the whole-layer / multi-
 * stage single dispatch of [A19] "The parked levers" (mega-kernel item),
 * against the per-dispatch tax of "What moved the needle".  Each op computes
 * exactly what the matching qmv_gemv / qmv_fused_rmsnorm_gemv call computes
 * (bit for bit, same mode), in order.  The weight stream runs across op
 * boundaries; a grid-wide barrier is inserted only before an op whose
 * activation reads (x, residual, gamma) overlap the outputs (y, h_out) of an
 * earlier op since the last barrier, or whose outputs overlap the reads or
 * outputs of such an op.  Packed weights must not change while a chain runs.
 * Every op needs K % 256 == 0.
 *
 * qmv_chain_workspace_bytes -- device bytes a chain of up to max_ops ops
 * needs (barrier words + op table); 0 if max_ops < 1.
 */
QMV_API size_t qmv_chain_workspace_bytes(int max_ops);

/*
 * qmv_chain_create -- an empty chain using the caller's device workspace
 * (256-byte aligned, at least qmv_chain_workspace_bytes(max_ops) bytes; it
 * must outlive the chain and must not be shared by two chains that run at
 * the same time).  Host only.
 * Errors: INVALID_ARG (NULL, max_ops < 1, workspace too small), ALIGNMENT.
 */
QMV_API int qmv_chain_create(qmv_chain **out, int max_ops, void *d_workspace,
                             size_t workspace_bytes);

/*
 * qmv_chain_create_no_alloc -- an empty chain whose barrier words and op table
 * live in the library's own scratch array (a file-scope device array, one per
 * device, room for 1024 ops), so neither the caller nor the library allocates
 * device memory for it.  The source pages have no counterpart: it is an interface
 * variant of qmv_chain_create.  The array's address is looked up here, once per
 * device (host bookkeeping behind a lock, so chains may be made and run from
 * several host threads); the chain must run on the device that was current
 * here.  Every run clears the barrier words; a run after another chain used
 * the array re-copies this chain's op table on the run's stream, so runs of
 * such chains queued one after another on one stream are ordered.  Chains
 * made this way share the array: runs of two of them that overlap in time
 * on the GPU (different streams) race, and so would a run overlapping its
 * own earlier run on another stream.
 * Errors: INVALID_ARG (NULL, max_ops < 1), UNSUPPORTED (max_ops > 1024), CUDA.
 */
QMV_API int qmv_chain_create_no_alloc(qmv_chain **out, int max_ops);

/*
 * qmv_chain_add_gemv / qmv_chain_add_fused_rmsnorm_gemv -- append one M = 1
 * matvec with the arguments of qmv_gemv / qmv_fused_rmsnorm_gemv (pointers
 * are recorded, not read, until qmv_chain_run).  Host only.
 * Errors: INVALID_ARG (NULL, chain full, bad enum), ALIGNMENT, UNSUPPORTED
 * (K % 256 != 0, or K too large for the chain's shared memory).
 */
QMV_API int qmv_chain_add_gemv(qmv_chain *c, const qmv_pack *p, const void *x, void *y,
                               int y_dtype, int mode);
QMV_API int qmv_chain_add_fused_rmsnorm_gemv(qmv_chain *c, const qmv_pack *p, const void *x,
                                             const void *residual, const void *gamma, float eps,
                                             void *h_out, void *y, int y_dtype, int mode);

/*
 * qmv_chain_run -- run every op of the chain, in order, as one cooperative
 * launch of one CTA per SM on `stream` (INVALID_ARG for a chain from
 * qmv_chain_create_no_alloc run on another device).  The first run after ops
 * were added copies the op table to the workspace with an asynchronous copy
 * on `stream` (ordered after the work queued there before); a run that needs
 * that copy while `stream` is capturing returns UNSUPPORTED.  Later runs only
 * clear the barrier words (an async memset) and launch.  Two runs of chains
 * that share a workspace must not overlap on the GPU.  A bounded device wait
 * that runs out shows in qmv_device_error.
 * Errors: INVALID_ARG, UNSUPPORTED (kernel does not fit an SM, or a table
 * copy during stream capture), CUDA.
 */
QMV_API int qmv_chain_run(qmv_chain *c, void *stream);

/* qmv_chain_info -- ops, inserted grid barriers, and the kernel's dynamic
 * shared memory (any out pointer may be NULL). */
QMV_API int qmv_chain_info(const qmv_chain *c, int *n_ops, int *n_barriers, int *smem_bytes);

/* qmv_chain_destroy -- free the host descriptor (never the workspace). */
QMV_API int qmv_chain_destroy(qmv_chain *c);

/*
 * The verification step of drafted tokens: a chunk of M = S + 1 tokens (S
 * drafted ones and the last accepted one) goes through the blocks at once, and
 * its logits decide how many of the drafted tokens stand ([A19] "The parked
 * levers", the multi-token-prediction item; [PLAY] prefill-regimes table, S = 4
 * chunks on the verify lane).  Four operators of that step: the matvec for
 * 4-bit weights with a scale and a zero point a group, the norms between two
 * blocks, logits to probabilities, and the verification itself.  These calls
 * take row strides (ld*, in elements, at least the row's length), fp16 and
 * bf16, and pointers aligned to their element; the conventions at the top of
 * this file hold for the rest.  They keep no device state and need no
 * workspace, so calls may overlap on several streams.  An output that shares
 * memory with an input or another output is refused (INVALID_ARG) but where a call
 * allows it; rows of one stride may lie between each other's, as two halves of a
 * wider tensor do.
 */

/*
 * qmv_w4_create -- describe 4-bit weights w[n][k] = (q[n][k] - z[n][g]) * s[n][g]
 * with g = k / group.
 *   N, K         output and input features; N >= 1, 32 <= K <= 131072, K % 32 == 0.
 *   group        32, 64 or 128 consecutive k of a row (the last group of a row
 *                is short where K is not a multiple).
 *   scale_dtype  QMV_F16 or QMV_BF16.
 *   has_zeros    0: symmetric weights, every z is 8.
 *   packed_bytes (out, nullable) bytes the caller must allocate for the packed
 *                weights, codes, scales and zero points together.
 * Packed layout: blocks of 32 rows x 128 k, in k order within 32 rows.  A block
 * holds its codes as the tensor cores read them (two 16-row halves, two 64-k
 * tiles, 16 bytes for each lane of a warp), then its scales (groups x 32 x
 * fp16/bf16), then its zero points (groups x 32 bytes).  Rows and k past the
 * end are padded with zero scales.
 * Errors: INVALID_ARG (out NULL, group or scale_dtype not allowed), SHAPE,
 * UNSUPPORTED (K > 131072).  Host only.
 */
QMV_API int qmv_w4_create(qmv_w4pack **out, int N, int K, int group, int scale_dtype,
                          int has_zeros, size_t *packed_bytes);

/*
 * qmv_w4_pack -- pack on the device and bind the pack to d_packed.
 *   d_codes_in   device uint8 [N][K], one code a byte, 0..15 (masked to 4 bits),
 *                8-byte aligned.
 *   d_scales_in  device fp16/bf16 [N][ceil(K/group)].
 *   d_zeros_in   device uint8 [N][ceil(K/group)], 0..15 (masked); NULL exactly
 *                when has_zeros was 0.
 *   d_packed     device, packed_bytes, 16-byte aligned; the pack keeps it.
 * Errors: INVALID_ARG, ALIGNMENT, CUDA.
 */
QMV_API int qmv_w4_pack(qmv_w4pack *p, const uint8_t *d_codes_in, const void *d_scales_in,
                        const uint8_t *d_zeros_in, void *d_packed, void *stream);

/* qmv_w4_bind -- bind a device buffer that already holds the packed bytes of
 * this shape (as qmv_w4_pack left them).  Errors: INVALID_ARG, ALIGNMENT.  Host only. */
QMV_API int qmv_w4_bind(qmv_w4pack *p, void *d_packed);

/* qmv_w4_unpack -- the codes back as device uint8 [N][K] (a check of the
 * layout, not on the hot path).  Errors: INVALID_ARG, CUDA. */
QMV_API int qmv_w4_unpack(const qmv_w4pack *p, uint8_t *d_codes_out, void *stream);

/* qmv_w4_info -- read back a pack's description (any out pointer may be NULL). */
QMV_API int qmv_w4_info(const qmv_w4pack *p, int *N, int *K, int *group, int *scale_dtype,
                        int *has_zeros);

/* qmv_w4_destroy -- free the host descriptor (never the device buffer). */
QMV_API int qmv_w4_destroy(qmv_w4pack *p);

/*
 * qmv_w4_gemv -- y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] * (q[n][k] - z[n][g])
 * for M columns, computed as s * (sum(x * q) - z * sum(x)) a group, with exact
 * products and fp32 sums in a fixed order and one rounding to y's type at the
 * end.  x in bf16 is first taken to within 2^-39 of its column's largest magnitude.
 * Infinities and NaN of x act as the definition has them: each result that is
 * not finite is formed again from it, which takes far longer (43008 x 5376, one
 * column: 1.1 ms instead of 24 us).  Repeated calls give the same bits.
 *   M        1 .. 4096.
 *   x        device [M][K] of x_dtype (QMV_F16 or QMV_BF16, any mix with the
 *            scales' type), row stride ldx.
 *   y        device [M][N] of y_dtype, row stride ldy.
 * Errors: INVALID_ARG, SHAPE (ldx < K or ldy < N), ALIGNMENT, CUDA.
 */
QMV_API int qmv_w4_gemv(const qmv_w4pack *p, int M, const void *x, int ldx, int x_dtype, void *y,
                        int ldy, int y_dtype, void *stream);

/*
 * qmv_block_norm -- from a block's output y to the next block's input, for M
 * rows of D:
 *   u = y;  with gamma_post: u = u / sqrt(mean(u^2) + eps) * (gamma_post + gamma_offset);
 *   with gate: u = gate * u;
 *   h = round(residual_scale * residual + branch_scale * u)          (h_out)
 *   z = round(h / sqrt(mean(h^2) + eps) * (gamma_pre + gamma_offset)) (out)
 * with every step in fp32 but the two roundings to dtype; the second norm takes
 * h as it is stored, as qmv_fused_rmsnorm_gemv does.
 *   y          device [M][D] of y_dtype (QMV_F32, QMV_F16 or QMV_BF16), row stride ldy.
 *   residual   device [M][D] of dtype (QMV_F16 or QMV_BF16), row stride ldr.
 *   gamma_post, gamma_pre  device [D] of dtype; gamma_post nullable.
 *   gate       nullable device [M][D] of dtype, row stride ldg; ldg = 0 takes one
 *              row [D] for every m.
 *   h_out      nullable device [M][D] of dtype, row stride ldh; may be residual
 *              itself (same pointer, ldh == ldr).
 *   out        device [M][D] of dtype, row stride ldo.
 *   D          1 .. 65536.  eps >= 0.
 * out overlaps nothing; h_out overlaps nothing but residual as above.
 * Errors: INVALID_ARG, SHAPE (a stride below D), UNSUPPORTED (D), ALIGNMENT, CUDA.
 */
QMV_API int qmv_block_norm(int M, int D, const void *y, int ldy, int y_dtype, const void *residual,
                           int ldr, const void *gamma_post, const void *gate, int ldg,
                           float residual_scale, float branch_scale, const void *gamma_pre,
                           float gamma_offset, float eps, void *h_out, int ldh, void *out, int ldo,
                           int dtype, void *stream);

/*
 * qmv_softmax -- rows of logits to probabilities:
 * out[r][v] = exp((x[r][v] - max_r) / T_r) / sum_v exp((x[r][v] - max_r) / T_r).
 *   logits  device [rows][V] of dtype (QMV_F32, QMV_F16 or QMV_BF16), row stride ldl.
 *   d_temperature  nullable device fp32 [rows]: T_r; NULL takes `temperature`
 *           for every row.  T = 0 gives 1 to the row's first maximum and 0 to
 *           the rest; a negative or NaN T of d_temperature counts as 0.
 *   out     device fp32 [rows][V], row stride ldo; may be logits itself (fp32,
 *           same pointer, ldo == ldl).
 * A logit of -inf gets 0; a row of nothing but -inf gets all zeros.  A row that
 * holds NaN or +inf gives NaN in every place.
 * All steps are fp32: a probability is off by at most 2^-24 * (70 + V / 128 +
 * 3.25 |x - max| / T) of itself, and what is below 2^-126 may be 0.  T acts as it
 * is from 2^-125 to 1e37 and as those beyond.
 * Errors: INVALID_ARG (also temperature < 0 or NaN), SHAPE, ALIGNMENT, CUDA.
 */
QMV_API int qmv_softmax(int rows, int V, const void *logits, int ldl, int dtype,
                        const float *d_temperature, float temperature, float *out, int ldo,
                        void *stream);

/*
 * qmv_verify_draft -- verification of drafted tokens against the target's
 * probabilities, for B sequences of n = n_draft[b] drafted tokens (S without
 * n_draft; values are clamped to 0..S):
 *   drafted token i stands while u_accept[b][i] * q_i(d_i) < p_i(d_i), compared
 *   exactly; at the first that does not, j, the new token is drawn from
 *   max(p_j - q_j, 0) (from p_j where that has no mass); with none refused, from p_n.
 * The draw: each weight, clamped to 0..1, counts in whole units of 2^-42
 * (truncated), T is their total, U = floor(2^31 * u_sample[b]), and the token is
 * the lowest id whose running sum is above floor(U * T / 2^31).  Sums of whole
 * numbers do not depend on their order, so the result is the same on every run.
 *   target      device fp32 [B][S+1][V], p_0 .. p_S.
 *   draft_probs device fp32 [B][S][V], q; NULL for a drafter that is sure of
 *               its tokens (q is 1 at d_i and 0 elsewhere).
 *   draft       device int32 [B][S]; an id outside [0, V) is refused.
 *   n_draft     nullable device int32 [B].
 *   u_accept    device fp32 [B][S], u_sample device fp32 [B], in [0, 1).
 *   tokens      device int32 [B][S+1]: the accepted tokens, the new one, then -1.
 *               The new token is -1 where p has no mass at all.
 *   n_accepted  device int32 [B]: drafted tokens that stand.
 * S may be 0 (draft, draft_probs and u_accept are then not read and may be NULL).
 *   B 1 .. 65535, S 0 .. 1024, V 1 .. 2^20.
 * NaN in p or q refuses its token; in the draw an id whose weight is NaN (p, or where
 * max(p - q, 0) is drawn from, p or q) counts 0.
 * Errors: INVALID_ARG, UNSUPPORTED (sizes), ALIGNMENT (4 bytes), CUDA.
 */
QMV_API int qmv_verify_draft(int B, int S, int V, const float *target, const float *draft_probs,
                             const int *draft, const int *n_draft, const float *u_accept,
                             const float *u_sample, int *tokens, int *n_accepted, void *stream);

/*
 * What a decode step does around its matvecs: the heads of the fused q/k/v matvec are
 * normed and rotated, tokens are routed to experts and multiplied with their weights,
 * and the next token is drawn from the logits.  As the verification-step calls above,
 * these take row strides, fp16 and bf16, and pointers aligned to their element, refuse
 * an output that shares memory with an input or another output but where a call allows
 * it (INVALID_ARG), keep no device state, and may overlap on several streams.
 */
typedef enum { QMV_ROPE_HALF = 0, QMV_ROPE_INTERLEAVED = 1 } qmv_rope_layout;
typedef enum { QMV_SCALE_NONE = 0, QMV_SCALE_LINEAR = 1, QMV_SCALE_NTK = 2, QMV_SCALE_YARN = 3 } qmv_rope_scaling;
typedef enum { QMV_SCORE_SOFTMAX = 0, QMV_SCORE_SIGMOID = 1 } qmv_score;
typedef enum { QMV_ACT_NONE = 0, QMV_ACT_SILU = 1, QMV_ACT_GELU = 2 } qmv_act;

/*
 * qmv_rope_inv_freq -- the angle a position of each of rot / 2 pairs, in radians:
 *   QMV_SCALE_NONE    w_i = base^(-2 i / rot)
 *   QMV_SCALE_LINEAR  w_i / factor
 *   QMV_SCALE_NTK     w_i of the base base * factor^(rot / (rot - 2))
 *   QMV_SCALE_YARN    w_i / factor * r_i + w_i * (1 - r_i), with the ramp r_i = (i - lo) / (hi - lo)
 *                     kept in 0..1 between lo, the pair that turns beta_fast times in
 *                     original_length positions (rounded down), and hi, the one that turns
 *                     beta_slow times (rounded up); *amplitude = 0.1 ln(factor) + 1 for
 *                     factor > 1.
 *   rot        even, 2 .. 1024 (above 2 for QMV_SCALE_NTK).   base > 1, factor > 0.
 *   inv_freq   host double [rot / 2];  amplitude (nullable) receives 1 where not stated.
 * Errors: INVALID_ARG (also original_length or a beta that is not above 0 for YARN),
 * SHAPE (rot).  Host only.
 */
QMV_API int qmv_rope_inv_freq(int rot, double base, int scaling, double factor, double original_length,
                              double beta_fast, double beta_slow, double *inv_freq, float *amplitude);

/*
 * qmv_rope_turns -- frequencies as qmv_qk_norm_rope takes them: turns a position, without
 * the whole ones, in units of 2^-64 (host int64 [n], for the caller to copy to the device).
 * A position times this, modulo 2^64, is its angle: exact however far the position, up to
 * the frequency's own 53 bits.  Any finite frequencies will do.
 * Errors: INVALID_ARG (NULL, n < 1, a frequency that is not finite).  Host only.
 */
QMV_API int qmv_rope_turns(int n, const double *inv_freq, int64_t *turns);

/*
 * qmv_qk_norm_rope -- norms of query and key heads and their position rotation, for M
 * rows as a fused q/k/v matvec leaves them: n_q query heads of D, then n_k key heads, then
 * anything (values), which is not read.  For each head
 *   u = x;  with its gamma: u = x / sqrt(mean(x^2) + eps) * (gamma + gamma_offset);
 *   pairs (a, b) of the first rot elements become amplitude * (a cos t - b sin t,
 *   b cos t + a sin t), t = position * frequency; the others stay u.
 * QMV_ROPE_HALF pairs element i with i + rot / 2, QMV_ROPE_INTERLEAVED 2 i with 2 i + 1.
 * Steps are fp32 with one rounding to dtype; cosines and sines are within 2^-21.  (So the squares of a
 * normed head have to stay below 2^128: with values from 2^64 / sqrt(D) on it becomes 0.)
 *   qkv        device [M][(n_q + n_k) * D, at least] of x_dtype (QMV_F32, QMV_F16 or QMV_BF16),
 *              row stride ld.
 *   positions  device int32 [M] (negative ones turn back); NULL exactly when rot is 0.
 *   turns      device int64 [rot / 2] from qmv_rope_turns, 8-byte aligned; NULL exactly when rot is 0.
 *   gamma_q, gamma_k  nullable device [D] of dtype.
 *   q, k       device [M][n_q * D] and [M][n_k * D] of dtype (QMV_F16 or QMV_BF16), row strides
 *              ldq, ldk; q is NULL exactly when n_q is 0, k when n_k is 0.  Either may be its
 *              own place in qkv (same pointer, stride and type).
 *   M >= 1; n_q, n_k 0 .. 4096, not both 0; D 1 .. 1024; rot even, 0 .. D; eps >= 0.
 * Errors: INVALID_ARG, SHAPE (a stride below its row, rot), UNSUPPORTED (sizes), ALIGNMENT, CUDA.
 */
QMV_API int qmv_qk_norm_rope(int M, int n_q, int n_k, int D, const void *qkv, int ld, int x_dtype,
                             const int *positions, const int64_t *turns, int rot, int layout,
                             float amplitude, const void *gamma_q, const void *gamma_k,
                             float gamma_offset, float eps, void *q, int ldq, void *k, int ldk,
                             int dtype, void *stream);

/*
 * qmv_route -- the T experts of each of M tokens and their weights, from router logits:
 *   s[e] = softmax or sigmoid of the row;  r[e] = s[e] + bias[e] (s[e] without bias);
 *   with groups > 1 (of E / groups neighbouring experts): a group counts the sum of its
 *   group_top largest r, and only the experts of the best group_k groups remain;
 *   ids = the T largest r, the largest first;  weights = s of those, over their sum where
 *   renormalise is not 0 (0 where that sum is 0 in 64 bits), times scale.
 * Equal ones go to the lowest index.  r is compared as 64-bit arithmetic would have it: where
 * fp32 cannot tell two apart they are formed again in 64 bits.  Without bias experts are compared
 * by their logits, which is the order of exact scores also where those of 64 bits are equal: of
 * sigmoid logits 40 and 41, both scores 1 there, 41 comes first, with a bias of 0 the lower
 * index.  The sums of two that groups count are of 64-bit scores, with a bias or without.
 * Weights are fp32, within 2^-20 of themselves, or 2^-126 of scale.
 * An expert whose logit or bias is NaN or -inf is never chosen (nor counted in a
 * group, as -inf: with group_top 2 a group of one expert alone counts as -inf); places
 * that are left over hold id -1 and weight 0.  Logits of +inf share a softmax evenly.
 *   logits   device [M][E] of dtype (QMV_F32, QMV_F16 or QMV_BF16), row stride ldl.
 *   bias     nullable device fp32 [E].
 *   ids      device int32 [M][T], as qmv_w4_experts and (a row at a time) qmv_gemv_gather take them.
 *   weights  device fp32 [M][T].
 *   M >= 1; E 1 .. 1024; T 1 .. 64; groups 1 .. 32 divides E; group_k 1 .. groups; group_top 1 or 2;
 *   T <= group_k * E / groups, group_top <= E / groups.
 * Errors: INVALID_ARG (also score), SHAPE (counts that do not go together, ldl), UNSUPPORTED
 * (E, T or groups above their limits), ALIGNMENT, CUDA.
 */
QMV_API int qmv_route(int M, int E, int T, const void *logits, int ldl, int dtype, int score,
                      const float *bias, int groups, int group_k, int group_top, int renormalise,
                      float scale, int *ids, float *weights, void *stream);

/*
 * qmv_w4_experts -- products of 4-bit expert weights with the tokens routed to them.  The
 * pack holds E = N / rows_per_expert experts of R = rows_per_expert rows, stacked; for token m
 * and its j-th expert e = ids[m][j]
 *   y[m][j] = W_e . x(m, j)       (weights NULL), or   y[m] = sum_j weights[m][j] * (W_e . x(m, j)),
 * with x(m, j) row m of x (per_pair 0) or its row m * T + j (per_pair not 0); with act that
 * row is [2 K], gate then up, and x(m, j) = act(gate) * up, formed in fp32 and rounded to
 * x_dtype, as an activation of its own would leave it: QMV_ACT_SILU g / (1 + exp(-g)),
 * QMV_ACT_GELU g / 2 * (1 + tanh(sqrt(2 / pi) * (g + 0.044715 g^3))).
 * Exact products, fp32 sums in a fixed order, one rounding to y's type; x in bf16 as in
 * qmv_w4_gemv.  Repeated calls give the same bits; among other tokens a token's fp32 sums may be
 * split, and so rounded, in another way.  Infinities and NaN of x act as the definition has
 * them, in their own row; products that are not finite are formed one by one, which takes some
 * hundred times as long.
 *   rows_per_expert  divides the pack's N and is a multiple of 32.
 *   ids      device int32 [M][T]; may come from the kernel just before.  An id outside [0, E)
 *            has the product 0; but for -1 it sets the device error word (8).
 *   weights  nullable device fp32 [M][T].
 *   x        device, M or M * T rows of K (2 K with act) of x_dtype (QMV_F16 or QMV_BF16), row stride ldx.
 *   y        device [M][T][R], or [M][R] with weights, of y_dtype, row stride ldy (of M * T or M rows of R).
 *   d_workspace, workspace_bytes  caller scratch, 256-byte aligned, at least
 *            qmv_w4_experts_workspace_bytes(p, rows_per_expert, M, T) bytes, which is enough for calls of
 *            every form of up to M tokens and T experts (0 where such a call is refused); its contents on
 *            entry do not matter; calls that share a workspace must not overlap.
 *   M 1 .. 4096; T 1 .. 64; M * T <= 32768; E <= 1024; K <= 16384; R <= 2^20.
 * Errors: INVALID_ARG, SHAPE (rows_per_expert, strides), UNSUPPORTED (sizes), ALIGNMENT, WORKSPACE, CUDA.
 */
QMV_API size_t qmv_w4_experts_workspace_bytes(const qmv_w4pack *p, int rows_per_expert, int M, int T);
QMV_API int qmv_w4_experts(const qmv_w4pack *p, int rows_per_expert, int M, int T, const int *ids,
                           const float *weights, const void *x, int ldx, int per_pair, int x_dtype,
                           int act, void *y, int ldy, int y_dtype, void *d_workspace,
                           size_t workspace_bytes, void *stream);

/*
 * qmv_w4_experts_form -- the same call with scratch for its own form alone: at least
 * qmv_w4_experts_form_bytes of its arguments.  That counts the pairs in order where M * T > 128, the rows of
 * x that are made (none for fp16 without act, x 16-byte aligned and ldx a multiple of 8; M, or with
 * per_pair M * T, of K otherwise) and the products that are summed (M * T of R, weights only).  It may be 0,
 * and d_workspace NULL then.  (4096 tokens of 8 experts of 4096 rows, K = 2048, fp16 without weights: 0.7 MB;
 * for every form 672 MB.)
 *   weighted  not 0 where the call has weights.   x  read for its alignment alone.
 */
QMV_API size_t qmv_w4_experts_form_bytes(const qmv_w4pack *p, int rows_per_expert, int M, int T, int weighted,
                                         const void *x, int ldx, int per_pair, int x_dtype, int act);
QMV_API int qmv_w4_experts_form(const qmv_w4pack *p, int rows_per_expert, int M, int T, const int *ids,
                                const float *weights, const void *x, int ldx, int per_pair, int x_dtype,
                                int act, void *y, int ldy, int y_dtype, void *d_workspace,
                                size_t workspace_bytes, void *stream);

/*
 * qmv_sample -- one token a row of logits, from given random numbers.  In a row, with T its
 * temperature and top its largest logit, the weight of id v is in whole units of 2^-42
 *   w[v] = floor(2^42 * 2^-z),  z = min((top - x[v]) * c, 64),  c = log2(e) / T,
 * each step one fp32 operation: with n = z rounded to a whole number (ties to even) and
 * f = n - z, 2^-z is 2^-n * P(f), P the polynomial with the coefficients 1,
 * 0.6931471824645996, 0.2402234971523285, 0.055503811687231064, 0.00966636836528778,
 * 0.0013381302123889327 (from f^0 on) in fused multiply-adds, the highest first: within 2^-21
 * of 2^f.  Sums of whole numbers do not depend on their order, so a row gives the same token
 * on every run.  In the order of logits, the largest first, equal ones by id:
 *   top-k  the first k stay (k = 0: all);
 *   top-p  of those the fewest first ones stay whose sum is at least floor(P * S / 2^31), S the sum
 *          of what top-k left, P = floor(2^31 * top_p); the first one in any case (top_p >= 1: all);
 *   min-p  of those stay the ones with w >= floor(2^42 * min_p) (min_p = 0: all).
 * The token is the lowest id, among those that stay, whose running sum in the order of ids
 * is above floor(U * W / 2^31), W the whole sum and U = floor(2^31 * u).
 * T = 0 gives the row's first maximum.  NaN and -inf are never drawn; a row of nothing else
 * gives -1.  +inf is drawn evenly among its like.
 *   logits  device [rows][V] of dtype (QMV_F32, QMV_F16 or QMV_BF16), row stride ldl.
 *   d_temperature, d_top_k, d_top_p, d_min_p  nullable device [rows] (int32 for top_k, fp32
 *           otherwise): a row's own setting; NULL takes the number beside it for all.
 *           Their values act as the nearest allowed ones, NaN as 0 (top_p: as 1); a T below 2^-100 that
 *           is not 0 as that.
 *   u       device fp32 [rows] in [0, 1).
 *   tokens  device int32 [rows].
 *   rows >= 1; V 1 .. 2^20; temperature >= 0, top_k >= 0, top_p and min_p 0 .. 1.
 * Errors: INVALID_ARG, SHAPE (ldl), UNSUPPORTED (V), ALIGNMENT, CUDA.
 */
QMV_API int qmv_sample(int rows, int V, const void *logits, int ldl, int dtype,
                       const float *d_temperature, float temperature, const int *d_top_k, int top_k,
                       const float *d_top_p, float top_p, const float *d_min_p, float min_p,
                       const float *u, int *tokens, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_H */
