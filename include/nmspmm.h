/*
 * nmspmm.h -- C ABI of the B200 (sm_100a) N:M sparse weight x dense activation
 * GEMM library (libnmspmm.so).
 *
 * The operation is the one of "Realizable N:M Sparse Transformer Inference via
 * Search-Kernel Co-Design" (arXiv 2607.12505):
 *   - section 2.1: N:M semi-structured sparsity keeps N non-zeros in every
 *     group of M weights of the projection and FFN linears;
 *   - section 4.1: the kernel rests on three mechanisms -- weight packing for
 *     decode-friendly storage, micro-dense execution, adaptive parallelism;
 *   - section 4.2: only the N kept values of each window are materialised in
 *     dense, MMA-shaped tiles; the packed weight carries values and their
 *     in-window positions together, so no separate index load is needed.
 *
 * Conventions for every entry point:
 *   - Pointers named *_dev are device pointers of the current CUDA device;
 *     *_host are host pointers.  The caller owns every buffer it passes.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Calls are stream-ordered and never synchronise the host unless
 *     stated.
 *   - Errors are returned as nm_status, never thrown or trapped; a message for
 *     the last failing call of the calling thread is in nm_last_error().
 *   - Layouts are row-major: W [n_out][k] (the PyTorch Linear layout),
 *     X [T][k], Y [T][n_out].
 */
#ifndef NMSPMM_H
#define NMSPMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NM_OK = 0,
    NM_ERR_INVALID = 1,     /* bad argument: null pointer, bad size, misalignment */
    NM_ERR_UNSUPPORTED = 2, /* valid request the library does not implement       */
    NM_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed                  */
    NM_ERR_OOM = 4,         /* device allocation failed                           */
    NM_ERR_TIMEOUT = 5      /* a kernel gave up a bounded wait (see nm_device_status) */
} nm_status;

typedef enum {
    NM_INT8 = 0,
    NM_FP16 = 1,
    NM_BF16 = 2,
    NM_FP32 = 3,            /* nm_compress_mx, nm_mx_quantize and nm_mx_dequantize only */
    NM_MXFP4 = 4            /* what nm_query reports for a handle of nm_compress_mx    */
} nm_dtype;

/* Opaque handle holding one compressed weight; owns all device memory it allocates. */
typedef struct nm_handle nm_handle;

/*
 * nm_compress -- prune and pack one weight (paper sections 2.1 and 4.2,
 * "weight packing").
 *
 * For every row n and every group g of M consecutive k positions (aligned at
 * k = 0) keeps the N entries of largest |W|, ties to the lower position, and
 * builds two device images inside the new handle:
 *   - the canonical compressed format (see nm_export), and
 *   - the packed operand image the SpMM kernel streams: per 128-row x k-block
 *     tile, the kept values already laid out as swizzled tensor-core operand
 *     rows, followed by their 2-bit in-window positions in the layout the
 *     sparse tensor core reads.
 *
 * W_dev   [n_out][k] of dtype `dt`, 16-byte aligned.  It may be freed once the
 *         stream has passed this call.
 * (N, M)  one of (1,4), (2,4), (2,8), (4,8), or N == M with M in {4, 8}
 *         (dense pass-through).  Other pairs -> NM_ERR_UNSUPPORTED.
 * k       multiple of M (else NM_ERR_INVALID); n_out, k > 0, at most 2^24;
 *         for NM_INT8 k at most 2^17 (so that k * 128 * 127 fits the int32
 *         accumulator exactly), else NM_ERR_UNSUPPORTED.
 * out     receives the handle; *out is NULL on failure.
 * Allocates device memory (NM_ERR_OOM on failure); returns without waiting
 * for the kernels.
 */
nm_status nm_compress(const void* W_dev, int64_t n_out, int64_t k, nm_dtype dt, int N, int M,
                      void* stream, nm_handle** out);

/*
 * nm_spmm_noalloc -- the same product as nm_spmm for callers that cannot
 * allocate device memory.  (The paper has no counterpart: this is a
 * deployment variant.)  Such callers include serving engines that hand
 * nearly all of HBM to their own pool up front, so a library cudaMalloc would
 * fail, and latency-critical code that must not call cudaMalloc/cudaFree,
 * which can synchronise the device and take a process-wide lock.
 *
 * Arguments, layouts, rounding and results are those of nm_spmm.  The
 * difference is where the scratch of a global-memory split-K (partial tiles
 * and per-tile arrival counters) lives: in one fixed array inside the
 * library, 4 MiB of partials plus 1024 counters.  Every GPU that loads the
 * library holds that array until the process exits.  This call never calls
 * cudaMalloc, cudaFree or any allocating routine.
 *   - The planner's own plans never use the array: they either do not split
 *     k or reduce the splits on chip (see nm_spmm).  Only a global-memory
 *     split forced through the environment (NMSPMM_FORCE_SPLITK with
 *     NMSPMM_SPLIT_GLOBAL=1, or more than 8 splits) uses it, and only then do
 *     the size limit and the race below apply.
 *   - The first call on a device looks up the array's device address with
 *     cudaGetSymbolAddress (set-up, once per device, with that device
 *     current); make that first call before any stream capture.
 *   - A shape whose split-K plan needs more than the array holds is rejected
 *     with NM_ERR_UNSUPPORTED and a message naming the sizes; nm_spmm handles
 *     it instead.
 *   - All calls share the array and it keeps the last call's contents; each
 *     call clears the counters it uses (an asynchronous memset on `stream`).
 *     Calls whose kernels overlap on the GPU (different streams, or different
 *     host threads) race on the array: order them.
 */
nm_status nm_spmm_noalloc(const nm_handle* h, const void* X_dev, int64_t T, void* Y_dev,
                          const float* scale_dev, void* stream);

/*
 * nm_recompress -- prune and pack a new weight of the handle's shape, dtype and
 * N:M into the handle's existing device buffers (a weight update; same rule
 * and layouts as nm_compress).  Allocates nothing; stream-ordered, so an
 * nm_spmm on the same stream afterwards sees the new weight.  W_dev element
 * aligned, [n_out][k].
 */
nm_status nm_recompress(nm_handle* h, const void* W_dev, void* stream);

/*
 * nm_spmm -- Y = X . Wm^T with Wm the masked weight of `h` (paper section 4.2,
 * micro-dense execution; section 4.1, adaptive parallelism).
 *
 * X_dev     [T][k] of the handle's dtype, 16-byte aligned, k * sizeof(dtype)
 *           a multiple of 16 bytes (else NM_ERR_UNSUPPORTED).
 * Y_dev     [T][n_out]:
 *             INT8, scale_dev == NULL : int32, exact integer result;
 *             INT8, scale_dev != NULL : float32, (float)acc * scale[n]
 *                                       (round-to-nearest, one multiply);
 *             FP16/BF16               : same dtype as X, rounded to nearest
 *                                       once from the fp32 accumulator
 *                                       (times scale[n] when given).  The
 *                                       accumulator is the tensor core's, which
 *                                       truncates: it is within (k / 8 + 4) 2^-23
 *                                       sum |x| |w| of the exact sum.
 *           Must be 16-byte aligned and must not overlap X.
 * scale_dev float32 [n_out] or NULL.
 * T         in [0, 2^31 - 256] (above: NM_ERR_UNSUPPORTED); T == 0 is a no-op
 *           returning NM_OK.
 * The kernel, token tile and split-K factor are chosen per (T, k, n_out,
 * N:M, dtype) so that small token counts still occupy the SMs (section 4.1,
 * mechanism 3; nm_plan_query reports the choice).  A split chosen by the
 * planner puts the k-splits of one output tile on the CTAs of one
 * thread-block cluster, which sum their partial tiles through distributed
 * shared memory: no workspace, no allocation.  A global-memory split-K
 * (forced through the environment: NMSPMM_FORCE_SPLITK with
 * NMSPMM_SPLIT_GLOBAL=1, or more than 8 splits) uses the handle's workspace:
 * calls on one handle must then not overlap on the GPU, and the first such
 * call allocates the workspace (after a device synchronisation; make it
 * before any stream capture).  Otherwise never synchronises.
 */
nm_status nm_spmm(const nm_handle* h, const void* X_dev, int64_t T, void* Y_dev,
                  const float* scale_dev, void* stream);

/*
 * Fused output stage of nm_spmm_ex.  The paper stops at the MMA (section 4.2)
 * and does not discuss the output stage; this is the library's definition.
 * Per output element, in fp32, each step rounded to nearest:
 *   v = acc                         INT8: (float)acc; FP16/BF16: the fp32 sum
 *   v = v * scale[n]                if scale != NULL
 *   v = v + bias[n]                 if bias != NULL
 *   v = v/2 * (1 + erf(v/sqrt 2))   if act == NM_ACT_GELU (erf form of GELU)
 * then stored as the output type:
 *   NM_OUT_FP32                     v
 *   NM_OUT_FP16 / NM_OUT_BF16       v rounded to nearest even
 *   NM_OUT_INT8                     clamp(round_half_even(v * out_scale), -128, 127)
 *   NM_OUT_INT32                    the raw INT8 accumulator (no scale, bias
 *                                   or activation allowed)
 *   NM_OUT_DEFAULT                  INT8: INT32 when scale, bias and act are
 *                                   all absent, else FP32; FP16/BF16: the
 *                                   input's type.
 * With act == NM_ACT_NONE and an INT8 handle the result is exactly fixed.  The
 * GELU evaluates erf by formula 7.1.26 of Abramowitz and Stegun (absolute error
 * at most 1.5e-7) with the GPU's approximate reciprocal and power of two; the
 * GELU value g of a pre-activation v is within 4e-7 |v| + 2e-6 |GELU(v)| of the
 * exact one.
 */
typedef enum {
  NM_OUT_DEFAULT = 0,
  NM_OUT_INT32 = 1,
  NM_OUT_FP32 = 2,
  NM_OUT_FP16 = 3,
  NM_OUT_BF16 = 4,
  NM_OUT_INT8 = 5
} nm_out_type;

typedef enum {
  NM_ACT_NONE = 0,
  NM_ACT_GELU = 1,
  NM_ACT_SILU = 2,     /* gated products only: v / (1 + exp(-v)) */
  NM_ACT_RELU = 3      /* gated products only: max(v, 0)         */
} nm_act;

typedef struct nm_epilogue {
  nm_out_type out;     /* element type of Y */
  nm_act act;          /* activation after scale and bias */
  const float* scale;  /* device float32 [n_out], 4-byte aligned, or NULL */
  const float* bias;   /* device float32 [n_out], 4-byte aligned, or NULL */
  float out_scale;     /* NM_OUT_INT8 only: multiplier before rounding; finite and > 0 */
} nm_epilogue;

/*
 * nm_spmm_ex -- nm_spmm with the fused output stage above: Y = out(act(
 * (X . Wm^T) * scale + bias)).  Arguments, alignment, the no-op for T == 0,
 * the workspace rule and the never-synchronise rule are those of nm_spmm; Y_dev
 * holds elements of the chosen output type.  ep == NULL is nm_spmm with no
 * scale.
 * Errors: NM_ERR_INVALID for an unknown out/act value, NM_OUT_INT32 together
 * with scale, bias or act, a misaligned scale/bias, or NM_OUT_INT8 with an
 * out_scale that is not finite and positive; NM_ERR_UNSUPPORTED for
 * NM_OUT_INT32 or NM_OUT_INT8 on an FP16/BF16 handle.
 */
nm_status nm_spmm_ex(const nm_handle* h, const void* X_dev, int64_t T, void* Y_dev,
                     const nm_epilogue* ep, void* stream);

/*
 * nm_compress_tile -- prune and pack one weight with a pattern shared by each
 * tile of 128 consecutive output channels (the vector-wise reading of the
 * paper's section 4.2: kept values become dense MMA tiles and the activations
 * are gathered to match, which needs one set of kept positions per tile of
 * channels).
 *
 * For every tile of rows [128t, 128t + 128) (the last may be shorter) and
 * every group g of M consecutive k positions, the score of position p is
 * sum over the tile's rows of |W[n][gM + p]|, computed exactly; the N
 * positions of largest score are kept, ties to the lower position, and every
 * row of the tile keeps them.  The handle holds the canonical format (exactly
 * as nm_compress lays it out, nm_export) and a dense operand image over the
 * kept k only (K' = k * N / M per row) plus the tile's kept k list, which
 * nm_spmm_gather uses to gather rows of the activation.
 *
 * Arguments as nm_compress, except:
 *   dt      NM_INT8 or NM_FP16 (scores of bfloat16 weights are not exact in
 *           any fixed-width sum: NM_ERR_UNSUPPORTED);
 *   (N, M)  one of (1,4), (2,4), (2,8), (4,8), or N == M with M in {4, 8}.
 * nm_recompress, nm_decompress, nm_export, nm_query and nm_destroy accept the
 * handle; nm_spmm, nm_spmm_ex and nm_spmm_noalloc reject it (NM_ERR_INVALID):
 * its product is nm_spmm_gather.
 */
nm_status nm_compress_tile(const void* W_dev, int64_t n_out, int64_t k, nm_dtype dt, int N, int M,
                           void* stream, nm_handle** out);

/*
 * nm_spmm_gather -- Y = X . Wm^T for a handle made by nm_compress_tile, with
 * the activation given feature-major: Xt_dev [k][ldx] holds X[t][kk] at
 * Xt_dev[kk * ldx + t].  Per 128-channel tile the kernel gathers the kept rows
 * of Xt (16-byte asynchronous copies, eight threads per 128-byte token run)
 * into a dense operand and runs dense tensor-core MMAs over K' = k * N / M
 * only, so both the MMA work and the activation bytes read per tile shrink by
 * N / M.  Environment NMSPMM_GATHER_TMA=1 gathers with four-row tensor copies
 * instead (same results; slower on B200).
 *
 * Xt_dev    16-byte aligned; ldx >= T and ldx * sizeof(dtype) a multiple of
 *           16 bytes (else NM_ERR_INVALID).  Columns t >= T are not read.
 * Y_dev     [T][n_out], 16-byte aligned, not overlapping Xt; element type and
 *           rounding exactly as nm_spmm (INT8: int32, or float32 with scale;
 *           FP16: fp16 from the fp32 accumulator).
 * scale_dev float32 [n_out] or NULL.
 * T         in [0, 2^31 - 256] (above: NM_ERR_UNSUPPORTED); T == 0 is a no-op.
 * The default plan never splits k, so the call allocates nothing and never
 * synchronises; a split-K plan forced through NMSPMM_FORCE_SPLITK reduces in
 * global memory and uses the handle's workspace under the rules of nm_spmm
 * (the first such call allocates it, after a device synchronisation).
 */
nm_status nm_spmm_gather(const nm_handle* h, const void* Xt_dev, int64_t ldx, int64_t T, void* Y_dev,
                         const float* scale_dev, void* stream);

/*
 * nm_spmm_gather_ex -- nm_spmm_gather with the fused output stage of
 * nm_spmm_ex (nm_epilogue above): Y = out(act((X . Wm^T) * scale + bias)), the same
 * definition, element types, rounding and argument checks as nm_spmm_ex; the
 * activation arguments (Xt_dev, ldx, T) and their checks are those of
 * nm_spmm_gather.  ep == NULL is nm_spmm_gather without a scale.
 */
nm_status nm_spmm_gather_ex(const nm_handle* h, const void* Xt_dev, int64_t ldx, int64_t T, void* Y_dev,
                            const nm_epilogue* ep, void* stream);

/*
 * Gated feed-forward block.  (No counterpart in the paper, whose feed-forward
 * linears are ungated: it is the same N:M product with a gated output stage.)
 *
 * nm_compress_gated -- prune and pack the two projections of a gated block.
 * W_dev [2 n_ff][k] holds the n_ff rows of the gate projection, then the n_ff
 * rows of the up projection.  Pruning, formats, limits and errors are those of
 * nm_compress for the [2 n_ff][k] weight; the packed image interleaves 16 gate
 * rows with their 16 up rows so that one accumulator tile holds both.
 * nm_recompress, nm_decompress, nm_export and nm_query (n_out = 2 n_ff) accept
 * the handle and see W's own row order; the ungated products reject it.
 */
nm_status nm_compress_gated(const void* W_dev, int64_t n_ff, int64_t k, nm_dtype dt, int N, int M, void* stream,
                            nm_handle** out);

/*
 * nm_spmm_gated -- both projections, the activation and the product in one
 * kernel:
 *   p[t][r] = acc(X . Wm^T)[t][r] * scale[r] + bias[r]      r in [0, 2 n_ff)
 *   Y[t][f] = act(p[t][f]) * p[t][n_ff + f]                 f in [0, n_ff)
 * with acc the accumulator of nm_spmm, in fp32, each step rounded to nearest as in
 * nm_spmm_ex, Y rounded once to its type.  act is any nm_act.  ep->scale and
 * ep->bias are [2 n_ff] (or NULL); output types, errors and defaults are
 * nm_spmm_ex's, but NM_OUT_INT32 is refused, and the default of an INT8 handle is
 * fp32.  ep == NULL: NM_ACT_SILU, default output.  The SiLU is within
 * (6e-7 + 1.3e-7 max(0, -v)) |SiLU(v)| + 1.1e-36 of the exact one (below -87.33,
 * where the reciprocal of 1 + exp(-v) is subnormal, it is -0).
 *
 * P_dev, if not NULL, receives p itself, [T][2 n_ff] in the handle's type
 * (FP16/BF16; an INT8 handle refuses it with NM_ERR_UNSUPPORTED): what
 * nm_gated_backward needs.  16-byte aligned, overlapping neither X nor Y.
 * X, T (at most 2^31 - 256), alignment and streams as nm_spmm.  Never allocates or
 * synchronises and keeps nothing between calls: calls on one handle may overlap.
 */
nm_status nm_spmm_gated(const nm_handle* h, const void* X_dev, int64_t T, void* Y_dev, void* P_dev,
                        const nm_epilogue* ep, void* stream);

/*
 * nm_gated_backward -- gradients of the gated block of an FP16 or BF16 handle
 * (made by nm_compress_gated; INT8: NM_ERR_UNSUPPORTED).  With g, u the two
 * halves of p (as nm_spmm_gated saved it, computed without a scale):
 *   dp[t][f]        = dY[t][f] * u * act'(g)      (RELU: act'(0) = 0)
 *   dp[t][n_ff + f] = dY[t][f] * act(g)
 *   dX [T][k]       = dp . Wm
 *   dW [2 n_ff][k]  = dp^T . X      the gradient of Wm at every position; a
 *                     pruned weight's own gradient is zero (mask it), while
 *                     straight-through training uses all of it
 *   dbias [2 n_ff]  = sum over t of dp, fp32
 * dX and dW have the handle's type.  dp is computed in fp32; the two products
 * read it rounded to the handle's type (their tensor-core operand), sum in fp32
 * and round once; dbias sums the unrounded fp32 values, in a fixed order.
 * Results do not depend on timing.  The tensor core truncates its accumulator, so
 * one holds at most 2^14 products; the runs of a longer sum are added in fp32,
 * rounded to nearest.  With h half a unit of the handle's type (2^-11, 2^-8) and A
 * the sum of |dp| |Wm| (dW: |dp| |X|) over the n = 2 n_ff (dW: T) terms, a result r
 * is within (h + min(n, 2^14) 2^-26 + 2^-17 + n 2^-38) A + h |r| of the exact one.
 * FP16: dp keeps the range of fp32, not fp16's.  Where the largest finite |dp| is
 * outside [2^-4, 2^15) it is stored times a power of two, which the products undo
 * (a second pass over P and dY); an element of dp is then off by h |dp| + 2^-21
 * of the largest |dp| at most.
 *
 * dX_dev, dW_dev, dbias_dev: any may be NULL (not computed), not all three.
 * X_dev [T][k] (needed for dW only, else may be NULL), P_dev [T][2 n_ff],
 * dY_dev [T][n_ff], all in the handle's type, all pointers 16-byte aligned;
 * k a multiple of 8 and T at most 2^26 (else NM_ERR_UNSUPPORTED).  T == 0 writes
 * zeros to dW and dbias.  ws_dev: device workspace of at least nm_gated_backward_workspace
 * bytes, 16-byte aligned, for this call alone until it has run; calls that
 * overlap need one each.  Outputs and workspace overlap nothing else.
 */
nm_status nm_gated_backward_workspace(const nm_handle* h, int64_t T, size_t* bytes);
nm_status nm_gated_backward(const nm_handle* h, const void* X_dev, const void* P_dev, const void* dY_dev, int64_t T,
                            nm_act act, void* dX_dev, void* dW_dev, float* dbias_dev, void* ws_dev, size_t ws_bytes,
                            void* stream);

/*
 * nm_gated_backward_plan_for_shape -- test and diagnostic hook: how
 * nm_gated_backward would share out the two products of this shape (those asked
 * for) over a GPU with `sms` SMs.  Touches no device.  The environment overrides
 * NMSPMM_FORCE_GRAD_BN and NMSPMM_GRAD_SPLIT apply.  Errors: NM_ERR_INVALID for a
 * null pointer or a bad shape, NM_ERR_UNSUPPORTED for one beyond the call's limits.
 */
typedef struct nm_grad_plan_info {
  int bn;                    /* columns of a tile (256 rows) */
  int grid;                  /* CTA pairs launched */
  int splits_dx, splits_dw;  /* parts of a tile's sum (1: whole, 0: not asked for) */
  int runs_dx, runs_dw;      /* accumulator runs of a part */
  int64_t stages;            /* 64-deep stages of the fullest pair */
  int complete;              /* 1: every stage of every tile is one pair's, every part has its slot */
} nm_grad_plan_info;
nm_status nm_gated_backward_plan_for_shape(int64_t n_ff, int64_t k, int64_t T, int want_dx, int want_dw, int sms,
                                           nm_grad_plan_info* out);

/*
 * Microscaled 4-bit floating point (the MXFP4 format of the OCP Microscaling
 * Formats specification, version 1.0).  (No counterpart in the paper: it is a
 * further storage format for the same linears.)  Along k, every block of 32
 * values shares one scale 2^e, kept as the byte e + 127 (E8M0); a value is a
 * 4-bit code (E2M1): a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0 to 7
 * in that order, the sign in bit 3).  Quantisation:
 *   e    = floor(log2(max |x| of the block)) - 2, at least -127
 *   code = x / 2^e rounded to the nearest of those, a tie to the even code;
 *          above 6 it becomes 6
 * A block of zeros has scale byte 0.  A block that holds an infinity or a NaN
 * has scale byte 255 (which makes every value of the block NaN) and codes 0.
 * All of it is exact arithmetic, so the result does not depend on the GPU.
 *
 * Layout of a quantised matrix [rows][k]:
 *   codes   [rows][k / 2] bytes, two per byte, the lower k in the low nibble;
 *   scales  tiles of 128 rows x 256 k (1024 bytes), row tiles outermost: the
 *           byte of row r and block b (k in [32b, 32b + 32)) is at
 *             ((r / 128) * ceil(k / 256) + b / 8) * 1024 + ((b % 8) / 4) * 512
 *             + (r % 32) * 16 + ((r % 128) / 32) * 4 + b % 4,
 *           which is how the tensor core reads them.  Bytes of rows and blocks
 *           beyond the matrix are 0.  nm_mx_scale_bytes gives the total.
 */
nm_status nm_mx_scale_bytes(int64_t rows, int64_t k, size_t* bytes);

/*
 * nm_mx_quantize -- X [T][k] (row stride ldx elements; NM_FP32, NM_FP16 or
 * NM_BF16) to codes Q_dev [T][k / 2] and scales S_dev (nm_mx_scale_bytes(T, k)
 * bytes, all written).  k > 0 and a multiple of 32, ldx >= k, ldx * sizeof a
 * multiple of 16 bytes, all pointers 16-byte aligned, T >= 0 (0 is a no-op),
 * else NM_ERR_INVALID.  Q and S must not overlap X.
 */
nm_status nm_mx_quantize(const void* X_dev, int64_t T, int64_t k, int64_t ldx, nm_dtype dt, void* Q_dev,
                         void* S_dev, void* stream);

/*
 * nm_mx_dequantize -- the values that codes and scales stand for, into X_dev
 * [T][k] of type dt (NM_FP32 and NM_BF16 hold every one exactly; NM_FP16 rounds
 * to nearest even).  Arguments as nm_mx_quantize with ldx = k.
 */
nm_status nm_mx_dequantize(const void* Q_dev, const void* S_dev, int64_t T, int64_t k, nm_dtype dt, void* X_dev,
                           void* stream);

/*
 * nm_compress_mx -- prune W [n_out][k] (NM_FP32, NM_FP16 or NM_BF16) to N:M by
 * nm_compress's rule (N == M keeps everything), quantise what is kept as above
 * and lay it out for nm_spmm_mx.  (N, M) as nm_compress; k a multiple of 32,
 * at most 2^24 (n_out too); W 16-byte aligned.
 * gated != 0: W is [2 n_ff][k], the n_ff gate rows first (n_out = 2 n_ff, even),
 * and the handle's product is nm_spmm_mx_gated.
 * nm_recompress (W of the same type), nm_decompress (the pruned, quantised
 * values as BF16, which holds them exactly), nm_query (reports NM_MXFP4),
 * nm_device_status and nm_destroy accept the handle; the other calls reject it.
 */
nm_status nm_compress_mx(const void* W_dev, int64_t n_out, int64_t k, nm_dtype dt, int N, int M, int gated,
                         void* stream, nm_handle** out);

/*
 * nm_spmm_mx -- Y = X . Wm^T with X given quantised (codes Q_dev [T][k / 2] and
 * scales S_dev of nm_mx_quantize) and the handle's quantised weight: products
 * of 4-bit values times their blocks' scales, summed in fp32 (by the tensor core,
 * within (k / 32 + 4) 2^-23 sum |x| |w|), then the fused output stage of
 * nm_spmm_ex (scale, bias, NM_ACT_GELU; fp32, fp16 or bf16).
 * NM_OUT_DEFAULT is the type of the handle's source weight; ep == NULL is that
 * with nothing else.  Y_dev [T][n_out], 16-byte aligned, overlapping neither Q
 * nor S; T >= 0 (0 is a no-op).  Allocates nothing, never synchronises, keeps
 * nothing between calls: calls on one handle may overlap.
 */
nm_status nm_spmm_mx(const nm_handle* h, const void* Q_dev, const void* S_dev, int64_t T, void* Y_dev,
                     const nm_epilogue* ep, void* stream);

/*
 * nm_spmm_mx_gated -- the gated block of nm_spmm_gated for a gated handle of
 * nm_compress_mx: Y [T][n_ff] = act(g) * u.  ep as in nm_spmm_gated (scale and
 * bias are [2 n_ff]); fp32, fp16 or bf16 output.  Otherwise as nm_spmm_mx.
 */
nm_status nm_spmm_mx_gated(const nm_handle* h, const void* Q_dev, const void* S_dev, int64_t T, void* Y_dev,
                           const nm_epilogue* ep, void* stream);

/*
 * nm_decompress -- write the masked dense weight Wm [n_out][k] (dtype of the
 * handle) decoded from the packed operand image the SpMM kernel reads, so the
 * image can be checked against the top-N rule.  W_dev_out 16-byte aligned.
 */
nm_status nm_decompress(const nm_handle* h, void* W_dev_out, void* stream);

/*
 * nm_export -- copy the canonical compressed format to the host.  Synchronises
 * the device.
 *   values_host: [n_out][k/M][N] elements of the weight dtype, kept values in
 *                ascending in-group position (nm_export_sizes gives bytes);
 *   idx_host:    [n_out][idx_pitch] bytes, one 4-bit in-group position per
 *                kept element in the same order, two per byte, low nibble
 *                first; idx_pitch = ceil(N * k / M / 2) so rows never share a
 *                byte.  For N == M, positions are 0..M-1.
 */
nm_status nm_export(const nm_handle* h, void* values_host, uint8_t* idx_host);
nm_status nm_export_sizes(const nm_handle* h, size_t* values_bytes, size_t* idx_bytes);

/*
 * nm_plan_query -- the launch plan nm_spmm (scaled != 0: with a scale; the
 * INT8 fp32-output kernels) would use for T tokens on the current device,
 * without launching anything (section 4.1, mechanism 3, adaptive
 * parallelism).  For a handle from nm_compress_tile it is nm_spmm_gather's
 * plan, for one from nm_compress_gated nm_spmm_gated's without P.  Environment
 * overrides (NMSPMM_FORCE_*) apply as they would to the call.  T > 0, else
 * NM_ERR_INVALID.
 */
typedef struct nm_plan_info {
  int pair;     /* 1: two-SM kernel (M = 256 per MMA, grid counts CTA pairs) */
  int bn;       /* token tile (MMA N) */
  int splits;   /* k-splits per output tile (1: none) */
  int cluster;  /* 1: the splits of a tile are one cluster, reduced on chip */
  int grid;     /* CTAs launched (CTA pairs for the two-SM kernel) */
  int units;    /* (tile, split) work units */
} nm_plan_info;
nm_status nm_plan_query(const nm_handle* h, int64_t T, int scaled, nm_plan_info* out);

/*
 * nm_plan_for_shape -- test and diagnostic hook (no counterpart in the paper):
 * the plan nm_plan_query would report for a handle of this shape (nm_compress
 * with dt, n_out, k, N, M) and T tokens on a GPU with `sms` SMs whose
 * resident-cluster capacities are given instead of queried, so the planner's
 * rules can be checked without a GPU.  Touches no device and allocates
 * nothing.
 *
 * pair_clusters    int[3]: CTA pairs of the two-SM kernel that fit on the GPU
 *                  at the token tiles 224, 192 and 128 (<= 0: that tile cannot
 *                  run); nm_plan_query queries these from the device for the
 *                  output the call would write.
 * stream_clusters  int[8]: clusters of S one-SM CTAs that fit, S = 1 .. 8
 *                  (<= 0: none).
 * The NMSPMM_FORCE_* environment overrides apply as in nm_spmm.  Errors:
 * NM_ERR_INVALID for null pointers, a bad dtype, shape, T or sms;
 * NM_ERR_UNSUPPORTED for an N:M nm_compress rejects.
 */
nm_status nm_plan_for_shape(nm_dtype dt, int64_t n_out, int64_t k, int N, int M, int64_t T, int sms,
                            const int* pair_clusters, const int* stream_clusters, nm_plan_info* out);

/* nm_query -- shape and format of a handle; any output pointer may be NULL. */
nm_status nm_query(const nm_handle* h, int64_t* n_out, int64_t* k, int* N, int* M, nm_dtype* dt);

/*
 * nm_device_status -- read (and clear) the handle's device error word, which a
 * kernel sets instead of trapping when a bounded wait runs out.  Synchronises
 * the device.  Returns NM_OK or NM_ERR_TIMEOUT.
 */
nm_status nm_device_status(const nm_handle* h);

/* nm_destroy -- free the handle and its device memory (synchronises). NULL is a no-op. */
void nm_destroy(nm_handle* h);

/* nm_last_error -- message of the calling thread's last failing call ("" if none). */
const char* nm_last_error(void);

/* nm_version -- library version string. */
const char* nm_version(void);

/*
 * Test hook (no counterpart in the paper): run nm_spmm with the SpMM kernel's
 * producer leaving pipeline stage number `skip_stage` (counted over the CTA's
 * whole run) unfilled, and every bounded wait limited to `timeout_ns`
 * (0 < timeout_ns <= 2e9).  The MMA warp's wait on that stage then runs out:
 * the kernel records the timeout in the handle's error word, drains its own
 * copies and MMAs, frees its tensor memory and returns, so the context stays
 * usable.  Exists so tests can exercise the failure path without faulting or
 * hanging a GPU; Y is left partially written.
 */
nm_status nm_test_spmm_skip_stage(const nm_handle* h, const void* X_dev, int64_t T, void* Y_dev,
                                  const float* scale_dev, void* stream, int skip_stage, int64_t timeout_ns);

#ifdef __cplusplus
}
#endif

#endif /* NMSPMM_H */
