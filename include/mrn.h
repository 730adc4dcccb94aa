/*
 * mrn.h -- C ABI of libmrn: RMSNorm, post-norm-then-add and the dual-epsilon
 * sandwich tail on NVIDIA GB300 (sm_103a), hand-written CUDA kernels.
 *
 * Operations (row r of a contiguous row-major [rows x n] matrix, j = 0..n-1):
 *
 *   mrn_rmsnorm             y[r,j]   = x[r,j] * inv(x[r,:]; eps) * gamma[j]
 *   mrn_rmsnorm_then_add    out[r,j] = x[r,j] * inv(x[r,:]; eps) * gamma[j] + residual[r,j]
 *   mrn_norm_residual_norm  out_stream[r,j] = block_out[r,j] * inv(block_out[r,:]; eps_post)
 *                                             * gamma_post[j] + residual[r,j]
 *                           normed[r,j]     = out_stream[r,j] * inv(out_stream[r,:]; eps_pre)
 *                                             * gamma_pre[j]
 *   with inv(v; eps) = 1 / sqrt((1/n) sum_j v_j^2 + eps).
 * Built on the same row reduction (declared further down, same conventions):
 *   mrn_add_rmsnorm, mrn_rmsnorm_then_add_scale, mrn_rmsnorm_q8_1 (Hesper
 *   "RMSNorm Layer" kernels) and the split-norm seam mrn_rmsnorm_seam,
 *   mrn_rmsnorm_unweighted, mrn_seam_scale ("Chapter 12", section 12.7).
 * The sandwich tail with a gate on the block and a scale on the residual:
 *   mrn_norm_gate_residual_norm.
 * For training: mrn_layernorm, mrn_dropout_add, mrn_dropout_add_layernorm and the
 *   gradients mrn_layernorm_backward, mrn_dropout_add_layernorm_backward,
 *   mrn_rmsnorm_backward, mrn_norm_gate_residual_norm_backward; and the global norm
 *   of all gradients, mrn_grad_norm, with clipping, mrn_clip_grad_norm.
 *
 * Sources: "Chapter 12 -- RMSNorm and the dual-epsilon sandwich" section 12.1
 * (definition), 12.2 (two epsilons: 1e-8 for the post norms, 1e-5 for the pre
 * norms), 12.4.3 (the fused tail: hidden += rms_norm(src, eps1) * w1, then
 * output = rms_norm(hidden, eps2) * w2, in one dispatch); the Hesper "RMSNorm
 * Layer" page, rmsNormThenAddKernel / rmsNormThenAddBatchKernel (post norm then
 * residual add, row-major batch) and rmsNormThenAddBatchInPlaceKernel (in-place
 * residual update).
 *
 * Common conventions for the operations
 * -------------------------------------
 * Pointers   All data pointers are CUDA device pointers (or managed memory)
 *            owned by the caller.  The library allocates no memory, keeps no
 *            per-call state and never frees anything.
 * Layout     Row operands are contiguous row-major [rows x n]: element (r, j)
 *            at base + r*n + j.  gamma vectors are [n] and shared by all rows.
 * dtype      MRN_F32: every operand is float.  MRN_BF16: every operand (row
 *            data and gamma) is bfloat16; arithmetic is f32 and each output is
 *            rounded once to bf16 (to nearest, ties to even).  In the bf16
 *            sandwich, normed is computed from the rounded out_stream that is
 *            stored (the split route's publication boundary, section 12.4.4).
 * eps        float, finite and > 0; used as given (the f32 value).
 * Sizes      n >= 1; rows >= 0.  rows == 0 is a no-op that returns MRN_OK
 *            without reading any pointer.  rows * n * element size must fit
 *            in int64.
 * Alignment  Each pointer must be aligned to its element size.  When every
 *            pointer is 16-byte aligned and n * element size is a multiple
 *            of 16, rows are moved in 16-byte vectors.  Otherwise, batches of
 *            the plain, then-add, then-add-scale and sandwich operations whose
 *            row operands and outputs all sit at one offset within 16 bytes
 *            (a row pitch that is not a multiple of 16 bytes on aligned
 *            buffers, or buffers offset alike) are still read as 16-byte
 *            granules: each row's granules are copied whole, including up to
 *            15 bytes before its first and after its last element within the
 *            same granules (never more), and its edge elements are written
 *            one by one.  Everything else moves element-wise.
 * Aliasing   An output may be the very same buffer as a row input (same base
 *            pointer): y == x, out == x or out == residual, out_stream ==
 *            residual (the in-place residual update) or out_stream ==
 *            block_out, normed == block_out or normed == residual.  Any
 *            other overlap -- partial overlaps, two outputs overlapping, an
 *            output overlapping a gamma -- is rejected with MRN_ERR_ALIASING.
 * Stream     Work is enqueued on `stream` (0 = the legacy default stream) and
 *            runs asynchronously; the call returns once it is enqueued.
 * Errors     Argument errors are detected before anything is enqueued; nothing
 *            is written.  MRN_ERR_CUDA means the launch itself failed (see
 *            mrn_last_cuda_error).  Faults during execution surface at the
 *            caller's next synchronisation, as for any CUDA kernel.  Every
 *            wait inside a kernel is bounded (about one second); one that runs
 *            out is counted on the device and reported only by
 *            mrn_wait_timeouts(), never as the status of the call that
 *            enqueued the kernel (that call returned MRN_OK at enqueue time).
 *            The affected rows' outputs are then not written (staged kernels)
 *            or unspecified (cluster reductions of the register kernel).
 * Threads    All entry points are thread-safe.
 */
#ifndef MRN_H
#define MRN_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mrn_dtype {
    MRN_F32 = 0,
    MRN_BF16 = 1,
    MRN_F16 = 2    /* IEEE binary16: only as the publication format of the seam
                      operations below; every other use is MRN_ERR_UNSUPPORTED_DTYPE */
} mrn_dtype;

typedef enum mrn_status {
    MRN_OK = 0,
    MRN_ERR_NULL_POINTER = 1,      /* a required pointer is NULL (rows > 0) */
    MRN_ERR_INVALID_SIZE = 2,      /* n < 1, rows < 0, rows*n*size overflows, a
                                      workspace smaller than the call needs, a number
                                      of tensors or elements < 0, or a factor of no
                                      known kind */
    MRN_ERR_INVALID_EPS = 3,       /* eps not finite or not > 0, a dropout
                                      probability outside 0 .. 1, or a largest norm
                                      that is not >= 0 */
    MRN_ERR_UNSUPPORTED_DTYPE = 4, /* dtype not MRN_F32 / MRN_BF16 (seam format not
                                      MRN_F16 / MRN_BF16) */
    MRN_ERR_ALIASING = 5,          /* a forbidden overlap between buffers */
    MRN_ERR_MISALIGNED = 6,        /* a pointer not aligned to its element size */
    MRN_ERR_CUDA = 7,              /* the CUDA runtime refused the launch */
    MRN_ERR_INVALID_GEOMETRY = 8   /* a forced geometry cannot cover the row */
    /* A kernel whose bounded wait ran out is never reported as a call status
       (the call has returned long before): only mrn_wait_timeouts() reports it. */
} mrn_status;

/*
 * RMSNorm of every row ("Chapter 12", section 12.1; the ferrite-lineage
 * rms_norm_batch of section 12.4.1 computes the same thing):
 *   x      [rows x n]  input rows
 *   gamma  [n]         per-channel gain
 *   y      [rows x n]  output; may be x itself
 */
mrn_status mrn_rmsnorm(const void *x, const void *gamma, void *y,
                       int64_t rows, int64_t n, float eps,
                       mrn_dtype dtype, cudaStream_t stream);

/*
 * Post norm then residual add (Hesper "RMSNorm Layer", rmsNormThenAddKernel and
 * its row-major batch form rmsNormAddBatchRowsKernel):
 *   x         [rows x n]  the block output that is normalised
 *   gamma     [n]
 *   residual  [rows x n]  added after the norm
 *   out       [rows x n]  may be x or residual itself (in-place residual update,
 *                         rmsNormThenAddBatchInPlaceKernel)
 */
mrn_status mrn_rmsnorm_then_add(const void *x, const void *gamma,
                                const void *residual, void *out,
                                int64_t rows, int64_t n, float eps,
                                mrn_dtype dtype, cudaStream_t stream);

/*
 * Dual-epsilon sandwich tail in one kernel ("Chapter 12", section 12.4.3,
 * muser_fused_norm_residual_rms_norm_32sg; roles: src = block_out,
 * hidden = residual / out_stream, weight1 = gamma_post, weight2 = gamma_pre,
 * eps1 = eps_post (1e-8 on the pages' model), eps2 = eps_pre (1e-5)):
 *   block_out   [rows x n]  sub-block output (attention o_proj or FFN down)
 *   residual    [rows x n]  residual stream before the update
 *   gamma_post  [n]         the post norm's gain
 *   gamma_pre   [n]         the next pre norm's gain
 *   out_stream  [rows x n]  updated stream; may be residual (in place) or block_out
 *   normed      [rows x n]  next sub-block's input; may be block_out or residual,
 *                           never overlapping out_stream
 */
mrn_status mrn_norm_residual_norm(const void *block_out, const void *residual,
                                  const void *gamma_post, const void *gamma_pre,
                                  void *out_stream, void *normed,
                                  int64_t rows, int64_t n,
                                  float eps_post, float eps_pre,
                                  mrn_dtype dtype, cudaStream_t stream);

/*
 * Residual add, then RMSNorm of the sum, in one kernel (Hesper "RMSNorm Layer",
 * residualAddRmsNormKernel / forwardResidualAdd; the pre-norm shape: the stream
 * is updated, then normalised for the next sub-block):
 *   residual_out[r,j] = a[r,j] + b[r,j]
 *   normed[r,j]       = residual_out[r,j] * inv(residual_out[r,:]; eps) * gamma[j]
 *   a, b          [rows x n]  the two summands (stream and sub-block output)
 *   gamma         [n]
 *   residual_out  [rows x n]  the sum; may be a or b (in-place accumulate)
 *   normed        [rows x n]  may be a or b, never overlapping residual_out
 * bf16: the sum is rounded once to bf16, stored, and that rounded value is
 * normalised (the same publication boundary as the sandwich's stream).
 */
mrn_status mrn_add_rmsnorm(const void *a, const void *b, const void *gamma,
                           void *residual_out, void *normed,
                           int64_t rows, int64_t n, float eps,
                           mrn_dtype dtype, cudaStream_t stream);

/*
 * Post norm, residual add, then a broadcast scalar (Hesper "RMSNorm Layer",
 * rmsNormThenAddThenBroadcastScaleKernel; a per-layer output scale):
 *   out[r,j] = (x[r,j] * inv(x[r,:]; eps) * gamma[j] + residual[r,j]) * out_scale[0]
 *   out_scale  one element of `dtype` in device memory, read by the kernel
 *   out        [rows x n]  may be x or residual; must not overlap out_scale
 * Arithmetic: fma(x * inv, gamma, residual) in f32, times out_scale, rounded
 * once to the output type.
 */
mrn_status mrn_rmsnorm_then_add_scale(const void *x, const void *gamma, const void *residual,
                                      const void *out_scale, void *out,
                                      int64_t rows, int64_t n, float eps,
                                      mrn_dtype dtype, cudaStream_t stream);

/*
 * RMSNorm fused with Q8_1 block quantisation (Hesper "RMSNorm Layer",
 * fusedRMSNormQ8_1Kernel: the norm's output goes straight to the quantised
 * input of the next matvec, with no f32 round trip through memory):
 *   x_normed[j] = x[r,j] * gamma[j] * inv(x[r,:]; eps)            (f32)
 *   per block of 32 consecutive elements of a row:
 *     d = max |x_normed| / 127,  q = round(x_normed / d)  (nearest, ties to
 *     even; clamped to [-128, 127]; q = 0 and d = 0 for an all-zero block)
 *   x       [rows x n]  f32 or bf16 (dtype); n must be a multiple of 32
 *   gamma   [n]         same dtype
 *   blocks  [rows x n/32] blocks of 36 bytes: f16 d (bytes 0-1), f16 s = 0
 *           (bytes 2-3; unused by the page's consumer), int8 q[32]
 *           (bytes 4-35); 4-byte aligned; must not overlap x or gamma
 * n % 32 != 0 gives MRN_ERR_INVALID_SIZE.
 */
mrn_status mrn_rmsnorm_q8_1(const void *x, const void *gamma, void *blocks,
                            int64_t rows, int64_t n, float eps,
                            mrn_dtype dtype, cudaStream_t stream);

/*
 * Split-norm seam: the rounding point between the weightless norm and the
 * weight multiply kept ("Chapter 12", section 12.7, the cross-vendor seam: a
 * producer that publishes the unweighted norm in F16 and applies its scale as
 * a second F16 operation; a receiver that fuses the two loses that rounding
 * point).  S is the 16-bit publication format `seam` (MRN_F16 or MRN_BF16),
 * S(v) rounds an f32 value to S (nearest, ties to even; overflow gives
 * infinity, gradual underflow).
 *   mrn_rmsnorm_unweighted  u[r,j] = S(x[r,j] * inv(x[r,:]; eps))
 *   mrn_seam_scale          y[r,j] = S(u[r,j] * gamma[j])
 *   mrn_rmsnorm_seam        y[r,j] = S(S(x[r,j] * inv(x[r,:]; eps)) * gamma[j])
 * The weight multiply is the IEEE multiply of S (the exact product of two S
 * values rounded once).  The fused form gives, bit for bit, what the two split
 * operations give on the same rows: the reduction (hence inv) is the same for
 * the fused and the weightless call.
 *   x      [rows x n]  f32 or bf16 (dtype)
 *   gamma  [n]         16-bit values of S
 *   u, y   [rows x n]  16-bit values of S; y may be x itself when dtype is
 *                      MRN_BF16 (same element positions), and mrn_seam_scale's
 *                      y may be u itself; no other overlap is allowed
 * Vector paths need 16-byte aligned pointers and n * element size (of x; of
 * u for mrn_seam_scale) a multiple of 16; otherwise element-wise.
 */
mrn_status mrn_rmsnorm_seam(const void *x, const void *gamma, void *y,
                            int64_t rows, int64_t n, float eps,
                            mrn_dtype dtype, mrn_dtype seam, cudaStream_t stream);
mrn_status mrn_rmsnorm_unweighted(const void *x, void *u, int64_t rows, int64_t n, float eps,
                                  mrn_dtype dtype, mrn_dtype seam, cudaStream_t stream);
mrn_status mrn_seam_scale(const void *u, const void *gamma, void *y, int64_t rows, int64_t n,
                          mrn_dtype seam, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* The dual-epsilon sandwich tail with a gate on the block and a scale on the
 * residual.  Not on the pages, whose blocks have neither.                     */

/* How the values of a factor are shared by the elements of [rows x n]. */
typedef enum mrn_factor {
    MRN_FACTOR_NONE = 0,     /* the factor is one; its pointer is not read */
    MRN_FACTOR_SCALAR = 1,   /* one value */
    MRN_FACTOR_CHANNEL = 2,  /* [n]: one per channel, shared by all rows */
    MRN_FACTOR_ROW = 3       /* [rows]: one per row (the gate only) */
} mrn_factor;

/*
 * The tail in one kernel:
 *   out_stream[r,j] = res_scale * residual[r,j]
 *                     + gate * gamma_post[j] * block_out[r,j] * inv(block_out[r,:]; eps_post)
 *   normed[r,j]     = out_stream[r,j] * inv(out_stream[r,:]; eps_pre) * gamma_pre[j]
 *   block_out   [rows x n]  sub-block output
 *   residual    [rows x n]  residual stream before the update
 *   gamma_post  [n]         the post norm's gain
 *   gamma_pre   [n]         the next pre norm's gain
 *   gate                    the block's gate, gate_kind any mrn_factor
 *   res_scale               the residual's scale; MRN_FACTOR_ROW is MRN_ERR_INVALID_SIZE
 *   out_stream  [rows x n]  may be block_out or residual (in place)
 *   normed      [rows x n]  may be block_out or residual, never overlapping out_stream
 * Factors are device memory of `dtype`, read when the kernel runs, so that a captured
 * graph takes the values of its replay; of a bf16 gate per row the four bytes that hold
 * a value are read.  Factors are multiplied as they are: a gate of zero does not hide an
 * infinity or NaN of the block.  The two factors of a channel (gate and gamma_post) are
 * multiplied first, in f32; bf16: out_stream is rounded once and normed is computed from
 * the rounded values, as in mrn_norm_residual_norm.
 * Speed, alignment and geometry: as of the training operations below (bf16 with a scale per
 * channel: rows of up to 196,608 elements at full speed); weights and factors of rows that
 * are all aligned should be 16-byte aligned too.
 */
mrn_status mrn_norm_gate_residual_norm(const void *block_out, const void *residual,
                                       const void *gamma_post, const void *gamma_pre,
                                       const void *gate, mrn_factor gate_kind,
                                       const void *res_scale, mrn_factor res_scale_kind,
                                       void *out_stream, void *normed,
                                       int64_t rows, int64_t n, float eps_post, float eps_pre,
                                       mrn_dtype dtype, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Training: LayerNorm, dropout before the residual add, and the gradients of
 * LayerNorm and RMSNorm.  Not on the pages, which only run a model.  The
 * conventions above hold (pointers, layout, dtype, alignment, aliasing, stream,
 * errors); rows == 0 is a no-op except where a gradient of weights is due,
 * which is then zero.
 *
 * Speed and alignment: operands whose base pointers share one offset from a multiple
 * of eight elements (16 bytes of bf16, 32 of f32), zero as a rule, are moved in whole
 * slots of eight elements, whatever the row pitch; up to seven elements at either end
 * of a row whose pitch is not a multiple of eight go one by one (bf16: the four bytes
 * that hold the element are read, which may take in one element beside the row, never
 * more).  Operands at different offsets, rows wider than a cluster of CTAs holds (over
 * 131,072 elements; 262,144 in a bf16 forward) and, with a dropout, operands off a multiple
 * of eight go element by element: several times slower, with the same meaning.  Sums are
 * then taken in another order: such a call and one with operands elsewhere agree within
 * roundings, not bit for bit.
 * Launches: one kernel per call, two for a gradient with weights (the rows, then the
 * sum of what the CTAs left of dgamma and dbeta); mrn_force_geometry does not apply.
 * Rows that are split over a cluster wait for each other for about a second at most;
 * if one runs out, mrn_wait_timeouts() counts it, and the call's remaining rows and its
 * gradients of weights are unspecified.
 *
 * Dropout and its generator
 *   Element e = r*n + j of the flattened matrix is kept when u16(e) >= t, with
 *   t = round(p * 2^16), and kept values are multiplied by 2^16 / (2^16 - t) (the
 *   exact inverse of the probability kept; 0 when t = 2^16).  p is a double in
 *   0 .. 1, taken to the nearest multiple of 2^-16.  u16(e) is 16-bit lane e % 8 (low half
 *   of each word first) of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
 *   random numbers: as easy as 1, 2, 3", 2011) with key rng[0] and counter
 *   (e / 8, rng[1] + site), 64 bits each, the lower words e / 8.
 *   rng is device memory, read when the kernel runs: a captured graph draws new
 *   masks at each replay when rng[1] is advanced between replays.  Call sites
 *   that share rng within a step take different `site`s, and rng[1] is advanced
 *   past the largest.  The mask is never stored: a gradient evaluates it again
 *   from the same rng values, site, p and shape.  A dropped value does not reach
 *   the result, whatever it is (infinities and NaN included).  rng may be NULL
 *   when t = 0.
 */

/*
 * LayerNorm of every row:
 *   mean = sum_j x[r,j] / n,  rstd = 1 / sqrt(sum_j (x[r,j] - mean)^2 / n + eps)
 *   y[r,j] = (x[r,j] - mean) * rstd * gamma[j] + beta[j]
 *   x           [rows x n]
 *   gamma       [n]
 *   beta        [n]         or NULL (no bias)
 *   y           [rows x n]  may be x itself
 *   mean, rstd  [rows]      f32, the row statistics kept for the gradient; both or
 *                           neither NULL
 * The variance is summed from the deviations in f32, not from the squares.
 */
mrn_status mrn_layernorm(const void *x, const void *gamma, const void *beta, void *y,
                         float *mean, float *rstd, int64_t rows, int64_t n, float eps,
                         mrn_dtype dtype, cudaStream_t stream);

/*
 * Dropout, then the residual add, in one kernel:
 *   out[r,j] = residual[r,j] + dropout(x)[r,j]        (one rounding)
 *   residual  [rows x n]  or NULL: out = dropout(x), which is also the gradient's
 *                         own form (dx = dropout(dout))
 *   out       [rows x n]  may be x or residual
 */
mrn_status mrn_dropout_add(const void *x, const void *residual, void *out,
                           const uint64_t *rng, uint64_t site, double p,
                           int64_t rows, int64_t n, mrn_dtype dtype, cudaStream_t stream);

/*
 * The tail of a training sub-block in one kernel: dropout, residual add, and the
 * LayerNorm of the new stream:
 *   out_stream = residual + dropout(x), rounded once to dtype and stored
 *   normed     = layernorm(out_stream as stored)
 *   out_stream  [rows x n]  may be x or residual
 *   normed      [rows x n]  may be x or residual, never overlapping out_stream
 *   beta, mean, rstd as in mrn_layernorm.  p = 0 is the residual add and LayerNorm.
 */
mrn_status mrn_dropout_add_layernorm(const void *x, const void *residual, const void *gamma,
                                     const void *beta, void *out_stream, void *normed,
                                     float *mean, float *rstd, const uint64_t *rng,
                                     uint64_t site, double p, int64_t rows, int64_t n, float eps,
                                     mrn_dtype dtype, cudaStream_t stream);

/*
 * Bytes of the workspace of a gradient of rows x n (either norm, either dtype) on
 * the current device.  The workspace is scratch: 16-byte aligned device memory that
 * holds nothing between calls, used by the call's kernels until they have run.  Calls
 * that may run at the same time (two streams, two graphs replayed together) need a
 * workspace each.
 */
mrn_status mrn_norm_backward_workspace(int64_t rows, int64_t n, int64_t *bytes);

/*
 * Gradient of mrn_layernorm.  With xh = (x - mean) * rstd and w = dy * gamma:
 *   dx[r,j]   = rstd * (w - sum_j w / n - xh * sum_j (w * xh) / n) + dstream[r,j]
 *   dgamma[j] = sum_r dy * xh,   dbeta[j] = sum_r dy
 *   dy          [rows x n]  gradient of y
 *   x           [rows x n]  the forward's input;  mean, rstd [rows] f32, its statistics
 *   dstream     [rows x n]  or NULL: the gradient that reaches x beside the norm (the
 *                           residual stream's), added to dx
 *   dx          [rows x n]  may be dy, x or dstream
 *   dgamma      [n]         f32 whatever the dtype (a sum over all rows)
 *   dbeta       [n]         f32, or NULL
 * The sums over rows are taken in a fixed order: the same call gives the same bits.
 * rows == 0 writes zeros to dgamma and dbeta; the other pointers are not read.
 */
mrn_status mrn_layernorm_backward(const void *dy, const void *x, const void *gamma,
                                  const float *mean, const float *rstd, const void *dstream,
                                  void *dx, float *dgamma, float *dbeta,
                                  void *workspace, int64_t workspace_bytes,
                                  int64_t rows, int64_t n, mrn_dtype dtype, cudaStream_t stream);

/*
 * Gradient of mrn_dropout_add_layernorm, with the forward's out_stream, mean, rstd,
 * rng values, site and p:
 *   ds        = layernorm gradient of dnormed at out_stream, + dstream
 *   dresidual = ds                       (rounded once)
 *   dx        = dropout(ds)              (from the f32 ds, rounded once)
 *   dx, dresidual  [rows x n]  each may be dnormed, out_stream or dstream, not each other
 */
mrn_status mrn_dropout_add_layernorm_backward(
    const void *dnormed, const void *out_stream, const void *gamma, const float *mean,
    const float *rstd, const void *dstream, void *dx, void *dresidual, float *dgamma,
    float *dbeta, const uint64_t *rng, uint64_t site, double p, void *workspace,
    int64_t workspace_bytes, int64_t rows, int64_t n, mrn_dtype dtype, cudaStream_t stream);

/*
 * Gradient of mrn_rmsnorm (and, with dstream, of mrn_add_rmsnorm: both summands get
 * dx; of mrn_norm_residual_norm: once at out_stream with gamma_pre and dstream, then
 * once at block_out with gamma_post).  inv is recomputed from x, so no statistics are
 * kept.  With w = dy * gamma:
 *   dx[r,j]   = inv * (w - x * inv^2 * sum_j (w * x) / n) + dstream[r,j]
 *   dgamma[j] = sum_r dy * x * inv
 * Operands as in mrn_layernorm_backward.
 */
mrn_status mrn_rmsnorm_backward(const void *dy, const void *x, const void *gamma,
                                const void *dstream, void *dx, float *dgamma,
                                void *workspace, int64_t workspace_bytes,
                                int64_t rows, int64_t n, float eps,
                                mrn_dtype dtype, cudaStream_t stream);

/*
 * Bytes of the workspace of mrn_norm_gate_residual_norm_backward for rows x n (either
 * dtype, any factors) on the current device; as mrn_norm_backward_workspace otherwise.
 */
mrn_status mrn_norm_gate_backward_workspace(int64_t rows, int64_t n, int64_t *bytes);

/*
 * Gradient of mrn_norm_gate_residual_norm (with no factors: of mrn_norm_residual_norm),
 * from its operands and its out_stream; no statistics are kept, both inv are taken again.
 * With i = inv(out_stream; eps_pre), w = dnormed * gamma_pre, xh = block_out *
 * inv(block_out; eps_post):
 *   ds          = i * (w - out_stream * i^2 * sum_j (w * out_stream) / n) + dstream
 *   u           = ds * gate * gamma_post
 *   dblock      = inv(block_out; eps_post) * (u - xh * sum_j (u * xh) / n)
 *   dresidual   = res_scale * ds
 *   dgamma_pre  = sum_r dnormed * out_stream * i,   dgamma_post = sum_r ds * gate * xh
 *   dgate       = ds * gamma_post * xh  summed over the elements that share a gate
 *   dres_scale  = ds * residual         summed over the elements that share a scale
 * dblock and dresidual come from the f32 ds, each rounded once.
 * Range: a row has six sums of products of its operands as they are, before inv scales
 * them: out_stream^2, block_out^2 and, with cb = block_out * gamma_post (times a gate per
 * channel), w * out_stream, w * cb, out_stream * cb and dstream * cb.  Where the magnitudes
 * of one add up past f32's largest number, the row's gradients and those of the weights are
 * unspecified (most often infinite or NaN), and products under f32's normal range (1e-38)
 * lose bits: in both cases also where each gradient is an ordinary number.
 *   dnormed     [rows x n]  gradient of normed
 *   dstream     [rows x n]  or NULL: the gradient that reaches out_stream beside the norm
 *   residual    [rows x n]  the forward's; read only when dres_scale is asked for (else
 *                           it may be NULL), and then not a stream updated in place
 *   dblock, dresidual  [rows x n]  each may be one of the row inputs, not each other
 *   dgamma_post, dgamma_pre  [n]  f32
 *   dgate, dres_scale  f32, as many values as the factor has; NULL: not computed.  With
 *                           MRN_FACTOR_NONE they must be NULL (else
 *                           MRN_ERR_NULL_POINTER: the factor is missing).
 * The same call gives the same bits.  rows == 0 writes zeros to the gradients of weights
 * and of factors; the other pointers are not read.
 */
mrn_status mrn_norm_gate_residual_norm_backward(
    const void *dnormed, const void *dstream, const void *block_out, const void *out_stream,
    const void *residual, const void *gamma_post, const void *gamma_pre, const void *gate,
    mrn_factor gate_kind, const void *res_scale, mrn_factor res_scale_kind, void *dblock,
    void *dresidual, float *dgamma_post, float *dgamma_pre, float *dgate, float *dres_scale,
    void *workspace, int64_t workspace_bytes, int64_t rows, int64_t n, float eps_post,
    float eps_pre, mrn_dtype dtype, cudaStream_t stream);

/*
 * Bytes of the workspace of mrn_grad_norm and mrn_clip_grad_norm for lists of up to
 * `tensors` tensors on the current device: scratch, 8-byte aligned device memory, a
 * workspace each for calls that may run at the same time.
 */
mrn_status mrn_grad_norm_workspace(int64_t tensors, int64_t *bytes);

/*
 * The norm of all elements of a list of tensors:  norm = sqrt(sum_t sum_e grads[t][e]^2)
 *   grads, counts, dtypes  host arrays of `tensors` entries, read by the call itself (a
 *           captured graph keeps the entries, not the arrays): the address of a tensor in
 *           device memory, its number of elements (0: the address is not read) and its
 *           type, MRN_F32 or MRN_BF16, mixed as they come
 *   norm    one f32 in device memory; 0 for an empty list
 * Sums over blocks of elements in f32, over the blocks in 64 bits, in a fixed order: the
 * same call gives the same bits.  Squares that leave f32's range are taken in 64 bits, so
 * that norm is right wherever it is an f32 number itself; infinities give infinity, NaN gives
 * NaN.  A tensor that is listed twice counts twice.
 * Launches: one kernel per 960 tensors, and one.
 */
mrn_status mrn_grad_norm(const void *const *grads, const int64_t *counts, const mrn_dtype *dtypes,
                         int64_t tensors, float *norm, void *workspace, int64_t workspace_bytes,
                         cudaStream_t stream);

/*
 * The norm as above, and the tensors scaled to a norm of max_norm at most:
 *   out[t][e] = grads[t][e] * (norm > max_norm ? max_norm / norm : 1)
 * (the factor rounded once to f32, each product once to the tensor's type).  A norm that is
 * not finite leaves the values as they are: the caller reads it and skips the step.
 *   out       host array of addresses; out[t] may be grads[t] itself (in place; nothing is
 *             written when the factor is one), and must not overlap any other entry of
 *             grads or out, norm or the workspace
 *   max_norm  >= 0; infinity: nothing is scaled
 * Tensors whose two addresses share an offset from a multiple of 32 bytes (16 of bf16) are
 * moved in whole vectors, others element by element.
 * Launches: two kernels per 960 tensors (for an empty list, one kernel).
 */
mrn_status mrn_clip_grad_norm(const void *const *grads, void *const *out, const int64_t *counts,
                              const mrn_dtype *dtypes, int64_t tensors, double max_norm,
                              float *norm, void *workspace, int64_t workspace_bytes,
                              cudaStream_t stream);

/* Static, human-readable name of a status code; never NULL. */
const char *mrn_status_string(mrn_status status);

/* cudaError_t of the most recent MRN_ERR_CUDA returned on the calling thread
 * (0 if none). */
int mrn_last_cuda_error(void);

/* ------------------------------------------------------------------------ */
/* Introspection and test hooks.  These are not on the pages: they expose the
 * kernel geometry the library picks so that tests can drive every variant
 * and benchmarks can report it.                                              */

typedef enum mrn_op {
    MRN_OP_RMSNORM = 0,
    MRN_OP_THEN_ADD = 1,
    MRN_OP_SANDWICH = 2,
    MRN_OP_ADD_RMSNORM = 3,
    MRN_OP_THEN_ADD_SCALE = 4,
    MRN_OP_RMSNORM_Q8_1 = 5,
    MRN_OP_RMSNORM_SEAM = 6,       /* mrn_rmsnorm_seam (either format) */
    MRN_OP_RMSNORM_UNWEIGHTED = 7  /* mrn_rmsnorm_unweighted (either format) */
} mrn_op;

typedef enum mrn_geometry_kind {
    MRN_GEOM_AUTO = 0,          /* (for mrn_force_geometry) let the library choose */
    MRN_GEOM_ROWS_PER_WARP = 1, /* lanes_per_row (1..32) lanes per row, several rows
                                   per CTA of `threads` (a multiple of 32 up to 256;
                                   0 when forced: 256), shuffle-only reduction */
    MRN_GEOM_CTA = 2,           /* one row per CTA, or per thread-block cluster of
                                   `cluster` CTAs whose partial sums travel as
                                   st.async messages to the peers' shared memory;
                                   row held in registers */
    MRN_GEOM_STREAM = 3,        /* one row per CTA, or per cluster of `cluster` CTAs
                                   each looping over its slice of the row: any n */
    MRN_GEOM_TMA = 4,           /* persistent CTAs; `stages` future rows are copied
                                   into shared memory by cp.async.bulk while the
                                   current one is reduced; gammas kept in shared
                                   memory; needs 16-byte aligned rows.  cluster > 1
                                   (groups 1; plain, then-add, then-add-scale and
                                   the sandwich): a cluster per row, each CTA
                                   staging a 16-byte-multiple slice, the partial
                                   sums exchanged as st.async messages */
    MRN_GEOM_Q8_BLOCKS = 5      /* RMSNorm + Q8_1 only: one row per CTA, `k` (1 or 2)
                                   whole 32-element blocks per thread, `threads` <= 512;
                                   needs 16-byte aligned rows */
} mrn_geometry_kind;

typedef struct mrn_geometry {
    int32_t kind;          /* mrn_geometry_kind */
    int32_t vec;           /* elements per load: 16 / element size, or 1 */
    int32_t k;             /* loads per operand per thread (register slots) */
    int32_t threads;       /* threads per CTA */
    int32_t cluster;       /* CTAs per row, 1..16 (MRN_GEOM_CTA, MRN_GEOM_TMA or
                              MRN_GEOM_STREAM) */
    int32_t lanes_per_row; /* threads per row for MRN_GEOM_ROWS_PER_WARP */
    int32_t rows_per_cta;  /* rows one CTA handles at a time */
    int32_t stages;        /* MRN_GEOM_TMA: rows staged in shared memory (1..8) */
    int32_t ctas;          /* MRN_GEOM_TMA: persistent CTAs (0 = fill the device) */
    int32_t groups;        /* MRN_GEOM_TMA: warp groups per CTA (1 or 2), each
                              reducing its own rows; threads is the CTA total */
    int32_t edge;          /* MRN_GEOM_TMA, cluster 1, groups 2: rows that are not
                              16-byte aligned (plain, then-add, then-add-scale,
                              sandwich; every row operand and output at one offset
                              within 16 bytes), each staged as the 16-byte granules
                              that cover it, the edge elements masked and stored one
                              by one; k * threads / 2 must cover
                              (n * size + 15) / 16 + 1 granules */
} mrn_geometry;

/*
 * The geometry an operation would launch with.  aligned16: 1 states that all
 * pointers would be 16-byte aligned; 2 that they would not, but that every
 * row operand and output would sit at one offset within 16 bytes; 0 neither.
 * sm_count 0 means: ask the current device; a positive value is used as
 * given (lets host-only tests query).  The thread's forced geometry, if any,
 * is reported instead.
 */
mrn_status mrn_query_geometry(mrn_op op, int64_t rows, int64_t n, mrn_dtype dtype,
                              int32_t aligned16, int32_t sm_count, mrn_geometry *out);

/*
 * Force the geometry of the calling thread's later calls (NULL or kind
 * MRN_GEOM_AUTO restores the automatic choice).  Fields 0 mean "automatic"
 * for vec.  A forced geometry that cannot cover a call's row makes that call
 * return MRN_ERR_INVALID_GEOMETRY.  The geometry is checked for internal
 * consistency here (MRN_ERR_INVALID_GEOMETRY if not).
 */
mrn_status mrn_force_geometry(const mrn_geometry *geometry);

/* Number of kernels this library has launched in the process (all threads). */
uint64_t mrn_launch_count(void);

/*
 * Launch options of the calling thread's later calls (default MRN_LAUNCH_PDL;
 * 0 = plain stream-ordered launches).
 *   MRN_LAUNCH_PDL  programmatic dependent launch: a kernel may be scheduled
 *                   before the previous kernel on the stream has finished.
 *                   Every kernel of this library first waits for that
 *                   previous grid to complete and publish its memory
 *                   (griddepcontrol.wait), so results are unchanged; the
 *                   launch latency of a call overlaps the previous kernel
 *                   instead of following it (measured on GB300: ~2 us per
 *                   call in a chain of 4096 x 6656 sandwich calls, ~0.2 us
 *                   per decode call in a CUDA graph).  The previous kernel
 *                   need not be ours; a kernel launched after ours without
 *                   the attribute is ordered as usual.
 *   MRN_LAUNCH_TEST_WAIT_TIMEOUT
 *                   test hook, never for use: the first wait of every CTA
 *                   of the staged kernels (MRN_GEOM_TMA, staged
 *                   MRN_GEOM_Q8_BLOCKS: its gamma copy) and of cluster
 *                   reductions in MRN_GEOM_CTA and the training operations (its
 *                   first message exchange) expects 16 bytes more than ever arrive, so it runs out
 *                   after about one second.  The staged kernels then write
 *                   nothing; the register kernel's outputs and the training
 *                   operations' are unspecified.
 *                   mrn_wait_timeouts() reports the waits; the context stays
 *                   usable.  Lets a test drive the timeout path with no fault.
 * Unknown bits give MRN_ERR_INVALID_GEOMETRY.  Not on the pages: a launch
 * option of this library.
 */
#define MRN_LAUNCH_PDL 1u
#define MRN_LAUNCH_TEST_WAIT_TIMEOUT 0x80000000u
mrn_status mrn_set_launch_options(uint32_t options);
uint32_t mrn_launch_options(void);

/*
 * Number of bounded waits (on the shared-memory copy barriers of the staged
 * kernels and the message barriers of cluster reductions) that ran out on the
 * current device since the previous mrn_wait_timeouts() call on that device;
 * -1 if the count could not be read.  This is the only place a timeout is
 * reported: no entry point returns a status for it.  The device-side counts
 * only grow; the library keeps the last value it reported per device (under
 * a lock), so a timeout counted while this function runs is reported by the
 * next call, never lost.  Every wait gives up after about one second of wall
 * time (%globaltimer, which also runs while the context is time-sliced out on
 * a shared GPU); a staged CTA then drains its copies and returns without
 * writing its remaining rows, so the context stays usable.
 * Synchronises the device (it reads device memory with cudaMemcpyFromSymbol).
 * Not on the pages: a diagnostic of this library.
 */
int mrn_wait_timeouts(void);

#ifdef __cplusplus
}
#endif

#endif /* MRN_H */
