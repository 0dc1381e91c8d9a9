/*
 * cbr.h -- C ABI of libcbr.so: the training-mode Conv2d -> BatchNorm -> ReLU (CBR) operator
 * on NVIDIA GB300 (sm_103a), forward, backward and folded inference.
 *
 * What is computed (all citations are to the source pages, by title and section):
 *   z      = conv(x, W)          cross-correlation, no bias, dilation 1
 *                                ("CBR fused operator" (Tech-Renaissance), section 4.1;
 *                                 "TileLang Conv2D+ReLU fusion", basic convolution section)
 *   mean, var over the M = N*P*Q rows of each output channel (biased var for normalising)
 *   inv_std = 1/sqrt(var + eps)
 *   y      = max(0, gamma*(z - mean)*inv_std + beta)        (CBR page, sections 4.2-4.3)
 *   mask   = (gamma*(z - mean)*inv_std + beta > 0), one bit per element (section 4.3, CMP_GT)
 *   running_mean <- (1-momentum)*running_mean + momentum*mean
 *   running_var  <- (1-momentum)*running_var  + momentum*var*M/(M-1)   (unbiased)
 *                                (CBR page section 4.2; "BatchNorm CUDA implementation",
 *                                 section 2.4)
 *   backward: g = dy*mask; dbeta = sum g; dgamma = sum g*xhat;
 *             dz = gamma*inv_std*(g - dbeta/M - xhat*dgamma/M);  dW = wgrad(dz, x);
 *             dx = dgrad(dz, W)   (CBR page sections 5.1-5.3; BatchNorm page section 3.1)
 *   inference: W_fold = W*gamma/sqrt(rv+eps), b_fold = (b - rm)*gamma/sqrt(rv+eps) + beta,
 *             y = relu(conv(x, W_fold) + b_fold)   (CBR page sections 2 and 6;
 *                                                    BatchNorm page section 4.4)
 *
 * Layouts (CBR page, section 8): activations NHWC, filters KRSC ([Cout][R][S][Cin]), both in
 * the storage dtype (fp16 or bf16).  gamma, beta, statistics and dW are fp32.  Output size
 * P = (H + 2*pad - R)/stride + 1, Q likewise.
 *
 * Conventions for every call:
 *   - The caller owns every buffer; pointers are device pointers unless stated otherwise.
 *     The library allocates no device memory on any call.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream).
 *     A returned CBR_OK means the work was validated and enqueued.  Device-side failures
 *     (a bounded wait that ran out) are reported by cbr_stream_status().
 *   - Arguments are validated on the host before anything is enqueued; on any error nothing
 *     is launched and no output is touched.
 *   - Activation / filter / workspace pointers must be 16-byte aligned, fp32 vectors 4-byte.
 *   - No call throws; the library holds no per-call state.
 *   - Supported shapes (else CBR_ERR_UNSUPPORTED): Cout in {16, 32, 64, 128}; and either
 *     stride 1 with Cin a multiple of 8, Cin <= 128, W + 2*pad <= 256; or the first-layer
 *     form Cin = 3 (any stride, R <= 8, S <= 8, pad <= 10, Q <= 128).  Cout % 8 != 0 is
 *     CBR_ERR_INVALID_ARG
 *     (CBR page, section 8: output channels must be a multiple of 8).
 */
#ifndef CBR_H_
#define CBR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* cbr_stream_t; /* identical to cudaStream_t */

typedef enum {
  CBR_OK = 0,
  CBR_ERR_INVALID_ARG = 1, /* null pointer, bad shape, bad scalar, dx aliases x, M < 2 */
  CBR_ERR_MISALIGNED = 2,  /* pointer alignment rule violated */
  CBR_ERR_UNSUPPORTED = 3, /* valid arguments outside the shapes/dtypes this library runs */
  CBR_ERR_WORKSPACE = 4,   /* ws_bytes smaller than cbr_workspace_size() requires */
  CBR_ERR_DEVICE = 5,      /* no CUDA device, or the current device is not compute 10.3 */
  CBR_ERR_CUDA = 6,        /* a CUDA runtime / driver call failed */
  CBR_ERR_TIMEOUT = 7      /* (cbr_stream_status) a kernel gave up on a bounded wait */
} cbr_status_t;

/* CBR_F32 is taken by the token operators only. */
typedef enum { CBR_F16 = 0, CBR_BF16 = 1, CBR_F32 = 2 } cbr_dtype_t;

/* Source of the ReLU mask for cbr_backward. */
typedef enum {
  CBR_MASK_BITS = 0,   /* bit-packed mask written by cbr_forward_train */
  CBR_MASK_FROM_Y = 1, /* recompute the mask as y > 0 from the forward output y */
  CBR_MASK_BYTES = 2   /* one byte per NHWC element, non-zero = active (a standalone ReLU's
                          INT8 mask); packed into the workspace before use */
} cbr_mask_kind_t;

/* One CBR layer.  dtype is a cbr_dtype_t. */
typedef struct {
  int32_t n, h, w, c_in, c_out, r, s, stride, pad;
  int32_t dtype;
} cbr_desc_t;

/* Version of this ABI (major*100 + minor). */
int32_t cbr_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* cbr_status_string(cbr_status_t status);

/*
 * Workspace bytes needed by cbr_forward_train (fwd_bytes) and cbr_backward (bwd_bytes) for
 * `desc`, assuming the caller passes z_saved = NULL (the largest case; with z_saved the calls
 * need less, and check the actual need).  Pure host computation; either output may be NULL.
 * The first 256 bytes of a workspace hold arrival counters: they must be zero the first
 * time a workspace is used (e.g. allocate it zero-filled); every call leaves them at zero.
 */
cbr_status_t cbr_workspace_size(const cbr_desc_t* desc, size_t* fwd_bytes, size_t* bwd_bytes);

/*
 * Training forward (CBR page, sections 4.1-4.3).
 *   x [n][h][w][c_in], w [c_out][r][s][c_in]          storage dtype, read only
 *   gamma, beta [c_out]                                fp32, read only
 *   running_mean, running_var [c_out]                  fp32, updated in place
 *   momentum in [0,1] (weight of the new batch), eps > 0
 *   y [n][p][q][c_out]                                 storage dtype, written
 *   relu_mask: ceil(n*p*q*c_out/32) uint32 words or NULL; bit i of word j is the mask of
 *              NHWC element 32*j + i (bits past the last element are unspecified)
 *   z_saved [n][p][q][c_out] or NULL: receives the conv output; pass it to cbr_backward to
 *              avoid recomputing the convolution there
 *   saved_mean, saved_inv_var [c_out]                  fp32 batch mean and 1/sqrt(var+eps)
 *   ws, ws_bytes                                       workspace (see cbr_workspace_size)
 * Errors: INVALID_ARG (null required pointer, bad desc, momentum/eps out of range,
 * n*p*q < 2), MISALIGNED, UNSUPPORTED, WORKSPACE, DEVICE, CUDA.
 */
cbr_status_t cbr_forward_train(const cbr_desc_t* desc, const void* x, const void* w,
                               const float* gamma, const float* beta, float* running_mean,
                               float* running_var, float momentum, float eps, void* y,
                               uint32_t* relu_mask, void* z_saved, float* saved_mean,
                               float* saved_inv_var, void* ws, size_t ws_bytes,
                               cbr_stream_t stream);

/*
 * The same training forward in one persistent, cooperative kernel launch: the convolution, the
 * statistics, the finalize by the last CTA, then (every CTA waiting, with a time limit, for the
 * finalize) BatchNorm and ReLU applied to the accumulators still held in tensor memory.  z is
 * never re-read (the single-read fusion of the BatchNorm CUDA page, section 4.1).  Arguments,
 * outputs and errors as cbr_forward_train, whose results it reproduces bit for bit (y is
 * computed from the accumulator rounded to the storage dtype, as z is stored).  It takes stride-1
 * convolutions of at most 64 input channels, 32 or 64 output channels, a filter that fits in
 * shared memory, y 32-byte aligned, and batches of at most 4 units of 256 output rows per SM
 * (for example 46 images of 56x56); otherwise it returns CBR_ERR_UNSUPPORTED and does nothing.
 * It is not faster than cbr_forward_train on the measured shapes (the finalize and the apply
 * phase then run one after the other inside one launch); it is there for callers who want one
 * launch per forward.  The runtime refuses the launch (CBR_ERR_CUDA) if the whole grid cannot be
 * resident at once.
 */
cbr_status_t cbr_forward_train_persistent(const cbr_desc_t* desc, const void* x, const void* w,
                                          const float* gamma, const float* beta, float* running_mean,
                                          float* running_var, float momentum, float eps, void* y,
                                          uint32_t* relu_mask, void* z_saved, float* saved_mean,
                                          float* saved_inv_var, void* ws, size_t ws_bytes,
                                          cbr_stream_t stream);

/*
 * Training backward (CBR page, sections 5.1-5.3; BatchNorm page, section 3.1).
 *   dy [n][p][q][c_out]            upstream gradient, storage dtype
 *   x, w                           the forward's inputs
 *   y_or_relu_mask, mask_kind      the forward's relu_mask words (CBR_MASK_BITS, 4-byte
 *                                  aligned), its y (CBR_MASK_FROM_Y) or a byte-per-element
 *                                  mask (CBR_MASK_BYTES, n*p*q*c_out bytes, 16-byte aligned)
 *   z_saved                        the forward's z_saved, or NULL to recompute conv(x, W)
 *   gamma, saved_mean, saved_inv_var   fp32 [c_out] (saved_* from cbr_forward_train)
 *   dx [n][h][w][c_in] or NULL     NULL = first layer: the data gradient is skipped
 *                                  (CBR page, section 5.3).  dx must not overlap x
 *                                  (section 5.2's write-after-read hazard): INVALID_ARG.
 *   dw [c_out][r][s][c_in]         fp32, written
 *   dgamma, dbeta [c_out]          fp32, written
 *   ws, ws_bytes                   workspace (see cbr_workspace_size); it also holds dz, which
 *                                  is evaluated once and read by both convolutions
 * Errors: INVALID_ARG (null required pointer, bad desc or mask_kind, dx overlapping x),
 * MISALIGNED, UNSUPPORTED (also: dx requested with a non-square filter or pad > R-1, or for
 * the 3-channel first layer), WORKSPACE, DEVICE, CUDA.
 */
cbr_status_t cbr_backward(const cbr_desc_t* desc, const void* dy, const void* x, const void* w,
                          const void* y_or_relu_mask, int32_t mask_kind, const void* z_saved,
                          const float* gamma, const float* saved_mean,
                          const float* saved_inv_var, void* dx, float* dw, float* dgamma,
                          float* dbeta, void* ws, size_t ws_bytes, cbr_stream_t stream);

/*
 * Synchronised BatchNorm across data-parallel ranks ("BatchNorm CUDA implementation",
 * section 7.1: the per-channel statistics of every rank's share of the batch are combined
 * before normalising, and so are the backward's per-channel sums).  Each call pair brackets
 * one collective that the caller runs (e.g. with NCCL); the library itself stays on one GPU.
 *
 * Forward, first half: conv and this rank's statistics, no finalize and no apply.
 *   z [n][p][q][c_out]     the conv output (required: the second half normalises it)
 *   moments [2*c_out + 1]  fp32 out: per-channel mean [c_out], M2 (sum of squared deviations
 *                          from the mean) [c_out], then this rank's row count n*p*q
 *   ws, ws_bytes           the forward workspace (cbr_workspace_size's fwd_bytes suffices)
 * The caller gathers every rank's moments, in rank order, into moments_all
 * [world][2*c_out + 1] (an all-gather, not a sum: moments merge exactly, sums of squares
 * would cancel), then calls
 * Forward, second half: merges the `world` moment sets in that order (Chan's parallel
 * formula), writes saved_mean / saved_inv_var, updates the running statistics with the
 * global unbiased variance (M = the sum of the counts), and applies BN + ReLU to this rank's z,
 * as cbr_forward_train does.  Every rank computes identical statistics.
 * Errors: INVALID_ARG (NULL, world < 1, momentum / eps out of range), MISALIGNED,
 * UNSUPPORTED, WORKSPACE, DEVICE, CUDA.
 */
cbr_status_t cbr_forward_train_stats(const cbr_desc_t* desc, const void* x, const void* w, void* z,
                                     float* moments, void* ws, size_t ws_bytes, cbr_stream_t stream);
cbr_status_t cbr_forward_train_finish(const cbr_desc_t* desc, const float* moments_all, int32_t world,
                                      const float* gamma, const float* beta, float* running_mean,
                                      float* running_var, float momentum, float eps, const void* z,
                                      void* y, uint32_t* relu_mask, float* saved_mean,
                                      float* saved_inv_var, void* ws, size_t ws_bytes,
                                      cbr_stream_t stream);

/*
 * Backward, first half: this rank's masked per-channel sums, written to sums [2*c_out] as
 * [sum of dy*mask][sum of dy*mask*(z - saved_mean)] (saved_mean: the merged mean from
 * cbr_forward_train_finish; z and the mask as for cbr_backward; ws: the backward workspace).
 * The caller sums them over the ranks (an all-reduce) into sums_all and calls
 * Backward, second half: dgamma, dbeta and the BN data gradient from the global sums over
 * m_total = the global n*p*q, then wgrad and dgrad of this rank's share, as cbr_backward does.
 * dgamma and dbeta are the global ones (identical on every rank); dW is this rank's share (the
 * caller's data-parallel gradient all-reduce sums it).
 * Errors as for cbr_backward, and INVALID_ARG for a NULL sums / sums_all or m_total < 2.
 */
cbr_status_t cbr_backward_sums(const cbr_desc_t* desc, const void* dy, const void* y_or_relu_mask,
                               int32_t mask_kind, const void* z_saved, const float* saved_mean,
                               float* sums, void* ws, size_t ws_bytes, cbr_stream_t stream);
cbr_status_t cbr_backward_finish(const cbr_desc_t* desc, const float* sums_all, int64_t m_total,
                                 const void* dy, const void* x, const void* w,
                                 const void* y_or_relu_mask, int32_t mask_kind, const void* z_saved,
                                 const float* gamma, const float* saved_mean,
                                 const float* saved_inv_var, void* dx, float* dw, float* dgamma,
                                 float* dbeta, void* ws, size_t ws_bytes, cbr_stream_t stream);

/*
 * BN folding for inference (CBR page, section 2; BatchNorm page, section 4.4):
 *   w_fold[k,...] = w[k,...]*gamma[k]/sqrt(running_var[k]+eps)   (computed in fp32, stored
 *                   rounded to the storage dtype, same layout as w)
 *   b_fold[k]     = (conv_bias[k] - running_mean[k])*gamma[k]/sqrt(running_var[k]+eps)
 *                   + beta[k]                                    (fp32; conv_bias may be NULL)
 */
cbr_status_t cbr_fold_bn(const cbr_desc_t* desc, const void* w, const float* conv_bias,
                         const float* gamma, const float* beta, const float* running_mean,
                         const float* running_var, float eps, void* w_fold, float* b_fold,
                         cbr_stream_t stream);

/*
 * Folded inference forward (CBR page, section 6): y = relu(conv(x, w_fold) + b_fold), with
 * the bias and ReLU applied to the fp32 accumulator before rounding.
 */
cbr_status_t cbr_forward_infer(const cbr_desc_t* desc, const void* x, const void* w_fold,
                               const float* b_fold, void* y, cbr_stream_t stream);

/*
 * Inference with BatchNorm applied to the convolution's fp32 accumulator, the CBR page's
 * single-graph form (section 6: conv, MUL by eq_scale, ADD eq_bias, ReLU):
 *   y = relu(conv(x, w)*scale + shift),  scale = gamma/sqrt(running_var + eps),
 *   shift = beta + (conv_bias - running_mean)*scale          (conv_bias may be NULL: 0)
 * Unlike cbr_fold_bn + cbr_forward_infer, the filter is used as trained, so nothing is rounded
 * to the storage dtype before the convolution.  Stride-1 layers only: the 3-channel first layer
 * returns UNSUPPORTED (fold it instead).  Errors: INVALID_ARG (NULL, eps <= 0), MISALIGNED,
 * UNSUPPORTED, DEVICE, CUDA.
 */
cbr_status_t cbr_forward_infer_bn(const cbr_desc_t* desc, const void* x, const void* w,
                                  const float* conv_bias, const float* gamma, const float* beta,
                                  const float* running_mean, const float* running_var, float eps,
                                  void* y, cbr_stream_t stream);

/*
 * Training forward that allocates nothing and takes no workspace.  The pages have no
 * counterpart; this exists for callers that must not allocate device memory on their
 * execution path, such as plug-ins that run inside another framework's execution loop with
 * no access to its allocator, or latency-critical loops where cudaMalloc's cost and implicit
 * synchronisation are unacceptable.
 *   Same arguments and results as cbr_forward_train, except: no ws / ws_bytes, and z_saved
 *   is required (INVALID_ARG when NULL), because the conv output cannot live in the fixed
 *   scratch.
 *   Scratch: a 320 KiB array compiled into the library, held by every GPU that loads it
 *   until the process exits.  A problem whose scratch need exceeds it returns
 *   CBR_ERR_WORKSPACE before anything is enqueued (with Cout <= 128 the need is about
 *   261 KiB, so supported shapes fit).
 *   The first call on each device looks up the array's device address (one
 *   cudaGetSymbolAddress with that device current); make that first call before any stream
 *   capture.  Each call clears the array's arrival counters with an asynchronous memset on
 *   `stream`.  All calls share the one array: calls that overlap on the GPU (different streams
 *   without ordering) race and give undefined results.  No cudaMalloc, cudaFree or other
 *   allocating routine is called.
 */
cbr_status_t cbr_forward_train_noalloc(const cbr_desc_t* desc, const void* x, const void* w,
                                       const float* gamma, const float* beta, float* running_mean,
                                       float* running_var, float momentum, float eps, void* y,
                                       uint32_t* relu_mask, void* z_saved, float* saved_mean,
                                       float* saved_inv_var, cbr_stream_t stream);

/*
 * ReLU-mask transcoding between this library's bit-packed mask (bit i of 32-bit word j is NHWC
 * element 32*j + i) and one byte per element (0 or 1), the form a standalone ReLU keeps
 * (CBR page, sections 8 and 9: the fused operator's BOOLEAN mask against the standalone
 * ReLU's INT8 mask, transcoded by its equivalence tests).
 *   count       elements (>= 0; 0 is a no-op)
 *   bits        ceil(count/32) uint32 words, 4-byte aligned
 *   bytes       count bytes, 16-byte aligned
 * cbr_mask_bits_to_bytes writes 0 or 1 per element.  cbr_mask_bytes_to_bits sets a bit for
 * every non-zero byte and writes the bits past `count` in the last word as 0.  Asynchronous on
 * `stream`.  Errors: INVALID_ARG (count < 0, or a NULL buffer with count > 0), MISALIGNED,
 * DEVICE, CUDA.
 */
cbr_status_t cbr_mask_bits_to_bytes(const uint32_t* bits, uint8_t* bytes, int64_t count,
                                    cbr_stream_t stream);
cbr_status_t cbr_mask_bytes_to_bits(const uint8_t* bytes, uint32_t* bits, int64_t count,
                                    cbr_stream_t stream);

/*
 * Synchronise `stream`, then read and clear the device error word of the current device.
 * Returns CBR_OK, CBR_ERR_TIMEOUT if a kernel abandoned a bounded wait (its outputs are then
 * undefined), or CBR_ERR_CUDA if the stream reports a CUDA error.
 */
cbr_status_t cbr_stream_status(cbr_stream_t stream);

/*
 * Failure-detection self-test (the pages have no counterpart; it exercises the library's own
 * error path).  Launches one warp on `stream` that waits, with the same bounded barrier wait
 * the library's kernels use, on a barrier nothing completes; after `limit_us` microseconds it
 * gives up, records the timeout in the device error word and exits.  The following
 * cbr_stream_status(stream) then returns CBR_ERR_TIMEOUT and clears the word, and the CUDA
 * context stays usable: no fault, trap or hang is involved.  Returns CBR_ERR_INVALID_ARG unless
 * 1 <= limit_us <= 1,000,000, CBR_ERR_DEVICE if the current device is not compute 10.3, else
 * CBR_OK (the wait itself runs asynchronously).
 */
cbr_status_t cbr_selftest_bounded_wait(int32_t limit_us, cbr_stream_t stream);

/*
 * Profiling hook for the calling host thread.  When `events` is non-NULL, the next
 * cbr_forward_train / cbr_backward / cbr_forward_infer call records events[0] before its
 * first kernel and events[i] after its i-th kernel (cudaEvent_t handles owned by the caller,
 * at most `count`), then clears the hook.  cbr_profile_last_count() returns how many events
 * that call recorded.  Used to time each kernel inside the real calls.  When the call is made
 * while its stream is being captured into a CUDA graph, the events are recorded as external
 * event-record nodes (cudaEventRecordExternal), so they timestamp every replay of the graph.
 */
cbr_status_t cbr_profile_next_call(void* const* events, int32_t count);
int32_t cbr_profile_last_count(void);

/* ======================================================================= token operators
 *
 * What a trunk of blocks and a training objective need on top of a CBR stem, whose NHWC feature
 * map is a grid of tokens: norms around a gated residual block, rotary positions over several
 * axes, and a distillation loss from a teacher's top logits.  The conventions above hold (caller
 * owns every buffer, asynchronous on `stream`, host-side validation before anything is enqueued),
 * with these differences: strides are in elements and counted in 64 bits (each up to 2^40, and up
 * to 2^58 times the steps of its axis); a tensor need only be aligned to its element; a call whose output is empty (no rows, no tokens) does nothing and
 * returns CBR_OK; and device data is never trusted (an entry id outside the vocabulary is an
 * absent entry, an axis outside the position's axes is the last one).
 * Rows of one output may not overlap, and no output may overlap an input except where it says so.
 */

/*
 * Distillation from a teacher's top logits.  For each row r of student logits s (temperature T):
 *   x = s / T,  log q_v = x_v - log sum_u exp x_u
 *   the row's entries k are (top_ids[r][k], top_logits[r][k]); an id outside [0, vocab) marks an
 *   absent entry, whose logit is not used
 *   teacher_lse NULL: p = softmax of t / T over the present entries, no tail (p_rest = 0)
 *   teacher_lse set:  p_k = exp(t_k / T - teacher_lse[r]) (the log-sum-exp of t / T over the
 *                     teacher's whole vocabulary), p_rest = max(0, 1 - sum p_k), and q_rest is the
 *                     student's mass outside the listed ids; p_rest = 0 where q_rest is 0 (below
 *                     2^-1074: e^-744, so words masked with the type's lowest value leave no tail)
 *   loss_r  = w_r T^2 (sum_k p_k (log p_k - log q_k) + p_rest (log p_rest - log q_rest))
 *   dlogits = dloss_r w_r T (q_v (sum p + p_rest) - sum over the entries of v of p_k
 *                            - [v is not listed] q_v p_rest / q_rest)
 * An id listed twice counts twice in the sums.  0 log 0 is 0.  w = row_weight, or 1 where NULL.
 * A row has loss 0, gradient 0 and statistics 0, whatever its other values (NaN included), if
 * w_r = 0; or no entry is present (teacher_lse NULL: none above -infinity); or no student logit
 * is above -infinity.  Other NaN and infinities go through the formulas, in their row alone.
 * Of 16-bit logits, exponentials below 2^-126 of the largest logit's (with a tail: of the largest
 * unlisted one's, for the unlisted words' share of it) count as 0, so a bf16 gradient that small is 0.
 */
typedef struct {
  int64_t rows, vocab;      /* rows >= 0; 1 <= vocab <= 393216 */
  int64_t topk;             /* entries a row, 0 <= topk <= 1024 */
  int64_t logits_stride;    /* elements between rows, >= vocab */
  int64_t dlogits_stride;
  int64_t ids_stride;       /* elements between rows of top_ids, >= topk */
  int64_t top_stride;       /* elements between rows of top_logits, >= topk */
  int32_t dtype;            /* of logits and dlogits */
  int32_t top_dtype;        /* of top_logits */
  int32_t id_bytes;         /* 4 (int32) or 8 (int64) */
  float temperature;        /* > 0; log2(e) / temperature has to be finite */
} cbr_distill_desc_t;

/*
 * Loss.  logits [rows][vocab], top_ids and top_logits [rows][topk], teacher_lse [rows] fp32 or
 * NULL, row_weight [rows] fp32 or NULL -> loss [rows] fp32, stats [rows][3] fp32 (the largest
 * logit, the sum of exp((s - largest) / T) over the row and over its unlisted ids; with
 * teacher_lse, the latter's logarithm to base 2 instead where it is below 2^-64, a negative
 * number, and 0 below 2^-1074) for the backward.  Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED, DEVICE, CUDA.
 */
cbr_status_t cbr_distill_forward(const cbr_distill_desc_t* desc, const void* logits, const void* top_ids,
                                 const void* top_logits, const float* teacher_lse, const float* row_weight,
                                 float* loss, float* stats, cbr_stream_t stream);

/*
 * Gradient, from the forward's stats and dloss [rows] fp32 (NULL: ones) -> dlogits [rows][vocab].
 * dlogits may be logits itself (same address and stride).
 */
cbr_status_t cbr_distill_backward(const cbr_distill_desc_t* desc, const float* dloss, const void* logits,
                                  const void* top_ids, const void* top_logits, const float* teacher_lse,
                                  const float* row_weight, const float* stats, void* dlogits, cbr_stream_t stream);

/*
 * Loss and gradient (of the loss itself: dloss = 1) in one call that reads the logits once.  loss
 * and dlogits are those of the two calls above; stats may be NULL.  dlogits may be logits itself.
 */
cbr_status_t cbr_distill_forward_backward(const cbr_distill_desc_t* desc, const void* logits, const void* top_ids,
                                          const void* top_logits, const float* teacher_lse,
                                          const float* row_weight, float* loss, float* stats, void* dlogits,
                                          cbr_stream_t stream);

/*
 * The norms around a block f, its gate and its residual scale, in one pass over the rows:
 *   n     = (f - m1) r1 post_weight                    the norm after the block
 *   x_out = residual_scale x + branch_scale gate n     the join
 *   h     = (x_out - m2) r2 pre_weight                 the norm before the next block
 * with r = 1 / sqrt(mean((a - m)^2) + eps) over a row, m its mean (CBR_NORM_LAYER) or 0
 * (CBR_NORM_RMS); neither kind has a bias.  h is computed from x_out before it is rounded.  Sums are
 * kept in fp32: r is 0 for a row whose squares pass its range, as for one with an infinity.  Either
 * half may stand alone: post_weight and branch NULL: h = norm of x (there is no x_out); pre_weight
 * NULL: x_out only.
 * gate [rows / gate_rows][dim]: one row for each gate_rows consecutive rows (gate_rows = rows: one
 * gate vector; 1: a gate for every row); NULL: no gate.  Weights, gate and their gradients are
 * fp32, the rest has the storage dtype.
 */
typedef enum { CBR_NORM_RMS = 0, CBR_NORM_LAYER = 1 } cbr_norm_kind_t;
typedef struct {
  int64_t rows;             /* >= 0 */
  int64_t dim;              /* 1 .. 16384 */
  int64_t gate_rows;        /* rows is a multiple of it; not used without a gate */
  int64_t x_stride, branch_stride, x_out_stride, h_stride;           /* elements between rows, >= dim */
  int64_t dx_out_stride, dh_stride, dx_stride, dbranch_stride;       /* backward */
  int32_t dtype, kind;
  float eps;                /* > 0 (forward) */
  float residual_scale, branch_scale;
} cbr_block_norm_desc_t;

/*
 * Forward -> x_out [rows][dim], h [rows][dim], stats [rows][4] fp32 (m1, r1, m2, r2; 0 for a norm
 * that is not there), which may be NULL.  x_out may be x or branch itself, and h branch itself or
 * (without a branch) x itself: same address and stride.
 */
cbr_status_t cbr_block_norm_forward(const cbr_block_norm_desc_t* desc, const void* x, const void* branch,
                                    const float* post_weight, const float* gate, const float* pre_weight,
                                    void* x_out, void* h, float* stats, cbr_stream_t stream);

/* Workspace bytes of the backward for this desc (dim, dtype): per-block sums of the parameter gradients. */
cbr_status_t cbr_block_norm_workspace_size(const cbr_block_norm_desc_t* desc, size_t* bytes);

/*
 * Backward.  dx_out [rows][dim] is the gradient that reaches x_out from later in the residual
 * stream (NULL where there is none: only h is used), dh that at h (unused without pre_weight).
 * x_out is the forward's (without a branch: x itself).  With u = dh pre_weight, c = (x_out - m2) r2:
 *   D = dx_out + r2 (u - [LAYER] mean(u) - c mean(u c));     dpre_weight = sum over rows of dh c
 *   dx = residual_scale D  (without a branch: D)
 *   with e = (f - m1) r1:  dgate = sum over a gate's rows of branch_scale D e post_weight
 *   dpost_weight = sum over rows of branch_scale D gate e;  v = branch_scale D gate post_weight
 *   dbranch = r1 (v - [LAYER] mean(v) - e mean(v e))
 * Sums over rows are kept in fp32 and added in a fixed order, so results repeat bit for bit.
 * dx may be dx_out itself, dbranch may be branch or dh itself.
 */
cbr_status_t cbr_block_norm_backward(const cbr_block_norm_desc_t* desc, const void* dx_out, const void* dh,
                                     const void* x_out, const void* branch, const float* post_weight,
                                     const float* gate, const float* pre_weight, const float* stats, void* dx,
                                     void* dbranch, float* dpost_weight, float* dgate, float* dpre_weight,
                                     void* ws, size_t ws_bytes, cbr_stream_t stream);

/*
 * Rotary positions over several axes (time, height, width, ...), on queries and keys in one call.
 * The first rot_dim elements of a head are rot_dim / 2 pairs: (i, i + rot_dim / 2) in
 * CBR_ROTARY_HALVES, (2 i, 2 i + 1) in CBR_ROTARY_NEIGHBOURS; the others are copied.  Pair i
 * follows the position's axis axis[i], at freq[i] turns a step:
 *   angle = 2 pi positions[b][t][axis[i]] freq[i] / 2^64
 *   (y1, y2) = (x1 cos(angle) - x2 sin(angle), x2 cos(angle) + x1 sin(angle))
 * freq is the frequency f_i (radians a step) as a fixed-point fraction of a turn,
 * round(f_i / (2 pi) 2^64): the product with a position is taken modulo 2^64, that is modulo whole
 * turns, without rounding, so far positions lose nothing.  Positions may be negative.
 */
typedef enum { CBR_ROTARY_HALVES = 0, CBR_ROTARY_NEIGHBOURS = 1 } cbr_rotary_layout_t;
typedef struct {
  int64_t batch, tokens;                 /* >= 0 */
  int64_t q_stride[3], k_stride[3];      /* elements between batches, tokens, heads; the head's own are adjacent */
  int64_t q_out_stride[3], k_out_stride[3];
  int64_t pos_stride[3];                 /* elements between batches, tokens, axes; 0 repeats */
  int32_t heads_q, heads_k;              /* 0 without q or k */
  int32_t head_dim, rot_dim;             /* head_dim <= 1024; rot_dim even, 2 .. head_dim */
  int32_t axes;                          /* 1 .. 8 */
  int32_t layout, dtype;
} cbr_rotary_desc_t;

/*
 * q_out may be q itself and k_out k itself (same address and strides).  An output's axes may lie in any
 * order in memory, each stepping past all that the smaller ones reach.
 */
cbr_status_t cbr_rotary_forward(const cbr_rotary_desc_t* desc, const void* q, const void* k,
                                const int32_t* positions, const int64_t* freq, const uint8_t* axis, void* q_out,
                                void* k_out, cbr_stream_t stream);

/* The gradients at q and k from those at q_out and k_out: the rotation by the opposite angle. */
cbr_status_t cbr_rotary_backward(const cbr_rotary_desc_t* desc, const void* dq_out, const void* dk_out,
                                 const int32_t* positions, const int64_t* freq, const uint8_t* axis, void* dq,
                                 void* dk, cbr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CBR_H_ */
