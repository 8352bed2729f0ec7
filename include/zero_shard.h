/*
 * zero_shard.h -- C ABI of the MI355X (gfx950) ZeRO-1/2 shard optimizer step.
 *
 * One data-parallel rank owns partition r of the flat parameter vector
 * theta = [theta_1 .. theta_N] and keeps the fp32 optimizer state for that
 * partition only ("Data parallelism and ZeRO optimization", sections
 * "ZeRO-1: Optimizer State Partitioning" and "ZeRO-2: Gradient
 * Partitioning"; "ZeRO (딥 러닝)", stage table of "ZeRO-DP의 세 단계").
 * Between the reduce-scatter of the gradients and the all-gather of the
 * updated weights ("ZeRO (딥 러닝)", "왜 통신량이 늘지 않는가") the rank:
 *
 *   a1  sums the N_d incoming bf16 gradient contributions for its slice in
 *       rank order and averages them ("大模型并行技术", "优化状态与梯度分割",
 *       step 2; "How Standard Data Parallelism Works": the average);
 *   a2  optionally clips by the global L2 norm of the averaged gradient
 *       ("ZeRO (딥 러닝)", "DeepSpeed에서 쓰기": gradient_clipping);
 *   a3  runs mixed-precision AdamW on its fp32 master weights, momentum and
 *       variance ("Memory Consumption Analysis"; "精度混合训练");
 *   a4  writes the bf16 copy of the updated master weights, the buffer the
 *       all-gather sends;
 *   a5  optionally block-quantizes that copy to int8 codes plus one fp32
 *       scale per block (ZeRO++ qwZ, "ZeRO (딥 러닝)", follow-ups table
 *       "후속 기법").
 *
 * Arithmetic (what every call computes, element i of the shard):
 *   s_i    = sum_{k=0}^{n_d-1} bf16(contrib[k][i])   binary64, k ascending
 *   gbar_i = binary32(s_i / n_d)                      one rounding
 *   g_i    = coef * gbar_i                            binary64; coef = 1
 *            unless clipping: coef = min(1, max_norm / (sqrt(S) + 1e-6)),
 *            S = global sum of gbar^2 handed to zero_shard_step
 *   m'     = b1 m + (1-b1) g        v' = b2 v + (1-b2) (g g)
 *   theta' = theta - (lr wd) theta - lr (m'/bc1) / (sqrt(v'/bc2) + eps)
 *            bc = 1 - beta^t with bias correction, else 1; all binary64
 *            from the binary32 state, each result rounded once to binary32
 *   p_i    = bf16(theta'_i), round to nearest even
 *   int8:  block b = elements [b*B, b*B+B) of the shard (last one partial);
 *          a = max |p|, scale = binary32(a / 127), code = round-half-even(
 *          binary32(p / scale)) clamped to +-127; scale 0 => codes 0;
 *          a non-finite quotient gives code 0.
 * With int8 contributions (the _q8 calls) element i of row k stands for
 * code_k[i] * scale_k[i / block], an exact binary64 product, and s_i sums
 * those products in the same k order.
 * Non-finite inputs propagate per IEEE; no step is skipped.
 *
 * Memory: every pointer in zs_desc and every contribution pointer is a
 * device pointer (HBM of the current device), allocated and owned by the
 * caller, and must stay valid until the work queued on the stream is done.
 * Layouts are flat, contiguous, element i at offset i.  fp32 and bf16
 * arrays and every contribution row must be 16-byte aligned; q_codes 8-byte
 * aligned.  The library owns only the handle and a small device scratch
 * (one fp64 partial of the norm per 16384 shard elements, or per 4096 with
 * int8 contributions), allocated at init; the bucketed calls add worker
 * streams and per-bucket scratch on first use.
 *
 * Errors: every call returns ZS_OK (0) or a negative zs_status.  Arguments
 * are validated before anything is queued: on an error nothing is launched
 * and no output is touched.  Launch failures are reported as ZS_EHIP;
 * faults inside a kernel surface at the caller's next synchronisation.
 * Calls are asynchronous on the handle's stream; a handle is used by one
 * host thread at a time.
 */
#ifndef ZERO_SHARD_H
#define ZERO_SHARD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zs_handle zs_handle; /* opaque */
typedef uint16_t zs_bf16;           /* bf16 bit pattern */

typedef enum zs_status {
  ZS_OK = 0,
  ZS_EINVAL = -1,  /* bad size, index, hyper-parameter or missing pointer */
  ZS_EALIGN = -2,  /* a pointer is not aligned as required                */
  ZS_ENOMEM = -3,  /* the library's own scratch could not be allocated     */
  ZS_EHIP = -4,    /* a HIP runtime call or kernel launch failed           */
  ZS_EDEVICE = -5, /* the current device is not gfx950                     */
  ZS_ESTATE = -6,  /* call out of order (step reading a gradient spill
                      that no norm pass has written) or a dead handle      */
  ZS_ETOOBIG = -7  /* shard longer than zero_shard_gnorm_noalloc's static
                      scratch allows                                       */
} zs_status;

#define ZS_MAX_ND 64 /* most contributions one call can average */

/* How the work of a call is split into kernel launches (on the call's
 * stream, in order; the split changes no result).  The norm pass over n
 * elements (the shard, or one bucket) queues ceil(n / ZS_NORM_LAUNCH_LEN)
 * partial-sum launches and one final reduction.  An update that reads the
 * contribution rows (no spill) runs in its wide form, as
 * ceil(n / ZS_WIDE_LAUNCH_LEN) launches, from ZS_WIDE_MIN_ROWS bf16 rows
 * (ZS_WIDE_MIN_ROWS_QUANT when it also writes int8) or ZS_WIDE_MIN_ROWS_Q8
 * int8 rows; any other update is one launch. */
#define ZS_NORM_LAUNCH_LEN (INT64_C(1) << 26)
#define ZS_WIDE_LAUNCH_LEN (INT64_C(1) << 25)
#define ZS_WIDE_MIN_ROWS 18
#define ZS_WIDE_MIN_ROWS_QUANT 32
#define ZS_WIDE_MIN_ROWS_Q8 16

typedef struct zs_desc {
  /* partition geometry */
  int64_t phi;       /* parameters in the whole flat buffer, >= 0           */
  int32_t n_d;       /* data-parallel degree, 1..ZS_MAX_ND                  */
  int32_t r;         /* partition index, 0 <= r < n_d                       */
  int64_t shard_len; /* elements of partition r: min(ceil(phi/n_d),
                        phi - r*ceil(phi/n_d)) clamped at 0; or phi with
                        r == 0 for the unpartitioned (stage 0) update        */
  /* optimizer: binary32 values, used widened to binary64 */
  float beta1, beta2; /* in [0, 1)                                          */
  float eps;          /* > 0                                                */
  float weight_decay; /* >= 0, decoupled; 0 = plain Adam                    */
  int32_t bias_correction; /* 1: divide by 1 - beta^t; 0: do not          */
  float max_norm;     /* > 0: clip by the global norm; <= 0: no clipping   */
  int32_t quant_block; /* 0: no int8; else 32, 64, 128, 256 or 512: the
                          step also writes codes and scales (fused)        */
  /* state and outputs (device pointers, caller-owned) */
  float *master, *m, *v; /* fp32[shard_len], updated in place; these four  */
  zs_bf16 *param_out;    /* bf16[shard_len]  may all be NULL for a norm-only
                            handle (state offloaded to the host, see
                            zero_shard_host_step), which needs gbar_ws and
                            refuses zero_shard_step / zero_shard_quant     */
  int8_t *q_codes;       /* int8[shard_len]; needed iff quant_block > 0 or
                            zero_shard_quant is called                     */
  float *q_scales;       /* fp32[ceil(shard_len / block)], same condition  */
  float *gbar_ws;        /* optional fp32[shard_len] workspace; with
                            clipping, zero_shard_gnorm stores the averaged
                            gradient there and zero_shard_step reads it
                            instead of re-reading the contributions        */
  void *stream;          /* hipStream_t for every call; NULL = null stream */
} zs_desc;

/* Validate d, check that the current device is gfx950, allocate the norm
 * scratch, and return a handle in *out.  The descriptor is copied.
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_ENOMEM, ZS_EHIP. */
int zero_shard_init(const zs_desc *d, zs_handle **out);

/* a2, first sweep: this shard's sum of squares of the averaged gradient,
 * S_local = sum_i gbar_i^2 (binary64), reduced over a grid fixed by the
 * shard length, in a fixed order, with no atomics (same inputs => same
 * bits).  contrib is a HOST array of n_d device pointers, contrib[k] =
 * rank k's bf16 gradient for this shard (shard-local index).  Writes
 * S_local to *sumsq_dev (device, one double).  With gbar_ws set, also
 * stores gbar there for the next step.
 * Summing S_local over the shards (one scalar all-reduce across ranks) gives
 * the S that zero_shard_step takes.  Errors: ZS_EINVAL, ZS_EALIGN, ZS_EHIP,
 * ZS_ESTATE. */
int zero_shard_gnorm(zs_handle *h, const zs_bf16 *const *contrib, double *sumsq_dev);

/* zero_shard_gnorm for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same sum of squares S_local and the same spill (when
 * d->gbar_ws is set), bit for bit, without a handle.  Takes the descriptor
 * itself (d->n_d, d->shard_len, d->gbar_ws and d->stream are used; the
 * state pointers and hyper-parameters are ignored), contrib and sumsq_dev as
 * for zero_shard_gnorm.  It allocates nothing: the block partials live in a
 * static device array of the library (512 KiB on each GPU the library runs
 * on, kept until the process ends), which bounds the shard at one partial
 * per 16384 elements, 65536 partials: shard_len <= 2^30 (ZS_ETOOBIG
 * beyond).  Every call on one GPU uses that GPU's one array: calls that
 * overlap on one GPU (other streams, other threads) race and must be
 * ordered by the caller; the partials need no clearing (each call writes
 * all it reads).  Queues ceil(shard_len / ZS_NORM_LAUNCH_LEN) + 1 kernel
 * launches (at least two) on d->stream and nothing else.
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_ETOOBIG, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_gnorm_noalloc(const zs_desc *d, const zs_bf16 *const *contrib,
                             double *sumsq_dev);

/* a1 + a3 + a4 (+ a5 when quant_block > 0): one optimizer step at 1-based
 * step counter t with learning rate lr >= 0.  contrib as for gnorm; it may
 * be NULL when clipping with gbar_ws (the spill written by the preceding
 * zero_shard_gnorm is read instead).  global_sumsq_dev (device, one double)
 * is S and is required iff max_norm > 0; it is read on the device, so no
 * host synchronisation is needed between gnorm and step.  gnorm and step
 * queue kernel launches only (no allocation, no memset), so they can be
 * captured in a HIP graph on the handle's stream; t and lr are then fixed
 * in the captured launches (zero_shard_step_dev reads them from device
 * memory instead).
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_ESTATE, ZS_EHIP. */
int zero_shard_step(zs_handle *h, const zs_bf16 *const *contrib, float lr, int64_t t,
                    const double *global_sumsq_dev);

/* The constants of step t at learning rate lr as the library computes them
 * on the host for zero_shard_step: out[0] = lr, out[1] = lr * weight_decay,
 * out[2] = bc1 = 1 - beta1^t, out[3] = bc2 = 1 - beta2^t (1 and 1 without
 * bias correction), binary64 from d's binary32 values (pow of the C
 * library).  out is a HOST array of 4 doubles; only d's hyper-parameters are
 * read.  Errors: ZS_EINVAL (bad d, lr or t). */
int zero_shard_step_consts(const zs_desc *d, float lr, int64_t t, double *out);

/* zero_shard_step with the step's constants read on the device, when the
 * kernel runs, from consts_dev (device, 4 doubles, 8-byte aligned, laid out
 * as zero_shard_step_consts writes them) instead of fixed at the call.  A
 * step captured in a HIP graph then serves every step: before each replay
 * the caller writes that step's constants to consts_dev (outside the graph,
 * e.g. an asynchronous copy on the same stream).  With the constants of
 * (lr, t) the results are zero_shard_step's at (lr, t), bit for bit.  The
 * constants are trusted as given.  Errors: ZS_EINVAL, ZS_EALIGN, ZS_ESTATE,
 * ZS_EHIP. */
int zero_shard_step_dev(zs_handle *h, const zs_bf16 *const *contrib, const double *consts_dev,
                        const double *global_sumsq_dev);

/* a1 with int8 contributions: ZeRO++ qgZ ("ZeRO (딥 러닝)", follow-ups table
 * "후속 기법": gradients are quantized and averaged after an all-to-all).
 * Row k is codes[k], int8[shard_len] (8-byte aligned), with one fp32 scale
 * per `block` contiguous shard elements starting at element 0, scales[k],
 * fp32[ceil(shard_len / block)] (4-byte aligned); codes and scales are HOST
 * arrays of n_d device pointers; block is 32, 64, 128, 256 or 512.
 * Otherwise exactly zero_shard_gnorm and zero_shard_step (codes and scales
 * may be NULL when the step reads the gradient spill).  Errors: as there. */
int zero_shard_gnorm_q8(zs_handle *h, const int8_t *const *codes, const float *const *scales,
                        int32_t block, double *sumsq_dev);
int zero_shard_step_q8(zs_handle *h, const int8_t *const *codes, const float *const *scales,
                       int32_t block, float lr, int64_t t, const double *global_sumsq_dev);

/* Bucketed step ("ZeRO (딥 러닝)", "DeepSpeed에서 쓰기": overlap_comm,
 * contiguous_gradients, reduce_bucket_size in the configuration example;
 * "ZeRO-R: 잔여 메모리 최적화": gradient communication through buffers of a
 * fixed size, independent of the model).  Gradients reach the owner rank
 * bucket by bucket, so the shard's elements [0, shard_len) are processed in
 * buckets of bucket_len elements (bucket j: [j*bucket_len, ...), the last
 * one shorter), each as soon as its slice of the contributions is in place,
 * overlapping the arrival of later buckets.
 *
 * contrib is a HOST array of n_d device pointers to the whole shard's rows,
 * as for zero_shard_gnorm (contiguous gradients: bucket j of row k starts at
 * contrib[k] + j*bucket_len).  bucket_len > 0 is a multiple of 512 (every
 * bucket starts on a vector and a quantizer-block boundary).  ready is NULL
 * (everything in place) or a HOST array of ceil(shard_len / bucket_len)
 * hipEvent_t, entries may be NULL: bucket j's work waits for ready[j],
 * which the caller has recorded (e.g. on its communication stream after
 * bucket j's reduce-scatter) before this call.  Buckets are distributed
 * round-robin over `streams` (1..4) worker streams that the handle creates
 * on first use (default priority) and that start after the work already
 * queued on the handle's stream; the handle's stream waits for all of them
 * before the call returns, so later calls on it are ordered after every
 * bucket.  The first call, or one with more buckets than before, allocates
 * the per-bucket scratch.
 *
 * zero_shard_gnorm_bucketed: a2's first sweep per bucket (spilling gbar as
 * zero_shard_gnorm does), then S_local = the per-bucket sums added in
 * bucket order, to *sumsq_dev.  Same result as zero_shard_gnorm up to the
 * association of the binary64 sum.
 * zero_shard_step_bucketed: the fused step (a1, a3, a4, a5) per bucket;
 * each element's result is bit-identical to zero_shard_step's.  With
 * clipping and gbar_ws it reads the spill and contrib may be NULL.
 * Errors: as zero_shard_gnorm / zero_shard_step; ZS_EINVAL also for a bad
 * bucket_len or streams; ZS_ENOMEM. */
int zero_shard_gnorm_bucketed(zs_handle *h, const zs_bf16 *const *contrib, int64_t bucket_len,
                              int32_t streams, const void *const *ready, double *sumsq_dev);
int zero_shard_step_bucketed(zs_handle *h, const zs_bf16 *const *contrib, int64_t bucket_len,
                             int32_t streams, const void *const *ready, float lr, int64_t t,
                             const double *global_sumsq_dev);

/* The bucketed calls with int8 contributions (qgZ, as the _q8 calls above):
 * codes[k] / scales[k] are rank k's whole-shard rows; bucket j of row k
 * starts at codes[k] + j*bucket_len and scales[k] + j*bucket_len/block
 * (bucket_len is a multiple of 512, so of every block).  Errors: as the
 * bucketed calls and the _q8 calls. */
int zero_shard_gnorm_bucketed_q8(zs_handle *h, const int8_t *const *codes,
                                 const float *const *scales, int32_t block, int64_t bucket_len,
                                 int32_t streams, const void *const *ready, double *sumsq_dev);
int zero_shard_step_bucketed_q8(zs_handle *h, const int8_t *const *codes,
                                const float *const *scales, int32_t block, int64_t bucket_len,
                                int32_t streams, const void *const *ready, float lr, int64_t t,
                                const double *global_sumsq_dev);

/* a5 as a separate pass: quantize param_out into q_codes / q_scales with
 * the given block (32, 64, 128, 256 or 512); q_scales must hold
 * ceil(shard_len / block) floats.  Errors: ZS_EINVAL, ZS_EHIP. */
int zero_shard_quant(zs_handle *h, int32_t block);

/* qwZ receive side (ZeRO++, "ZeRO (딥 러닝)" follow-ups table "후속 기법"):
 * after the all-gather of the n_d int8 shards, rebuild the whole bf16
 * parameter vector.  Shard r holds flat elements [r*ceil(phi/n_d), ...) of
 * length zero_shard_len(phi, n_d, r); codes[r] is its int8[len] (8-byte
 * aligned) and scales[r] its fp32[ceil(len / block)] (4-byte aligned), one
 * scale per `block` elements counted from the shard's own element 0, as
 * zero_shard_step writes them.  codes and scales are HOST arrays of n_d
 * device pointers (entries of empty shards may be NULL).  Writes
 * param_out[i] = bf16(binary32(code * scale)) (nearest even) for all phi
 * elements of param_out (device, 16-byte aligned).  No handle: it reads
 * every rank's shard.  Asynchronous on `stream` (hipStream_t, NULL = null
 * stream).  Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_dequant(const int8_t *const *codes, const float *const *scales, int32_t n_d,
                       int64_t phi, int32_t block, zs_bf16 *param_out, void *stream);

/* ZeRO-Offload host step ("ZeRO (딥 러닝)", follow-ups table "후속 기법":
 * optimizer states and the update in CPU memory, an optimized CPU Adam, a
 * one-step delayed update).  a3 + a4 (+ a5) on the CPU for the shard
 * described by d, whose master/m/v/param_out/q_codes/q_scales are HOST
 * pointers here (d->stream and d->gbar_ws are ignored); gbar is the host
 * fp32[shard_len] averaged gradient, e.g. the device spill that
 * zero_shard_gnorm wrote, copied to the host.  global_sumsq is S, used iff
 * d->max_norm > 0.  The arithmetic is the device step's, so the result is
 * bit-identical to zero_shard_step on the same inputs.  Synchronous; runs
 * on `threads` host threads (>= 1), which take contiguous 2^18-element,
 * block-aligned pieces of the shard in turn (the split changes no bit).
 * Errors: ZS_EINVAL. */
int zero_shard_host_step(const zs_desc *d, const float *gbar, float lr, int64_t t,
                         double global_sumsq, int32_t threads);

/* ZeRO-Offload pipeline for one rank's shard ("ZeRO (딥 러닝)", follow-ups
 * table "후속 기법": optimizer states and their update on the CPU, the
 * update hidden behind the GPU's next step by a one-step delayed update).
 *
 * zero_shard_offload_init: `host` describes the shard with HOST pointers
 * for master/m/v (and q_codes/q_scales when quant_block > 0), as for
 * zero_shard_host_step; its param_out, gbar_ws and stream are ignored.
 * param_dev0/param_dev1 are two device bf16[shard_len] buffers (16-byte
 * aligned) that the updated parameters are uploaded into, alternately;
 * `stream` is the caller's compute stream; `threads` (>= 1) host threads
 * run the update.  The library allocates a device spill and S scalar, two
 * pinned gradient slots and two pinned bf16 slots, a download and an
 * upload stream, and one event per 2^24-element chunk of each gradient slot.
 *
 * zero_shard_offload_step: step t.  Queues on `stream` the norm pass over
 * contrib (a HOST array of n_d device pointers, as for zero_shard_gnorm),
 * then copies S_local and the averaged gradient to pinned memory (the
 * gradient in chunks of 2^24 elements), waits for the host update of the
 * previous step to finish, orders `stream` after that step's upload, starts
 * this step's host update (a3-a5 with S = S_local + s_other, s_other >= 0
 * being the other shards' sum) on a host thread, and returns.  The host
 * update takes each chunk as soon as its copy has landed and uploads each
 * chunk of its bf16 parameters into buffer (call index mod 2) as soon as
 * it is written.  Work queued on `stream` after the call
 * sees the parameters of the previous step: zero_shard_offload_params
 * names that buffer (NULL before any update has been uploaded).
 * zero_shard_offload_wait: finish the running host update and order
 * `stream` after its upload; zero_shard_offload_params then names the
 * newest parameters.  zero_shard_offload_init rejects a descriptor the host
 * update would reject (geometry, beta, eps, weight decay, max_norm, block)
 * before it allocates anything, and zero_shard_offload_step rejects a bad
 * lr, t or s_other (negative or non-finite) before it queues anything; an
 * error inside a running host update is returned by the next step or wait
 * call.  zero_shard_offload_free waits and releases.
 * The results are those of zero_shard_step on the same inputs, bit for bit.
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_ENOMEM, ZS_EHIP, ZS_ESTATE. */
typedef struct zs_offload zs_offload;
int zero_shard_offload_init(const zs_desc *host, zs_bf16 *param_dev0, zs_bf16 *param_dev1,
                            void *stream, int32_t threads, zs_offload **out);
int zero_shard_offload_step(zs_offload *o, const zs_bf16 *const *contrib, float lr, int64_t t,
                            double s_other);
zs_bf16 *zero_shard_offload_params(zs_offload *o);
int zero_shard_offload_wait(zs_offload *o);
int zero_shard_offload_free(zs_offload *o);

/* ---------------------------------------------------------------------------
 * The optimizer and the norm of the parameters around the shard step: the
 * Muon update for a rank's weight matrices, and layer norm, whose gains and
 * biases stay with the shard step.  These calls take no handle: they queue
 * kernel launches on the descriptor's stream and nothing else (no allocation,
 * no memset, no synchronisation), so they can be captured in a HIP graph, and
 * every scratch byte is a workspace the caller owns, which holds nothing
 * between calls.  Calls that overlap on different streams need different
 * workspaces.  Same inputs => same bits.  Errors as above: everything is
 * checked before anything is queued; sizes of zero are valid and queue
 * nothing, except that gradients of no rows are written as zeros. */
typedef enum zs_dtype { ZS_F32 = 0, ZS_BF16 = 1, ZS_F16 = 2 } zs_dtype;

/* Layer norm over rows of `cols` elements, column stride 1, row strides ld_*
 * in elements (0: cols).  Statistics, sums and products are binary32, each
 * output is rounded once to its type (nearest even). */
typedef struct zs_layernorm_desc {
  int64_t rows, cols;  /* rows >= 0, 1 <= cols <= 2^31                        */
  int32_t dtype;       /* zs_dtype of x, residual, sum, y, dy, dsum, dx       */
  int32_t param_dtype; /* of gamma, beta, dgamma, dbeta: ZS_F32 or dtype      */
  float eps;           /* >= 0, finite                                        */
  int64_t ld_x, ld_residual, ld_sum, ld_y; /* forward                         */
  int64_t ld_dy, ld_dsum, ld_dx;           /* backward (which uses ld_x too)  */
  void *stream;        /* hipStream_t, NULL = null stream                     */
} zs_layernorm_desc;

/* Forward:  s = round(x + residual), stored to sum, or s = x when residual
 * and sum are NULL (both or neither);
 *   mean = sum_c s / cols;  rstd = 1 / sqrt(sum_c (s - mean)^2 / cols + eps);
 *   y = (s - mean) rstd gamma + beta.
 * gamma and beta (cols elements) may each be NULL (1 and 0); mean and rstd
 * (fp32[rows]) may each be NULL when no backward pass follows.  A row that
 * holds an infinity or NaN gives NaN in that row only, as does one whose sum is
 * beyond binary32; where the deviations' squares are, rstd is 0.  A constant row
 * gives beta up to rounding (eps > 0; with eps = 0 it has no value).  sum may be x's or
 * residual's own buffer with the same row stride, y may be x's (or
 * residual's) unless sum is; otherwise outputs overlap nothing.
 * Errors: ZS_EINVAL, ZS_EALIGN (a pointer not aligned to its element),
 * ZS_EDEVICE, ZS_EHIP. */
int zero_shard_layernorm(const zs_layernorm_desc *d, const void *x, const void *residual,
                         const void *gamma, const void *beta, void *sum, void *y, float *mean,
                         float *rstd);

/* Bytes of workspace that zero_shard_layernorm_bwd needs for d when dgamma or
 * dbeta is asked for, or -1 for an invalid descriptor. */
int64_t zero_shard_layernorm_workspace(const zs_layernorm_desc *d);

/* Backward of y = h gamma + beta, h = (x - mean) rstd, where x is what was
 * normalised (the forward pass's sum when it had a residual), with its saved
 * mean and rstd:
 *   g = dy gamma;  dx = rstd (g - sum_c g / cols - h sum_c (g h) / cols) + dsum
 *   dgamma = sum_rows dy h;  dbeta = sum_rows dy
 * dsum, the gradient that reaches the sum from elsewhere (the residual path),
 * may be NULL; dx is then the gradient of x and of residual alike.  gamma
 * may be NULL (1); dgamma and dbeta may each be NULL (not computed); they are
 * written, not added to.  dx may be dy's, x's or dsum's own buffer with the same
 * row stride.  workspace: device, 16-byte aligned, at least
 * zero_shard_layernorm_workspace(d) bytes (may be NULL when neither gradient
 * is asked for).  Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_layernorm_bwd(const zs_layernorm_desc *d, const void *dy, const void *x,
                             const void *gamma, const float *mean, const float *rstd,
                             const void *dsum, void *dx, void *dgamma, void *dbeta,
                             void *workspace, int64_t workspace_bytes);

/* The Muon update over a flat range of n elements: one weight matrix, or
 * several of the same shape one after another.  A rank owns whole matrices;
 * contributions are rows as for zero_shard_step.  All arrays 16-byte aligned. */
typedef struct zs_muon_desc {
  int64_t n;           /* elements, >= 0                                      */
  int32_t n_d;         /* contributions averaged, 1..ZS_MAX_ND                */
  int32_t nesterov;    /* 1: look ahead; 0: plain momentum                    */
  int32_t dtype;       /* of the update matrix: ZS_F32 or ZS_BF16             */
  float mu;            /* momentum, in [0, 1)                                 */
  float weight_decay;  /* >= 0, decoupled                                     */
  void *stream;        /* hipStream_t, NULL = null stream                     */
} zs_muon_desc;

/* gbar as in the shard step (binary64 sum in rank order, averaged, rounded to
 * binary32);  M' = mu M + gbar;  u = gbar + mu M' (nesterov) or M'; binary64
 * from binary32 values, M' and u rounded to binary32 once each.  A bf16 u is the
 * bf16 of that binary32 value (as the bf16 weights are of the master's).
 * contrib: HOST array of n_d device pointers to bf16[n]; m_in, m_out: fp32[n],
 * may be the same buffer; update: u.
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_muon_momentum(const zs_muon_desc *d, const zs_bf16 *const *contrib,
                             const float *m_in, float *m_out, void *update);

/* theta' = theta - (lr wd) theta - (lr scale) o, binary64 from binary32 and
 * bf16 values, rounded once; p = bf16(theta').  o: bf16[n], the
 * orthogonalised update; scale: the caller's adjustment for the matrix's
 * shape, e.g. 0.2 sqrt(max(rows, cols)); master_in, master_out: fp32[n], may be
 * the same buffer; param_out: bf16[n], the buffer the all-gather sends.  lr and
 * scale are taken at the call: a captured graph keeps those of its capture.
 * Errors: ZS_EINVAL (lr negative or not finite, ...), ZS_EALIGN, ZS_EDEVICE,
 * ZS_EHIP. */
int zero_shard_muon_apply(const zs_muon_desc *d, const zs_bf16 *o, float lr, float scale,
                          const float *master_in, float *master_out, zs_bf16 *param_out);

#define ZS_ORTHO_MAX_STEPS 32 /* most Newton-Schulz steps of one call */

/* Orthogonalisation of `batch` matrices of rows x cols, column stride 1. */
typedef struct zs_ortho_desc {
  int64_t batch, rows, cols;  /* >= 0; batch <= 65535, sides <= 2^20          */
  int64_t ld_in, ld_out;      /* row strides in elements (0: cols)            */
  int64_t stride_in, stride_out; /* from matrix to matrix (0: rows * ld); the
                                 output's matrices must not overlap           */
  int32_t dtype;              /* zs_dtype of the input                        */
  int32_t steps;              /* Newton-Schulz steps, 1..ZS_ORTHO_MAX_STEPS    */
  const float *coeffs;        /* HOST array of 3 * steps floats, (a, b, c) of
                                 each step; NULL: (3.4445, -4.7750, 2.0315)   */
  float eps;                  /* >= 0, added to the norm                      */
  void *stream;               /* hipStream_t, NULL = null stream              */
} zs_ortho_desc;

/* Bytes of workspace that zero_shard_ortho needs for d, or -1 for an invalid
 * descriptor, among them one with a product of 2^23 or more tiles of 256 x 256,
 * which no launch takes (and no card holds). */
int64_t zero_shard_ortho_workspace(const zs_ortho_desc *d);

/* Per matrix: X = G / (|G|_F + eps) (the norm in binary64), then `steps` times
 *   A = X X^T;  X = a X + (b A + c A A) X
 * (X^T X and products from the right when rows > cols); o = bf16(X).
 * Products are summed in binary32; X, A and B = a I + b A + c A A are rounded
 * to binary16 times 2^-11 between products, and what that takes off A's and B's
 * diagonals is kept in binary32 and made good.  Of a matrix much longer than wide
 * two steps whose a have a product in (0, 16] are taken together: the second A
 * is B A B and X becomes (B' B) X, the same products in another order; B A and
 * B' B are rounded likewise.  The entries of all of them must stay below 32
 * (coefficients that bring singular values in [0, 1] towards 1 keep them below
 * 16), and entries of X under 2^-36 vanish: a matrix whose norm is far below eps
 * gives zeros.  A zero matrix gives zeros (eps > 0; NaN with eps = 0); a matrix
 * that holds an infinity or NaN gives NaN in that matrix only.
 * g: input; o: bf16 output, overlapping nothing else; workspace: device,
 * 256-byte aligned, at least zero_shard_ortho_workspace(d) bytes.
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_ortho(const zs_ortho_desc *d, const void *g, zs_bf16 *o, void *workspace,
                     int64_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * The seam between two blocks of a network: the norm of a block's output, its
 * gate, the scaled residual sum, and the norm before the next block.  No
 * handle; launches only, as for layer norm.
 *
 * Rows of `cols` elements, column stride 1, row strides ld_* in elements (0:
 * cols).  Sums, statistics and products are binary32, each output is rounded once to
 * its type (nearest even). */
#define ZS_BLOCKNORM_MAX_COLS 16384
typedef enum zs_norm_kind { ZS_NORM_LAYER = 0, ZS_NORM_RMS = 1 } zs_norm_kind;
typedef enum zs_gate {
  ZS_GATE_NONE = 0,
  ZS_GATE_COLUMN = 1, /* a factor for each column: param_dtype, cols elements  */
  ZS_GATE_SIGMOID = 2 /* sigmoid(z) for each element: z is dtype, rows x cols;
                         it and its slope are 0 where they are below 2^-126   */
} zs_gate;

typedef struct zs_blocknorm_desc {
  int64_t rows, cols;  /* rows >= 0, 1 <= cols <= ZS_BLOCKNORM_MAX_COLS       */
  int32_t dtype;       /* zs_dtype of x, block, sum, y, their gradients, and z */
  int32_t param_dtype; /* of gains, biases, column gates: ZS_F32 or dtype     */
  int32_t kind;        /* zs_norm_kind of both norms                          */
  int32_t post;        /* 1: the block's output is normalised; 0: it is not   */
  int32_t gate;        /* zs_gate                                             */
  float eps;           /* >= 0, finite                                        */
  float residual_scale;  /* finite                                            */
  int64_t ld_x, ld_block, ld_gate, ld_sum, ld_y;      /* ld_gate: of z        */
  int64_t ld_dy, ld_dsum, ld_dx, ld_dblock, ld_dgate; /* ld_dgate: of z's     */
  void *stream;        /* hipStream_t, NULL = null stream                     */
} zs_blocknorm_desc;

/* Forward:
 *   n = N(block) gamma_post + beta_post  (post)  or  block
 *   s = round(residual_scale x + g n),  g = 1, the column's gate or sigmoid(z)
 *   y = N(s) gamma + beta
 * N(a) = (a - mean) rstd for layer norm, as zero_shard_layernorm; for RMS norm
 * N(a) = a rstd, rstd = 1 / sqrt(sum_c a^2 / cols + eps).  Gains and biases may each be
 * NULL (1 and 0; gamma_post and beta_post have to be without post), gate is NULL iff
 * the descriptor has none.  s is stored to sum.  stats (may be NULL when no
 * backward pass follows): fp32[4][rows] (layer) or fp32[2][rows] (RMS), the rows'
 * rstd of the first norm, rstd of the second, mean of the first, mean of the
 * second; those of the first are not written without post.
 * block and sum may both be NULL: then s = x and y = N(x) gamma + beta, with post 0,
 * no gate and residual_scale 1.
 * An infinity or NaN stays in its row: a layer norm's row is NaN, an RMS norm's
 * too for a NaN; where an RMS norm's sum of squares is beyond binary32, rstd is 0
 * (an infinity itself gives NaN).  A row of zeros gives beta (eps > 0).
 * sum may be x's or block's own buffer with the same row stride, y may be
 * x's, block's or z's unless sum is; otherwise outputs overlap nothing.
 * Errors: ZS_EINVAL, ZS_EALIGN (a pointer not aligned to its element),
 * ZS_EDEVICE, ZS_EHIP. */
int zero_shard_blocknorm(const zs_blocknorm_desc *d, const void *x, const void *block,
                         const void *gate, const void *gamma_post, const void *beta_post,
                         const void *gamma, const void *beta, void *sum, void *y, float *stats);

/* Bytes of workspace that zero_shard_blocknorm_bwd needs for d when a gradient of
 * columns is asked for, or -1 for an invalid descriptor. */
int64_t zero_shard_blocknorm_workspace(const zs_blocknorm_desc *d);

/* Backward, from dy and dsum (the gradient that reaches sum from elsewhere; may
 * be NULL), with the forward pass's sum, block and stats.  h0, h1: N(block) (block
 * itself without post) and N(sum):
 *   D = N'(dy gamma) + dsum;  dx = residual_scale D;  dn = g D
 *   dblock = N'(dn gamma_post)  (post)  or  dn
 *   N'(u) = rstd (u - sum_c u / cols - h sum_c (u h) / cols), RMS without the first sum
 *   dgamma = sum_rows dy h1;  dbeta = sum_rows dy
 *   dgamma_post = sum_rows dn h0;  dbeta_post = sum_rows dn
 *   dgate = sum_rows D n  (column)  or the gradient of z, D n g (1 - g)
 * The five parameters' gradients may each be NULL (not computed; those of what the
 * descriptor lacks have to be); they are written, not added to.  Without a block
 * (as in the forward pass) sum is x and dblock is NULL.  Of no rows the columns'
 * gradients are zeros.
 * dx and dblock may each be dy's, dsum's, sum's or block's own buffer with the same
 * row stride, and dgate z's; otherwise outputs overlap nothing.  workspace: device,
 * 16-byte aligned, at least zero_shard_blocknorm_workspace(d) bytes (may be NULL when
 * no gradient of columns is asked for).
 * Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_blocknorm_bwd(const zs_blocknorm_desc *d, const void *dy, const void *dsum,
                             const void *sum, const void *block, const void *gate,
                             const void *gamma_post, const void *beta_post, const void *gamma,
                             const float *stats, void *dx, void *dblock, void *dgate,
                             void *dgamma_post, void *dbeta_post, void *dgamma, void *dbeta,
                             void *workspace, int64_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * The embedding of tokens, and the gradient of its table.  No handle; launches
 * only, as for layer norm.  The table may be a rank's part of a larger one: its
 * rows stand for the ids first, first + 1, ..; other ids (negative ones too)
 * belong to other ranks, give rows of zeros and no gradient, so that the ranks'
 * outputs add up to the whole table's. */
#define ZS_EMBEDDING_MAX_TOKENS (INT64_C(1) << 27)
#define ZS_EMBEDDING_MAX_VOCAB (INT64_C(1) << 30)
typedef struct zs_embedding_desc {
  int64_t tokens;      /* 0 .. ZS_EMBEDDING_MAX_TOKENS; below 2^34 elements,
                          with cols counted as the multiple of 8 from it on    */
  int64_t vocab;       /* rows of the table, 1 .. ZS_EMBEDDING_MAX_VOCAB;
                          vocab * cols <= 2^37                                */
  int64_t cols;        /* 1 .. 2^20                                           */
  int64_t first;       /* the id of the table's first row; the last row's has to fit */
  int64_t padding;     /* an id whose tokens give no gradient                 */
  int32_t pad_set;     /* 1: padding counts; 0: there is none                 */
  int32_t id_bytes;    /* 4 or 8: ids are int32_t or int64_t                  */
  int32_t dtype;       /* zs_dtype of y and dy                                */
  int32_t table_dtype; /* of table: ZS_F32 or dtype                           */
  int32_t grad_dtype;  /* of dtable: ZS_F32 or dtype                          */
  int32_t accumulate;  /* 1: dtable is added to; 0: it is written             */
  float scale;         /* finite                                              */
  int64_t ld_table, ld_y, ld_dy, ld_dtable; /* row strides in elements (0: cols) */
  void *stream;        /* hipStream_t, NULL = null stream                     */
} zs_embedding_desc;

/* y[t] = scale table[ids[t] - first] (binary32, rounded once), zeros where that is
 * no row of the table.  ids: tokens of them; table: vocab x cols; y: tokens x
 * cols, overlapping nothing.  Errors: ZS_EINVAL, ZS_EALIGN (a pointer not aligned to
 * its element), ZS_EDEVICE, ZS_EHIP. */
int zero_shard_embedding(const zs_embedding_desc *d, const void *ids, const void *table, void *y);

/* Bytes of workspace that zero_shard_embedding_bwd needs for d, or -1 for an
 * invalid descriptor. */
int64_t zero_shard_embedding_workspace(const zs_embedding_desc *d);

/* dtable[v] = scale sum dy[t] over the tokens t of row v, in binary32 and in the
 * order of t: runs of 32 tokens of the row each (8 up to 2048 tokens in all), the runs
 * then in order (four stretches of runs side by side); rounded once.  accumulate:
 * dtable[v] + that, rounded once; rows without tokens are left as they are.  Otherwise
 * they become zeros.
 * dtable overlaps nothing; workspace: device, 256-byte aligned, at least
 * zero_shard_embedding_workspace(d) bytes (NULL where that is 0).  Errors: as above. */
int zero_shard_embedding_bwd(const zs_embedding_desc *d, const void *ids, const void *dy,
                             void *dtable, void *workspace, int64_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * AdamW over many tensors at once: what Muon leaves, or whole models.  Each
 * tensor has its own length, weight decay and learning-rate factor, gradients of
 * its own type, and moments in 32 or in 8 bits.  One launch takes up to 440
 * tensors of a kind of moments (further ones follow in launches of their own).
 *
 * A plan of the tensors is filled on the host, and copied to device memory by the
 * caller, once; the calls take both copies.  They queue kernel launches only, so
 * they can be captured in a HIP graph (with the gradients' addresses of the
 * capture).  Calls of one plan must not overlap.  Same inputs => same bits.
 *
 * Arithmetic, element i of a tensor, gradient g:
 *   g'  = coef g, coef as in zero_shard_step (1 without clipping)
 *   m'  = b1 m + (1-b1) g'      v' = b2 v + (1-b2) g'^2
 *   theta' = theta - (lr f wd) theta - lr f (m'/bc1) / (sqrt(v'/bc2) + eps)
 * with the tensor's lr_scale f and weight_decay wd, in binary64 from the stored
 * values, each result rounded once to binary32: with n_d = 1 and a bf16
 * gradient whose values are the averages, zero_shard_step's bits.
 *
 * ZS_STATE_8: m and r = sqrt(v) are each an e4m3 number (sign, 4 bits of exponent with
 * bias 7, 3 of mantissa; no infinities) times the scale of its block, the
 * tensor's elements [256 b, 256 b + 256).  Their moments are binary32 throughout (with
 * coef, b, 1-b and 1/sqrt(bc2) rounded to it), every operation rounded (u's quotient
 * within two steps of binary32):
 *   m' = b1 m + (1-b1) g'      r' = sqrt((b2 r) r + ((1-b2) g') g')
 *   u = m' / (r' / sqrt(bc2) + eps)
 *   theta' = theta - (lr f wd) theta - (lr f / bc1) u   (binary64, rounded once)
 * (b2 and 1-b2 times 2^32 there, the root times 2^-16, so that an r' from 2^48 on is an
 * infinity and one below 2^-91 a zero).
 * Storing values x of a block (of m', or of r'):
 *   top = max |x|;  scale = top / 256
 *   y = |x| binary32(1 / scale), at most 256, and at least 2^-9 for an r' > 0, becomes
 *   an e4m3 number (with x's sign, a zero's too) by chance, the one below or above it
 *   in proportion to how near each is: above where the 2^20ths of its way from the one
 *   below to the one above, cut to a whole number, plus 16 d + 8 reach 2^20.  d is 16
 *   bits of h (the lower ones for m, the upper ones for r):
 *   h = mix(mix(key + c (k + 1)) + c mix(i >> 32) + i), modulo 2^32, k the tensor's number,
 *   c = 0x9e3779b9, mix(x): x ^= x >> 16; x *= 0x6a09e667; x ^= x >> 15;
 *   x *= 0xbb67ae85; x ^= x >> 16
 * so that the average of what is stored is what was computed: to nearest, a moment
 * whose step is below half a step of the type (v's, with beta2 = 0.999) would never
 * move.  top < 2^-100: the block is zeros.  A block that holds an infinity or NaN
 * has no finite scale from then on.  All zeros are the state at the start. */
#define ZS_ADAMW_BLOCK 256
#define ZS_ADAMW_MAX_TENSORS (INT64_C(1) << 20)
#define ZS_ADAMW_MAX_ELEMENTS (INT64_C(1) << 33) /* of a tensor; of all, 2^24 - 1
                                     chunks of 1024 (32 bits) or 2048 (8) */
typedef enum zs_state { ZS_STATE_32 = 0, ZS_STATE_8 = 1 } zs_state;

/* A tensor.  All arrays are flat and contiguous, aligned to their elements; *_out
 * may be the *_in of the same tensor, otherwise outputs overlap nothing (a plan whose
 * outputs overlap each other is refused). */
typedef struct zs_adamw_tensor {
  int64_t n;                 /* elements, >= 0                                */
  const float *master_in;    /* fp32[n]                                       */
  float *master_out;
  const void *m_in, *v_in;   /* fp32[n], or e4m3 bytes [n] of m and sqrt(v)   */
  void *m_out, *v_out;
  const float *m_scale_in, *v_scale_in; /* fp32[ceil(n / 256)], 8 bits only:  */
  float *m_scale_out, *v_scale_out;     /* NULL with 32                       */
  void *param_out;           /* NULL, or the 16-bit copy of the new weights   */
  float weight_decay, lr_scale; /* >= 0                                       */
  int32_t state;             /* zs_state                                      */
  int32_t grad_dtype;        /* zs_dtype of its gradient                      */
  int32_t param_dtype;       /* of param_out: ZS_BF16 or ZS_F16               */
} zs_adamw_tensor;

typedef struct zs_adamw_desc {
  int64_t count;             /* tensors, 0 .. ZS_ADAMW_MAX_TENSORS            */
  float beta1, beta2, eps;   /* as in zs_desc                                 */
  int32_t bias_correction;   /* 0 or 1                                        */
  float max_norm;            /* > 0: clip by the global norm; <= 0: no        */
  void *stream;              /* hipStream_t, NULL = null stream               */
} zs_adamw_desc;

/* Bytes of a plan of d->count tensors (a HOST array), or -1 where a count or a
 * length is out of range (or all of them together). */
int64_t zero_shard_adamw_plan_bytes(const zs_adamw_desc *d, const zs_adamw_tensor *tensors);

/* Fill a plan (HOST memory, 16-byte aligned).  The caller then copies it to
 * device memory, 256-byte aligned, plan_bytes long, and keeps both for the calls
 * below; the device copy also holds the norm's partial sums.  Tensors keep the
 * addresses given here.  Errors: ZS_EINVAL, ZS_EALIGN, ZS_ENOMEM. */
int zero_shard_adamw_plan(const zs_adamw_desc *d, const zs_adamw_tensor *tensors, void *plan,
                          int64_t plan_bytes);

/* The sum of squares of all gradients (binary64, a fixed order), to *sumsq_dev
 * (device).  grads: HOST array of count device pointers, aligned to their elements
 * (NULL for an empty tensor).  Summed over ranks whose tensors differ it is the step's
 * global_sumsq_dev.  Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_adamw_gnorm(const zs_adamw_desc *d, const void *plan, void *plan_dev,
                           const void *const *grads, double *sumsq_dev);

/* The step t >= 1 at learning rate lr >= 0.  key: any number, another one each step
 * (the step's own will do); it is used by 8-bit states only.  global_sumsq_dev: iff
 * max_norm > 0.  Errors: ZS_EINVAL, ZS_EALIGN, ZS_EDEVICE, ZS_EHIP. */
int zero_shard_adamw(const zs_adamw_desc *d, const void *plan, void *plan_dev,
                     const void *const *grads, float lr, int64_t t, uint32_t key,
                     const double *global_sumsq_dev);

/* The step with its constants read on the device when the kernel runs, so that a
 * captured step serves every step: consts_dev (device, 4 doubles, 8-byte aligned) as
 * zero_shard_adamw_consts writes them (HOST): lr, bc1, bc2, key.  They are trusted as
 * given.  Errors: as above. */
int zero_shard_adamw_consts(const zs_adamw_desc *d, float lr, int64_t t, uint32_t key,
                            double *out);
int zero_shard_adamw_dev(const zs_adamw_desc *d, const void *plan, void *plan_dev,
                         const void *const *grads, const double *consts_dev,
                         const double *global_sumsq_dev);

/* Wait for the handle's stream, release its scratch and the handle.
 * Passing NULL is a no-op returning ZS_OK. */
int zero_shard_free(zs_handle *h);

/* Static description of a status code (never NULL). */
const char *zero_shard_strerror(int code);

/* Length of partition r of phi parameters over n_d ranks (the geometry
 * zero_shard_init checks), or -1 for invalid arguments. */
int64_t zero_shard_len(int64_t phi, int32_t n_d, int32_t r);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_SHARD_H */
