/*
 * ob.h — C ABI of the 1-bit Adam compression-phase step on one AMD Instinct
 * MI355X (gfx950).
 *
 * The method: the nubint.ai review of "1-bit Adam: Communication Efficient
 * Large-Scale Training with Adam's Convergence Speed" (Tang, Gan et al.),
 * called "the 1-bit Adam review" in the Source line of each declaration.
 * After a full-precision Adam warmup, Adam's variance is frozen and used as a
 * fixed preconditioner (Abstract; Proposed method, bullet 2), and training
 * continues as momentum SGD whose momentum is exchanged with 1-bit
 * error-compensated compression (One-line summary; Proposed method, bullets
 * 1 and 3).  The review's system exchanges the compressed messages with
 * custom collectives (Proposed method, bullet 4).  Here all W workers'
 * buffers live in one GPU's HBM and the exchange is a local reduction over
 * the W packed messages.  Declared below with their sources as well: the
 * warmup phase and the switch to compression, a partitioned server, a
 * layer-wise trust ratio, and ScaleCom's cyclic local top-k codec.
 *
 * Arithmetic (the pages give no formulas; these are the readings taken):
 *   c1 = fp32(beta1), c2 = fp32(1 - beta1) (complement in double, rounded once)
 *   worker w, element i of tensor t (every fp32 operation rounded once, no FMA):
 *     x        = (c1*m[i] + c2*g_w[i]) + e_w[i]
 *     bit      = x >= 0            (+0 and -0 give 1, NaN gives 0)
 *     s_w,t    = fp32( sqrt( fl64(sum over tensor t of x^2) / n_t ) )
 *     e_w[i]   = bit ? x - s_w,t : x + s_w,t
 *   server:
 *     y        = (sum over w = 0..W-1, ascending, from +0, of (bit_w ? s_w,t : -s_w,t)) / W
 *     z        = y + e_s[i];  bit_s = z >= 0;  s_s,t as above over z
 *     e_s[i]   = bit_s ? z - s_s,t : z + s_s,t
 *   update:
 *     m[i]     = bit_s ? s_s,t : -s_s,t
 *     p[i]     = p[i] - lr * (m[i] / (sqrt(v[i]) + eps))   (correctly rounded sqrt and /)
 *   A tensor holding a non-finite x (or z) gets a NaN scale.
 *
 * Layout.  T tensors with n_t >= 1 elements.  Every flat buffer uses the same
 * padded layout: tensor t occupies elements [off[t], off[t] + n_t) with
 * off[0] = 0 and off[t+1] = off[t] + 64*ceil(n_t/64); N = off[T].  Elements in
 * [off[t] + n_t, off[t+1]) are padding: never read, never written.
 * Per-worker buffers are [W][N] with row stride N.  A packed sign message is
 * uint64 words, Nw = N/64 per worker: word j, bit k holds element 64*j + k;
 * each tensor starts on a word; bits past a tensor's end are written as 0.
 * Scales are fp32: scale_w is [W][T] (row stride T), scale_s is [S]: one
 * per tensor (S = T) unless the server is partitioned (ob_set_server_chunks).
 *
 * Ownership.  The caller owns every buffer passed in: device memory (HBM)
 * pointers, each aligned to 16 bytes.  The library owns only the context and
 * its scratch: a tile table, server-piece tables and partial sums per tile
 * and, for the residual worker pass, per 1024-element chunk (allocated in
 * ob_init), and the CLT-k codec's
 * histograms, candidate lists, masks and per-tile counts (allocated in
 * ob_cltk_configure); ob_destroy frees both.
 *
 * Streams.  Every device call enqueues its kernels on the given stream (a
 * hipStream_t; NULL means the null stream) and returns without waiting.  A
 * context's scratch lives on the device that was current at ob_init: later
 * calls must pass buffers and a stream of that device, with it current.
 * Results are visible to later work on that stream.  Concurrent calls on one
 * context from several host threads, or on several streams at once, race on
 * the context's scratch and are not allowed (but for the calls that fill a
 * gradient row, below, which use none of it).
 *
 * Errors.  Calls return OB_OK or an ob_status code.  Argument errors are
 * detected before anything is enqueued.  A failed launch returns
 * OB_ERR_DEVICE; faults inside a kernel surface at the caller's next
 * synchronization with the stream.
 */
#ifndef OB_H
#define OB_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ob_ctx ob_ctx;

typedef enum {
  OB_OK = 0,
  OB_ERR_INVALID = 1,   /* null pointer, bad count, bad range, non-finite hyper-parameter */
  OB_ERR_ALIGN = 2,     /* a device pointer not aligned to 16 bytes */
  OB_ERR_NOMEM = 3,     /* device or host allocation failed */
  OB_ERR_DEVICE = 4,    /* a HIP runtime call or kernel launch failed */
  OB_ERR_SCRATCH = 5    /* the list needs more than ob_step_residual_noalloc's static scratch */
} ob_status;

typedef enum {
  OB_GRAD_F32 = 0,      /* gradients are IEEE binary32 */
  OB_GRAD_BF16 = 1      /* gradients are bfloat16 (widened exactly to fp32) */
} ob_grad_dtype;

/* Element types of activations and their gradients are ob_grad_dtype codes. */
typedef enum {
  OB_ID_I32 = 0,        /* token ids are int32 */
  OB_ID_I64 = 1         /* token ids are int64 */
} ob_id_dtype;

typedef enum {
  OB_ACT_E4M3 = 0,      /* 8-bit floats: 4 exponent and 3 mantissa bits, no infinities (OCP) */
  OB_ACT_INT8 = 1       /* two's complement integers -127..127 */
} ob_act_format;

typedef enum {
  OB_FN_NONE = 0,
  OB_FN_GELU = 1,       /* x * Phi(x), Phi the normal distribution function */
  OB_FN_GELU_TANH = 2,  /* x * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) / 2 */
  OB_FN_SILU = 3        /* x / (1 + exp(-x)) */
} ob_act_fn;

typedef enum {
  OB_MOMENTS_F32 = 0,   /* Adam's moments as fp32 */
  OB_MOMENTS_8BIT = 1   /* as 8-bit codes with a scale byte for every 64 elements */
} ob_moments;

/* Human-readable name of a status code (static storage; never NULL). */
const char *ob_status_string(int status);

/* Host only (no device access).  Fills elem_off[0..T] with the padded layout
 * described above for numel[0..T-1].  Returns OB_ERR_INVALID if T < 1, a
 * pointer is NULL or some numel[t] is < 1 or > 2^40. */
int ob_layout(int32_t num_tensors, const int64_t *numel, int64_t *elem_off);

/* Source: the 1-bit Adam review, Proposed method, bullets 1 and 2: after the
 * Adam warmup the optimizer is momentum SGD (momentum coefficient beta1)
 * preconditioned by the frozen variance (eps in the denominator).  The flat
 * tensor list and its layout are this library's.
 *
 * Creates a context for T tensors of numel[] elements (host array, copied),
 * 1 <= W <= 4096 simulated workers, gradients of grad_dtype, and the fixed
 * hyper-parameters beta1 (momentum, in [0, 1)) and eps (> 0 also once rounded
 * to fp32, the precision the kernels use it in).  Allocates the
 * context's device scratch on the current HIP device and uploads its tables
 * with synchronous copies.  OB_ERR_INVALID also when a launch over the list
 * would exceed the device's grid limit (2^32 - 1 work-items, i.e. 16,777,215
 * workgroups of 256): the (worker group, tile) grid of 8192-element tiles,
 * the 1024-element chunks of the residual worker pass, or one workgroup per
 * (worker, tensor) for the scales.  OB_ERR_NOMEM when the
 * scratch cannot be allocated.  Blocking calls of this library: ob_init,
 * ob_destroy, ob_set_server_chunks, ob_cltk_configure and ob_profile_read;
 * every other call only enqueues work on the given stream. */
int ob_init(ob_ctx **out, int32_t num_tensors, const int64_t *numel, int32_t num_workers,
            int32_t grad_dtype, double beta1, double eps);

/* Frees the context and its scratch (waits for the device as hipFree does).
 * NULL is ignored. */
void ob_destroy(ob_ctx *ctx);

/* Source: the 1-bit Adam review, Proposed method, bullet 3 (error-compensated
 * compression applied to the momentum, not the gradient), Abstract (error
 * compensation keeps convergence robust under 1-bit compression) and One-line
 * summary (1-bit compression).  The scale ||x||_2/sqrt(n) and the bit layout
 * are readings: the pages give no formula.
 *
 * Workers [w_begin, w_end) ⊆ [0, W): momentum, error feedback, 1-bit
 * compression and the new worker error.
 *   grads    [W][N] grad_dtype, read (rows w_begin..w_end-1)
 *   m        [N]    fp32, read (the shared momentum)
 *   err_w    [W][N] fp32, read and overwritten with the new errors
 *   packed_w [W][Nw] uint64, written (the messages)
 *   scale_w  [W][T] fp32, written */
int ob_compress_worker(ob_ctx *ctx, int32_t w_begin, int32_t w_end, const void *grads,
                       const float *m, float *err_w, uint64_t *packed_w, float *scale_w,
                       void *stream);

/* Source: the 1-bit Adam review, Proposed method, bullet 4 (the compressed
 * messages are exchanged through custom collectives).  The pages describe the
 * collective only in prose; a server that averages the W decompressed messages
 * and re-compresses the average with its own error buffer is the reading
 * taken, and here the exchange is a local reduction in one GPU's memory.
 *
 * Server: decompress and average all W messages, add the server error,
 * re-compress, store the new server error.
 *   packed_w [W][Nw], scale_w [W][T] read; err_s [N] read and overwritten;
 *   packed_s [Nw] and scale_s [S] written (the server message; S = T unless the
 *   server is partitioned, see ob_set_server_chunks). */
int ob_server_reduce(ob_ctx *ctx, const uint64_t *packed_w, const float *scale_w,
                     float *err_s, uint64_t *packed_s, float *scale_s, void *stream);

/* Source: the 1-bit Adam review, Abstract (the variance, stable after warmup,
 * is a fixed preconditioner for the rest of training), Proposed method, bullet
 * 2, and One-line summary (preconditioned momentum SGD).  No bias correction,
 * eps outside the root.
 *
 * Update from the server message with the frozen variance:
 *   packed_s [Nw], scale_s [S], v [N] read; m [N] written; params [N] read and
 *   overwritten.  lr must be finite. */
int ob_apply_update(ob_ctx *ctx, const uint64_t *packed_s, const float *scale_s,
                    const float *v, float *m, float *params, double lr, void *stream);

/* Source: the 1-bit Adam review, One-line summary and Proposed method, bullets
 * 1 to 4: one step of the compression phase (compressed momentum, exchange,
 * preconditioned update).
 *
 * One whole compression-phase step: ob_compress_worker over all W workers,
 * ob_server_reduce and ob_apply_update, with the server's second pass and the
 * update fused into one kernel.  Same buffers and results as the three calls
 * in sequence. */
int ob_step(ob_ctx *ctx, const void *grads, float *m, const float *v, float *params,
            float *err_w, float *err_s, uint64_t *packed_w, float *scale_w,
            uint64_t *packed_s, float *scale_s, double lr, void *stream);

/* Source: as ob_step (the 1-bit Adam review, One-line summary and Proposed
 * method, bullets 1 to 4).  The residual form of the state between steps is
 * this library's: the pages say nothing of what is stored between steps.
 *
 * The same step with the error and momentum state kept in residual form,
 * one pass per phase instead of two.
 *
 * Residual form: err_w[w] holds x_w, the value worker w compressed in the
 * last step, and scale_w its scales; err_s holds z, the value the server
 * compressed, and scale_s / packed_s its scales and message.  The state of
 * the strict form is an exact function of it (see ob_materialize):
 *   e_w = x_w - s_w,t*sign(x_w),  e_s = z - s_s,t*sign(z),  m = s_s,t*sign(z),
 * the same fp32 operations the strict form performs, so both forms follow
 * bit-identical trajectories (the momentum of this phase is the server's
 * 1-bit message, so it needs no separate buffer).
 *
 *   first != 0: err_w, err_s and m hold strict-form errors and momentum (for
 *               example zeros at the start of the compression phase);
 *               packed_s and scale_s are only written.
 *   first == 0: the buffers hold the residual form left by the previous call;
 *               m is not read and may be NULL.
 * On return err_w, err_s, packed_w, scale_w, packed_s and scale_s hold this
 * step's residual form and messages, params is updated, m is untouched. */
int ob_step_residual(ob_ctx *ctx, int32_t first, const void *grads, const float *m,
                     const float *v, float *params, float *err_w, float *err_s,
                     uint64_t *packed_w, float *scale_w, uint64_t *packed_s, float *scale_s,
                     double lr, void *stream);

/* For callers that cannot allocate device memory when they step: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * The same step as ob_step_residual (same arguments, buffers and results),
 * with every per-step scratch buffer -- the per-tile and per-chunk partial
 * sums of squares and the trust ratios -- in one static device array of this
 * library (64 MiB per GPU, held from the library's first use on that GPU
 * until the process ends) instead of the context's scratch.  It allocates
 * nothing: no hipMalloc, hipFree, event creation or allocating library call
 * (so its launches are not timed by ob_profile_*); its device address is
 * looked up once per GPU by ob_init.  A list needs (W+1)*tiles*16 +
 * W*tiles*128 + T*4 bytes of it (tiles = its 8192-element tiles; each of the
 * three sections rounded up to 256 bytes): 48 MB for the BERT-Large-shaped
 * list at W = 8.  A list needing more than 64 MiB returns OB_ERR_SCRATCH
 * before anything is enqueued; OB_ERR_DEVICE if ob_init could not look the
 * array up.  Every context and call on one GPU shares that GPU's array: calls
 * that overlap on one GPU (two streams, two host threads) race on it.  Each
 * call writes every scratch entry before reading it, so nothing is cleared
 * between calls. */
int ob_step_residual_noalloc(ob_ctx *ctx, int32_t first, const void *grads, const float *m,
                             const float *v, float *params, float *err_w, float *err_s,
                             uint64_t *packed_w, float *scale_w, uint64_t *packed_s,
                             float *scale_s, double lr, void *stream);

/* Source: the 1-bit Adam review, Proposed method, bullet 3: the error left by
 * compressing x is x minus its 1-bit reconstruction.
 *
 * Writes the strict-form state of a residual-form state:
 *   err_w [W][N] = x_w - s_w,t*sign(x_w),  err_s [N] = z - s_s,t*sign(z),
 *   m [N] = s_s,t*sign(z).
 * x_w [W][N], scale_w [W][T], z [N], scale_s [S] are read.  Outputs may be
 * the same buffers as the inputs (in place). */
int ob_materialize(ob_ctx *ctx, const float *x_w, const float *scale_w, const float *z,
                   const float *scale_s, float *err_w, float *err_s, float *m, void *stream);

/* Source: the 1-bit Adam review, Proposed method, bullet 1 (full-precision
 * Adam for about the first 20% of steps).
 *
 * Warmup phase: one uncompressed Adam step on the workers' average gradient,
 * the first phase of the method (the review of "1-bit Adam ...", Proposed
 * method, bullet 1: full-precision Adam for about the first 20% of steps,
 * whose variance the compression phase then keeps fixed, bullet 2):
 *   gbar = (sum over w = 0..W-1, ascending, from +0, of g_w[i]) / W
 *   m[i] = c1*m[i] + c2*gbar
 *   v[i] = fp32(beta2)*v[i] + fp32(1 - beta2)*(gbar*gbar)
 *   p[i] = p[i] - lr * (m[i] / (sqrt(v[i]) + eps))      (no bias correction)
 * grads [W][N] read; m, v, params [N] read and overwritten.  beta2 in [0, 1),
 * lr finite. */
int ob_warmup_step(ob_ctx *ctx, const void *grads, float *m, float *v, float *params,
                   double beta2, double lr, void *stream);

/* Source: the 1-bit Adam review, Proposed method, bullet 1 (the warmup is
 * Adam at full precision).  AdamW's form of it (bias correction, decay beside
 * the gradient) and the 8-bit moments are this library's.
 *
 * One AdamW step over the whole list, on the workers' average gradient:
 *   g    = (sum over w = 0..W-1, ascending, from +0, of g_w[i]) / W, times *grad_scale if given
 *   m[i] = c1*m[i] + c2*g;  v[i] = fp32(beta2)*v[i] + fp32(1 - beta2)*(g*g);  r = sqrt(v[i])
 *   p[i] = (p[i] - p[i]*(fp32(lr*weight_decay)*decay[t])) - (m[i] / (r*root + eps))*rate
 * with rate = fp32(lr / (1 - beta1^step)), root = fp32(1 / sqrt(1 - beta2^step)),
 * step >= 1, every fp32 operation rounded once.  decay [T] (device; NULL: 1
 * for every tensor) scales the decay by tensor, *grad_scale (device, one float;
 * NULL: none) all gradients: a clipping factor that the device has computed.
 * With model [N] bf16 not NULL the new parameters are also written there, rounded
 * to nearest even: what ob_linear multiplies with.  grads [W][N] read; m, v
 * [N] and params [N] read and overwritten; lr finite, weight_decay >= 0, beta2 in [0, 1);
 * decay and *grad_scale need their element's alignment only.
 * A captured call keeps its step, lr and seed at every replay: one step's bias correction and,
 * in 8 bits, one dither, over which rounding is not unbiased.  A graph that is replayed as
 * step after step leaves this call outside.
 *
 * moments = OB_MOMENTS_F32: m, v [N] fp32; m_scale and v_scale are NULL.
 * moments = OB_MOMENTS_8BIT: m, v [N] are codes, m_scale, v_scale [N/64] scale
 * bytes: a block of 64 consecutive elements (no block spans two tensors, and
 * padding is no part of one) stands for code * 2^(scale - 127), the scale the
 * smallest, and at least 2^-111, for which the block's largest magnitude fits.  m:
 * e4m3 codes; magnitudes past 1.875 * 2^127 count as that.  v: codes of its root,
 * code 16k + f standing for f if k = 0 and (16 + f)*2^(k-1) otherwise (the
 * largest is 31 * 2^14); v is the square, in fp32.  The step reads these values, computes
 * as above and writes m and r back, rounded with a dither: of h = M(lo(i) ^ (key + hi(i)*0x9E3779B9)),
 * i the element's place in the list, M(x) = x ^= x >> 16, x *= 0x85EBCA6B, x ^= x >> 13, x *=
 * 0xC2B2AE35, x ^= x >> 16 and key = M(lo(seed) ^ M(hi(seed) + 0x9E3779B9)), all modulo 2^32 (lo,
 * hi: the 32-bit halves), the low 16 bits are m's and the high 16 r's.  A magnitude
 * between two codes takes the upper one if its remainder in steps plus the
 * dither / 2^16 reaches 1 (below the smallest normal code the remainder is first rounded
 * to nearest even at 2^-20 of a step, of r 2^-19), so over seeds rounding is unbiased to within
 * 2^-16 of a step (a remainder below that never rounds up): give every step another seed.
 * A root above 0 takes code 1 at least.  A block with a NaN or an infinity has scale 255 and
 * codes 0 and stands for NaN throughout.  Zero-filled buffers stand for zeros: the state to
 * start from.  m_scale and v_scale are aligned to 16 bytes as well. */
int ob_adamw_step(ob_ctx *ctx, int32_t moments, const void *grads, const float *grad_scale, void *m, uint8_t *m_scale,
                  void *v, uint8_t *v_scale, float *params, uint16_t *model, int64_t step, double lr, double beta2,
                  double weight_decay, const float *decay, uint64_t seed, void *stream);

/* The values of 8-bit moments: m_out, v_out [N] of type dtype, written (fp32:
 * exact; what the compression phase starts from).  Padding stays untouched. */
int ob_adamw_load(ob_ctx *ctx, const uint8_t *m, const uint8_t *m_scale, const uint8_t *v, const uint8_t *v_scale,
                  int32_t dtype, void *m_out, void *v_out, void *stream);

/* Source: the 1-bit Adam review, Proposed method, bullets 1 and 2 (the switch
 * to compressed momentum SGD, with the variance kept fixed from then on).
 *
 * The switch from warmup to compression: v is kept as it is from now on
 * (frozen) and the error buffers start from zero.  Writes 0 to every tensor
 * element of err_w [W][N] and err_s [N] (padding untouched).  The next step
 * is ob_step, or ob_step_residual with first != 0. */
int ob_begin_compression(ob_ctx *ctx, float *err_w, float *err_s, void *stream);

/* Source: the 1-bit Adam review, Proposed method, bullet 4 (the custom
 * collective).  One scale per server chunk is the reading for a server role
 * split across ranks; the pages do not say.
 *
 * Partitioned server: when the server role is split C ways, rank j holds
 * chunk j of every tensor and compresses it with its own scale.  Chunk j of
 * an n-element tensor covers elements [j*S_t, min((j+1)*S_t, n)) with
 * S_t = 8192*ceil(ceil(n/8192)/C) (whole 8192-element blocks, so a chunk
 * boundary never splits a sign word); a tensor has ceil(n/S_t) <= C chunks.
 * After this call every server scale (scale_s, the server message) is per
 * chunk, in tensor order then chunk order; ob_server_scale_count gives their
 * number S.  C = 1 (the default) is one scale per tensor; any C at or above
 * a tensor's tile count gives that tensor one scale per 8192-element block.
 * Synchronous: waits for the stream of this context's latest launch (which
 * must still exist), then uploads small tables; if an upload fails it
 * restores the previous setting's tables and returns OB_ERR_DEVICE.  Changes
 * of C between steps also change what scale_s holds, so use it before the
 * first step. */
int ob_set_server_chunks(ob_ctx *ctx, int32_t chunks);
int32_t ob_server_scale_count(const ob_ctx *ctx);

/* Source: the fugumt page on "1-bit LAMB: Communication Efficient Large-Scale
 * Large-Batch Training with LAMB's Convergence Speed", Abstract (LAMB's layer-
 * wise adaptive learning rates kept under 1-bit compression).
 *
 * Layer-wise trust ratio (the fugumt page on "1-bit LAMB": LAMB's layer-wise
 * adaptive learning rates kept under compressed communication; the page gives
 * no formula, this is the plainest reading).  With enable != 0 every update of
 * this context (ob_step, ob_step_residual, ob_apply_update) becomes, per
 * tensor t:
 *   u[i] = m[i] / (sqrt(v[i]) + eps)   (+ fp32(weight_decay) * p[i] if > 0)
 *   r_t  = fp32( sqrt(fl64(sum p^2)) / sqrt(fl64(sum u^2)) ), 1 if a sum is 0
 *   p[i] = p[i] - lr * (r_t * u[i])
 * with the sums exact up to one rounding, as for the scales.  It costs two
 * more launches per step (the ratio needs the whole tensor's update) and one
 * more read of v and params.  weight_decay >= 0 and finite. */
int ob_set_trust_ratio(ob_ctx *ctx, int32_t enable, double weight_decay);

/* Source: the nubint.ai review of "ScaleCom: Scalable Sparsified Gradient
 * Compression for Communication-Efficient Distributed Training", Proposed
 * method, bullet 1 (a cyclically chosen leader's top-k indices shared by all
 * workers) and Main results, bullet 3.
 *
 * Cyclic local top-k (CLT-k), an alternative codec for the exchange: the
 * commutative compressor of the review of "ScaleCom: Scalable Sparsified
 * Gradient Compression for Communication-Efficient Distributed Training"
 * (Proposed method, bullet 1; Main results, bullet 3).  Per tensor t with
 * k_t = max(1, ceil(density * n_t)) entries kept:
 *   x_w     = memory_w + g_w                              (fp32, every worker)
 *   index   = the k_t positions of largest |x_leader|, leader = step mod W,
 *             ties to the lower position, listed in ascending order
 *   values_w = x_w at index;  memory_w = x_w with those positions set to 0
 *   average = (sum over w ascending, from +0, of values_w) / W
 * The page names a low-pass filter on the memory without its form; none is
 * applied.  Inputs must be finite.
 *
 * ob_cltk_configure allocates the codec's scratch for the given density
 * (0 < density <= 1; every n_t at most INT32_MAX, else OB_ERR_INVALID;
 * synchronous: waits for the stream of this context's latest launch, then
 * allocates and uploads) and returns K = sum of k_t; ob_cltk_layout writes the host
 * array k_off[0..T] (tensor t's entries are k_off[t] .. k_off[t+1]-1).
 * ob_cltk_step: grads [W][N] read; memory [W][N] fp32 read and overwritten;
 * index [K] int32 (position within the tensor), values [W][K] fp32 and
 * average [K] fp32 written. */
int ob_cltk_configure(ob_ctx *ctx, double density, int64_t *k_total);
int ob_cltk_layout(const ob_ctx *ctx, int64_t *k_off);
int ob_cltk_step(ob_ctx *ctx, int64_t step, const void *grads, float *memory, int32_t *index,
                 float *values, float *average, void *stream);

/* ------------------------------------------------------------------------
 * What fills a worker's gradient row: embedding lookup and gradient, 8-bit
 * activation checkpoints, and the linear layer: its forward, the gradient to
 * its input, and its weight's gradient from a checkpoint.
 *
 * Matrices are [rows][cols] with a row stride of ld >= cols elements; their
 * pointers need the alignment of their element only (rows that all start on
 * 16 bytes are read and written faster).  params, grads, codes, scales and
 * work are aligned to 16 bytes as everywhere.  The *_grad calls write one
 * tensor's gradient into row `worker` of grads [W][N] (the context's gradient
 * type); padding and all other tensors and rows stay untouched.  With
 * accumulate != 0 they add to what the tensor's gradient holds (in fp32,
 * rounded once), otherwise they overwrite it.  Sums over tokens are fp32, in
 * an order that the sizes, types, ids and, for dy, its row stride and alignment
 * to 16 bytes settle: the same call gives the same bits, one with the same
 * values in a dy of another stride or alignment may not.  A call with no rows (tokens) reads nothing: its matrices and
 * checkpoint may be NULL, and a gradient is written as 0 or left as it was.
 *
 * `work` is the caller's scratch of at least the bytes that the matching
 * *_work call gives (host only; NULL when that is 0): each call writes what it
 * reads there, so it needs no clearing and may be reused by the next call on
 * the stream.  These calls use no scratch of the context: unlike its other
 * calls, those on different streams may overlap, and several host threads may
 * make them on one context at once, as long as their buffers and work do not
 * overlap (the context is neither destroyed nor given another profiling
 * setting meanwhile).  With profiling off they allocate nothing and may be
 * captured into a HIP graph.
 * ------------------------------------------------------------------------ */

/* Source: the jarxiv page on "Activations and Gradients Compression for
 * Model-Parallel Training", Abstract (activations kept or sent in compressed
 * form).  The page gives no format; this one is the library's.
 *
 * 8-bit activation checkpoint of x [rows][cols]: codes [rows][pitch] bytes and
 * scales [ceil(rows/32)][pitch] bytes, pitch = 64*ceil(cols/64).  Element
 * (r, c) stands for code(r, c) * 2^(scales(r/32, c) - 127): 32 consecutive
 * rows of a column share a power-of-two scale, the smallest (and at least
 * 2^-111) for which the block's largest |x| fits the format (448 for e4m3, 127
 * for int8); magnitudes past 1.875 * 2^127 count as that; codes are rounded to
 * nearest even.  A block with a NaN or an
 * infinity has scale byte 255 and stands for NaN throughout.  Every value is
 * exact in bf16.  Bytes cols..pitch-1 of a row are never written and their
 * content never reaches a result.
 *
 * ob_act_layout (host only): the pitch and the two sizes; rows up to 2^31,
 * cols up to 2^30. */
int ob_act_layout(int64_t rows, int64_t cols, int64_t *pitch, int64_t *code_bytes, int64_t *scale_bytes);

/* Writes x's checkpoint and, with fn != OB_FN_NONE, y = fn(x) in the same
 * pass.  x and y have type dtype; y may be x itself (with the same ld),
 * and is NULL with OB_FN_NONE.  In fp32 a value of fn is off by at most 2^-20
 * of itself (16 half steps), and where Phi or sigma is below 2^-126 it may be 0. */
int ob_act_save(int32_t format, int32_t fn, int64_t rows, int64_t cols, int32_t dtype, const void *x, int64_t ldx,
                void *y, int64_t ldy, uint8_t *codes, uint8_t *scales, void *stream);

/* The checkpoint's values; with dtype bf16 or fp32 alike they are exact. */
int ob_act_load(int32_t format, int64_t rows, int64_t cols, const uint8_t *codes, const uint8_t *scales, int32_t dtype,
                void *out, int64_t ldo, void *stream);

/* dx = dy * fn'(checkpoint's values); dx may be dy itself (with the same ld).  fn is
 * not OB_FN_NONE.  In fp32 fn' = F + x*F' is off by at most 2^-19 of the larger
 * of its two terms. */
int ob_act_backward(int32_t format, int32_t fn, int64_t rows, int64_t cols, const uint8_t *codes, const uint8_t *scales,
                    int32_t dtype, const void *dy, int64_t lddy, void *dx, int64_t lddx, void *stream);

/* Gradient of a linear layer y = x W^T + b whose input x [rows][in_features]
 * was kept as a checkpoint:
 *   dW[o][i] = sum over r of dy[r][o] * xhat[r][i],  db[o] = sum over r of dy[r][o]
 * tensor `weight` of the list is W [out_features][in_features], tensor `bias`
 * is b [out_features] (-1: none).  dy is [rows][out_features], fp32 or bf16;
 * products are exact (of an fp32 dy, bits below 2^-133 are dropped) and summed
 * in fp32.  rows and in_features at most 2^24. */
int ob_linear_grad_work(int64_t rows, int64_t out_features, int64_t in_features, int32_t dy_dtype, int32_t bias,
                        int64_t *work_bytes);
int ob_linear_grad(ob_ctx *ctx, int32_t worker, int32_t weight, int32_t bias, int64_t rows, int64_t out_features,
                   int64_t in_features, int32_t format, const uint8_t *codes, const uint8_t *scales, int32_t dy_dtype,
                   const void *dy, int64_t lddy, int32_t accumulate, void *grads, void *work, int64_t work_bytes,
                   void *stream);

/* A linear layer's forward, y = fn(x W^T + b) + residual, with W (tensor
 * `weight`, [out_features][in_features]) and b (tensor `bias`, [out_features]; -1: none)
 * read from a list in the padded layout of list_dtype: params itself, or the bf16 copy
 * that ob_adamw_step writes.
 *   h[t][o] = sum over i of x[t][i] * W[o][i] + b[o];  y[t][o] = fn(h[t][o]) + residual[t][o]
 * x [rows][in_features], residual (NULL: none) and y [rows][out_features] have type dtype;
 * y may be residual (with the same row stride), not x.  With codes and scales not NULL the
 * checkpoint of h (its fp32 values, in the format and layout of ob_act_save) is
 * written in the same pass: what ob_act_backward or ob_linear_input_grad take.
 * Sums are fp32 in an order that the sizes, types and x's row stride and
 * alignment settle; the matrix units may cut, not round, what lies below 2^-24 of an addition's
 * largest term.  Products of bf16 operands are exact; an fp32 operand is cut into three
 * bf16 parts (bits below 2^-133 are dropped), and of two fp32 operands the
 * products of parts below 2^-25 of the whole are left out.  Where an operand is fp32, an infinity
 * in either gives an infinity or NaN where plain arithmetic gives an infinity, by the kernel that
 * the sizes settle, and so may a product or sum within 2^-6 of fp32's largest; never a finite
 * value.  fn as in ob_act_save (gelu_tanh of bf16 results takes fewer operations here, so a
 * result that lies between two of them may round the other way).
 * rows up to 2^24, features up to 2^21, and ceil(rows/128) * ceil(f/128) at most
 * 8,388,607 for the larger f of the two.
 *
 * ob_linear_work (host only): the scratch of a call.  aligned != 0 promises that
 * x (dy) starts on 16 bytes, its row stride is a multiple of 16 bytes and at most
 * 2^21 elements: bf16 matrices that are not get a copy there. */
int ob_linear_work(int64_t rows, int64_t out_features, int64_t in_features, int32_t dtype, int32_t list_dtype,
                   int32_t aligned, int32_t input_grad, int64_t *work_bytes);
int ob_linear(ob_ctx *ctx, int32_t weight, int32_t bias, int64_t rows, int64_t out_features, int64_t in_features,
              int32_t dtype, const void *x, int64_t ldx, int32_t list_dtype, const void *list, int32_t fn, int32_t format,
              uint8_t *codes, uint8_t *scales, const void *residual, int64_t ldr, void *y, int64_t ldy, void *work,
              int64_t work_bytes, void *stream);

/* The gradient to a linear layer's input,
 *   dx[t][i] = (sum over o of dy[t][o] * W[o][i]) * fn'(kept[t][i]) + add[t][i]
 * with kept the values of the checkpoint [rows][in_features] in codes and scales (fn =
 * OB_FN_NONE: no such factor, codes and scales are NULL) and add a gradient that reached
 * the same place another way (NULL: none).  dy [rows][out_features], add and dx
 * [rows][in_features] have type dtype; dx may be add (with the same row stride), not dy.
 * W, sums, products, limits and scratch as for ob_linear (ob_linear_work with
 * input_grad != 0); fn' as in ob_act_backward, with the same remark. */
int ob_linear_input_grad(ob_ctx *ctx, int32_t weight, int64_t rows, int64_t out_features, int64_t in_features,
                         int32_t dtype, const void *dy, int64_t lddy, int32_t list_dtype, const void *list, int32_t fn,
                         int32_t format, const uint8_t *codes, const uint8_t *scales, const void *add, int64_t ldadd,
                         void *dx, int64_t lddx, void *work, int64_t work_bytes, void *stream);

/* Embedding lookup: out[t] = fp32(scale) * E[ids[t]], with tensor `tensor` of
 * params [N] as the table E [numel/dim][dim], and at most 16,777,215 tokens;
 * fp32(scale) is finite.  A negative id is padding and gives a row of zeros;
 * an id past the table gives a row of NaN.  out is [tokens][dim] of out_dtype. */
int ob_embedding_lookup(ob_ctx *ctx, int32_t tensor, int64_t dim, int64_t tokens, const void *ids, int32_t id_dtype,
                        const float *params, double scale, int32_t out_dtype, void *out, int64_t ldo, void *stream);

/* Its gradient: dE[v] = fp32(scale) * (sum over t with ids[t] = v of dy[t]);
 * ids outside the table contribute nothing.  dy is [tokens][dim] of dy_dtype.
 * At most 16,777,215 tokens, 2^31 - 1 rows and 2^30 columns, and
 * ceil(tokens/32) * ceil(dim/64) at most 16,777,215. */
int ob_embedding_grad_work(int64_t tokens, int64_t dim, int64_t *work_bytes);
int ob_embedding_grad(ob_ctx *ctx, int32_t worker, int32_t tensor, int64_t dim, int64_t tokens, const void *ids,
                      int32_t id_dtype, double scale, int32_t dy_dtype, const void *dy, int64_t lddy,
                      int32_t accumulate, void *grads, void *work, int64_t work_bytes, void *stream);

/* Kernel timing for measurement.  With profiling on, every kernel the context
 * launches is bracketed by HIP events on its stream.  ob_profile_read waits for
 * the recorded events, writes per kernel kind the summed milliseconds and the
 * launch count (arrays of ob_profile_kinds() entries), and with reset != 0
 * forgets them.  ob_profile_kind_name names kind k (NULL when out of range). */
int ob_profile_enable(ob_ctx *ctx, int32_t enable);
int32_t ob_profile_kinds(void);
const char *ob_profile_kind_name(int32_t kind);
int ob_profile_read(ob_ctx *ctx, double *total_ms, int64_t *launches, int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* OB_H */
