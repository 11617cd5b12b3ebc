/*
 * signmuon_layers.h -- C ABI of libsignmuon.so, continued: the parts of a
 * training pass over M workers' rows that are not weight products, on the
 * flat W and the per-worker flat G[m] of a signmuon_t handle.
 *
 * One backward pass over the joined batch of M workers gives one gradient;
 * the step needs M.  These calls keep what belongs to a worker apart: rows
 * (tokens) are joined in worker order, and the gradients of an embedding table
 * and of a layer norm's weights come out in every G[m] at their place in the
 * flat vector, as signmuon_step reads them; the loss comes out per worker.
 *
 * Conventions, besides those of signmuon.h
 *   - `mat` is the index of one of the handle's matrices (the order of
 *     `shapes` at signmuon_init).  Vote-only handles may make these calls.
 *   - Activations (X, Y, dY, ...) are device matrices of `type` elements with
 *     a row stride of ld >= cols elements; their pointers need the alignment
 *     of one element.  Rows and W/G offsets that allow 16-byte accesses take a
 *     faster path.  Results are computed in fp32 and rounded once.
 *   - rows is a host array of M row counts (>= 0): worker m's rows follow
 *     worker m-1's.  Rows behind the last one are neither read nor written.
 *   - No call waits or allocates, except signmuon_layers_reserve and
 *     signmuon_layers_sync; the others can be captured into a CUDA graph on
 *     the handle's stream (row counts and scalars are then fixed).
 *   - The calls use one workspace per handle: calls, and replays of graphs
 *     that hold them, must not overlap each other on different streams.
 *   - Sums have a fixed order: equal inputs give equal bits.
 *   - The M vectors of G are written by these calls and must not overlap.
 *   - Outputs must not overlap inputs, except where a call says so.
 */
#ifndef SIGNMUON_LAYERS_H
#define SIGNMUON_LAYERS_H

#include "signmuon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of activations */
#define SIGNMUON_F32  0
#define SIGNMUON_BF16 1
#define SIGNMUON_F16  2
/* index types */
#define SIGNMUON_I32  0
#define SIGNMUON_I64  1

/* limits: E_UNSUPPORTED beyond them */
#define SIGNMUON_LAYERNORM_MAX_COLS 16384
#define SIGNMUON_DISTILL_MAX_K      1024

/* ------------------------------------------------------------------------
 * signmuon_layers_reserve -- allocate the workspace of the calls below for up
 * to max_rows rows (all workers together) and embedding / layer norm rows of
 * up to max_cols entries.  Call it once after signmuon_init; a later call
 * with larger sizes allocates a larger workspace and keeps the old one until
 * signmuon_destroy (graphs captured before stay valid).  Waits for the
 * handle's stream; not during capture.  1 <= max_rows, max_cols <= 2^30.
 * Errors: E_INVALID, E_NOMEM, E_CUDA.  The calls below return E_UNSUPPORTED
 * before it, and E_INVALID where they need more than was reserved.
 * ---------------------------------------------------------------------- */
int signmuon_layers_reserve(signmuon_t h, int64_t max_rows, int64_t max_cols);

/* ------------------------------------------------------------------------
 * signmuon_layers_sync -- wait for the handle's stream and report the calls
 * since the last one: E_INVALID when an index was at or above the number of
 * rows or columns it points into (such an index counts as absent, like a
 * negative one), E_CUDA when the device failed, else OK.
 * ---------------------------------------------------------------------- */
int signmuon_layers_sync(signmuon_t h);

/* ------------------------------------------------------------------------
 * signmuon_embed -- out[r] = scale * W[mat][ids[r]], r < n.
 *   W     device float[d].   mat: a V x E table.
 *   ids   device int32/int64[n]; a negative id (padding) gives a row of zeros.
 *   out   n x E, row stride ld.  0 <= n <= 2^30, E <= 2^30.
 * ---------------------------------------------------------------------- */
int signmuon_embed(signmuon_t h, const float* W, int mat, const void* ids, int id_type, int64_t n,
                   float scale, void* out, int type, int64_t ld);

/* ------------------------------------------------------------------------
 * signmuon_embed_grad -- the table's gradient, per worker:
 *   G[m][mat][v] = scale * sum of dY[r] over worker m's rows with ids[r] = v,
 * zero where there are none.  With accumulate, the sum is added to what
 * G[m][mat] holds (a tied table's gradient from elsewhere) and rows without
 * tokens are not touched.  Rows of dY with a negative id are not read.
 *   G     host array of M device pointers, float[d], 16-byte aligned.
 * The tokens are sorted by id, so a row's sum is made in registers over its
 * tokens in order, without floating-point atomics.
 * ---------------------------------------------------------------------- */
int signmuon_embed_grad(signmuon_t h, int mat, const void* ids, int id_type, const int64_t* rows,
                        float scale, const void* dY, int type, int64_t ld, float* const* G,
                        int accumulate);

/* ------------------------------------------------------------------------
 * signmuon_layernorm -- Y = (X - mean) * rstd * gamma + beta per row, with
 * mean = sum X / E and rstd = 1 / sqrt(sum (X - mean)^2 / E + eps).
 *   gamma, beta  matrices with E = rows*cols entries each; beta = -1: none.
 *   n, X, Y      n x E, row strides ldx, ldy, both of `type`; 0 <= n <= 2^30.
 *   mean, rstd   device float[n], what signmuon_layernorm_grad reads; may be
 *                NULL (both).
 * eps > 0.  The statistics are held in fp32; the variance is summed around
 * the mean.  E <= SIGNMUON_LAYERNORM_MAX_COLS (E_UNSUPPORTED).
 * ---------------------------------------------------------------------- */
int signmuon_layernorm(signmuon_t h, const float* W, int gamma, int beta, int64_t n, const void* X,
                       int64_t ldx, void* Y, int64_t ldy, int type, float eps, float* mean,
                       float* rstd);

/* ------------------------------------------------------------------------
 * signmuon_layernorm_grad -- with xh = (X - mean) * rstd and g = dY * gamma:
 *   dX = rstd * (g - mean_E(g) - xh * mean_E(g * xh)),
 *   G[m][gamma] = sum over worker m's rows of dY * xh,
 *   G[m][beta]  = sum over worker m's rows of dY  (beta = -1: none),
 * zero for a worker without rows; with accumulate the sums are added to G.
 *   dX may be dY itself (same pointer and row stride).
 * ---------------------------------------------------------------------- */
int signmuon_layernorm_grad(signmuon_t h, const float* W, int gamma, int beta, const int64_t* rows,
                            const void* X, int64_t ldx, const void* dY, int64_t ldy,
                            const float* mean, const float* rstd, void* dX, int64_t ldd, int type,
                            float* const* G, int accumulate);

/* ------------------------------------------------------------------------
 * signmuon_distill -- distillation from a teacher's top logits: loss per
 * worker and, unless dZ is NULL, the gradient of the sum of the workers'
 * losses with respect to the student's logits, times gscale.
 * Row r has student logits Z[r] (V of them) and up to K teacher entries
 * (idx, t); an entry counts when 0 <= idx < V and t > -inf (or NaN).  With
 * q = softmax of t/T over the row's entries and p = softmax(Z[r]/T):
 *   row_loss[r] = T^2 * sum_k q_k (log q_k - log p[idx_k]),
 *   loss[m] = sum over worker m's rows / count[m],
 *   dZ[r][v] = gscale * T / count[m] * (p[v] - sum of q_k with idx_k = v),
 * count[m] the worker's rows with at least one entry.  A row without entries
 * has loss 0 and a gradient of zeros, whatever its logits hold; a worker
 * without rows that count has loss 0.  Entries with the same idx add up.  K = 1 is
 * the cross-entropy with the label idx (for T = 1).  A logit of -inf is a
 * masked entry (p = 0); a row whose logits are all -inf gives NaN.
 *   Z      rows x V of `type`, row stride ldz.
 *   idx, t rows x K, row stride ldt both; t of t_type.
 *   loss   device float[M].  count: device int32[M], may be NULL.
 *   row_loss  device float[rows], may be NULL.
 *   dZ     rows x V of `type`, row stride ldd; may be Z itself (same pointer
 *          and row stride).
 * Masks may be any finite value too: p is 0 where it is below 2^-126.  Rows whose
 * largest logit is beyond about 1.1e7 temperature, on either side of zero, take
 * longer (their logits are read once more, one by one).
 * 1e-18 <= temperature <= 1e18, 1 <= V <= 2^30, 1 <= K; K <= SIGNMUON_DISTILL_MAX_K
 * (E_UNSUPPORTED).
 * ---------------------------------------------------------------------- */
int signmuon_distill(signmuon_t h, const void* Z, int type, int64_t ldz, int64_t V, const void* idx,
                     int id_type, const void* t, int t_type, int64_t ldt, int K,
                     const int64_t* rows, float temperature, float gscale, float* loss,
                     int32_t* count, float* row_loss, void* dZ, int64_t ldd);

#ifdef __cplusplus
}
#endif
#endif /* SIGNMUON_LAYERS_H */
