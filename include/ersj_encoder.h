/*
 * ersj_encoder.h -- operators of the encoder whose vectors the join compares,
 * on AMD Instinct MI355X (gfx950).  Part of libersj.so.
 *
 * A token-table encoder looks the tokens of a text up in a table of rows,
 * normalises them and pools them into the vector that ersj_build_index then
 * indexes.  These entry points are that encoder's forward and backward
 * passes: token embedding with scaling and its gradient, layer norm and its
 * gradient, and the clipping of all gradients by their global norm.
 *
 * Conventions are those of ersj.h (device pointers, streams, error codes,
 * ersj_last_error, arguments validated before any HIP call), and further:
 *  - No call waits for the device, allocates device memory or copies to the
 *    host, except ersj_grads_create and ersj_grads_free.  Every call can be
 *    captured into a graph, those two excepted.  Host arrays are read before
 *    the call returns.
 *  - Working memory is the caller's (d_work); its contents need no
 *    preparation and mean nothing afterwards.  Calls that overlap in time
 *    need one each.
 *  - Element types are ERSJ_F32, ERSJ_F16 and ERSJ_BF16.  All arithmetic is
 *    in 32 bits or more; a result is rounded to its type once, to nearest.
 *  - Rows may be spaced by more than their length (ld* counts elements) and
 *    start at any multiple of the element size.
 *  - An output may lie on an input only where its entry says so.  Overlaps are
 *    looked for among the tensors of a set of gradients alone.
 *  - The same inputs give the same bits on every call: sums are taken in a
 *    fixed order.  It depends on the sizes and element types; for the gradient
 *    of a table on the ids as well; for the global norm on where each tensor
 *    lies, modulo 128 bytes.
 */
#ifndef ERSJ_ENCODER_H
#define ERSJ_ENCODER_H

#include "ersj.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { ERSJ_F32 = 0, ERSJ_F16 = 1, ERSJ_BF16 = 2 }; /* element types */
enum { ERSJ_I32 = 0, ERSJ_I64 = 1 };                /* token id types */

#define ERSJ_ENCODER_MAX_DIM 65536

/*
 * Token embedding: out[t, :] = scale * table[ids[t], :].
 *  d_table    : device [rows][ld_table] of table_type; 1 <= rows < 2^31 - 1.
 *  dim        : 1 <= dim <= ERSJ_ENCODER_MAX_DIM; ld_table, ld_out >= dim.
 *  d_ids      : device [n] of id_type; 0 <= n < 2^31.
 *  padding_id : tokens with this id get a row of zeros (-1: none have).  Any
 *               other id outside [0, rows) gets a row of NaN; no memory
 *               outside the table is read for it.
 *  d_out      : device [n][ld_out] of out_type: table_type, or any type
 *               where the table is ERSJ_F32.
 * Errors: INVALID_ARG, HIP.
 */
int ersj_embed(const void *d_table, int32_t table_type, int64_t rows, int32_t dim, int64_t ld_table,
               const void *d_ids, int32_t id_type, int64_t n, float scale, int64_t padding_id, void *d_out,
               int32_t out_type, int64_t ld_out, void *stream);

/*
 * Gradient of the table:
 *   out[v, :] = scale * sum over t with ids[t] = v of grad[t, :].
 * Tokens with the padding id, or with an id outside [0, rows), add nothing.
 * Each row's terms are added in 32 bits in an order that the ids and sizes
 * determine: a row's tokens side by side, in the order of t, in stretches
 * whose sums are then added.
 *  d_grad     : device [n][ld_grad] of grad_type.
 *  d_out      : device [rows][ld_out] of out_type: grad_type, or ERSJ_F32.
 *               Every row is written; a row without tokens gets zeros, also
 *               where the scale is infinite or NaN.
 *  accumulate : nonzero: add the sums to out instead (rows without tokens
 *               are left alone); the addition is made in 32 bits and rounded
 *               once.
 *  d_work     : at least ersj_embed_grad_work(n, rows, dim) bytes, aligned
 *               to 256; d_work_bytes is what it holds.
 * Errors: INVALID_ARG, HIP.
 */
int ersj_embed_grad(const void *d_grad, int32_t grad_type, int64_t ld_grad, const void *d_ids, int32_t id_type,
                    int64_t n, float scale, int64_t padding_id, void *d_out, int32_t out_type, int64_t rows,
                    int32_t dim, int64_t ld_out, int32_t accumulate, void *d_work, uint64_t d_work_bytes,
                    void *stream);
/* Bytes of working memory for those sizes (0 also for sizes that are refused,
 * and for few tokens, where none is needed and d_work may be NULL). */
uint64_t ersj_embed_grad_work(int64_t n, int64_t rows, int32_t dim);

/*
 * Layer norm of each row:
 *   mean = sum x / dim,  rstd = 1 / sqrt(sum (x - mean)^2 / dim + eps),
 *   y = (x - mean) * rstd * weight + bias.
 *  d_x, d_y        : device [n][ld_*] of type; 0 <= n < 2^31.  d_y may be d_x
 *                    (with ld_y = ld_x).
 *  d_weight, d_bias: device [dim] of param_type (type or ERSJ_F32); NULL: 1
 *                    and 0.
 *  eps             : finite, >= 0 (with 0, a row of one value gives NaN).
 *  d_mean, d_rstd  : device [n] float; NULL where not wanted.
 * Errors: INVALID_ARG, HIP.
 */
int ersj_layer_norm(const void *d_x, int32_t type, int64_t n, int32_t dim, int64_t ld_x, const void *d_weight,
                    const void *d_bias, int32_t param_type, float eps, void *d_y, int64_t ld_y, float *d_mean,
                    float *d_rstd, void *stream);

/*
 * Gradient of layer norm, with xh = (x - mean) * rstd and g = grad_y * weight:
 *   grad_x      = rstd * (g - sum g / dim - xh * sum (g xh) / dim)
 *   grad_weight = sum over rows of grad_y * xh
 *   grad_bias   = sum over rows of grad_y
 *  d_grad_y, d_x   : device [n][ld_*] of type.
 *  d_mean, d_rstd  : device [n] float, as ersj_layer_norm wrote them.
 *  d_weight        : device [dim] of param_type, NULL: 1.
 *  d_grad_x        : device [n][ld_grad_x] of type; NULL: not wanted.  It may
 *                    be d_grad_y or d_x (with the same spacing).
 *  d_grad_weight, d_grad_bias : device [dim] of param_type; NULL: not wanted.
 *  d_work          : at least ersj_layer_norm_grad_work(n, dim) bytes,
 *                    aligned to 256; not used (NULL) where neither of these
 *                    two gradients is wanted.
 * Errors: INVALID_ARG, HIP.
 */
int ersj_layer_norm_grad(const void *d_grad_y, int64_t ld_grad_y, const void *d_x, int64_t ld_x, int32_t type,
                         int64_t n, int32_t dim, const float *d_mean, const float *d_rstd, const void *d_weight,
                         int32_t param_type, void *d_grad_x, int64_t ld_grad_x, void *d_grad_weight,
                         void *d_grad_bias, void *d_work, uint64_t d_work_bytes, void *stream);
/* Bytes of working memory for those sizes (0 also for sizes that are refused,
 * and for few rows, where none is needed and d_work may be NULL). */
uint64_t ersj_layer_norm_grad_work(int64_t n, int32_t dim);

/*
 * A set of gradient tensors, for clipping by their global norm.  The handle
 * holds a device table of the tensors' addresses and sizes, never their
 * values; the tensors have to outlive it.
 *  count  : 1 <= count <= 65536 tensors.
 *  d_grad : host array [count] of device pointers (NULL where size is 0).
 *  d_out  : host array [count] of device pointers for the clipped tensors, or
 *           NULL to clip in place.  A tensor's own entry may equal its
 *           d_grad; otherwise no output may overlap an input or another
 *           output (INVALID_ARG; ersj_grads_create looks for it once it knows
 *           its device, all other arguments are checked before).
 *  size   : host array [count], elements of each tensor, >= 0, contiguous.
 *  type   : host array [count], ERSJ_F32, ERSJ_F16 or ERSJ_BF16; input and
 *           output have the same type.
 * For tensors that are clipped many times: the table comes from the library's
 * device memory, and the call waits for its stream, and for the whole device
 * where it takes a table that ersj_grads_free has returned since the last such
 * wait.  For tensors whose addresses change from call to call there is
 * ersj_clip_tensors.  Errors: INVALID_ARG, HIP, OOM.
 */
typedef struct ersj_grads ersj_grads;
int ersj_grads_create(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                      const int32_t *type, void *stream, ersj_grads **out);

/*
 * norm = sqrt(sum of the squares of every element of every tensor), squares
 * and sums in binary64; factor = min(1, max_norm / (norm + 1e-6)); every
 * element is multiplied by the factor (binary64 rounded to 32 bits) in 32
 * bits and rounded once.  A norm of infinity makes the factor 0, with a
 * max_norm of infinity 1; a norm of NaN makes it NaN.
 *  max_norm : >= 0 (+inf: the norm alone is wanted; outputs are copies unless
 *             the norm is NaN).
 *  d_norm   : device float, the norm before clipping; NULL where not wanted.
 *  d_work   : ERSJ_GRADS_WORK bytes, aligned to 8.
 * Calls on one handle write the same outputs and must not overlap in time.
 * Errors: INVALID_ARG, HIP.
 */
#define ERSJ_GRADS_WORK 16384
int ersj_grads_clip(const ersj_grads *h, float max_norm, float *d_norm, void *d_work, uint64_t d_work_bytes,
                    void *stream);

/*
 * ersj_grads_clip of tensors given as to ersj_grads_create, without a handle:
 * the table is made in d_work by kernels that carry the tensors' addresses in
 * their arguments, and nothing is waited for.
 *  d_work   : at least ersj_clip_tensors_work(count, size, type) bytes,
 *             aligned to 8.
 * Errors: INVALID_ARG, HIP, OOM.
 */
int ersj_clip_tensors(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                      const int32_t *type, float max_norm, float *d_norm, void *d_work, uint64_t d_work_bytes,
                      void *stream);
/* Bytes of working memory for tensors of those sizes, wherever they lie (0 for
 * sizes that are refused). */
uint64_t ersj_clip_tensors_work(int32_t count, const int64_t *size, const int32_t *type);

/* Release the handle (NULL is a no-op).  Work enqueued with it may still be
 * running: its memory is kept, as ersj_free keeps an index's, and handed out
 * again only after the device has finished what was enqueued. */
void ersj_grads_free(ersj_grads *h);

#ifdef __cplusplus
}
#endif

#endif /* ERSJ_ENCODER_H */
