/*
 * ra_operators.h -- C ABI of the training-step operators of the GB300 ring
 * all-reduce library (libgradient_ring_all.so): the calls that produce the
 * gradients which the ring averages.
 *
 *   ra_embedding_lookup    rows of an embedding table, scaled
 *   ra_embedding_grad      the table's gradient, summed by sorted token
 *   ra_linear              act(x w + bias) + residual on the tensor cores
 *   ra_linear_dgrad        (dy w^T) * act'(z) + residual
 *   ra_linear_wgrad        act(z)^T dy and the column sums of dy
 *   ra_checkpoint8_pack    an activation kept in 8 bits
 *   ra_checkpoint8_unpack  and restored
 *
 * The layers are those of the Transformer whose gradients the library's
 * workloads average ("How GPipe works", section 1: embedding V x d, weights
 * d x h and h x d with biases).  A checkpoint is what section 6 of the same
 * page (re-materialisation) trades for recomputation: the activation that the
 * backward pass needs, here at 33/32 byte a value.
 *
 * Conventions, besides those of ring_allreduce.h (asynchronous on `stream`,
 * arguments checked before anything is queued, the caller owns all device
 * memory, no state kept between calls):
 *   - a matrix is row-major: element (r, c) of `a` at a[r * ld + c], ld >= its
 *     columns; ld is not looked at where there is one row.  Rows and columns
 *     stay below 2^31, byte offsets may be larger.
 *   - an output shares no byte with an input, unless the call says so
 *     (RA_ERR_OVERLAP).  Column slices of one array with one ld may interleave.
 *   - a size of zero is allowed: nothing to write is RA_OK without a launch, an
 *     empty sum is zero.
 *   - results do not change from call to call: every sum is added in an order
 *     that the sizes, the token ids, whether ws has the room that
 *     ra_linear_split_bytes asks for, and the device's number of SMs alone decide.
 *   - NaN and infinities go through by the formulas.
 *   - products are summed in binary32 by the tensor cores, which round toward
 *     zero: a bf16 result over up to 16384 of k may be short by a fifth of half a
 *     bf16 step where all products have one sign, and by far less where they
 *     have not.  Longer sums, and binary32 results, are made in chunks of 512
 *     that are added with rounding to nearest.
 *   - the products' kernels wait for their own copies and tensor-core work with
 *     the library's limit; ra_check_device_errors reports a wait that gave up.
 *     What the blocks concerned would have stored keeps its former value.
 *   - gelu, silu and their slopes are within 2^-20 of |z| (of 1 + |z| for a
 *     slope); far out on gelu's negative side, where the values are that small
 *     themselves, they do not keep their relative accuracy (0.2 % at z = -5).
 *   - a call may be the first to look up a driver entry point, and loads the
 *     kernels it is the first to launch; which these are depends on sizes, types,
 *     row alignment, activation, and whether a checkpoint, a bias gradient and
 *     the room for parts are there.  Before capturing a call, make the same call
 *     once outside any stream capture.
 */
#ifndef RA_OPERATORS_H
#define RA_OPERATORS_H

#include "ring_allreduce.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, computed in binary32:
 *   relu  max(z, 0)
 *   gelu  z * (1 + erf(z / sqrt 2)) / 2
 *   silu  z / (1 + exp(-z)) */
typedef enum { RA_ACT_NONE = 0, RA_ACT_RELU = 1, RA_ACT_GELU = 2, RA_ACT_SILU = 3 } ra_act;

/*
 * An activation of rows x cols in 8 bits.  RA_CHECKPOINT8_GROUP neighbours of
 * a row (the last group of a row may be short) share one step, a power of two;
 * each value is the nearest whole number of steps (ties to even), -127 .. 127:
 *   q  rows * groups * 32 bytes, group g of row r at q + (r * groups + g) * 32,
 *      the short group's rest zero; 16-byte aligned
 *   e  rows * groups bytes; the step is 2^(e - 127)
 * with groups = ceil(cols / 32).  e is 6 below the (biased) exponent of the
 * group's largest magnitude, one more where that would round to 128 steps, and
 * between 1 and 248.  A value is off by at most half a step: 1/127.5 of that
 * magnitude, or 2^-127 where the magnitude is below 2^-120.  Only a group whose
 * largest magnitude is 255 * 2^120 or more, of which a restored value could be
 * infinite, is taken times 127/128: there a value is off by at most 1.5 steps,
 * 1/85 of the magnitude.  A power-of-two step makes every restored value exact
 * in bf16 (and in binary32), so the tensor cores read a checkpoint without a
 * second rounding.
 * A group with an infinity or a NaN is marked (e = 255, q = 0) and reads back as
 * NaN throughout, so that such a value is not lost.
 */
#define RA_CHECKPOINT8_GROUP 32

ra_status ra_checkpoint8_pack(const void *x, int64_t ld, int dtype, int64_t rows, int64_t cols, int8_t *q, uint8_t *e,
                              void *stream);

/* out = act(the values that q and e stand for) in `dtype`. */
ra_status ra_checkpoint8_unpack(const int8_t *q, const uint8_t *e, int64_t rows, int64_t cols, int act, void *out,
                                int64_t ld, int dtype, void *stream);

/*
 * ra_embedding_lookup -- out[t, :] = scale * table[ids[t], :], t in [0, tokens);
 * the binary32 product is rounded to `dtype`.  An id outside [0, vocab) is padding:
 * its row is zero.
 *   table   vocab x d, out  tokens x d, both of `dtype`
 *   ids     tokens integers of id_bytes (4 or 8), contiguous
 */
ra_status ra_embedding_lookup(const void *table, int64_t ld_table, int dtype, int64_t vocab, int64_t d, const void *ids,
                              int id_bytes, int64_t tokens, float scale, void *out, int64_t ld_out, void *stream);

/*
 * ra_embedding_grad -- the gradient of that lookup:
 *   out[v, :] = scale * sum over t with ids[t] = v of grad[t, :]
 * for every v in [0, vocab), zero where no token has id v.  The sum is
 * binary32; it and, with `accumulate`, out's former value are rounded to
 * out_dtype once.  accumulate != 0 adds to out (micro-batches, tied weights)
 * and leaves rows without a token alone.  Ids outside [0, vocab) count for
 * nothing, whatever their rows of grad hold.
 *   ws, ws_bytes  device workspace of at least
 *                 ra_embedding_grad_workspace_bytes(tokens, vocab, d), 16-byte
 *                 aligned
 */
size_t ra_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d);
ra_status ra_embedding_grad(const void *grad, int64_t ld_grad, int grad_dtype, const void *ids, int id_bytes, int64_t tokens,
                            float scale, int accumulate, void *out, int64_t ld_out, int out_dtype, int64_t vocab, int64_t d,
                            void *ws, size_t ws_bytes, void *stream);

/*
 * ra_linear -- y = act(x w + bias) + residual.
 *   x, w      m x k and k x n, bf16; products are summed in binary32
 *   bias      n values of bias_dtype (RA_F32 or RA_BF16), or NULL
 *   residual  m x n of res_dtype, or NULL; may be y itself (same address, ld
 *             and type)
 *   save_q, save_e  NULL, or the 8-bit checkpoint (m x n) that receives
 *             z = x w + bias, for ra_linear_dgrad and ra_linear_wgrad
 *   y         m x n of y_dtype, rounded once
 *   ws        device workspace, 16-byte aligned, for two things:
 *             - ra_linear_workspace_bytes(m, k, n) where x or w does not start on
 *               a 16-byte boundary or its rows are not multiples of 16 bytes
 *               apart: TMA reads others in place, these are laid out first;
 *             - ra_linear_split_bytes(m, n, k) more, by choice: where it is not
 *               0, the last tiles would leave most SMs idle, and with this room
 *               they are made in parts along k (faster; the sums are then
 *               grouped differently, the same way in every such call).
 *             NULL where neither is wanted.
 */
size_t ra_linear_workspace_bytes(int64_t m, int64_t k, int64_t n);
/* for an output of rows x cols summed over k: (m, n, k) for ra_linear, (m, k, n)
 * for ra_linear_dgrad, (k, n, m) for ra_linear_wgrad */
size_t ra_linear_split_bytes(int64_t rows, int64_t cols, int64_t k);
ra_status ra_linear(const void *x, int64_t ld_x, const void *w, int64_t ld_w, int64_t m, int64_t k, int64_t n,
                    const void *bias, int bias_dtype, int act, const void *residual, int64_t ld_res, int res_dtype,
                    int8_t *save_q, uint8_t *save_e, void *y, int64_t ld_y, int y_dtype, void *ws, size_t ws_bytes,
                    void *stream);

/*
 * ra_linear_dgrad -- dx = (dy w^T) * act'(z) + residual: the gradient with
 * respect to the layer's input, carried on through the activation that made
 * that input from z.
 *   dy, w     m x n and k x n, bf16
 *   z_q, z_e  the 8-bit checkpoint of z (m x k); NULL with RA_ACT_NONE
 *   residual  m x k of res_dtype, or NULL; may be dx itself
 *   dx        m x k of dx_dtype, rounded once
 *   ws        as for ra_linear, for dy and w
 */
ra_status ra_linear_dgrad(const void *dy, int64_t ld_dy, const void *w, int64_t ld_w, int64_t m, int64_t k, int64_t n,
                          const int8_t *z_q, const uint8_t *z_e, int act, const void *residual, int64_t ld_res, int res_dtype,
                          void *dx, int64_t ld_dx, int dx_dtype, void *ws, size_t ws_bytes, void *stream);

/*
 * ra_linear_wgrad -- dw = a^T dy and db = the column sums of dy.
 *   x         m x k, bf16: a = x; or NULL and
 *   z_q, z_e  the 8-bit checkpoint of z (m x k): a = act(z), recomputed here
 *             (act is RA_ACT_NONE with x); an empty checkpoint's pointers may
 *             be NULL too.  With RA_ACT_NONE a is exact; else act(z) is
 *             rounded to bf16 for the tensor cores, whatever type dw has: the
 *             forward layer's own product read its input rounded so, and a
 *             second product over what the rounding drops would double the work
 *   dy        m x n, bf16
 *   dw        k x n of dw_dtype; accumulate != 0 adds to it (micro-batches)
 *   db        n binary32 values, or NULL; accumulate holds for it too
 *   ws        as for ra_linear, for x and dy; needed for a checkpoint
 */
ra_status ra_linear_wgrad(const void *x, int64_t ld_x, const int8_t *z_q, const uint8_t *z_e, int act, const void *dy,
                          int64_t ld_dy, int64_t m, int64_t k, int64_t n, int accumulate, void *dw, int64_t ld_dw,
                          int dw_dtype, float *db, void *ws, size_t ws_bytes, void *stream);

/*
 * ra_selftest_linear_stall -- exercises the products' time limit on purpose: in
 * the product that this host thread queues next through ra_linear (other than
 * a single token's), ra_linear_dgrad or ra_linear_wgrad, block `block` of the
 * grid makes no copies, and every wait is limited to timeout_us (1 .. 10^7).
 * The waits that run out are recorded (ra_check_device_errors: RA_ERR_TIMEOUT)
 * and the blocks return; nothing hangs, and no memory is touched that the call
 * would not touch.  What a block that gave up would have stored stays as it
 * was, but for db, which waits for nothing.
 */
ra_status ra_selftest_linear_stall(int block, int timeout_us);

#ifdef __cplusplus
}
#endif

#endif /* RA_OPERATORS_H */
