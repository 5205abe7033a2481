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
 *   ra_dropout             values dropped by a counter-based generator, + residual
 *   ra_norm_block          the join behind a block and the norm before the next
 *   ra_norm_block_grad     its gradients
 *   ra_logprobs            log probabilities of given tokens, entropy, alternatives
 *   ra_logprobs_grad       the logits' gradient
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

/*
 * ra_dropout -- y = residual + (kept ? x * 1/(1-p) : 0), a value kept or dropped
 * by 16 bits that its place and the seed alone decide: the mask is never stored.
 * The gradient with respect to x is the same call on dy without a residual; a
 * recomputation in the backward pass, and a micro-batch of a larger batch
 * (first_row), meet the same mask again.
 *   x         rows x cols of x_dtype
 *   p         in [0, 1]: a value is dropped with probability t / 65536, t =
 *             65536 p rounded to a whole number (ties to even), and the others are
 *             scaled by 65536 / (65536 - t), so that the mean is kept exactly.
 *             Nothing is kept at t = 65536.  What is dropped counts as 0, whatever
 *             it holds.
 *   seed      the generator's key; with seed_at (8-byte aligned device memory, or
 *             NULL) the 64-bit number found there when the kernel runs is added to
 *             it, so that a captured call takes another mask at each replay
 *   site      tells the calls of one step apart
 *   first_row, >= 0: row r of x is row first_row + r of the mask
 *   residual  rows x cols of res_dtype, or NULL
 *   y         rows x cols of y_dtype, rounded once; may be x or the residual itself
 *             (same address, ld and type)
 * The bits: Philox4x32-10 (Salmon, Moraes, Dror and Shaw 2011) under the key (low,
 * high word of the seed) makes four words of the counter (column / 8, site, low,
 * high word of the row); column 8 g + j takes the low half of word j / 2 where j
 * is even, the high half where it is odd; a value is kept where they are t or more.
 */
ra_status ra_dropout(const void *x, int64_t ld_x, int x_dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                     const uint64_t *seed_at, uint32_t site, int64_t first_row, const void *residual, int64_t ld_res,
                     int res_dtype, void *y, int64_t ld_y, int y_dtype, void *stream);

/* A norm over a row v of d values: (v - m) * rstd * gain + bias,
 *   m = mean of v (RA_NORM_LAYER) or 0 (RA_NORM_RMS), rstd = (mean of (v - m)^2 + eps)^-1/2.
 * Moments are binary32, the second one of the differences from the first (or of the
 * values, less m^2, where that costs 4 bits at most).  Where the sum of these squares
 * is no binary32 number rstd is 0; where that of the values is none the row is NaN. */
typedef enum { RA_NORM_NONE = 0, RA_NORM_LAYER = 1, RA_NORM_RMS = 2 } ra_norm_kind;
#define RA_NORM_MAX_D 32768

typedef struct {
    const void *gain; /* d values of dtype, or NULL: ones */
    const void *bias; /* d values of dtype, or NULL: zeros */
    int dtype;        /* of both */
    int kind;         /* ra_norm_kind; RA_NORM_NONE: no norm, the rest is not looked at */
    float eps;        /* >= 0 */
    int reserved;     /* 0 */
} ra_norm;

typedef enum { RA_GATE_NONE = 0, RA_GATE_VECTOR = 1, RA_GATE_MATRIX = 2 } ra_gate_kind;

/*
 * ra_norm_block -- what lies between two blocks of a layer, in one pass over its
 * rows:
 *   x' = alpha x + beta gate * post(f),   h = pre(x')
 * x is the residual stream, f the output of the block behind, h the input of the
 * block ahead.  x' is rounded to its type and pre() is that of the rounded row, so
 * that h is what a call of its own would make of x' and the backward pass, which
 * reads x', differentiates what was computed.
 *   f      NULL: x' is x, x_out is not written, and only pre() is computed
 *   post   RA_NORM_NONE: f itself;  pre  RA_NORM_NONE: no h (only with f)
 *   gate   d values of gate_dtype, or rows x d of f_dtype; RA_GATE_NONE: ones
 *   x_out  rows x d of x_dtype; may be x itself (same address and ld)
 *   h      rows x d of f_dtype, which is the type of f too
 *   kept   4 values a row, contiguous and 16-byte aligned, or NULL: m and rstd of
 *          post and of pre (zeros where there is no such norm), for the backward pass
 * x_dtype and f_dtype: both RA_F32, both RA_BF16, or RA_F32 and RA_BF16.
 * d is at most RA_NORM_MAX_D (RA_ERR_UNSUPPORTED).  Beside an infinite gate or gain a
 * value may be NaN where the formula has an infinity.
 */
typedef struct {
    int64_t rows, d;
    const void *x;
    int64_t ld_x;
    const void *f;
    int64_t ld_f;
    const void *gate;
    int64_t ld_gate; /* of a matrix */
    void *x_out;
    int64_t ld_x_out;
    void *h;
    int64_t ld_h;
    float *kept;
    ra_norm post, pre;
    int x_dtype, f_dtype, gate_kind, gate_dtype; /* gate_dtype: of a vector */
    float alpha, beta;
} ra_norm_block_args;

ra_status ra_norm_block(const ra_norm_block_args *args, void *stream);

/*
 * ra_norm_block_grad -- the gradients of ra_norm_block, from dh (of h) and dx_new
 * (of x', what the later part of the stream sends back).  With v = (x' - m) rstd of
 * pre and w = (f - m) rstd of post:
 *   D  = dx_new + the gradient of pre() with respect to x'
 *   dx = alpha D  (D where there is no f),   dgate = beta D post(f)
 *   df = the gradient of post() for  u = beta gate D
 *   dpre_gain = sum of dh v,  dpre_bias = sum of dh,  dpost_gain = sum of u w,
 *   dpost_bias = sum of u, sums over the rows
 *   dh     rows x d of f_dtype; NULL exactly where pre is RA_NORM_NONE
 *   dx_new rows x d of x_dtype, or NULL: zeros (not where dh is NULL too)
 *   x      x' as ra_norm_block left it (or took it, without an f); not read without pre
 *   f, gate, kept, post, pre, alpha, beta  as there
 *   dx     rows x d of x_dtype, may be dx_new itself;  df  rows x d of f_dtype
 *   dgate  d binary32 values (a vector's: summed over the rows), or rows x d of
 *          f_dtype (a matrix's)
 *   dpost_gain, ...  d binary32 values each, 4-byte aligned
 *   accumulate != 0 adds to the vectors of d values (micro-batches); dx, df and a
 *          matrix's dgate are always overwritten
 * Any output may be NULL; then it is not made.  With rows 0 the vectors become 0
 * (or stay, with accumulate), whatever parts there are.  ws: device workspace of
 * at least ra_norm_block_grad_workspace_bytes(rows, d), 16-byte aligned, where a
 * vector of sums is wanted; else it may be NULL.
 */
typedef struct {
    int64_t rows, d;
    const void *dh;
    int64_t ld_dh;
    const void *dx_new;
    int64_t ld_dx_new;
    const void *x;
    int64_t ld_x;
    const void *f;
    int64_t ld_f;
    const void *gate;
    int64_t ld_gate;
    const float *kept;
    void *dx;
    int64_t ld_dx;
    void *df;
    int64_t ld_df;
    void *dgate;
    int64_t ld_dgate;
    float *dpost_gain, *dpost_bias, *dpre_gain, *dpre_bias;
    void *ws;
    size_t ws_bytes;
    ra_norm post, pre;
    int x_dtype, f_dtype, gate_kind, gate_dtype; /* gate_dtype: of a vector */
    float alpha, beta;
    int accumulate, reserved;
} ra_norm_block_grad_args;

size_t ra_norm_block_grad_workspace_bytes(int64_t rows, int64_t d);
ra_status ra_norm_block_grad(const ra_norm_block_grad_args *args, void *stream);

/*
 * ra_logprobs -- for each row of logits, z = scale * logits[r, :]:
 *   lse[r]     = log of the sum of exp z
 *   logp[r]    = z[ids[r]] - lse[r]; 0 for an id outside [0, vocab) (padding)
 *   entropy[r] = - sum of p log p, p = exp(z - lse)
 *   top_ids, top_logp  the `top` most likely tokens, by falling logit and, among
 *              equals, by rising index, with their log probabilities
 * A logit of minus infinity is a token that cannot be: it adds nothing, its log
 * probability is minus infinity, and it is no alternative.  Where fewer than `top`
 * tokens can be, the rest of the row is -1 and minus infinity.  A row in which no
 * token can be has lse minus infinity, entropy 0 and logp minus infinity (0 for
 * padding).  A row with a NaN or plus infinity gives NaN in place of every number
 * but a padding's logp, and -1 as its alternatives.  Finite logits may lie anywhere:
 * sums are of exp of differences from logits of the row, so that rows far from zero,
 * or masked by any finite value, keep their digits; lse itself is a binary32 number
 * (an infinity beyond the range).  A difference that is none counts as infinite.
 *   logits   rows x vocab of dtype;  ids  rows integers of id_bytes (4 or 8)
 *   scale    the inverse of a temperature: > 0, and 1.443 scale is finite
 *   logp, lse, entropy  rows binary32 values each; logp (then ids too) and entropy
 *            may be NULL
 *   top      0 .. RA_LOGPROBS_MAX_TOP;  top_ids, top_logp  rows x top, contiguous
 */
#define RA_LOGPROBS_MAX_TOP 32
#define RA_LOGPROBS_MAX_VOCAB (1 << 30) /* RA_ERR_UNSUPPORTED beyond, for the gradient too */
ra_status ra_logprobs(const void *logits, int64_t ld, int dtype, int64_t rows, int64_t vocab, const void *ids, int id_bytes,
                      float scale, float *logp, float *lse, float *entropy, int top, int64_t *top_ids, float *top_logp,
                      void *stream);

/*
 * ra_logprobs_grad -- the gradient with respect to the logits, from those of logp
 * (g) and of the entropy (e), p = exp(z - lse):
 *   out[r, j] = scale * (g[r] ([j = ids[r]] - p_j) - e[r] p_j (z_j - lse[r] + entropy[r]))
 * Padding's g counts for nothing, whatever it holds.  A token that cannot be has
 * p = 0 and adds no entropy; a row in which none can be has gradient 0.  lse is a
 * binary32 number: its rounding makes p off by a factor of up to exp(2^-24 |lse|),
 * never above 1.  So a row with lse below -2^24, of which p would have no digit (a
 * row masked throughout by a finite value such as -10^9), has gradient 0 too.
 *   lse, entropy  as ra_logprobs left them; entropy only with grad_entropy
 *   grad_logp, grad_entropy  rows binary32 values, or NULL: zeros; without
 *            grad_logp ids are not looked at
 *   out      rows x vocab of out_dtype, rounded once; may be the logits themselves
 *            (same address, ld and type)
 */
ra_status ra_logprobs_grad(const void *logits, int64_t ld, int dtype, int64_t rows, int64_t vocab, const void *ids,
                           int id_bytes, float scale, const float *lse, const float *entropy, const float *grad_logp,
                           const float *grad_entropy, void *out, int64_t ld_out, int out_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RA_OPERATORS_H */
