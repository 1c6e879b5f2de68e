/*
 * fno_ops.h -- C ABI of the sequence and training operators of the library:
 *
 *   fno_sandwich_*     norms before and after a block, with the block's gate,
 *                      residual scale and residual sum, and their gradients;
 *   fno_act8_*         activation checkpoints in 8 bits, and GELU's backward
 *                      from one;
 *   fno_linear_grad_*  weight and bias gradient of a 1x1 linear from the 8-bit
 *                      checkpoint of its input;
 *   fno_linattn_*      linear attention with a decay for each head: prompts,
 *                      single tokens, gradients;
 *   fno_rotary_*       rotary positions of its queries and keys;
 *   fno_causal_conv_*  short causal convolutions along time, and
 *   fno_scan_*         the selective state space scan behind them: prompts, single
 *                      tokens, gradients.
 *
 * They surround the spectral layers of fno.h in a deep or time-dependent
 * neural operator: the sandwich norm and the checkpoints work on the layers'
 * channels-first fields as well as on token rows, and the linear attention or
 * the scan carries the history of a simulation from frame to frame.
 *
 * The conventions of fno.h hold: fno_status_t from every call, nothing thrown
 * or printed; device pointers are the caller's, 16-byte aligned
 * (FNO_ERR_MISALIGNED) and dense row-major; work is enqueued on `stream`; no
 * call but the plan calls allocates or waits, so that every other call can be
 * captured in a CUDA graph; an output may not overlap an input, another output
 * or the workspace (FNO_ERR_ALIASING) except where a call says so.  Parameters
 * and their gradients are float32; fields have the storage type; sums, norms
 * and states are float32 and results do not depend on the order in which the
 * GPU runs its blocks.  Where operands or functions have fewer digits than
 * that, a call says so.  Calls that may run at the same time need their own
 * workspaces; a plan may be shared.
 */
#ifndef FNO_OPS_H_
#define FNO_OPS_H_

#include "fno.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------------------------
 * Sandwich norm.
 *
 * For a block f = F(u) of a residual stack (F a spectral layer, attention, a
 * pointwise network):
 *   y = x + s * a * (n2(f) * w2 + b2)        the block's output joins the stream
 *   u = n1(y) * w1 + b1                      the next block's input
 * with, over the channels of each point,
 *   n(v) = v / sqrt(mean(v^2) + eps)                       (FNO_NORM_RMS, no b)
 *   n(v) = (v - mean v) / sqrt(mean((v - mean v)^2) + eps) (FNO_NORM_LAYER)
 * s the residual scale of each channel, and the gate a = g or 1 / (1 + e^-g).
 * ------------------------------------------------------------------------- */
typedef enum fno_layout_e {
    FNO_LAYOUT_GRID = 0,    /* (batch, channels, points): the spectral layers' fields     */
    FNO_LAYOUT_TOKENS = 1   /* (batch, points, channels)                                  */
} fno_layout_t;

typedef enum fno_norm_e { FNO_NORM_RMS = 0, FNO_NORM_LAYER = 1 } fno_norm_t;

typedef enum fno_gate_e {
    FNO_GATE_NONE = 0,      /* a = 1                                                      */
    FNO_GATE_CHANNEL = 1,   /* g is float32 (batch, channels)                             */
    FNO_GATE_FULL = 2       /* g has the field's shape and storage type                   */
} fno_gate_t;

typedef struct fno_sandwich_s *fno_sandwich_t;

typedef struct fno_sandwich_desc_s {
    int64_t batch, points;    /* >= 1                                                     */
    int32_t channels;         /* 1 .. 65536                                               */
    fno_layout_t layout;
    fno_norm_t norm;
    fno_gate_t gate;
    int32_t gate_sigmoid;     /* 0: a = g, 1: a = 1 / (1 + e^-g) (1e-6 relative for       */
                              /* |g| up to 10)                                            */
    float eps;                /* >= 0                                                     */
    fno_dtype_t dtype;        /* storage type of x, f, y, u and a full gate               */
} fno_sandwich_desc_t;

/* Validate the description and make a plan (host memory only).  *plan is NULL
 * on failure.  Errors: INVALID_ARG, UNSUPPORTED (more than 2^38 elements, than
 * 2^34 - 8 points in all samples, than 65535 samples with FNO_GATE_CHANNEL, for
 * either direction), OUT_OF_MEMORY, CUDA.                                     */
fno_status_t fno_sandwich_plan(fno_sandwich_t *plan, const fno_sandwich_desc_t *desc);

/* Device workspace bytes of fno_sandwich_backward (the forward needs none). */
fno_status_t fno_sandwich_workspace_size(fno_sandwich_t plan, size_t *bytes);

/* y and u of the formulas above.
 *   x        residual stream, the field's shape
 *   f        the block's output; NULL: no block, u = n1(x) w1 + b1 (the norm
 *            in front of the first block) and y, gate, s, w2, b2, f8,
 *            f8_scale must be NULL
 *   gate     as desc.gate says, NULL for FNO_GATE_NONE
 *   s, w2, w1  (channels) float32; b2, b1 for FNO_NORM_LAYER, else NULL
 *   y        the field's shape; may be x itself (the stream updated in place)
 *   u        the field's shape; NULL: not wanted (then w1, b1 are NULL)
 *   f8, f8_scale  both or neither: also keep f in 8 bits, exactly as
 *            fno_act8_pack(rows, cols) would, rows of the layout's last axis
 * u is computed from y before y is rounded to its storage type.               */
fno_status_t fno_sandwich_forward(fno_sandwich_t plan, const void *x, const void *f,
                                  const void *gate, const float *s, const float *w2,
                                  const float *b2, const float *w1, const float *b1, void *y,
                                  void *u, int8_t *f8, float *f8_scale, fno_stream_t stream);

/* Gradients, given dy = dL/dy (from the stream) and du = dL/du:
 *   dY = dy + (gradient of n1 at y, of du w1),  dx = dY,
 *   df, dgate, ds, dw2, db2, dw1, db1 by the chain rule from dY and du.
 *   y        the forward's output as stored
 *   f        the block's output, or NULL with f8, f8_scale its 8-bit
 *            checkpoint (then the gradients are those at the values that the
 *            codes stand for); all three NULL: the norm alone (f NULL forward)
 *   dy       NULL: zero.    du  NULL: u was not computed (w1 is NULL)
 *   dx       the field's shape; may be dy itself
 *   df       the field's shape, with f or f8; may not be NULL then
 *   dgate    float32 (batch, channels) for FNO_GATE_CHANNEL, the field's shape
 *            and type for FNO_GATE_FULL, NULL for FNO_GATE_NONE or not wanted
 *   ds, dw2, db2, dw1, db1  (channels) float32; each NULL if not wanted
 * workspace: fno_sandwich_workspace_size bytes.                               */
fno_status_t fno_sandwich_backward(fno_sandwich_t plan, const void *y, const void *f,
                                   const int8_t *f8, const float *f8_scale, const void *gate,
                                   const float *s, const float *w2, const float *b2,
                                   const float *w1, const void *dy, const void *du, void *dx,
                                   void *df, void *dgate, float *ds, float *dw2, float *db2,
                                   float *dw1, float *db1, void *workspace, fno_stream_t stream);

/* Release the plan; NULL is accepted. */
fno_status_t fno_sandwich_destroy(fno_sandwich_t plan);

/* -------------------------------------------------------------------------
 * Activation checkpoints in 8 bits.
 *
 * x is rows x cols.  Each run of FNO_ACT8_GROUP consecutive elements of a row
 * (the last one of a row may be shorter) shares a float32 scale:
 *   m = max |x|,  scale = m / 127,  code = rint(x * (127 / m)),
 * in float32, ties to even; a group with m < 1e-30 has scale 0.  The value of
 * a code is code * scale, at most m / 254 (and rounding) from x.  A group that
 * holds a NaN or an infinity has that scale, and reads back as NaN.
 * codes: int8, rows x cols.  scales: float32, rows x ceil(cols / GROUP).
 * rows, cols >= 1, at most 2^38 elements and 2^36 - 32 groups (else
 * FNO_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------- */
#define FNO_ACT8_GROUP 128

fno_status_t fno_act8_pack(int64_t rows, int64_t cols, fno_dtype_t dtype, const void *x,
                           int8_t *codes, float *scales, fno_stream_t stream);

/* x = code * scale, rounded to the storage type. */
fno_status_t fno_act8_unpack(int64_t rows, int64_t cols, fno_dtype_t dtype, const int8_t *codes,
                             const float *scales, void *x, fno_stream_t stream);

/* dx = dy * GELU'(v), v the checkpoint's values, GELU the exact form
 * v/2 (1 + erf(v / sqrt 2)), its slope to 3e-7 absolute (erf by a published
 * polynomial, as in the pointwise layers).  dx may be dy itself.              */
fno_status_t fno_act8_gelu_backward(int64_t rows, int64_t cols, fno_dtype_t dtype,
                                    const int8_t *codes, const float *scales, const void *dy,
                                    void *dx, fno_stream_t stream);

/* -------------------------------------------------------------------------
 * Weight and bias gradient of the 1x1 linear  t[b,o,p] = sum_i W[o,i] x[b,i,p]
 * + bias[o]  (the pointwise linears of fno_forward), from dy = dL/dt and the
 * 8-bit checkpoint of x (rows = batch * cin, cols = points):
 *   dw[o,i] = sum_{b,p} dy[b,o,p] x[b,i,p],   db[o] = sum_{b,p} dy[b,o,p].
 * The products are exact (codes are small integers) and summed in float32; the
 * scales are applied in float32.
 * ------------------------------------------------------------------------- */
typedef struct fno_linear_grad_s *fno_linear_grad_t;

/* batch, points >= 1; 1 <= cin, cout <= 4096.  dtype: storage of dy.  Errors:
 * INVALID_ARG, UNSUPPORTED, OUT_OF_MEMORY, CUDA.                             */
fno_status_t fno_linear_grad_plan(fno_linear_grad_t *plan, int64_t batch, int32_t cin,
                                  int32_t cout, int64_t points, fno_dtype_t dtype);
fno_status_t fno_linear_grad_workspace_size(fno_linear_grad_t plan, size_t *bytes);

/* dw (cout, cin), db (cout) float32; db may be NULL. */
fno_status_t fno_linear_grad(fno_linear_grad_t plan, const void *dy, const int8_t *codes,
                             const float *scales, float *dw, float *db, void *workspace,
                             fno_stream_t stream);

/* Synchronise `stream`, read and clear the plan's device error word (as
 * fno_plan_get_device_error).                                                */
fno_status_t fno_linear_grad_get_device_error(fno_linear_grad_t plan, fno_stream_t stream);
fno_status_t fno_linear_grad_destroy(fno_linear_grad_t plan);

/* -------------------------------------------------------------------------
 * Linear attention with a decay for each head.
 *   S_t = e^{log_decay[h]} S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
 * per sequence and query head h; query head h reads key/value head
 * h / (heads / kv_heads).  S is dk x dv.
 *   q (batch, length, heads, dk), k (batch, length, kv_heads, dk),
 *   v (batch, length, kv_heads, dv), o (batch, length, heads, dv): storage type
 *   log_decay (heads) float32, <= 0 (-inf: the state holds the last token
 *     only); the decay is a constant of the head and has no gradient
 *   states (batch, heads, dk, dv) float32
 *   lengths (batch) int32 or NULL: sequence b has max(0, min(lengths[b],
 *     length)) tokens; o and the gradients beyond are 0 and q, k, v beyond are
 *     not looked at; a sequence of no tokens returns its initial state
 * Up to 128 tokens are worked on together: an infinity or a NaN in one of a
 * sequence's tokens may reach the outputs of that many before it in its head,
 * and an infinity may come out as a NaN.
 * The sums and the state are float32.  The decayed products of queries and keys,
 * the state that a query meets and what a token adds to the state keep float32's
 * digits for float32, and 16 bits or more for fp16 and bfloat16, in front of the
 * rounding of the result (final states and ds0: float32's digits for all).
 * ------------------------------------------------------------------------- */
typedef struct fno_linattn_s *fno_linattn_t;

#define FNO_LINATTN_BACKWARD 1u   /* the plan's workspace also covers the backward          */

/* batch, length >= 1; 1 <= kv_heads <= heads, heads a multiple of kv_heads;
 * 1 <= dk, dv <= 256.  Errors: INVALID_ARG, UNSUPPORTED, OUT_OF_MEMORY, CUDA. */
fno_status_t fno_linattn_plan(fno_linattn_t *plan, int64_t batch, int64_t length, int32_t heads,
                              int32_t kv_heads, int32_t dk, int32_t dv, fno_dtype_t dtype,
                              uint32_t flags);
fno_status_t fno_linattn_workspace_size(fno_linattn_t plan, size_t *bytes);

/* Prompts.  s0 NULL: zero initial state; sT NULL: final state not wanted; sT
 * may be s0 itself.                                                          */
fno_status_t fno_linattn_forward(fno_linattn_t plan, const void *q, const void *k, const void *v,
                                 const float *log_decay, float scale, const int32_t *lengths,
                                 const float *s0, void *o, float *sT, void *workspace,
                                 fno_stream_t stream);

/* Gradients of L given go = dL/do and gsT = dL/dS_T (NULL: zero).  dq, dk, dv
 * have the shapes of q, k, v (a shared key/value head sums over its query
 * heads); ds0 NULL: not wanted; ds0 may be gsT itself.  Needs
 * FNO_LINATTN_BACKWARD.                                                       */
fno_status_t fno_linattn_backward(fno_linattn_t plan, const void *q, const void *k, const void *v,
                                  const float *log_decay, float scale, const int32_t *lengths,
                                  const float *s0, const void *go, const float *gsT, void *dq,
                                  void *dk, void *dv, float *ds0, void *workspace,
                                  fno_stream_t stream);

/* One token for each of the plan's `batch` rows: q (batch, heads, dk), k
 * (batch, kv_heads, dk), v (batch, kv_heads, dv), o (batch, heads, dv); the
 * plan's length is not used.  state, new_state: (num_slots, heads, dk, dv)
 * float32; row b reads state[slots[b]] and writes new_state[slots[b]]
 * (new_state may be state itself).  slots NULL: row b uses slot b.  A row whose
 * slot is outside [0, num_slots) is idle: its o is 0 and no state is touched.
 * Two rows of one call may not share a slot.                                 */
fno_status_t fno_linattn_step(fno_linattn_t plan, const void *q, const void *k, const void *v,
                              const float *log_decay, float scale, const int32_t *slots,
                              int64_t num_slots, const float *state, float *new_state, void *o,
                              fno_stream_t stream);

/* Synchronise `stream`, read and clear the plan's device error word (as
 * fno_plan_get_device_error).                                                */
fno_status_t fno_linattn_get_device_error(fno_linattn_t plan, fno_stream_t stream);
fno_status_t fno_linattn_destroy(fno_linattn_t plan);

/* -------------------------------------------------------------------------
 * Rotary positions.
 * The first `rotary_dim` elements of each head are pairs (a, b), pair i of
 * rotary_dim / 2: elements i and i + rotary_dim / 2 (FNO_ROTARY_HALF) or 2 i and
 * 2 i + 1 (FNO_ROTARY_INTERLEAVED).  A token at position p turns pair i to
 *   m (a cos(p f_i) - b sin(p f_i)),  m (b cos(p f_i) + a sin(p f_i)),
 *   f_i = base^(-2 i / rotary_dim),  m = 1,
 * and the rest of the head is copied.  For contexts longer than those trained on
 * (`factor` times):
 *   FNO_ROTARY_LINEAR  f_i / factor
 *   FNO_ROTARY_BASE    base times factor^(rotary_dim / (rotary_dim - 2)), which has to be finite
 *                      (rotary_dim > 2)
 *   FNO_ROTARY_RAMP    f_i (k + (1 - k) / factor), where a pair that makes `fast` turns or
 *                      more over `original` positions has k = 1 (it stays), one that makes
 *                      `slow` or fewer k = 0, and k is linear in the turns between;
 *                      m = 1 + 0.1 log(factor)
 * A position's fraction of a turn is exact to 2^-32 of a turn and to what f_i's 53 bits give at
 * any position of 32 bits, then rounded to float32 (2^-26 of a turn at most); cosines and sines
 * are float32's (for 16-bit types good to 2^-20).
 * ------------------------------------------------------------------------- */
typedef enum fno_rotary_layout_e {
    FNO_ROTARY_HALF = 0, FNO_ROTARY_INTERLEAVED = 1
} fno_rotary_layout_t;

typedef enum fno_rotary_scaling_e {
    FNO_ROTARY_NONE = 0, FNO_ROTARY_LINEAR = 1, FNO_ROTARY_BASE = 2, FNO_ROTARY_RAMP = 3
} fno_rotary_scaling_t;

typedef struct fno_rotary_s *fno_rotary_t;

typedef struct fno_rotary_desc_s {
    int64_t batch, length;    /* >= 1                                                     */
    int32_t heads;            /* of q, >= 1                                               */
    int32_t kv_heads;         /* of k, >= 0 (0: there is no k)                            */
    int32_t dim;              /* of a head, 1 .. 1024; (heads + kv_heads) dim <= 65536    */
    int32_t rotary_dim;       /* even, 2 .. min(dim, 256)                                 */
    fno_rotary_layout_t layout;
    fno_rotary_scaling_t scaling;
    double base;              /* > 1                                                      */
    double factor;            /* >= 1 (unless FNO_ROTARY_NONE)                            */
    double original, fast, slow;    /* FNO_ROTARY_RAMP: > 0, fast > slow >= 0             */
    fno_dtype_t dtype;        /* storage type of q and k                                  */
} fno_rotary_desc_t;

/* Errors: INVALID_ARG, UNSUPPORTED, OUT_OF_MEMORY, CUDA. */
fno_status_t fno_rotary_plan(fno_rotary_t *plan, const fno_rotary_desc_t *desc);

/* q (batch, length, heads, dim), k (batch, length, kv_heads, dim) -> qo, ko, which may be
 * q and k themselves.  k and ko are NULL for kv_heads = 0.  Token t of sequence b has
 *   positions  int32 (batch, length): its position, or NULL
 *   offsets    int32 (batch): position offsets[b] + t, or NULL (at most one of the two)
 * or, both NULL, position t.  transpose != 0: the gradients of q and k from those of qo and
 * ko (each pair turned back, times m).                                        */
fno_status_t fno_rotary_apply(fno_rotary_t plan, const void *q, const void *k,
                              const int32_t *positions, const int32_t *offsets,
                              int32_t transpose, void *qo, void *ko, fno_stream_t stream);
fno_status_t fno_rotary_destroy(fno_rotary_t plan);

/* -------------------------------------------------------------------------
 * Short causal convolution of each channel along time.
 *   y_t = act(bias[c] + sum_j w[c, j] x_{t - width + 1 + j}),   j = 0 .. width - 1
 *   x, y (batch, length, channels): storage type; w (channels, width), bias (channels)
 *     float32, bias NULL: zero
 *   act: none, or v / (1 + e^-v) (1e-6 relative for |v| up to 10)
 *   states (batch, width - 1, channels), storage type: the inputs in front of the first
 *     token, oldest first
 *   lengths (batch) int32 or NULL: sequence b has max(0, min(lengths[b], length)) tokens; y
 *     and dx beyond are 0 and x and dy beyond are not looked at
 * ------------------------------------------------------------------------- */
typedef enum fno_act_e { FNO_ACT_NONE = 0, FNO_ACT_SILU = 1 } fno_act_t;

typedef struct fno_causal_conv_s *fno_causal_conv_t;

#define FNO_CAUSAL_CONV_BACKWARD 1u   /* the workspace is that of the backward              */

/* batch, length, channels >= 1, length below 2^31 - 64, channels up to 65535 x 64;
 * 2 <= width <= 8.
 * Errors: INVALID_ARG, UNSUPPORTED, OUT_OF_MEMORY, CUDA.                      */
fno_status_t fno_causal_conv_plan(fno_causal_conv_t *plan, int64_t batch, int64_t length,
                                  int32_t channels, int32_t width, fno_act_t act,
                                  fno_dtype_t dtype, uint32_t flags);
fno_status_t fno_causal_conv_workspace_size(fno_causal_conv_t plan, size_t *bytes);

/* s0 NULL: zeros; sT (the last width - 1 inputs, s0's among them where the sequence is
 * shorter) NULL: not wanted.  Needs no workspace.                             */
fno_status_t fno_causal_conv_forward(fno_causal_conv_t plan, const void *x, const float *w,
                                     const float *bias, const int32_t *lengths, const void *s0,
                                     void *y, void *sT, fno_stream_t stream);

/* Gradients given dy = dL/dy and dsT = dL/dsT (NULL: zero).  dw (channels, width) and dbias
 * (channels) float32; dbias, ds0 NULL: not wanted.  Needs FNO_CAUSAL_CONV_BACKWARD. */
fno_status_t fno_causal_conv_backward(fno_causal_conv_t plan, const void *x, const float *w,
                                      const float *bias, const int32_t *lengths, const void *s0,
                                      const void *dy, const void *dsT, void *dx, float *dw,
                                      float *dbias, void *ds0, void *workspace,
                                      fno_stream_t stream);

/* One token for each of the plan's `batch` rows: x, y (batch, channels).  state, new_state
 * (num_slots, width - 1, channels): row b reads state[slots[b]] and writes
 * new_state[slots[b]] (new_state may be state itself).  slots NULL: row b uses slot b.  A row
 * whose slot is outside [0, num_slots) is idle: its y is 0 and no state is touched.  Two rows
 * of one call may not share a slot.                                           */
fno_status_t fno_causal_conv_step(fno_causal_conv_t plan, const void *x, const float *w,
                                  const float *bias, const int32_t *slots, int64_t num_slots,
                                  const void *state, void *new_state, void *y,
                                  fno_stream_t stream);
fno_status_t fno_causal_conv_destroy(fno_causal_conv_t plan);

/* -------------------------------------------------------------------------
 * Selective state space scan.  For each channel c (of group g = c / (channels / groups)) and
 * state n of a sequence
 *   d_t = softplus(dt_t[c] + dt_bias[c])   (or dt_t[c] + dt_bias[c])
 *   h_t[c, n] = e^{d_t A[c, n]} h_{t-1}[c, n] + d_t x_t[c] B_t[g, n]
 *   y_t[c] = (sum_n C_t[g, n] h_t[c, n] + D[c] x_t[c]) * silu(z_t[c])
 *   x, dt, z, y (batch, length, channels), B, C (batch, length, groups, states): storage
 *     type; z NULL: no gate
 *   A (channels, states), D, dt_bias (channels) float32; D, dt_bias NULL: zero
 *   states h (batch, channels, states) float32
 *   lengths (batch) int32 or NULL: sequence b has max(0, min(lengths[b], length)) tokens; y
 *     and the gradients beyond are 0 and the inputs beyond are not looked at; a sequence of
 *     no tokens returns its initial state
 * All arithmetic is float32 on the stored inputs.  A decay e^{d A} is good to 1.5e-7 +
 * 1.4e-7 |d A| of itself (below 2^-126 it is 0), a state that remembers n tokens to n times
 * that and its sums' roundings; softplus to 1e-6 (a step below 2^-126 is 0), silu to 1e-6 for
 * |z| up to 10.  A is finite, and d A meant to be at most 0: time is split, so that where states
 * grow the product of all of a sequence's e^{d A} has to be below 2^127.  An infinity in a token
 * may come out as a NaN, in that token or a later one of its channel.
 * ------------------------------------------------------------------------- */
typedef struct fno_scan_s *fno_scan_t;

#define FNO_SCAN_BACKWARD 1u   /* the workspace also covers the backward                    */

typedef struct fno_scan_desc_s {
    int64_t batch, length;    /* >= 1, below 2^30 - 64 and 2^31 - 16                      */
    int32_t channels;         /* >= 1, below 2^31 - 256, a multiple of groups              */
    int32_t states;           /* 1 .. 64                                                  */
    int32_t groups;           /* >= 1                                                     */
    int32_t softplus;         /* 0: d = dt + dt_bias                                      */
    fno_dtype_t dtype;
    uint32_t flags;
} fno_scan_desc_t;

/* Errors: INVALID_ARG, UNSUPPORTED (also of a workspace beyond 2^38 bytes: the backward keeps
 * the states, padded to at most twice the channels and a power of two of states, of every
 * eighth token), OUT_OF_MEMORY, CUDA.                                         */
fno_status_t fno_scan_plan(fno_scan_t *plan, const fno_scan_desc_t *desc);
fno_status_t fno_scan_workspace_size(fno_scan_t plan, size_t *bytes);

/* s0 NULL: zero initial state; sT NULL: final state not wanted. */
fno_status_t fno_scan_forward(fno_scan_t plan, const void *x, const void *dt, const float *A,
                              const void *B, const void *C, const float *D, const void *z,
                              const float *dt_bias, const int32_t *lengths, const float *s0,
                              void *y, float *sT, void *workspace, fno_stream_t stream);

/* Gradients given dy = dL/dy and dsT = dL/dsT (NULL: zero).  dx, ddt, dz, dB, dC have the
 * shapes and type of x, dt, z, B, C (of B and C, the sums over a group's channels); dA, dD,
 * ddt_bias float32.  dz is NULL without z; dD, ddt_bias, ds0 NULL: not wanted.  Needs
 * FNO_SCAN_BACKWARD.                                                          */
fno_status_t fno_scan_backward(fno_scan_t plan, const void *x, const void *dt, const float *A,
                               const void *B, const void *C, const float *D, const void *z,
                               const float *dt_bias, const int32_t *lengths, const float *s0,
                               const void *dy, const float *dsT, void *dx, void *ddt, float *dA,
                               void *dB, void *dC, float *dD, void *dz, float *ddt_bias,
                               float *ds0, void *workspace, fno_stream_t stream);

/* One token for each of the plan's `batch` rows: x, dt, z, y (batch, channels), B, C (batch,
 * groups, states).  state, new_state (num_slots, channels, states) float32; slots as for
 * fno_causal_conv_step.                                                       */
fno_status_t fno_scan_step(fno_scan_t plan, const void *x, const void *dt, const float *A,
                           const void *B, const void *C, const float *D, const void *z,
                           const float *dt_bias, const int32_t *slots, int64_t num_slots,
                           const float *state, float *new_state, void *y, fno_stream_t stream);
fno_status_t fno_scan_destroy(fno_scan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* FNO_OPS_H_ */
