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
 *                      single tokens, gradients.
 *
 * They surround the spectral layers of fno.h in a deep or time-dependent
 * neural operator: the sandwich norm and the checkpoints work on the layers'
 * channels-first fields as well as on token rows, and the linear attention
 * carries the history of a simulation from frame to frame.
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

#ifdef __cplusplus
}
#endif

#endif /* FNO_OPS_H_ */
