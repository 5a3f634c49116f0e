/*
 * vsa_block.h -- C ABI of the operators around the VSA layer of vsa.h: what a
 * video transformer block does to the layer's inputs and outputs.
 *   - rotary positions with three axes (time, height, width), vsa_rope_*;
 *   - the norm of every query and key head with the rotation in the same pass,
 *     on its own (vsa_norm_rope) or fused into step 1 of the layer
 *     (vsa_norm_rope_permute_pool), and its backward;
 *   - linears with bias, activation and residual in the product's epilogue
 *     (vsa_linear), and their backward.
 *
 * The conventions of vsa.h hold for every call (ownership, alignment, streams,
 * errors, NVTX ranges), with one difference: tensors that come with a vsa_view
 * may be strided.  Calls on a plan keep nothing in it but a recorded fault, and
 * may overlap on the GPU (several streams) and come from several host threads; a workspace and an output belong to one call
 * at a time, and calls or captured graphs that may overlap need their own.
 */
#ifndef VSA_BLOCK_H_
#define VSA_BLOCK_H_

#include "vsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of parameter vectors (gains, biases). */
enum { VSA_BF16 = 0, VSA_F32 = 1 };

/* Activations.  gelu_tanh(x) = x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))),
 * silu(x) = x sigmoid(x). */
enum { VSA_ACT_IDENTITY = 0, VSA_ACT_SIGMOID = 1, VSA_ACT_GELU_TANH = 2, VSA_ACT_SILU = 3 };

/* A bf16 tensor [B,H,N,D] with its last dimension contiguous: element
 * (b,h,n,d) is at ptr + b*stride_b + h*stride_h + n*stride_n + d.  Strides
 * are in elements, multiples of 8, and not negative; ptr is 16-byte aligned.  A
 * stride of a dimension of extent 1 is not looked at.  Inputs of the norm_rope
 * calls may have strides of 0 (a broadcast tensor); the elements of an output must not
 * share memory with each other. */
typedef struct vsa_view {
  void* ptr;
  int64_t stride_b, stride_h, stride_n;
} vsa_view;

/* ------------------------------------------------------------------- rope
 * Rotary positions.  P = (dim[0] + dim[1] + dim[2]) / 2 pairs of channels turn;
 * pair p belongs to the axis whose block of dim[a]/2 pairs holds it (time, then
 * height, then width) and turns by
 *   angle(n, p) = pos[n][a] * inv_freq[p],
 *   (x, x') -> (x cos - x' sin, x sin + x' cos).
 * Channels from 2P to D pass through unchanged.  A token's position is a triple:
 * video token (t, h, w) stands at offset[a] + step[a] * coordinate, a prefix
 * token where prefix_pos says. */
typedef struct vsa_rope_s* vsa_rope;

typedef struct vsa_rope_desc {
  int32_t dim[3];            /* channels of each axis: even, >= 0, sum in [2, 128]        */
  int32_t halves;            /* 0: pairs (2p, 2p+1); 1: pairs (p, P + p), P a multiple of 4 */
  double theta[3];           /* inv_freq = theta^(-2i/dim) for pair i of its axis          */
  double offset[3], step[3]; /* positions of the video grid                                */
  const double* inv_freq;    /* host, P entries, or NULL: from theta                       */
  const double* prefix_pos;  /* host, [prefix tokens][3], or NULL: (0, 0, 0), no rotation  */
} vsa_rope_desc;

/* Builds the rotation of a plan's tokens: angles, cosines and sines in double,
 * kept as fp32 for every distinct position of each axis.  The tables live on
 * the plan's device (host only for a host-only plan), are there for any stream when the call
 * returns, and are owned by the handle, which does not refer to the plan afterwards: it goes with
 * every plan of the same device, number of prefix tokens and video grid, however these are cut into
 * segments and tiles, and calls with any other plan refuse it.  Errors: VSA_ERR_INVALID_ARG
 * for dimensions out of range or numbers that are not finite, VSA_ERR_CUDA. */
vsa_status vsa_rope_create(vsa_plan plan, const vsa_rope_desc* desc, vsa_rope* out);

/* The rotation of every token as the kernels use it: cos_sin[n][p] = (cos, sin),
 * host fp32 [N][P][2].  pairs (nullable) receives P. */
vsa_status vsa_rope_tables(vsa_rope rope, int32_t* pairs, float* cos_sin);

/* Frees the tables (after the work that uses them has finished: cudaFree
 * synchronises).  NULL is a no-op. */
vsa_status vsa_rope_destroy(vsa_rope rope);

/* y = R x (inverse = 0) or R^T x (inverse = 1: the gradient of the rotation) for
 * x, y bf16 [B,H,N,D] in natural order, N the plan's tokens.  fp32 arithmetic,
 * one rounding.  y may be x itself (same pointer and strides); otherwise they
 * must not overlap. */
vsa_status vsa_rope_apply(vsa_plan plan, vsa_rope rope, const vsa_view* x, const vsa_view* y,
                          int inverse, int B, int H, int D, void* stream);

/* --------------------------------------------------------------- norm_rope
 * Per head and token, over the D channels:
 *   z = x / sqrt(mean(x^2) + eps) * gain     (norm = 1; z = x for norm = 0)
 *   y = R z                                  (rotate = 1; y = z for rotate = 0)
 * in fp32 with one rounding to bf16 at the end.  A row of zeros gives zeros.
 * The squares are summed in fp32: rows with elements beyond about 1e18 overflow. */
#define VSA_MAX_HEAD_TENSORS 4

typedef struct vsa_head_tensor {
  vsa_view x;          /* bf16 [B,H,N,D], natural order                                */
  const void* gain;    /* [D] of gain_type, 16-byte aligned, or NULL: 1                */
  int32_t gain_type;   /* VSA_BF16 or VSA_F32                                          */
  int32_t norm, rotate;
  vsa_view y;          /* vsa_norm_rope: bf16 [B,H,N,D]; permute_pool: ptr only, bf16
                          [B,H,N_pad,D] contiguous                                     */
  float* pooled;       /* permute_pool only: fp32 [B,H,T,D], or NULL: no means         */
} vsa_head_tensor;

/* One launch for n tensors (1 .. VSA_MAX_HEAD_TENSORS), natural order in and out.
 * y may be x itself; an output must not overlap anything else of the call.  rope may
 * be NULL when no tensor rotates (and is not looked at then). */
vsa_status vsa_norm_rope(vsa_plan plan, vsa_rope rope, const vsa_head_tensor* tensors, int n,
                         float eps, int B, int H, int D, void* stream);

/* The same fused with vsa_permute_pool (step 1 of the layer): rows are written in
 * tile order (pad rows 0) and pooled receives the fp32 mean of each tile's live rows,
 * taken before the rounding to bf16.  With norm = rotate = 0 the rows are those of
 * vsa_permute_pool to the bit; the means are summed in another order (equal up to fp32 rounding, so
 * that a selection made from them may differ where scores tie that closely).  Q, K and V of a
 * layer take one launch; finish with vsa_coarse_topk_pooled.  y must not overlap x. */
vsa_status vsa_norm_rope_permute_pool(vsa_plan plan, vsa_rope rope, const vsa_head_tensor* tensors,
                                      int n, float eps, int B, int H, int D, void* stream);

typedef struct vsa_head_grad {
  vsa_view dy;         /* tiled = 0: bf16 [B,H,N,D]; tiled = 1: ptr only, bf16 [B,H,N_pad,D] */
  vsa_view x;          /* the forward's input (norm = 1; not read otherwise)                 */
  const void* gain;
  int32_t gain_type;
  int32_t norm, rotate;
  vsa_view dx;         /* bf16 [B,H,N,D], natural order                                      */
  float* d_gain;       /* fp32 [D], 16-byte aligned, or NULL                                 */
} vsa_head_grad;

/* Bytes of workspace vsa_norm_rope_backward needs for n tensors (the sums of d_gain
 * of each block).  Nothing in it has to be set before the call. */
vsa_status vsa_norm_rope_backward_workspace_size(vsa_plan plan, int n, int D, size_t* bytes);

/* Backward of both forms (tiled = 1: dy in tile order, the unpermute fused in).
 * With g = R^T dy, r = 1/sqrt(mean(x^2) + eps) and u = x r:
 *   dx = r (g gain - u mean(g gain u)),   d_gain = sum over b, h, n of g u
 * (dx = g without the norm, where d_gain has to be NULL).  The rows are read once; r is computed again from
 * x.  d_gain is summed in fp32 in a fixed order.  dx may be dy itself when tiled =
 * 0.  x of a head that several tensors share (a stride of 0) gets each tensor's own
 * dx: the caller adds them up. */
vsa_status vsa_norm_rope_backward(vsa_plan plan, vsa_rope rope, const vsa_head_grad* grads, int n,
                                  float eps, int tiled, int B, int H, int D, void* ws,
                                  size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ linear
 * Rows are tokens: tensors are [B,N,C] (heads = 0; the view's stride_h is not
 * looked at) or [B,heads,N,C/heads] with C/heads in {64, 128} (channel c = h *
 * C/heads + d).  N is any number of tokens (not the plan's); the plan gives the
 * device and the status word. */
typedef struct vsa_linear_args {
  int32_t B, x_heads, C, y_heads, O;
  int64_t N;
  vsa_view x;          /* bf16 input                                              */
  const void* w;       /* bf16 [O,C] (nn.Linear layout)                           */
  const void* bias;    /* [O] of bias_type, 16-byte aligned, or NULL              */
  int32_t bias_type;
  int32_t act;
  vsa_view residual;   /* laid out as y, or ptr = NULL; may be y itself           */
  vsa_view pre;        /* laid out as y, or ptr = NULL: receives x w^T + bias     */
  vsa_view y;
} vsa_linear_args;

/* Bytes of workspace with which vsa_linear splits a product of few rows over more of the GPU
 * (fp32 partial sums); 0 where it would not.  Nothing in it has to be set. */
vsa_status vsa_linear_workspace_size(vsa_plan plan, int B, int64_t N, int C, int O, size_t* bytes);

/* y = residual + act(x w^T + bias).  fp32 accumulation and epilogue, one
 * rounding to bf16; pre is rounded on its own.  C and O are multiples of 8.  y
 * and pre must not overlap x or w.  ws: at least vsa_linear_workspace_size bytes,
 * or NULL: the same result up to fp32 summation order, without the split. */
vsa_status vsa_linear(vsa_plan plan, const vsa_linear_args* args, void* ws, size_t ws_bytes,
                      void* stream);

typedef struct vsa_linear_grad_args {
  int32_t B, x_heads, C, y_heads, O;
  int64_t N;
  vsa_view dy;         /* gradient of x w^T + bias (see vsa_act_backward)          */
  vsa_view x;          /* the forward's input (read for dw)                        */
  const void* w;
  vsa_view x_pre;      /* laid out as x, or ptr = NULL; with it x = x_act(x_pre)   */
  int32_t x_act;
  vsa_view dx;         /* laid out as x, or ptr = NULL                             */
  void* dw;            /* bf16 [O,C], or NULL                                      */
  float* db;           /* fp32 [O], or NULL                                        */
  vsa_view dx_add;     /* laid out as x, or ptr = NULL: added to dx                */
} vsa_linear_grad_args;

/* Bytes of workspace of vsa_linear_backward.  Nothing in it has to be set. */
vsa_status vsa_linear_backward_workspace_size(vsa_plan plan, int B, int64_t N, int C, int O,
                                              size_t* bytes);

/* dx = dy w, times x_act'(x_pre) when x_pre is given (the gradient then goes
 * through the activation that made x, in the product's epilogue), or plus dx_add
 * (what reaches x by another way, a residual connection for instance; dx_add may be dx
 * itself, and does not go with x_pre);
 * dw = dy^T x, db = column sums of dy.  fp32 accumulation in a fixed order.  The tensor core
 * cuts the products' sums to fp32 and does not round them: over 33,920 rows dw comes out some 3e-5 of
 * itself too small, a fraction of its rounding to bf16 (2^-9 to 2^-8).  The
 * gradient of vsa_linear's residual is dy of its output itself.  With no rows dw
 * and db are 0. */
vsa_status vsa_linear_backward(vsa_plan plan, const vsa_linear_grad_args* args, void* ws,
                               size_t ws_bytes, void* stream);

/* out = dy * act'(pre), n bf16 elements each (n a multiple of 8), contiguous; out may
 * be dy or pre itself.  What is left of an activation's backward where its output does
 * not go into vsa_linear (there x_pre does it in the product's epilogue). */
vsa_status vsa_act_backward(vsa_plan plan, const void* dy, const void* pre, int act, void* out,
                            int64_t n, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VSA_BLOCK_H_ */
