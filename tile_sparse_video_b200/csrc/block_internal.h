// Internal declarations of the operators of include/vsa_block.h.
#pragma once

#include <vector>

#include "../../include/vsa_block.h"
#include "vsa_internal.h"

// Rotation of a plan's tokens.  For every axis a the distinct positions of its
// tokens have one row of P_a = dim[a]/2 (cos, sin) entries in `tab`; a token
// holds, for each axis, the index of its row's first entry less the axis's
// first pair, so that pair p of axis a is tab[tok[n][a] + p].
struct vsa_rope_s {
  int device = -1;
  int64_t n_tokens = 0, n_prefix = 0;
  int grid[3] = {0, 0, 0};   // the plan's; (0, 0, 0) where it has no video tokens
  int P = 0;                 // rotated pairs
  int start1 = 0, start2 = 0;  // first pair of the height and the width axis
  int halves = 0;
  std::vector<float2> tab;   // host copies
  std::vector<int4> tok;
  float2* d_tab = nullptr;
  int4* d_tok = nullptr;
};

namespace vsa {

struct HeadTensorArgs {
  const uint16_t* x;
  int64_t xb, xh, xn;
  const void* gain;
  int gain_f32, norm, rotate;
  uint16_t* y;
  int64_t yb, yh, yn;
  float* pooled;
};

struct HeadGradArgs {
  const uint16_t* dy;
  int64_t gb, gh, gn;
  const uint16_t* x;
  int64_t xb, xh, xn;
  const void* gain;
  int gain_f32, norm, rotate;
  uint16_t* dx;
  int64_t db, dh, dn;
  float* d_gain;
};

// Forward; tiled: y in tile order with the plan's tables, pooled means; else
// natural order.  inverse turns the rotation back.
vsa_status launch_norm_rope(const vsa_plan_s* p, const vsa_rope_s* rope, const HeadTensorArgs* t,
                            int n, float eps, int inverse, bool tiled, int B, int H, int D,
                            cudaStream_t stream);
size_t norm_rope_backward_bytes(const vsa_plan_s* p, int n, int D);
vsa_status launch_norm_rope_backward(const vsa_plan_s* p, const vsa_rope_s* rope,
                                     const HeadGradArgs* t, int n, float eps, bool tiled, int B,
                                     int H, int D, void* ws, cudaStream_t stream);

// ws: linear_bytes of it, or NULL (the K blocks are then not split).
size_t linear_bytes(const vsa_plan_s* p, int B, int64_t N, int C, int O);
vsa_status launch_linear(const vsa_plan_s* p, const vsa_linear_args& a, void* ws, cudaStream_t stream);
size_t linear_backward_bytes(const vsa_plan_s* p, int B, int64_t N, int C, int O);
vsa_status launch_linear_backward(const vsa_plan_s* p, const vsa_linear_grad_args& a, void* ws,
                                  cudaStream_t stream);
cudaError_t launch_act_backward(const void* dy, const void* pre, int act, void* out, int64_t n,
                                int num_sms, cudaStream_t stream);

}  // namespace vsa
