// Head norm and rotary positions in one pass over Q, K (and V): natural order, or
// fused with the permute and the tile means of the layer's step 1, and the
// backward of both.
//
//   z = x r gain,  r = 1/sqrt(mean(x^2) + eps);   y = R z
//   g = R^T dy;  u = x r;  dx = r (g gain - u mean(g gain u));  d_gain = sum g u
//
// HBM-bound: a row is D bf16 (128 or 256 bytes), read once and written once.
// One warp takes an item (a head's tile, or a run of rows in natural order);
// D/8 lanes share a row, each with 8 channels in registers, and the row's sums
// go through shuffles among them.  Items run head by head for the same rows, so
// that the warps of a block use the same rows of the (cos, sin) tables, which then
// come from L1, and so that a [B,N,H,D] input is read along its memory.
//
// A lane's 8 channels are four pairs of the rotation: 8c .. 8c+7 where pairs are
// neighbours, and 4c .. 4c+3 with P+4c .. P+4c+3 where they are halves (two 8-byte
// accesses in place of one of 16 bytes, and no exchange between lanes).
#include <algorithm>

#include "block_internal.h"
#include "sm100.cuh"

namespace vsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kU = 8;                 // rows in flight per lane

struct RopeArgs {
  const float2* tab;
  const int4* tok;
  int P, start1, start2;
  float sign;                         // -1: R^T in place of R
};

struct FwdArgs {
  HeadTensorArgs t[VSA_MAX_HEAD_TENSORS];
  RopeArgs rope;
  const int32_t* row_src;
  const int32_t* block_len;
  int64_t N;
  int H, T, R;                        // items per batch element: T of R rows
  unsigned n_items;
  float eps;
};

struct BwdArgs {
  HeadGradArgs t[VSA_MAX_HEAD_TENSORS];
  RopeArgs rope;
  const int32_t* row_src;
  const int32_t* block_len;
  int64_t N;
  int H, T, R;
  unsigned n_items;
  float eps;
  float* partial;                     // [n][gridDim.x][D]
};

// Not .nc: in-place calls write what other lanes of the launch read.
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  using sm100::pack_bf16;
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// The channels of a lane and the pairs they make.
template <int kD, bool kHalves>
struct Lane {
  int o0, o1;        // first channel of each half of the lane's eight
  int p0;            // first pair
  int n_rot;         // how many of its four pairs turn
  __device__ __forceinline__ Lane(int c, int P) {
    p0 = 4 * c;
    if (kHalves) {
      const bool rot = p0 < P;
      o0 = rot ? p0 : 2 * P + 8 * (c - P / 4);
      o1 = rot ? P + p0 : o0 + 4;
      n_rot = rot ? 4 : 0;
    } else {
      o0 = 8 * c;
      o1 = o0 + 4;
      n_rot = min(4, max(0, P - p0));
    }
  }
  __device__ __forceinline__ uint4 load(const uint16_t* row) const {
    if (!kHalves) return load16(row + o0);
    const uint2 a = load8(row + o0), b = load8(row + o1);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void store(uint16_t* row, const uint4& v) const {
    if (!kHalves) {
      *reinterpret_cast<uint4*>(row + o0) = v;
    } else {
      *reinterpret_cast<uint2*>(row + o0) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(row + o1) = make_uint2(v.z, v.w);
    }
  }
  __device__ __forceinline__ void store_f32(float* row, const float (&f)[8]) const {
    *reinterpret_cast<float4*>(row + o0) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(row + o1) = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void load_gain(const void* gain, int f32, float (&g)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = (i < 4 ? o0 + i : o1 + i - 4);
      g[i] = gain == nullptr ? 1.0f
             : f32          ? __ldg(static_cast<const float*>(gain) + d)
                            : __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(gain) + d)) << 16);
    }
  }
  // Turn f by the token's angles.
  __device__ __forceinline__ void rotate(const RopeArgs& a, int64_t token, float (&f)[8]) const {
    if (n_rot == 0) return;
    const int4 off = __ldg(a.tok + token);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= n_rot) break;
      const int p = p0 + i;
      const int base = p < a.start1 ? off.x : (p < a.start2 ? off.y : off.z);
      const float2 cs = __ldg(a.tab + base + p);
      const float s = a.sign * cs.y;
      float& u = f[kHalves ? i : 2 * i];
      float& v = f[kHalves ? i + 4 : 2 * i + 1];
      const float t = fmaf(u, cs.x, -v * s);
      v = fmaf(u, s, v * cs.x);
      u = t;
    }
  }
};

template <int kCpr>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 1; off < kCpr; off <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}

template <int kD, bool kHalves, bool kTiled>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int kCpr = kD / 8, kRpp = 32 / kCpr;
  const HeadTensorArgs& t = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const Lane<kD, kHalves> ln(lane % kCpr, a.rope.P);
  const int sub = lane / kCpr;
  float gain[8];
  ln.load_gain(t.gain, t.gain_f32, gain);
  const bool plain = !t.norm && !t.rotate;
  for (unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5); item < a.n_items;
       item += gridDim.x * kWarps) {
    const unsigned h = item % a.H, bt = item / a.H;
    const unsigned ti = bt % a.T, b = bt / a.T;
    const int64_t first = int64_t(ti) * a.R;
    const int n = kTiled ? __ldg(a.block_len + ti) : int(min(int64_t(a.R), a.N - first));
    const uint16_t* x = t.x + b * t.xb + h * t.xh;
    uint16_t* y = kTiled ? t.y + ((int64_t(b) * a.H + h) * a.T + ti) * a.R * kD
                         : t.y + b * t.yb + h * t.yh;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int rows = kTiled ? a.R : n;
    for (int r0 = 0; r0 < rows; r0 += kRpp * kU) {
      uint4 raw[kU];
      int32_t src[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int r = r0 + u * kRpp + sub;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        src[u] = -1;
        if (r < n) {
          src[u] = kTiled ? __ldg(a.row_src + first + r) : int32_t(first + r);
          raw[u] = ln.load(x + int64_t(src[u]) * t.xn);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int r = r0 + u * kRpp + sub;
        float f[8];
        unpack(raw[u], f);
        if (t.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
          const float rs = rsqrtf(fmaf(row_sum<kCpr>(ss), 1.0f / kD, a.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= rs * gain[i];
        }
        if (t.rotate && src[u] >= 0) ln.rotate(a.rope, src[u], f);
        if (kTiled) {
          if (r < n) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
          }
          if (r < rows) ln.store(y + int64_t(r) * kD, plain ? raw[u] : pack(f));
        } else if (r < n) {
          ln.store(y + int64_t(src[u]) * t.yn, plain ? raw[u] : pack(f));
        }
      }
    }
    if (kTiled) {
#pragma unroll
      for (int off = kCpr; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], off);
      if (sub == 0) {
        const float inv = 1.0f / float(n);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] *= inv;
        ln.store_f32(t.pooled + ((int64_t(b) * a.H + h) * a.T + ti) * kD, acc);
      }
    }
  }
}

template <int kD, bool kHalves, bool kTiled>
__global__ void __launch_bounds__(kThreads)
    norm_rope_backward_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int kCpr = kD / 8, kRpp = 32 / kCpr;
  constexpr int kUb = kU / 2;         // two tensors are read, so half the rows in flight
  const HeadGradArgs& t = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const Lane<kD, kHalves> ln(lane % kCpr, a.rope.P);
  const int sub = lane / kCpr;
  float gain[8], dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  ln.load_gain(t.gain, t.gain_f32, gain);
  const bool plain = !t.norm && !t.rotate;
  for (unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5); item < a.n_items;
       item += gridDim.x * kWarps) {
    const unsigned h = item % a.H, bt = item / a.H;
    const unsigned ti = bt % a.T, b = bt / a.T;
    const int64_t first = int64_t(ti) * a.R;
    const int n = kTiled ? __ldg(a.block_len + ti) : int(min(int64_t(a.R), a.N - first));
    const uint16_t* x = t.x + b * t.xb + h * t.xh;
    const uint16_t* dy = kTiled ? t.dy + ((int64_t(b) * a.H + h) * a.T + ti) * a.R * kD
                                : t.dy + b * t.gb + h * t.gh;
    uint16_t* dx = t.dx + b * t.db + h * t.dh;
    for (int r0 = 0; r0 < n; r0 += kRpp * kUb) {
      uint4 rg[kUb], rx[kUb];
      int32_t src[kUb];
#pragma unroll
      for (int u = 0; u < kUb; ++u) {
        const int r = r0 + u * kRpp + sub;
        rg[u] = rx[u] = make_uint4(0u, 0u, 0u, 0u);
        src[u] = -1;
        if (r < n) {
          src[u] = kTiled ? __ldg(a.row_src + first + r) : int32_t(first + r);
          rg[u] = ln.load(dy + (kTiled ? int64_t(r) * kD : int64_t(src[u]) * t.gn));
          if (t.norm) rx[u] = ln.load(x + int64_t(src[u]) * t.xn);
        }
      }
#pragma unroll
      for (int u = 0; u < kUb; ++u) {
        float g[8];
        unpack(rg[u], g);
        if (t.rotate && src[u] >= 0) ln.rotate(a.rope, src[u], g);
        if (t.norm) {
          // with r = 1/sqrt(mean(x^2) + eps): sum of g gain u = r * (sum of g gain x)
          float f[8], ss = 0.f, gx = 0.f;
          unpack(rx[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(f[i], f[i], ss);
            gx = fmaf(g[i] * gain[i], f[i], gx);
          }
          const float rs = rsqrtf(fmaf(row_sum<kCpr>(ss), 1.0f / kD, a.eps));
          const float m = row_sum<kCpr>(gx) * rs * (1.0f / kD);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float un = f[i] * rs;
            dw[i] = fmaf(g[i], un, dw[i]);
            g[i] = rs * fmaf(-un, m, g[i] * gain[i]);
          }
        }
        if (src[u] >= 0) ln.store(dx + int64_t(src[u]) * t.dn, plain ? rg[u] : pack(g));
      }
    }
  }
  if (t.d_gain == nullptr) return;
  // the block's sum, by lanes of a channel first and then by warps, in a fixed order
  __shared__ float part[kWarps][kD];
#pragma unroll
  for (int off = kCpr; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] += __shfl_xor_sync(0xFFFFFFFFu, dw[i], off);
  if (sub == 0) ln.store_f32(part[threadIdx.x >> 5], dw);
  __syncthreads();
  if (threadIdx.x < kD) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
    a.partial[(int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kD + threadIdx.x] = s;
  }
}

struct GainOut {
  float* d_gain[VSA_MAX_HEAD_TENSORS];
};

// d_gain[c] = sum over the blocks' partial sums, in block order per thread row and then by
// rows: one block for 32 channels of a tensor.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const float* partial, int blocks, int D,
                                                        const GainOut out) {
  __shared__ float part[32][33];
  float* d = out.d_gain[blockIdx.y];
  if (d == nullptr) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const float* p = partial + int64_t(blockIdx.y) * blocks * D + c;
  float s = 0.f;
#pragma unroll 8
  for (int i = row; i < blocks; i += 32) s += p[int64_t(i) * D];
  part[row][threadIdx.x & 31] = s;
  __syncthreads();
  if (row == 0) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += part[i][threadIdx.x];
    d[c] = v;
  }
}

int max_blocks(const vsa_plan_s* p) { return (p->num_sms > 0 ? p->num_sms : 148) * 8; }

RopeArgs rope_args(const vsa_rope_s* r, int inverse) {
  RopeArgs a = {};
  a.sign = inverse ? -1.0f : 1.0f;
  if (r != nullptr) {
    a.tab = r->d_tab;
    a.tok = r->d_tok;
    a.P = r->P;
    a.start1 = r->start1;
    a.start2 = r->start2;
  }
  return a;
}

// Rows of an item and items per batch element.
template <class Args>
bool set_items(Args* a, const vsa_plan_s* p, bool tiled, int natural_rows, int B, int H) {
  a->row_src = p->d_row_src;
  a->block_len = p->d_block_len;
  a->N = p->n_tokens;
  a->H = H;
  a->R = tiled ? p->R : natural_rows;
  const int64_t T = tiled ? p->n_tiles : (p->n_tokens + a->R - 1) / a->R;
  a->T = int(T);
  const int64_t items = int64_t(B) * H * T;
  a->n_items = unsigned(items);
  return items < (int64_t(1) << 31);
}

}  // namespace

vsa_status launch_norm_rope(const vsa_plan_s* p, const vsa_rope_s* rope, const HeadTensorArgs* t,
                            int n, float eps, int inverse, bool tiled, int B, int H, int D,
                            cudaStream_t stream) {
  FwdArgs a = {};
  for (int i = 0; i < n; ++i) a.t[i] = t[i];
  a.rope = rope_args(rope, inverse);
  a.eps = eps;
  if (!set_items(&a, p, tiled, kU * 256 / D, B, H))
    return fail(VSA_ERR_UNSUPPORTED, "too many heads and rows for one launch");
  const int64_t want = (int64_t(a.n_items) + kWarps - 1) / kWarps;
  const dim3 grid(unsigned(std::min<int64_t>(want, max_blocks(p))), unsigned(n));
  const bool halves = rope != nullptr && rope->halves;
#define VSA_LAUNCH(DD, HV, TL) norm_rope_kernel<DD, HV, TL><<<grid, kThreads, 0, stream>>>(a)
#define VSA_PICK(DD)                                                     \
  (halves ? (tiled ? (VSA_LAUNCH(DD, true, true), 0) : (VSA_LAUNCH(DD, true, false), 0)) \
          : (tiled ? (VSA_LAUNCH(DD, false, true), 0) : (VSA_LAUNCH(DD, false, false), 0)))
  if (D == 128)
    (void)VSA_PICK(128);
  else
    (void)VSA_PICK(64);
#undef VSA_PICK
#undef VSA_LAUNCH
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK
                          : fail(VSA_ERR_CUDA, std::string("norm_rope launch: ") + cudaGetErrorString(e));
}

size_t norm_rope_backward_bytes(const vsa_plan_s* p, int n, int D) {
  return size_t(n) * size_t(max_blocks(p)) * size_t(D) * sizeof(float);
}

vsa_status launch_norm_rope_backward(const vsa_plan_s* p, const vsa_rope_s* rope,
                                     const HeadGradArgs* t, int n, float eps, bool tiled, int B,
                                     int H, int D, void* ws, cudaStream_t stream) {
  BwdArgs a = {};
  bool gains = false;
  GainOut out = {};
  for (int i = 0; i < n; ++i) {
    a.t[i] = t[i];
    out.d_gain[i] = t[i].d_gain;
    gains = gains || t[i].d_gain != nullptr;
  }
  a.rope = rope_args(rope, 1);
  a.eps = eps;
  a.partial = static_cast<float*>(ws);
  if (!set_items(&a, p, tiled, kU * 256 / D, B, H))
    return fail(VSA_ERR_UNSUPPORTED, "too many heads and rows for one launch");
  const int64_t want = (int64_t(a.n_items) + kWarps - 1) / kWarps;
  const dim3 grid(unsigned(std::min<int64_t>(want, max_blocks(p))), unsigned(n));
  const bool halves = rope != nullptr && rope->halves;
#define VSA_LAUNCH(DD, HV, TL) norm_rope_backward_kernel<DD, HV, TL><<<grid, kThreads, 0, stream>>>(a)
#define VSA_PICK(DD)                                                     \
  (halves ? (tiled ? (VSA_LAUNCH(DD, true, true), 0) : (VSA_LAUNCH(DD, true, false), 0)) \
          : (tiled ? (VSA_LAUNCH(DD, false, true), 0) : (VSA_LAUNCH(DD, false, false), 0)))
  if (D == 128)
    (void)VSA_PICK(128);
  else
    (void)VSA_PICK(64);
#undef VSA_PICK
#undef VSA_LAUNCH
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && gains) {
    gain_sum_kernel<<<dim3(D / 32, n), 1024, 0, stream>>>(a.partial, int(grid.x), D, out);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? VSA_OK
                          : fail(VSA_ERR_CUDA, std::string("norm_rope backward launch: ") + cudaGetErrorString(e));
}

}  // namespace vsa
