// Head norm and rotary positions in one pass over Q, K (and V): natural order, or
// fused with the permute and the tile means of the layer's step 1, and the
// backward of both.
//
//   z = x r gain,  r = 1/sqrt(mean(x^2) + eps);   y = R z
//   g = R^T dy;  u = x r;  dx = r (g gain - u mean(g gain u));  d_gain = sum g u
//
// HBM-bound: a row is D bf16 (128 or 256 bytes), read once and written once.
// D/8 lanes share a row, each with 8 channels in registers, and the row's sums go
// through shuffles among them.  A block takes a run of rows (a tile, or rows in natural
// order) for a group of heads: a lane keeps the cosines and sines of its rows in
// registers and walks the heads.  The rows of the next heads are on their way meanwhile:
// each lane copies its own chunks into slots of shared memory that it alone reads, so that
// kStages heads are in flight with no register held and no barrier.
//
// A lane's 8 channels are four pairs of the rotation: 8c .. 8c+7 where pairs are
// neighbours, and 4c .. 4c+3 with P+4c .. P+4c+3 where they are halves (two 8-byte
// accesses in place of one of 16 bytes, and no exchange between lanes).
//
// Measured (B200, device time of a pass replayed from a graph, share of the measured 6,549 GB/s copy
// rate; in brackets called one after another through the binding, inputs changing): Q, K and V of 104,704
// tokens x 42 heads into tiles with their means 1,091-1,135 us (6.81 GB, 92-95 %; [1,155]); the rotation
// alone of 33,920 x 42 on a [B,N,H,D] tensor 116 us (96 %; [125]); the backward of Q, K and V there
// 459-468 us (95-97 %; [497]); Q and K of 9,772 x 8 out of one [B,N,3,H,D] projection 17.8 us (80 MB, 69 %:
// start and end of so short a kernel; [18.8]); two heads of 366 tokens 2.4 us (launch; [9.9], host time);
// the backward of three tensors of a ragged batch 6.9 us ([31.5], host time).  A warp per tile and head with its loads in registers, which
// looked the angles up for every row and head, took 2,031, 252, 815, 39 and 8 us.
#include <algorithm>
#include <cmath>

#include "block_internal.h"
#include "sm100.cuh"

namespace vsa {
namespace {

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
  int H, T, R;                        // heads; row blocks (tiles) of a batch element, tile rows
  int group, groups;                  // heads of an item, items of a row block
  float eps;
};

struct BwdArgs {
  HeadGradArgs t[VSA_MAX_HEAD_TENSORS];
  RopeArgs rope;
  const int32_t* row_src;
  int64_t rows;                       // rows of dy (padded in tile order)
  int H, T, group, groups;
  unsigned n_items;
  float eps;
  float* partial;                     // [n][gridDim.x][D]
};

// Copies into shared memory that wait for no register; zeros where the row is not there.
__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t* p, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint16_t* p, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(p), "r"(live ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 slot_load(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
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
  __device__ __forceinline__ void fetch(uint32_t slot, const uint16_t* row, bool live) const {
    if (!kHalves) {
      copy16(slot, row + o0, live);
    } else {
      copy8(slot, row + o0, live);
      copy8(slot + 8, row + o1, live);
    }
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
  // The lane's own place in shared memory: f, added to what an earlier pass left there.
  __device__ __forceinline__ void add_f32(float* row, float (&f)[8], bool add) const {
    if (add) {
      const float4 a = *reinterpret_cast<const float4*>(row + o0);
      const float4 b = *reinterpret_cast<const float4*>(row + o1);
      f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
      f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
    }
    store_f32(row, f);
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
  // The four (cos, sin) of a token; (1, 0) where the pair does not turn.
  __device__ __forceinline__ void angles(const RopeArgs& a, int32_t token, float2 (&cs)[4]) const {
    const int4 off = n_rot > 0 && token >= 0 ? __ldg(a.tok + token) : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = make_float2(1.0f, 0.0f);
      if (i < n_rot && token >= 0) {
        const int p = p0 + i;
        cs[i] = __ldg(a.tab + (p < a.start1 ? off.x : (p < a.start2 ? off.y : off.z)) + p);
        cs[i].y *= a.sign;
      }
    }
  }
  static __device__ __forceinline__ void rotate(const float2 (&cs)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& u = f[kHalves ? i : 2 * i];
      float& v = f[kHalves ? i + 4 : 2 * i + 1];
      const float t = fmaf(u, cs[i].x, -v * cs[i].y);
      v = fmaf(u, cs[i].y, v * cs[i].x);
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

// Rows of a block: kThreads / (D/8) at a time, kU of them in each lane.
template <int kD, int kThreads, int kU>
struct Block {
  static constexpr int kCpr = kD / 8, kRpp = 32 / kCpr, kWarps = kThreads / 32;
  static constexpr int kPass = kWarps * kRpp;      // rows side by side
  static constexpr int kRows = kPass * kU;
  static constexpr uint32_t kStage = kThreads * kU * 16;   // slots of one tensor's rows
};
// Heads in flight.  With two the tiles take 1,125 us in place of 1,101; with four only one block of
// the backward fits an SM (550 us in place of 460).
constexpr int kStages = 3;
// Heads of an item of the forward, at most.  Tiles: their column sums (4 KB a head of 128 channels,
// 64 KB) and the slots (48 KB) leave room for two blocks on an SM.  Natural order: 42 x 33,920 take 116.7 us
// with 14, 118.7 with 21 and 123.6 with all heads an item.
constexpr int kMaxGroup = 16;
constexpr int kGradRows = 64;         // rows of an item of the backward

template <int kD, bool kHalves, bool kTiled, int kThreads, int kU>
__global__ void __launch_bounds__(kThreads, kTiled ? 2 : 6)
    norm_rope_kernel(const __grid_constant__ FwdArgs a) {
  using Bl = Block<kD, kThreads, kU>;
  constexpr int kCpr = Bl::kCpr;
  extern __shared__ __align__(16) uint8_t slots[];
  // tiles: the column sums of each head and warp
  float* part = reinterpret_cast<float*>(slots + kStages * Bl::kStage);
  const HeadTensorArgs& t = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<kD, kHalves> ln(lane % kCpr, a.rope.P);
  const unsigned g = blockIdx.x % a.groups, bt = blockIdx.x / a.groups;
  const unsigned ti = bt % a.T, b = bt / a.T;
  const int h0 = g * a.group, h1 = min(a.H, h0 + a.group);
  const int R = kTiled ? a.R : Bl::kRows;          // rows of the item, kRows at a time
  const int64_t first = int64_t(ti) * R;
  const int n = kTiled ? __ldg(a.block_len + ti) : int(min(int64_t(R), a.N - first));
  const uint32_t slot = sm100::smem_u32(slots) + threadIdx.x * 16;
  const bool plain = !t.norm && !t.rotate;
  float gain[8];
  ln.load_gain(t.gain, t.gain_f32, gain);
  for (int base = 0; base < R; base += Bl::kRows) {
    const int r0 = base + warp * Bl::kRpp + lane / kCpr;   // this lane's rows: r0 + u * kPass
    int32_t src[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = r0 + u * Bl::kPass;
      src[u] = r >= n ? -1 : kTiled ? __ldg(a.row_src + first + r) : int32_t(first + r);
    }
    const uint16_t* x = t.x + b * t.xb + h0 * t.xh;
    uint32_t in = 0, out = 0;                      // stage of the next fetch, of the next head
    int hf = h0;                                   // head of the next fetch
    const auto fetch = [&]() {
      if (hf < h1) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
          ln.fetch(slot + in * Bl::kStage + u * kThreads * 16, x + max(src[u], 0) * t.xn, src[u] >= 0);
        x += t.xh;
        ++hf;
      }
      copy_commit();                               // a group a step, empty at the end
      in = in + 1 == kStages ? 0 : in + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
    float2 cs[kU][4];
    if (t.rotate) {
#pragma unroll
      for (int u = 0; u < kU; ++u) ln.angles(a.rope, src[u], cs[u]);
    }
    uint16_t* y = kTiled ? t.y + (((int64_t(b) * a.H + h0) * a.T + ti) * R + r0) * kD
                         : t.y + b * t.yb + h0 * t.yh;
    const int64_t y_head = kTiled ? int64_t(a.T) * R * kD : t.yh;
    for (int h = h0; h < h1; ++h) {
      fetch();
      copy_wait<kStages - 1>();
      uint4 raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) raw[u] = slot_load(slot + out * Bl::kStage + u * kThreads * 16);
      out = out + 1 == kStages ? 0 : out + 1;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < kU; ++u) {
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
        if (t.rotate) ln.rotate(cs[u], f);
        if (kTiled) {
          // pad rows are zeros, whatever the gain
          if (src[u] >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
          }
          ln.store(y + u * (Bl::kPass * kD), plain || src[u] < 0 ? raw[u] : pack(f));
        } else if (src[u] >= 0) {
          ln.store(y + src[u] * t.yn, plain ? raw[u] : pack(f));
        }
      }
      y += y_head;
      if (kTiled && t.pooled != nullptr) {
#pragma unroll
        for (int off = kCpr; off < 32; off <<= 1)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], off);
        if (lane < kCpr) ln.add_f32(part + ((h - h0) * Bl::kWarps + warp) * kD, acc, base > 0);
      }
    }
  }
  if (kTiled && t.pooled != nullptr) {
    // the tile's means: the warps' sums, a head after the other
    __syncthreads();
    const float inv = 1.0f / float(n);
    for (int i = threadIdx.x; i < (h1 - h0) * kD; i += kThreads) {
      const int h = i / kD, d = i % kD;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < Bl::kWarps; ++w) s += part[(h * Bl::kWarps + w) * kD + d];
      t.pooled[((int64_t(b) * a.H + h0 + h) * a.T + ti) * kD + d] = s * inv;
    }
  }
}

template <int kD, bool kHalves, bool kTiled, int kThreads, int kU>
__global__ void __launch_bounds__(kThreads, 512 / kThreads)
    norm_rope_backward_kernel(const __grid_constant__ BwdArgs a) {
  using Bl = Block<kD, kThreads, kU>;
  constexpr int kCpr = Bl::kCpr;
  extern __shared__ __align__(16) uint8_t slots[];
  const HeadGradArgs& t = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<kD, kHalves> ln(lane % kCpr, a.rope.P);
  const int r0 = warp * Bl::kRpp + lane / kCpr;
  float gain[8], dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  ln.load_gain(t.gain, t.gain_f32, gain);
  const bool plain = !t.norm && !t.rotate;
  const uint32_t slot = sm100::smem_u32(slots) + threadIdx.x * 16;
  uint32_t in = 0, out = 0;
  for (unsigned item = blockIdx.x; item < a.n_items; item += gridDim.x) {
    const unsigned g = item % a.groups, bt = item / a.groups;
    const unsigned ti = bt % a.T, b = bt / a.T;
    const int h0 = g * a.group, h1 = min(a.H, h0 + a.group);
    const int64_t first = int64_t(ti) * Bl::kRows;
    int32_t src[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t r = first + r0 + u * Bl::kPass;
      src[u] = r >= a.rows ? -1 : kTiled ? __ldg(a.row_src + r) : int32_t(r);
    }
    // dy of row u: at tile row first + r, or at the token
    const uint16_t* dy = kTiled ? t.dy + ((int64_t(b) * a.H + h0) * a.rows + first) * kD
                                : t.dy + b * t.gb + h0 * t.gh;
    const int64_t dy_head = kTiled ? a.rows * kD : t.gh;
    const uint16_t* x = t.x + b * t.xb + h0 * t.xh;
    uint16_t* dx = t.dx + b * t.db + h0 * t.dh;
    int hf = h0;
    const auto fetch = [&]() {
      if (hf < h1) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const uint32_t s = slot + in * (2 * Bl::kStage) + u * kThreads * 16;
          const bool live = src[u] >= 0;
          const int64_t row = max(src[u], 0);
          ln.fetch(s, kTiled ? dy + (live ? (r0 + u * Bl::kPass) * kD : 0) : dy + row * t.gn, live);
          if (t.norm) ln.fetch(s + Bl::kStage, x + row * t.xn, live);
        }
        dy += dy_head;
        x += t.xh;
        ++hf;
      }
      copy_commit();
      in = in + 1 == kStages ? 0 : in + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
    float2 cs[kU][4];
    if (t.rotate) {
#pragma unroll
      for (int u = 0; u < kU; ++u) ln.angles(a.rope, src[u], cs[u]);
    }
    for (int h = h0; h < h1; ++h) {
      fetch();
      copy_wait<kStages - 1>();
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t s = slot + out * (2 * Bl::kStage) + u * kThreads * 16;
        const uint4 rg = slot_load(s);
        float gr[8];
        unpack(rg, gr);
        if (t.rotate) ln.rotate(cs[u], gr);
        if (t.norm) {
          // with r = 1/sqrt(mean(x^2) + eps): sum of g gain u = r * (sum of g gain x)
          float f[8], ss = 0.f, gx = 0.f;
          unpack(slot_load(s + Bl::kStage), f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(f[i], f[i], ss);
            gx = fmaf(gr[i] * gain[i], f[i], gx);
          }
          const float rs = rsqrtf(fmaf(row_sum<kCpr>(ss), 1.0f / kD, a.eps));
          const float m = row_sum<kCpr>(gx) * rs * (1.0f / kD);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float un = f[i] * rs;
            dw[i] = fmaf(gr[i], un, dw[i]);
            gr[i] = rs * fmaf(-un, m, gr[i] * gain[i]);
          }
        }
        if (src[u] >= 0) ln.store(dx + src[u] * t.dn, plain ? rg : pack(gr));
      }
      out = out + 1 == kStages ? 0 : out + 1;
      dx += t.dh;
    }
    // the item's last fetches brought nothing; the stages go on from here
    in = out;
  }
  if (t.d_gain == nullptr) return;
  // the block's sum, by lanes of a channel first and then by warps, in a fixed order
  __shared__ float part[Bl::kWarps][kD];
#pragma unroll
  for (int off = kCpr; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] += __shfl_xor_sync(0xFFFFFFFFu, dw[i], off);
  if (lane < kCpr) ln.store_f32(part[warp], dw);
  __syncthreads();
  if (threadIdx.x < kD) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < Bl::kWarps; ++w) s += part[w][threadIdx.x];
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

int sms(const vsa_plan_s* p) { return p->num_sms > 0 ? p->num_sms : 148; }
// Blocks of a tensor in the backward, at most: two of 256 threads an SM.
int max_blocks(const vsa_plan_s* p) { return sms(p) * 2; }

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

// Heads of an item, at most max_group: an item costs its heads and a start of about two more (its
// rows' indices and angles, and the first heads' way from memory).  Two blocks an SM with
// their items in step come in waves of `slots`: the group that makes the waves shortest (one head an
// item: small layer 41 us, eight: 27 us; all 42 heads an item or a sixteenth of the waves: 1,186 and
// 1,318 us at 104,704 tokens).  Six (natural order) share the memory whatever the wave, and the
// last items cost a third of their heads: Q and K of 8 x 9,772 36.2, 24.6, 19.2 and 17.1 us with one, two,
// four and eight heads an item (by whole waves it would be four), 42 x 700 15.3 with one, 8.7
// with six and 16.0 with 42.
template <class Args>
bool set_items(Args* a, const vsa_plan_s* p, int64_t row_blocks, int B, int H, int n, int64_t slots,
               int max_group, bool in_step, int64_t* items) {
  a->row_src = p->d_row_src;
  a->H = H;
  a->T = int(row_blocks);
  double least = 1e300;
  for (int g = 1; g <= std::min(H, max_group); ++g) {
    const int64_t groups = (H + g - 1) / g;
    const double waves = double(int64_t(B) * row_blocks * n * groups) / double(slots);
    const double cost = in_step ? std::ceil(waves) * (g + 2) : waves * (g + 2.3) + 0.35 * g;
    if (cost < least) {
      least = cost;
      a->group = g;
      a->groups = int(groups);
    }
  }
  *items = int64_t(B) * row_blocks * a->groups;
  return *items < (int64_t(1) << 31) && row_blocks < (int64_t(1) << 31);
}

// smem: this call's shared memory; most: the most that any call of the kernel takes.  The leave is the
// function's, not the call's: every thread asks for the same, so that none takes from another's
// between its leave and its launch.
template <class Kernel, class Args>
cudaError_t launch(Kernel k, int64_t items, int n, int threads, uint32_t smem, uint32_t most, const Args& a,
                   cudaStream_t stream) {
  // 48 KB need no leave, less the 4 KB a kernel has besides
  if (most > 44 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
    if (e != cudaSuccess) return e;
  }
  k<<<dim3(unsigned(items), unsigned(n)), threads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

vsa_status launch_norm_rope(const vsa_plan_s* p, const vsa_rope_s* rope, const HeadTensorArgs* t,
                            int n, float eps, int inverse, bool tiled, int B, int H, int D,
                            cudaStream_t stream) {
  FwdArgs a = {};
  for (int i = 0; i < n; ++i) a.t[i] = t[i];
  a.rope = rope_args(rope, inverse);
  a.eps = eps;
  a.block_len = p->d_block_len;
  a.N = p->n_tokens;
  // rows of an item: a tile, or 16 (32 of 64 channels) in natural order, where a row a lane leaves room
  // for six blocks an SM (two rows and four blocks: 123 us in place of 116 at 33,920 x 42)
  const int64_t row_blocks = tiled ? p->n_tiles : (p->n_tokens + 2048 / D - 1) / (2048 / D);
  a.R = p->R;
  int64_t items = 0;
  if (!set_items(&a, p, row_blocks, B, H, n, int64_t(sms(p)) * (tiled ? 2 : 6), kMaxGroup, tiled, &items))
    return fail(VSA_ERR_UNSUPPORTED, "too many heads and rows for one launch");
  const bool halves = rope != nullptr && rope->halves;
  cudaError_t e;
#define VSA_LAUNCH(DD, TL, U)                                                                     \
  {                                                                                               \
    static_assert(Block<DD, 256, U>::kRows == (TL ? 64 : 2048 / DD), "rows of a pass or an item"); \
    const uint32_t rows = kStages * Block<DD, 256, U>::kStage, head = TL ? 8 * DD * 4 : 0;        \
    const uint32_t smem = rows + a.group * head, most = rows + kMaxGroup * head;                  \
    e = halves ? launch(norm_rope_kernel<DD, true, TL, 256, U>, items, n, 256, smem, most, a, stream)   \
               : launch(norm_rope_kernel<DD, false, TL, 256, U>, items, n, 256, smem, most, a, stream); \
  }
  if (D == 128) {
    if (tiled)
      VSA_LAUNCH(128, true, 4)
    else
      VSA_LAUNCH(128, false, 1)
  } else {
    if (tiled)
      VSA_LAUNCH(64, true, 2)
    else
      VSA_LAUNCH(64, false, 1)
  }
#undef VSA_LAUNCH
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
  a.rows = tiled ? p->n_padded : p->n_tokens;
  int64_t items = 0;
  if (!set_items(&a, p, (a.rows + kGradRows - 1) / kGradRows, B, H, n, max_blocks(p), H, true, &items))
    return fail(VSA_ERR_UNSUPPORTED, "too many heads and rows for one launch");
  a.n_items = unsigned(items);
  const int64_t blocks = std::min<int64_t>(items, max_blocks(p));
  const bool halves = rope != nullptr && rope->halves;
  cudaError_t e;
#define VSA_LAUNCH(DD, TL, U)                                                                 \
  {                                                                                           \
    static_assert(Block<DD, 256, U>::kRows == kGradRows, "rows of an item");                  \
    const uint32_t smem = 2 * kStages * Block<DD, 256, U>::kStage;                            \
    e = halves ? launch(norm_rope_backward_kernel<DD, true, TL, 256, U>, blocks, n, 256,      \
                        smem, smem, a, stream)                                                \
               : launch(norm_rope_backward_kernel<DD, false, TL, 256, U>, blocks, n, 256,     \
                        smem, smem, a, stream);                                               \
  }
  if (D == 128) {
    if (tiled)
      VSA_LAUNCH(128, true, 4)
    else
      VSA_LAUNCH(128, false, 4)
  } else {
    if (tiled)
      VSA_LAUNCH(64, true, 2)
    else
      VSA_LAUNCH(64, false, 2)
  }
#undef VSA_LAUNCH
  if (e == cudaSuccess && gains) {
    gain_sum_kernel<<<dim3(D / 32, n), 1024, 0, stream>>>(a.partial, int(blocks), D, out);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? VSA_OK
                          : fail(VSA_ERR_CUDA, std::string("norm_rope backward launch: ") + cudaGetErrorString(e));
}

}  // namespace vsa
