// Linears with a fused epilogue and their gradients, one tcgen05 GEMM kernel in
// three operand orders:
//   forward   y  = residual + act(x w^T + bias)     A = x  [rows, C],  B = w [O, C]
//   dgrad     dx = (dy w) * act'(x_pre)             A = dy [rows, O],  B = w read along C
//   wgrad     dw = dy^T x                           A = dy read along O, B = x read along C,
//                                                   K = the rows
// "Read along" operands are MN-major for the tensor core: the same row-major
// tensors in memory, with no transposed copy.
//
// Tensors come as 4-D views [B, heads, N, D] (heads = 1: rows), so the products read
// and write head layouts and strided tensors through the TMA maps and the
// epilogue's addresses; a 64-column block never crosses a head (D is 64 or 128).
//
// Design: pairs of CTAs (a cluster of two SMs) over output tiles of 256 rows x 256 or 128
// columns, persistent.  Each CTA loads its half of the A rows and of the B columns of a
// 64-wide K block (16 + 16 KB, 128-byte swizzle) into a 6-stage ring by TMA; one lane of the
// leading CTA issues tcgen05.mma.cta_group::2, M = 256, for both; each CTA has its 128 rows of
// the accumulator in its own TMEM, twice (2 x 256 columns), so that the epilogue of a
// tile (biases, activations, residuals) runs under the products of the next.  Epilogue warps
// pass the accumulator through 2 KB of shared memory of their own, and read residuals and
// write results in whole 64-byte row pieces.
//
// Every wait is bounded (abort flag and status word); the pair meets at cluster
// barriers before its first and after its last signal.
//
// Measured (B200, device time of calls in a row or replayed from a graph): 33,920 x 5,376 -> 7,168 with
// bias, GELU and pre-activation out 1.77-2.02 ms = 1,295-1,477 TFLOP/s, the library's plain product of the
// same operands 1.65-1.9 ms in the same runs; both gradients 3.85-4.12 ms = 1,270-1,358.  The tensor pipe is active 99 % of the time (ncu) at the 1.1-1.25 GHz to which the 1 kW cap takes the
// clock: power bounds it.  2,048 x 5,376 x 5,376: 86 us forward, 77 us weight gradient (library 86-88 and 79).
// 9,772 x 1,024 -> 1,024 18.8 us (library 18.7), with bias and residual 21.7-22.9 (called through the
// binding 26.7).  On the way: one lane on the
// producer's and issuer's loops with divisions in them 1,050-1,250 TFLOP/s, whole warps without
// divisions 1,400-1,500; branches for every eight values and
// scalar arithmetic in the epilogue 45 us in place of 34 (4,096 x 1,024 -> 4,096, GELU); cluster-scope
// releases, which wait for a warp's stores, another 2 us.
#include <algorithm>

#include "block_internal.h"
#include "sm100.cuh"

namespace vsa {
namespace {
using namespace sm100;

constexpr int kBM = 256, kBK = 64, kStages = 6;
constexpr int kThreads = 320;                     // TMA, MMA, 8 epilogue warps
constexpr int kABytes = 128 * kBK * 2;            // a CTA's half of the A block
constexpr int kStageBytes = 2 * kABytes;          // and at most as much of B
constexpr int kMnAtom = 64 * kBK * 2;             // one 64-column x 64-row box
constexpr int kStaging = 8 * 32 * 64;             // each epilogue warp's 32 rows x 64 bytes
// full[S], empty[S], acc_full[2], acc_empty[2], drain
constexpr int kNBar = 2 * kStages + 5;
constexpr size_t kSmem = size_t(kStages) * kStageBytes + kStaging + 8 * 128 * 4 + kNBar * 8 + 16 + 1024;

enum Order { kForward = 0, kDgrad = 1, kWgrad = 2 };

// Column c of a view -> (head, channel).
struct Cols {
  int D;          // channels of a head (all of them for rows)
  int blocks;     // 64-wide blocks of a head
};

struct OutView {
  uint16_t* ptr;
  int64_t sb, sh, sn;
  int shift;      // column >> shift is its head: log2 of a head's 64 or 128 channels, 31 for rows
};

// Division of 0 <= n < 2^31 by a number fixed at launch: n * mul / 2^(32 + shift) with
// mul = ceil(2^(32 + shift) / d).  mul * d exceeds 2^(32 + shift) by less than
// d <= 2^(shift + 1), and n times that stays below 2^(32 + shift): the quotient is exact.
struct Div {
  uint32_t d, mul, shift;
};
__host__ __forceinline__ Div make_div(int64_t d) {
  Div v = {uint32_t(d), 0, 0};
  while ((int64_t(2) << v.shift) < d) ++v.shift;
  v.mul = uint32_t(((uint64_t(1) << (32 + v.shift)) + d - 1) / d);
  return v;
}
__device__ __forceinline__ uint32_t operator/(uint32_t n, const Div& v) {
  return v.d == 1 ? n : __umulhi(n, v.mul) >> v.shift;
}

// Column sums of dy [B, heads, N, D] -> part [runs][O] in fp32, to be summed in order by
// colsum_join_kernel.  A unit is 256 columns (32 lanes of 8) of a run of rows.
struct ColSums {
  OutView dy;
  Div by_n, by_cols;               // rows of a batch element; units of 256 columns in a run
  int M, O, rows, units;           // rows of a run
  float* part;
};

struct GemmArgs {
  unsigned int* status;
  unsigned long long wait_ns;      // bound of every wait
  int bn;                          // columns of a tile: 256 or 128
  int m_tiles, n_tiles, group;     // output tiles and the column group of the order
  Div by_group, by_width, by_last; // tiles of a group; its columns, and the last group's
  Div by_parts, by_rows_b, by_nrow; // by_parts: splits or strips of a tile
  // whole tiles come first, in full waves; the rest are split along K, k_split blocks each, or
  // cut into strips of columns
  int k_blocks, k_split, splits, strips, whole;
  int rows_b;                      // row blocks (tiles, or K blocks in wgrad) per batch element
  int64_t N;                       // rows of a batch element of the TMA views
  int64_t M;                       // valid rows of the output (rows of dw in wgrad)
  int cols;                        // valid columns of the output
  Cols ac, bc;                     // columns of A and B along the contiguous dimension
  // epilogue
  int64_t Nrow;                    // rows per batch element of the output views
  OutView y, res, pre;
  const void* bias;
  int bias_f32, act;
  int add;                         // dgrad: res is added, and not the pre-activation
  float* partial;                  // fp32 [splits][tiles - whole][256][bn]
  ColSums sum;                     // wgrad: dy's column sums, made on the way (units = 0: not)
};

// The barrier may be the other CTA's.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The leading CTA's copy of a shared address.
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Relaxed: the accumulator's reads are ordered by the tcgen05 fence before it, and a release at
// cluster scope would first wait for this thread's stores to global memory (1-2 us a tile).
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this place in both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"(uint16_t(3))
      : "memory");
}

// Output tile -> its row and column tile: the column tiles in groups, m-major within one.
__device__ __forceinline__ void decode(uint32_t tile, const GemmArgs& a, int& m, int& n) {
  const uint32_t g = tile / a.by_group, r = tile - g * a.by_group.d;
  const int first = int(g) * a.group;
  const bool last = first + a.group >= a.n_tiles;
  m = int(last ? r / a.by_last : r / a.by_width);
  n = first + int(r) - m * int(last ? a.by_last.d : a.by_width.d);
}
// Work item t: `width` columns from column `col` of a tile; sp >= 0 is a split of its K.
struct Item {
  int tile, sp, k0, k1, col, width;
};
__device__ __forceinline__ Item item_of(int t, const GemmArgs& a) {
  if (t < a.whole) return {t, -1, 0, a.k_blocks, 0, a.bn};
  const int u = t - a.whole, i = int(uint32_t(u) / a.by_parts), part = u - i * int(a.by_parts.d);
  if (a.strips > 1) {
    const int width = a.bn / a.strips;
    return {a.whole + i, -1, 0, a.k_blocks, part * width, width};
  }
  return {a.whole + i, a.splits > 1 ? part : -1, part * a.k_split, min(a.k_blocks, (part + 1) * a.k_split), 0, a.bn};
}

// Two fp32 values at a time: the epilogue's arithmetic is bound by its instructions.
__device__ __forceinline__ uint64_t bits(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 floats(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return floats(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return floats(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return floats(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 1 / (1 + 2^t): the logistic function of x for t = -x log2(e).  2^t = inf gives 0.
__device__ __forceinline__ float2 logistic2(float2 t) {
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = add2(e, both(1.0f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  return e;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 1.5957691216057308f;     // 2 sqrt(2/pi)
// sigmoid(kGeluC (x + 0.044715 x^3)): gelu_tanh(x) / x
__device__ __forceinline__ float2 gelu_gate2(float2 x) {
  const float2 q = fma2(mul2(x, x), both(-kLog2e * kGeluC * 0.044715f), both(-kLog2e * kGeluC));
  return logistic2(mul2(x, q));
}

// f = act(f) for a run of values; the choice is uniform and taken once a run.
template <int kN>
__device__ __forceinline__ void act_run(int act, float2 (&f)[kN]) {
  if (act == VSA_ACT_GELU_TANH) {
#pragma unroll
    for (int e = 0; e < kN; ++e) f[e] = mul2(f[e], gelu_gate2(f[e]));
  } else if (act == VSA_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < kN; ++e) f[e] = mul2(f[e], logistic2(mul2(f[e], both(-kLog2e))));
  } else if (act == VSA_ACT_SIGMOID) {
#pragma unroll
    for (int e = 0; e < kN; ++e) f[e] = logistic2(mul2(f[e], both(-kLog2e)));
  }
}

// act'(x) of a pair.
__device__ __forceinline__ float2 act_slope2(int act, float2 x) {
  if (act == VSA_ACT_GELU_TANH) {
    // s is 0 in fp32 for x < -10 and 1 - s for x > 6, so the clamp only keeps an overflow
    // of the square from meeting that 0
    const float2 s = gelu_gate2(x);
    const float2 c = make_float2(fminf(fmaxf(x.x, -20.0f), 20.0f), fminf(fmaxf(x.y, -20.0f), 20.0f));
    const float2 d = fma2(mul2(c, c), both(kGeluC * 0.134145f), both(kGeluC));
    return fma2(mul2(mul2(c, s), fma2(s, both(-1.0f), both(1.0f))), d, s);
  }
  const float2 s = logistic2(mul2(x, both(-kLog2e)));
  // sigmoid's slope is s(x) s(-x): 1 - s in place of s(-x) loses bits to the right, from x = 17 all of them
  if (act == VSA_ACT_SIGMOID) return mul2(s, logistic2(mul2(x, both(kLog2e))));
  return fma2(mul2(x, s), fma2(s, both(-1.0f), both(1.0f)), s);      // there x s (1 - s) adds to 1
}
// f *= act'(x).
template <int kN>
__device__ __forceinline__ void slope_run(int act, const float2 (&x)[kN], float2 (&f)[kN]) {
  if (act == VSA_ACT_IDENTITY) return;
#pragma unroll
  for (int e = 0; e < kN; ++e) f[e] = mul2(f[e], act_slope2(act, x[e]));
}

__device__ __forceinline__ void unpack(const uint4& v, float2* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack(const float2* f) {
  return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                    pack_bf16(f[3].x, f[3].y));
}

// wait_bar by a whole warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          const GemmArgs& a, unsigned int where) {
  return __all_sync(0xFFFFFFFFu, wait_bar(bar, parity, abort_flag, a.status, where, a.wait_ns));
}

// Column col of a view (a block of 64 columns lies within a head), less its row.
__device__ __forceinline__ int64_t col_offset(const OutView& v, int col) {
  const int h = col >> v.shift;
  return h * v.sh + (col - (h << v.shift));
}

// Programmatic launch: the tiles' kernel and those that join and sum for it are put on the GPU while
// the one before them on the stream still runs, where that is one of them (they let the next
// at their start; behind anything else they start as usual).  They set themselves up, and wait for
// that one's end before they touch memory; as each of them waits, its end is the end of all before it.
// What another of them may have written is read with plain loads: one through the read-only path
// could be moved up over the wait.  (Calls one after the other: 9,772 x 1,024 -> 1,024 20.6 us without and
// 19.3 with it, 366 x 256 -> 256 5.8 and 4.6.  The kernels that only stream their operands lose as much as
// they gain and are launched plainly: eight rows of 1,024 2.4 and 2.8 us.)
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// An epilogue warp's 32 x 64 bytes of shared memory: 16-byte chunk q of row r at chunk q ^ (r/2 & 3),
// so that neither a lane per row nor four lanes per row meet in a bank.
__device__ __forceinline__ uint4* chunk_at(uint8_t* staging, int r, int q) {
  return reinterpret_cast<uint4*>(staging + r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}

// 16 bytes that are read once: volatile, so that the loads of a step stay ahead of its arithmetic.
__device__ __forceinline__ uint4 load_once(const uint16_t* p, bool live) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (live)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

// A unit by eight warps with eight rows each in flight; `sync` is a barrier of theirs, and `s`
// 256 floats a warp, kStride apart.
constexpr int kColsumRows = 64;
template <int kStride, class Sync>
__device__ __forceinline__ void colsum_unit(const ColSums& a, uint32_t unit, int warp, int lane, float* s,
                                            const Sync& sync) {
  const uint32_t run = unit / a.by_cols, cols = unit - run * a.by_cols.d;
  const int col = int(cols) * 256 + 8 * lane;
  float2 acc[4] = {};
  const int r0 = int(run) * a.rows, r1 = int(min(uint32_t(a.M), uint32_t(r0) + uint32_t(a.rows)));
  if (col < a.O) {
    const uint16_t* base = a.dy.ptr + col_offset(a.dy, col);
    for (int r = r0 + warp; r < r1; r += kColsumRows) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t ri = r + 8 * i, b = ri / a.by_n;
        v[i] = load_once(base + b * a.dy.sb + (ri - b * a.by_n.d) * a.dy.sn, int(ri) < r1);
      }
      // nothing is added before all eight are asked for
      asm volatile("" : "+r"(v[0].x), "+r"(v[1].x), "+r"(v[2].x), "+r"(v[3].x), "+r"(v[4].x), "+r"(v[5].x),
                        "+r"(v[6].x), "+r"(v[7].x));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f[4];
        unpack(v[i], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = add2(acc[e], f[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(s + warp * kStride + 8 * lane + 2 * e) = acc[e];
  sync();
  const int c = warp * 32 + lane;
  if (int(cols) * 256 + c < a.O) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += s[w * kStride + c];
    a.part[int64_t(run) * a.O + cols * 256 + c] = v;
  }
  sync();
}

template <int kOrder>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_strip, const __grid_constant__ GemmArgs a) {
  constexpr bool kAMn = kOrder == kWgrad, kBMn = kOrder != kForward;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t s_base = smem_u32(smem);
  uint8_t* staging = smem + kStages * kStageBytes;
  float* s_bias = reinterpret_cast<float*>(staging + kStaging);
  uint8_t* tail = staging + kStaging + 8 * 128 * 4;
  const uint32_t full = smem_u32(tail), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + kNBar * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + kNBar * 8 + 4);
  // K blocks the producer asked for (a register of all roles for it made the epilogue spill)
  uint32_t* issued = reinterpret_cast<uint32_t*>(tail + kNBar * 8 + 8);
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0);
  const int rank = int(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int items = a.whole + (a.m_tiles * a.n_tiles - a.whole) * int(a.by_parts.d);

  let_next_start();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);      // the leader's: its producer, and both CTAs' bytes
      mbar_init(empty + 8 * s, 1);     // each CTA's own: the commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 16);  // the leader's: 8 epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                      // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_last();

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    // The whole warp walks the blocks and one lane issues: what the instructions need is then
    // uniform, and stands in uniform registers.  (One lane alone on the loop took
    // some 100 cycles for every product and copy.)
    {
      // The block index is split into coordinates step by step, with no division on the way: a K
      // block of products takes 512 cycles, and a division by a variable some hundred.
      uint32_t g = 0, s = 0, phase = 1;  // K block, its stage, parity of the stage's last use
      bool ok = true;
      const uint32_t lead = at_leader(full);
      for (int t = pair; t < items && ok; t += pairs) {
        const Item it = item_of(t, a);
        int m, n;
        decode(it.tile, a, m, n);
        const int half = it.width / 2;   // this CTA's columns of the B block
        const int b0 = n * a.bn + it.col + rank * half;
        const CUtensorMap* map_b = kOrder == kForward && it.width < a.bn ? &tm_strip : &tm_b;
        const int k0 = it.k0, k1 = it.k1;
        // along K: block `i` of `per` in head (or batch element) `o`
        const int per = kAMn ? a.rows_b : a.ac.blocks;
        int o = k0 / per, i = k0 - o * per;
        // across K: boxes of 64 columns (wgrad), or the tile's rows
        int ca[2] = {0, 0}, ha[2] = {0, 0}, cb[2] = {0, 0}, hb[2] = {0, 0};
        if (kAMn) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = m * kBM + rank * 128 + 64 * j, d = b0 + 64 * j;
            ha[j] = c / a.ac.D;
            ca[j] = c - ha[j] * a.ac.D;
            hb[j] = d / a.bc.D;
            cb[j] = d - hb[j] * a.bc.D;
          }
        } else {
          ha[0] = int(uint32_t(m) / a.by_rows_b);
          ca[0] = (m - ha[0] * a.rows_b) * kBM + rank * 128;
        }
        for (int kb = k0; kb < k1; ++kb, ++g) {
          if (g >= uint32_t(kStages) && !wait_warp(empty + 8 * s, phase, abort_flag, a, 31)) {
            ok = false;
            break;
          }
          const uint32_t sa = s_base + s * kStageBytes, sb = sa + kABytes, bar = lead + 8 * s;
          if (elect_one()) {
            if (rank == 0) mbar_expect_tx(full + 8 * s, 2 * (kABytes + half * kBK * 2));
            if (!kAMn) {
              tma_load_4d(sa, &tm_a, bar, i * kBK, ca[0], o, ha[0]);
              const int k = o * a.ac.D + i * kBK;
              if (!kBMn) {
                tma_load_4d(sb, map_b, bar, k, b0, 0, 0);
              } else {
                tma_load_4d(sb, &tm_b, bar, b0, k, 0, 0);
                if (half > 64) tma_load_4d(sb + kMnAtom, &tm_b, bar, b0 + 64, k, 0, 0);
              }
            } else {
              tma_load_4d(sa, &tm_a, bar, ca[0], i * kBK, ha[0], o);
              tma_load_4d(sa + kMnAtom, &tm_a, bar, ca[1], i * kBK, ha[1], o);
              tma_load_4d(sb, &tm_b, bar, cb[0], i * kBK, hb[0], o);
              if (half > 64) tma_load_4d(sb + kMnAtom, &tm_b, bar, cb[1], i * kBK, hb[1], o);
            }
          }
          __syncwarp();
          if (++i == per) {
            i = 0;
            ++o;
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (lane == 0) *issued = g;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA, for the pair
    if (rank == 0) {
      uint32_t s = 0, phase = 0;
      int lt = 0;
      bool ok = true;
      for (int t = pair; t < items && ok; t += pairs, ++lt) {
        const Item it = item_of(t, a);
        const int nk = it.k1 - it.k0;
        const uint32_t idesc = idesc_bf16(kBM, it.width, kAMn, kBMn);
        const int buf = lt & 1;
        if (lt >= 2 && !wait_warp(acc_empty + 8 * buf, ((lt >> 1) - 1) & 1, abort_flag, a, 32)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + buf * 256;
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait_warp(full + 8 * s, phase, abort_flag, a, 33)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = s_base + s * kStageBytes, sb = sa + kABytes;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
              // K-major: 16 columns on; MN-major: 16 rows of 128 bytes on, 64-column atoms
              // kMnAtom apart
              const uint64_t ad = kAMn ? sdesc_sw128(sa + ks * 2048, kMnAtom, 1024)
                                       : sdesc_sw128(sa + ks * 32, 16, 1024);
              const uint64_t bd = kBMn ? sdesc_sw128(sb + ks * 2048, kMnAtom, 1024)
                                       : sdesc_sw128(sb + ks * 32, 16, 1024);
              umma_pair(acc, ad, bd, idesc, (kb > 0 || ks > 0) ? 1u : 0u);
            }
            commit_pair(empty + 8 * s);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok && elect_one()) commit_pair(acc_full + 8 * buf);
        __syncwarp();
      }
      // every product issued above completes before either CTA frees its TMEM
      if (elect_one()) commit_pair(drain);
      __syncwarp();
    }
    if (lane == 0) wait_bar_drain(drain, 0);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;                       // TMEM lane quadrant of this warp
    const int side = (warp - 2) >> 2;                // first or second half of the columns
    uint8_t* st = staging + (warp - 2) * (32 * 64);
    float* bias = s_bias + (warp - 2) * 128;
    const int row0 = rank * 128 + quad * 32;         // first row of the warp in the tile
    if (kOrder == kWgrad) {
      // these warps have nothing else to do during the first products
      for (uint32_t u = blockIdx.x; u < uint32_t(a.sum.units); u += gridDim.x)
        colsum_unit<512>(a.sum, u, warp - 2, lane, reinterpret_cast<float*>(staging),
                         [] { asm volatile("bar.sync 1, 256;" ::: "memory"); });
    }
    float next_bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // column 32 i + lane of the next tile
    const auto read_bias = [&](int t) {
      int m, n;
      const Item it = item_of(t, a);
      const int half = it.width / 2;
      decode(it.tile, a, m, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = n * a.bn + it.col + side * half + 32 * i + lane;
        next_bias[i] = 0.0f;
        if (32 * i < half && col < a.cols)
          next_bias[i] =
              a.bias_f32 ? static_cast<const float*>(a.bias)[col]
                         : __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.bias)[col]) << 16);
      }
    };
    if (kOrder == kForward && a.bias != nullptr && pair < items) read_bias(pair);
    int lt = 0;
    for (int t = pair; t < items; t += pairs, ++lt) {
      const Item it = item_of(t, a);
      int m, n;
      decode(it.tile, a, m, n);
      const int buf = lt & 1, half = it.width / 2;
      const uint32_t acc = tmem + buf * 256 + (uint32_t(quad * 32) << 16) + uint32_t(side * half);
      // four lanes write a row's 64 bytes: this lane's rows are 8 i + lane / 4
      uint32_t tok[4], bat[4];
      uint32_t live = 0;
      const uint32_t mb = kOrder == kWgrad ? 0 : uint32_t(m) / a.by_rows_b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int in_tile = row0 + 8 * i + (lane >> 2);
        if (kOrder == kWgrad) {
          tok[i] = uint32_t(m) * kBM + in_tile;
          bat[i] = 0;
          live |= uint32_t(tok[i] < a.M) << i;
        } else {
          const uint32_t in_b = (uint32_t(m) - mb * uint32_t(a.rows_b)) * kBM + in_tile;
          const uint32_t r = mb * uint32_t(a.N) + in_b;
          live |= uint32_t(in_b < a.N) << i;
          bat[i] = r / a.by_nrow;
          tok[i] = r - bat[i] * uint32_t(a.Nrow);
        }
      }
      const int q = lane & 3;                        // and its chunk of them
      const int col_w = n * a.bn + it.col + side * half;      // first column of the warp
      const bool with_bias = kOrder == kForward && a.bias != nullptr;
      if (with_bias) {
        // the tile's biases were read during the tile before
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[32 * i + lane] = next_bias[i];
        __syncwarp();
        if (t + pairs < items) read_bias(t + pairs);
      }
      const bool with_res = kOrder != kWgrad && a.res.ptr != nullptr && it.sp < 0;
      const bool with_pre = kOrder == kForward && a.pre.ptr != nullptr;
      // nothing of the warp's rows and columns is over the edge
      const bool inside = __all_sync(0xFFFFFFFFu, live == 15u) && col_w + half <= a.cols;
      const int chunks = half / 32;
      // residuals: a chunk of 32 columns is on its way, the first under the products
      uint4 rr[4];
      const auto load_res = [&](int c) {
        const int col = col_w + 32 * c;
        if (!with_res || col + 8 * q >= a.cols) return;
        const uint16_t* p = a.res.ptr + col_offset(a.res, col) + 8 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (live >> i & 1)
            rr[i] = *reinterpret_cast<const uint4*>(p + bat[i] * a.res.sb + tok[i] * a.res.sn);
      };
      // the warp's 32 rows x 32 columns, a row a lane, through shared memory to the rows of a view
      const auto store_rows = [&](const OutView& v, int c, const uint4 (&o)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) *chunk_at(st, lane, e) = o[e];
        __syncwarp();
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *chunk_at(st, 8 * i + (lane >> 2), q);
        const int col = col_w + 32 * c;
        uint16_t* p = v.ptr + col_offset(v, col) + 8 * q;
        if (inside) {
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(p + bat[i] * v.sb + tok[i] * v.sn) = w[i];
        } else if (col + 8 * q < a.cols) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (live >> i & 1) *reinterpret_cast<uint4*>(p + bat[i] * v.sb + tok[i] * v.sn) = w[i];
        }
        __syncwarp();
      };
      // the accumulator is out: the products of the tile after the next may start
      const auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(at_leader(acc_empty + 8 * buf));
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) rr[i] = make_uint4(0u, 0u, 0u, 0u);
      load_res(0);
      if (!wait_warp(acc_full + 8 * buf, (lt >> 1) & 1, abort_flag, a, 34)) break;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(acc, v);
      if (it.sp >= 0) {
        // fp32 partial products of the tile's rows, 16 columns (64 bytes) at a time
        float* slot = a.partial + (int64_t(it.sp) * (a.m_tiles * a.n_tiles - a.whole) + it.tile - a.whole) *
                                      (kBM * a.bn) +
                      (row0 + (lane >> 2)) * a.bn + side * half + 4 * q;
        for (int c = 0; c < chunks; ++c) {
          tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *chunk_at(st, lane, e) = make_uint4(v[16 * j + 4 * e], v[16 * j + 4 * e + 1],
                                                  v[16 * j + 4 * e + 2], v[16 * j + 4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (live >> i & 1)
                *reinterpret_cast<uint4*>(slot + 8 * i * a.bn + 32 * c + 16 * j) =
                    *chunk_at(st, 8 * i + (lane >> 2), q);
            __syncwarp();
          }
          if (c + 1 < chunks) tmem_ld32(acc + 32 * c + 32, v);
        }
        release();
        continue;
      }
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        uint4 x4[4];
        if (with_res) {
          // residuals: rows as they were read -> a row per lane
#pragma unroll
          for (int i = 0; i < 4; ++i) *chunk_at(st, 8 * i + (lane >> 2), q) = rr[i];
          if (c + 1 < chunks) load_res(c + 1);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) x4[e] = *chunk_at(st, lane, e);
          __syncwarp();
        }
        tmem_wait_ld(v);
        float2 f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          f[e] = make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
        if (with_bias) {
          const float4* bp = reinterpret_cast<const float4*>(bias + 32 * c);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 w = bp[e];
            f[2 * e] = add2(f[2 * e], make_float2(w.x, w.y));
            f[2 * e + 1] = add2(f[2 * e + 1], make_float2(w.z, w.w));
          }
        }
        uint4 o[4];
        if (with_pre) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = pack(&f[4 * e]);
          store_rows(a.pre, c, o);
        }
        if (kOrder == kForward) act_run(a.act, f);
        if (with_res) {
          float2 x[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) unpack(x4[e], &x[4 * e]);
          if (kOrder == kForward || a.add) {
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = add2(f[e], x[e]);
          } else {
            slope_run(a.act, x, f);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack(&f[4 * e]);
        if (c + 1 < chunks)
          tmem_ld32(acc + 32 * c + 32, v);
        else
          release();
        store_rows(a.y, c, o);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0 && *abort_flag) {
    // Abort, whichever warp's: none of our TMA writes may still be in flight.  (Without one all
    // accumulators came out, and with that all copies in.)  They complete on the leader's
    // barriers, whose phases stay open where the other CTA stopped before them: one bound for all.
    // The other CTA gives its own a millisecond, some thousand times what a copy takes.
    const unsigned long long t0 = globaltimer();
    if (rank == 0) {
      const uint32_t end = *issued;
      uint32_t x = end > uint32_t(kStages) ? end - kStages : 0;
      while (x < end && globaltimer() - t0 < kWaitLimitNs)
        if (mbar_try_wait(full + 8 * (x % kStages), (x / kStages) & 1)) ++x;
    } else {
      while (globaltimer() - t0 < 1000000ull) {
      }
    }
    __syncwarp();
  }
  cluster_sync();                      // no signal to either CTA is on its way
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

// ---------------------------------------------------------------- few rows
// Forward for up to eight rows, where reading w is all there is (2 O C bytes; 8.8 us at the copy
// rate for 5,376 x 5,376) and tiles of 256 rows would leave most SMs without work.
// A block takes eight rows of w; its warps share out C.  A lane reads 16 bytes along C of a row
// of w and of a row of x straight into the fragments of mma.m16n8k16 (x in the first
// eight of 16 rows): the order of C within 32 columns does not matter to a sum, so lane t's eight
// neighbours stand for the pairs 2t, 2t + 1, 2t + 8, 2t + 9 of two products.  The warps'
// fp32 sums meet in shared memory, in warp order.
constexpr int kFewThreads = 256, kFewRows = 8;

struct FewArgs {
  const uint16_t *x, *w;
  int64_t xb, xh, xn;
  int x_shift;                     // column >> x_shift is the head of x
  int M, N, C, O;
  OutView y, res, pre;
  const void* bias;
  int bias_f32, act;
};

// d += a b for the first eight rows of a.
__device__ __forceinline__ void mma_8x8(float (&d)[2], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  float d2 = 0.0f, d3 = 0.0f;
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d2), "+f"(d3)
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_or_zero(const uint16_t* p, bool live) {
  return live ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// The epilogue of two neighbouring columns of row r.
__device__ __forceinline__ void finish(const FewArgs& a, int r, int o, float2 (&f)[1]) {
  if (a.bias != nullptr) {
    const float* bf = static_cast<const float*>(a.bias) + o;
    const uint16_t* bh = static_cast<const uint16_t*>(a.bias) + o;
    f[0].x += a.bias_f32 ? bf[0] : __uint_as_float(uint32_t(bh[0]) << 16);
    f[0].y += a.bias_f32 ? bf[1] : __uint_as_float(uint32_t(bh[1]) << 16);
  }
  const int b = r / a.N;
  const int64_t n = r - b * a.N;
  const auto at = [&](const OutView& v) {
    return reinterpret_cast<uint32_t*>(v.ptr + b * v.sb + n * v.sn + col_offset(v, o));
  };
  if (a.pre.ptr != nullptr) *at(a.pre) = pack_bf16(f[0].x, f[0].y);
  act_run(a.act, f);
  if (a.res.ptr != nullptr) {
    const uint32_t w = *at(a.res);
    f[0] = add2(f[0], make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)));
  }
  *at(a.y) = pack_bf16(f[0].x, f[0].y);
}

// kPieces 16-byte pieces of w in flight a lane and step, kPerSm blocks an SM.
template <int kPieces, int kPerSm>
__global__ void __launch_bounds__(kFewThreads, kPerSm) linear_few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kWarps = kFewThreads / 32, kStep = kWarps * 32;
  __shared__ float sum[kWarps][8][8 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int o0 = blockIdx.x * 8;                    // O is a multiple of 8
  const uint16_t* w = a.w + int64_t(o0 + g) * a.C;
  const int bx = g / a.N;
  const bool live = g < a.M;
  const uint16_t* x = a.x + bx * a.xb + int64_t(g - bx * a.N) * a.xn;
  float acc[2] = {0.0f, 0.0f};
  const int first = warp * 32 + 8 * t;
  uint4 next[kPieces];                            // the step's pieces of w, a step ahead
#pragma unroll
  for (int i = 0; i < kPieces; ++i) next[i] = load_once(w + first + i * kStep, first + i * kStep < a.C);
  for (int k0 = first; k0 - 8 * t < a.C; k0 += kStep * kPieces) {
    uint4 u[kPieces], v[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int k = k0 + i * kStep, h = k >> a.x_shift, kn = k + kStep * kPieces;
      u[i] = next[i];
      v[i] = load_or_zero(x + h * a.xh + (k - (h << a.x_shift)), live && k < a.C);
      next[i] = load_once(w + kn, kn < a.C);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      mma_8x8(acc, v[i].x, v[i].y, u[i].x, u[i].y);
      mma_8x8(acc, v[i].z, v[i].w, u[i].z, u[i].w);
    }
  }
  // row g of x, columns 2t and 2t + 1
  sum[warp][g][2 * t] = acc[0];
  sum[warp][g][2 * t + 1] = acc[1];
  __syncthreads();
  // a thread for two neighbouring columns of a row
  if (threadIdx.x >= 32) return;
  const int c = 2 * t, r = g, o = o0 + c;
  if (r >= a.M) return;
  float2 f[1] = {make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int v = 0; v < kWarps; ++v) f[0] = add2(f[0], make_float2(sum[v][r][c], sum[v][r][c + 1]));
  finish(a, r, o, f);
}

// The join of split tiles: partials are summed in split order, and what the tiles' epilogue
// would have done follows.  A thread takes eight columns of a row, a block 2,048 elements of a tile.
template <int kOrder>
__global__ void __launch_bounds__(256) split_join_kernel(const __grid_constant__ GemmArgs a) {
  let_next_start();
  wait_for_last();
  const int octs = a.bn / 8, per_block = 256 / octs;       // rows of a block
  const int i = blockIdx.x / (kBM / per_block), part = blockIdx.x % (kBM / per_block);
  const int in_tile = part * per_block + threadIdx.x / octs, in_row = (threadIdx.x % octs) * 8;
  int m, tn;
  decode(a.whole + i, a, m, tn);
  const int col = tn * a.bn + in_row;
  uint32_t r;                                              // row of the output
  if (kOrder == kWgrad) {
    r = uint32_t(m) * kBM + in_tile;
    if (r >= a.M) return;
  } else {
    const uint32_t mb = uint32_t(m) / a.by_rows_b, in_b = (uint32_t(m) - mb * uint32_t(a.rows_b)) * kBM + in_tile;
    if (in_b >= a.N) return;
    r = mb * uint32_t(a.N) + in_b;
  }
  if (col >= a.cols) return;
  float2 f[4] = {};
  const float* p = a.partial + int64_t(i) * (kBM * a.bn) + in_tile * a.bn + in_row;
  const int64_t next = int64_t(a.m_tiles * a.n_tiles - a.whole) * (kBM * a.bn);
  for (int k = 0; k < a.splits; ++k, p += next) {
    const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
    f[0] = add2(f[0], make_float2(u.x, u.y));
    f[1] = add2(f[1], make_float2(u.z, u.w));
    f[2] = add2(f[2], make_float2(v.x, v.y));
    f[3] = add2(f[3], make_float2(v.z, v.w));
  }
  const uint32_t b = r / a.by_nrow;
  const int64_t n = r - b * a.by_nrow.d;
  const auto at = [&](const OutView& v) {
    return reinterpret_cast<uint4*>(v.ptr + b * v.sb + n * v.sn + col_offset(v, col));
  };
  if (kOrder == kForward) {
    if (a.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* bf = static_cast<const float*>(a.bias) + col + 2 * e;
        const uint16_t* bh = static_cast<const uint16_t*>(a.bias) + col + 2 * e;
        f[e] = add2(f[e], a.bias_f32 ? make_float2(bf[0], bf[1])
                                     : make_float2(__uint_as_float(uint32_t(bh[0]) << 16),
                                                   __uint_as_float(uint32_t(bh[1]) << 16)));
      }
    }
    if (a.pre.ptr != nullptr) *at(a.pre) = pack(f);
    act_run(a.act, f);
  }
  if (kOrder != kWgrad && a.res.ptr != nullptr) {
    float2 x[4];
    unpack(*at(a.res), x);
    if (kOrder == kForward || a.add) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = add2(f[e], x[e]);
    } else {
      slope_run(a.act, x, f);
    }
  }
  *at(a.y) = pack(f);
}

// Column sums by themselves: a block a unit.
__global__ void __launch_bounds__(256) colsum_kernel(const __grid_constant__ ColSums a) {
  __shared__ float s[8 * 256];
  let_next_start();
  wait_for_last();
  colsum_unit<256>(a, blockIdx.x, threadIdx.x >> 5, threadIdx.x & 31, s, [] { __syncthreads(); });
}

__global__ void __launch_bounds__(1024) colsum_join_kernel(const float* part, int runs, int O, float* db) {
  __shared__ float s[32][33];
  let_next_start();
  wait_for_last();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < O) {
#pragma unroll 8
    for (int i = warp; i < runs; i += 32) v += part[int64_t(i) * O + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < O) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += s[w][lane];
    db[c] = t;
  }
}

__global__ void __launch_bounds__(256) act_backward_kernel(const uint4* dy, const uint4* pre, int act,
                                                           uint4* out, int64_t n8) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n8; i += int64_t(gridDim.x) * 256) {
    float2 g[4], x[4];
    unpack(dy[i], g);
    unpack(pre[i], x);
    slope_run(act, x, g);
    out[i] = pack(g);
  }
}

// ---------------------------------------------------------------- host side

template <class... Params, class... Args>
cudaError_t launch_on(cudaStream_t stream, void (*kernel)(Params...), dim3 blocks, int threads, size_t smem,
                      const Args&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A view as the products see it: heads >= 1, rows as one batch element when they are
// evenly spaced over all of them.
struct View {
  const uint16_t* ptr;
  int64_t sb, sh, sn, B, N;
  int H, D;
};

View make_view(const vsa_view& v, int B, int64_t N, int heads, int C) {
  View o = {static_cast<const uint16_t*>(v.ptr), v.stride_b, v.stride_h, v.stride_n, B, N, 1, C};
  if (heads > 0) {
    o.H = heads;
    o.D = C / heads;
  }
  return o;
}

bool rows_even(const View& v) { return v.B == 1 || v.N == 1 || v.sb == v.N * v.sn; }

void flatten(View* v) {
  if (v->N == 1 && v->B > 1) v->sn = v->sb;
  v->N *= v->B;
  v->B = 1;
}

// TMA map of a view, box 64 channels x box_rows rows.
bool map_view(CUtensorMap* m, const View& v, int box_rows) {
  const cuuint64_t dims[4] = {cuuint64_t(v.D), cuuint64_t(v.N), cuuint64_t(v.H), cuuint64_t(v.B)};
  // the stride of a dimension of extent 1 is not used, but has to be valid
  const auto bytes = [](int64_t extent, int64_t stride) {
    return extent > 1 ? cuuint64_t(stride) * 2 : cuuint64_t(16);
  };
  const cuuint64_t strides[3] = {bytes(v.N, v.sn), bytes(v.H, v.sh), bytes(v.B, v.sb)};
  const cuuint32_t box[4] = {64u, cuuint32_t(box_rows), 1u, 1u};
  return encode_map(m, v.ptr, 4, dims, strides, box);
}

View matrix(const void* p, int64_t rows, int cols) {
  return View{static_cast<const uint16_t*>(p), 0, 0, cols, 1, rows, 1, cols};
}

OutView out_view(const vsa_view& v, int heads, int C) {
  return OutView{static_cast<uint16_t*>(v.ptr), v.stride_b, heads > 0 ? v.stride_h : 0, v.stride_n,
                 heads > 0 ? (C / heads == 64 ? 6 : 7) : 31};
}

Cols cols_of(const View& v) { return Cols{v.D, (v.D + kBK - 1) / kBK}; }

int sms(const vsa_plan_s* p) { return p->num_sms > 0 ? p->num_sms : 148; }

int pairs_of(const vsa_plan_s* p) { return std::max(1, sms(p) / 2); }

// Columns of a tile (256 or 128), and what becomes of the tiles that are over after the full waves:
// whole, split along K, or cut into strips of columns (64 or 128 wide; the gradients' boxes of 64
// columns a CTA leave them 128), by the time it should take, in us.  A wave of tiles over the pairs
// of SMs takes 0.35 a K block with 256 columns, 0.25 with 128 and 0.22 with 64 (measured: 29 and
// 20 us at K = 5,376 for the first two; narrow tiles want more operand bytes a product), and one
// for its turn; its epilogue takes 14 ns a column and runs under the next wave's products.  Splits
// of K cost the join: a launch under the products' end and two passes over their fp32 partial sums, at
// some 4 TB/s.
// Strips cost their operands' bytes, and shorten the last epilogue along with the last products.
// Measured with whole tiles, the best strips and the best split: 9,772 x 1,024 -> 1,024 with residual
// 24.4, 21.6, 27.6 us; 3,000 x 512 -> 2,048 11.7, 10.6, 17.1; 9,772 x 4,096 -> 1,024 71.5, 68.6, 68.1;
// 1,024 x 5,376 -> 5,376 56.5, 50.8, 49.4; 256 rows of it 22.7 (128 columns), 22.9, 21.0.
struct Tiling {
  int bn, splits, k_split, strips;
  int64_t whole, split_tiles;
  size_t bytes() const {
    return splits > 1 ? size_t(splits) * size_t(split_tiles) * kBM * size_t(bn) * sizeof(float) : 0;
  }
};
Tiling tiling(const vsa_plan_s* p, int64_t m_tiles, int64_t M, int cols, int k_blocks, bool may_split, bool narrow) {
  const auto products = [](int width, int blocks) {
    return blocks * (width == 256 ? 0.35 : width == 128 ? 0.25 : 0.22) + 1;
  };
  const auto epilogue = [](int width) { return 0.014 * width; };
  Tiling best = {256, 1, k_blocks, 1, 0, 0};
  double least = 1e300;
  for (const int bn : {256, 128}) {
    const int64_t tiles = m_tiles * ((cols + bn - 1) / bn), rest = tiles % pairs_of(p);
    const double waves = double(tiles / pairs_of(p)), P = products(bn, k_blocks), E = epilogue(bn);
    // when the epilogues of the full waves end, and when a product after them may start (its
    // accumulator is that of the wave before the last)
    const double done = waves > 0 ? waves * std::max(P, E) + std::min(P, E) : 0;
    const double idle = std::max(waves * P, done - std::max(P, E));
    const auto consider = [&](int splits, int k_split, int strips) {
      const int width = bn / strips;
      const double sums = double(splits) * double(rest) * double(std::min<int64_t>(M, kBM)) * bn * 8;
      const double join = splits > 1 ? 1.0 + sums / 4e6 : 0.0;
      const double t = rest > 0 ? std::max(done, idle + products(width, k_split)) + epilogue(width) + join : done;
      if (t < least) {
        least = t;
        best = {bn, splits, k_split, strips, splits * strips > 1 ? tiles - rest : tiles, splits > 1 ? rest : 0};
      }
    };
    const int64_t parts = rest > 0 ? pairs_of(p) / rest : 1;
    consider(1, k_blocks, 1);
    for (int strips = 2; strips <= parts && bn / strips >= (narrow ? 64 : 128); strips *= 2)
      consider(1, k_blocks, strips);
    const int most = may_split && rest > 0 ? int(std::min<int64_t>({16, k_blocks / 4, parts})) : 1;
    for (int want = 2; want <= most; ++want) {
      const int k_split = (k_blocks + want - 1) / want;
      consider((k_blocks + k_split - 1) / k_split, k_split, 1);
    }
  }
  return best;
}

void set_tiles(const vsa_plan_s* p, GemmArgs* a, bool may_split, bool narrow) {
  const Tiling t = tiling(p, a->m_tiles, a->M, a->cols, a->k_blocks, may_split, narrow);
  a->bn = t.bn;
  a->n_tiles = (a->cols + t.bn - 1) / t.bn;
  a->k_split = t.k_split;
  a->splits = t.splits;
  a->strips = t.strips;
  a->whole = int(t.whole);
}

int row_blocks(const View& v, int rows) { return int((v.N + rows - 1) / rows); }

// Runs of rows of the column sums: 64 rows each, more where that made more than 512 runs.
int colsum_rows(int64_t M) {
  const int64_t per = (M + 511) / 512;
  return int(std::max<int64_t>(1, (per + kColsumRows - 1) / kColsumRows) * kColsumRows);
}
int colsum_runs(int64_t M) { return int(std::max<int64_t>(1, (M + colsum_rows(M) - 1) / colsum_rows(M))); }

ColSums col_sums(const vsa_linear_grad_args& q, float* part) {
  ColSums a = {};
  a.dy = out_view(q.dy, q.y_heads, q.O);
  a.M = int(q.B * q.N);
  a.O = int(q.O);
  a.rows = colsum_rows(a.M);
  const int cols = (a.O + 255) / 256;
  a.units = cols * colsum_runs(a.M);
  a.by_n = make_div(q.N);
  a.by_cols = make_div(cols);
  a.part = part;
  return a;
}

template <int kOrder>
vsa_status launch(const vsa_plan_s* p, const View& av, int a_box, const View& bv, int b_box,
                  GemmArgs a, cudaStream_t stream) {
  if (int64_t(a.m_tiles) * a.n_tiles >= (int64_t(1) << 31))
    return fail(VSA_ERR_UNSUPPORTED, "too many output tiles");
  CUtensorMap ma, mb, strip;         // a strip's box of w: a map of its own in the forward product
  const int strip_box = kOrder == kForward ? b_box / a.strips : b_box;
  if (!map_view(&ma, av, a_box) || !map_view(&mb, bv, b_box) || !map_view(&strip, bv, strip_box))
    return fail(VSA_ERR_CUDA, "cuTensorMapEncodeTiled failed (driver entry point or arguments)");
  cudaError_t e = cudaFuncSetAttribute(linear_kernel<kOrder>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return fail(VSA_ERR_CUDA, cudaGetErrorString(e));
  // Groups of at most 14 column tiles: the 74 tiles in work at a time are then some 5 x 14, and share
  // their rows of A and columns of B in L2.  At 33,920 x 5,376 x 7,168 (28 or 21 column tiles) the weight
  // gradient took 2,040 us with 14, 2,064 with 10 and 2,138 with all 28 (its DRAM reads fall from 8.5 to
  // 5.5 GB, the column sums' 0.4 among them, and with them the power that holds the clock down); the others stay within 2 %.
  const int groups = (a.n_tiles + 13) / 14;
  a.group = (a.n_tiles + groups - 1) / groups;
  a.by_group = make_div(int64_t(a.m_tiles) * a.group);
  a.by_width = make_div(a.group);
  a.by_last = make_div(a.n_tiles - (a.n_tiles - 1) / a.group * a.group);
  a.by_parts = make_div(int64_t(a.splits) * a.strips);
  a.by_rows_b = make_div(a.rows_b);
  a.by_nrow = make_div(a.Nrow);
  a.status = p->d_status;
  a.wait_ns = wait_limit_ns();
  const int64_t rest = int64_t(a.m_tiles) * a.n_tiles - a.whole, items = a.whole + rest * a.splits * a.strips;
  const int grid = 2 * int(std::min<int64_t>(items, pairs_of(p)));
  e = launch_on(stream, linear_kernel<kOrder>, dim3(unsigned(grid)), kThreads, kSmem, ma, mb, strip, a);
  if (e == cudaSuccess && a.splits > 1)
    e = launch_on(stream, split_join_kernel<kOrder>, dim3(unsigned(rest * (kBM * a.bn / 2048))), 256, 0, a);
  return e == cudaSuccess ? VSA_OK
                          : fail(VSA_ERR_CUDA, std::string("linear launch: ") + cudaGetErrorString(e));
}

vsa_status launch_few(const vsa_plan_s* p, const vsa_linear_args& q, cudaStream_t stream) {
  FewArgs a = {};
  const View x = make_view(q.x, q.B, q.N, q.x_heads, q.C);
  a.x = x.ptr;
  a.w = static_cast<const uint16_t*>(q.w);
  a.xb = x.sb;
  a.xh = x.H > 1 ? x.sh : 0;
  a.xn = x.sn;
  a.x_shift = q.x_heads > 0 ? (x.D == 64 ? 6 : 7) : 31;
  a.M = int(q.B * q.N);
  a.N = int(q.N);
  a.C = q.C;
  a.O = q.O;
  a.y = out_view(q.y, q.y_heads, q.O);
  a.res = out_view(q.residual, q.y_heads, q.O);
  a.pre = out_view(q.pre, q.y_heads, q.O);
  a.bias = q.bias;
  a.bias_f32 = q.bias_type == VSA_F32;
  a.act = q.act;
  // Blocks that fit the SMs four apiece keep four pieces in flight (1,024 x 1,024: 2.7 against 3.4 us,
  // 5,376 x 640: 7.2 against 7.8 us); more of them go five apiece with three (5,376 x 5,376: 12.0
  // against 15.7 us, w from memory each time).
  if (q.O / 8 <= 4 * sms(p))
    linear_few_kernel<4, 4><<<q.O / 8, kFewThreads, 0, stream>>>(a);
  else
    linear_few_kernel<3, 5><<<q.O / 8, kFewThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK
                          : fail(VSA_ERR_CUDA, std::string("linear launch: ") + cudaGetErrorString(e));
}

}  // namespace

size_t linear_bytes(const vsa_plan_s* p, int B, int64_t N, int C, int O) {
  const int64_t M = int64_t(B) * N;
  if (M <= kFewRows) return 0;
  // tiles and K blocks of either flattening, rows or heads
  const int64_t m1 = (M + kBM - 1) / kBM, m2 = int64_t(B) * ((N + kBM - 1) / kBM);
  const int kb = (C + kBK - 1) / kBK;
  return std::max(tiling(p, m1, M, O, kb, true, true).bytes(), tiling(p, m2, M, O, kb, true, true).bytes());
}

vsa_status launch_linear(const vsa_plan_s* p, const vsa_linear_args& q, void* ws, cudaStream_t stream) {
  if (int64_t(q.B) * q.N <= kFewRows) return launch_few(p, q, stream);
  View x = make_view(q.x, q.B, q.N, q.x_heads, q.C);
  if (rows_even(x)) flatten(&x);
  GemmArgs a = {};
  a.rows_b = row_blocks(x, kBM);
  a.m_tiles = int(x.B) * a.rows_b;
  a.ac = cols_of(x);
  a.k_blocks = x.H * a.ac.blocks;
  a.N = x.N;
  a.M = x.B * x.N;
  a.cols = q.O;
  set_tiles(p, &a, ws != nullptr, true);
  a.partial = static_cast<float*>(ws);
  a.Nrow = q.N;
  a.y = out_view(q.y, q.y_heads, q.O);
  a.res = out_view(q.residual, q.y_heads, q.O);
  a.pre = out_view(q.pre, q.y_heads, q.O);
  a.bias = q.bias;
  a.bias_f32 = q.bias_type == VSA_F32;
  a.act = q.act;
  return launch<kForward>(p, x, 128, matrix(q.w, q.O, q.C), a.bn / 2, a, stream);
}

size_t linear_backward_bytes(const vsa_plan_s* p, int B, int64_t N, int C, int O) {
  if (int64_t(B) * N == 0) return 0;
  // one buffer, used in turn by the products' partial sums, the column sums behind those of
  // dw; tiles and K blocks of either flattening, rows or heads
  const int64_t M = int64_t(B) * N;
  const int64_t m1 = (M + kBM - 1) / kBM, m2 = int64_t(B) * ((N + kBM - 1) / kBM);
  const int64_t k1 = (M + kBK - 1) / kBK, k2 = int64_t(B) * ((N + kBK - 1) / kBK);
  const int ko = (O + kBK - 1) / kBK;
  const int64_t mo = (O + kBM - 1) / kBM;
  return std::max({tiling(p, m1, M, C, ko, true, false).bytes(), tiling(p, m2, M, C, ko, true, false).bytes(),
                   std::max(tiling(p, mo, O, C, int(k1), true, false).bytes(),
                            tiling(p, mo, O, C, int(k2), true, false).bytes()) +
                       size_t(colsum_runs(M)) * O * sizeof(float)});
}

vsa_status launch_linear_backward(const vsa_plan_s* p, const vsa_linear_grad_args& q, void* ws,
                                  cudaStream_t stream) {
  const int64_t M = int64_t(q.B) * q.N;
  if (M == 0) {
    cudaError_t e = cudaSuccess;
    if (q.dw != nullptr) e = cudaMemsetAsync(q.dw, 0, size_t(q.O) * q.C * 2, stream);
    if (e == cudaSuccess && q.db != nullptr) e = cudaMemsetAsync(q.db, 0, size_t(q.O) * 4, stream);
    return e == cudaSuccess ? VSA_OK : fail(VSA_ERR_CUDA, cudaGetErrorString(e));
  }
  const View dy = make_view(q.dy, q.B, q.N, q.y_heads, q.O);
  if (q.dx.ptr != nullptr) {
    View g = dy;
    if (rows_even(g)) flatten(&g);
    GemmArgs a = {};
    a.rows_b = row_blocks(g, kBM);
    a.m_tiles = int(g.B) * a.rows_b;
    a.ac = cols_of(g);
    a.k_blocks = g.H * a.ac.blocks;
    a.N = g.N;
    a.M = M;
    a.cols = q.C;
    set_tiles(p, &a, true, false);
    a.partial = static_cast<float*>(ws);
    a.Nrow = q.N;
    a.y = out_view(q.dx, q.x_heads, q.C);
    a.add = q.dx_add.ptr != nullptr;
    a.res = out_view(a.add ? q.dx_add : q.x_pre, q.x_heads, q.C);
    a.act = q.x_act;
    const vsa_status st = launch<kDgrad>(p, g, 128, matrix(q.w, q.O, q.C), kBK, a, stream);
    if (st != VSA_OK) return st;
  }
  float* sums = static_cast<float*>(ws);           // column sums, behind dw's partial sums
  // The product for dw takes the column sums along where it reads dy for more than one tile of
  // columns: 9,772 x 1,024 -> 1,024 (dx, dw, db) 52 -> 46.4 us, 33,920 x 512 -> 1,024 (dw, db) 55.3 -> 50.6.
  // With one there is too little to hide them under: 33,920 x 64 -> 7,168 168 us apart, 186 along.
  const bool along = q.dw != nullptr && q.db != nullptr && q.C > 256;
  if (q.dw != nullptr) {
    View g = dy, x = make_view(q.x, q.B, q.N, q.x_heads, q.C);
    if (rows_even(g) && rows_even(x)) {
      flatten(&g);
      flatten(&x);
    }
    GemmArgs a = {};
    a.rows_b = row_blocks(g, kBK);
    a.k_blocks = int(g.B) * a.rows_b;
    a.m_tiles = (q.O + kBM - 1) / kBM;
    a.ac = cols_of(g);
    a.bc = cols_of(x);
    a.N = g.N;
    a.M = q.O;
    a.cols = q.C;
    set_tiles(p, &a, true, false);
    a.Nrow = q.O;
    a.y = OutView{static_cast<uint16_t*>(q.dw), 0, 0, q.C, 31};
    a.partial = static_cast<float*>(ws);
    if (along) {
      const int64_t rest = int64_t(a.m_tiles) * a.n_tiles - a.whole;
      sums += a.splits > 1 ? a.splits * rest * kBM * a.bn : 0;
      a.sum = col_sums(q, sums);
    }
    const vsa_status st = launch<kWgrad>(p, g, kBK, x, kBK, a, stream);
    if (st != VSA_OK) return st;
  }
  if (q.db != nullptr) {
    const ColSums a = col_sums(q, sums);
    cudaError_t e = cudaSuccess;
    if (!along) e = launch_on(stream, colsum_kernel, dim3(unsigned(a.units)), 256, 0, a);
    if (e == cudaSuccess)
      e = launch_on(stream, colsum_join_kernel, dim3(unsigned((q.O + 31) / 32)), 1024, 0,
                    static_cast<const float*>(sums), colsum_runs(M), int(q.O), q.db);
    if (e != cudaSuccess) return fail(VSA_ERR_CUDA, cudaGetErrorString(e));
  }
  return VSA_OK;
}

cudaError_t launch_act_backward(const void* dy, const void* pre, int act, void* out, int64_t n,
                                int num_sms, cudaStream_t stream) {
  const int64_t n8 = n / 8;
  const int blocks = int(std::min<int64_t>((n8 + 255) / 256, int64_t(num_sms > 0 ? num_sms : 148) * 8));
  act_backward_kernel<<<blocks, 256, 0, stream>>>(static_cast<const uint4*>(dy),
                                                  static_cast<const uint4*>(pre), act,
                                                  static_cast<uint4*>(out), n8);
  return cudaGetLastError();
}

}  // namespace vsa
