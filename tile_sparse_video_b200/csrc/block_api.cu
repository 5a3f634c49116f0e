// C entry points of include/vsa_block.h: argument checks, the rotation's tables and
// dispatch to the kernels.
#include <algorithm>
#include <cmath>
#include <exception>
#include <new>
#include <string>

#include "block_internal.h"

namespace vsa {
namespace {

vsa_status cuda_fail(cudaError_t e, const char* what) {
  return fail(VSA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

vsa_status check_device(const vsa_plan_s* p) {
  if (p == nullptr) return fail(VSA_ERR_INVALID_ARG, "plan is NULL");
  if (p->device < 0) return fail(VSA_ERR_INVALID_ARG, "host-only plan (device = -1) cannot launch");
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (cur != p->device)
    return fail(VSA_ERR_INVALID_ARG, "current CUDA device differs from the plan's device");
  return VSA_OK;
}

vsa_status check_heads(const vsa_plan_s* p, int B, int H, int D) {
  if (p == nullptr) return fail(VSA_ERR_INVALID_ARG, "plan is NULL");
  if (p->device < 0) return fail(VSA_ERR_INVALID_ARG, "host-only plan (device = -1) cannot launch");
  if (B < 0 || H < 0) return fail(VSA_ERR_INVALID_ARG, "B and H must be >= 0");
  if (D != 64 && D != 128) return fail(VSA_ERR_UNSUPPORTED, "head dim D must be 64 or 128");
  return check_device(p);
}

vsa_status check_ptr(const void* ptr, const char* name) {
  if (ptr == nullptr) return fail(VSA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!aligned16(ptr)) return fail(VSA_ERR_INVALID_ARG, std::string(name) + " is not 16-byte aligned");
  return VSA_OK;
}

// One stride: a multiple of 8, and no smaller than `least` (0 lets a broadcast through).
// The stride of an extent of 1 is not used.
vsa_status check_stride(int64_t stride, int64_t extent, int64_t least, const char* name) {
  if (extent <= 1) return VSA_OK;
  if (stride < least || stride % 8 != 0 || stride >= (int64_t(1) << 38))
    return fail(VSA_ERR_INVALID_ARG,
                std::string(name) + ": strides must be multiples of 8 elements, not negative, and " +
                    "keep the elements of an output apart");
  return VSA_OK;
}

#define VSA_TRY(expr)            \
  do {                           \
    vsa_status _s = (expr);      \
    if (_s != VSA_OK) return _s; \
  } while (0)

// A view [B,H,N,D].  Outputs: no two elements may share memory, so that the dimensions, from the
// smallest stride to the largest, each step over all that lies inside.
vsa_status check_view(const vsa_view& v, int64_t B, int64_t H, int64_t N, int64_t D, bool output,
                      int64_t least, const char* name) {
  VSA_TRY(check_ptr(v.ptr, name));
  VSA_TRY(check_stride(v.stride_b, B, output ? 8 : least, name));
  VSA_TRY(check_stride(v.stride_h, H, output ? 8 : least, name));
  VSA_TRY(check_stride(v.stride_n, N, output ? 8 : least, name));
  if (output) {
    std::pair<int64_t, int64_t> d[3] = {{v.stride_b, B}, {v.stride_h, H}, {v.stride_n, N}};
    std::sort(d, d + 3);
    int64_t inside = D;
    for (const auto& e : d) {
      if (e.second <= 1) continue;
      if (e.first < inside)
        return fail(VSA_ERR_INVALID_ARG, std::string(name) + ": the output's elements share memory");
      inside = e.first * (e.second - 1) + inside;
    }
  }
  return VSA_OK;
}

bool same_view(const vsa_view& a, const vsa_view& b, int64_t B, int64_t H, int64_t N) {
  return a.ptr == b.ptr && (B <= 1 || a.stride_b == b.stride_b) &&
         (H <= 1 || a.stride_h == b.stride_h) && (N <= 1 || a.stride_n == b.stride_n);
}

// In place means the very same elements.
vsa_status check_in_place(const vsa_view& out, const vsa_view& in, int64_t B, int64_t H, int64_t N,
                          const char* name) {
  if (out.ptr == in.ptr && !same_view(out, in, B, H, N))
    return fail(VSA_ERR_INVALID_ARG,
                std::string(name) + ": in place needs the strides of the input");
  return VSA_OK;
}

vsa_status check_eps(float eps) {
  if (!(eps > 0.0f) || !std::isfinite(eps))
    return fail(VSA_ERR_INVALID_ARG, "eps must be finite and > 0");
  return VSA_OK;
}

// Extent a of a plan's grid, as it tells tokens' positions apart: of an empty grid, none does.
int extent(const vsa_plan_s* p, int a) { return p->n_tokens > p->n_prefix_tokens ? p->grid[a] : 0; }

vsa_status check_rope(const vsa_plan_s* p, const vsa_rope_s* r, int D) {
  if (r == nullptr) return fail(VSA_ERR_INVALID_ARG, "rope is NULL, and a tensor rotates");
  if (r->device != p->device || r->n_tokens != p->n_tokens)
    return fail(VSA_ERR_INVALID_ARG, "rope was built for another device or number of tokens");
  // as many tokens in another prefix or grid would turn by the wrong positions
  bool same = r->n_prefix == p->n_prefix_tokens;
  for (int a = 0; a < 3; ++a) same = same && r->grid[a] == extent(p, a);
  if (!same) return fail(VSA_ERR_INVALID_ARG, "rope was built for another prefix length or video grid");
  if (2 * r->P > D) return fail(VSA_ERR_INVALID_ARG, "rope turns more channels than D");
  return VSA_OK;
}

vsa_status check_gain(const void* gain, int type) {
  if (type != VSA_BF16 && type != VSA_F32)
    return fail(VSA_ERR_INVALID_ARG, "gain_type must be VSA_BF16 or VSA_F32");
  return gain == nullptr ? VSA_OK : check_ptr(gain, "gain");
}

vsa_status check_flags(int norm, int rotate) {
  if ((norm != 0 && norm != 1) || (rotate != 0 && rotate != 1))
    return fail(VSA_ERR_INVALID_ARG, "norm and rotate must be 0 or 1");
  return VSA_OK;
}

vsa_status check_act(int act) {
  if (act < VSA_ACT_IDENTITY || act > VSA_ACT_SILU)
    return fail(VSA_ERR_INVALID_ARG, "unknown activation");
  return VSA_OK;
}

// Channels of one side of a linear.
vsa_status check_width(int heads, int C, const char* name) {
  if (C <= 0 || C % 8 != 0 || C >= (1 << 20))
    return fail(VSA_ERR_INVALID_ARG, std::string(name) + " must be a multiple of 8 in (0, 2^20)");
  if (heads < 0 || (heads > 0 && C % heads != 0))
    return fail(VSA_ERR_INVALID_ARG, std::string(name) + " must split evenly into its heads");
  if (heads > 0 && C / heads != 64 && C / heads != 128)
    return fail(VSA_ERR_UNSUPPORTED, std::string(name) + ": heads must have 64 or 128 channels");
  return VSA_OK;
}

vsa_status check_rows(int B, int64_t N) {
  if (B < 0 || N < 0) return fail(VSA_ERR_INVALID_ARG, "B and N must be >= 0");
  if (N >= (int64_t(1) << 31) || int64_t(B) * N >= (int64_t(1) << 31) - 512)
    return fail(VSA_ERR_UNSUPPORTED, "too many rows for 32-bit TMA coordinates");
  return VSA_OK;
}

vsa_status check_linear_view(const vsa_view& v, int B, int64_t N, int heads, int C, bool output,
                             const char* name) {
  const int H = heads > 0 ? heads : 1;
  return check_view(v, B, H, N, C / H, output, 8, name);
}

vsa_status build_rope(const vsa_plan_s* p, const vsa_rope_desc& d, vsa_rope_s* r) {
  int width = 0;
  for (int a = 0; a < 3; ++a) {
    if (d.dim[a] < 0 || d.dim[a] % 2 != 0 || d.dim[a] > 128)
      return fail(VSA_ERR_INVALID_ARG, "rope: dim must be even and in [0, 128]");
    width += d.dim[a];
    if (!std::isfinite(d.offset[a]) || !std::isfinite(d.step[a]))
      return fail(VSA_ERR_INVALID_ARG, "rope: offset and step must be finite");
    if (d.inv_freq == nullptr && (!(d.theta[a] > 0.0) || !std::isfinite(d.theta[a])))
      return fail(VSA_ERR_INVALID_ARG, "rope: theta must be finite and > 0");
  }
  if (width < 2 || width > 128)
    return fail(VSA_ERR_INVALID_ARG, "rope: the dimensions must add up to 2 .. 128");
  if (d.halves != 0 && d.halves != 1) return fail(VSA_ERR_INVALID_ARG, "rope: halves must be 0 or 1");
  const int P = width / 2;
  if (d.halves == 1 && P % 4 != 0)
    return fail(VSA_ERR_UNSUPPORTED, "rope: halves needs a multiple of 8 rotated channels");
  if (d.inv_freq != nullptr)
    for (int i = 0; i < P; ++i)
      if (!std::isfinite(d.inv_freq[i]))
        return fail(VSA_ERR_INVALID_ARG, "rope: inv_freq must be finite");
  if (d.prefix_pos != nullptr)
    for (int64_t i = 0; i < 3 * p->n_prefix_tokens; ++i)
      if (!std::isfinite(d.prefix_pos[i]))
        return fail(VSA_ERR_INVALID_ARG, "rope: prefix_pos must be finite");

  r->device = p->device;
  r->n_tokens = p->n_tokens;
  r->n_prefix = p->n_prefix_tokens;
  for (int a = 0; a < 3; ++a) r->grid[a] = extent(p, a);
  r->P = P;
  r->halves = d.halves;
  r->start1 = d.dim[0] / 2;
  r->start2 = (d.dim[0] + d.dim[1]) / 2;
  r->tok.assign(size_t(p->n_tokens), int4{0, 0, 0, 0});
  const int64_t n_prefix = p->n_prefix_tokens;
  const auto prefix_at = [&](int64_t n, int a) {
    return d.prefix_pos != nullptr ? d.prefix_pos[3 * n + a] : 0.0;
  };
  std::vector<double> distinct;
  std::vector<int> row_of;             // table row of each coordinate of the grid's axis
  int start = 0;
  for (int a = 0; a < 3; ++a) {
    const int pairs = d.dim[a] / 2;
    distinct.clear();
    for (int64_t n = 0; n < n_prefix; ++n) distinct.push_back(prefix_at(n, a));
    for (int c = 0; c < p->grid[a]; ++c) distinct.push_back(d.offset[a] + d.step[a] * c);
    std::sort(distinct.begin(), distinct.end());
    distinct.erase(std::unique(distinct.begin(), distinct.end()), distinct.end());
    const auto find = [&](double x) {
      return int(std::lower_bound(distinct.begin(), distinct.end(), x) - distinct.begin());
    };
    const int64_t base = int64_t(r->tab.size());
    if (base + int64_t(distinct.size()) * pairs >= (int64_t(1) << 31))
      return fail(VSA_ERR_UNSUPPORTED, "rope: too many distinct positions");
    for (const double x : distinct)
      for (int i = 0; i < pairs; ++i) {
        const double f = d.inv_freq != nullptr ? d.inv_freq[start + i]
                                               : std::pow(d.theta[a], -2.0 * i / d.dim[a]);
        const double angle = x * f;
        if (!std::isfinite(angle))
          return fail(VSA_ERR_INVALID_ARG, "rope: an angle is not finite");
        r->tab.push_back(float2{float(std::cos(angle)), float(std::sin(angle))});
      }
    const auto set = [&](int64_t n, int row) {
      const int off = int(base + int64_t(row) * pairs - start);
      int4& t = r->tok[size_t(n)];
      (a == 0 ? t.x : a == 1 ? t.y : t.z) = off;
    };
    for (int64_t n = 0; n < n_prefix; ++n) set(n, find(prefix_at(n, a)));
    row_of.clear();
    for (int c = 0; c < p->grid[a]; ++c) row_of.push_back(find(d.offset[a] + d.step[a] * c));
    int64_t n = n_prefix;
    for (int i = 0; i < p->grid[0]; ++i)
      for (int j = 0; j < p->grid[1]; ++j)
        for (int k = 0; k < p->grid[2]; ++k, ++n) set(n, row_of[size_t(a == 0 ? i : a == 1 ? j : k)]);
    start += pairs;
  }
  return VSA_OK;
}

void free_rope(vsa_rope_s* r) {
  if (r->device >= 0) {
    int prev = -1;
    cudaGetDevice(&prev);
    cudaSetDevice(r->device);
    const RelaxedCapture relaxed;
    cudaFree(r->d_tab);
    cudaFree(r->d_tok);
    if (prev >= 0) cudaSetDevice(prev);
  }
  delete r;
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" {

vsa_status vsa_rope_create(vsa_plan p, const vsa_rope_desc* desc, vsa_rope* out) {
  if (p == nullptr || desc == nullptr || out == nullptr)
    return fail(VSA_ERR_INVALID_ARG, "NULL argument");
  *out = nullptr;
  vsa_rope_s* r = new (std::nothrow) vsa_rope_s();
  if (r == nullptr) return fail(VSA_ERR_INVALID_ARG, "out of host memory");
  vsa_status st;
  try {
    st = build_rope(p, *desc, r);
  } catch (const std::exception& e) {
    st = fail(VSA_ERR_INVALID_ARG, "out of host memory");
  }
  if (st != VSA_OK) {
    delete r;
    return st;
  }
  if (r->device >= 0) {
    int prev = -1;
    cudaError_t e = cudaGetDevice(&prev);
    if (e == cudaSuccess) e = cudaSetDevice(r->device);
    const size_t nt = r->tab.size() * sizeof(float2), nk = r->tok.size() * sizeof(int4);
    if (e == cudaSuccess) e = cudaMalloc(&r->d_tab, std::max<size_t>(16, nt));
    if (e == cudaSuccess) e = cudaMalloc(&r->d_tok, std::max<size_t>(16, nk));
    if (e == cudaSuccess) {
      Upload up;
      up.copy(r->d_tab, r->tab.data(), nt);
      up.copy(r->d_tok, r->tok.data(), nk);
      e = up.finish();
    }
    if (prev >= 0) cudaSetDevice(prev);
    if (e != cudaSuccess) {
      free_rope(r);
      return cuda_fail(e, "uploading rope tables");
    }
  }
  *out = r;
  return VSA_OK;
}

vsa_status vsa_rope_tables(vsa_rope r, int32_t* pairs, float* cos_sin) {
  if (r == nullptr) return fail(VSA_ERR_INVALID_ARG, "rope is NULL");
  if (pairs != nullptr) *pairs = r->P;
  if (cos_sin == nullptr) return VSA_OK;
  for (int64_t n = 0; n < r->n_tokens; ++n)
    for (int i = 0; i < r->P; ++i) {
      const int4& t = r->tok[size_t(n)];
      const int off = i < r->start1 ? t.x : (i < r->start2 ? t.y : t.z);
      const float2 cs = r->tab[size_t(off + i)];
      cos_sin[2 * (n * r->P + i)] = cs.x;
      cos_sin[2 * (n * r->P + i) + 1] = cs.y;
    }
  return VSA_OK;
}

vsa_status vsa_rope_destroy(vsa_rope r) {
  if (r != nullptr) free_rope(r);
  return VSA_OK;
}

vsa_status vsa_rope_apply(vsa_plan p, vsa_rope rope, const vsa_view* xv, const vsa_view* yv, int inverse,
                          int B, int H, int D, void* stream) {
  VSA_NVTX_RANGE();
  VSA_TRY(check_heads(p, B, H, D));
  if (xv == nullptr || yv == nullptr) return fail(VSA_ERR_INVALID_ARG, "x or y is NULL");
  const vsa_view x = *xv, y = *yv;
  VSA_TRY(check_rope(p, rope, D));
  if (inverse != 0 && inverse != 1) return fail(VSA_ERR_INVALID_ARG, "inverse must be 0 or 1");
  if (int64_t(B) * H == 0 || p->n_tokens == 0) return VSA_OK;
  VSA_TRY(check_view(x, B, H, p->n_tokens, D, false, 0, "x"));
  VSA_TRY(check_view(y, B, H, p->n_tokens, D, true, 8, "y"));
  VSA_TRY(check_in_place(y, x, B, H, p->n_tokens, "y"));
  HeadTensorArgs t = {};
  t.x = static_cast<const uint16_t*>(x.ptr);
  t.xb = x.stride_b, t.xh = x.stride_h, t.xn = x.stride_n;
  t.y = static_cast<uint16_t*>(y.ptr);
  t.yb = y.stride_b, t.yh = y.stride_h, t.yn = y.stride_n;
  t.rotate = 1;
  return launch_norm_rope(p, rope, &t, 1, 1.0f, inverse, false, B, H, D,
                          static_cast<cudaStream_t>(stream));
}

static vsa_status norm_rope_forward(vsa_plan p, vsa_rope rope, const vsa_head_tensor* tensors, int n,
                                    float eps, int B, int H, int D, bool tiled, void* stream) {
  VSA_TRY(check_heads(p, B, H, D));
  if (n < 1 || n > VSA_MAX_HEAD_TENSORS || tensors == nullptr)
    return fail(VSA_ERR_INVALID_ARG, "n must be in [1, 4] and tensors not NULL");
  VSA_TRY(check_eps(eps));
  const bool empty = int64_t(B) * H == 0 || p->n_tokens == 0;
  bool turns = false;
  HeadTensorArgs t[VSA_MAX_HEAD_TENSORS] = {};
  for (int i = 0; i < n; ++i) {
    const vsa_head_tensor& s = tensors[i];
    VSA_TRY(check_flags(s.norm, s.rotate));
    VSA_TRY(check_gain(s.gain, s.gain_type));
    if (s.gain != nullptr && !s.norm)
      return fail(VSA_ERR_INVALID_ARG, "a gain needs norm = 1");
    if (s.rotate) VSA_TRY(check_rope(p, rope, D));
    turns = turns || s.rotate;
    if (empty) continue;
    VSA_TRY(check_view(s.x, B, H, p->n_tokens, D, false, 0, "x"));
    if (tiled) {
      VSA_TRY(check_ptr(s.y.ptr, "y"));
      if (s.pooled != nullptr) VSA_TRY(check_ptr(s.pooled, "pooled"));
      if (s.y.ptr == s.x.ptr) return fail(VSA_ERR_INVALID_ARG, "the permute is not done in place");
    } else {
      VSA_TRY(check_view(s.y, B, H, p->n_tokens, D, true, 8, "y"));
      VSA_TRY(check_in_place(s.y, s.x, B, H, p->n_tokens, "y"));
    }
    t[i].x = static_cast<const uint16_t*>(s.x.ptr);
    t[i].xb = s.x.stride_b, t[i].xh = s.x.stride_h, t[i].xn = s.x.stride_n;
    t[i].gain = s.gain;
    t[i].gain_f32 = s.gain_type == VSA_F32;
    t[i].norm = s.norm;
    t[i].rotate = s.rotate;
    t[i].y = static_cast<uint16_t*>(s.y.ptr);
    t[i].yb = s.y.stride_b, t[i].yh = s.y.stride_h, t[i].yn = s.y.stride_n;
    t[i].pooled = s.pooled;
  }
  if (empty) return VSA_OK;
  // a rope that no tensor asked for was not looked at, and is not used
  return launch_norm_rope(p, turns ? rope : nullptr, t, n, eps, 0, tiled, B, H, D,
                          static_cast<cudaStream_t>(stream));
}

vsa_status vsa_norm_rope(vsa_plan p, vsa_rope rope, const vsa_head_tensor* tensors, int n, float eps,
                         int B, int H, int D, void* stream) {
  VSA_NVTX_RANGE();
  return norm_rope_forward(p, rope, tensors, n, eps, B, H, D, false, stream);
}

vsa_status vsa_norm_rope_permute_pool(vsa_plan p, vsa_rope rope, const vsa_head_tensor* tensors,
                                      int n, float eps, int B, int H, int D, void* stream) {
  VSA_NVTX_RANGE();
  return norm_rope_forward(p, rope, tensors, n, eps, B, H, D, true, stream);
}

vsa_status vsa_norm_rope_backward_workspace_size(vsa_plan p, int n, int D, size_t* bytes) {
  if (p == nullptr || bytes == nullptr) return fail(VSA_ERR_INVALID_ARG, "plan or bytes is NULL");
  if (n < 1 || n > VSA_MAX_HEAD_TENSORS) return fail(VSA_ERR_INVALID_ARG, "n must be in [1, 4]");
  if (D != 64 && D != 128) return fail(VSA_ERR_UNSUPPORTED, "head dim D must be 64 or 128");
  *bytes = norm_rope_backward_bytes(p, n, D);
  return VSA_OK;
}

vsa_status vsa_norm_rope_backward(vsa_plan p, vsa_rope rope, const vsa_head_grad* grads, int n,
                                  float eps, int tiled, int B, int H, int D, void* ws,
                                  size_t ws_bytes, void* stream) {
  VSA_NVTX_RANGE();
  VSA_TRY(check_heads(p, B, H, D));
  if (n < 1 || n > VSA_MAX_HEAD_TENSORS || grads == nullptr)
    return fail(VSA_ERR_INVALID_ARG, "n must be in [1, 4] and grads not NULL");
  if (tiled != 0 && tiled != 1) return fail(VSA_ERR_INVALID_ARG, "tiled must be 0 or 1");
  VSA_TRY(check_eps(eps));
  const bool empty = int64_t(B) * H == 0 || p->n_tokens == 0;
  const int64_t N = p->n_tokens;
  bool gains = false, turns = false;
  HeadGradArgs t[VSA_MAX_HEAD_TENSORS] = {};
  for (int i = 0; i < n; ++i) {
    const vsa_head_grad& s = grads[i];
    VSA_TRY(check_flags(s.norm, s.rotate));
    VSA_TRY(check_gain(s.gain, s.gain_type));
    if ((s.gain != nullptr || s.d_gain != nullptr) && !s.norm)
      return fail(VSA_ERR_INVALID_ARG, "a gain needs norm = 1");
    if (s.d_gain != nullptr) VSA_TRY(check_ptr(s.d_gain, "d_gain"));
    if (s.rotate) VSA_TRY(check_rope(p, rope, D));
    gains = gains || s.d_gain != nullptr;
    turns = turns || s.rotate;
    if (empty) continue;
    if (s.norm) VSA_TRY(check_view(s.x, B, H, N, D, false, 0, "x"));
    VSA_TRY(check_view(s.dx, B, H, N, D, true, 8, "dx"));
    if (tiled) {
      VSA_TRY(check_ptr(s.dy.ptr, "dy"));
      if (s.dy.ptr == s.dx.ptr) return fail(VSA_ERR_INVALID_ARG, "the unpermute is not done in place");
    } else {
      VSA_TRY(check_view(s.dy, B, H, N, D, false, 0, "dy"));
      VSA_TRY(check_in_place(s.dx, s.dy, B, H, N, "dx"));
    }
    t[i].dy = static_cast<const uint16_t*>(s.dy.ptr);
    t[i].gb = s.dy.stride_b, t[i].gh = s.dy.stride_h, t[i].gn = s.dy.stride_n;
    t[i].x = static_cast<const uint16_t*>(s.x.ptr);
    t[i].xb = s.x.stride_b, t[i].xh = s.x.stride_h, t[i].xn = s.x.stride_n;
    t[i].gain = s.gain;
    t[i].gain_f32 = s.gain_type == VSA_F32;
    t[i].norm = s.norm;
    t[i].rotate = s.rotate;
    t[i].dx = static_cast<uint16_t*>(s.dx.ptr);
    t[i].db = s.dx.stride_b, t[i].dh = s.dx.stride_h, t[i].dn = s.dx.stride_n;
    t[i].d_gain = s.d_gain;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) {
    for (int i = 0; i < n; ++i)
      if (grads[i].d_gain != nullptr) {
        const cudaError_t e = cudaMemsetAsync(grads[i].d_gain, 0, size_t(D) * sizeof(float), st);
        if (e != cudaSuccess) return cuda_fail(e, "clearing d_gain");
      }
    return VSA_OK;
  }
  if (gains) {
    if (ws == nullptr || ws_bytes < norm_rope_backward_bytes(p, n, D))
      return fail(VSA_ERR_WORKSPACE,
                  "workspace missing or too small (see vsa_norm_rope_backward_workspace_size)");
    VSA_TRY(check_ptr(ws, "ws"));
  }
  return launch_norm_rope_backward(p, turns ? rope : nullptr, t, n, eps, tiled == 1, B, H, D, ws, st);
}

vsa_status vsa_linear_workspace_size(vsa_plan p, int B, int64_t N, int C, int O, size_t* bytes) {
  if (p == nullptr || bytes == nullptr) return fail(VSA_ERR_INVALID_ARG, "plan or bytes is NULL");
  VSA_TRY(check_rows(B, N));
  VSA_TRY(check_width(0, C, "C"));
  VSA_TRY(check_width(0, O, "O"));
  *bytes = linear_bytes(p, B, N, C, O);
  return VSA_OK;
}

vsa_status vsa_linear(vsa_plan p, const vsa_linear_args* q, void* ws, size_t ws_bytes, void* stream) {
  VSA_NVTX_RANGE();
  VSA_TRY(check_device(p));
  if (q == nullptr) return fail(VSA_ERR_INVALID_ARG, "args is NULL");
  VSA_TRY(check_rows(q->B, q->N));
  VSA_TRY(check_width(q->x_heads, q->C, "C"));
  VSA_TRY(check_width(q->y_heads, q->O, "O"));
  VSA_TRY(check_act(q->act));
  if (q->bias_type != VSA_BF16 && q->bias_type != VSA_F32)
    return fail(VSA_ERR_INVALID_ARG, "bias_type must be VSA_BF16 or VSA_F32");
  if (q->bias != nullptr) VSA_TRY(check_ptr(q->bias, "bias"));
  VSA_TRY(check_ptr(q->w, "w"));
  if (int64_t(q->B) * q->N == 0) return VSA_OK;
  VSA_TRY(check_linear_view(q->x, q->B, q->N, q->x_heads, q->C, false, "x"));
  VSA_TRY(check_linear_view(q->y, q->B, q->N, q->y_heads, q->O, true, "y"));
  if (q->y.ptr == q->x.ptr || q->y.ptr == q->w)
    return fail(VSA_ERR_INVALID_ARG, "y must not overlap x or w");
  if (q->residual.ptr != nullptr) {
    VSA_TRY(check_linear_view(q->residual, q->B, q->N, q->y_heads, q->O, false, "residual"));
    VSA_TRY(check_in_place(q->y, q->residual, q->B, q->y_heads, q->N, "y"));
  }
  if (q->pre.ptr != nullptr) {
    VSA_TRY(check_linear_view(q->pre, q->B, q->N, q->y_heads, q->O, true, "pre"));
    if (q->pre.ptr == q->x.ptr || q->pre.ptr == q->w || q->pre.ptr == q->y.ptr ||
        q->pre.ptr == q->residual.ptr)
      return fail(VSA_ERR_INVALID_ARG, "pre must not overlap another tensor");
  }
  if (ws != nullptr) {
    VSA_TRY(check_ptr(ws, "ws"));
    if (ws_bytes < linear_bytes(p, q->B, q->N, q->C, q->O))
      return fail(VSA_ERR_WORKSPACE, "workspace too small (see vsa_linear_workspace_size)");
  }
  return launch_linear(p, *q, ws, static_cast<cudaStream_t>(stream));
}

vsa_status vsa_linear_backward_workspace_size(vsa_plan p, int B, int64_t N, int C, int O,
                                              size_t* bytes) {
  if (p == nullptr || bytes == nullptr) return fail(VSA_ERR_INVALID_ARG, "plan or bytes is NULL");
  VSA_TRY(check_rows(B, N));
  VSA_TRY(check_width(0, C, "C"));
  VSA_TRY(check_width(0, O, "O"));
  *bytes = linear_backward_bytes(p, B, N, C, O);
  return VSA_OK;
}

vsa_status vsa_linear_backward(vsa_plan p, const vsa_linear_grad_args* q, void* ws, size_t ws_bytes,
                               void* stream) {
  VSA_NVTX_RANGE();
  VSA_TRY(check_device(p));
  if (q == nullptr) return fail(VSA_ERR_INVALID_ARG, "args is NULL");
  VSA_TRY(check_rows(q->B, q->N));
  VSA_TRY(check_width(q->x_heads, q->C, "C"));
  VSA_TRY(check_width(q->y_heads, q->O, "O"));
  VSA_TRY(check_act(q->x_act));
  if (q->dw != nullptr) VSA_TRY(check_ptr(q->dw, "dw"));
  if (q->db != nullptr) VSA_TRY(check_ptr(q->db, "db"));
  if (int64_t(q->B) * q->N > 0) {
    VSA_TRY(check_linear_view(q->dy, q->B, q->N, q->y_heads, q->O, false, "dy"));
    if (q->dx.ptr != nullptr) {
      VSA_TRY(check_ptr(q->w, "w"));
      VSA_TRY(check_linear_view(q->dx, q->B, q->N, q->x_heads, q->C, true, "dx"));
      if (q->dx.ptr == q->dy.ptr || q->dx.ptr == q->w || q->dx.ptr == q->x.ptr)
        return fail(VSA_ERR_INVALID_ARG, "dx must not overlap dy, x or w");
      if (q->x_pre.ptr != nullptr) {
        VSA_TRY(check_linear_view(q->x_pre, q->B, q->N, q->x_heads, q->C, false, "x_pre"));
        VSA_TRY(check_in_place(q->dx, q->x_pre, q->B, q->x_heads, q->N, "dx"));
      }
      if (q->dx_add.ptr != nullptr) {
        if (q->x_pre.ptr != nullptr)
          return fail(VSA_ERR_INVALID_ARG, "dx_add does not go with x_pre");
        VSA_TRY(check_linear_view(q->dx_add, q->B, q->N, q->x_heads, q->C, false, "dx_add"));
        VSA_TRY(check_in_place(q->dx, q->dx_add, q->B, q->x_heads, q->N, "dx"));
      }
    }
    if (q->dw != nullptr) {
      VSA_TRY(check_linear_view(q->x, q->B, q->N, q->x_heads, q->C, false, "x"));
      if (q->dw == q->dy.ptr || q->dw == q->x.ptr || q->dw == q->w || q->dw == q->dx.ptr)
        return fail(VSA_ERR_INVALID_ARG, "dw must not overlap another tensor");
    }
    if (q->dx.ptr != nullptr || q->dw != nullptr || q->db != nullptr) {
      if (ws == nullptr || ws_bytes < linear_backward_bytes(p, q->B, q->N, q->C, q->O))
        return fail(VSA_ERR_WORKSPACE,
                    "workspace missing or too small (see vsa_linear_backward_workspace_size)");
      VSA_TRY(check_ptr(ws, "ws"));
    }
  }
  return launch_linear_backward(p, *q, ws, static_cast<cudaStream_t>(stream));
}

vsa_status vsa_act_backward(vsa_plan p, const void* dy, const void* pre, int act, void* out,
                            int64_t n, void* stream) {
  VSA_NVTX_RANGE();
  VSA_TRY(check_device(p));
  VSA_TRY(check_act(act));
  if (n < 0 || n % 8 != 0) return fail(VSA_ERR_INVALID_ARG, "n must be a multiple of 8, >= 0");
  if (n == 0) return VSA_OK;
  VSA_TRY(check_ptr(dy, "dy"));
  VSA_TRY(check_ptr(pre, "pre"));
  VSA_TRY(check_ptr(out, "out"));
  const cudaError_t e = launch_act_backward(dy, pre, act, out, n, p->num_sms,
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSA_OK : cuda_fail(e, "act backward launch");
}

}  // extern "C"
