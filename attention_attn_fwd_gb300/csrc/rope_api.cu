// C ABI of the norm and rotation of queries and keys: argument checks and
// launches.  No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "attn_host.h"
#include "rope_common.cuh"

namespace {

constexpr size_t kWorkspaceAlign = 256;
constexpr int kMaxTokens = 0x7fffffff - 4096;  // group numbers stay in 32 bits
constexpr int kMaxHeads = 1 << 20;

bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

struct Range {
  const void* p;
  size_t n;
};

struct Sizes {
  int B, S, D;
};

// A strided view with the strides of dimensions of one element at 0, its
// heads, and the elements from its first to its last.
struct View {
  const void* p;
  long long b, s, h;
  int H;
  long long extent;
  Range range() const { return {p, static_cast<size_t>(extent) * 2}; }
};

attn_status_t make_view(const attn_heads_t* v, const Sizes& z, int H,
                        View* out) {
  if (v == nullptr || v->p == nullptr) return ATTN_ERR_INVALID_ARG;
  out->p = v->p;
  out->H = H;
  out->b = z.B > 1 ? v->stride_b : 0;
  out->s = z.S > 1 ? v->stride_s : 0;
  out->h = H > 1 ? v->stride_h : 0;
  if (out->b < 0 || out->s < 0 || out->h < 0) return ATTN_ERR_INVALID_ARG;
  if (out->b % 8 || out->s % 8 || out->h % 8 || misaligned(v->p, 16))
    return ATTN_ERR_ALIGNMENT;
  constexpr long long kMost = 1LL << 46;  // elements of a view
  if (out->b > kMost || out->s > kMost || out->h > kMost)
    return ATTN_ERR_INVALID_ARG;
  const __int128 e = static_cast<__int128>(z.B - 1) * out->b +
                     static_cast<__int128>(z.S - 1) * out->s +
                     static_cast<__int128>(H - 1) * out->h + z.D;
  if (e > kMost) return ATTN_ERR_INVALID_ARG;
  out->extent = static_cast<long long>(e);
  return ATTN_OK;
}

// A dimension of places: its stride and how many there are.
struct Dim {
  long long stride;
  int n;
};

// Whether runs of `extent` elements at the places of `count` dimensions share no
// element: each dimension, from the smallest stride up, steps over all that
// lies within.
bool nested(long long extent, Dim* d, int count) {
  std::sort(d, d + count,
            [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  for (int i = 0; i < count; ++i) {
    if (d[i].n == 1) continue;
    if (d[i].stride < extent) return false;
    extent += d[i].stride * (d[i].n - 1);
  }
  return true;
}

// Whether no two places of a view share an element.
bool writable(const View& v, const Sizes& z) {
  Dim d[3] = {{v.b, z.B}, {v.s, z.S}, {v.h, v.H}};
  return nested(z.D, d, 3);
}

// Whether two writable views share no element: for some of the dimensions, all
// of x's places along these lie before y's, and so they do at every step of the
// others, which both views take alike and which step over what lies within.
// (All dimensions: apart altogether.  Heads alone: side by side in a token, as
// parts of a packed projection.  Heads and tokens: parts of a packed tensor
// with the heads ahead of the tokens.  None: in turn.)
bool apart(const View& x, const View& y, const Sizes& z) {
  const long long off =
      (reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p)) / 2;
  if (off < 0) return apart(y, x, z);
  const Dim dx[3] = {{x.b, z.B}, {x.s, z.S}, {x.h, x.H}};
  const Dim dy[3] = {{y.b, z.B}, {y.s, z.S}, {y.h, y.H}};
  for (int within = 0; within < 8; ++within) {
    long long ex = z.D, ey = z.D;
    Dim rest[3];
    int count = 0;
    bool alike = true;
    for (int i = 0; i < 3; ++i) {
      if (within >> i & 1) {
        ex += dx[i].stride * (dx[i].n - 1);
        ey += dy[i].stride * (dy[i].n - 1);
        continue;
      }
      // (The stride of a dimension of one element says nothing.)
      const Dim& longer = dx[i].n >= dy[i].n ? dx[i] : dy[i];
      alike &= std::min(dx[i].n, dy[i].n) == 1 ||
               dx[i].stride == dy[i].stride;
      rest[count++] = longer;
    }
    if (alike && off >= ex && nested(off + ey, rest, count)) return true;
  }
  return false;
}

bool any_overlap(const Range& a, const Range* others, int count) {
  for (int i = 0; i < count; ++i)
    if (attn::ranges_overlap(a.p, a.n, others[i].p, others[i].n)) return true;
  return false;
}

attn_status_t check_rope(const attn_rope_t* r) {
  if (r == nullptr || r->D <= 0 || r->rot < 0 || r->rot > r->D || r->axes < 1 ||
      r->axes > 255)
    return ATTN_ERR_INVALID_ARG;
  if ((r->D != 64 && r->D != 128) || r->rot % 8 != 0)
    return ATTN_ERR_UNSUPPORTED;
  if (r->rot > 0 &&
      (r->phase == nullptr || (r->axes > 1 && r->axis == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (misaligned(r->phase, 8)) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

attn_status_t check_sizes(int B, int S, int Hq, int Hkv, float eps,
                          int weight_f32, const void* wq, const void* wk,
                          attn_dtype_t dtype) {
  if (B < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || Hq > kMaxHeads ||
      Hkv > kMaxHeads || (dtype != ATTN_F16 && dtype != ATTN_BF16) ||
      static_cast<long long>(B) * S > kMaxTokens)
    return ATTN_ERR_INVALID_ARG;
  // Thread blocks of a launch: 8 tokens of 8 heads of a kind at least.
  const long long blocks = (Hq + 7) / 8 + 2LL * ((Hkv + 7) / 8);
  if ((static_cast<long long>(B) * S / 8 + 1) * blocks > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  if (wq != nullptr || wk != nullptr) {
    if (!(eps > 0.f) || !std::isfinite(eps)) return ATTN_ERR_INVALID_ARG;
    const uintptr_t a = weight_f32 ? 4 : 2;
    if (misaligned(wq, a) || misaligned(wk, a)) return ATTN_ERR_ALIGNMENT;
  }
  return ATTN_OK;
}

bool on_device_or_null(const void* const* p, int n, int dev) {
  for (int i = 0; i < n; ++i)
    if (p[i] != nullptr && !attn::on_device(p[i], dev)) return false;
  return true;
}

void fill_rope(attn::rope::RopeParams* p, const attn_rope_t* r) {
  p->phase = r->phase;
  p->axis = r->axes > 1 ? r->axis : nullptr;
  p->rot = r->rot;
}

attn_status_t fwd_impl(const attn_rope_t* rope, const attn_heads_t* q,
                       const attn_heads_t* k, const attn_heads_t* v,
                       const void* wq, const void* wk, int weight_f32,
                       float eps, const int* positions, const int* lens,
                       const int* new_lens, const int* offset, void* q_out,
                       void* k_out, void* v_out, int B, int S, int Hq, int Hkv,
                       int capacity, attn_dtype_t dtype, cudaStream_t stream) {
  attn_status_t st = check_rope(rope);
  if (st != ATTN_OK) return st;
  st = check_sizes(B, S, Hq, Hkv, eps, weight_f32, wq, wk, dtype);
  if (st != ATTN_OK) return st;
  if (positions != nullptr && offset != nullptr) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || S == 0) return ATTN_OK;
  if (capacity < S) return ATTN_ERR_INVALID_ARG;
  if ((v == nullptr) != (v_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  const Sizes z{B, S, rope->D};
  const attn_heads_t* src[3] = {q, k, v};
  const int H[3] = {Hq, Hkv, Hkv};
  const int n = v != nullptr ? 3 : 2;
  View x[3];
  for (int i = 0; i < n; ++i) {
    st = make_view(src[i], z, H[i], &x[i]);
    if (st != ATTN_OK) return st;
  }
  void* y[3] = {q_out, k_out, v_out};
  for (int i = 0; i < n; ++i) {
    if (y[i] == nullptr) return ATTN_ERR_INVALID_ARG;
    if (misaligned(y[i], 16)) return ATTN_ERR_ALIGNMENT;
  }
  if (misaligned(positions, 4) || misaligned(lens, 4) ||
      misaligned(new_lens, 4) || misaligned(offset, 4))
    return ATTN_ERR_ALIGNMENT;
  const size_t tokens = static_cast<size_t>(B) * S;
  const size_t len_bytes = static_cast<size_t>(B) * 4;
  const size_t w_bytes = static_cast<size_t>(rope->D) * (weight_f32 ? 4 : 2);
  const size_t kv_bytes = static_cast<size_t>(B) * Hkv * capacity * rope->D * 2;
  const Range in[] = {
      x[0].range(),
      x[1].range(),
      n == 3 ? x[2].range() : Range{nullptr, 0},
      {wq, wq ? w_bytes : 0},
      {wk, wk ? w_bytes : 0},
      {positions, positions ? tokens * rope->axes * 4 : 0},
      {lens, lens ? len_bytes : 0},
      {new_lens, new_lens ? len_bytes : 0},
      {offset, offset ? size_t(4) : 0},
      {rope->phase, static_cast<size_t>(rope->rot) * 4},
      {rope->axis, rope->axes > 1 ? static_cast<size_t>(rope->rot / 2) : 0}};
  const Range out[] = {{q_out, tokens * Hq * rope->D * 2},
                       {k_out, kv_bytes},
                       {v_out, v_out ? kv_bytes : 0}};
  for (int i = 0; i < 3; ++i)
    if (any_overlap(out[i], in, 11) || any_overlap(out[i], out + i + 1, 2 - i))
      return ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  const void* mem[] = {x[0].p, x[1].p, n == 3 ? x[2].p : nullptr,
                       q_out,  k_out,  v_out,
                       wq,     wk,     positions,
                       lens,   new_lens, offset,
                       rope->rot > 0 ? rope->phase : nullptr,
                       rope->axes > 1 ? rope->axis : nullptr};
  if (!on_device_or_null(mem, 14, dev)) return ATTN_ERR_INVALID_ARG;
  attn::rope::RopeParams p{};
  fill_rope(&p, rope);
  for (int i = 0; i < n; ++i) {
    p.x[i] = static_cast<const uint16_t*>(x[i].p);
    p.x_b[i] = x[i].b;
    p.x_s[i] = x[i].s;
    p.x_h[i] = x[i].h;
    p.y[i] = static_cast<uint16_t*>(y[i]);
  }
  p.pos = positions;
  p.offset = offset;
  p.lens = lens;
  p.new_lens = new_lens;
  p.w[0] = wq;
  p.w[1] = wk;
  p.w_f32 = weight_f32 != 0;
  p.eps = eps;
  p.B = B;
  p.S = S;
  p.tokens = B * S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.heads = Hq + (n - 1) * Hkv;
  p.capacity = capacity;
  p.status = attn::device_status_word(dev);
  const int sms = attn::device_sms(dev);
  if (p.status == nullptr || sms <= 0) return ATTN_ERR_CUDA;
  const cudaError_t err = attn::rope::launch_rope(
      rope->D, dtype == ATTN_BF16, rope->interleaved != 0, p, sms, stream);
  return err == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int current_sms() {
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = attn::device_sms(dev);
  cudaGetLastError();  // no device: not an error of the caller's
  return sms > 0 ? sms : 152;  // a GB300's without a device
}

size_t bwd_workspace(int sms, int D) {
  return static_cast<size_t>(attn::rope::bwd_ctas(sms)) * D * 4;
}

attn_status_t bwd_impl(const attn_rope_t* rope, const void* dq, const void* dk,
                       const void* dv, const attn_heads_t* q,
                       const attn_heads_t* k, const void* wq, const void* wk,
                       int weight_f32, float eps, const int* positions,
                       const int* offset, const attn_heads_t* dxq,
                       const attn_heads_t* dxk, const attn_heads_t* dxv,
                       float* dwq, float* dwk, int B, int S, int Hq, int Hkv,
                       attn_dtype_t dtype, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  attn_status_t st = check_rope(rope);
  if (st != ATTN_OK) return st;
  st = check_sizes(B, S, Hq, Hkv, eps, weight_f32, wq, wk, dtype);
  if (st != ATTN_OK) return st;
  if (positions != nullptr && offset != nullptr) return ATTN_ERR_INVALID_ARG;
  // Gradients of weights that are there, and of no others.
  if ((dwq != nullptr) != (wq != nullptr) || (dwk != nullptr) != (wk != nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (misaligned(dwq, 4) || misaligned(dwk, 4)) return ATTN_ERR_ALIGNMENT;
  const bool norm = wq != nullptr || wk != nullptr;
  const bool empty = B == 0 || S == 0;
  const int n = dv != nullptr ? 3 : 2;
  const Sizes z{B, S, rope->D};
  const void* dy[3] = {dq, dk, dv};
  const attn_heads_t* dst[3] = {dxq, dxk, dxv};
  const int H[3] = {Hq, Hkv, Hkv};
  View x[2] = {}, dx[3] = {};
  if (!empty) {
    if ((dv == nullptr) != (dxv == nullptr)) return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
      if (dy[i] == nullptr) return ATTN_ERR_INVALID_ARG;
      if (misaligned(dy[i], 16)) return ATTN_ERR_ALIGNMENT;
      st = make_view(dst[i], z, H[i], &dx[i]);
      if (st != ATTN_OK) return st;
      if (!writable(dx[i], z)) return ATTN_ERR_INVALID_ARG;
    }
    // What was normed is read again.
    if (wq != nullptr && (st = make_view(q, z, Hq, &x[0])) != ATTN_OK) return st;
    if (wk != nullptr && (st = make_view(k, z, Hkv, &x[1])) != ATTN_OK)
      return st;
    if (misaligned(positions, 4) || misaligned(offset, 4))
      return ATTN_ERR_ALIGNMENT;
  }
  if (empty && !norm) return ATTN_OK;
  if (norm && (workspace == nullptr || misaligned(workspace, kWorkspaceAlign)))
    return ATTN_ERR_ALIGNMENT;
  const int sms = current_sms();
  const size_t need = norm ? bwd_workspace(sms, rope->D) : 0;
  if (norm && workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  const size_t tokens = static_cast<size_t>(B) * S;
  const size_t w_bytes = static_cast<size_t>(rope->D) * (weight_f32 ? 4 : 2);
  const size_t row = static_cast<size_t>(rope->D) * 2;
  const Range in[] = {
      {dq, tokens * Hq * row},
      {dk, tokens * Hkv * row},
      {dv, dv ? tokens * Hkv * row : 0},
      wq != nullptr && !empty ? x[0].range() : Range{nullptr, 0},
      wk != nullptr && !empty ? x[1].range() : Range{nullptr, 0},
      {wq, wq ? w_bytes : 0},
      {wk, wk ? w_bytes : 0},
      {positions, positions ? tokens * rope->axes * 4 : 0},
      {offset, offset ? size_t(4) : 0},
      {rope->phase, static_cast<size_t>(rope->rot) * 4},
      {rope->axis, rope->axes > 1 ? static_cast<size_t>(rope->rot / 2) : 0}};
  const size_t dw_bytes = static_cast<size_t>(rope->D) * 4;
  const Range none{nullptr, 0};
  const Range out[] = {{dwq, dwq ? dw_bytes : 0},
                       {dwk, dwk ? dw_bytes : 0},
                       {workspace, need},
                       empty ? none : dx[0].range(),
                       empty ? none : dx[1].range(),
                       empty || n < 3 ? none : dx[2].range()};
  for (int i = 0; i < 6; ++i) {
    if (any_overlap(out[i], in, 11)) return ATTN_ERR_INVALID_ARG;
    if (i < 3 && any_overlap(out[i], out + i + 1, 5 - i))
      return ATTN_ERR_INVALID_ARG;
  }
  if (!empty)
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if (!apart(dx[i], dx[j], z)) return ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  const void* mem[] = {dq, dk, dv, x[0].p, x[1].p, dx[0].p, dx[1].p,
                       n == 3 ? dx[2].p : nullptr, wq, wk, dwq, dwk,
                       positions, offset, norm ? workspace : nullptr,
                       rope->rot > 0 ? rope->phase : nullptr,
                       rope->axes > 1 ? rope->axis : nullptr};
  if (!on_device_or_null(mem, 17, dev)) return ATTN_ERR_INVALID_ARG;
  if (empty) {  // no rows: the weights' gradients are sums of nothing
    if (dwq != nullptr &&
        cudaMemsetAsync(dwq, 0, dw_bytes, stream) != cudaSuccess)
      return ATTN_ERR_CUDA;
    if (dwk != nullptr &&
        cudaMemsetAsync(dwk, 0, dw_bytes, stream) != cudaSuccess)
      return ATTN_ERR_CUDA;
    return ATTN_OK;
  }
  attn::rope::RopeParams p{};
  fill_rope(&p, rope);
  for (int i = 0; i < n; ++i) {
    p.y[i] = static_cast<uint16_t*>(const_cast<void*>(dy[i]));
    p.dx[i] = static_cast<uint16_t*>(const_cast<void*>(dx[i].p));
    p.dx_b[i] = dx[i].b;
    p.dx_s[i] = dx[i].s;
    p.dx_h[i] = dx[i].h;
  }
  for (int i = 0; i < 2; ++i) {
    p.x[i] = static_cast<const uint16_t*>(x[i].p);
    p.x_b[i] = x[i].b;
    p.x_s[i] = x[i].s;
    p.x_h[i] = x[i].h;
  }
  p.pos = positions;
  p.offset = offset;
  p.w[0] = wq;
  p.w[1] = wk;
  p.dw[0] = dwq;
  p.dw[1] = dwk;
  p.w_f32 = weight_f32 != 0;
  p.eps = eps;
  p.part = static_cast<float*>(workspace);
  p.B = B;
  p.S = S;
  p.tokens = B * S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.heads = Hq + (n - 1) * Hkv;
  p.capacity = S;
  p.status = attn::device_status_word(dev);
  if (p.status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t err = attn::rope::launch_rope_bwd(
      rope->D, dtype == ATTN_BF16, rope->interleaved != 0, p, sms, stream);
  return err == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_rope_phase(const double* freq, int n,
                              unsigned long long* phase) {
  if (n < 0 || (n > 0 && (freq == nullptr || phase == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(freq[i]) <= 0x1p32)) return ATTN_ERR_INVALID_ARG;
  // 1 / (2 pi) as the sum of two doubles; the product's rounding error is kept,
  // so that the fraction of a turn is right to 2^-64 or so.
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  for (int i = 0; i < n; ++i) {
    const double f = std::fabs(freq[i]);
    const double hi = f * kHi;
    const double lo = std::fma(f, kHi, -hi) + f * kLo;
    const double frac = hi - std::floor(hi);  // exact
    const double part = std::floor(std::ldexp(frac, 63));
    const double rest = std::ldexp(frac, 64) - 2 * part + std::ldexp(lo, 64);
    const unsigned long long turn =
        2 * static_cast<unsigned long long>(part) +
        static_cast<unsigned long long>(std::llrint(rest));
    phase[i] = freq[i] < 0 ? 0 - turn : turn;
  }
  return ATTN_OK;
}

attn_status_t attn_qk_rope(const attn_rope_t* rope, const attn_heads_t* q,
                           const attn_heads_t* k, const attn_heads_t* v,
                           const void* q_weight, const void* k_weight,
                           int weight_f32, float eps, const int* positions,
                           const int* lens, const int* new_lens,
                           const int* offset, void* q_out, void* k_out,
                           void* v_out, int B, int S, int Hq, int Hkv,
                           int capacity, attn_dtype_t dtype,
                           attn_stream_t stream) {
  return fwd_impl(rope, q, k, v, q_weight, k_weight, weight_f32, eps,
                  positions, lens, new_lens, offset, q_out, k_out, v_out, B, S,
                  Hq, Hkv, capacity, dtype,
                  reinterpret_cast<cudaStream_t>(stream));
}

attn_status_t attn_qk_rope_bwd(
    const attn_rope_t* rope, const void* dq_out, const void* dk_out,
    const void* dv_out, const attn_heads_t* q, const attn_heads_t* k,
    const void* q_weight, const void* k_weight, int weight_f32, float eps,
    const int* positions, const int* offset, const attn_heads_t* dq,
    const attn_heads_t* dk, const attn_heads_t* dv, float* dq_weight,
    float* dk_weight, int B, int S, int Hq, int Hkv, attn_dtype_t dtype,
    void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  return bwd_impl(rope, dq_out, dk_out, dv_out, q, k, q_weight, k_weight,
                  weight_f32, eps, positions, offset, dq, dk, dv, dq_weight,
                  dk_weight, B, S, Hq, Hkv, dtype, workspace, workspace_bytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

size_t attn_qk_rope_bwd_workspace_bytes(int D) {
  if (D != 64 && D != 128) return 0;
  return bwd_workspace(current_sms(), D);
}

}  // extern "C"
