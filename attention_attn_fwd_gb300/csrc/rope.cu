// Norms of queries and keys and their rotation by position, on the way from
// the projections to the attention, and the backward pass.
//
// Mathematics, for a row x of D numbers (one head of one token):
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps)      (n = x without weights)
//   pair (a, b) of n at angle t:  (a cos t - b sin t, a sin t + b cos t);
// and back, from the gradient dy of the result:
//   dn: the pairs of dy turned by -t,  g = dn w,  dw = sum over rows of dn x r,
//   dx = r (g - x r^2 mean(g x)).
//
// Angles: position times frequency in 64-bit fixed point of a turn.  The
// product modulo 2^64 drops whole turns exactly, so far positions lose
// nothing; the upper 32 bits as a fraction of a turn go to sincospif.
//
// Layout: a group of D / 8 lanes holds one row, eight elements a lane, chosen
// so that both numbers of its four pairs are its own: two runs of four
// elements, rot / 2 apart (or eight neighbours).  No exchange but the sums of
// squares, and no angle is computed twice for a row; a group keeps its token's
// sines for a block of heads.  Everything between load and store is fp32; one
// rounding, to the output.
#include <algorithm>

#include "kv8_common.cuh"
#include "rope_common.cuh"

namespace attn {
namespace rope {
namespace {

using kv8::launch_pdl;
using kv8::start_after_previous;
using kv8::unpack2;

constexpr unsigned kFull = 0xffffffffu;

// What a lane holds of each row.
template <int D, bool kInterleaved>
struct Lane {
  int at[2];     // first elements of its two runs of four
  int pair;      // its first pair; -1: not rotated
  __device__ __forceinline__ explicit Lane(int lane, int rot) {
    if (kInterleaved) {
      at[0] = 8 * lane;
      at[1] = at[0] + 4;
      pair = at[0] < rot ? 4 * lane : -1;
    } else if (8 * lane < rot) {
      at[0] = 4 * lane;
      at[1] = rot / 2 + 4 * lane;
      pair = at[0];
    } else {
      at[0] = 8 * lane;
      at[1] = at[0] + 4;
      pair = -1;
    }
  }
};

// Numbers i and j of the lane's eight that pair e rotates.
template <bool kInterleaved>
__host__ __device__ constexpr int first_of(int e) {
  return kInterleaved ? 2 * e : e;
}
template <bool kInterleaved>
__host__ __device__ constexpr int second_of(int e) {
  return kInterleaved ? 2 * e + 1 : e + 4;
}

// A token and what its rows need.
struct Token {
  int b, s;
  int row;      // its row in K's and V's outputs
  bool in;      // there is such a token
  long long pos;
};

__device__ __forceinline__ Token find_token(const RopeParams& p, int t) {
  Token k;
  k.in = t < p.tokens;
  k.b = k.in ? t / p.S : 0;
  k.s = k.in ? t - k.b * p.S : 0;
  int len = p.S, n = p.S, start = 0;
  if (p.lens != nullptr) {
    len = kv8::clamp_len(p.lens[k.b], p.capacity, p.status);
    n = p.new_lens == nullptr
            ? kv8::clamp_len(p.S, len, p.status)
            : kv8::clamp_len(p.new_lens[k.b], min(p.S, len), p.status);
    start = len - n;
  } else if (p.new_lens != nullptr) {
    n = kv8::clamp_len(p.new_lens[k.b], p.S, p.status);
  }
  k.in = k.in && k.s < n;
  k.row = start + k.s;
  k.pos = k.row;
  if (p.offset != nullptr) k.pos += *p.offset;
  return k;
}

// cos and sin of the lane's four pairs at a token.
__device__ __forceinline__ void turns(const RopeParams& p, const Token& k,
                                      int pair, float* c, float* s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (pair < 0 || !k.in) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    long long pos = k.pos;
    if (p.pos != nullptr) {
      const int a = p.axis == nullptr ? 0 : __ldg(p.axis + pair + e);
      pos = __ldg(p.pos + (static_cast<long long>(a) * p.B + k.b) * p.S + k.s);
    }
    const unsigned long long turn =
        static_cast<unsigned long long>(pos) * __ldg(p.phase + pair + e);
    // Half turns in [-1, 1): off by 2^-24 of itself at most.
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f,
              &s[e], &c[e]);
  }
}

template <bool kBF16>
__device__ __forceinline__ void load8(const uint16_t* row, const int* at,
                                      uint2* w) {
  w[0] = __ldg(reinterpret_cast<const uint2*>(row + at[0]));
  w[1] = __ldg(reinterpret_cast<const uint2*>(row + at[1]));
}
template <bool kBF16>
__device__ __forceinline__ void widen(const uint2* w, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2<kBF16>(w[i].x), b = unpack2<kBF16>(w[i].y);
    x[4 * i] = a.x;
    x[4 * i + 1] = a.y;
    x[4 * i + 2] = b.x;
    x[4 * i + 3] = b.y;
  }
}
template <bool kBF16>
__device__ __forceinline__ void store8(uint16_t* row, const int* at,
                                       const float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint2*>(row + at[i]) =
        make_uint2(ptx::pack2<kBF16>(x[4 * i], x[4 * i + 1]),
                   ptx::pack2<kBF16>(x[4 * i + 2], x[4 * i + 3]));
}

// The lane's norm weights.
template <bool kBF16>
__device__ __forceinline__ void load_weights(const RopeParams& p, int kind,
                                             const int* at, float* w) {
  if (p.w[kind] == nullptr) return;
  if (p.w_f32) {
    const float* f = static_cast<const float*>(p.w[kind]);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __ldg(f + at[i / 4] + i % 4);
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p.w[kind]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = __ldg(h + at[i / 4] + i % 4);
      w[i] = unpack2<kBF16>(word).x;
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int i = kLanes / 2; i > 0; i /= 2) x += __shfl_xor_sync(kFull, x, i);
  return x;
}

// x becomes x f, and the row's norm factor is r f: f is 1 but for rows whose
// squares pass fp32's largest number.  Returns r.
template <int D>
__device__ __forceinline__ float norm_factor(float* x, float eps, float* f) {
  *f = 1.f;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = group_sum<D / 8>(ss);
  if (__any_sync(kFull, ss == INFINITY)) {
    const bool big = ss == INFINITY;
    if (big) *f = 0x1p-96f;
    float again = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= *f;
      again = fmaf(x[i], x[i], again);
    }
    again = group_sum<D / 8>(again);
    if (big) {
      ss = again;
      eps = 0.f;
    }
  }
  return rsqrtf(fmaf(ss, 1.f / D, eps));
}

// The kind of a head (0 Q, 1 K, 2 V) in the list of all, and its number there.
__device__ __forceinline__ int head_kind(const RopeParams& p, int h, int* at) {
  const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
  *at = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
  return kind;
}

// ---------------------------------------------------------------- forward
constexpr int kAhead = 4;  // rows of a group in flight

template <int D, bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;
  const Lane<D, kInterleaved> lane(threadIdx.x % kLanes, p.rot);
  start_after_previous();
  const Token k =
      find_token(p, blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes);
  const int h0 = blockIdx.y * p.head_block;
  const int h1 = min(h0 + p.head_block, p.heads);

  auto load = [&](int h, uint2* w) {
    int at;
    const int kind = head_kind(p, h, &at);
    load8<kBF16>(p.x[kind] + k.b * p.x_b[kind] + k.s * p.x_s[kind] +
                     at * p.x_h[kind],
                 lane.at, w);
  };
  uint2 in[kAhead][2];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    in[i][0] = in[i][1] = make_uint2(0u, 0u);
    if (k.in && h0 + i < h1) load(h0 + i, in[i]);
  }
  float wq[8], wk[8], c[4], s[4];
  load_weights<kBF16>(p, 0, lane.at, wq);
  load_weights<kBF16>(p, 1, lane.at, wk);
  turns(p, k, lane.pair, c, s);

  for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (h + i >= h1) break;
      int at;
      const int kind = head_kind(p, h + i, &at);
      const int H = kind == 0 ? p.Hq : p.Hkv;
      const int rows = kind == 0 ? p.S : p.capacity;
      uint16_t* out =
          p.y[kind] + ((static_cast<long long>(k.b) * H + at) * rows +
                       (kind == 0 ? k.s : k.row)) * D;
      if (kind == 2) {
        if (k.in) {
          *reinterpret_cast<uint2*>(out + lane.at[0]) = in[i][0];
          *reinterpret_cast<uint2*>(out + lane.at[1]) = in[i][1];
        }
      } else {
        float x[8], y[8];
        widen<kBF16>(in[i], x);
        if (p.w[kind] != nullptr) {
          float f;
          const float r = norm_factor<D>(x, p.eps, &f);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= r * (kind == 0 ? wq[e] : wk[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int a = first_of<kInterleaved>(e);
          const int b = second_of<kInterleaved>(e);
          y[a] = x[a];
          y[b] = x[b];
          if (lane.pair >= 0) {
            y[a] = x[a] * c[e] - x[b] * s[e];
            y[b] = x[a] * s[e] + x[b] * c[e];
          }
        }
        if (k.in) store8<kBF16>(out, lane.at, y);
      }
      if (k.in && h + i + kAhead < h1) load(h + i + kAhead, in[i]);
    }
  }
}

// --------------------------------------------------------------- backward
constexpr int kAheadBwd = 2;

template <int D, bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
    rope_bwd_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  const int group = threadIdx.x / kLanes;
  const Lane<D, kInterleaved> lane(threadIdx.x % kLanes, p.rot);
  start_after_previous();
  const int h0 = blockIdx.y * p.head_block;
  const int h1 = min(h0 + p.head_block, p.heads);
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  load_weights<kBF16>(p, 0, lane.at, wq);
  load_weights<kBF16>(p, 1, lane.at, wk);

  const int blocks = (p.tokens + kGroups - 1) / kGroups;
  for (int blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const Token k = find_token(p, blk * kGroups + group);
    auto load = [&](int h, uint2* dy, uint2* x) {
      int at;
      const int kind = head_kind(p, h, &at);
      const int H = kind == 0 ? p.Hq : p.Hkv;
      load8<kBF16>(
          p.y[kind] +
              ((static_cast<long long>(k.b) * H + at) * p.S + k.s) * D,
          lane.at, dy);
      if (kind < 2 && p.w[kind] != nullptr)
        load8<kBF16>(p.x[kind] + k.b * p.x_b[kind] + k.s * p.x_s[kind] +
                         at * p.x_h[kind],
                     lane.at, x);
    };
    uint2 gy[kAheadBwd][2], gx[kAheadBwd][2];
#pragma unroll
    for (int i = 0; i < kAheadBwd; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) gy[i][j] = gx[i][j] = make_uint2(0u, 0u);
      if (k.in && h0 + i < h1) load(h0 + i, gy[i], gx[i]);
    }
    float c[4], s[4];
    turns(p, k, lane.pair, c, s);
    for (int h = h0; h < h1; h += kAheadBwd) {
#pragma unroll
      for (int i = 0; i < kAheadBwd; ++i) {
        if (h + i >= h1) break;
        int at;
        const int kind = head_kind(p, h + i, &at);
        uint16_t* out = p.dx[kind] + k.b * p.dx_b[kind] +
                        k.s * p.dx_s[kind] + at * p.dx_h[kind];
        if (kind == 2) {
          if (k.in) {
            *reinterpret_cast<uint2*>(out + lane.at[0]) = gy[i][0];
            *reinterpret_cast<uint2*>(out + lane.at[1]) = gy[i][1];
          }
        } else {
          float dy[8], dn[8];
          widen<kBF16>(gy[i], dy);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = first_of<kInterleaved>(e);
            const int b = second_of<kInterleaved>(e);
            dn[a] = dy[a];
            dn[b] = dy[b];
            if (lane.pair >= 0) {
              dn[a] = dy[a] * c[e] + dy[b] * s[e];
              dn[b] = dy[b] * c[e] - dy[a] * s[e];
            }
          }
          if (p.w[kind] != nullptr) {
            float x[8];
            widen<kBF16>(gx[i], x);
            float f, dot = 0.f;
            const float r = norm_factor<D>(x, p.eps, &f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] *= r;  // x^
              const float add = dn[e] * x[e];
              if (kind == 0)
                dwq[e] += add;
              else
                dwk[e] += add;
              dn[e] *= kind == 0 ? wq[e] : wk[e];
              dot = fmaf(dn[e], x[e], dot);
            }
            dot = group_sum<kLanes>(dot) * (1.f / D);
#pragma unroll
            for (int e = 0; e < 8; ++e) dn[e] = r * f * (dn[e] - x[e] * dot);
          }
          if (k.in) store8<kBF16>(out, lane.at, dn);
        }
        if (k.in && h + i + kAheadBwd < h1)
          load(h + i + kAheadBwd, gy[i], gx[i]);
      }
    }
  }
  if (p.w[0] == nullptr && p.w[1] == nullptr) return;
  // The CTA's sums over its groups, in their order.
  __shared__ float sums[kGroups][D];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      sums[group][lane.at[e / 4] + e % 4] = kind == 0 ? dwq[e] : dwk[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) sum += sums[g][threadIdx.x];
      const int cta = blockIdx.y * gridDim.x + blockIdx.x;
      p.part[(2LL * cta + kind) * D + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// Sums of the CTAs' rows: 32 columns a CTA, a warp takes every 32nd row.
constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads)
    rope_dw_kernel(const float* part, float* dwq, float* dwk, int D,
                   int ctas) {
  __shared__ float sums[32][33];
  start_after_previous();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
  float sum = 0.f;
#pragma unroll 4
  for (int i = warp; i < ctas; i += 32) sum += part[2LL * i * D + col];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp != 0) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += sums[i][lane];
  float* out = col < D ? dwq : dwk;
  if (out != nullptr) out[col % D] = sum;
}

template <class Kernel, class... Args>
cudaError_t launch_grid(Kernel kernel, dim3 grid, cudaStream_t stream,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Heads that a group of lanes takes.
int pick_head_block(const RopeParams& p, int groups, int sms) {
  const long long blocks = (p.tokens + groups - 1) / groups;
  int block = p.heads;
  while (block > kAhead &&
         blocks * ((p.heads + block - 1) / block) < 8LL * sms)
    block = (block + 1) / 2;
  return std::max(block, (p.heads + kMaxHeadBlocks - 1) / kMaxHeadBlocks);
}

template <int D, bool kBF16, bool kInterleaved>
cudaError_t launch_fwd(RopeParams p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  p.head_block = pick_head_block(p, kGroups, sms);
  const dim3 grid((p.tokens + kGroups - 1) / kGroups,
                  (p.heads + p.head_block - 1) / p.head_block);
  return launch_grid(rope_kernel<D, kBF16, kInterleaved>, grid, stream, p);
}

template <int D, bool kBF16, bool kInterleaved>
cudaError_t launch_bwd(RopeParams p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  p.head_block = pick_head_block(p, kGroups, sms);
  const int ny = (p.heads + p.head_block - 1) / p.head_block;
  const int nx = std::min((p.tokens + kGroups - 1) / kGroups,
                     bwd_ctas(sms) / ny);
  cudaError_t err =
      launch_grid(rope_bwd_kernel<D, kBF16, kInterleaved>, dim3(nx, ny),
                  stream, p);
  if (err != cudaSuccess || (p.w[0] == nullptr && p.w[1] == nullptr))
    return err;
  return launch_pdl(rope_dw_kernel, 2 * D / 32, kSumThreads, 0, stream,
                    static_cast<const float*>(p.part), p.dw[0], p.dw[1], D,
                    nx * ny);
}

template <int D>
cudaError_t launch_d(bool bwd, bool bf16, bool interleaved,
                     const RopeParams& p, int sms, cudaStream_t stream) {
  if (bwd) {
    if (interleaved)
      return bf16 ? launch_bwd<D, true, true>(p, sms, stream)
                  : launch_bwd<D, false, true>(p, sms, stream);
    return bf16 ? launch_bwd<D, true, false>(p, sms, stream)
                : launch_bwd<D, false, false>(p, sms, stream);
  }
  if (interleaved)
    return bf16 ? launch_fwd<D, true, true>(p, sms, stream)
                : launch_fwd<D, false, true>(p, sms, stream);
  return bf16 ? launch_fwd<D, true, false>(p, sms, stream)
              : launch_fwd<D, false, false>(p, sms, stream);
}

}  // namespace

cudaError_t launch_rope(int D, bool bf16, bool interleaved,
                        const RopeParams& p, int sms, cudaStream_t stream) {
  return D == 64 ? launch_d<64>(false, bf16, interleaved, p, sms, stream)
                 : launch_d<128>(false, bf16, interleaved, p, sms, stream);
}
cudaError_t launch_rope_bwd(int D, bool bf16, bool interleaved,
                            const RopeParams& p, int sms,
                            cudaStream_t stream) {
  return D == 64 ? launch_d<64>(true, bf16, interleaved, p, sms, stream)
                 : launch_d<128>(true, bf16, interleaved, p, sms, stream);
}

}  // namespace rope
}  // namespace attn
