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
// nothing; the fraction of a turn, rounded to fp32, goes to sincospif.
//
// Layout: a group of D / 8 lanes holds one row, eight elements a lane, chosen
// so that both numbers of its four pairs are its own: two runs of four
// elements, rot / 2 apart (or eight neighbours).  No exchange but the sums of
// squares, and no angle is computed twice for a row; a group keeps its token's
// sines for a block of heads.  Everything between load and store is fp32; one
// rounding, to the output.
//
// What bounds it: the bytes, each read and written once.  The prompt's 168 MB
// take 28.9 us, 5.8 TB/s (a copy's rate would be 25.0); the video tokens' 100 MB
// 18.7, 5.3 TB/s (of the rest, three axes' positions and angles for no more than
// 8 heads of a token); one token of 8 sequences 3.1 us on the device, a launch.
// Registers limit what is in flight, hence a CTA's one kind of head, whose
// factors of norm and rotation are made once, and packed arithmetic.
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
// Times of: a prompt of 8192 tokens, 32 + 4 + 4 heads of 128, norms; 8102 video
// tokens, 16 + 16 + 16 heads of 64, norms, three axes; a training step's
// backward, 16384 tokens, 32 + 8 + 8 heads of 128, norms.
// Rows of a group, all in flight at once (28.9 and 18.6 us; 4: 31.9 and 21.5).
constexpr int kRows = 8;
// CTAs an SM holds, which caps a thread's registers (6, 7, 8 and 9: 31.1, 29.9,
// 28.9 and 30.7 us of heads of 128; 19.1, 18.7, 19.6 and 21.1 of 64).
constexpr int fwd_blocks(int D) { return D == 128 ? 8 : 7; }
// The backward's ring: rows of a group (2, 4 and 8: 106.2, 106.1 and 107.4 us).
constexpr int kStagesBwd = 4;
// Heads of a group (4, 8 and 16: 129, 106 and 127 us).
constexpr int kHeadsBwd = 8;
// CTAs an SM holds, and the launch has (4, 6 and 8: 113, 106 and 108 us).
constexpr int kBwdBlocks = 6;

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
    // Half turns in [-1, 1]: the upper half of the fraction, rounded, and what
    // that leaves, each rounded to fp32: off by 2^-23 of itself at most, also
    // where the angle is small.  (By one conversion of 64 bits a prompt took 0.2
    // us longer, the padded batch 3.98 for 3.77.)
    const int hi = static_cast<int>((turn + 0x80000000u) >> 32);
    const int lo = static_cast<int>(static_cast<unsigned>(turn));
    sincospif(fmaf(static_cast<float>(hi), 0x1p-31f,
                   static_cast<float>(lo) * 0x1p-63f),
              &s[e], &c[e]);
  }
}

// Two fp32 numbers and packed arithmetic on them.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r.v)
      : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 swapped(F2 a) {
  const float2 p = parts(a);
  return f2(p.y, p.x);
}
__device__ __forceinline__ F2 chosen(bool first, F2 a, F2 b) {
  F2 r;
  r.v = first ? a.v : b.v;
  return r;
}

// A lane's eight numbers of a row as they lie in memory, and as fp32.
struct Row {
  uint2 w[2];
};
__device__ __forceinline__ Row load_row(const uint16_t* row, const int* at) {
  Row r;
  r.w[0] = __ldg(reinterpret_cast<const uint2*>(row + at[0]));
  r.w[1] = __ldg(reinterpret_cast<const uint2*>(row + at[1]));
  return r;
}
template <bool kBF16>
__device__ __forceinline__ void widen(const Row& r, F2* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2<kBF16>(r.w[i].x), b = unpack2<kBF16>(r.w[i].y);
    x[2 * i] = f2(a.x, a.y);
    x[2 * i + 1] = f2(b.x, b.y);
  }
}
template <bool kBF16>
__device__ __forceinline__ void store_row(uint16_t* row, const int* at,
                                          const F2* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = parts(x[2 * i]), b = parts(x[2 * i + 1]);
    *reinterpret_cast<uint2*>(row + at[i]) = make_uint2(
        ptx::pack2<kBF16>(a.x, a.y), ptx::pack2<kBF16>(b.x, b.y));
  }
}

// The lane's norm weights (1 without).
template <bool kBF16>
__device__ __forceinline__ void load_weights(const RopeParams& p, int kind,
                                             const int* at, float* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
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

// The rotation of a lane's numbers n = x w by angles t as products with
// factors made once: of pair (a, b) the turned ones are
//   a w_a cos t - b w_b sin t,  b w_b cos t + a w_a sin t.
// Packed, own[i] multiplies x[i] and other[i] the numbers that x[i]'s partners
// are: x[i ^ 2], or neighbours with each other.
struct Turn {
  F2 own[4], other[4];
};
// sign: -1 turns back.
template <bool kInterleaved>
__device__ __forceinline__ Turn make_turn(const float* w, const float* c,
                                          const float* s, float sign) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInterleaved) {
      const float u = sign * s[i];
      t.own[i] = f2(w[2 * i] * c[i], w[2 * i + 1] * c[i]);
      t.other[i] = f2(-w[2 * i + 1] * u, w[2 * i] * u);
    } else {
      const int e = 2 * (i % 2);  // first of its two pairs
      const float u = i < 2 ? -sign : sign;
      const float* v = i < 2 ? w + 4 : w;
      t.own[i] = f2(w[2 * i] * c[e], w[2 * i + 1] * c[e + 1]);
      t.other[i] = f2(u * v[e] * s[e], u * v[e + 1] * s[e + 1]);
    }
  }
  return t;
}
// whole: every lane's numbers are rotated; turns: this lane's are.
template <bool kInterleaved>
__device__ __forceinline__ void rotate(const Turn& t, const F2* x, F2* y,
                                       bool whole, bool turns) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 o = mul(x[i], t.own[i]);
    y[i] = fma(kInterleaved ? swapped(x[i]) : x[i ^ 2], t.other[i], o);
    // (Not x + 0 * partner: an infinity would make that NaN.)
    if (!whole) y[i] = chosen(turns, y[i], o);
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
__device__ __forceinline__ float norm_factor(F2* x, float eps, float* f) {
  auto squares = [&] {
    F2 ss = mul(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) ss = fma(x[i], x[i], ss);
    const float2 p = parts(ss);
    return group_sum<D / 8>(p.x + p.y);
  };
  *f = 1.f;
  float ss = squares();
  if (__any_sync(kFull, ss == INFINITY)) {
    const bool big = ss == INFINITY;
    if (big) *f = 0x1p-96f;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul(x[i], f2(*f, *f));
    const float again = squares();
    if (big) {
      ss = again;
      eps = 0.f;
    }
  }
  return rsqrtf(fmaf(ss, 1.f / D, eps));
}

// A block's heads: `count` of kind `kind` (0 Q, 1 K, 2 V) from `first` on.
struct Heads {
  int kind, first, count;
};
__device__ __forceinline__ Heads find_heads(const RopeParams& p, int y) {
  Heads h;
  h.kind = y < p.q_blocks ? 0 : y < p.q_blocks + p.kv_blocks ? 1 : 2;
  if (h.kind > 0) y -= p.q_blocks + (h.kind - 1) * p.kv_blocks;
  h.first = y * p.head_block;
  h.count = min(p.head_block, (h.kind == 0 ? p.Hq : p.Hkv) - h.first);
  return h;
}

// ---------------------------------------------------------------- forward
template <int D, bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, fwd_blocks(D))
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  const Lane<D, kInterleaved> lane(threadIdx.x % kLanes, p.rot);
  const int block = fast_div(blockIdx.x, p.fd_blocks);
  const Heads h = find_heads(p, blockIdx.x - block * p.blocks);
  start_after_previous();
  const Token k = find_token(p, block * kGroups + threadIdx.x / kLanes);
  const uint16_t* x = p.x[h.kind] + k.b * p.x_b[h.kind] +
                      k.s * p.x_s[h.kind] + h.first * p.x_h[h.kind];
  // Every row of the group at once.
  Row in[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    in[i].w[0] = in[i].w[1] = make_uint2(0u, 0u);
    if (k.in && i < h.count) in[i] = load_row(x + i * p.x_h[h.kind], lane.at);
  }
  const int rows = h.kind == 0 ? p.S : p.capacity;
  uint16_t* out =
      p.y[h.kind] +
      ((static_cast<long long>(k.b) * (h.kind == 0 ? p.Hq : p.Hkv) + h.first) *
           rows + (h.kind == 0 ? k.s : k.row)) * D;
  const long long step = static_cast<long long>(rows) * D;
  if (h.kind == 2) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (!k.in || i >= h.count) break;
      *reinterpret_cast<uint2*>(out + i * step + lane.at[0]) = in[i].w[0];
      *reinterpret_cast<uint2*>(out + i * step + lane.at[1]) = in[i].w[1];
    }
    return;
  }
  Turn turn;
  {
    float w[8], c[4], s[4];
    load_weights<kBF16>(p, h.kind, lane.at, w);
    turns(p, k, lane.pair, c, s);
    turn = make_turn<kInterleaved>(w, c, s, 1.f);
  }
  const bool norm = p.w[h.kind] != nullptr, whole = p.rot == D;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i >= h.count) break;
    F2 n[4], y[4];
    widen<kBF16>(in[i], n);
    if (norm) {
      float f;
      const float r = norm_factor<D>(n, p.eps, &f);
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = mul(n[e], f2(r, r));
    }
    rotate<kInterleaved>(turn, n, y, whole, lane.pair >= 0);
    if (k.in) store_row<kBF16>(out + i * step, lane.at, y);
  }
}

// --------------------------------------------------------------- backward
// Reads two rows and writes one, with twice the forward's arithmetic between: a
// training step's 570 MB take 107 us, 5.3 TB/s (a copy's rate would be 85).  Rows
// run ahead through shared memory, as registers have no room for them beside the
// weights' sums (121 us with loads just ahead of their use, 127 with the next
// row's in registers).  Each CTA keeps to a block of heads and walks over tokens,
// so that the weights' sums stay in registers; they meet as fp32 in a fixed
// order: results do not change from run to run.

__device__ __forceinline__ Row shared_row(uint32_t row, const int* at) {
  Row r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.w[i].x), "=r"(r.w[i].y)
                 : "r"(row + 2 * at[i])
                 : "memory");
  return r;
}

template <int D, bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBwdBlocks)
    rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  const int group = threadIdx.x / kLanes;
  const Lane<D, kInterleaved> lane(threadIdx.x % kLanes, p.rot);
  const int stripe = fast_div(blockIdx.x, p.fd_blocks);
  const int stripes = gridDim.x / p.blocks;
  const int y_block = blockIdx.x - stripe * p.blocks;
  const Heads h = find_heads(p, y_block);
  start_after_previous();
  const bool norm = h.kind < 2 && p.w[h.kind] != nullptr;
  const bool whole = p.rot == D;
  float w[8];
  F2 dw[4];
  if (h.kind < 2) load_weights<kBF16>(p, h.kind, lane.at, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[e] = f2(0.f, 0.f);

  // A warp's rows, one of each group at a time: token blocks of the stripe, and
  // the heads of each.  They run ahead through a ring in shared memory.
  __shared__ __align__(16) uint8_t ring[kThreads / 32][kStagesBwd][1024];
  const int token_blocks = (p.tokens + kGroups - 1) / kGroups;
  const long long step = static_cast<long long>(p.S) * D;
  const int in_warp = threadIdx.x % 32 / kLanes, l = threadIdx.x % kLanes;
  const uint32_t slots = ptx::smem_u32(ring[threadIdx.x / 32]);
  constexpr uint32_t kRowBytes = 2 * D;  // of an input; a slot: [group][dy, x]
  const uint32_t mine = slots + in_warp * 2 * kRowBytes;
  struct {
    int blk, i;
    bool in;
    const uint16_t *dy, *x;
  } ahead{};
  auto enter = [&] {
    const Token k = find_token(p, ahead.blk * kGroups + group);
    ahead.in = k.in;
    ahead.dy = p.y[h.kind] +
               ((static_cast<long long>(k.b) * (h.kind == 0 ? p.Hq : p.Hkv) +
                 h.first) * p.S + k.s) * D + 8 * l;
    if (norm)
      ahead.x = p.x[h.kind] + k.b * p.x_b[h.kind] + k.s * p.x_s[h.kind] +
                h.first * p.x_h[h.kind] + 8 * l;
  };
  auto load = [&](int stage) {
    if (ahead.blk < token_blocks) {
      const uint32_t to = mine + stage * 1024 + 16 * l;
      ptx::cp_async16_or_zero(to, ahead.dy, ahead.in);
      if (norm) ptx::cp_async16_or_zero(to + kRowBytes, ahead.x, ahead.in);
      ahead.dy += step;
      if (norm) ahead.x += p.x_h[h.kind];
      if (++ahead.i == h.count) {
        ahead.i = 0;
        ahead.blk += stripes;
        if (ahead.blk < token_blocks) enter();
      }
    }
    ptx::cp_async_commit();
  };
  ahead.blk = stripe;
  ahead.i = 0;
  enter();
#pragma unroll
  for (int i = 0; i < kStagesBwd; ++i) load(i);
  int stage = 0;
  for (int blk = stripe; blk < token_blocks; blk += stripes) {
    const Token k = find_token(p, blk * kGroups + group);
    uint16_t* dx = p.dx[h.kind] + k.b * p.dx_b[h.kind] +
                   k.s * p.dx_s[h.kind] + h.first * p.dx_h[h.kind];
    Turn back;
    if (h.kind < 2) {
      float one[8], c[4], s[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) one[e] = 1.f;
      turns(p, k, lane.pair, c, s);
      back = make_turn<kInterleaved>(one, c, s, -1.f);
    }
    for (int i = 0; i < h.count; ++i, dx += p.dx_h[h.kind]) {
      ptx::cp_async_wait<kStagesBwd - 1>();
      __syncwarp();
      Row gy, gx;
      const uint32_t from = mine + stage * 1024;
      gy = shared_row(from, lane.at);
      if (norm) gx = shared_row(from + kRowBytes, lane.at);
      __syncwarp();  // the slot has been read
      load(stage);
      stage = stage + 1 == kStagesBwd ? 0 : stage + 1;
      if (h.kind == 2) {
        if (k.in) {
          *reinterpret_cast<uint2*>(dx + lane.at[0]) = gy.w[0];
          *reinterpret_cast<uint2*>(dx + lane.at[1]) = gy.w[1];
        }
        continue;
      }
      F2 d[4], g[4];
      widen<kBF16>(gy, d);
      rotate<kInterleaved>(back, d, g, whole, lane.pair >= 0);
      if (norm) {
        F2 n[4];
        widen<kBF16>(gx, n);
        float f;
        const float r = norm_factor<D>(n, p.eps, &f);
        F2 sum = f2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          n[e] = mul(n[e], f2(r, r));  // x^
          dw[e] = fma(g[e], n[e], dw[e]);
          g[e] = mul(g[e], f2(w[2 * e], w[2 * e + 1]));
          sum = fma(g[e], n[e], sum);
        }
        const float2 both = parts(sum);
        const float mean = group_sum<kLanes>(both.x + both.y) * (-1.f / D);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          g[e] = mul(fma(n[e], f2(mean, mean), g[e]), f2(r * f, r * f));
      }
      if (k.in) store_row<kBF16>(dx, lane.at, g);
    }
  }
  if (!norm) return;
  // The CTA's sums over its groups, in their order.
  __shared__ float sums[kGroups][D];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = parts(dw[e]);
    float* at = &sums[group][lane.at[e / 2] + 2 * (e % 2)];
    at[0] = v.x;
    at[1] = v.y;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sum += sums[g][i];
    p.part[(static_cast<long long>(y_block) * stripes + stripe) * D + i] = sum;
  }
}

// Sums of the CTAs' rows: 32 columns a CTA, a warp takes every 32nd row.
constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads)
    rope_dw_kernel(const float* part, float* dwq, float* dwk, int D,
                   int q_ctas, int kv_ctas) {
  __shared__ float sums[32][33];
  start_after_previous();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int kind = blockIdx.x / (D / 32);
  const int col = blockIdx.x % (D / 32) * 32 + lane;
  float* out = kind == 0 ? dwq : dwk;
  if (out == nullptr) return;
  const int first = kind == 0 ? 0 : q_ctas;
  const int count = kind == 0 ? q_ctas : kv_ctas;
  float sum = 0.f;
#pragma unroll 8
  for (int i = warp; i < count; i += 32)
    sum += part[static_cast<long long>(first + i) * D + col];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp != 0) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += sums[i][lane];
  out[col] = sum;
}

// Cuts the heads into blocks of head_block.
void cut_heads(RopeParams* p, int head_block) {
  const bool values = p->heads > p->Hq + p->Hkv;
  p->head_block = head_block;
  p->q_blocks = (p->Hq + head_block - 1) / head_block;
  p->kv_blocks = (p->Hkv + head_block - 1) / head_block;
  p->blocks = p->q_blocks + p->kv_blocks * (values ? 2 : 1);
  p->fd_blocks = make_fast_div(p->blocks);
}

template <int D, bool kBF16, bool kInterleaved>
cudaError_t launch_fwd(RopeParams p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const long long token_blocks = (p.tokens + kGroups - 1LL) / kGroups;
  // Fewer heads a group where these would not fill the machine (8 tokens of 48
  // heads: 3.1 us, by 8 heads 4.5).
  int head_block = kRows;
  cut_heads(&p, head_block);
  while (head_block > 1 && token_blocks * p.blocks < 2LL * sms)
    cut_heads(&p, head_block /= 2);
  return launch_pdl(rope_kernel<D, kBF16, kInterleaved>,
                    token_blocks * p.blocks, kThreads, 0, stream, p);
}

template <int D, bool kBF16, bool kInterleaved>
cudaError_t launch_bwd(RopeParams p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const int token_blocks = (p.tokens + kGroups - 1) / kGroups;
  int head_block = kHeadsBwd;
  cut_heads(&p, head_block);
  while (head_block > 1 &&
         static_cast<long long>(token_blocks) * p.blocks < 2LL * sms)
    cut_heads(&p, head_block /= 2);
  // (Each CTA of Q and K leaves a row of sums.)
  while (p.blocks > bwd_ctas(sms)) cut_heads(&p, head_block *= 2);
  const int stripes = std::min(token_blocks, bwd_ctas(sms) / p.blocks);
  cudaError_t err =
      launch_pdl(rope_bwd_kernel<D, kBF16, kInterleaved>,
                 static_cast<long long>(stripes) * p.blocks, kThreads, 0,
                 stream, p);
  if (err != cudaSuccess || (p.w[0] == nullptr && p.w[1] == nullptr))
    return err;
  return launch_pdl(rope_dw_kernel, 2 * D / 32, kSumThreads, 0, stream,
                    static_cast<const float*>(p.part), p.dw[0], p.dw[1], D,
                    p.q_blocks * stripes, p.kv_blocks * stripes);
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
