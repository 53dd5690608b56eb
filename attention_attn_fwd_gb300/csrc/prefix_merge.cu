// Joins the parts of a query row's attention behind a shared prefix.  With part
// s the average O_s and the log-sum-exp L_s of its keys (in log2 units),
//   O = sum_s 2^(L_s - m) O_s / sum_s 2^(L_s - m),  LSE = m + log2(the sum).
// All in fp32; one rounding, to the output.
//
// What bounds it: a chain of loads (lengths, where the parts are, their L,
// their O), some 4 us, each as far as a cold cache; so the O are asked for
// before their factors are known, and rows are spread over warps where they are
// few. Where they are many, warps take four at once: 32768 rows of 128, two
// parts each, in 18 us (a row a warp 31).
//
// A part's weight 2^(L_s - m) is held times kSlack: the weights of all parts of
// a row then sum to 1 at most, and their products with O_s stay within fp32 where
// V (and so each O_s) comes near its largest number.  A power of two, so that
// nothing is rounded by it and the results' bits are those without it.
#include "prefix_common.cuh"

namespace attn {
namespace prefix {
namespace {

using kv8::kNone;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kAhead = 8;  // parts whose O a warp has in flight
// 1 / (more parts than a row has: one per CTA over the prefix, and over the own
// keys one per CTA or, of few rows, per warp of the CTAs set aside for them;
// 1369 of 152 CTAs).
constexpr float kSlack = 0x1p-11f;
static_assert((1 + kFewWarps) * 224 < 2048, "parts of a row (SMs: 224)");
// Rows an SM from which on warps take four (2520 rows in all, 35 a head: 24 us
// of the whole call, 27 by four).
constexpr long long kManyRows = 32;

// What a warp has of a row: the sum over its parts, relative to 2^mx.
struct Sum {
  float mx, sum;
  float4 acc;
};

__device__ __forceinline__ void add(float4& acc, const float4& y, float f) {
  if (f == 0.f) return;  // a part that sees nothing has no O
  acc.x += y.x * f;
  acc.y += y.y * f;
  acc.z += y.z * f;
  acc.w += y.w * f;
}

// Parts [s0, s1) by one warp, where at(s, &o, &lse2) gives the places of part
// s's O and LSE.  (O is on its way before its factor is known.)
template <int D, class At>
__device__ __forceinline__ Sum add_parts(int s0, int s1, int lane, At at) {
  constexpr int kCols = D / 4;          // float4 columns
  constexpr int kGroups = 32 / kCols;   // parts a warp reads at a time
  constexpr int kBatch = kAhead * kGroups;
  const int col = lane % kCols, sub = lane / kCols;
  Sum t{kNone, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (; s0 < s1; s0 += 32) {
    const int count = min(32, s1 - s0);
    const float4* o = nullptr;
    float x = -INFINITY;
    if (lane < count) {
      const float* lse2;
      at(s0 + lane, &o, &lse2);
      x = *lse2;
    }
    const unsigned long long place = reinterpret_cast<unsigned long long>(o);
    float f_all = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      float4 y[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = k0 + i * kGroups + sub;
        const float4* from = reinterpret_cast<const float4*>(
            __shfl_sync(0xffffffffu, place, k % 32));
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < count) y[i] = from[col];
      }
      if (k0 == 0) {
        float m = fmaxf(t.mx, x);
#pragma unroll
        for (int k = 16; k > 0; k /= 2)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        const float before = ptx::ex2(t.mx - m);
        f_all = ptx::ex2(x - m) * kSlack;
        t.mx = m;
        t.acc.x *= before;
        t.acc.y *= before;
        t.acc.z *= before;
        t.acc.w *= before;
        t.sum = t.sum * before + f_all;  // (a lane's share)
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = k0 + i * kGroups + sub;
        const float f = __shfl_sync(0xffffffffu, f_all, k % 32);
        if (k < count) add(t.acc, y[i], f);
      }
    }
  }
  // (The lanes' shares were scaled alike.)
#pragma unroll
  for (int k = 16; k > 0; k /= 2)
    t.sum += __shfl_xor_sync(0xffffffffu, t.sum, k);
  if constexpr (kGroups == 2) {
    t.acc.x += __shfl_xor_sync(0xffffffffu, t.acc.x, 16);
    t.acc.y += __shfl_xor_sync(0xffffffffu, t.acc.y, 16);
    t.acc.z += __shfl_xor_sync(0xffffffffu, t.acc.z, 16);
    t.acc.w += __shfl_xor_sync(0xffffffffu, t.acc.w, 16);
  }
  return t;
}

template <int D, bool kBF16>
__device__ __forceinline__ void write_row(const PrefixParams& p, long long row,
                                          const Sum& t, int lane) {
  const float inv = t.sum == 0.f ? 0.f : 1.f / t.sum;
  if (lane < D / 4) {
    uint2 out;
    out.x = ptx::pack2<kBF16>(t.acc.x * inv, t.acc.y * inv);
    out.y = ptx::pack2<kBF16>(t.acc.z * inv, t.acc.w * inv);
    reinterpret_cast<uint2*>(p.o + row * D)[lane] = out;
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = t.sum == 0.f ? -INFINITY
                              : (t.mx + log2f(t.sum * (1.f / kSlack))) *
                                    0.69314718055994531f;
}

// First part and number of parts within `n` slots: a kernel ahead whose wait
// ran out may not have written them.
__device__ __forceinline__ int2 within(int2 x, int n) {
  x.y = min(max(x.y, 0), n);
  x.x = min(max(x.x, 0), n - x.y);
  return x;
}

// What the rows of a K/V head of a sequence have in common (kFew, kPacked):
// the CTAs (or warps) and numbers of their parts over the prefix and over the
// own keys.
struct Parts {
  int2 pre, own;
  long long base, bh;
  int in_unit;

  __device__ __forceinline__ Parts(const PrefixParams& p, int bh_, int b,
                                   int h, int np, int len, int n_new) {
    bh = bh_;
    const int tile = fast_div(b, p.fd_tile_seqs);
    in_unit = tile % 2 * kTM + (b - tile * p.tile_seqs) * p.rows;
    base = (static_cast<long long>(h) * p.B + b) * p.rows;
    pre = own = make_int2(0, 0);
    if (np > 0)
      pre = within(p.info[static_cast<long long>(tile / 2) * p.Hkv + h],
                   p.grid);
    if (p.mode == kFew) {
      if (len > 0) own = p.own_info[bh];
    } else if (tiles_seen(p, len, n_new, 0, p.rows) > 0) {
      own = within(
          p.info[(static_cast<long long>(p.pack_blocks) + b) * p.Hkv + h],
          p.grid);
    }
  }
  // Row r's part s: those over the prefix first.
  __device__ __forceinline__ void at(const PrefixParams& p, int s, int r,
                                     int cols, const float4** o,
                                     const float** lse2) const {
    const float *from = p.base_o, *from2 = p.base_lse2;
    long long i;
    if (s == 0 && pre.y > 0) {
      i = base + r;
    } else if (s < pre.y) {
      from = p.slot_o;
      from2 = p.slot_lse2;
      i = static_cast<long long>(pre.x + s) * kUnitRows + in_unit + r;
    } else if (p.mode == kFew) {
      from = p.few_o;
      from2 = p.few_lse2;
      i = (static_cast<long long>(own.x + s - pre.y) + bh) *
              few_rows(p.rows) + r;
    } else if (s == pre.y) {
      i = (static_cast<long long>(p.Hkv) * p.B + bh) * p.rows + r;
    } else {
      from = p.slot_o;
      from2 = p.slot_lse2;
      i = static_cast<long long>(own.x + s - pre.y) * kUnitRows + r;
    }
    *o = reinterpret_cast<const float4*>(from) + i * cols;
    *lse2 = from2 + i;
  }
};

// kFew and kPacked, where rows are few: each by row_warps warps.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 4)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p,
                        int row_warps) {
  __shared__ float2 sm_sum[kWarps];
  __shared__ float4 sm_acc[kWarps][D / 4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long id =
      (static_cast<long long>(blockIdx.x) * kWarps + warp) / row_warps;
  // (b, h, r), r fastest.
  const bool in = id < static_cast<long long>(p.B) * p.rows * p.Hkv;
  const int bh =
      !in ? 0
      : id < 0x7fffffff ? fast_div(static_cast<int>(id), p.fd_rows)
                        : static_cast<int>(id / p.rows);
  const int r =
      in ? static_cast<int>(id - static_cast<long long>(bh) * p.rows) : 0;
  const int b = fast_div(bh, p.fd_hkv), h = bh - b * p.Hkv;
  const int len = kv8::seq_len(p, b), n_new = kv8::seq_new(p, b);
  const int np = prefix_tiles(p);
  // (Lengths are read ahead of the wait: the kernels ahead do not write them.)
  kv8::start_after_previous();
  const bool live = in && r < n_new * p.group;
  Sum t{kNone, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  const int w = warp % row_warps;
  if (live) {
    const Parts parts(p, bh, b, h, np, len, n_new);
    const int n = parts.pre.y + parts.own.y;
    t = add_parts<D>(n * w / row_warps, n * (w + 1) / row_warps, lane,
                     [&](int s, const float4** o, const float** lse2) {
                       parts.at(p, s, r, D / 4, o, lse2);
                     });
  }
  if (row_warps > 1) {
    if (lane == 0) sm_sum[warp] = make_float2(t.mx, t.sum);
    if (lane < D / 4) sm_acc[warp][lane] = t.acc;
    __syncthreads();
    if (w != 0) return;
    float mx = t.mx;
    for (int i = 1; i < row_warps; ++i) mx = fmaxf(mx, sm_sum[warp + i].x);
    Sum all_of{mx, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int i = 0; i < row_warps; ++i) {
      const float f = ptx::ex2(sm_sum[warp + i].x - mx);
      const float4 y = sm_acc[warp + i][lane % (D / 4)];
      all_of.sum += sm_sum[warp + i].y * f;
      all_of.acc.x += y.x * f;
      all_of.acc.y += y.y * f;
      all_of.acc.z += y.z * f;
      all_of.acc.w += y.w * f;
    }
    t = all_of;
  }
  if (live) write_row<D, kBF16>(p, q_row_index(p, b, h, r), t, lane);
}

// `n` rows, kJoinRows at most, of `parts` parts each by one warp, all rows at
// once: at(s, i, &o, &lse2) as above for row i, row_at(i) its row of O.
constexpr int kJoinRows = 4;
constexpr int kJoinParts = 32 / kJoinRows;  // whose LSEs a warp reads at once

template <int D, bool kBF16, class At, class RowAt>
__device__ __forceinline__ void join_rows(const PrefixParams& p, int n,
                                          int parts, int lane, At at,
                                          RowAt row_at) {
  constexpr int kCols = D / 4;
  constexpr int kGroups = 32 / kCols;  // rows a warp reads at a time
  constexpr int kLoads = kJoinRows / kGroups;
  constexpr int kBatch = kAhead / kLoads;  // parts in flight
  const int col = lane % kCols, sub = lane / kCols;
  const int i_lane = lane / kJoinParts, s_lane = lane % kJoinParts;
  float mx = kNone, sum = 0.f;  // of the lane's row, its share of the sum
  float4 acc[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 0; s0 < parts; s0 += kJoinParts) {
    const int count = min(kJoinParts, parts - s0);
    const float4* o = nullptr;
    float x = -INFINITY, f_all = 0.f;
    if (s_lane < count && i_lane < n) {
      const float* lse2;
      at(s0 + s_lane, i_lane, &o, &lse2);
      x = *lse2;
    }
    const unsigned long long place = reinterpret_cast<unsigned long long>(o);
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      float4 y[kBatch][kLoads];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const float4* from = reinterpret_cast<const float4*>(__shfl_sync(
              0xffffffffu, place,
              (j * kGroups + sub) * kJoinParts + (k0 + k) % kJoinParts));
          y[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < count && from != nullptr) y[k][j] = from[col];
        }
      if (k0 == 0) {
        float m = fmaxf(mx, x);
#pragma unroll
        for (int k = kJoinParts / 2; k > 0; k /= 2)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        const float before = ptx::ex2(mx - m);
        f_all = ptx::ex2(x - m) * kSlack;
        mx = m;
        sum = sum * before + f_all;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const float f = __shfl_sync(0xffffffffu, before,
                                      (j * kGroups + sub) * kJoinParts);
          acc[j].x *= f;
          acc[j].y *= f;
          acc[j].z *= f;
          acc[j].w *= f;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const float f = __shfl_sync(
              0xffffffffu, f_all,
              (j * kGroups + sub) * kJoinParts + (k0 + k) % kJoinParts);
          if (k0 + k < count) add(acc[j], y[k][j], f);
        }
    }
  }
#pragma unroll
  for (int k = kJoinParts / 2; k > 0; k /= 2)
    sum += __shfl_xor_sync(0xffffffffu, sum, k);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int i = j * kGroups + sub;
    const float f = __shfl_sync(0xffffffffu, inv, i * kJoinParts);
    if (i >= n) continue;
    uint2 out;
    out.x = ptx::pack2<kBF16>(acc[j].x * f, acc[j].y * f);
    out.y = ptx::pack2<kBF16>(acc[j].z * f, acc[j].w * f);
    reinterpret_cast<uint2*>(p.o + row_at(i) * D)[col] = out;
  }
  if (s_lane == 0 && i_lane < n && p.lse != nullptr)
    p.lse[row_at(i_lane)] =
        sum == 0.f ? -INFINITY
                   : (mx + log2f(sum * (1.f / kSlack))) *
                         0.69314718055994531f;
}

// kFew and kPacked, where rows are many: four of a (sequence, K/V head) by a
// warp.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kJoinThreads, 8)
    prefix_rows_kernel(const __grid_constant__ PrefixParams p, int chunks,
                       FastDiv fd_chunks) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int id = blockIdx.x * kJoinWarps + warp;
  const bool in = id < chunks;
  const int bh = in ? fast_div(id, fd_chunks) : 0;
  const int b = fast_div(bh, p.fd_hkv), h = bh - b * p.Hkv;
  const int len = kv8::seq_len(p, b), n_new = kv8::seq_new(p, b);
  const int np = prefix_tiles(p);
  kv8::start_after_previous();
  if (!in) return;
  const int r0 =
      (id - bh * ((p.rows + kJoinRows - 1) / kJoinRows)) * kJoinRows;
  const int n = min(kJoinRows, n_new * p.group - r0);
  if (n <= 0) return;
  const Parts parts(p, bh, b, h, np, len, n_new);
  join_rows<D, kBF16>(
      p, n, parts.pre.y + parts.own.y, lane,
      [&](int s, int i, const float4** o, const float** lse2) {
        parts.at(p, s, r0 + i, D / 4, o, lse2);
      },
      [&](int i) { return q_row_index(p, b, h, r0 + i); });
}

// kJoint: the rows of each CTA's unit that went on behind it.
constexpr int kParts = kUnitRows / kJoinWarps / kJoinRows;  // CTAs per unit

template <int D, bool kBF16>
__global__ void __launch_bounds__(kJoinThreads, 8)
    prefix_join_kernel(const __grid_constant__ PrefixParams p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x / kParts;
  const int i0 =
      ((blockIdx.x - cta * kParts) * kJoinWarps + warp) * kJoinRows;
  kv8::start_after_previous();
  const int4 split = p.split[cta];
  const int b = split.x, h = split.y, parts = split.w;
  if (parts == 0) return;
  const int rows = kv8::seq_new(p, b) * p.group;
  const int tile = i0 / kTM, in_tile = i0 % kTM;
  const int r0 = (2 * split.z + tile) * p.tile_rows + in_tile;
  const int n = min(kJoinRows, min(p.tile_rows - in_tile, rows - r0));
  if (n <= 0) return;
  join_rows<D, kBF16>(
      p, n, parts, lane,
      [&](int s, int i, const float4** o, const float** lse2) {
        const long long j =
            static_cast<long long>(s == 0 ? p.grid + cta : cta + s) *
                kUnitRows + i0 + i;
        *o = reinterpret_cast<const float4*>(p.slot_o) + j * (D / 4);
        *lse2 = p.slot_lse2 + j;
      },
      [&](int i) { return q_row_index(p, b, h, r0 + i); });
}

template <int D, bool kBF16>
cudaError_t launch(PrefixParams p, cudaStream_t stream) {
  if (p.mode == kJoint)
    return kv8::launch_pdl(prefix_join_kernel<D, kBF16>,
                           static_cast<long long>(p.grid) * kParts,
                           kJoinThreads, 0, stream, p);
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  const long long rows = heads * p.rows;
  const int per_head = (p.rows + kJoinRows - 1) / kJoinRows;
  if (p.rows >= kJoinRows && rows > kManyRows * p.grid)
    return kv8::launch_pdl(prefix_rows_kernel<D, kBF16>,
                           (heads * per_head + kJoinWarps - 1) / kJoinWarps,
                           kJoinThreads, 0, stream, p,
                           static_cast<int>(heads * per_head),
                           make_fast_div(per_head));
  // Warps a row: as many as make the machine's warps busy, rows having some 20
  // parts where they are few (8 sequences behind 4096 tokens: 18.2 us of the
  // whole call, 20.6 by a warp a row; 32 behind 65531: 52 and 57).
  int row_warps = kWarps;
  while (row_warps > 1 && rows * row_warps > 32LL * p.grid)
    row_warps /= 2;
  return kv8::launch_pdl(prefix_merge_kernel<D, kBF16>,
                         (rows * row_warps + kWarps - 1) / kWarps, kThreads, 0,
                         stream, p, row_warps);
}

}  // namespace

cudaError_t launch_merge(int D, bool bf16, const PrefixParams& p,
                         cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return bf16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace prefix
}  // namespace attn
