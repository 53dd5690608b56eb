// Joins the parts of a query row's attention behind a shared prefix.  With part s the average O_s and the log-sum-exp L_s of its keys,
//   O = sum_s 2^(L_s - m) O_s / sum_s 2^(L_s - m),  LSE = m + log2(the sum).
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
        f_all = ptx::ex2(x - m);
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
                              : (t.mx + log2f(t.sum)) * 0.69314718055994531f;
}

// kFew and kPacked: every row, with the parts over the prefix first, by
// row_warps warps.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 4)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p,
                        int row_warps) {
  __shared__ float2 sm_sum[kWarps];
  __shared__ float4 sm_acc[kWarps][D / 4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long id =
      (static_cast<long long>(blockIdx.x) * kWarps + warp) / row_warps;
  const int R = p.rows;
  const long long all = static_cast<long long>(p.B) * R;  // rows of a head
  const bool in = id < all * p.Hkv;
  // (b, h, r), r fastest.
  const int bh =
      !in ? 0
      : id < 0x7fffffff ? fast_div(static_cast<int>(id), p.fd_rows)
                        : static_cast<int>(id / R);
  const int r = in ? static_cast<int>(id - static_cast<long long>(bh) * R) : 0;
  const int b = fast_div(bh, p.fd_hkv), h = bh - b * p.Hkv;
  const int len = kv8::seq_len(p, b), n_new = kv8::seq_new(p, b);
  const int np = prefix_tiles(p);
  // Its Q tiles over the prefix and over the own keys, and places in their
  // units.
  const int tile = fast_div(b, p.fd_tile_seqs);
  const int in_unit = tile % 2 * kTM + (b - tile * p.tile_seqs) * R + r;
  const int own_tile = fast_div(r, p.fd_tile_rows);
  const int own_in_unit =
      own_tile % 2 * kTM + r - own_tile * p.tile_rows;
  const int u = own_tile / 2, r0 = u * 2 * p.tile_rows;
  // (Lengths are read ahead of the wait: the kernels ahead do not write them.)
  kv8::start_after_previous();
  const bool live = in && r < n_new * p.group;
  int2 pre = make_int2(0, 0), own = make_int2(0, 0);
  if (live) {
    if (np > 0)
      pre = p.info[static_cast<long long>(tile / 2) * p.Hkv + h];
    if (p.mode == kFew) {
      if (len > 0) own = p.own_info[bh];
    } else if (tiles_seen(p, len, n_new, r0, r0 + 2 * p.tile_rows) > 0) {
      own = p.info[(static_cast<long long>(p.pack_blocks) +
                    static_cast<long long>(b) * p.row_blocks + u) * p.Hkv + h];
    }
  }
  auto at = [&](int s, const float4** o, const float** lse2) {
    const float *from = p.base_o, *from2 = p.base_lse2;
    long long i;
    if (s == 0 && pre.y > 0) {
      i = h * all + static_cast<long long>(b) * R + r;
    } else if (s < pre.y) {
      from = p.slot_o;
      from2 = p.slot_lse2;
      i = static_cast<long long>(pre.x + s) * kUnitRows + in_unit;
    } else if (p.mode == kFew) {
      from = p.few_o;
      from2 = p.few_lse2;
      i = (static_cast<long long>(own.x + s - pre.y) + bh) * few_rows(R) + r;
    } else if (s == pre.y) {
      i = p.Hkv * all + static_cast<long long>(bh) * R + r;
    } else {
      from = p.slot_o;
      from2 = p.slot_lse2;
      i = static_cast<long long>(own.x + s - pre.y) * kUnitRows +
          own_in_unit;
    }
    *o = reinterpret_cast<const float4*>(from) + i * (D / 4);
    *lse2 = from2 + i;
  };
  const int n = pre.y + own.y, w = warp % row_warps;
  Sum t = add_parts<D>(n * w / row_warps, n * (w + 1) / row_warps, lane, at);
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

// kJoint: the rows of each CTA's unit that went on behind it, four by a warp.
constexpr int kJoinRows = 4;
constexpr int kParts = kUnitRows / kJoinWarps / kJoinRows;  // CTAs per unit

template <int D, bool kBF16>
__global__ void __launch_bounds__(kJoinThreads, 8)
    prefix_join_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kCols = D / 4;
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
  auto place = [&](int s, int i) {
    return static_cast<long long>(s == 0 ? p.grid + cta : cta + s) *
               kUnitRows + i;
  };
  if (parts == 2 && D == 128) {
    // The usual case, all rows at once: lane 2 i + s has row i's part s.
    float x = -INFINITY;
    if (lane < 2 * n) x = p.slot_lse2[place(lane % 2, i0 + lane / 2)];
    float4 y[kJoinRows][2];
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        y[i][s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n)
          y[i][s] = reinterpret_cast<const float4*>(
              p.slot_o)[place(s, i0 + i) * kCols + lane % kCols];
      }
    const float m = fmaxf(kNone, fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1)));
    const float f = ptx::ex2(x - m);
    const float sum = f + __shfl_xor_sync(0xffffffffu, f, 1);
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
      Sum t;
      t.mx = __shfl_sync(0xffffffffu, m, 2 * i);
      t.sum = __shfl_sync(0xffffffffu, sum, 2 * i);
      t.acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        add(t.acc, y[i][s], __shfl_sync(0xffffffffu, f, 2 * i + s));
      if (i < n)
        write_row<D, kBF16>(p, q_row_index(p, b, h, r0 + i), t, lane);
    }
    return;
  }
  for (int i = 0; i < n; ++i) {
    const Sum t = add_parts<D>(
        0, parts, lane, [&](int s, const float4** o, const float** lse2) {
          const long long j = place(s, i0 + i);
          *o = reinterpret_cast<const float4*>(p.slot_o) + j * kCols;
          *lse2 = p.slot_lse2 + j;
        });
    write_row<D, kBF16>(p, q_row_index(p, b, h, r0 + i), t, lane);
  }
}

template <int D, bool kBF16>
cudaError_t launch(PrefixParams p, cudaStream_t stream) {
  if (p.mode == kJoint)
    return kv8::launch_pdl(prefix_join_kernel<D, kBF16>,
                           static_cast<long long>(p.grid) * kParts,
                           kJoinThreads, 0, stream, p);
  const long long rows = static_cast<long long>(p.B) * p.rows * p.Hkv;
  // Warps a row: as many as make the machine's warps busy, rows having some 20
  // parts where they are few.
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
