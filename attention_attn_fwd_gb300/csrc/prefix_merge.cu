// Joins the parts of a query row's attention behind a shared prefix: a warp per
// row.  With part s the average O_s and the log-sum-exp L_s of its keys,
//   O = sum_s 2^(L_s - m) O_s / sum_s 2^(L_s - m),  LSE = m + log2(the sum).
#include "prefix_common.cuh"

namespace attn {
namespace prefix {
namespace {

using kv8::kNone;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The sum over parts 0 .. n - 1, where at(s) gives the row of part s in an
// array of O rows and one of LSEs.  (A part that sees nothing has the factor 0
// and no O.)
template <int D, bool kBF16, class At>
__device__ __forceinline__ void join(const PrefixParams& p, int n,
                                     long long row, int lane, At at) {
  constexpr int kCols = D / 4;          // float4 columns
  constexpr int kGroups = 32 / kCols;   // parts a warp reads at a time
  const int col = lane % kCols, sub = lane / kCols;
  float mx = kNone, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += 32) {
    float x = -INFINITY;
    if (s0 + lane < n) {
      const float *o, *lse2;
      const long long i = at(s0 + lane, &o, &lse2);
      x = lse2[i];
    }
    float m = mx;
    m = fmaxf(m, x);
#pragma unroll
    for (int k = 16; k > 0; k /= 2)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float before = ptx::ex2(mx - m);
    const float f_all = ptx::ex2(x - m);
    mx = m;
    acc.x *= before;
    acc.y *= before;
    acc.z *= before;
    acc.w *= before;
    sum = sum * before + f_all;  // (a lane's share)
    const int count = min(32, n - s0);
#pragma unroll 4
    for (int k = 0; k < count; k += kGroups) {
      const int s = k + sub;
      const float f = __shfl_sync(0xffffffffu, f_all, s % 32);
      if (s < count && f != 0.f) {
        const float *o, *lse2;
        const long long i = at(s0 + s, &o, &lse2);
        const float4 y = reinterpret_cast<const float4*>(o)[i * kCols + col];
        acc.x += y.x * f;
        acc.y += y.y * f;
        acc.z += y.z * f;
        acc.w += y.w * f;
      }
    }
  }
  // (The lanes' shares were scaled alike.)
#pragma unroll
  for (int k = 16; k > 0; k /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  if constexpr (kGroups == 2) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (lane < kCols) {
    uint2 out;
    out.x = ptx::pack2<kBF16>(acc.x * inv, acc.y * inv);
    out.y = ptx::pack2<kBF16>(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(p.o + row * D)[col] = out;
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = sum == 0.f ? -INFINITY
                            : (mx + log2f(sum)) * 0.69314718055994531f;
}

// kFew and kPacked: every row, with the parts over the prefix first.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long id = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int R = p.rows;
  const long long all = static_cast<long long>(p.B) * R;  // rows of a head
  const bool in = id < all * p.Hkv;
  // (b, h, r), r fastest.
  const int bh = in ? static_cast<int>(id / R) : 0;
  const int r = in ? static_cast<int>(id - static_cast<long long>(bh) * R) : 0;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int len = kv8::seq_len(p, b), n_new = kv8::seq_new(p, b);
  const int np = prefix_tiles(p);
  const int x = b * R + r;
  const int u = r / kUnitRows;
  // (Lengths are read ahead of the wait: the kernels ahead do not write them.)
  int few_first = 0, few_n = 0;
  if (p.mode == kFew && len > 0 && in) {
    constexpr int kKeys = few_keys<D>();
    const int tiles = (len + kKeys - 1) / kKeys;
    int first;
    const int total = kv8::list_tiles<kKeys, kFewOver>(p, b, lane, &first);
    const kv8::Cut cut = kv8::make_cut<kFewWarps>(p, total);
    first += h * (tiles + kFewOver) + kFewOver;
    few_first = cut.owner(first);
    few_n = cut.owner(first + tiles - 1) - few_first + 1;
  }
  kv8::start_after_previous();
  if (!in || r >= n_new * p.group) return;
  int2 pre = make_int2(0, 0), own = make_int2(0, 0);
  if (np > 0)
    pre = p.info[static_cast<long long>(x / kUnitRows) * p.Hkv + h];
  if (p.mode == kFew)
    own = make_int2(few_first, few_n);
  else if (tiles_seen(p, len, n_new, u * kUnitRows, (u + 1) * kUnitRows) > 0)
    own = p.info[(static_cast<long long>(p.pack_blocks) +
                  static_cast<long long>(b) * p.row_blocks + u) * p.Hkv + h];
  auto at = [&](int s, const float** o, const float** lse2) -> long long {
    *o = p.base_o;
    *lse2 = p.base_lse2;
    if (s == 0 && pre.y > 0) return h * all + x;
    if (s < pre.y) {
      *o = p.slot_o;
      *lse2 = p.slot_lse2;
      return static_cast<long long>(pre.x + s) * kUnitRows + x % kUnitRows;
    }
    s -= pre.y;
    if (p.mode == kFew) {
      *o = p.few_o;
      *lse2 = p.few_lse2;
      return (static_cast<long long>(own.x + s) + bh) * few_rows(R) + r;
    }
    if (s == 0) return p.Hkv * all + static_cast<long long>(bh) * R + r;
    *o = p.slot_o;
    *lse2 = p.slot_lse2;
    return static_cast<long long>(own.x + s) * kUnitRows + r % kUnitRows;
  };
  join<D, kBF16>(p, pre.y + own.y, q_row_index(p, b, h, r), lane, at);
}

// kJoint: the rows of each CTA's unit that went on behind it.
constexpr int kParts = kUnitRows / kWarps;  // CTAs per unit

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads)
    prefix_join_kernel(const __grid_constant__ PrefixParams p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x / kParts;
  const int i = (blockIdx.x - cta * kParts) * kWarps + warp;
  kv8::start_after_previous();
  const int4 split = p.split[cta];
  const int b = split.x, h = split.y, parts = split.w;
  if (parts == 0) return;
  const int r = split.z * kUnitRows + i;
  if (r >= kv8::seq_new(p, b) * p.group) return;
  auto at = [&](int s, const float** o, const float** lse2) -> long long {
    *o = p.slot_o;
    *lse2 = p.slot_lse2;
    return static_cast<long long>(s == 0 ? p.many_grid + cta : cta + s) *
               kUnitRows + i;
  };
  join<D, kBF16>(p, parts, q_row_index(p, b, h, r), lane, at);
}

template <int D, bool kBF16>
cudaError_t launch(PrefixParams p, cudaStream_t stream) {
  if (p.mode == kJoint)
    return kv8::launch_pdl(prefix_join_kernel<D, kBF16>,
                           static_cast<long long>(p.many_grid) * kParts,
                           kThreads, 0, stream, p);
  p.grid = p.few_grid;
  const long long rows = static_cast<long long>(p.B) * p.rows * p.Hkv;
  return kv8::launch_pdl(prefix_merge_kernel<D, kBF16>,
                         (rows + kWarps - 1) / kWarps, kThreads, 0, stream, p);
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
