// Accumulated attention weights of many query rows over the 8-bit cache.
//
// w_j += sum over the rows i that see key j of 2^(s_ij - LSE_i), with the
// rows' LSEs (log2 units) of the forward launch ahead of this one.  The scores
// are computed again -- a stored score costs 8 bytes of traffic, a recomputed
// one D / 8 MMAs of the 256 keys x 8 rows -- as S^T = K Q^T with mma.sync in
// fp16 like the few-row kernel's (its header comment has the fragments and
// the roundings): a warp keeps the fragments of its 32 keys in registers, the
// rows pass through shared memory 64 at a time, the next 64 being loaded
// meanwhile.  Each key has one owner that takes the rows in order: no atomics,
// one order of sums.  Bound by issue (MMA, exp2 and their addressing).
#include "attn_sync.cuh"
#include "kv8_common.cuh"

namespace attn {
namespace kv8 {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 32 * (kThreads / 32);  // keys of a CTA
constexpr int kRowsAt = 64;                  // rows in shared memory at a time

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 2)
    kv8_weights_kernel(const FwdParams p, int tiles, int lse2_rows) {
  constexpr int kPitch = D + 8;  // halves: rows 16 bytes apart in the banks
  constexpr int kPer = D / 8;    // threads that load a row
  constexpr int kLoads = kRowsAt * kPer / kThreads;
  __shared__ __align__(16) uint16_t sq[2][kRowsAt * kPitch];
  __shared__ float s_mult[2][kRowsAt], s_lse[2][kRowsAt];
  start_after_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g8 = lane / 4, c = lane % 4;
  const int bh = blockIdx.x / tiles;
  const int tile0 = (blockIdx.x - bh * tiles) * kKeys;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int len = seq_len(p, b), n_new = seq_new(p, b);
  if (tile0 >= len) return;
  const int rows = n_new * p.group;
  // Rows before r_first see nothing of this tile.
  const int r_first =
      p.causal ? max(0, tile0 - (len - n_new)) * p.group : 0;
  const int key0 = tile0 + warp * 32;

  // Fragments of keys key0 + 16 u + g8 (+ 8).
  uint32_t a[2][D / 16][4];
  float ks[2];
  const uint8_t* k = p.k + static_cast<long long>(bh) * p.capacity * D;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        const int key = key0 + 16 * u + g8 + 8 * i;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (key < len)
          x = __ldg(reinterpret_cast<const uint4*>(
              k + static_cast<long long>(key) * D + 64 * hf + 16 * c));
        e4m3x4_to_half2(x.x, a[u][4 * hf][i], a[u][4 * hf][2 + i]);
        e4m3x4_to_half2(x.y, a[u][4 * hf + 1][i], a[u][4 * hf + 1][2 + i]);
        e4m3x4_to_half2(x.z, a[u][4 * hf + 2][i], a[u][4 * hf + 2][2 + i]);
        e4m3x4_to_half2(x.w, a[u][4 * hf + 3][i], a[u][4 * hf + 3][2 + i]);
      }
    ks[u] = 0.f;
    if (key0 + 16 * u < len)
      ks[u] = __ldg(p.k_scale + static_cast<long long>(bh) * p.nblk +
                    ((key0 + 16 * u) >> p.block_shift));
  }

  // Rows r0 .. r0 + 63: this thread's chunks, and its row's LSE.
  uint4 x[kLoads];
  float lse[kLoads];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int i = threadIdx.x + e * kThreads;
      const int r = r0 + i / kPer;
      x[e] = make_uint4(0u, 0u, 0u, 0u);
      lse[e] = INFINITY;  // a row of no weight
      if (r < rows) {
        const int tok = r / p.group, hd = r - tok * p.group;
        x[e] = __ldg(reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) +
            ((static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq +
             tok) * D + i % kPer * 8));
        lse[e] = p.lse2[static_cast<long long>(bh) * lse2_rows + r];
        if (lse[e] == -INFINITY) lse[e] = INFINITY;  // sees nothing
      }
    }
  };
  auto store_rows = [&](int buf) {
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int i = threadIdx.x + e * kThreads;
      const int r = i / kPer, ch = i % kPer;
      const uint32_t in[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
      float2 f[4];
      float amax = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[q] = unpack2<kBF16>(in[q]);
        amax = fmaxf(amax, fmaxf(fabsf(f[q].x), fabsf(f[q].y)));
      }
#pragma unroll
      for (int s = kPer / 2; s > 0; s /= 2)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
      const int up = row_shift(amax);
      const float f_up = exp2_int(up);
      uint32_t out[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        out[q] = ptx::pack2<false>(f[q].x * f_up, f[q].y * f_up);
      *reinterpret_cast<uint4*>(&sq[buf][r * kPitch + ch * 8]) =
          make_uint4(out[0], out[1], out[2], out[3]);
      if (ch == 0) {
        s_mult[buf][r] = p.scale_log2 * exp2_int(-up);
        s_lse[buf][r] = lse[e];
      }
    }
  };

  float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  auto add_rows = [&](int buf, int r0, auto masked_tag) {
    constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll 1
    for (int nt = 0; nt < kRowsAt / 8; ++nt) {
      uint32_t bw[D / 64][8];
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        const uint16_t* row =
            &sq[buf][(8 * nt + g8) * kPitch + 64 * hf + 16 * c];
        const uint4 w0 = *reinterpret_cast<const uint4*>(row);
        const uint4 w1 = *reinterpret_cast<const uint4*>(row + 8);
        bw[hf][0] = w0.x; bw[hf][1] = w0.y; bw[hf][2] = w0.z; bw[hf][3] = w0.w;
        bw[hf][4] = w1.x; bw[hf][5] = w1.y; bw[hf][6] = w1.z; bw[hf][7] = w1.w;
      }
      const float2 mult =
          *reinterpret_cast<const float2*>(&s_mult[buf][8 * nt + 2 * c]);
      const float2 l2 =
          *reinterpret_cast<const float2*>(&s_lse[buf][8 * nt + 2 * c]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            mma_f16((w & 1) ? s2 : s, a[u][4 * hf + w][0], a[u][4 * hf + w][1],
                    a[u][4 * hf + w][2], a[u][4 * hf + w][3], bw[hf][2 * w],
                    bw[hf][2 * w + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float m = (e & 1) ? mult.y : mult.x;
          const float l = (e & 1) ? l2.y : l2.x;
          const float w = ptx::ex2(fmaf(s[e] + s2[e], m * ks[u], -l));
          if constexpr (kMasked) {
            const int key = key0 + 16 * u + g8 + 8 * (e >> 1);
            const int r = r0 + 8 * nt + 2 * c + (e & 1);
            if (r < rows && key < row_end(p, len, n_new, r))
              sum[u][e >> 1] += w;
          } else {
            sum[u][e >> 1] += w;
          }
        }
      }
    }
  };

  load_rows(r_first);
  int buf = 0;
  for (int r0 = r_first; r0 < rows; r0 += kRowsAt, buf ^= 1) {
    store_rows(buf);
    __syncthreads();  // one buffer is written while the other may be read
    if (r0 + kRowsAt < rows) load_rows(r0 + kRowsAt);
    if (key0 >= len) continue;
    // Rows see more and more tokens: the first one decides.
    if (key0 + 32 > row_end(p, len, n_new, r0))
      add_rows(buf, r0, BoolTag<true>{});
    else
      add_rows(buf, r0, BoolTag<false>{});
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float w = sum[u][e];
      w += __shfl_xor_sync(0xffffffffu, w, 1);
      w += __shfl_xor_sync(0xffffffffu, w, 2);
      const int key = key0 + 16 * u + g8 + 8 * e;
      if (c == 0 && key < len && w != 0.f)
        p.weights[static_cast<long long>(bh) * p.capacity + key] += w;
    }
}

template <int D, bool kBF16>
cudaError_t launch(const FwdParams& p, int lse2_rows, cudaStream_t stream) {
  const int tiles = (p.capacity - 1) / kKeys + 1;
  return launch_pdl(kv8_weights_kernel<D, kBF16>,
                    static_cast<long long>(p.B) * p.Hkv * tiles, kThreads, 0,
                    stream, p, tiles, lse2_rows);
}

}  // namespace

cudaError_t launch_weights(int D, bool bf16, int lse2_rows,
                           const FwdParams& p, cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch<64, true>(p, lse2_rows, stream)
                : launch<64, false>(p, lse2_rows, stream);
  return bf16 ? launch<128, true>(p, lse2_rows, stream)
              : launch<128, false>(p, lse2_rows, stream);
}

}  // namespace kv8
}  // namespace attn
