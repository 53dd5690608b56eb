// Quantising new K and V tokens into the 8-bit cache.
//
// One unit = one block of tokens of one (batch, K/V head) of K or of V.  Its
// threads hold the block's new tokens in registers (64 elements a thread),
// reduce the largest finite magnitude, settle the block's scale and store the
// codes: each input element is read once and each code written once.  A block
// begun by an earlier call whose scale has to grow also has its held codes
// read, shifted to the new scale and written back.  Powers of two make both
// the product with the scale's reciprocal and the requantisation of normal
// codes exact, so the only rounding is the one to E4M3.
//
// Bound by memory traffic (2 bytes in, 1 out per element) on prompts: 8 x 4096
// tokens of 8 heads, D = 128, 201 MB in 33.8 us, 5.95 TB/s (88 % of a copy's
// rate); 8-byte stores and a division per element took 39.6.  One new token
// per sequence: 6.0 us, the call itself.
#include "kv8_common.cuh"
#include "kv8_index.h"

namespace attn {
namespace kv8 {
namespace {

// Threads of a unit: 64 elements each, at least one warp.
template <int D, int kBlock>
__host__ __device__ constexpr int unit_threads() {
  return kBlock * D / 64 < 32 ? 32 : kBlock * D / 64;
}

template <int D, int kBlock, bool kBF16>
__global__ void __launch_bounds__(unit_threads<D, kBlock>(),
                                  896 / unit_threads<D, kBlock>())
    kv8_append_kernel(const AppendParams p) {
  constexpr int kThreads = unit_threads<D, kBlock>();
  constexpr int kWarps = kThreads / 32;
  constexpr int kPerRow = D / 16;                       // 16-element chunks
  constexpr int kChunks = kBlock * kPerRow / kThreads;  // per thread
  static_assert(kChunks * kThreads == kBlock * kPerRow, "whole chunks");
  __shared__ float red[kWarps];

  start_after_previous();
  // Unit = (batch, head), block of that head, K or V.
  const int kv = blockIdx.x & 1;
  const int bh = (blockIdx.x >> 1) / p.units_per_seq;
  const int u = (blockIdx.x >> 1) - bh * p.units_per_seq;
  const int b = bh / p.Hkv;
  const int len = clamp_len(p.lens[b], p.capacity, p.status);
  const int n_new =
      p.new_lens == nullptr
          ? clamp_len(p.Sq, len, p.status)
          : clamp_len(p.new_lens[b], min(p.Sq, len), p.status);
  const int start = len - n_new;  // position of the first new token
  if (n_new == 0) return;
  const int blk = append_block(start, len, kBlock, u);
  if (blk < 0) return;
  const int base = blk * kBlock;  // first token of the block

  // Tokens [base, start) of the block are held already, [t0, t1) are new.
  const int t0 = max(start, base), t1 = min(len, base + kBlock);
  const uint16_t* x = static_cast<const uint16_t*>(p.x[kv]) +
                      (static_cast<long long>(bh) * p.Sq - start) * D;
  uint8_t* code = p.code[kv] + static_cast<long long>(bh) * p.capacity * D;
  float* scale = p.scale[kv] + static_cast<long long>(bh) * p.nblk + blk;

  uint4 in[kChunks][2];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = threadIdx.x + i * kThreads;
    const int tok = base + c / kPerRow;
    in[i][0] = in[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (tok >= t0 && tok < t1) {
      const uint4* at = reinterpret_cast<const uint4*>(
          x + static_cast<long long>(tok) * D + (c % kPerRow) * 16);
      in[i][0] = __ldg(at);
      in[i][1] = __ldg(at + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t w[4] = {in[i][q].x, in[i][q].y, in[i][q].z, in[i][q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<kBF16>(w[e]);
        amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
    }
#pragma unroll
  for (int s = 16; s > 0; s /= 2)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
  const bool begun = base < start;
  float old = 0.f;
  if (begun) old = *scale;
  if constexpr (kWarps > 1) {
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = amax;
    __syncthreads();  // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kWarps; ++i) amax = fmaxf(amax, red[i]);
  } else {
    __syncwarp();
  }
  const int e = tight_exponent(amax);
  const bool keep = begun && amax <= kE4m3Max * old;
  const float now = keep ? old : exp2_int(e);
  if (threadIdx.x == 0 && !keep) *scale = now;

  if (!is_power_of_two(now)) {
    // A kept scale of other origin: quotients rounded to fp32.  (A rounded
    // reciprocal would move quotients that are ties.)  The tokens are read
    // again, so that this path costs the usual one no registers.
    for (int c = threadIdx.x; c < kBlock * (D / 8); c += kThreads) {
      const int tok = base + c / (D / 8);
      if (tok < t0 || tok >= t1) continue;
      const long long at = static_cast<long long>(tok) * D + c % (D / 8) * 8;
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(x + at));
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2<kBF16>(w[j]);
        f[2 * j] = v.x / now;
        f[2 * j + 1] = v.y / now;
      }
      *reinterpret_cast<uint2*>(code + at) =
          make_uint2(ptx::pack4_e4m3(f[0], f[1], f[2], f[3]),
                     ptx::pack4_e4m3(f[4], f[5], f[6], f[7]));
    }
    return;
  }
  const float inv = reciprocal(now);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = threadIdx.x + i * kThreads;
    const int tok = base + c / kPerRow;
    if (tok < t0 || tok >= t1) continue;
    uint32_t out[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t w[4] = {in[i][q].x, in[i][q].y, in[i][q].z, in[i][q].w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2<kBF16>(w[j]);
        f[2 * j] = v.x;
        f[2 * j + 1] = v.y;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= inv;
      out[2 * q] = ptx::pack4_e4m3(f[0], f[1], f[2], f[3]);
      out[2 * q + 1] = ptx::pack4_e4m3(f[4], f[5], f[6], f[7]);
    }
    *reinterpret_cast<uint4*>(code + static_cast<long long>(tok) * D +
                              (c % kPerRow) * 16) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
  if (begun && !keep) {
    // The block's scale grew: the codes it holds move to the new one.
    for (int c = threadIdx.x; c < (start - base) * (D / 8); c += kThreads) {
      uint2* at = reinterpret_cast<uint2*>(
          code + static_cast<long long>(base) * D + c * 8);
      const uint2 held = *at;
      float f[8];
      e4m3x4_to_float(held.x, f);
      e4m3x4_to_float(held.y, f + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * old * inv;
      *at = make_uint2(ptx::pack4_e4m3(f[0], f[1], f[2], f[3]),
                       ptx::pack4_e4m3(f[4], f[5], f[6], f[7]));
    }
  }
}

template <int D, int kBlock>
cudaError_t launch(bool bf16, const AppendParams& p, long long grid,
                   cudaStream_t stream) {
  constexpr int kThreads = unit_threads<D, kBlock>();
  return bf16 ? launch_pdl(kv8_append_kernel<D, kBlock, true>, grid, kThreads,
                           0, stream, p)
              : launch_pdl(kv8_append_kernel<D, kBlock, false>, grid, kThreads,
                           0, stream, p);
}

template <int D>
cudaError_t launch_d(int block, bool bf16, const AppendParams& p, long long grid,
                     cudaStream_t stream) {
  switch (block) {
    case 16: return launch<D, 16>(bf16, p, grid, stream);
    case 32: return launch<D, 32>(bf16, p, grid, stream);
    case 64: return launch<D, 64>(bf16, p, grid, stream);
    default: return launch<D, 128>(bf16, p, grid, stream);
  }
}

}  // namespace

cudaError_t launch_append(int D, int block, bool bf16, const AppendParams& p,
                          int B, cudaStream_t stream) {
  const long long grid = 2LL * B * p.Hkv * p.units_per_seq;
  return D == 64 ? launch_d<64>(block, bf16, p, grid, stream)
                 : launch_d<128>(block, bf16, p, grid, stream);
}

}  // namespace kv8
}  // namespace attn
