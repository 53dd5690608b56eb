// Eviction from the 8-bit cache by accumulated attention weight.
//
// Kernel 1 (select), one CTA per (batch, K/V head): the candidates' weights
// as order-preserving 32-bit keys; a radix select (four 8-bit digits from the
// top, one histogram pass each) finds the key of the last token kept and how
// many tokens of that very key stay (the earliest ones); a counting pass and
// a writing pass then list the kept places in ascending order.
//
// Kernel 2 (move), one cluster of CTAs per (batch, K/V head) and of K, V or
// the weights: blocks of destination tokens in ascending rounds, each CTA of
// the cluster one block a round: gather the codes to registers, reduce the
// largest magnitude, settle the block's power-of-two scale, shift the codes
// to it, store.  In place this is safe with one cluster barrier per round
// between its reads and its writes: the n-th kept token comes from a place
// >= n, so a round only overwrites places that no later round reads.
#include "kv8_common.cuh"

namespace attn {
namespace kv8 {
namespace {

// Order-preserving key: larger weight, larger key; -0 equals +0; NaN is
// less than every number (key 0).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

// Exclusive sum of two counters over the CTA's warps (lane 0's values
// count); every thread of a warp gets its warp's offsets.
__device__ __forceinline__ int2 warp_offsets(int2 v, int2* sm) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) sm[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const int2 x = sm[lane];
    int a = x.x, b = x.y;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const int ua = __shfl_up_sync(0xffffffffu, a, s);
      const int ub = __shfl_up_sync(0xffffffffu, b, s);
      if (lane >= s) {
        a += ua;
        b += ub;
      }
    }
    sm[lane] = make_int2(a - x.x, b - x.y);
  }
  __syncthreads();
  const int2 r = sm[warp];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kSelThreads)
    kv8_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int2 sm_warp[32];
  __shared__ uint32_t s_digit;
  __shared__ int s_left;
  start_after_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int bh = blockIdx.x;
  const int b = bh / p.Hkv;
  const int len = clamp_len(p.src_lens[b], p.src_capacity, p.status);
  int* idx = p.indices + static_cast<long long>(bh) * p.keep;
  if (len <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += kSelThreads)
      idx[i] = i < len ? i : -1;
    return;
  }
  const float* w = p.weights + static_cast<long long>(bh) * p.src_capacity;
  const int cand = len - p.recent;        // candidates: places [0, cand)
  const int want = p.keep - p.recent;     // of which so many stay
  // Radix select of the want-th largest key.
  uint32_t prefix = 0u, mask = 0u;
  int left = want;  // tokens still wanted among keys matching the prefix
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = threadIdx.x; j < cand; j += kSelThreads) {
        const uint32_t key = weight_key(w[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // Digits from the top, eight per lane (lane 0 holds 255 .. 248).
        int n[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          n[e] = hist[255 - (8 * lane + e)];
          sum += n[e];
        }
        int incl = sum;
#pragma unroll
        for (int s = 1; s < 32; s *= 2) {
          const int up = __shfl_up_sync(0xffffffffu, incl, s);
          if (lane >= s) incl += up;
        }
        int before = incl - sum;
        if (before < left && incl >= left) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (before < left && before + n[e] >= left) {
              s_digit = 255u - (8 * lane + e);
              s_left = left - before;
            }
            before += n[e];
          }
        }
      }
      __syncthreads();
      prefix |= s_digit << shift;
      mask |= 255u << shift;
      left = s_left;
      __syncthreads();
    }
  }
  // Kept: keys above the threshold, the first `left` tokens of its very key,
  // and the recent ones.  Each warp takes a consecutive range of places.
  const int per = (len + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int j0 = min(len, warp * per), j1 = min(len, j0 + per);
  auto flags = [&](int j, unsigned* above, unsigned* equal) {
    bool a = false, q = false;
    if (j < j1) {
      if (j >= cand) {
        a = true;
      } else if (want > 0) {
        const uint32_t key = weight_key(w[j]);
        a = key > prefix;
        q = key == prefix;
      }
    }
    *above = __ballot_sync(0xffffffffu, a);
    *equal = __ballot_sync(0xffffffffu, q);
  };
  int2 n = make_int2(0, 0);
  for (int j = j0; j < j1; j += 32) {
    unsigned a, q;
    flags(j + lane, &a, &q);
    n.x += __popc(a);
    n.y += __popc(q);
  }
  const int2 off = warp_offsets(n, sm_warp);
  int above = off.x, equal = off.y;
  for (int j = j0; j < j1; j += 32) {
    unsigned a, q;
    flags(j + lane, &a, &q);
    const unsigned lower = (1u << lane) - 1u;
    const int eq_rank = equal + __popc(q & lower);
    const bool is_eq = (q >> lane) & 1u;
    const bool kept = ((a >> lane) & 1u) || (is_eq && eq_rank < left);
    if (kept) {
      const int at = above + __popc(a & lower) + min(eq_rank, left);
      idx[at] = j + lane;
    }
    above += __popc(a);
    equal += __popc(q);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kCluster = 8;

// One round of the codes: destination block `nb` of one head.
template <int D>
__device__ __forceinline__ void move_codes(const EvictParams& p, int kv,
                                           int bh, int rank, int len,
                                           int n_kept) {
  constexpr int kPerRow = D / 16;                       // 16-byte chunks
  constexpr int kMax = 128 * kPerRow / kMoveThreads;    // chunks per thread
  __shared__ float red[kMoveThreads / 32];
  const int block = 1 << p.block_shift;
  const bool whole = len <= p.keep;  // nothing leaves: bit for bit
  const int* idx = p.indices + static_cast<long long>(bh) * p.keep;
  const uint8_t* src = p.src_code[kv] +
                       static_cast<long long>(bh) * p.src_capacity * D;
  const float* src_scale = p.src_scale[kv] +
                           static_cast<long long>(bh) * p.src_nblk;
  uint8_t* dst = p.dst_code[kv] +
                 static_cast<long long>(bh) * p.dst_capacity * D;
  float* dst_scale = p.dst_scale[kv] + static_cast<long long>(bh) * p.dst_nblk;
  const int blocks = (n_kept + block - 1) >> p.block_shift;
  const int rounds = (blocks + kCluster - 1) / kCluster;
  const int chunks = block * kPerRow;
  for (int rd = 0; rd < rounds; ++rd) {
    const int nb = rd * kCluster + rank;
    const int t0 = nb << p.block_shift;
    uint4 held[kMax];
    float factor[kMax];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int ch = threadIdx.x + i * kMoveThreads;
      const int tok = t0 + ch / kPerRow;
      held[i] = make_uint4(0u, 0u, 0u, 0u);
      factor[i] = 0.f;
      if (ch < chunks && tok < n_kept) {
        const int from = whole ? tok : idx[tok];
        held[i] = *reinterpret_cast<const uint4*>(
            src + static_cast<long long>(from) * D + (ch % kPerRow) * 16);
        factor[i] = src_scale[from >> p.block_shift];
        const uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f[4];
          e4m3x4_to_float(w[e], f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, finite_abs(f[j] * factor[i]));
        }
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s /= 2)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = amax;
    float first = 0.f;
    if (whole && threadIdx.x == 0 && nb < blocks) first = src_scale[nb];
    if (p.in_place) {
      // Every CTA of the cluster has read what this round overwrites.
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kMoveThreads / 32; ++i) amax = fmaxf(amax, red[i]);
    const float now = exp2_int(tight_exponent(amax));
    const float inv = 1.f / now;
    if (threadIdx.x == 0 && nb < blocks) dst_scale[nb] = whole ? first : now;
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int ch = threadIdx.x + i * kMoveThreads;
      const int tok = t0 + ch / kPerRow;
      if (ch < chunks && tok < n_kept) {
        uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f[4];
            e4m3x4_to_float(w[e], f);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = f[j] * factor[i] * inv;
            w[e] = ptx::pack4_e4m3(f[0], f[1], f[2], f[3]);
          }
        }
        *reinterpret_cast<uint4*>(dst + static_cast<long long>(tok) * D +
                                  (ch % kPerRow) * 16) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncthreads();  // red is free again
  }
}

__device__ __forceinline__ void move_weights(const EvictParams& p, int bh,
                                             int rank, int n_kept) {
  const int* idx = p.indices + static_cast<long long>(bh) * p.keep;
  const float* src = p.weights + static_cast<long long>(bh) * p.src_capacity;
  float* dst = p.dst_weights + static_cast<long long>(bh) * p.dst_capacity;
  constexpr int kPer = 4 * kMoveThreads;  // tokens a CTA moves per round
  const int step = kPer * kCluster;
  const int rounds = (n_kept + step - 1) / step;
  for (int rd = 0; rd < rounds; ++rd) {
    const int t0 = rd * step + rank * kPer + threadIdx.x;
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t0 + i * kMoveThreads;
      w[i] = tok < n_kept ? src[idx[tok]] : 0.f;
    }
    if (p.in_place) {
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t0 + i * kMoveThreads;
      if (tok < n_kept) dst[tok] = w[i];
    }
  }
  if (p.in_place && rounds == 0) {
    ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
  }
  // Every read of the sources is behind the last round's barrier.
  for (int tok = n_kept + rank * kMoveThreads + threadIdx.x;
       tok < p.dst_capacity; tok += kCluster * kMoveThreads)
    dst[tok] = 0.f;
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads)
    kv8_move_kernel(const EvictParams p) {
  start_after_previous();
  const int rank = blockIdx.x % kCluster;
  const int unit = blockIdx.x / kCluster;
  const int part = unit % 3;  // K, V, weights
  const int bh = unit / 3;
  const int b = bh / p.Hkv;
  const int len = clamp_len(p.src_lens[b], p.src_capacity, p.status);
  const int n_kept = min(len, p.keep);
  if (part < 2) {
    if (p.in_place && len <= p.keep) return;  // stays as it is
    move_codes<D>(p, part, bh, rank, len, n_kept);
  } else {
    move_weights(p, bh, rank, n_kept);
    if (bh % p.Hkv == 0 && rank == 0 && threadIdx.x == 0)
      p.dst_lens[b] = n_kept;
  }
}

template <int D>
cudaError_t launch_move(const EvictParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * 3 * kCluster, 1, 1);
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv8_move_kernel<D>, p);
}

}  // namespace

cudaError_t launch_evict(int D, const EvictParams& p, cudaStream_t stream) {
  const cudaError_t err =
      launch_pdl(kv8_select_kernel, static_cast<long long>(p.B) * p.Hkv,
                 kSelThreads, 0, stream, p);
  if (err != cudaSuccess) return err;
  return D == 64 ? launch_move<64>(p, stream) : launch_move<128>(p, stream);
}

}  // namespace kv8
}  // namespace attn
