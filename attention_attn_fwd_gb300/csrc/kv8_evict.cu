// Eviction from the 8-bit cache by accumulated attention weight.
//
// Kernel 1 (select), a cluster of 1 to 8 CTAs per (batch, K/V head), each with
// a consecutive part of the tokens: the candidates' weights become
// order-preserving 32-bit keys in registers (one pass over them in memory up
// to 131072 tokens); a radix select (four 8-bit digits from the top, the
// parts' histograms summed over the cluster) finds the key of the last token
// kept and how many tokens of that very key stay (the earliest ones); counts
// of kept tokens, summed over the parts before, give each its place in the
// ascending list.
//
// Kernel 2 (move), CTAs by (batch, K/V head) and K, V or the weights, one
// block of destination tokens at a time: gather the codes to registers,
// reduce the largest magnitude, settle the block's power-of-two scale, shift
// the codes to it, store.  Into another cache every block is a CTA of its
// own.  In place a cluster of eight takes the blocks in ascending rounds with
// one cluster barrier per round between its reads and its writes: the n-th
// kept token comes from a place >= n, so a round only overwrites places that
// no later round reads.
//
// Measured: 8 x 8 heads of 4096 tokens to 2048, D = 128, 24.0 us; 4 heads of
// 131072 tokens to 16384, 27.5 us; one call by itself, 29 and 33 us, in place
// 41 and 64 (its rounds wait for one another).  Select is bound by latency
// (four digits of a cluster barrier and two block barriers each: 9 and 20 us
// of the two when launched alone), move by the gather (17 and 11 us, 69 and 36
// MB: a block's largest magnitude is known only after the last of its
// scattered rows has come).  Keys one per lane instead of in quads: 31.8 us on
// the long one; one CTA per head for the select 191 us.
#include "kv8_common.cuh"
#include "kv8_index.h"

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
constexpr int kMaxCluster = 8;
constexpr int kQuadsAt = 4;         // most quads of keys a thread holds

// Shared memory of a select CTA that peers read.
struct Shared {
  int hist[2][256];      // of the digit, double-buffered
  int sum[256];          // the same, of the whole cluster
  int2 count;            // kept for certain, equal to the threshold
  int2 warp[kQuadsAt * kSelWarps];  // the same, before each 128 places
  int2 group[kQuadsAt];             // per 4096
  unsigned digit;
  int left;
};

__device__ __forceinline__ uint32_t ld_peer(const void* p, uint32_t rank) {
  return static_cast<uint32_t>(ptx::ld_shared_cluster_s32(
      ptx::mapa_shared(ptx::smem_u32(p), rank)));
}
// kQuads: quads of keys a thread holds; element e of quad i of thread t is
// place 4 (1024 i + t) + e of the CTA's part.  Longer parts are walked in
// turns of 4096 kQuads places, their keys read again in each pass.
template <int kQuads>
__global__ void __launch_bounds__(kSelThreads, 1)
    kv8_select_kernel(const EvictParams p, int ranks) {
  __shared__ Shared sh;
  start_after_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int bh = blockIdx.x / ranks, rank = blockIdx.x - bh * ranks;
  const int b = bh / p.Hkv;
  const int len = clamp_len(p.src_lens[b], p.src_capacity, p.status);
  int* idx = p.indices + static_cast<long long>(bh) * p.keep;
  if (len <= p.keep) {  // the whole cluster
    for (int i = rank * kSelThreads + threadIdx.x; i < p.keep;
         i += ranks * kSelThreads)
      idx[i] = i < len ? i : -1;
    return;
  }
  const float* w = p.weights + static_cast<long long>(bh) * p.src_capacity;
  const int cand = len - p.recent;        // candidates: places [0, cand)
  const int want = p.keep - p.recent;     // of which so many stay
  constexpr int kTurn = 4 * kSelThreads * kQuads;
  const int part = ((len + ranks - 1) / ranks + 3) / 4 * 4;
  const int a0 = min(len, rank * part), a1 = min(len, a0 + part);
  const int c1 = min(a1, cand);  // candidates of this CTA: [a0, c1)
  const int turns = (part + kTurn - 1) / kTurn;
  const bool aligned = (reinterpret_cast<uintptr_t>(w + a0) & 15) == 0;
  uint32_t key[kQuads][4];
  auto load = [&](int at) {  // the turn that begins at place `at`
    float4 x[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int j = at + 4 * (i * kSelThreads + threadIdx.x);
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (aligned && j + 4 <= c1) {
        x[i] = __ldg(reinterpret_cast<const float4*>(w + j));
      } else {
        if (j < c1) x[i].x = __ldg(w + j);
        if (j + 1 < c1) x[i].y = __ldg(w + j + 1);
        if (j + 2 < c1) x[i].z = __ldg(w + j + 2);
        if (j + 3 < c1) x[i].w = __ldg(w + j + 3);
      }
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      key[i][0] = weight_key(x[i].x);
      key[i][1] = weight_key(x[i].y);
      key[i][2] = weight_key(x[i].z);
      key[i][3] = weight_key(x[i].w);
    }
  };
  load(a0);
  if (threadIdx.x < 512) sh.hist[threadIdx.x / 256][threadIdx.x % 256] = 0;
  __syncthreads();

  // Radix select of the want-th largest key.
  uint32_t prefix = 0u, mask = 0u;
  int left = want;  // tokens still wanted among keys matching the prefix
  for (int shift = 24, buf = 0; shift >= 0 && want > 0; shift -= 8, buf ^= 1) {
    for (int t = 0; t < turns; ++t) {
      const int at = a0 + t * kTurn;
      if (turns > 1) load(at);
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = at + 4 * (i * kSelThreads + threadIdx.x) + e;
          if (j < c1 && (key[i][e] & mask) == prefix)
            atomicAdd(&sh.hist[buf][(key[i][e] >> shift) & 255u], 1);
        }
    }
    if (ranks > 1)
      cluster_barrier();
    else
      __syncthreads();
    if (threadIdx.x < 256) {
      int n = 0;
      if (ranks > 1) {
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < ranks)
            n += static_cast<int>(ld_peer(&sh.hist[buf][threadIdx.x], r));
      } else {
        n = sh.hist[buf][threadIdx.x];
      }
      sh.sum[threadIdx.x] = n;
    } else if (threadIdx.x < 512 && shift < 24) {
      // The other buffer was read ahead of this digit's barrier: clear it
      // for the next one.
      sh.hist[buf ^ 1][threadIdx.x - 256] = 0;
    }
    __syncthreads();
    if (warp == 0) {
      // Digits from the top, eight per lane (lane 0 holds 255 .. 248).
      int n[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] = sh.sum[255 - (8 * lane + e)];
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
            sh.digit = 255u - (8 * lane + e);
            sh.left = left - before;
          }
          before += n[e];
        }
      }
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= 255u << shift;
    left = sh.left;
  }
  // Kept: keys above the threshold, the first `left` tokens of its very key,
  // and the recent ones.
  // Bits e: element e of quad i is above the threshold (or recent); bits
  // 4 + e: equal to it.
  auto flags = [&](int at, int i) {
    unsigned f = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = at + 4 * (i * kSelThreads + threadIdx.x) + e;
      const bool c = j < c1 && want > 0;
      if ((j >= cand && j < a1) || (c && key[i][e] > prefix)) f |= 1u << e;
      if (c && key[i][e] == prefix) f |= 16u << e;
    }
    return f;
  };
  // Kept for certain (low half) and equal (high half) before this thread's
  // quads among its warp's 128 places; sh.warp: before those in the turn.
  unsigned lower[kQuads];
  auto count = [&](int at) -> int2 {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const unsigned f = flags(at, i);
      const unsigned x = __popc(f & 15u) | (__popc(f >> 4) << 16);
      unsigned incl = x;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const unsigned up = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += up;
      }
      lower[i] = incl - x;
      if (lane == 31)
        sh.warp[i * kSelWarps + warp] =
            make_int2(static_cast<int>(incl & 0xffffu),
                      static_cast<int>(incl >> 16));
    }
    __syncthreads();
    int2 x = make_int2(0, 0), incl = x;
    if (warp < kQuads) {  // warp i: the 32 counts of quad i
      x = incl = sh.warp[warp * kSelWarps + lane];
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const int ua = __shfl_up_sync(0xffffffffu, incl.x, s);
        const int uq = __shfl_up_sync(0xffffffffu, incl.y, s);
        if (lane >= s) {
          incl.x += ua;
          incl.y += uq;
        }
      }
      if (lane == 31) sh.group[warp] = incl;
    }
    __syncthreads();
    int2 total = make_int2(0, 0), before = total;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      if (i == warp) before = total;
      total.x += sh.group[i].x;
      total.y += sh.group[i].y;
    }
    if (warp < kQuads)
      sh.warp[warp * kSelWarps + lane] = make_int2(
          before.x + incl.x - x.x, before.y + incl.y - x.y);
    __syncthreads();
    return total;
  };
  int2 total = make_int2(0, 0);
  for (int t = 0; t < turns; ++t) {
    if (turns > 1) load(a0 + t * kTurn);
    const int2 n = count(a0 + t * kTurn);
    total.x += n.x;
    total.y += n.y;
  }
  int above = 0, equal = 0;  // kept, equal ones before this turn's places
  if (ranks > 1) {
    if (threadIdx.x == 0) sh.count = total;
    cluster_barrier();
    for (int r = 0; r < rank; ++r) {
      above += static_cast<int>(ld_peer(&sh.count.x, r));
      equal += static_cast<int>(ld_peer(&sh.count.y, r));
    }
    cluster_arrive();  // awaited at the end: peers' reads
  }
  for (int t = 0; t < turns; ++t) {
    const int at = a0 + t * kTurn;
    int2 n = total;
    if (turns > 1) {
      load(at);
      n = count(at);
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const unsigned f = flags(at, i);
      const int2 pre = sh.warp[i * kSelWarps + warp];
      int a = above + pre.x + static_cast<int>(lower[i] & 0xffffu);
      int q = equal + pre.y + static_cast<int>(lower[i] >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_eq = (f >> (4 + e)) & 1u;
        if (((f >> e) & 1u) || (is_eq && q < left))
          idx[a + min(q, left)] =
              at + 4 * (i * kSelThreads + threadIdx.x) + e;
        a += (f >> e) & 1u;
        q += is_eq;
      }
    }
    above += n.x;
    equal += n.y;
    if (turns > 1) __syncthreads();  // the counts have been read
  }
  if (ranks > 1) cluster_wait();
}

constexpr int kMoveThreads = 512;  // most; two chunks of 16 codes a thread
constexpr int kCluster = 8;  // CTAs per unit in place

// Largest magnitude of 16 codes (NaN codes do not count).
__device__ __forceinline__ float codes_amax(uint4 c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t m = 0u;  // two halves
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t lo, hi;
    e4m3x4_to_half2(w[e] & 0x7f7f7f7fu, lo, hi);
    asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(lo));
    asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(hi));
  }
  const float2 f = unpack2<false>(m);
  return fmaxf(f.x, f.y);
}

// Four halves to four E4M3 codes, round to nearest even, saturating.
__device__ __forceinline__ uint32_t half2x2_to_e4m3(uint32_t lo, uint32_t hi) {
  uint32_t d;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(d)
      : "r"(lo), "r"(hi));
  return d;
}

// Key of a magnitude for the comparison of magnitudes and for a scale: its
// bits as an fp32 number, and past fp32's range (a code of 448 under a scale of
// 2^127 is 2^136) what they would be with another exponent bit.
__device__ __forceinline__ uint32_t magnitude_key(float code, float factor) {
  const uint32_t key = __float_as_uint(code * factor);
  return key < 0x7f800000u
             ? key
             : __float_as_uint(code * (factor * 0x1p-16f)) + (16u << 23);
}

// Its tight scale's exponent (cf. tight_exponent), fp32's largest at most: a
// scale between 2^127 and 2^128 may have made numbers past 448 * 2^127, which
// become 448.
__device__ __forceinline__ int tight_exponent_of_key(uint32_t key) {
  const int e = static_cast<int>(key >> 23) - 127 - 8 +
                ((key & 0x7fffff) > 0x600000);
  return min(max(e, -126), 127);
}

// The codes of K or V of one head: destination blocks rank, rank + ranks, ...
template <int D, bool kInPlace>
__device__ __forceinline__ void move_codes(const EvictParams& p, int kv,
                                           int bh, int rank, int ranks,
                                           int len, int n_kept) {
  constexpr int kPerRow = D / 16;                       // 16-byte chunks
  constexpr int kMax = 2;
  __shared__ uint32_t red[kMoveThreads / 32];
  const int threads = blockDim.x;  // of a block's chunks, half as many
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
  const int rounds = (blocks + ranks - 1) / ranks;
  for (int rd = 0; rd < rounds; ++rd) {
    const int nb = rd * ranks + rank;
    if (!kInPlace && nb >= blocks) break;
    const int t0 = nb << p.block_shift;
    uint4 held[kMax];
    float factor[kMax];
    uint32_t largest = 0u;
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int ch = threadIdx.x + i * threads;
      const int tok = t0 + ch / kPerRow;
      held[i] = make_uint4(0u, 0u, 0u, 0u);
      factor[i] = 0.f;
      if (tok < n_kept) {
        const int from = whole ? tok : idx[tok];
        held[i] = *reinterpret_cast<const uint4*>(
            src + static_cast<long long>(from) * D + (ch % kPerRow) * 16);
        factor[i] = src_scale[from >> p.block_shift];
      }
    }
#pragma unroll
    for (int i = 0; i < kMax; ++i)
      largest = max(largest, magnitude_key(codes_amax(held[i]), factor[i]));
    largest = __reduce_max_sync(0xffffffffu, largest);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = largest;
    float first = 0.f;  // the block's scale, where nothing leaves
    if (whole && threadIdx.x == 0 && nb < blocks) first = src_scale[nb];
    if constexpr (kInPlace) {
      // Every CTA of the cluster has read what this round overwrites.
      cluster_barrier();
    } else {
      __syncthreads();
    }
    for (int i = 0; i < threads / 32; ++i) largest = max(largest, red[i]);
    const float now = exp2_int(tight_exponent_of_key(largest));
    const float inv = reciprocal(now);
    if (threadIdx.x == 0 && nb < blocks) dst_scale[nb] = whole ? first : now;
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int ch = threadIdx.x + i * threads;
      const int tok = t0 + ch / kPerRow;
      if (tok >= n_kept) continue;
      uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
      const float ratio = factor[i] * inv;
      if (whole || ratio == 1.f) {
        // As it is.
      } else if ((__float_as_int(ratio) & 0x7fffff) == 0 && ratio > 1e-30f &&
                 ratio <= 32768.f) {
        // A shift of the exponent, in fp16: exact where a code above zero
        // can result (its last bit is 2^-24 or more then).
        const uint32_t r2 = ptx::pack2<false>(ratio, ratio);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t lo, hi;
          e4m3x4_to_half2(w[e], lo, hi);
          w[e] = half2x2_to_e4m3(hmul2(lo, r2), hmul2(hi, r2));
        }
      } else {  // a scale of other origin, or out of fp16's range
        // (Past 2^18 only for zeros, which stay zeros.)
        const float r = fminf(ratio, 0x1p100f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f[4];
          e4m3x4_to_float(w[e], f);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] *= r;
          w[e] = ptx::pack4_e4m3(f[0], f[1], f[2], f[3]);
        }
      }
      *reinterpret_cast<uint4*>(dst + static_cast<long long>(tok) * D +
                                (ch % kPerRow) * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();  // red is free again
  }
}

template <bool kInPlace>
__device__ __forceinline__ void move_weights(const EvictParams& p, int bh,
                                             int rank, int ranks,
                                             int n_kept) {
  const int* idx = p.indices + static_cast<long long>(bh) * p.keep;
  const float* src = p.weights + static_cast<long long>(bh) * p.src_capacity;
  float* dst = p.dst_weights + static_cast<long long>(bh) * p.dst_capacity;
  const int threads = blockDim.x;
  const int per = 4 * threads;  // tokens a CTA moves per round
  const int step = per * ranks;
  const int rounds = round_count(n_kept, step);
  for (int rd = 0; rd < rounds; ++rd) {
    const int t0 = rd * step + rank * per + threadIdx.x;
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t0 + i * threads;
      w[i] = tok < n_kept ? src[idx[tok]] : 0.f;
    }
    if constexpr (kInPlace) cluster_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t0 + i * threads;
      if (tok < n_kept) dst[tok] = w[i];
    }
  }
  // Every read of the sources is behind the last round's barrier.
  for (long long tok = cleared_place(n_kept, rank, threads, threadIdx.x);
       tok < p.dst_capacity; tok += ranks * threads)
    dst[tok] = 0.f;
}

template <int D, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads)
    kv8_move_kernel(const EvictParams p, int ranks, int weight_ranks) {
  start_after_previous();
  // K and V of every head, `ranks` CTAs each, then its weights.
  const int heads = p.B * p.Hkv;
  int x = blockIdx.x;
  const bool codes = x < 2 * heads * ranks;
  if (!codes) {
    x -= 2 * heads * ranks;
    ranks = weight_ranks;
  }
  const int unit = x / ranks, rank = x - unit * ranks;
  const int bh = codes ? unit / 2 : unit;
  const int b = bh / p.Hkv;
  const int len = clamp_len(p.src_lens[b], p.src_capacity, p.status);
  const int n_kept = min(len, p.keep);
  if (codes) {
    if (kInPlace && len <= p.keep) return;  // stays as it is
    move_codes<D, kInPlace>(p, unit % 2, bh, rank, ranks, len, n_kept);
  } else {
    move_weights<kInPlace>(p, bh, rank, ranks, n_kept);
    if (bh % p.Hkv == 0 && rank == 0 && threadIdx.x == 0)
      p.dst_lens[b] = n_kept;
  }
}

template <int D>
cudaError_t launch_move(const EvictParams& p, cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  const int threads = (D / 16 << p.block_shift) / 2;  // 32 to 512
  if (p.in_place)
    return launch_cluster(kv8_move_kernel<D, true>, heads * 3 * kCluster,
                          threads, 0, kCluster, stream, p, kCluster, kCluster);
  const int blocks = ((p.keep - 1) >> p.block_shift) + 1;
  const int weight_ranks = (p.dst_capacity - 1) / (4 * threads) + 1;
  return launch_cluster(kv8_move_kernel<D, false>,
                        heads * (2 * blocks + weight_ranks), threads, 0, 1,
                        stream, p, blocks, weight_ranks);
}

}  // namespace

cudaError_t launch_evict(int D, const EvictParams& p, cudaStream_t stream) {
  // CTAs per head: parts of up to 4096 tokens (four keys a thread), eight at
  // most; then 16 keys a thread.
  int ranks = 1;
  while (ranks < kMaxCluster && p.src_capacity > ranks * 4 * kSelThreads)
    ranks *= 2;
  const long long grid = static_cast<long long>(p.B) * p.Hkv * ranks;
  const cudaError_t err =
      p.src_capacity <= ranks * 4 * kSelThreads
          ? launch_cluster(kv8_select_kernel<1>, grid, kSelThreads, 0, ranks,
                           stream, p, ranks)
          : launch_cluster(kv8_select_kernel<kQuadsAt>, grid, kSelThreads, 0,
                           ranks, stream, p, ranks);
  if (err != cudaSuccess) return err;
  return D == 64 ? launch_move<64>(p, stream) : launch_move<128>(p, stream);
}

}  // namespace kv8
}  // namespace attn
