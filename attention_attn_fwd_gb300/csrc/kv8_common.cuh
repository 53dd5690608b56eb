// Parameters and arithmetic shared by the kernels of the 8-bit KV cache:
// E4M3 codes [B, Hkv, capacity, D] with one fp32 scale per block of tokens
// and head.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_host.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace kv8 {

constexpr float kE4m3Max = 448.f;

// A length read from device memory, brought into [0, most]; a value outside
// sets the status word's length bit.
__device__ __forceinline__ int clamp_len(int n, int most,
                                         unsigned int* status) {
  if (n < 0 || n > most) {
    atomicOr(status, kStatusBadLength);
    return n < 0 ? 0 : most;
  }
  return n;
}

// Exponent of the smallest power of two s with amax <= 448 s, 2^-126 at
// least: 448 = 1.75 * 2^8, so it is amax's exponent - 8, one more when its
// mantissa exceeds 1.75.  Exact for every finite amax >= 0.
__device__ __forceinline__ int tight_exponent(float amax) {
  const int bits = __float_as_int(amax);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return max(e, -126);
}

__device__ __forceinline__ float exp2_int(int e) {  // -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}

__device__ __forceinline__ bool is_power_of_two(float s) {  // s normal
  return (__float_as_int(s) & 0x7fffff) == 0;
}

// 1 / s of a normal power of two, exact (2^127's is the subnormal 2^-127).
__device__ __forceinline__ float reciprocal(float s) {
  return __int_as_float(max((254 << 23) - __float_as_int(s), 1 << 22));
}

// Magnitude that counts for a scale: finite values only.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;  // inf and NaN compare false
}

// Two 16-bit elements of a word as floats.
template <bool kBF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kBF16) {
    return make_float2(__uint_as_float(w << 16),
                       __uint_as_float(w & 0xffff0000u));
  } else {
    __half2 h;
    *reinterpret_cast<uint32_t*>(&h) = w;
    return __half22float2(h);
  }
}

// Two E4M3 codes (low byte first) as a packed fp16 pair: exact, E4M3's
// values (2^-9 steps up to 448, NaN) are all fp16 values.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}

// The four halves of a word of four codes.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t codes, uint32_t& lo,
                                                uint32_t& hi) {
  lo = e4m3x2_to_half2(static_cast<uint16_t>(codes & 0xffffu));
  hi = e4m3x2_to_half2(static_cast<uint16_t>(codes >> 16));
}

__device__ __forceinline__ void e4m3x4_to_float(uint32_t codes, float* x) {
  uint32_t lo, hi;
  e4m3x4_to_half2(codes, lo, hi);
  const float2 a = unpack2<false>(lo), b = unpack2<false>(hi);
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Programmatic dependent launches: every kernel of the 8-bit cache may be
// scheduled before the one ahead of it on the stream has ended, so that its
// launch overlaps that one's tail.  Each begins with start_after_previous():
// it waits for the kernel ahead (whatever that is) to end and be visible,
// and only then lets the next one be scheduled -- so a kernel that reads
// memory before its own wait can rely on everything but the kernel directly
// ahead, and every thread block waits, also one without work (else a kernel
// of idle blocks could end before the one ahead of it).
__device__ __forceinline__ void start_after_previous() {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
}

// Launch with clusters of `cluster` CTAs (1: none).
template <class Kernel, class... Args>
cudaError_t launch_cluster(Kernel kernel, long long grid, int threads,
                           int smem, int cluster, cudaStream_t stream,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class Kernel, class... Args>
cudaError_t launch_pdl(Kernel kernel, long long grid, int threads, int smem,
                       cudaStream_t stream, Args... args) {
  return launch_cluster(kernel, grid, threads, smem, 1, stream, args...);
}

// (The cluster's barrier wants whole warps, as loops may have left them apart.)
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  ptx::cluster_arrive_release();
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  ptx::cluster_wait_acquire();
}
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
}

// Few-row forward: warps of a CTA, and CTAs an SM holds at 8 and 16 query
// rows each.
constexpr int kDecodeWarps = 4;
__host__ __device__ constexpr int decode_ctas(int D, int rows) {
  return rows <= 8 ? (D == 128 ? 3 : 4) : 2;
}

struct AppendParams {
  uint8_t* code[2];       // K, V
  float* scale[2];
  const void* x[2];       // new K, V [B, Hkv, Sq, D]
  const int* lens;
  const int* new_lens;    // or nullptr
  int Hkv, Sq, capacity, nblk;
  int units_per_seq;      // blocks of a head one call may touch
  unsigned int* status;
};

struct FwdParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int* lens;
  const int* new_lens;    // or nullptr
  const void* q;
  void* o;
  float* lse;             // or nullptr
  float* weights;         // or nullptr
  int B, Hq, Hkv, Sq, capacity, nblk, block_shift;
  int group;              // query heads per K/V head
  int row_blocks;         // many rows: units of 256 per (batch, K/V head)
  int causal;
  int whole;              // many rows: units are not split
  int ranks;              // few rows: CTAs of a cluster that takes a segment
  float scale_log2;       // scale * log2(e)
  // Workspace: rows of the parts of a split segment or unit, each the average
  // that it is, and their LSEs in log2 units (-inf: sees nothing; few rows) or
  // (max, sum) (many: the logarithm is cheaper in the merge there); few rows:
  // the scores of every key; many rows: the unit that goes on behind each CTA,
  // and the rows' LSEs in log2 units.
  float* part_o;          // [slots, rows, D]
  float* part_lse2;       // [slots, rows]
  float2* part_ml;        // [slots, rows]
  float* scores;          // [B * Hkv, capacity, 1 << score_shift]
  int4* split;            // [grid]: b, h, unit, number of CTAs (0: none)
  float* lse2;            // [B * Hkv, row_blocks * 256]
  int grid;               // CTAs of the forward launch
  int score_shift;        // few rows: log2 of the scores' rows per key
  unsigned long long timeout_ns;  // limit of a pipeline wait
  unsigned int* status;
};

// ------------------------------------------------ shared by the forwards
constexpr float kNone = -3.402823466e38f;  // running maximum of no score

__device__ __forceinline__ int seq_len(const FwdParams& p, int b) {
  return clamp_len(p.lens[b], p.capacity, p.status);
}
__device__ __forceinline__ int seq_new(const FwdParams& p, int b) {
  return p.new_lens == nullptr ? p.Sq
                               : clamp_len(p.new_lens[b], p.Sq, p.status);
}
// Visible tokens of row r (token-major: row r = token r / group, head
// r % group) of a sequence.
__device__ __forceinline__ int row_end(const FwdParams& p, int len, int n_new,
                                       int r) {
  if (!p.causal) return len;
  return min(len, max(0, len - n_new + r / p.group + 1));
}
// The list of tiles: sequence b contributes Hkv segments of
// ceil(lens[b] / kKeys) tiles, and kOver empty places before each, which stand
// for the time that a segment takes besides its tiles.  (Counts fit 32 bits:
// a tile of one segment holds 4 KB of codes.)
template <int kKeys, int kOver>
__device__ __forceinline__ int places(int len) {
  return len > 0 ? (len + kKeys - 1) / kKeys + kOver : 0;
}

// Places before sequence `seq` and of all sequences, for every lane of the
// calling warp.
template <int kKeys, int kOver>
__device__ __forceinline__ int list_tiles(const FwdParams& p, int seq,
                                          int lane, int* before) {
  int t = 0, pre = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int n = places<kKeys, kOver>(seq_len(p, b));
    t += n;
    if (b < seq) pre += n;
  }
#pragma unroll
  for (int s = 16; s > 0; s /= 2) {
    t += __shfl_xor_sync(0xffffffffu, t, s);
    pre += __shfl_xor_sync(0xffffffffu, pre, s);
  }
  *before = pre * p.Hkv;
  return t * p.Hkv;
}

// The cut: CTA c of n takes q places, the first `rest` CTAs one more.
struct Cut {
  int n, q, rest;
  __device__ __forceinline__ int first(int c) const {
    return c * q + min(c, rest);
  }
  __device__ __forceinline__ int owner(int x) const {
    const int fat = rest * (q + 1);
    return x < fat ? x / (q + 1) : rest + (x - fat) / q;
  }
};
// kLeast places a CTA are the finest cut.
template <int kLeast>
__device__ __forceinline__ Cut make_cut(const FwdParams& p, int total) {
  Cut c;
  c.n = max(1, min(p.grid, (total + kLeast - 1) / kLeast));
  c.q = total / c.n;
  c.rest = total - c.q * c.n;
  return c;
}

// A segment of the list as a CTA walks its share: its tiles lie at [pos, end)
// counted from the share's start (pos < 0: it began earlier).
struct Segment {
  int pos, end;
  int b, h;  // sequence, K/V head
  int len, tiles;
};

// CTA's share: its number of places (0: none) and first segment.
template <int kKeys, int kOver, int kLeast>
__device__ __forceinline__ int take_share(const FwdParams& p, int cta,
                                          int lane, Segment* s) {
  int first = 0, count = 0, base = 0;
  if (p.B > 32) {
    const int total = list_tiles<kKeys, kOver>(p, 0, lane, &base);
    const Cut cut = make_cut<kLeast>(p, total);
    first = cut.first(cta);
    count = cta < cut.n ? cut.first(cta + 1) - first : 0;
    if (count == 0) return 0;
  }
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int len = b < p.B ? seq_len(p, b) : 0;
    const int t = places<kKeys, kOver>(len) * p.Hkv;
    int incl = t;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, incl, i);
      if (lane >= i) incl += up;
    }
    const int sum = __shfl_sync(0xffffffffu, incl, 31);
    if (p.B <= 32) {  // one load per lane tells all
      const Cut cut = make_cut<kLeast>(p, sum);
      first = cut.first(cta);
      count = cta < cut.n ? cut.first(cta + 1) - first : 0;
      if (count == 0) return 0;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > first);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      const int before = base + __shfl_sync(0xffffffffu, incl - t, l);
      s->b = b0 + l;
      s->len = __shfl_sync(0xffffffffu, len, l);
      s->tiles = (s->len + kKeys - 1) / kKeys;
      s->h = (first - before) / (s->tiles + kOver);
      s->pos = kOver - ((first - before) - s->h * (s->tiles + kOver));
      s->end = s->pos + s->tiles;
      return count;
    }
    base += sum;
  }
  return 0;
}

template <int kKeys, int kOver>
__device__ __forceinline__ void next_segment(const FwdParams& p, Segment& c) {
  c.pos = c.end + kOver;
  if (++c.h == p.Hkv) {
    c.h = 0;
    do {  // some later sequence has tokens: the share is not at its end
      ++c.b;
      c.len = seq_len(p, c.b);
    } while (c.len == 0);
    c.tiles = (c.len + kKeys - 1) / kKeys;
  }
  c.end = c.pos + c.tiles;
}

// Exponent of the power of two that brings a query row's largest element to
// [2^13, 2^14) (rows of zeros or of the smallest numbers: as far as it goes).
__device__ __forceinline__ int row_shift(float amax) {
  const int e = (__float_as_int(amax) >> 23) - 127;
  return max(-114, min(13 - e, 126));
}

// C (16 x 8, fp32) += A (16 x 16) B (16 x 8) in fp16.
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1,
                                        uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct EvictParams {
  const uint8_t* src_code[2];
  const float* src_scale[2];
  uint8_t* dst_code[2];
  float* dst_scale[2];
  const int* src_lens;
  int* dst_lens;
  const float* weights;
  float* dst_weights;
  int* indices;           // [B, Hkv, keep]
  int B, Hkv, src_capacity, dst_capacity, src_nblk, dst_nblk, block_shift;
  int keep, recent;
  int in_place;
  unsigned int* status;
};

cudaError_t launch_append(int D, int block, bool bf16, const AppendParams& p,
                          int B, cudaStream_t stream);
cudaError_t launch_decode(int D, bool bf16, int rows, const FwdParams& p,
                          cudaStream_t stream);
cudaError_t launch_prefill(int D, bool bf16, const FwdParams& p,
                           cudaStream_t stream);
cudaError_t launch_weights(int D, bool bf16, int lse2_rows,
                           const FwdParams& p, cudaStream_t stream);
cudaError_t launch_evict(int D, const EvictParams& p, cudaStream_t stream);

}  // namespace kv8
}  // namespace attn
