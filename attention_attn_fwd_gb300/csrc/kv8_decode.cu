// Attention of a few query rows per K/V head over the 8-bit cache, and the
// merge of its partial results.
//
// Mathematics: flash-decoding.  The keys of all (batch, K/V head) segments
// form one list of tiles (2 KB of K codes each), cut into equal consecutive
// shares, one per CTA; a CTA's warps take its tiles in turn, each with its
// own running maximum m, sum l and accumulator O, which meet in shared memory
// at the end of a segment.  A partial result goes to workspace slot
// (CTA + segment): both only grow along the list, so no two share one.  The
// merge kernel joins a segment's partials by their maxima.  Lengths come from
// device memory, so the cut follows them without the host's knowing: ragged
// batches are balanced to a tile.  Over short caches a cluster of 1 to 8 CTAs
// takes each segment instead and writes the results itself (cluster_ranks
// below): its CTAs' sums meet in distributed shared memory.
//
// Products: S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16 in fp16,
// 16 keys (or 16 of D) by 8 query rows: with 8 or 16 rows a 128-row
// tcgen05 tile would be nearly empty, and the codes' bytes bound the kernel.
// E4M3 codes are fp16 values, so K and V convert exactly; Q is multiplied by
// a power of two per row that brings its largest element to [2^13, 2^14),
// which makes bf16 -> fp16 exact down to 2^-37 of the row's largest element
// (below fp32 accumulation's own rounding).  Block scales multiply scores and
// weights in fp32.  P is rounded to fp16 (2^-11 relative, the rounding of an
// fp16 output itself and an eighth of a bf16 one's), shifted by 2^7 so that
// weights down to 2^-21 of the row's largest stay normal numbers.  V's scales
// are kept out of it, for each factor of two between two blocks would cost P a
// bit of its range: O is held in units of a power of two, that of the keys at
// hand, and moved to another, in fp32, when that changes.  The row sums take P
// unrounded.
//
// Codes reach shared memory by 16-byte asynchronous copies, a ring of tiles
// per warp that runs ahead across segments (128 to 144 KB in flight per SM;
// with the codes loaded straight to registers one tile ahead, 64 KB, the
// kernel ran at 2.8 TB/s on 8 x 4096 tokens and 4.4 TB/s on 131072, without
// its merge).  Fragments are read
// 16 bytes at a time: the d index of both products may be permuted freely, so
// lane c of a quad owns bytes 16c.. of a 64-byte half row of K and lane group
// g8 owns bytes (D/8) g8.. of four V rows; 16-byte chunks of a row are stored
// XORed by its row so that those reads do not share banks.  No transposes but
// a byte permute and one movmatrix per 8 x 8 weights.
//
// Measured, cut and merged: 8 x 4096 tokens, 8 heads of 4 rows, D = 128, with
// accumulated weights 23.8 us (69 MB); 131072 tokens, 4 heads of 8 rows 32.5
// us (134 MB, 4.1 TB/s).  With the products taken out the first two thirds of
// that stay (15.8 and 25.0 us, the loads), the products add about 4 us and the
// merge's launch behind the last CTA 4 to 7: on short caches latency bounds
// the pair, on long ones the codes' bytes.
#include "kv8_common.cuh"

namespace attn {
namespace kv8 {
namespace {

// A segment takes a CTA time besides its tiles (2 us: query rows and scales
// fetched, partials joined and stored).  Without empty places for it in the
// cut, heads of short sequences that share a CTA held the whole launch up: 16
// sequences of 0 .. 2048 tokens, 16 heads, 20-44 us by the draw; with 4 places
// 20-22, with 12 19-20 (8 x 4096 tokens 25.0 -> 23.5, 16 or 24 about the same).
constexpr int kOver = 12;
constexpr float kTau = 8.f;        // lazy rescale threshold (log2 units)
constexpr float kPScale = 128.f;   // 2^7: P <= 2^(8 + 7) < 65504
// Exponents of O's unit: the least one, and how far below that of the largest
// V scale met it may lie (O stays below 2^128: 2^64 times 448, 2^15 of P and up
// to 2^31 keys).
constexpr int kMinUnit = -125;
constexpr int kUnitDepth = 64;

// Keys of a list tile: 2 KB of K codes.
template <int D>
__host__ __device__ constexpr int tile_keys() {
  return 2048 / D;
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

// One tile of a warp's ring: 2 KB of K codes, then 2 KB of V codes.  Chunk j
// (16 bytes) of row r lies at chunk j ^ swizzle(r): the rows read together by
// the 8 lanes of a phase (K: rows 2q, 2q + 1; V: rows of one parity) then lie
// in different banks (64-byte V rows: two lanes share one).
template <int D>
__device__ __forceinline__ int k_swizzle(int r) {
  return D == 128 ? (r & 1) << 2 : 0;
}
template <int D>
__device__ __forceinline__ int v_swizzle(int r) {
  return D == 128 ? ((r >> 1) & 3) << 1 : ((r >> 1) & 1) << 1;
}

// A warp's loads: they run ahead of its products, across segments.  Lane i
// copies chunks i, i + 32, i + 64 and i + 96 of a tile.
template <int D>
struct Loader {
  static constexpr int kKeys = tile_keys<D>();
  static constexpr int kPerRow = D / 16;
  static constexpr int kRowStep = 32 / kPerRow;  // rows between the chunks
  Segment seg;
  int pos;                 // next tile, counted from the share's start
  const uint8_t* k;        // this lane's first chunk of tile 0 of the segment
  const uint8_t* v;
  uint32_t dst_k, dst_v0, dst_v1;  // its places in a ring slot

  __device__ __forceinline__ void set_segment(const FwdParams& p, int lane) {
    const long long at =
        (static_cast<long long>(seg.b) * p.Hkv + seg.h) * p.capacity * D +
        16 * lane;
    k = p.k + at;
    v = p.v + at;
  }
  __device__ __forceinline__ void init(const FwdParams& p, const Segment& s,
                                       int warp, int lane, uint32_t ring) {
    seg = s;
    pos = warp;
    const int r = lane / kPerRow, j = lane % kPerRow;
    dst_k = ring + r * D + ((j ^ k_swizzle<D>(r)) << 4);
    dst_v0 = ring + 2048 + r * D + ((j ^ v_swizzle<D>(r)) << 4);
    dst_v1 = ring + 2048 + r * D + ((j ^ v_swizzle<D>(r + kRowStep)) << 4);
    set_segment(p, lane);
  }
  template <int kStep>
  __device__ __forceinline__ void next(const FwdParams& p, int count,
                                       int stage, int lane) {
    bool moved = false;
    while (pos < count) {
      if (pos >= seg.end) {
        next_segment<kKeys, kOver>(p, seg);
        moved = true;
      } else if (pos < seg.pos) {
        pos += kStep;
      } else {
        break;
      }
    }
    if (pos < count) {
      if (moved) set_segment(p, lane);
      const int t = pos - seg.pos;
      const long long off = static_cast<long long>(t) * 2048;
      const uint32_t to = stage * 4096;
      if ((t + 1) * kKeys <= seg.len) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ptx::cp_async16(dst_k + to + 512 * i, k + off + 512 * i);
          ptx::cp_async16(((i & 1) ? dst_v1 : dst_v0) + to + 512 * i,
                          v + off + 512 * i);
        }
      } else {  // rows past the length become zeros
        const int left = seg.len - t * kKeys - lane / kPerRow;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = i * kRowStep < left;
          const long long at = in ? off + 512 * i : 0;
          ptx::cp_async16_or_zero(dst_k + to + 512 * i, k + at, in);
          ptx::cp_async16_or_zero(
              ((i & 1) ? dst_v1 : dst_v0) + to + 512 * i, v + at, in);
        }
      }
      pos += kStep;
    }
    ptx::cp_async_commit();
  }
};

// NT: 8-row groups of query rows a CTA holds (8 or 16 rows of a K/V head).
// CTAs of four warps, as many as registers and shared memory allow: one CTA's
// start, end of a segment or tail runs under the others' loads (four CTAs an
// SM against one of 16 warps: 29.0 -> 27 us on 8 x 4096 tokens, 57 -> 32 on
// 256 segments of about 1000).
template <int D, int NT>
struct Config {
  static constexpr int kRows = 8 * NT;
  static constexpr int kThreads = 32 * kDecodeWarps;
  static constexpr int kCtas = decode_ctas(D, kRows);
  static constexpr int kStages = NT == 1 ? (D == 128 ? 3 : 2) : 4;
  static constexpr int kPitch = D + 4;  // floats: rows start 4 banks apart
  static constexpr int kRingBytes = kDecodeWarps * kStages * 4096;
  static constexpr int kBytes =
      kRingBytes + kDecodeWarps * kRows * (kPitch + 2) * 4 +
      (kRows + kDecodeWarps) * 4;
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory");
};

__device__ __forceinline__ long long out_row(const FwdParams& p, int b, int h,
                                             int r) {
  const int tok = r / p.group, hd = r - tok * p.group;
  return (static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq + tok;
}
// The LSE in log2 units of a row's maximum and sum, -inf for one that sees
// nothing.
__device__ __forceinline__ float lse2_of(float mx, float sum) {
  return sum == 0.f ? -INFINITY : mx + log2f(sum);
}

// The scores of one key that the forward left, rows beyond n_rows as hidden
// ones; and the weight they make under the rows' LSEs.
template <int kRows>
__device__ __forceinline__ void load_scores(const FwdParams& p, long long key,
                                            int n_rows, float4* x) {
  const float* at = p.scores + (key << p.score_shift);
#pragma unroll
  for (int k = 0; k < kRows / 4; ++k) {
    x[k] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (4 * k >= n_rows) continue;
    if (p.score_shift >= 2) {
      x[k] = *reinterpret_cast<const float4*>(at + 4 * k);
    } else {
      x[k].x = at[0];
      if (n_rows > 1) x[k].y = at[1];
    }
  }
}
template <int kRows>
__device__ __forceinline__ float weight_of(const float4* x, const float* lse2,
                                           int n_rows) {
  float add = 0.f;
#pragma unroll
  for (int k = 0; k < kRows / 4; ++k) {
    const float v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)  // hidden scores and padding rows: -inf
      if (4 * k + e < n_rows && v[e] != -INFINITY)
        add += ptx::ex2(v[e] - lse2[4 * k + e]);
  }
  return add;
}

constexpr int kMaxRanks = 8;

// kWhole: a CTA per segment, or a cluster of a few that divide its tiles
// evenly, which write the results themselves.
template <int D, int NT, bool kBF16, bool kWhole>
__global__ void __launch_bounds__(Config<D, NT>::kThreads, Config<D, NT>::kCtas)
    kv8_decode_kernel(const FwdParams p) {
  using C = Config<D, NT>;
  constexpr int kWarps = kDecodeWarps;
  constexpr int kRows = C::kRows;
  constexpr int kPitch = C::kPitch;
  constexpr int kStages = C::kStages;
  constexpr int kKeys = tile_keys<D>();
  constexpr int kSub = kKeys / 16;  // 16-key steps per tile
  constexpr int kKSteps = D / 16;
  constexpr int kMT = D / 16;       // m-tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  float* sm_o = reinterpret_cast<float*>(smem + C::kRingBytes);
  float* sm_m = sm_o + kWarps * kRows * kPitch;  // [kWarps][kRows]
  float* sm_l = sm_m + kWarps * kRows;
  float* sm_lse = sm_l + kWarps * kRows;  // kWhole: [kRows]
  int* sm_unit = reinterpret_cast<int*>(sm_lse + kRows);  // [kWarps]

  start_after_previous();

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g8 = lane / 4, c = lane % 4;
  const int cta = blockIdx.x;
  Segment seg;
  seg.pos = 0;
  int count;
  int rank = 0;
  if constexpr (kWhole) {
    const int bh = cta / p.ranks;
    rank = cta - bh * p.ranks;
    seg.b = bh / p.Hkv;
    seg.h = bh - seg.b * p.Hkv;
    seg.len = seq_len(p, seg.b);
    seg.tiles = (seg.len + kKeys - 1) / kKeys;
    seg.pos = -(seg.tiles * rank / p.ranks);
    seg.end = seg.tiles + seg.pos;
    count = seg.tiles * (rank + 1) / p.ranks + seg.pos;
  } else {
    count = take_share<kKeys, kOver, kDecodeWarps>(p, cta, lane, &seg);
    if (seg.pos >= count) return;  // (also: no share)
  }
  const uint32_t ring = ptx::smem_u32(smem) + warp * kStages * 4096;
  Loader<D> ld;
  ld.init(p, seg, warp, lane, ring);
#pragma unroll
  for (int i = 0; i < kStages; ++i)
    ld.template next<kWarps>(p, count, i, lane);

  int stage = 0;
  int pos = warp;  // this warp's next tile
  while (true) {
    const int seg_last = min(seg.end, count);  // end of the CTA's part
    const int b = seg.b, h = seg.h, len = seg.len;
    const int bh = b * p.Hkv + h;
    const int n_new = seq_new(p, b);
    const int n_rows = n_new * p.group;  // valid rows, kRows at most
    const int min_end = n_rows > 0 ? row_end(p, len, n_new, 0) : 0;
    const int max_end = n_rows > 0 ? len : 0;

    // This lane's two query rows per 8-row group (columns of S^T): how many
    // tokens they see, and the factor of their scores.
    int vis[NT][2];
    float mult[NT][2];
    uint32_t bq[NT][kKSteps][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g8;
      uint32_t raw[D / 64][8];
      float amax = 0.f;
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
        if (r < n_rows) {
          const int tok = r / p.group, hd = r % p.group;
          const uint16_t* q =
              static_cast<const uint16_t*>(p.q) +
              ((static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq +
               tok) * D + 64 * hf + 16 * c;
          w0 = __ldg(reinterpret_cast<const uint4*>(q));
          w1 = __ldg(reinterpret_cast<const uint4*>(q) + 1);
        }
        raw[hf][0] = w0.x; raw[hf][1] = w0.y; raw[hf][2] = w0.z; raw[hf][3] = w0.w;
        raw[hf][4] = w1.x; raw[hf][5] = w1.y; raw[hf][6] = w1.z; raw[hf][7] = w1.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = unpack2<kBF16>(raw[hf][i]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int up = row_shift(amax);
      const float f_up = exp2_int(up);
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = unpack2<kBF16>(raw[hf][2 * w + i]);
            bq[nt][4 * hf + w][i] = ptx::pack2<false>(f.x * f_up, f.y * f_up);
          }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 2 * c + e;  // row of the group this column is
        const int up_col = __shfl_sync(0xffffffffu, up, 4 * col);
        mult[nt][e] = p.scale_log2 * exp2_int(-up_col);
        const int rr = 8 * nt + col;
        vis[nt][e] = rr < n_rows ? row_end(p, len, n_new, rr) : len;
      }
    }

    const float* ksb = p.k_scale + static_cast<long long>(bh) * p.nblk;
    const float* vsb = p.v_scale + static_cast<long long>(bh) * p.nblk;

    float m[NT][2], l[NT][2], o[NT][kMT][4];
    // O is held in units of 2^unit (times 2^7): the least power of two that is
    // no less than the V scale of the keys before, vs_last, if kUnitDepth
    // allows; unit_most: of the largest one.
    int unit = kMinUnit, unit_most = kMinUnit;
    float vs_last = 0.f;
    float p_factor = 0.f;  // 2^7 vs_last / 2^unit, 2^7 at most
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    // Block scales of this warp's next 32 / kSub tiles, one per lane (lane
    // i: step i % kSub of tile i / kSub), fetched again when used up.
    float ks_all = 0.f, vs_all = 0.f;
    int held = 32 / kSub;  // tiles of the fetched ones that are used up
    while (pos < seg.pos) pos += kWarps;
    for (; pos < seg_last; pos += kWarps) {
      if (held == 32 / kSub) {
        const int key =
            (pos + (lane / kSub) * kWarps - seg.pos) * kKeys +
            16 * (lane % kSub);
        const bool in = key < len;
        ks_all = in ? __ldg(ksb + (key >> p.block_shift)) : 0.f;
        vs_all = in ? __ldg(vsb + (key >> p.block_shift)) : 0.f;
        held = 0;
      }
      ptx::cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t tile = ring + stage * 4096;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int key0 = (pos - seg.pos) * kKeys + 16 * u;
        const float ks =
            __shfl_sync(0xffffffffu, ks_all, held * kSub + u);
        const float vs =
            __shfl_sync(0xffffffffu, vs_all, held * kSub + u);
        if (key0 >= max_end) continue;  // no rows, or past the length
        // S^T of 16 keys, in two chains.
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          uint4 kr[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 16 * u + g8 + 8 * i;
            kr[i] = ptx::ld_shared_v4(
                tile + r * D + (((4 * hf + c) ^ k_swizzle<D>(r)) << 4));
          }
          const uint32_t k0[4] = {kr[0].x, kr[0].y, kr[0].z, kr[0].w};
          const uint32_t k1[4] = {kr[1].x, kr[1].y, kr[1].z, kr[1].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_half2(k0[w], a0, a2);
            e4m3x4_to_half2(k1[w], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16((w & 1) ? s2[nt] : s[nt], a0, a1, a2, a3,
                      bq[nt][4 * hf + w][0], bq[nt][4 * hf + w][1]);
          }
        }
        // Scores in log2 units; hidden ones are -inf.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[nt][e] = (s[nt][e] + s2[nt][e]) * (mult[nt][e & 1] * ks);
        if (key0 + 16 > min_end) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + g8 + 8 * (e >> 1) >= vis[nt][e & 1])
                s[nt][e] = -INFINITY;
        }
        if (p.scores != nullptr) {
          // [key][row], rows padded to a power of two.
          float* sc = p.scores + ((static_cast<long long>(bh) * p.capacity +
                                   key0 + g8) << p.score_shift);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = 8 * nt + 2 * c;
              if (key0 + g8 + 8 * i >= len || r >> p.score_shift) continue;
              float* at = sc + (8 * i << p.score_shift) + r;
              if (p.score_shift == 0)
                *at = s[nt][2 * i];
              else
                *reinterpret_cast<float2*>(at) =
                    make_float2(s[nt][2 * i], s[nt][2 * i + 1]);
            }
        }
        if (vs != vs_last) {
          vs_last = vs;
          const int bits = __float_as_int(vs), frac = bits & 0x7fffff;
          const int e = (bits >> 23) - 127;
          const int up = e + (frac != 0 ? 1 : 0);
          unit_most = max(unit_most, up);
          const int now = max(max(up, kMinUnit), unit_most - kUnitDepth);
          p_factor =
              __int_as_float(frac | (max(127 + 7 + e - now, 1) << 23));
          if (now != unit) {  // O to the unit of these keys
            const float f = exp2_int(max(unit - now, -126));
            unit = now;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nt][i][k] *= f;
          }
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            grow |= fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + kTau;
        // Lazy rescale: some row's maximum grew by more than 2^8.
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(s[nt][e], s[nt][e + 2]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float m_new = fmaxf(m[nt][e], mx);
              const float alpha = ptx::ex2(m[nt][e] - m_new);
              m[nt][e] = m_new;
              l[nt][e] *= alpha;
#pragma unroll
              for (int i = 0; i < kMT; ++i) {
                o[nt][i][e] *= alpha;
                o[nt][i][e + 2] *= alpha;
              }
            }
        }
        // P^T in fp16, times 2^7.
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // A hidden score is -inf, m never is: 0; NaN stays NaN.
            w[e] = ptx::ex2(s[nt][e] - m[nt][e & 1]);
            l[nt][e & 1] += w[e];
          }
          pb[nt][0] = ptx::movmatrix_trans(
              ptx::pack2<false>(w[0] * p_factor, w[1] * p_factor));
          pb[nt][1] = ptx::movmatrix_trans(
              ptx::pack2<false>(w[2] * p_factor, w[3] * p_factor));
        }
        // O^T += V^T P^T: V rows 2c, 2c + 1, 2c + 8, 2c + 9 of the step.
        constexpr int kVWords = D / 32;
        uint32_t v[4][kVWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * u + 2 * c + (i & 1) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 x = ptx::ld_shared_v4(
                tile + 2048 + r * D + ((g8 ^ v_swizzle<D>(r)) << 4));
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
          } else {
            const uint2 x = ld_shared_v2(
                tile + 2048 + r * D +
                (((g8 >> 1) ^ v_swizzle<D>(r)) << 4) + 8 * (g8 & 1));
            v[i][0] = x.x;
            v[i][1] = x.y;
          }
        }
#pragma unroll
        for (int w = 0; w < kVWords; ++w) {
          uint32_t a[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t lo =
                __byte_perm(v[2 * i][w], v[2 * i + 1][w], 0x5140);
            const uint32_t hi =
                __byte_perm(v[2 * i][w], v[2 * i + 1][w], 0x7362);
            e4m3x4_to_half2(lo, a[0][2 * i], a[0][2 * i + 1]);
            e4m3x4_to_half2(hi, a[1][2 * i], a[1][2 * i + 1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(o[nt][2 * w], a[0][0], a[0][1], a[0][2], a[0][3],
                    pb[nt][0], pb[nt][1]);
            mma_f16(o[nt][2 * w + 1], a[1][0], a[1][1], a[1][2], a[1][3],
                    pb[nt][0], pb[nt][1]);
          }
        }
      }
      __syncwarp();  // the tile has been read
      ld.template next<kWarps>(p, count, stage, lane);
      ++held;
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // The warps' results meet: maxima and units, then O and l under the common
    // ones.  O leaves as the average that it is: a sum of many V could pass
    // fp32's largest.
    __syncthreads();  // the previous segment's sums have been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[nt][e] = x;
        if (g8 == 0) sm_m[warp * kRows + 8 * nt + 2 * c + e] = m[nt][e];
      }
    if (lane == 0) sm_unit[warp] = unit;
    __syncthreads();
    int unit_cta = sm_unit[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) unit_cta = max(unit_cta, sm_unit[w]);
    const float f_unit = exp2_int(max(unit - unit_cta, -126));
    // (A unit of 2^128 has scales between that and 2^127.)
    const float v_unit = exp2_int(unit_cta - 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * c + e;
        float mx = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          mx = fmaxf(mx, sm_m[w * kRows + r]);
        const float f = ptx::ex2(m[nt][e] - mx);
        const float fo = f * f_unit;
        if (g8 == 0) sm_l[warp * kRows + r] = l[nt][e] * f;
        float* dst = sm_o + (warp * kRows + r) * kPitch + (D / 8) * g8;
#pragma unroll
        for (int i = 0; i < kMT; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(o[nt][i][e] * fo, o[nt][i][e + 2] * fo,
                          o[nt][i + 1][e] * fo, o[nt][i + 1][e + 2] * fo);
      }
    __syncthreads();
    // Row r's sum over the warps, and what they have of its O.
    auto cta_sum = [&](int r) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += sm_l[w * kRows + r];
      return sum;
    };
    auto cta_lse2 = [&](int r) {
      float mx = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w * kRows + r]);
      return lse2_of(mx, cta_sum(r));
    };
    auto cta_o = [&](int r, int d4) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(
            sm_o + (w * kRows + r) * kPitch + 4 * d4);
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      const float sum = cta_sum(r);
      // A row that sees nothing: 0, whatever its accumulators hold (NaN codes
      // of V reach them).
      if (sum == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
      const float inv = ptx::rcp(sum) * (2.f / kPScale);
      return make_float4(acc.x * inv * v_unit, acc.y * inv * v_unit,
                         acc.z * inv * v_unit, acc.w * inv * v_unit);
    };
    if constexpr (kWhole) {
      // This CTA's rows, then those of the cluster's.
      float4* own_o = reinterpret_cast<float4*>(smem);  // (the ring is free)
      float* own_lse2 = reinterpret_cast<float*>(smem + kRows * D * 4);
      for (int i = threadIdx.x; i < n_rows * (D / 4); i += C::kThreads)
        own_o[i] = cta_o(i / (D / 4), i % (D / 4));
      if (threadIdx.x < n_rows) own_lse2[threadIdx.x] = cta_lse2(threadIdx.x);
      if (p.ranks > 1)
        cluster_barrier();
      else
        __syncthreads();
      const uint32_t at_o = ptx::smem_u32(own_o);
      const uint32_t at_lse2 = ptx::smem_u32(own_lse2);
      // Row r's LSE, and the CTAs' shares of its sum.
      auto total = [&](int r, float* f) -> float {
        if (p.ranks == 1) return own_lse2[r];
        float x[kMaxRanks];
        float mx = kNone, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) {
          x[k] = -INFINITY;
          if (k < p.ranks)
            x[k] = ptx::ld_shared_cluster_f32(
                ptx::mapa_shared(at_lse2 + 4 * r, k));
        }
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) mx = fmaxf(mx, x[k]);
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) {
          f[k] = ptx::ex2(x[k] - mx);
          sum += f[k];
        }
        const float inv = sum == 0.f ? 0.f : ptx::rcp(sum);
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) f[k] *= inv;
        return lse2_of(mx, sum);
      };
      for (int i = rank * C::kThreads + threadIdx.x; i < n_rows * (D / 4);
           i += p.ranks * C::kThreads) {
        const int r = i / (D / 4), d4 = i % (D / 4);
        float f[kMaxRanks];
        const float lse2 = total(r, f);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.ranks == 1) {
          acc = own_o[i];
        } else {
#pragma unroll
          for (int k = 0; k < kMaxRanks; ++k) {
            if (k >= p.ranks) break;
            const float4 x = ptx::ld_shared_cluster_v4(
                ptx::mapa_shared(at_o + 16 * i, k));
            acc.x += x.x * f[k];
            acc.y += x.y * f[k];
            acc.z += x.z * f[k];
            acc.w += x.w * f[k];
          }
        }
        const long long row = out_row(p, b, h, r);
        uint2 out;
        out.x = ptx::pack2<kBF16>(acc.x, acc.y);
        out.y = ptx::pack2<kBF16>(acc.z, acc.w);
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D)[d4] =
            out;
        if (d4 == 0 && p.lse != nullptr)
          p.lse[row] = lse2 * 0.69314718055994531f;
      }
      if (p.scores != nullptr && threadIdx.x < n_rows) {
        float f[kMaxRanks];
        sm_lse[threadIdx.x] = total(threadIdx.x, f);
      }
      if (p.ranks > 1) cluster_arrive();  // peers' sums are read
      if (p.scores != nullptr && n_rows > 0) {
        __syncthreads();  // the part's scores and the LSEs have been written
        const long long key_at = static_cast<long long>(bh) * p.capacity;
        const int key_end = min(len, (count - seg.pos) * kKeys);
#pragma unroll 2
        for (int key = threadIdx.x - seg.pos * kKeys; key < key_end;
             key += C::kThreads) {
          const float before = p.weights[key_at + key];
          float4 x[kRows / 4];
          load_scores<kRows>(p, key_at + key, n_rows, x);
          const float add = weight_of<kRows>(x, sm_lse, n_rows);
          if (add != 0.f) p.weights[key_at + key] = before + add;
        }
      }
      if (p.ranks > 1) cluster_wait();
      return;
    }
    const long long slot = static_cast<long long>(cta) + bh;
#pragma unroll 2
    for (int i = threadIdx.x; i < n_rows * (D / 4); i += C::kThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      reinterpret_cast<float4*>(p.part_o)[(slot * kRows + r) * (D / 4) + d4] =
          cta_o(r, d4);
    }
    if (threadIdx.x < n_rows)
      p.part_lse2[slot * kRows + threadIdx.x] = cta_lse2(threadIdx.x);
    if (seg.end >= count) break;
    next_segment<kKeys, kOver>(p, seg);
    if (seg.pos >= count) break;
  }
}

// ------------------------------------------------------------------ merge
// CTAs 0 .. row_ctas - 1 of a segment join the rows' partials into O and LSE:
// a warp per row where a segment has few partials, else all eight warps (a
// single long sequence has 150 partials per head).  With accumulated weights
// further CTAs, one per 512 keys of a segment, add p = 2^(score - LSE) over
// the rows, read back from the scores the forward kernel left (4 bytes per
// key and row; recomputing them would read the keys' codes again).
constexpr int kMergeThreads = 256;
constexpr int kKeysPerPart = 512;

// Up to 256 partials' LSEs of a row, eight per lane and all loads in flight at
// once: lane l holds partials l, l + 32, ...; f becomes their factors
// 2^(LSE_s - mx - kSlack).  mx and the lanes' shares of sum carry on from the
// partials before; the return value is what those have to be multiplied by.
// (A NaN among the scores has made an LSE NaN, which sets no maximum.)
constexpr int kHeld = 8;
// log2 of the most partials (152 SMs of four CTAs): their sum times V stays
// within fp32.
constexpr float kSlack = 10.f;
template <int kRows>
__device__ __forceinline__ float take_partials(const float* lse2, int r, int s0,
                                               int n_slots, int lane,
                                               float* f, float& mx,
                                               float& sum) {
  float x[kHeld];
  float m = mx;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int s = s0 + 32 * i + lane;
    x[i] = s < n_slots ? lse2[s * kRows + r] : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) m = fmaxf(m, x[i]);
#pragma unroll
  for (int i = 16; i > 0; i /= 2)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  const float before = ptx::ex2(mx - m);
  sum *= before;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    f[i] = ptx::ex2((x[i] - m) - kSlack);
    sum += f[i];
  }
  mx = m;
  return before;
}

// LSE of row r over a segment's partials, by one warp (every lane gets it).
template <int kRows>
__device__ __forceinline__ float row_lse2(const float* lse2, int r,
                                          int n_slots, int lane) {
  float mx = kNone, sum = 0.f, f[kHeld];
  for (int s0 = 0; s0 < n_slots; s0 += 32 * kHeld)
    take_partials<kRows>(lse2, r, s0, n_slots, lane, f, mx, sum);
#pragma unroll
  for (int i = 16; i > 0; i /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, i);
  return lse2_of(mx, sum) + kSlack;
}

template <int D, int NT, bool kBF16>
__global__ void __launch_bounds__(kMergeThreads, 4)
    kv8_merge_kernel(const FwdParams p, int row_ctas, int parts,
                     int row_warps) {
  constexpr int kRows = 8 * NT;
  constexpr int kKeys = tile_keys<D>();
  constexpr int kCols = D / 4;               // float4 columns
  constexpr int kGroups = 32 / kCols;        // partials a warp reads at a time
  __shared__ float sm_lse[kRows];
  __shared__ float4 sm_acc[kMergeThreads / 32][kCols];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per_seg = row_ctas + parts;  // CTAs of a segment
  const int bh = blockIdx.x / per_seg;
  const int unit = blockIdx.x - bh * per_seg;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  // (Lengths are read ahead of the wait: the kernel ahead is the forward.)
  const int len = seq_len(p, b), n_new = seq_new(p, b);
  const int n_rows = n_new * p.group;
  const int rows_per_cta = kMergeThreads / 32 / row_warps;
  const int r = unit * rows_per_cta + warp / row_warps;
  const int key0 = (unit - row_ctas) * kKeysPerPart;
  const bool idle = unit < row_ctas ? unit * rows_per_cta >= n_rows
                                    : (n_rows <= 0 || key0 >= len);

  const int tiles = (len + kKeys - 1) / kKeys;
  long long c0 = 0;
  int n_slots = 0;
  if (tiles > 0 && !idle) {
    int first;
    const int total = list_tiles<kKeys, kOver>(p, b, lane, &first);
    const Cut cut = make_cut<kDecodeWarps>(p, total);
    first += h * (tiles + kOver) + kOver;
    c0 = cut.owner(first);
    n_slots = cut.owner(first + tiles - 1) - static_cast<int>(c0) + 1;
  }
  const float* part_lse2 = p.part_lse2 + (c0 + bh) * kRows;
  // Accumulated weights of this CTA's keys (the forward does not touch them).
  constexpr int kKeysPerThread = kKeysPerPart / kMergeThreads;
  const long long key_at = static_cast<long long>(bh) * p.capacity;
  float w[kKeysPerThread];
#pragma unroll
  for (int i = 0; i < kKeysPerThread; ++i) {
    const int key = key0 + threadIdx.x + i * kMergeThreads;
    w[i] = !idle && unit >= row_ctas && key < len ? p.weights[key_at + key]
                                                  : 0.f;
  }
  start_after_previous();
  if (idle) return;

  if (unit < row_ctas) {
    const bool live = r < n_rows;
    const int d4 = lane % kCols;
    // This lane's partials: sub, sub + step, ...
    const int sub = (warp % row_warps) * kGroups + lane / kCols;
    const int step = row_warps * kGroups;
    float2 t = make_float2(kNone, 0.f);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      const float4* po = reinterpret_cast<const float4*>(p.part_o) +
                         ((c0 + bh) * kRows + r) * kCols + d4;
      // The first partial's O is on its way while its factor is computed.
      float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (sub < n_slots) y0 = po[static_cast<long long>(sub) * kRows * kCols];
      for (int s0 = 0; s0 < n_slots; s0 += 32 * kHeld) {
        float f[kHeld];
        const float before = take_partials<kRows>(part_lse2, r, s0, n_slots,
                                                  lane, f, t.x, t.y);
        acc.x *= before;
        acc.y *= before;
        acc.z *= before;
        acc.w *= before;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (s0 + 32 * i >= n_slots) break;
#pragma unroll 4
          for (int k = sub; k < 32; k += step) {
            const float fk = __shfl_sync(0xffffffffu, f[i], k);
            const int s = s0 + 32 * i + k;
            if (s < n_slots) {
              const float4 y =
                  s == sub ? y0 : po[static_cast<long long>(s) * kRows * kCols];
              acc.x += y.x * fk;
              acc.y += y.y * fk;
              acc.z += y.z * fk;
              acc.w += y.w * fk;
            }
          }
        }
      }
#pragma unroll
      for (int i = 16; i > 0; i /= 2)
        t.y += __shfl_xor_sync(0xffffffffu, t.y, i);
      if constexpr (kGroups == 2) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
      }
    }
    if (row_warps > 1) {
      if (lane < kCols) sm_acc[warp][d4] = acc;
      __syncthreads();
      if (warp % row_warps != 0 || !live) return;
      for (int i = 1; i < row_warps; ++i) {
        const float4 y = sm_acc[warp + i][d4];
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
      }
    }
    if (!live) return;
    const float inv = t.y == 0.f ? 0.f : 1.f / t.y;
    const long long row = out_row(p, b, h, r);
    if (lane < kCols) {
      uint2 out;
      out.x = ptx::pack2<kBF16>(acc.x * inv, acc.y * inv);
      out.y = ptx::pack2<kBF16>(acc.z * inv, acc.w * inv);
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D)[d4] =
          out;
    }
    if (lane == 0 && p.lse != nullptr)
      p.lse[row] = (lse2_of(t.x, t.y) + kSlack) * 0.69314718055994531f;
    return;
  }
  // Scores and LSEs are fetched side by side.
  float4 x[kKeysPerThread][kRows / 4];
#pragma unroll
  for (int i = 0; i < kKeysPerThread; ++i) {
    const int key = key0 + threadIdx.x + i * kMergeThreads;
    load_scores<kRows>(p, key_at + key, key < len ? n_rows : 0, x[i]);
  }
  if (threadIdx.x < kRows) sm_lse[threadIdx.x] = 0.f;
  __syncthreads();
  for (int i = warp; i < n_rows; i += kMergeThreads / 32) {
    const float lse2 = row_lse2<kRows>(part_lse2, i, n_slots, lane);
    if (lane == 0) sm_lse[i] = lse2;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKeysPerThread; ++i) {
    const int key = key0 + threadIdx.x + i * kMergeThreads;
    const float add = weight_of<kRows>(x[i], sm_lse, n_rows);
    if (add != 0.f) p.weights[key_at + key] = w[i] + add;
  }
}

// CTAs of the cluster that takes a segment, which saves the partials and the
// second launch; 0: the list is cut and merged.  Decided by the capacity
// (lengths are not known here), and alike with and without weights, so that
// these change no bit of O: 256 tokens a CTA, fewer and larger parts where
// clusters of that size were not all on the machine at once, up to 512 tokens
// and only with segments enough to fill it.
//
// Cut against clusters, us a call (in a graph), D = 128, 4 rows: 512 tokens of
// 2 segments 9.4 (6.2) against 8.0 (6.5), of 32 10.1 (9.7) against 7.9 (6.9),
// of 256 15.4 (15.3) against 11.1 (10.9); 2048 tokens of 2 segments 9.5 (7.0)
// against 7.9 (7.3), of 32 12.9 (12.3) against 9.5 (8.9), of 96 18.6 against
// 14.5; 16 rows with weights, 512 tokens of 256 segments 28.7 against 19.5.
// In a graph a few segments with weights lose up to a fifth (1024 tokens of 2
// segments 6.6 against 8.2; call by call 10.0 against 8.6).  Larger parts pay
// for the longest sequence (16 of 0 to 2048 tokens, 16 heads of D = 64, with
// weights: 19 cut, 28 with a CTA each).
int cluster_ranks(const FwdParams& p, int ctas) {
  const long long segs = static_cast<long long>(p.B) * p.Hkv;
  constexpr int kPart = 256;
  int ranks = 1;
  while (ranks < kMaxRanks && p.capacity > ranks * kPart) ranks *= 2;
  while (ranks > 1 && segs * ranks > p.grid) ranks /= 2;
  const bool many = 8 * segs >= p.grid / ctas;
  return p.capacity <= ranks * (many ? 2 * kPart : kPart) ? ranks : 0;
}

template <int D, int NT, bool kBF16, bool kWhole>
cudaError_t launch_tiles(const FwdParams& p, long long grid,
                         cudaStream_t stream) {
  using C = Config<D, NT>;
  const cudaError_t err = cudaFuncSetAttribute(
      kv8_decode_kernel<D, NT, kBF16, kWhole>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (err != cudaSuccess) return err;
  return launch_cluster(kv8_decode_kernel<D, NT, kBF16, kWhole>, grid,
                        C::kThreads, C::kBytes, kWhole ? p.ranks : 1, stream,
                        p);
}

template <int D, int NT, bool kBF16>
cudaError_t launch_rows(FwdParams p, cudaStream_t stream) {
  const long long segs = static_cast<long long>(p.B) * p.Hkv;
  p.ranks = cluster_ranks(p, Config<D, NT>::kCtas);
  if (p.ranks > 0)
    return launch_tiles<D, NT, kBF16, true>(p, segs * p.ranks, stream);
  const cudaError_t err =
      launch_tiles<D, NT, kBF16, false>(p, p.grid, stream);
  if (err != cudaSuccess) return err;
  const int parts = p.scores == nullptr
                        ? 0
                        : (p.capacity + kKeysPerPart - 1) / kKeysPerPart;
  // Partials of a segment if all are equally long.
  const int row_warps = segs * 16 <= p.grid ? kMergeThreads / 32 : 1;
  const int rows_per_cta = kMergeThreads / 32 / row_warps;
  const int row_ctas = (p.group * p.Sq + rows_per_cta - 1) / rows_per_cta;
  return launch_pdl(kv8_merge_kernel<D, NT, kBF16>, segs * (row_ctas + parts),
                    kMergeThreads, 0, stream, p, row_ctas, parts, row_warps);
}

template <int D, bool kBF16>
cudaError_t launch_dt(int rows, const FwdParams& p, cudaStream_t stream) {
  return rows <= 8 ? launch_rows<D, 1, kBF16>(p, stream)
                   : launch_rows<D, 2, kBF16>(p, stream);
}

}  // namespace

cudaError_t launch_decode(int D, bool bf16, int rows, const FwdParams& p,
                          cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch_dt<64, true>(rows, p, stream)
                : launch_dt<64, false>(rows, p, stream);
  return bf16 ? launch_dt<128, true>(rows, p, stream)
              : launch_dt<128, false>(rows, p, stream);
}

}  // namespace kv8
}  // namespace attn
