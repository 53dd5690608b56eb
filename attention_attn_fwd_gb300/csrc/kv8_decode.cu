// Attention of a few query rows per K/V head over the 8-bit cache, and the
// merge of its partial results.
//
// Mathematics: flash-decoding.  The keys of all (batch, K/V head) segments
// form one list of 16-key tiles, cut into equal consecutive shares, one per
// CTA; a CTA's warps take its tiles in turn, each with its own running
// maximum m, sum l and accumulator O, which meet in shared memory at the end
// of a segment.  A partial result goes to workspace slot (CTA + segment):
// both only grow along the list, so no two share one.  The merge kernel
// joins a segment's partials by their maxima.  Lengths come from device
// memory, so the cut follows them without the host's knowing: ragged batches
// are balanced to a tile.
//
// Products: S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16 in fp16,
// 16 keys (or 16 of D) by 8 query rows.  E4M3 codes are fp16 values, so
// K and V convert exactly; Q is multiplied by a power of two per row that
// brings its largest element to [2^13, 2^14), which makes bf16 -> fp16 exact
// down to 2^-37 of the row's largest element (below fp32 accumulation's own
// rounding).  Block scales multiply scores and weights in fp32.  P is rounded
// to fp16 (2^-11 relative, the rounding of the 16-bit output itself or less)
// with 2^7 of headroom used up so that weights down to 2^-29 of the row's
// largest stay normal numbers.  The row sums take P unrounded.
//
// Codes go from global memory straight to the registers of the lanes whose
// MMA fragments need them, 16 bytes at a time: the d index of both products
// may be permuted freely, so lane c of a quad owns bytes 16c.. of a 64-byte
// half row of K (fragment columns) and lane group g8 owns bytes 16 g8.. of
// four V rows.  No shared memory, no transposes but a byte permute and one
// movmatrix per 8 x 8 weights.  Bound by the bytes of the codes: tiles are
// prefetched one ahead per warp, about 64 KB in flight per SM.
#include "kv8_common.cuh"

namespace attn {
namespace kv8 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;          // keys per warp step
constexpr float kTau = 8.f;        // lazy rescale threshold (log2 units)
constexpr float kPScale = 128.f;   // 2^7: P <= 2^(8 + 7) < 65504

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1,
                                        uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(y)
               : "r"(x));
  return y;
}

// Codes are read once: keep them out of L1.
__device__ __forceinline__ uint4 ld_codes16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_codes8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// The list of tiles: sequence b contributes Hkv * row_blocks segments of
// ceil(lens[b] / 16) tiles.
__device__ __forceinline__ int seq_len(const FwdParams& p, int b) {
  return clamp_len(p.lens[b], p.capacity, p.status);
}
__device__ __forceinline__ int seq_new(const FwdParams& p, int b) {
  return p.new_lens == nullptr ? p.Sq
                               : clamp_len(p.new_lens[b], p.Sq, p.status);
}

// Tiles of all sequences before `end` (every lane of the warp gets the sum).
__device__ __forceinline__ long long tiles_before(const FwdParams& p, int end,
                                                  int lane) {
  long long t = 0;
  for (int b = lane; b < end; b += 32)
    t += (seq_len(p, b) + kTile - 1) / kTile;
#pragma unroll
  for (int s = 16; s > 0; s /= 2) t += __shfl_xor_sync(0xffffffffu, t, s);
  return t * p.Hkv * p.row_blocks;
}

// Sequence that holds list position x (x < total), and the tiles before it.
__device__ __forceinline__ int find_seq(const FwdParams& p, long long x,
                                        int lane, long long* before) {
  long long base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    long long t = 0;
    if (b < p.B)
      t = static_cast<long long>((seq_len(p, b) + kTile - 1) / kTile) *
          p.Hkv * p.row_blocks;
    long long incl = t;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > x);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      *before = base + __shfl_sync(0xffffffffu, incl - t, l);
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  *before = base;  // not reached for x < total
  return p.B - 1;
}

// CTAs that take a share: at most one tile per warp is the finest cut.
__device__ __forceinline__ long long shares(const FwdParams& p,
                                            long long total) {
  const long long most = (total + kWarps - 1) / kWarps;
  return most < p.grid ? (most > 0 ? most : 1) : p.grid;
}

// Visible tokens of row r (token-major: row r = token r / group, head
// r % group) of a sequence.
__device__ __forceinline__ int row_end(const FwdParams& p, int len, int n_new,
                                       int r) {
  if (!p.causal) return len;
  return min(len, max(0, len - n_new + r / p.group + 1));
}

// One tile's codes in registers: K rows g8 and g8 + 8, V rows 2c, 2c + 1,
// 2c + 8, 2c + 9 of the tile.
template <int D>
struct Codes {
  static constexpr int kHalves = D / 64;   // 64-byte halves of a K row
  static constexpr int kVWords = D / 32;   // words of a V row per lane
  uint32_t k[2][kHalves][4];
  uint32_t v[4][kVWords];
};

template <int D>
__device__ __forceinline__ void load_k(Codes<D>& t, const uint8_t* k, int key0,
                                       int len, int g8, int c) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int key = key0 + g8 + 8 * i;
#pragma unroll
    for (int h = 0; h < Codes<D>::kHalves; ++h) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (key < len)
        w = ld_codes16(k + static_cast<long long>(key) * D + 64 * h + 16 * c);
      t.k[i][h][0] = w.x;
      t.k[i][h][1] = w.y;
      t.k[i][h][2] = w.z;
      t.k[i][h][3] = w.w;
    }
  }
}

template <int D>
__device__ __forceinline__ void load_v(Codes<D>& t, const uint8_t* v, int key0,
                                       int len, int g8, int c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = key0 + 2 * c + (i & 1) + 8 * (i >> 1);
    const uint8_t* at = v + static_cast<long long>(key) * D + (D / 8) * g8;
    if constexpr (D == 128) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (key < len) w = ld_codes16(at);
      t.v[i][0] = w.x;
      t.v[i][1] = w.y;
      t.v[i][2] = w.z;
      t.v[i][3] = w.w;
    } else {
      uint2 w = make_uint2(0u, 0u);
      if (key < len) w = ld_codes8(at);
      t.v[i][0] = w.x;
      t.v[i][1] = w.y;
    }
  }
}

// NT: 8-row groups of query rows a CTA holds (8 or 16 rows of a K/V head).
template <int D, int NT, bool kBF16>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1)
    kv8_decode_kernel(const FwdParams p) {
  constexpr int kRows = 8 * NT;
  constexpr int kKSteps = D / 16;
  constexpr int kMT = D / 16;      // m-tiles of O^T
  extern __shared__ float smem[];  // [kWarps][kRows][D + 4], then m, l
  constexpr int kPitch = D + 4;    // floats: rows start 4 banks apart
  float* sm_o = smem;
  float* sm_m = smem + kWarps * kRows * kPitch;  // [kWarps][kRows]
  float* sm_l = sm_m + kWarps * kRows;           // [kWarps][kRows]

  // The merge kernel may be scheduled early: its CTAs wait for this grid.
  ptx::griddep_launch_dependents();

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g8 = lane / 4, c = lane % 4;
  const long long total = tiles_before(p, p.B, lane);
  const long long n_cta = shares(p, total);
  const int cta = blockIdx.x;
  if (cta >= n_cta) return;
  long long at = total * cta / n_cta;
  const long long end = total * (cta + 1) / n_cta;
  if (at >= end) return;

  long long before;
  int b = find_seq(p, at, lane, &before);
  while (at < end) {
    int len = seq_len(p, b);
    long long tiles = (len + kTile - 1) / kTile;
    while (at - before >= tiles * p.Hkv * p.row_blocks) {  // next sequence
      before += tiles * p.Hkv * p.row_blocks;
      ++b;
      len = seq_len(p, b);
      tiles = (len + kTile - 1) / kTile;
    }
    const int seg_in_b = static_cast<int>((at - before) / tiles);
    const int t_first = static_cast<int>((at - before) % tiles);
    const int t_last = static_cast<int>(
        min(tiles, static_cast<long long>(t_first) + (end - at)));
    at += t_last - t_first;

    const int h = seg_in_b / p.row_blocks;
    const int rb = seg_in_b - h * p.row_blocks;
    const int r0 = rb * kRows;
    const int bh = b * p.Hkv + h;
    const int n_new = seq_new(p, b);
    const int n_rows = min(kRows, n_new * p.group - r0);  // valid rows
    if (n_rows <= 0) continue;
    const int min_end = row_end(p, len, n_new, r0);
    const int max_end = row_end(p, len, n_new, r0 + n_rows - 1);

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
          const int tok = (r0 + r) / p.group, hd = (r0 + r) % p.group;
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
      // Power of two that brings the row's largest element to [2^13, 2^14).
      const int ex = (__float_as_int(amax) >> 23) - 127;
      const int up = max(-114, min(13 - ex, 126));
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
        vis[nt][e] = rr < n_rows ? row_end(p, len, n_new, r0 + rr) : max_end;
      }
    }

    const uint8_t* kb = p.k + static_cast<long long>(bh) * p.capacity * D;
    const uint8_t* vb = p.v + static_cast<long long>(bh) * p.capacity * D;
    const float* ksb = p.k_scale + static_cast<long long>(bh) * p.nblk;
    const float* vsb = p.v_scale + static_cast<long long>(bh) * p.nblk;

    float m[NT][2], l[NT][2], o[NT][kMT][4];
    float unit = 0.f;  // O is held in units of this V scale (times 2^7)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    // Tiles past every row's horizon hold nothing for this row block.
    const int t_stop = min(t_last, (max_end + kTile - 1) / kTile);
    Codes<D> cur;
    int t = t_first + warp;
    float ks = 0.f, vs = 0.f;
    if (t < t_stop) {
      load_k<D>(cur, kb, t * kTile, len, g8, c);
      load_v<D>(cur, vb, t * kTile, len, g8, c);
      ks = __ldg(ksb + ((t * kTile) >> p.block_shift));
      vs = __ldg(vsb + ((t * kTile) >> p.block_shift));
    }
    for (; t < t_stop; t += kWarps) {
      const int key0 = t * kTile;
      const int t_next = t + kWarps;
      const bool more = t_next < t_stop;
      // S^T tile.
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_half2(cur.k[0][hf][w], a0, a2);
          e4m3x4_to_half2(cur.k[1][hf][w], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(s[nt], a0, a1, a2, a3, bq[nt][4 * hf + w][0],
                    bq[nt][4 * hf + w][1]);
        }
      const float ks_now = ks, vs_now = vs;
      if (more) {
        load_k<D>(cur, kb, t_next * kTile, len, g8, c);
        ks = __ldg(ksb + ((t_next * kTile) >> p.block_shift));
        vs = __ldg(vsb + ((t_next * kTile) >> p.block_shift));
      }
      // Scores in log2 units; hidden ones are -inf.
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] *= mult[nt][e & 1] * ks_now;
      if (key0 + kTile > min_end) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + g8 + 8 * (e >> 1) >= vis[nt][e & 1])
              s[nt][e] = -INFINITY;
      }
      if (p.scores != nullptr) {
        float* sc = p.scores +
                    (static_cast<long long>(bh) * p.capacity + key0 + g8) *
                        kRows + 2 * c;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (key0 + g8 < len)
            *reinterpret_cast<float2*>(sc + 8 * nt) =
                make_float2(s[nt][0], s[nt][1]);
          if (key0 + g8 + 8 < len)
            *reinterpret_cast<float2*>(sc + 8 * kRows + 8 * nt) =
                make_float2(s[nt][2], s[nt][3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          grow |= fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + kTau;
      grow |= vs_now > unit;
      // Lazy rescale: some row's maximum grew by more than 2^8, or a block's
      // V scale exceeds the unit O is held in.
      if (__any_sync(0xffffffffu, grow)) {
        const float unit_new = fmaxf(unit, vs_now);
        const float f_unit = unit_new > 0.f ? unit / unit_new : 1.f;
        unit = unit_new;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[nt][e], s[nt][e + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(m[nt][e], mx);
            const float alpha =
                m_new == -INFINITY ? 1.f : ptx::ex2(m[nt][e] - m_new);
            m[nt][e] = m_new;
            l[nt][e] *= alpha;
            const float f = alpha * f_unit;
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
              o[nt][i][e] *= f;
              o[nt][i][e + 2] *= f;
            }
          }
      }
      // P^T in fp16, times 2^7 and the block's V scale over the unit.
      const float pf = unit > 0.f ? kPScale * vs_now / unit : 0.f;
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // A column nothing of which is visible yet has m = -inf (NaN
          // scores stay NaN).
          w[e] = s[nt][e] == -INFINITY ? 0.f
                                       : ptx::ex2(s[nt][e] - m[nt][e & 1]);
          l[nt][e & 1] += w[e];
        }
        pb[nt][0] =
            movmatrix_trans(ptx::pack2<false>(w[0] * pf, w[1] * pf));
        pb[nt][1] =
            movmatrix_trans(ptx::pack2<false>(w[2] * pf, w[3] * pf));
      }
      // O^T += V^T P^T.
#pragma unroll
      for (int w = 0; w < Codes<D>::kVWords; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t lo = __byte_perm(cur.v[2 * i][w], cur.v[2 * i + 1][w],
                                          0x5140);
          const uint32_t hi = __byte_perm(cur.v[2 * i][w], cur.v[2 * i + 1][w],
                                          0x7362);
          e4m3x4_to_half2(lo, a[0][2 * i], a[0][2 * i + 1]);
          e4m3x4_to_half2(hi, a[1][2 * i], a[1][2 * i + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[nt][2 * w], a[0][0], a[0][1], a[0][2], a[0][3], pb[nt][0],
                  pb[nt][1]);
          mma_f16(o[nt][2 * w + 1], a[1][0], a[1][1], a[1][2], a[1][3],
                  pb[nt][0], pb[nt][1]);
        }
      }
      if (more) load_v<D>(cur, vb, t_next * kTile, len, g8, c);
    }

    // The warps' results meet: maxima, then O and l under the common one.
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
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * c + e;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          mx = fmaxf(mx, sm_m[w * kRows + r]);
        const float f =
            m[nt][e] == -INFINITY ? 0.f : ptx::ex2(m[nt][e] - mx);
        const float fo = f * unit * (1.f / kPScale);
        if (g8 == 0) sm_l[warp * kRows + r] = l[nt][e] * f;
        float* dst = sm_o + (warp * kRows + r) * kPitch + (D / 8) * g8;
#pragma unroll
        for (int i = 0; i < kMT; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(o[nt][i][e] * fo, o[nt][i][e + 2] * fo,
                          o[nt][i + 1][e] * fo, o[nt][i + 1][e + 2] * fo);
      }
    __syncthreads();
    const long long slot =
        cta + (static_cast<long long>(b) * p.Hkv + h) * p.row_blocks + rb;
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      if (r >= n_rows) break;
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
      reinterpret_cast<float4*>(p.part_o)[(slot * kRows + r) * (D / 4) + d4] =
          acc;
    }
    if (threadIdx.x < n_rows) {
      const int r = threadIdx.x;
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mx = fmaxf(mx, sm_m[w * kRows + r]);
        sum += sm_l[w * kRows + r];
      }
      p.part_ml[slot * kRows + r] = make_float2(mx, sum);
    }
  }
}

// ------------------------------------------------------------------ merge
// One CTA per segment and part: part 0 merges the segment's partial rows
// into O and LSE; with accumulated weights every part adds the weights of
// its share of the keys, p = 2^(score - LSE), read back from the scores the
// forward kernel left (4 bytes per key and row; recomputing them would read
// the keys' codes again).
constexpr int kMergeThreads = 256;
constexpr int kKeysPerPart = 512;

template <int D, int NT, bool kBF16>
__global__ void __launch_bounds__(kMergeThreads)
    kv8_merge_kernel(const FwdParams p, int parts) {
  constexpr int kRows = 8 * NT;
  __shared__ float sm_lse[kRows];
  ptx::griddep_wait();
  const int lane = threadIdx.x % 32;
  const long long seg = blockIdx.x / parts;
  const int part = static_cast<int>(blockIdx.x - seg * parts);
  const int rb = static_cast<int>(seg % p.row_blocks);
  const int bh = static_cast<int>(seg / p.row_blocks);
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int len = seq_len(p, b), n_new = seq_new(p, b);
  const int r0 = rb * kRows;
  const int n_rows = min(kRows, n_new * p.group - r0);
  if (n_rows <= 0) return;
  if (part > 0 && part * kKeysPerPart >= len) return;

  const long long tiles = (len + kTile - 1) / kTile;
  long long c0 = 0, n_slots = 0;
  if (tiles > 0) {
    const long long total = tiles_before(p, p.B, lane);
    const long long n_cta = shares(p, total);
    const long long first =
        tiles_before(p, b, lane) +
        (static_cast<long long>(h) * p.row_blocks + rb) * tiles;
    // CTA c holds positions [total c / n, total (c + 1) / n).
    c0 = ((first + 1) * n_cta - 1) / total;
    n_slots = ((first + tiles) * n_cta - 1) / total - c0 + 1;
  }
  const float2* ml = p.part_ml + (c0 + seg) * kRows;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) +
                     (c0 + seg) * kRows * (D / 4);
  for (int i = threadIdx.x; i < kRows * (D / 4); i += kMergeThreads) {
    const int r = i / (D / 4), d4 = i % (D / 4);
    if (r >= n_rows) break;
    if (part > 0 && d4 != 0) continue;  // only the row's LSE is wanted
    float mx = -INFINITY;
    for (int s = 0; s < n_slots; ++s) mx = fmaxf(mx, ml[s * kRows + r].x);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < n_slots; ++s) {
      const float2 x = ml[s * kRows + r];
      const float f = x.x == -INFINITY ? 0.f : ptx::ex2(x.x - mx);
      sum += x.y * f;
      if (part == 0) {
        const float4 y =
            po[(static_cast<long long>(s) * kRows + r) * (D / 4) + d4];
        acc.x += y.x * f;
        acc.y += y.y * f;
        acc.z += y.z * f;
        acc.w += y.w * f;
      }
    }
    // A sum of 0: the row sees no token.  (A NaN among the scores has made
    // the sum NaN, also where no other score set a maximum.)
    const float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
    if (d4 == 0) sm_lse[r] = lse2;
    if (part > 0) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = (r0 + r) / p.group, hd = (r0 + r) % p.group;
    const long long row =
        (static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq + tok;
    uint2 out;
    out.x = ptx::pack2<kBF16>(acc.x * inv, acc.y * inv);
    out.y = ptx::pack2<kBF16>(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D)[d4] = out;
    if (d4 == 0) {
      if (p.lse != nullptr) p.lse[row] = lse2 * 0.69314718055994531f;
      if (p.lse2 != nullptr)
        p.lse2[static_cast<long long>(bh) * p.row_blocks * kRows + r0 + r] =
            lse2;
    }
  }
  if (p.scores == nullptr) return;
  __syncthreads();
  const int k_end = min(len, (part + 1) * kKeysPerPart);
  for (int key = part * kKeysPerPart + threadIdx.x; key < k_end;
       key += kMergeThreads) {
    const float* s =
        p.scores + (static_cast<long long>(bh) * p.capacity + key) * kRows;
    float w = 0.f;
    for (int r = 0; r < n_rows; ++r) {
      const float x = s[r];
      if (x != -INFINITY) w += ptx::ex2(x - sm_lse[r]);
    }
    if (w != 0.f) p.weights[static_cast<long long>(bh) * p.capacity + key] += w;
  }
}

// ---------------------------------------------------------------- weights
// Accumulated weights of many query rows: the scores of a 128-key tile are
// computed again, S^T = K Q^T as above, with the keys' fragments kept in
// registers and the query rows passing through shared memory 64 at a time;
// p = 2^(score - LSE) summed over the rows.  Every key has one owner, so the
// sums have one order.
constexpr int kWRows = 64;

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 2)
    kv8_weights_kernel(const FwdParams p, int lse2_rows) {
  constexpr int kPitch = D + 8;  // halves: rows 16 bytes apart in the banks
  __shared__ __align__(16) uint16_t sq[kWRows * kPitch];
  __shared__ float s_mult[kWRows], s_lse[kWRows];
  __shared__ int s_vis[kWRows];
  ptx::griddep_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g8 = lane / 4, c = lane % 4;
  const int tiles = (p.capacity + 127) / 128;
  const int bh = blockIdx.x / tiles;
  const int tile0 = (blockIdx.x - bh * tiles) * 128;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int len = seq_len(p, b), n_new = seq_new(p, b);
  if (tile0 >= len) return;
  const int rows = n_new * p.group;
  // Rows before r_first see nothing of this tile.
  int r_first = 0;
  if (p.causal) r_first = max(0, tile0 - (len - n_new)) * p.group;
  const int key0 = tile0 + warp * 16;

  uint32_t a[D / 16][4];
  {
    Codes<D> t;
    load_k<D>(t, p.k + static_cast<long long>(bh) * p.capacity * D, key0, len,
              g8, c);
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        e4m3x4_to_half2(t.k[0][hf][w], a[4 * hf + w][0], a[4 * hf + w][2]);
        e4m3x4_to_half2(t.k[1][hf][w], a[4 * hf + w][1], a[4 * hf + w][3]);
      }
  }
  float ks = 0.f;
  if (key0 < len)
    ks = __ldg(p.k_scale + static_cast<long long>(bh) * p.nblk +
               (key0 >> p.block_shift));
  float sum[2] = {0.f, 0.f};
  for (int r0 = r_first; r0 < rows; r0 += kWRows) {
    __syncthreads();
    constexpr int kPer = D / 8;  // threads per row
    for (int i = threadIdx.x; i < kWRows * kPer; i += kThreads) {
      const int r = i / kPer, ch = i % kPer;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      const bool ok = r0 + r < rows;
      if (ok) {
        const int tok = (r0 + r) / p.group, hd = (r0 + r) % p.group;
        w = __ldg(reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) +
            ((static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq +
             tok) * D + ch * 8));
      }
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
      float2 f[4];
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = unpack2<kBF16>(in[e]);
        amax = fmaxf(amax, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
      }
#pragma unroll
      for (int s = kPer / 2; s > 0; s /= 2)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
      const int ex = (__float_as_int(amax) >> 23) - 127;
      const int up = max(-114, min(13 - ex, 126));
      const float f_up = exp2_int(up);
      uint32_t out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[e] = ptx::pack2<false>(f[e].x * f_up, f[e].y * f_up);
      *reinterpret_cast<uint4*>(sq + r * kPitch + ch * 8) =
          make_uint4(out[0], out[1], out[2], out[3]);
      if (ch == 0) {
        s_mult[r] = p.scale_log2 * exp2_int(-up);
        s_vis[r] = ok ? row_end(p, len, n_new, r0 + r) : 0;
        s_lse[r] =
            ok ? p.lse2[static_cast<long long>(bh) * lse2_rows + r0 + r]
               : INFINITY;
      }
    }
    __syncthreads();
    if (key0 >= len) continue;
#pragma unroll 2
    for (int nt = 0; nt < kWRows / 8; ++nt) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        const uint16_t* row = sq + (8 * nt + g8) * kPitch + 64 * hf + 16 * c;
        const uint4 w0 = *reinterpret_cast<const uint4*>(row);
        const uint4 w1 = *reinterpret_cast<const uint4*>(row + 8);
        const uint32_t bw[8] = {w0.x, w0.y, w0.z, w0.w,
                                w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w)
          mma_f16(s, a[4 * hf + w][0], a[4 * hf + w][1], a[4 * hf + w][2],
                  a[4 * hf + w][3], bw[2 * w], bw[2 * w + 1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 8 * nt + 2 * c + (e & 1);
        const int key = key0 + g8 + 8 * (e >> 1);
        if (key < s_vis[r])
          sum[e >> 1] += ptx::ex2(s[e] * (s_mult[r] * ks) - s_lse[r]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
    const int key = key0 + g8 + 8 * e;
    if (c == 0 && key < len && sum[e] != 0.f)
      p.weights[static_cast<long long>(bh) * p.capacity + key] += sum[e];
  }
}

template <class Kernel, class... Args>
cudaError_t launch_pdl(Kernel kernel, long long grid, int threads,
                       cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int NT, bool kBF16>
cudaError_t launch_rows(const FwdParams& p, cudaStream_t stream) {
  constexpr int kRows = 8 * NT;
  constexpr int kSmem = kWarps * kRows * (D + 4 + 2) * 4;
  cudaError_t err = cudaFuncSetAttribute(
      kv8_decode_kernel<D, NT, kBF16>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (err != cudaSuccess) return err;
  kv8_decode_kernel<D, NT, kBF16><<<p.grid, kThreads, kSmem, stream>>>(p);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const long long segs = static_cast<long long>(p.B) * p.Hkv * p.row_blocks;
  const int parts = p.scores == nullptr
                        ? 1
                        : (p.capacity + kKeysPerPart - 1) / kKeysPerPart;
  err = launch_pdl(kv8_merge_kernel<D, NT, kBF16>, segs * parts,
                   kMergeThreads, stream, p, parts);
  if (err != cudaSuccess || p.weights == nullptr || p.scores != nullptr)
    return err;
  const long long tiles = (p.capacity + 127) / 128;
  return launch_pdl(kv8_weights_kernel<D, kBF16>,
                    static_cast<long long>(p.B) * p.Hkv * tiles, kThreads,
                    stream, p, p.row_blocks * kRows);
}

template <int D, bool kBF16>
cudaError_t launch_dt(int rows, const FwdParams& p, cudaStream_t stream) {
  return rows <= 8 ? launch_rows<D, 1, kBF16>(p, stream)
                   : launch_rows<D, 2, kBF16>(p, stream);
}

}  // namespace

cudaError_t launch_fwd(int D, bool bf16, int rows, const FwdParams& p,
                       cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch_dt<64, true>(rows, p, stream)
                : launch_dt<64, false>(rows, p, stream);
  return bf16 ? launch_dt<128, true>(rows, p, stream)
              : launch_dt<128, false>(rows, p, stream);
}

}  // namespace kv8
}  // namespace attn
