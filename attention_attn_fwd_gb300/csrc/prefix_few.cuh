// Attention of up to 16 query rows per K/V head over each sequence's own keys,
// behind a shared prefix: the work of the thread blocks that the many-row
// kernel sets aside for it.
//
// Mathematics: flash-decoding.  The keys of all (sequence, K/V head) segments
// form one list of tiles (4 KB of keys), cut into equal consecutive shares, one
// per warp.  A warp has its own running maximum, sum and accumulator; a part of
// a segment goes to workspace slot (warp + segment) -- both only grow along the
// list, so no two share one -- and is joined with the others and the prefix's
// by the merge kernel.
//
// Products: S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16, 16 keys (or
// 16 of D) by 8 query rows: a 128-row tcgen05 tile would be nearly empty, and
// the bytes of K and V bound this work.  P is rounded to the inputs' type and
// held times 2^kShift as in the many-row kernel.
//
// Tiles reach shared memory by 16-byte asynchronous copies, a ring per warp
// that runs ahead across segments; rows past a length are filled with zeros
// and read nothing.  Chunk j of row r lies at chunk j ^ r % 8, so that
// ldmatrix reads share no banks.  Three tiles ahead: 192 KB of the CTA's eight
// warps are in flight or worked on, all that an SM holds.
//
// What bounds it: the bytes of K and V.  256 sequences of 300 own tokens, 16
// heads of 64 (157 MB with a prefix of 2048, which takes some CTAs): 36 us and
// 7 of the merge, of which loads can go for about 28; the rest is the start.
#pragma once

#include "prefix_common.cuh"

namespace attn {
namespace prefix {

__device__ __forceinline__ void ldmatrix4(uint32_t* a, uint32_t addr) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t* a, uint32_t addr) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
      : "r"(addr)
      : "memory");
}

// C (16 x 8, fp32) += A (16 x 16) B (16 x 8).
template <bool kBF16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kBF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    kv8::mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
  }
}

constexpr int kFewStages = 3;
constexpr int kFewTile = 4096;  // bytes of keys in a tile, and of values
constexpr int kFewRing = kFewStages * 2 * kFewTile;  // bytes of a warp's ring

// Places of a segment in the list.
template <int D>
__device__ __forceinline__ int few_places(int tiles) {
  return tiles > 0 ? tiles + kFewOver : 0;
}
// Tiles of a sequence (of each of its heads): none where no row wants them.
template <int D>
__device__ __forceinline__ int few_tiles_of(const PrefixParams& p, int len,
                                            int n_new) {
  len = kv8::clamp_len(len, p.capacity, p.status);
  n_new = kv8::clamp_len(n_new, p.Sq, p.status);
  return n_new > 0 ? (len + few_keys<D>() - 1) / few_keys<D>() : 0;
}
template <int D>
__device__ __forceinline__ int few_tiles(const PrefixParams& p, int b) {
  return few_tiles_of<D>(p, p.lens[b],
                         p.new_lens == nullptr ? p.Sq : p.new_lens[b]);
}

// The lengths of the lane's first sequence, fetched ahead of their use.
struct FewLens {
  int len, n_new;
  __device__ __forceinline__ void load(const PrefixParams& p, int lane) {
    len = 0;
    n_new = p.Sq;
    if (lane < p.B) {
      len = p.lens[lane];
      if (p.new_lens != nullptr) n_new = p.new_lens[lane];
    }
  }
};

// Places of all segments, for every lane of the calling warp.
template <int D>
__device__ __forceinline__ int few_total(const PrefixParams& p,
                                         const FewLens& ahead, int lane) {
  int t = lane < p.B ? few_places<D>(few_tiles_of<D>(p, ahead.len,
                                                     ahead.n_new))
                     : 0;
  for (int b = lane + 32; b < p.B; b += 32)
    t += few_places<D>(few_tiles<D>(p, b));
#pragma unroll
  for (int s = 16; s > 0; s /= 2) t += __shfl_xor_sync(0xffffffffu, t, s);
  return t * p.Hkv;
}

// A segment as a warp walks its share: its tiles lie at [pos, end) counted from
// the share's start (pos < 0: it began earlier).
struct FewSegment {
  int pos, end;
  int b, h, len, tiles;
};

template <int D>
__device__ __forceinline__ void few_enter(const PrefixParams& p, int b,
                                          FewSegment& s) {
  s.b = b;
  s.len = kv8::seq_len(p, b);
  s.tiles = few_tiles<D>(p, b);
}

// The segment that holds place `first` of the list (there is one).
template <int D>
__device__ __forceinline__ void few_find(const PrefixParams& p, int first,
                                         int lane, FewSegment& s) {
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int t =
        b < p.B ? few_places<D>(few_tiles<D>(p, b)) * p.Hkv : 0;
    int incl = t;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, incl, i);
      if (lane >= i) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > first);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      const int off = first - base - __shfl_sync(0xffffffffu, incl - t, l);
      few_enter<D>(p, b0 + l, s);
      s.h = off / few_places<D>(s.tiles);
      s.pos = kFewOver - (off - s.h * few_places<D>(s.tiles));
      s.end = s.pos + s.tiles;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <int D>
__device__ __forceinline__ void few_next(const PrefixParams& p,
                                         FewSegment& s) {
  s.pos = s.end + kFewOver;
  if (++s.h == p.Hkv) {
    s.h = 0;
    do {  // some later sequence has tiles: the share is not at its end
      few_enter<D>(p, s.b + 1, s);
    } while (s.tiles == 0);
  }
  s.end = s.pos + s.tiles;
}

// Byte offset of 16-byte chunk j of row r in a tile.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int j) {
  return r * (2 * D) + ((j ^ (r & 7)) << 4);
}

// A warp's loads: they run ahead of its products, across segments.
template <int D>
struct FewLoader {
  static constexpr int kKeys = few_keys<D>();
  static constexpr int kPerRow = D / 8;          // chunks
  static constexpr int kRowStep = 32 / kPerRow;  // rows between a lane's chunks
  static constexpr int kChunks = kFewTile / 16 / 32;
  FewSegment seg;
  int pos;                 // next tile, counted from the share's start
  const uint16_t* k;       // this lane's first chunk of the segment
  const uint16_t* v;

  __device__ __forceinline__ void set_segment(const PrefixParams& p,
                                              int lane) {
    const long long at =
        (static_cast<long long>(seg.b) * p.Hkv + seg.h) * p.capacity * D +
        8 * lane;
    k = p.k + at;
    v = p.v + at;
  }
  // The segment's query rows on their way to L1, a line a lane (64 sequences
  // behind 8192 tokens: 44.0 -> 43.2 us).
  __device__ __forceinline__ void prefetch_rows(const PrefixParams& p,
                                                int lane) {
    constexpr int kLines = D / 64;
    if (lane < p.rows * kLines) {
      const uint16_t* q = p.q +
                          q_row_index(p, seg.b, seg.h, lane / kLines) * D +
                          lane % kLines * 64;
      asm volatile("prefetch.global.L1 [%0];" ::"l"(q));
    }
  }
  __device__ __forceinline__ void next(const PrefixParams& p, int count,
                                       uint32_t to, int lane) {
    bool moved = false;
    while (pos < count && pos >= seg.end) {
      few_next<D>(p, seg);
      pos = seg.pos;
      moved = true;
    }
    if (pos < count) {
      if (moved) {
        set_segment(p, lane);
        prefetch_rows(p, lane);
      }
      const int t = pos - seg.pos;
      const long long off = static_cast<long long>(t) * kKeys * D;
      const int r0 = lane / kPerRow, j = lane % kPerRow;
      const int left = seg.len - t * kKeys;
      if (left >= kKeys) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint32_t dst = to + chunk_at<D>(r0 + i * kRowStep, j);
          ptx::cp_async16(dst, k + off + i * kRowStep * D);
          ptx::cp_async16(dst + kFewTile, v + off + i * kRowStep * D);
        }
      } else {
#pragma unroll 2
        for (int i = 0; i < kChunks; ++i) {
          const uint32_t dst = to + chunk_at<D>(r0 + i * kRowStep, j);
          const bool in = r0 + i * kRowStep < left;
          const long long at = in ? off + i * kRowStep * D : 0;
          ptx::cp_async16_or_zero(dst, k + at, in);
          ptx::cp_async16_or_zero(dst + kFewTile, v + at, in);
        }
      }
      ++pos;
    }
    ptx::cp_async_commit();
  }
};

// The share of warp `gw` of `warps` of a list of `total` places.  NT: 8-row
// groups of query rows.
template <int D, int NT, bool kBF16>
__device__ __forceinline__ void few_share(const PrefixParams& p, int gw,
                                          int warps, int total, int lane,
                                          uint32_t ring) {
  constexpr int kRows = 8 * NT;
  constexpr int kKeys = few_keys<D>();
  constexpr int kSub = kKeys / 16;  // 16-key steps per tile
  constexpr int kKSteps = D / 16;
  constexpr float kShift = kBF16 ? -24.f : 7.f;
  constexpr float kTau = 8.f;  // lazy rescale threshold (log2 units)

  if (total == 0) return;
  kv8::Cut cut;
  cut.n = min(warps, total);
  cut.q = total / cut.n;
  cut.rest = total - cut.q * cut.n;
  if (gw >= cut.n) return;
  const int first = cut.first(gw), count = cut.first(gw + 1) - first;
  FewSegment seg;
  few_find<D>(p, first, lane, seg);
  if (seg.pos >= count) return;  // empty places alone
  const int g8 = lane / 4, c = lane % 4;
  FewLoader<D> ld;
  ld.seg = seg;
  ld.pos = max(seg.pos, 0);
  ld.set_segment(p, lane);
#pragma unroll
  for (int i = 0; i < kFewStages; ++i)
    ld.next(p, count, ring + i * 2 * kFewTile, lane);
  // This lane's rows of ldmatrix's four 8 x 8 matrices: of K (keys 0-7 and
  // 8-15, then the next 8 of D) and of V (the next 8 of D, then keys 8-15).
  const int k_row = lane % 8 + 8 * ((lane / 8) & 1), k_col = lane / 16;
  const int v_row = lane % 8 + 8 * (lane / 16), v_col = (lane / 8) & 1;
  const float mult = p.negate ? -p.scale_log2 : p.scale_log2;

  int stage = 0;
  while (true) {
    const int b = seg.b, h = seg.h, len = seg.len;
    const int bh = b * p.Hkv + h;
    const int n_new = kv8::seq_new(p, b);
    const int n_rows = n_new * p.group;  // valid rows, kRows at most
    const int min_end = row_end(p, len, n_new, 0);
    if (seg.pos >= 0 && lane == 0)  // it begins here
      p.own_info[bh] =
          make_int2(gw, cut.owner(first + seg.end - 1) - gw + 1);

    // This lane's two query rows per 8-row group (columns of S^T): how many
    // tokens they see.
    int vis[NT][2];
    uint32_t bq[NT][kKSteps][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g8;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(
          p.q + (r < n_rows ? q_row_index(p, b, h, r) * D : 0));
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          bq[nt][ks][i] = r < n_rows ? __ldg(q + 8 * ks + 4 * i + c) : 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 8 * nt + 2 * c + e;
        vis[nt][e] = rr < n_rows ? row_end(p, len, n_new, rr) : len;
      }
    }

    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kv8::kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    const int last = min(seg.end, count);  // end of the warp's part
    for (int pos = max(seg.pos, 0); pos < last; ++pos) {
      ptx::cp_async_wait<kFewStages - 1>();
      __syncwarp();
      const uint32_t tile = ring + stage * 2 * kFewTile;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int key0 = (pos - seg.pos) * kKeys + 16 * u;
        if (key0 >= len) continue;
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < kKSteps; ++ks) {
          uint32_t a[4];
          ldmatrix4(a, tile + chunk_at<D>(16 * u + k_row, 2 * ks + k_col));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<kBF16>(s[nt], a, bq[nt][ks][0], bq[nt][ks][1]);
        }
        // Scores in log2 units; hidden ones are -inf.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] *= mult;
        if (key0 + 16 > min_end) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + g8 + 8 * (e >> 1) >= vis[nt][e & 1])
                s[nt][e] = -INFINITY;
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
              for (int i = 0; i < D / 16; ++i) {
                o[nt][i][e] *= alpha;
                o[nt][i][e + 2] *= alpha;
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // A hidden score is -inf, m never is: 0; NaN stays NaN.
            w[e] = ptx::ex2((s[nt][e] - m[nt][e & 1]) + kShift);
            l[nt][e & 1] += w[e];
          }
          pb[nt][0] = ptx::movmatrix_trans(ptx::pack2<kBF16>(w[0], w[1]));
          pb[nt][1] = ptx::movmatrix_trans(ptx::pack2<kBF16>(w[2], w[3]));
        }
        // O^T += V^T P^T: row i of a thread's O is element 16 i + g8 (+ 8).
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t a[4];
          ldmatrix4_trans(a, tile + kFewTile +
                                 chunk_at<D>(16 * u + v_row, 2 * i + v_col));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<kBF16>(o[nt][i], a, pb[nt][0], pb[nt][1]);
        }
      }
      __syncwarp();  // the tile has been read
      ld.next(p, count, tile, lane);
      stage = stage + 1 == kFewStages ? 0 : stage + 1;
    }

    // The part's averages and LSEs to its slot.
    const long long slot = static_cast<long long>(gw) + bh;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * c + e;
        float sum = l[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (r >= n_rows) continue;
        const bool seen = sum != 0.f;
        const float inv = seen ? 1.f / sum : 0.f;
        float* dst = p.few_o + (slot * kRows + r) * D + g8;
        if (seen) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            dst[16 * i] = o[nt][i][e] * inv;
            dst[16 * i + 8] = o[nt][i][e + 2] * inv;
          }
        }
        if (g8 == 0)
          p.few_lse2[slot * kRows + r] =
              seen ? m[nt][e] + log2f(sum) - kShift : -INFINITY;
      }
    if (seg.end >= count) break;
    few_next<D>(p, seg);
    if (seg.pos >= count) break;
  }
}

}  // namespace prefix
}  // namespace attn
