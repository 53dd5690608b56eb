// Attention of up to 16 query rows per K/V head over each sequence's own keys,
// behind a shared prefix.
//
// Mathematics: flash-decoding, as the few-row kernel of the 8-bit cache does
// it.  The keys of all (sequence, K/V head) segments form one list of tiles (4
// KB of keys), cut into equal consecutive shares, one per CTA; a CTA's warps
// take its tiles in turn, each with its own running maximum, sum and
// accumulator, which meet in shared memory at the end of a segment.  A result
// goes to workspace slot (CTA + segment) and is joined with the others and the
// prefix's by the merge kernel.
//
// Products: S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16, 16 keys (or
// 16 of D) by 8 query rows: a 128-row tcgen05 tile would be nearly empty, and
// the bytes of K and V bound the kernel.  P is rounded to the inputs' type and
// held times 2^kShift as in the many-row kernel.
//
// Tiles reach shared memory by 16-byte asynchronous copies, a ring per warp
// that runs ahead across segments; rows past a length are filled with zeros
// and read nothing.  Chunk j of row r lies at chunk j ^ r % 8, so that
// ldmatrix reads share no banks.
//
// The kernel reads what was there before the prefix's kernel ahead of it, not
// that one's results: it starts while that one drains, and waits for it only
// at its end (so that the merge behind has waited for both).
#include "prefix_common.cuh"

namespace attn {
namespace prefix {
namespace {

using kv8::kNone;
using kv8::Segment;

constexpr float kTau = 8.f;  // lazy rescale threshold (log2 units)

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(y)
               : "r"(x));
  return y;
}

// 16-byte asynchronous copy past L1; zeros, and nothing read, unless `in`.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst,
                                                   const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

template <int D, int NT>
struct Config {
  static constexpr int kRows = 8 * NT;
  static constexpr int kThreads = 32 * kFewWarps;
  static constexpr int kCtas = few_ctas(D, kRows);
  static constexpr int kStages = NT == 1 ? 3 : 2;
  static constexpr int kTile = 4096;     // bytes of K, and of V
  static constexpr int kPitch = D + 4;   // floats: rows start 4 banks apart
  static constexpr int kRingBytes = kFewWarps * kStages * 2 * kTile;
  static constexpr int kBytes =
      kRingBytes + kFewWarps * kRows * (kPitch + 2) * 4;
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory");
};

// Byte offset of 16-byte chunk j of row r in a tile.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int j) {
  return r * (2 * D) + ((j ^ (r & 7)) << 4);
}

// A warp's loads: they run ahead of its products, across segments.
template <int D, int NT>
struct Loader {
  using C = Config<D, NT>;
  static constexpr int kKeys = few_keys<D>();
  static constexpr int kPerRow = D / 8;          // chunks
  static constexpr int kRowStep = 32 / kPerRow;  // rows between a lane's chunks
  static constexpr int kChunks = C::kTile / 16 / 32;
  Segment seg;
  int pos;                 // next tile, counted from the share's start
  const uint16_t* k;       // this lane's first chunk of the segment
  const uint16_t* v;
  uint32_t ring;

  __device__ __forceinline__ void set_segment(const PrefixParams& p,
                                              int lane) {
    const long long at =
        (static_cast<long long>(seg.b) * p.Hkv + seg.h) * p.capacity * D +
        8 * lane;
    k = p.k + at;
    v = p.v + at;
  }
  __device__ __forceinline__ void init(const PrefixParams& p,
                                       const Segment& s, int warp, int lane,
                                       uint32_t ring_) {
    seg = s;
    pos = warp;
    ring = ring_;
    set_segment(p, lane);
  }
  __device__ __forceinline__ void next(const PrefixParams& p, int count,
                                       int stage, int lane) {
    bool moved = false;
    while (pos < count) {
      if (pos >= seg.end) {
        kv8::next_segment<kKeys, kFewOver>(p, seg);
        moved = true;
      } else if (pos < seg.pos) {
        pos += kFewWarps;
      } else {
        break;
      }
    }
    if (pos < count) {
      if (moved) set_segment(p, lane);
      const int t = pos - seg.pos;
      const long long off = static_cast<long long>(t) * kKeys * D;
      const uint32_t to = ring + stage * 2 * C::kTile;
      const int r0 = lane / kPerRow, j = lane % kPerRow;
      const int left = seg.len - t * kKeys - r0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int r = r0 + i * kRowStep;
        const uint32_t dst = to + chunk_at<D>(r, j);
        const bool in = i * kRowStep < left;
        const long long at = in ? off + i * kRowStep * D : 0;
        if (left >= kKeys) {
          cp_async16(dst, k + off + i * kRowStep * D);
          cp_async16(dst + C::kTile, v + off + i * kRowStep * D);
        } else {
          cp_async16_or_zero(dst, k + at, in);
          cp_async16_or_zero(dst + C::kTile, v + at, in);
        }
      }
      pos += kFewWarps;
    }
    cp_async_commit();
  }
};

template <int D, int NT, bool kBF16>
__device__ __forceinline__ void few_rows_share(const PrefixParams& p) {
  using C = Config<D, NT>;
  constexpr int kWarps = kFewWarps;
  constexpr int kRows = C::kRows;
  constexpr int kPitch = C::kPitch;
  constexpr int kStages = C::kStages;
  constexpr int kKeys = few_keys<D>();
  constexpr int kSub = kKeys / 16;  // 16-key steps per tile
  constexpr int kKSteps = D / 16;
  constexpr float kShift = kBF16 ? -24.f : 7.f;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sm_o = reinterpret_cast<float*>(smem + C::kRingBytes);
  float* sm_m = sm_o + kWarps * kRows * kPitch;  // [kWarps][kRows]
  float* sm_l = sm_m + kWarps * kRows;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g8 = lane / 4, c = lane % 4;
  const int cta = blockIdx.x;
  Segment seg;
  seg.pos = 0;
  const int count =
      kv8::take_share<kKeys, kFewOver, kWarps>(p, cta, lane, &seg);
  if (seg.pos >= count) return;  // (also: no share)
  const uint32_t ring =
      ptx::smem_u32(smem) + warp * kStages * 2 * C::kTile;
  Loader<D, NT> ld;
  ld.init(p, seg, warp, lane, ring);
#pragma unroll
  for (int i = 0; i < kStages; ++i) ld.next(p, count, i, lane);
  // This lane's rows of ldmatrix's four 8 x 8 matrices: of K (keys 0-7 and
  // 8-15, then the next 8 of D) and of V (the next 8 of D, then keys 8-15).
  const int k_row = lane % 8 + 8 * ((lane / 8) & 1), k_col = lane / 16;
  const int v_row = lane % 8 + 8 * (lane / 16), v_col = (lane / 8) & 1;
  const float mult = p.negate ? -p.scale_log2 : p.scale_log2;

  int stage = 0;
  int pos = warp;  // this warp's next tile
  while (true) {
    const int seg_last = min(seg.end, count);  // end of the CTA's part
    const int b = seg.b, h = seg.h, len = seg.len;
    const int n_new = kv8::seq_new(p, b);
    const int n_rows = n_new * p.group;  // valid rows, kRows at most
    const int min_end = n_rows > 0 ? kv8::row_end(p, len, n_new, 0) : 0;
    const int max_end = n_rows > 0 ? len : 0;

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
        vis[nt][e] = rr < n_rows ? kv8::row_end(p, len, n_new, rr) : len;
      }
    }

    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    while (pos < seg.pos) pos += kWarps;
    for (; pos < seg_last; pos += kWarps) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t tile = ring + stage * 2 * C::kTile;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int key0 = (pos - seg.pos) * kKeys + 16 * u;
        if (key0 >= max_end) continue;  // no rows, or past the length
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
        bool grow = false;
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
          pb[nt][0] = movmatrix_trans(ptx::pack2<kBF16>(w[0], w[1]));
          pb[nt][1] = movmatrix_trans(ptx::pack2<kBF16>(w[2], w[3]));
        }
        // O^T += V^T P^T: row i of a thread's O is element 16 i + g8 (+ 8).
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t a[4];
          ldmatrix4_trans(a, tile + C::kTile +
                                 chunk_at<D>(16 * u + v_row, 2 * i + v_col));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<kBF16>(o[nt][i], a, pb[nt][0], pb[nt][1]);
        }
      }
      __syncwarp();  // the tile has been read
      ld.next(p, count, stage, lane);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // The warps' results meet: maxima, then O and l under the common ones.
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
        float mx = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w * kRows + r]);
        const float f = ptx::ex2(m[nt][e] - mx);
        if (g8 == 0) sm_l[warp * kRows + r] = l[nt][e] * f;
        float* dst = sm_o + (warp * kRows + r) * kPitch + g8;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          dst[16 * i] = o[nt][i][e] * f;
          dst[16 * i + 8] = o[nt][i][e + 2] * f;
        }
      }
    __syncthreads();
    const long long slot =
        static_cast<long long>(cta) + static_cast<long long>(b) * p.Hkv + h;
    for (int i = threadIdx.x; i < n_rows * (D / 4); i += C::kThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f, mx = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(
            sm_o + (w * kRows + r) * kPitch + 4 * d4);
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
        sum += sm_l[w * kRows + r];
        mx = fmaxf(mx, sm_m[w * kRows + r]);
      }
      const bool seen = sum != 0.f;
      const float inv = seen ? 1.f / sum : 0.f;
      if (seen)
        reinterpret_cast<float4*>(p.few_o)[(slot * kRows + r) * (D / 4) + d4] =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (d4 == 0)
        p.few_lse2[slot * kRows + r] =
            seen ? mx + log2f(sum) - kShift : -INFINITY;
    }
    if (seg.end >= count) break;
    kv8::next_segment<kKeys, kFewOver>(p, seg);
    if (seg.pos >= count) break;
  }
}

template <int D, int NT, bool kBF16>
__global__ void __launch_bounds__(Config<D, NT>::kThreads,
                                  Config<D, NT>::kCtas)
    prefix_few_kernel(const __grid_constant__ PrefixParams p) {
  ptx::griddep_launch_dependents();
  few_rows_share<D, NT, kBF16>(p);
  ptx::griddep_wait();
}

template <int D, int NT, bool kBF16>
cudaError_t launch(PrefixParams p, cudaStream_t stream) {
  using C = Config<D, NT>;
  p.grid = p.few_grid;
  const cudaError_t err = cudaFuncSetAttribute(
      prefix_few_kernel<D, NT, kBF16>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (err != cudaSuccess) return err;
  return kv8::launch_pdl(prefix_few_kernel<D, NT, kBF16>, p.few_grid,
                         C::kThreads, C::kBytes, stream, p);
}

template <int D, bool kBF16>
cudaError_t launch_dt(const PrefixParams& p, cudaStream_t stream) {
  return p.rows <= 8 ? launch<D, 1, kBF16>(p, stream)
                     : launch<D, 2, kBF16>(p, stream);
}

}  // namespace

cudaError_t launch_few(int D, bool bf16, const PrefixParams& p,
                       cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch_dt<64, true>(p, stream)
                : launch_dt<64, false>(p, stream);
  return bf16 ? launch_dt<128, true>(p, stream)
              : launch_dt<128, false>(p, stream);
}

}  // namespace prefix
}  // namespace attn
