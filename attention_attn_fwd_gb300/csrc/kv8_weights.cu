// Accumulated attention weights of many query rows over the 8-bit cache.
//
// w_j += sum over the rows i that see key j of 2^(s_ij - LSE_i), with the
// rows' LSEs (log2 units) of the forward launches ahead of this one.  The
// scores are computed again (a stored score would cost 8 bytes of traffic),
// keys as rows: S^T = K Q^T for 128 keys and 256 query rows at a time, by
// tcgen05 in fp16 with the operands of the many-row forward kernel (its header
// comment has the roundings).  A thread of the epilogue owns one key: it adds
// up its 256 columns, so no value crosses threads, and the rows' factors and
// LSEs are broadcast from shared memory.
//
// The key tiles of all (batch, K/V head) segments are cut into equal
// consecutive shares, one per CTA.  A pass is a segment's part of the share
// under 256 query rows: their fp16 tile stays in shared memory while the key
// tiles stream past it.  Tile j goes to accumulator and epilogue warpgroup
// j % 2 in every pass, so a key has one owner, which adds the passes in order:
// no atomics, one order of sums.
//
// Roles (512 threads): warp 0 MMA issue, warp 1 bulk copies of raw key tiles,
// warps 4-7 conversion of key tiles, warps 8-15 query rows, then the epilogue
// of even (8-11) and odd tiles.  Every wait is bounded as in the forward
// kernel.  Measured: 2 x 64 rows of 32 heads over 8192 tokens, 7 key tiles a
// CTA, 24 us of the call's 62 (8 GFLOP of products run again: 4 us at cuBLAS's
// rate).  The start and the query rows take about 13000 clocks, a tile 3400,
// the epilogue's time (its exp2 alone would take 1000); a loop of 32 columns
// is kept rolled, for its code is fetched anew in every launch (unrolled twice
// 63.2 us, whole 66; 64 columns a turn 66; columns loaded a turn ahead 66).
// The first form, on mma.sync, took 77 us.
#include "attn_sync.cuh"
#include "kv8_common.cuh"

namespace attn {
namespace kv8 {
namespace {

constexpr int kThreads = 512;
constexpr int kTN = 128;    // keys of a tile
constexpr int kRows = 256;  // query rows of a pass
// Empty places of the cut per segment, for its query rows (2 x 64 rows over
// 8192 tokens, 32 heads, forward included: 69.0 us without, with 2 / 4 / 8
// places 65.4 / 63.8 / 65.1).
constexpr int kOver = 4;

template <int D>
struct Smem {
  static constexpr int kBox = kTN * 128;            // 128 keys x 128 bytes
  static constexpr int kTile = kBox * (D / 64);     // one fp16 key tile
  static constexpr int kQBox = kRows * 128;
  static constexpr int kRaw = kTN * D;              // one raw key tile
  static constexpr int kSlots = 3, kRawSlots = 3;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + kQBox * (D / 64);
  static constexpr int kRawRing = kRing + kSlots * kTile;
  static constexpr int kConst = kRawRing + kRawSlots * kRaw;
  // Per pair of rows: both factors, both negated LSEs.
  static constexpr int kBars = kConst + kRows * 8;
  // raw_full, raw_empty, full, empty, q, qfree, s[2], sfree[2], drain
  static constexpr int kNumBars = 2 * kRawSlots + 2 * kSlots + 7;
  static constexpr int kMisc = kBars + 8 * kNumBars;  // TMEM base, abort
  static constexpr int kBytes = kMisc + 8;
  static_assert(kBytes + 1024 <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// (x0, x1) * (m0, m1) + (a0, a1).
__device__ __forceinline__ void ffma2_pairs(float& y0, float& y1, float x0,
                                            float x1, float m0, float m1,
                                            float a0, float a1) {
  asm("{\n\t.reg .b64 x, m, a, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 m, {%4, %5};\n\t"
      "mov.b64 a, {%6, %7};\n\t"
      "fma.rn.ftz.f32x2 y, x, m, a;\n\t"
      "mov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y0), "=f"(y1)
      : "f"(x0), "f"(x1), "f"(m0), "f"(m1), "f"(a0), "f"(a1));
}

// 32 query rows to fp16 operand rows in shared memory (128-byte swizzled boxes
// of `box` bytes, the first row at `dst`, a multiple of 8 rows from its box's
// start), each times its row_shift's power of two.
// `off`: this lane's row, in elements from q, or -1 (zeros).  Returns the
// shift of this lane's row.  The rows come by coalesced asynchronous copies
// and are converted where they land, a row per lane, in small loops: a row of
// loads per lane, unrolled, touched 32 lines with each load and fetched its
// instructions anew at every call (weights kernel 31 -> 26 us at 2 x 64 rows
// over 8192 tokens; the forward kernel, whose softmax warps hold their rows in
// registers, gained nothing from it).
template <int D, bool kBF16>
__device__ __forceinline__ int stage_rows(const void* q, long long off,
                                          uint32_t dst, uint32_t box,
                                          int lane) {
  constexpr int kChunks = D / 8;         // lanes of a row
  constexpr int kAtOnce = 32 / kChunks;  // rows of an instruction
  {
    const int c = lane % kChunks, sub = lane / kChunks;
    const uint32_t to = dst + (c / 8) * box;
#pragma unroll 2
    for (int row = sub; row < 32; row += kAtOnce) {
      const long long at = __shfl_sync(0xffffffffu, off, row);
      const uint32_t d = to + row * 128 + (((c % 8) ^ (row % 8)) << 4);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                   "l"(static_cast<const uint16_t*>(q) +
                       (at < 0 ? 0 : at + 8 * c)),
                   "r"(at < 0 ? 0 : 16)
                   : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const uint32_t mine = dst + lane * 128;
  float amax = 0.f;
#pragma unroll 4
  for (int k = 0; k < kChunks; ++k) {
    const uint4 x = ptx::ld_shared_v4(mine + (k / 8) * box +
                                      (((k % 8) ^ (lane % 8)) << 4));
    const float2 a = unpack2<kBF16>(x.x), b = unpack2<kBF16>(x.y);
    const float2 c = unpack2<kBF16>(x.z), d = unpack2<kBF16>(x.w);
    amax = ptx::fmax3(amax, fabsf(a.x), fabsf(a.y));
    amax = ptx::fmax3(amax, fabsf(b.x), fabsf(b.y));
    amax = ptx::fmax3(amax, fabsf(c.x), fabsf(c.y));
    amax = ptx::fmax3(amax, fabsf(d.x), fabsf(d.y));
  }
  const int up = row_shift(amax);
  const float f = exp2_int(up);
#pragma unroll 2
  for (int k = 0; k < kChunks; ++k) {
    const uint32_t at = mine + (k / 8) * box + (((k % 8) ^ (lane % 8)) << 4);
    const uint4 x = ptx::ld_shared_v4(at);
    const float2 a = unpack2<kBF16>(x.x), b = unpack2<kBF16>(x.y);
    const float2 c = unpack2<kBF16>(x.z), d = unpack2<kBF16>(x.w);
    ptx::st_shared_v4(at, ptx::pack2<false>(a.x * f, a.y * f),
                      ptx::pack2<false>(b.x * f, b.y * f),
                      ptx::pack2<false>(c.x * f, c.y * f),
                      ptx::pack2<false>(d.x * f, d.y * f));
  }
  return up;
}

// The passes of a CTA's share, walked alike by every role: tiles [t0, t1) of
// a segment, query rows [256 u, 256 u + 256), of which tiles [t0, hi) see
// some.
struct Passes {
  Segment seg;
  int count;         // tiles of the share
  int t0, t1, hi;
  int u, n_new, rows;

  __device__ __forceinline__ void enter(const FwdParams& p) {
    n_new = seq_new(p, seg.b);
    rows = n_new * p.group;
    t0 = max(0, -seg.pos);
    t1 = min(seg.end, count) - seg.pos;
    u = 0;
    set_hi(p);
  }
  __device__ __forceinline__ void set_hi(const FwdParams& p) {
    const int last = min(rows, (u + 1) * kRows) - 1;
    hi = last < u * kRows
             ? t0
             : min(t1, (row_end(p, seg.len, n_new, last) + kTN - 1) / kTN);
  }
  __device__ __forceinline__ bool first(const FwdParams& p, int lane) {
    count =
        take_share<kTN, kOver, 1>(p, static_cast<int>(blockIdx.x), lane, &seg);
    if (count == 0 || seg.pos >= count) return false;
    enter(p);
    return hi > t0 || next(p);
  }
  __device__ __forceinline__ bool next(const FwdParams& p) {
    do {
      if ((u + 1) * kRows < rows) {
        ++u;
        set_hi(p);
      } else {
        if (seg.end >= count) return false;
        next_segment<kTN, kOver>(p, seg);
        if (seg.pos >= count) return false;
        enter(p);
      }
    } while (hi <= t0);
    return true;
  }
};

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_weights_kernel(const FwdParams p, int lse2_rows) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_base = ptx::smem_u32(smem);
  const uint32_t bar_rfull = s_base + L::kBars;
  const uint32_t bar_rempty = bar_rfull + 8 * L::kRawSlots;
  const uint32_t bar_full = bar_rempty + 8 * L::kRawSlots;
  const uint32_t bar_empty = bar_full + 8 * L::kSlots;
  const uint32_t bar_q = bar_empty + 8 * L::kSlots;
  const uint32_t bar_qfree = bar_q + 8;
  const uint32_t bar_s = bar_qfree + 8;      // [2]
  const uint32_t bar_sfree = bar_s + 16;     // [2]
  const uint32_t bar_drain = bar_sfree + 16;
  float* consts = reinterpret_cast<float*>(smem + L::kConst);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc + 4);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x < L::kNumBars) {
    const uint32_t bar = s_base + L::kBars + 8 * threadIdx.x;
    // One arrival per warp of the role that fills or frees; raw loads and
    // MMAs arrive once.
    uint32_t count = 1;
    if ((bar >= bar_rempty && bar < bar_empty) ||
        (bar >= bar_sfree && bar < bar_drain))
      count = 4;
    if (bar == bar_q || bar == bar_qfree) count = 8;
    ptx::mbar_init(bar, count);
    if (threadIdx.x == 0) *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  // Tensor memory is taken behind the wait for the kernel ahead (which may
  // still have to take its own) and before the one behind may start.
  ptx::griddep_wait();
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  Passes w;
  const bool first = (warp < 2 || warp >= 4) && w.first(p, lane);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_launch_dependents();

  bool ok = true;
  auto wait = [&](uint32_t bar, int phase, int role) {
    return __all_sync(0xffffffffu, wait_bounded(bar, phase & 1, abort_flag, p,
                                                role)) != 0;
  };
  bool more = first;

  if (warp == 1) {
    // ------------------------------------------------------ raw key tiles
    int it = 0;
    for (; more && ok; more = w.next(p)) {
      const uint8_t* k =
          p.k + (static_cast<long long>(w.seg.b) * p.Hkv + w.seg.h) *
                    p.capacity * D;
      for (int j = w.t0; j < w.hi && ok; ++j, ++it) {
        const int slot = it % L::kRawSlots, use = it / L::kRawSlots;
        if (use > 0) ok = wait(bar_rempty + 8 * slot, use - 1, 1);
        if (!ok) break;
        const uint32_t bytes = min(kTN, w.seg.len - j * kTN) * D;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(bar_rfull + 8 * slot, bytes);
          bulk_load(s_base + L::kRawRing + slot * L::kRaw,
                    k + static_cast<long long>(j) * L::kRaw, bytes,
                    bar_rfull + 8 * slot);
        }
      }
    }
    if (!ok) {  // let the copies in flight land
      for (int i = max(0, it - L::kRawSlots); i < it; ++i)
        drain_wait(bar_rfull + 8 * (i % L::kRawSlots),
                   (i / L::kRawSlots) & 1, p);
    }
    __syncwarp();
  } else if (warp == 0) {
    // ---------------------------------------------------------- MMA issue
    const uint32_t idesc = ptx::idesc_f16(false, kTN, kRows, false, false);
    constexpr uint32_t kHi = ptx::sdesc_hi_sw128(1024);
    const uint32_t q_lo = ptx::sdesc_lo(s_base + L::kQ, 16);
    const uint32_t k_lo = ptx::sdesc_lo(s_base + L::kRing, 16);
    int it = 0, pass = 0, uses[2] = {0, 0};
    bool issued = false;
    for (; more && ok; more = w.next(p), ++pass) {
      ok = wait(bar_q, pass, 2);
      // (Warp-uniform to the compiler: descriptors in uniform registers.)
      const int j0 = __reduce_max_sync(0xffffffffu, w.t0);
      const int j1 = __reduce_max_sync(0xffffffffu, w.hi);
      for (int j = j0; j < j1 && ok; ++j, ++it) {
        const int slot = it % L::kSlots, buf = j & 1;
        ok = wait(bar_full + 8 * slot, it / L::kSlots, 2);
        const int used = buf ? uses[1] : uses[0];
        if (ok && used > 0) ok = wait(bar_sfree + 8 * buf, used - 1, 2);
        if (!ok) break;
        if (buf) ++uses[1]; else ++uses[0];
        ptx::tc_fence_after();
        const uint32_t a0 = k_lo + slot * (L::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ptx::mma_ss_elect(
              tmem + buf * kRows,
              a0 + (((kk / 4) * L::kBox + (kk % 4) * 32) >> 4),
              q_lo + (((kk / 4) * L::kQBox + (kk % 4) * 32) >> 4), kHi, idesc,
              kk > 0 ? 1u : 0u);
        ptx::tc_commit_elect(bar_s + 8 * buf);
        ptx::tc_commit_elect(bar_empty + 8 * slot);
        issued = true;
      }
    }
    if (!ok && issued) {  // the MMAs issued end before TMEM is released
      ptx::tc_commit_elect(bar_drain);
      drain_wait(bar_drain, 0, p);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // --------------------------------------------------------- conversion
    const int cw = warp - 4;
    const int tid = cw * 32 + lane;
    constexpr int kItems = D / 16;          // 16-byte chunks of a tile
    constexpr int kRowStep = kTN / kItems;  // rows between them
    int row0, ch;  // as in the forward kernel: no bank shared
    if constexpr (D == 128) {
      const int odd = (tid >> 2) & 1;
      row0 = 2 * (tid / 16) + odd;
      ch = (((tid >> 3) & 1) ^ odd) * 4 + (tid & 3);
    } else {
      row0 = tid / 4;
      ch = tid % 4;
    }
    const uint32_t raw_off = row0 * D + ch * 16;
    const uint32_t out_off = (ch / 4) * L::kBox + row0 * 128;
    const uint32_t out0 = out_off + ((((ch % 4) * 2) ^ (row0 % 8)) << 4);
    const uint32_t out1 = out_off + ((((ch % 4) * 2 + 1) ^ (row0 % 8)) << 4);
    int it = 0;
    for (; more && ok; more = w.next(p)) {
      for (int j = w.t0; j < w.hi && ok; ++j, ++it) {
        const int rslot = it % L::kRawSlots, slot = it % L::kSlots;
        const int valid = w.seg.len - j * kTN;  // rows that hold tokens
        ok = wait(bar_rfull + 8 * rslot, it / L::kRawSlots, 8);
        if (ok && it >= L::kSlots)
          ok = wait(bar_empty + 8 * slot, it / L::kSlots - 1, 8);
        if (!ok) break;
        const uint32_t raw = s_base + L::kRawRing + rslot * L::kRaw + raw_off;
        const uint32_t out = s_base + L::kRing + slot * L::kTile;
        uint4 x[kItems];
#pragma unroll
        for (int e = 0; e < kItems; ++e)
          x[e] = ptx::ld_shared_v4(raw + e * kRowStep * D);
        if (valid < kTN) {  // rows past the length: zeros
#pragma unroll
          for (int e = 0; e < kItems; ++e)
            if (row0 + e * kRowStep >= valid) x[e] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int e = 0; e < kItems; ++e) {
          uint32_t h[8];
          e4m3x4_to_half2(x[e].x, h[0], h[1]);
          e4m3x4_to_half2(x[e].y, h[2], h[3]);
          e4m3x4_to_half2(x[e].z, h[4], h[5]);
          e4m3x4_to_half2(x[e].w, h[6], h[7]);
          const uint32_t at = out + e * kRowStep * 128;
          ptx::st_shared_v4(at + out0, h[0], h[1], h[2], h[3]);
          ptx::st_shared_v4(at + out1, h[4], h[5], h[6], h[7]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {  // (the raw values have been used: see the forward)
          ptx::mbar_arrive(bar_full + 8 * slot);
          ptx::mbar_arrive(bar_rempty + 8 * rslot);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ----------------------------------------------------------- epilogue
    const int buf = (warp - 8) / 4;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16) +
                         buf * kRows;
    const int r = threadIdx.x % kTN;  // key of the tile
    const int q_row = (warp - 8) * 32 + lane;  // query row this lane brings
    int pass = 0, uses = 0;
    for (; more && ok; more = w.next(p), ++pass) {
      // The rows of the pass, once every tile of the one before has been
      // added up.
      if (pass > 0) ok = wait(bar_qfree, pass - 1, 4);
      if (!ok) break;
      {
        const int row = w.u * kRows + q_row;
        const bool in = row < w.rows;
        const int tok = row / p.group, hd = row - tok * p.group;
        float lse = INFINITY;  // no weight: rows past the last, and rows
        if (in) {              // that see nothing
          lse = p.lse2[(static_cast<long long>(w.seg.b) * p.Hkv + w.seg.h) *
                           lse2_rows + row];
          if (lse == -INFINITY) lse = INFINITY;
        }
        const int up = stage_rows<D, kBF16>(
            p.q,
            in ? ((static_cast<long long>(w.seg.b) * p.Hq +
                   w.seg.h * p.group + hd) * p.Sq + tok) * D
               : -1,
            s_base + L::kQ + (warp - 8) * 32 * 128, L::kQBox, lane);
        consts[(q_row / 2) * 4 + q_row % 2] = p.scale_log2 * exp2_int(-up);
        consts[(q_row / 2) * 4 + 2 + q_row % 2] = -lse;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_q);
      ok = wait(bar_q, pass, 4);
      const int bh = w.seg.b * p.Hkv + w.seg.h;
      const int first_row = w.u * kRows;
      const int n_rows = min(kRows, w.rows - first_row);
      const int seen = row_end(p, w.seg.len, w.n_new, first_row);
      for (int j = w.t0; j < w.hi && ok; ++j) {
        if ((j & 1) != buf) continue;
        const int key = j * kTN + r;
        const bool in = key < w.seg.len;
        float ks = 0.f, before = 0.f;
        float* at = p.weights + static_cast<long long>(bh) * p.capacity + key;
        if (in) {
          ks = __ldg(p.k_scale + static_cast<long long>(bh) * p.nblk +
                     (key >> p.block_shift));
          before = *at;
        }
        // Rows below `low` do not see the key (rows see more and more).
        int low = 0;
        if ((j + 1) * kTN > seen && p.causal)
          low = max(0, (key - (w.seg.len - w.n_new))) * p.group - first_row;
        const bool masked =
            __any_sync(0xffffffffu, low > 0 || n_rows < kRows) != 0;
        ok = wait(bar_s + 8 * buf, uses, 4);
        if (!ok) break;
        ++uses;
        ptx::tc_fence_after();
        float sm[4] = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](auto masked_tag) {
          constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll 1
          for (int q = 0; q < kRows / 32; ++q) {
            uint32_t s[32];
            ptx::tmem_ld32(t_s + 32 * q, s);
            ptx::tmem_wait_ld();
            const float4* c4 =
                reinterpret_cast<const float4*>(consts) + 16 * q;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 k = c4[e];
              float x0, x1;
              // (The factors first: a score reaches 2^30 times K's scale
              // before its row's factor, past fp32 under large scales.)
              ffma2_pairs(x0, x1, __uint_as_float(s[2 * e]),
                          __uint_as_float(s[2 * e + 1]), ks * k.x, ks * k.y,
                          k.z, k.w);
              float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              if constexpr (kMasked) {
                const int c0 = 32 * q + 2 * e;
                if (c0 < low || c0 >= n_rows) p0 = 0.f;
                if (c0 + 1 < low || c0 + 1 >= n_rows) p1 = 0.f;
              }
              if (e & 1)
                ptx::fadd2(sm[2], sm[3], p0, p1);
              else
                ptx::fadd2(sm[0], sm[1], p0, p1);
            }
          }
        };
        if (masked)
          add(BoolTag<true>{});
        else
          add(BoolTag<false>{});
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_sfree + 8 * buf);
        const float sum = (sm[0] + sm[1]) + (sm[2] + sm[3]);
        if (in && sum != 0.f) *at = before + sum;
      }
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(bar_qfree);
    }
    __syncwarp();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kBF16>
cudaError_t launch(const FwdParams& p, int lse2_rows, cudaStream_t stream) {
  constexpr int kBytes = Smem<D>::kBytes + 1024;
  const cudaError_t err = cudaFuncSetAttribute(
      kv8_weights_kernel<D, kBF16>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (err != cudaSuccess) return err;
  return launch_pdl(kv8_weights_kernel<D, kBF16>, p.grid, kThreads, kBytes,
                    stream, p, lse2_rows);
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
