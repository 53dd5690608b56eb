// Attention of many query rows per K/V head over the 8-bit cache.
//
// The query rows of a K/V head, token-major (row r = token r / group, head
// r % group), are cut into units of two 128-row Q tiles that share one
// stream of 128-key tiles.  S = Q K^T and O += P V run as tcgen05 MMAs with
// fp16 operands and fp32 accumulators in TMEM, as in the 16-bit forward
// kernel; what differs is that the operands do not exist in memory:
//   - E4M3 codes are fp16 values, so a warpgroup converts each raw tile from
//     one shared-memory ring into the 128-byte-swizzled fp16 tiles of
//     another (exactly).  K's block scales multiply the scores in fp32, 16
//     keys at a time; V's scale over 2^-7 of the largest one of the part's
//     keys (codes times 2^7 are fp16 numbers still) multiplies V's halves:
//     exact for powers of two within 2^22 of the largest, else two fp16
//     roundings, 2^-11 each as P's own.  Further below, numbers are off by
//     2^-23 of the largest scale at most: the factor's half loses bits below
//     2^-14 and is 0 below 2^-25, a distance of 2^32 (448 * 2^-32 < 2^-23), and
//     the product is rounded to multiples of 2^-24;
//   - each softmax thread brings its Q row to fp16 with a power of two
//     (exact down to 2^-37 of the row's largest element) and the sign of the
//     scale, while the previous unit's last products run.
// P is kept shifted by 2^7 (it is at most 2^15, and normal down to 2^-21 of
// its row's largest), as are the row sums, which take P unrounded.
//
// Steps (unit, key tile) form one list, with some empty places before each
// unit's, cut into equal consecutive shares, one per CTA: lengths come from
// device memory and the cut follows them, whether there are few units with
// many keys or many units.  (Units of short caches are left whole, see
// whole_units.)  A unit that one CTA covers is finished by it; the parts of
// any other go to workspace slots (a CTA has two at most: a unit begun before
// its share, one going on after it) and are joined by the merge kernel.
//
// Roles (512 threads): warp 0 MMA issue, warp 1 bulk copies of the raw
// tiles, warp 2 walks the share and publishes its units in shared memory,
// warps 4-7 / 8-11 Q conversion, softmax and epilogue of Q tile 0 / 1, warps
// 12-15 K and V conversion.  Every wait is bounded as in the forward kernel.
//
// Measured: 8 x 512 rows of 32 heads over 4096 tokens of 8 heads, D = 128,
// causal (258 GFLOP): 236 us, 1.09 PFLOP/s, against 187 for the 16-bit forward
// kernel on the same numbers.  A step (256 rows, 128 keys) takes about 3400
// clocks against 2048 of MMAs.  Conversion and exp2 are not most of that gap:
// with the conversion left out the call (then 238 us) took 223, with exp2 left
// out 235, with both 212.  The rest has not been traced; three converted slots
// that K and V share, and shared memory that carries both operands of Q K^T,
// the raw tiles and the converted ones, are what differs from the 16-bit
// kernel.  A fifth warpgroup for V's conversion took 268 (spills), raw tiles
// read past shared memory 255, four converted and two raw slots 262.
#include "attn_sync.cuh"
#include "kv8_common.cuh"

namespace attn {
namespace kv8 {
namespace {

constexpr int kThreads = 512;
constexpr int kTM = 128;            // rows of a Q tile
constexpr int kTN = 128;            // keys of a tile
constexpr int kUnitRows = 2 * kTM;
constexpr float kTau = 8.f;         // lazy rescale threshold (log2 units)
constexpr float kShift = 7.f;       // log2 of P's scale
// Below this, a unit of V times 1 over a row's sum (2^46 at most, P's scale in
// it) may be no normal number.
constexpr float kSmallUnit = 0x1p-80f;
// Registers: the launch gives every thread 128; the shares of the four
// warpgroups add up to 4 * 128.
constexpr int kRegsControl = 64;
constexpr int kRegsSoftmax = 192;
constexpr int kRegsConvert = 64;
static_assert(kRegsControl + 2 * kRegsSoftmax + kRegsConvert <= 4 * 128,
              "register split exceeds the launch allocation");

constexpr int kUnits = 4;  // published units held at a time
// Empty places of the list before each unit's steps: they stand for what a
// part of a unit takes besides them (query rows, the first tile's fill, the
// output: about 13000 clocks against 3400 a step), so that CTAs with more
// parts get fewer steps.  8 x 512 rows over 4096 tokens, 32 heads: CTAs took
// 398k to 438k clocks without, 238 us; with 2 / 4 / 6 places 234.5 / 232 / 232
// (2 x 64 rows over 8192: 77 -> 73 / 70 / 68; 4 x 200 rows over 1500, 16 heads:
// 23.0 -> 21.9 / 22.6 / 23.9).
constexpr int kOver = 4;

// A unit's part as the roles need it.
struct Record {
  int n_kv;       // key tiles of the part; 0: no more units
  int j0;         // first of them
  int b, h, len, n_new;
  int row0;       // first row of tile 0
  int slot;       // workspace slot of a part; -1: this CTA has all of the unit
  int n[2];       // key tiles each Q tile sees
  int full[2];    // tiles below this one are seen whole by each valid row
  float v_unit;   // V's unit of the part (by the converters)
};

template <int D>
struct Smem {
  static constexpr int kBox = kTN * 128;             // 128 rows x 128 bytes
  static constexpr int kTile = kBox * (D / 64);      // one fp16 tile
  static constexpr int kRaw = kTN * D;               // one raw tile
  // fp16 tiles: V_j and K_j+1 in use, the next being written.  Raw tiles:
  // as many bytes in flight as fit.
  static constexpr int kSlots = D == 128 ? 3 : 5;
  static constexpr int kRawSlots = D == 128 ? 4 : 8;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTile;
  static constexpr int kRawRing = kRing + kSlots * kTile;
  static constexpr int kBars = kRawRing + kRawSlots * kRaw;
  // raw_full, raw_empty, kv_full, kv_empty, unit_full, unit_empty, q[2],
  // s[2], p[2], o[2], drain
  static constexpr int kNumBars = 2 * kRawSlots + 2 * kSlots + 2 * kUnits + 9;
  static constexpr int kMisc = kBars + 8 * kNumBars;  // TMEM base, abort
  static constexpr int kRecords = kMisc + 8;
  static constexpr int kBytes = kRecords + kUnits * sizeof(Record);
  static_assert(kBytes + 1024 <= 227 * 1024, "shared memory per CTA");
};

// ------------------------------------------------------------- the list
// Key tiles rows [r0, r1) of a sequence with `rows` rows see.
__device__ __forceinline__ int tiles_seen(const FwdParams& p, int len,
                                          int n_new, int r0, int r1) {
  const int last = min(r1, n_new * p.group) - 1;
  if (last < r0) return 0;
  return (row_end(p, len, n_new, last) + kTN - 1) / kTN;
}

__device__ __forceinline__ int places(const FwdParams& p, int steps) {
  return steps == 0 ? 0 : p.whole ? 1 : steps + kOver;
}

// A unit, or the part of one, that a CTA works on: key tiles [j0, j1) of its
// `steps`.  Units are numbered (b, u, h), h fastest.
struct Unit {
  int b, u, h;
  int len, n_new, steps;
  int j0, j1;
};

__device__ __forceinline__ int pair_steps(const FwdParams& p, int i, int* len,
                                          int* n_new) {
  const int b = i / p.row_blocks, u = i - b * p.row_blocks;
  *len = seq_len(p, b);
  *n_new = seq_new(p, b);
  return tiles_seen(p, *len, *n_new, u * kUnitRows, (u + 1) * kUnitRows);
}

// Walks a CTA's share.  take() and next() are warp-collective and return
// whether there is a unit.
struct Walk {
  Unit w;
  int left;      // steps of the share behind this unit's part
  int cta;
  int n, q, rest;  // the cut: CTA c of n takes q steps, the first rest one more

  __device__ __forceinline__ int first(int c) const {
    return c * q + min(c, rest);
  }
  __device__ __forceinline__ int owner(int x) const {
    const int fat = rest * (q + 1);
    return x < fat ? x / (q + 1) : rest + (x - fat) / q;
  }
  __device__ __forceinline__ void set_pair(const FwdParams& p, int i) {
    w.b = i / p.row_blocks;
    w.u = i - w.b * p.row_blocks;
  }

  __device__ __forceinline__ bool take(const FwdParams& p, int cta_, int lane) {
    cta = cta_;
    const int pairs = p.B * p.row_blocks;
    int total = 0;
    for (int i = lane; i < pairs; i += 32) {
      int len, n_new;
      total += places(p, pair_steps(p, i, &len, &n_new));
    }
#pragma unroll
    for (int s = 16; s > 0; s /= 2)
      total += __shfl_xor_sync(0xffffffffu, total, s);
    total *= p.Hkv;
    if (total == 0) return false;
    n = min(p.grid, total);
    q = total / n;
    rest = total - q * n;
    if (cta >= n) return false;
    const int x = first(cta);
    const int count = first(cta + 1) - x;
    int base = 0;
    for (int i0 = 0; i0 < pairs; i0 += 32) {
      const int i = i0 + lane;
      int len = 0, n_new = 0, steps = 0;
      if (i < pairs) steps = pair_steps(p, i, &len, &n_new);
      const int t = places(p, steps) * p.Hkv;
      int incl = t;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > x);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        set_pair(p, i0 + l);
        const int off = x - base - __shfl_sync(0xffffffffu, incl - t, l);
        w.len = __shfl_sync(0xffffffffu, len, l);
        w.n_new = __shfl_sync(0xffffffffu, n_new, l);
        w.steps = __shfl_sync(0xffffffffu, steps, l);
        w.h = off / places(p, w.steps);
        if (p.whole) {
          w.j0 = 0;
          w.j1 = w.steps;
          left = count - 1;
          return true;
        }
        // Steps of the unit before the share (negative: empty places).
        const int at = off - w.h * places(p, w.steps) - kOver;
        w.j0 = max(0, at);
        w.j1 = min(w.steps, at + count);
        left = count - (w.j1 - at);
        return w.j1 > w.j0;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }

  __device__ __forceinline__ bool next(const FwdParams& p) {
    if (left <= (p.whole ? 0 : kOver)) return false;
    if (++w.h == p.Hkv) {
      w.h = 0;
      int i = w.b * p.row_blocks + w.u;
      do {  // some later unit has steps: the share is not at its end
        ++i;
        w.steps = pair_steps(p, i, &w.len, &w.n_new);
      } while (w.steps == 0);
      set_pair(p, i);
    }
    w.j0 = 0;
    w.j1 = p.whole ? w.steps : min(w.steps, left - kOver);
    left -= places(p, w.j1);
    return true;
  }
};

__device__ __forceinline__ long long q_row_index(const FwdParams& p, int b,
                                                 int h, int r) {
  const int tok = r / p.group, hd = r - tok * p.group;
  return (static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq + tok;
}

__device__ __forceinline__ void fill_record(const FwdParams& p,
                                            const Walk& walk,
                                            volatile Record* rec) {
  const Unit& w = walk.w;
  rec->n_kv = w.j1 - w.j0;
  rec->j0 = w.j0;
  rec->b = w.b;
  rec->h = w.h;
  rec->len = w.len;
  rec->n_new = w.n_new;
  rec->row0 = w.u * kUnitRows;
  const bool whole = w.j0 == 0 && w.j1 == w.steps;
  rec->slot = whole ? -1 : 2 * walk.cta + (w.j0 == 0 ? 1 : 0);
  for (int t = 0; t < 2; ++t) {
    const int r0 = w.u * kUnitRows + t * kTM;
    const int hi = tiles_seen(p, w.len, w.n_new, r0, r0 + kTM);
    rec->n[t] = max(0, min(hi, w.j1) - w.j0);
    rec->full[t] = row_end(p, w.len, w.n_new, r0) / kTN;
  }
}

// Rows of units without steps (empty sequences, or rows before the first
// token) see nothing: the warp writes their O and LSE, each CTA its share of
// the units.
template <int D>
__device__ __forceinline__ void write_unseen(const FwdParams& p, int lane) {
  for (int i = blockIdx.x; i < p.B * p.row_blocks; i += gridDim.x) {
    int len, n_new;
    if (pair_steps(p, i, &len, &n_new) > 0) continue;
    const int b = i / p.row_blocks, r0 = (i - b * p.row_blocks) * kUnitRows;
    const int n = min(kUnitRows, n_new * p.group - r0);
    for (int j = lane; j < n * p.Hkv; j += 32) {
      const int h = j / n, r = r0 + j - h * n;
      const long long row = q_row_index(p, b, h, r);
      uint4* dst =
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D);
      for (int k = 0; k < D / 8; ++k) dst[k] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr) p.lse[row] = -INFINITY;
      if (p.lse2 != nullptr)
        p.lse2[(static_cast<long long>(b) * p.Hkv + h) * p.row_blocks *
                   kUnitRows + r] = -INFINITY;
    }
  }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// One 32-byte sector: a thread's row stores then fill sectors whole (16-byte
// stores of rows 256 or 512 bytes apart leave half-written ones behind).
__device__ __forceinline__ void store32(void* dst, const uint32_t* x) {
  asm volatile(
      "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]),
      "r"(x[6]), "r"(x[7])
      : "memory");
}
__device__ __forceinline__ void store_row(uint4* dst, const uint32_t* x,
                                          bool wide) {
  if (wide) {
    store32(dst, x);
  } else {
    dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
    dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// ------------------------------------------------------------ the kernel
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_prefill_kernel(const FwdParams p) {
  using L = Smem<D>;
  constexpr int kOCol = 2 * kTN;  // TMEM: S0, S1, then O0, O1
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_base = ptx::smem_u32(smem);
  const uint32_t bar_rfull = s_base + L::kBars;
  const uint32_t bar_rempty = bar_rfull + 8 * L::kRawSlots;
  const uint32_t bar_full = bar_rempty + 8 * L::kRawSlots;
  const uint32_t bar_empty = bar_full + 8 * L::kSlots;
  const uint32_t bar_unit = bar_empty + 8 * L::kSlots;  // [kUnits]
  const uint32_t bar_ufree = bar_unit + 8 * kUnits;     // [kUnits]
  const uint32_t bar_q = bar_ufree + 8 * kUnits;        // [2]
  const uint32_t bar_s = bar_q + 16;                    // [2]
  const uint32_t bar_p = bar_s + 16;                    // [2]
  const uint32_t bar_o = bar_p + 16;                    // [2]
  const uint32_t bar_drain = bar_o + 16;                // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc + 4);
  volatile Record* records = reinterpret_cast<Record*>(smem + L::kRecords);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x < L::kNumBars) {
    const uint32_t bar = s_base + L::kBars + 8 * threadIdx.x;
    // Converted tiles, freed raw tiles and Q tiles: one arrival per warp of
    // the four; units read: one per warp of the other roles (14); P: one per
    // softmax thread of the tile.
    uint32_t count = 1;
    if ((bar >= bar_rempty && bar < bar_empty) ||
        (bar >= bar_q && bar < bar_s))
      count = 4;
    if (bar >= bar_ufree && bar < bar_q) count = 14;
    if (bar >= bar_p && bar < bar_o) count = kTM;
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
  // The k-th unit, nullptr at the end of the share (or on abort); and its
  // release by this warp.
  auto get_unit = [&](int k) -> volatile Record* {
    ok = wait(bar_unit + 8 * (k % kUnits), k / kUnits, 1);
    if (!ok) return nullptr;
    volatile Record* rec = records + k % kUnits;
    return rec->n_kv > 0 ? rec : nullptr;
  };
  auto release_unit = [&](int k) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar_ufree + 8 * (k % kUnits));
  };

  if (warp < 4) {
    ptx::setmaxnreg_dec<kRegsControl>();
    if (warp == 2) {
      // ------------------------------------------------ units of the share
      Walk walk;
      bool more = walk.take(p, static_cast<int>(blockIdx.x), lane);
      // The unit that begins here and goes on in later CTAs, for the merge.
      int4 split = make_int4(0, 0, 0, 0);
      for (int k = 0; ok; ++k) {
        if (k >= kUnits)
          ok = wait(bar_ufree + 8 * (k % kUnits), k / kUnits - 1, 1);
        if (!ok) break;
        volatile Record* rec = records + k % kUnits;
        if (lane == 0) {
          if (more)
            fill_record(p, walk, rec);
          else
            rec->n_kv = 0;
          ptx::mbar_arrive(bar_unit + 8 * (k % kUnits));
        }
        __syncwarp();
        if (!more) break;
        const Unit& w = walk.w;
        if (w.j0 == 0 && w.j1 < w.steps) {
          const int last = walk.first(walk.cta + 1) - w.j1 + w.steps - 1;
          split = make_int4(w.b, w.h, w.u, walk.owner(last) - walk.cta + 1);
        }
        more = walk.next(p);
      }
      if (lane == 0) p.split[blockIdx.x] = split;
    } else if (warp == 3) {
      write_unseen<D>(p, lane);
    } else if (warp == 1) {
      // ---------------------------------------------------- raw tile loads
      int it = 0;
      for (int k = 0; ok; ++k) {
        volatile Record* rec = get_unit(k);
        if (rec == nullptr) break;
        const int n = rec->n_kv, j0 = rec->j0, len = rec->len;
        const long long head =
            (static_cast<long long>(rec->b) * p.Hkv + rec->h) * p.capacity * D;
        release_unit(k);
        for (int j = 0; j < n && ok; ++j) {
          const int key0 = (j0 + j) * kTN;
          const uint32_t bytes = min(kTN, len - key0) * D;
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = it % L::kRawSlots, use = it / L::kRawSlots;
            if (use > 0) ok = wait(bar_rempty + 8 * slot, use - 1, 1);
            if (!ok) break;
            if (lane == 0) {
              ptx::mbar_arrive_expect_tx(bar_rfull + 8 * slot, bytes);
              bulk_load(s_base + L::kRawRing + slot * L::kRaw,
                        (kv ? p.v : p.k) + head +
                            static_cast<long long>(key0) * D,
                        bytes, bar_rfull + 8 * slot);
            }
            ++it;
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
      // -------------------------------------------------------- MMA issue
      const uint32_t idesc_qk = ptx::idesc_f16(false, kTM, kTN, false, false);
      const uint32_t idesc_pv = ptx::idesc_f16(false, kTM, D, true, false);
      constexpr uint32_t kHi = ptx::sdesc_hi_sw128(1024);
      const uint32_t q_lo = ptx::sdesc_lo(s_base + L::kQ, 16);
      const uint32_t k_lo = ptx::sdesc_lo(s_base + L::kRing, 16);
      const uint32_t v_lo = ptx::sdesc_lo(s_base + L::kRing, L::kBox);
      constexpr uint32_t kTile16 = L::kTile >> 4;
      auto issue_qk = [&](int t, int slot) {
        const uint32_t a0 = q_lo + t * kTile16, b0 = k_lo + slot * kTile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * L::kBox + (kk % 4) * 32) >> 4;
          ptx::mma_ss_elect(tmem + t * kTN, a0 + off, b0 + off, kHi, idesc_qk,
                            kk > 0 ? 1u : 0u);
        }
        ptx::tc_commit_elect(bar_s + 8 * t);
      };
      auto issue_pv = [&](int t, int slot, bool acc) {
        const uint32_t b0 = v_lo + slot * kTile16;
#pragma unroll
        for (int kk = 0; kk < kTN / 16; ++kk)
          ptx::mma_ts_elect(tmem + kOCol + t * D, tmem + t * kTN + kk * 8,
                            b0 + ((kk * 16 * 128) >> 4), kHi, idesc_pv,
                            (acc || kk > 0) ? 1u : 0u);
      };
      int it = 0;  // converted tiles consumed
      int q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
      bool issued = false;
      for (int k = 0; ok; ++k) {
        ok = wait(bar_unit + 8 * (k % kUnits), k / kUnits, 1);
        if (!ok) break;
        // Through a warp reduction the counts are warp-uniform to the
        // compiler, and with them the ring position: descriptors then stay in
        // uniform registers (else every MMA moves them there first).
        volatile Record* rec = records + k % kUnits;
        const int n0 = __reduce_max_sync(0xffffffffu, rec->n[0]);
        const int n1 = __reduce_max_sync(0xffffffffu, rec->n[1]);
        const int n_kv = __reduce_max_sync(0xffffffffu, rec->n_kv);
        if (n_kv == 0) break;
        release_unit(k);
        ok = wait(bar_full + 8 * (it % L::kSlots), it / L::kSlots, 2);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = t ? n1 : n0;
          if (!ok || n == 0) continue;
          ok = wait(bar_q + 8 * t, q_uses[t], 2);
          if (!ok) break;
          ++q_uses[t];
          ptx::tc_fence_after();
          issue_qk(t, it % L::kSlots);
          issued = true;
        }
        if (!ok) break;
        ptx::tc_commit_elect(bar_empty + 8 * (it % L::kSlots));
        const int it0 = it;
        for (int j = 0; j < n_kv && ok; ++j) {
          const int it_v = it0 + 2 * j + 1, it_k = it0 + 2 * j + 2;
          const int slot_v = it_v % L::kSlots, slot_k = it_k % L::kSlots;
          ok = wait(bar_full + 8 * slot_v, it_v / L::kSlots, 2);
          if (!ok) break;
          bool k_ready = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int n = t ? n1 : n0;
            if (!ok || j >= n) continue;
            ok = wait(bar_p + 8 * t, p_uses[t], 2);
            if (!ok) break;
            ++p_uses[t];
            ptx::tc_fence_after();
            issue_pv(t, slot_v, j > 0);
            if (j == n - 1) {
              ptx::tc_commit_elect(bar_o + 8 * t);
              continue;
            }
            if (!k_ready) {
              ok = wait(bar_full + 8 * slot_k, it_k / L::kSlots, 2);
              if (!ok) break;
              k_ready = true;
              ptx::tc_fence_after();
            }
            issue_qk(t, slot_k);
          }
          if (!ok) break;
          ptx::tc_commit_elect(bar_empty + 8 * slot_v);
          if (j + 1 < n_kv) ptx::tc_commit_elect(bar_empty + 8 * slot_k);
        }
        it = it0 + 2 * n_kv;
      }
      if (!ok && issued) {  // the MMAs issued end before TMEM is released
        ptx::tc_commit_elect(bar_drain);
        drain_wait(bar_drain, 0, p);
      }
      __syncwarp();
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------- conversion
    ptx::setmaxnreg_dec<kRegsConvert>();
    const int cw = warp - 12;
    // Each thread converts one 16-byte raw chunk of every 16th (D = 64:
    // 32nd) row.  Eight lanes take four chunks of each of two rows: D = 128
    // the lower four of one row and the upper four of the next, so that
    // neither the reads nor the swizzled writes share a bank.
    constexpr int kItems = D / 16;
    constexpr int kRowStep = kTN / kItems;
    int row0, ch;
    {
      const int q = cw * 32 + lane;
      if constexpr (D == 128) {
        const int odd = (q >> 2) & 1;
        row0 = 2 * (q / 16) + odd;
        ch = (((q >> 3) & 1) ^ odd) * 4 + (q & 3);
      } else {
        row0 = q / 4;
        ch = q % 4;
      }
    }
    const uint32_t raw_off = row0 * D + ch * 16;
    const uint32_t out_off = (ch / 4) * L::kBox + row0 * 128;
    const uint32_t out0 = out_off + ((((ch % 4) * 2) ^ (row0 % 8)) << 4);
    const uint32_t out1 = out_off + ((((ch % 4) * 2 + 1) ^ (row0 % 8)) << 4);
    int it = 0;                 // tiles converted (K_0, V_0, K_1, ...)
    for (int k = 0; ok; ++k) {
      volatile Record* rec = get_unit(k);
      if (rec == nullptr) break;
      const int bh = rec->b * p.Hkv + rec->h;
      const int n_kv = rec->n_kv, j0 = rec->j0, len = rec->len;
      // Unit of V: 2^-7 of the largest scale of the part's keys.
      const float* vs = p.v_scale + static_cast<long long>(bh) * p.nblk;
      const int key_end = min(len, (j0 + n_kv) * kTN);
      float unit = 0x1p-119f;
      for (int i = ((j0 * kTN) >> p.block_shift) + lane;
           i <= (key_end - 1) >> p.block_shift; i += 32)
        unit = fmaxf(unit, __ldg(vs + i));
#pragma unroll
      for (int s = 16; s > 0; s /= 2)
        unit = fmaxf(unit, __shfl_xor_sync(0xffffffffu, unit, s));
      unit *= 0x1p-7f;
      if (cw == 0 && lane == 0) rec->v_unit = unit;
      const float inv_unit = 1.f / unit;
      release_unit(k);

      for (int i = 0; i < 2 * n_kv && ok; ++i) {
        const bool is_v = i & 1;
        const int rslot = it % L::kRawSlots, slot = it % L::kSlots;
        const int key0 = (j0 + (i >> 1)) * kTN;
        const int valid = len - key0;  // rows of the tile that hold tokens
        // V: lane g < 8 holds the factor of rows 16 g.. of the tile.
        float f_all = 1.f;
        if (is_v) {
          const int key = key0 + 16 * (lane & 7);
          if (key < len) f_all = __ldg(vs + (key >> p.block_shift)) * inv_unit;
        }
        ok = wait(bar_rfull + 8 * rslot, it / L::kRawSlots, 8);
        if (!ok) break;
        const uint32_t raw = s_base + L::kRawRing + rslot * L::kRaw + raw_off;
        const uint32_t out = s_base + L::kRing + slot * L::kTile;
        constexpr int kBatch = 4;  // chunks in registers at a time
#pragma unroll
        for (int e0 = 0; e0 < kItems; e0 += kBatch) {
          uint4 x[kBatch];
#pragma unroll
          for (int e = 0; e < kBatch; ++e)
            x[e] = ptx::ld_shared_v4(raw + (e0 + e) * kRowStep * D);
          if (valid < kTN) {  // rows past the length: zeros
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              if (row0 + (e0 + e) * kRowStep >= valid)
                x[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          if (e0 == 0 && it >= L::kSlots) {
            ok = wait(bar_empty + 8 * slot, it / L::kSlots - 1, 8);
            if (!ok) break;
          }
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            uint32_t h[8];
            e4m3x4_to_half2(x[e].x, h[0], h[1]);
            e4m3x4_to_half2(x[e].y, h[2], h[3]);
            e4m3x4_to_half2(x[e].z, h[4], h[5]);
            e4m3x4_to_half2(x[e].w, h[6], h[7]);
            if (is_v) {
              // Rows of this step lie in one 16-key group.
              const int g = D == 128 ? e0 + e : cw / 2 + 2 * (e0 + e);
              const float f = __shfl_sync(0xffffffffu, f_all, g);
              const uint32_t f2 = ptx::pack2<false>(f, f);
#pragma unroll
              for (int k = 0; k < 8; ++k) h[k] = hmul2(h[k], f2);
            }
            const uint32_t at = out + (e0 + e) * kRowStep * 128;
            ptx::st_shared_v4(at + out0, h[0], h[1], h[2], h[3]);
            ptx::st_shared_v4(at + out1, h[4], h[5], h[6], h[7]);
          }
        }
        if (!ok) break;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        // The raw tile is released only now that its values have been used: a
        // load that has been issued may still read shared memory after an
        // arrival issued behind it, when the next copy is already landing.
        if (lane == 0) {
          ptx::mbar_arrive(bar_full + 8 * slot);
          ptx::mbar_arrive(bar_rempty + 8 * rslot);
        }
        ++it;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------ softmax, correction, epilogue
    ptx::setmaxnreg_inc<kRegsSoftmax>();
    const int t = warp / 4 - 1;
    const int r = threadIdx.x % kTM;  // row within the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + t * kTN;
    const uint32_t t_o = tmem + lane_off + kOCol + t * D;
    int s_uses = 0, o_uses = 0;
    // This thread's Q row of unit `rec` to fp16 in shared memory; returns the
    // factor of its scores.  The buffer is free: every S of the tile has been
    // read.
    auto stage_q = [&](volatile Record* rec) -> float {
      const int row = rec->row0 + t * kTM + r;
      const bool in = row < rec->n_new * p.group;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) +
          (in ? q_row_index(p, rec->b, rec->h, row) * D : 0));
      uint32_t x[D / 2];
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint4 y = in ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
        x[4 * k] = y.x;
        x[4 * k + 1] = y.y;
        x[4 * k + 2] = y.z;
        x[4 * k + 3] = y.w;
      }
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < D / 2; ++k) {
        const float2 f = unpack2<kBF16>(x[k]);
        amax = ptx::fmax3(amax, fabsf(f.x), fabsf(f.y));
      }
      const int up = row_shift(amax);
      float f_up = exp2_int(up);
      if (p.scale_log2 < 0.f) f_up = -f_up;
      const uint32_t dst = s_base + L::kQ + t * L::kTile + r * 128;
      const uint32_t sw = r % 8;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float2 f = unpack2<kBF16>(x[4 * k + a]);
          o[a] = ptx::pack2<false>(f.x * f_up, f.y * f_up);
        }
        ptx::st_shared_v4(dst + (k / 8) * L::kBox + (((k % 8) ^ sw) << 4),
                          o[0], o[1], o[2], o[3]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_q + 8 * t);
      return fabsf(p.scale_log2) * exp2_int(-up);
    };
    volatile Record* rec = get_unit(0);
    float c_next = 0.f;
    if (rec != nullptr && rec->n[t] > 0) c_next = stage_q(rec);
    for (int k = 0; rec != nullptr; ++k) {
      const int n = rec->n[t], j0 = rec->j0, len = rec->len;
      const int full = rec->full[t];
      const float c = c_next;
      const float* ks_at =
          p.k_scale +
          (static_cast<long long>(rec->b) * p.Hkv + rec->h) * p.nblk;
      int vis;
      {
        const int row = rec->row0 + t * kTM + r, n_new = rec->n_new;
        vis = row < n_new * p.group ? row_end(p, len, n_new, row) : len;
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n; ++j) {
        const int key0 = (j0 + j) * kTN;
        // Lane g < 8 holds the K scale of keys 16 g.. of the tile.
        const int kg = key0 + 16 * (lane & 7);
        const float ks = kg < len ? __ldg(ks_at + (kg >> p.block_shift)) : 1.f;
        ok = wait(bar_s + 8 * t, s_uses, 4);
        if (!ok) break;
        ++s_uses;
        ptx::tc_fence_after();
        const bool masked = j0 + j >= full;
        const int lim = masked ? vis - key0 : kTN;
        uint32_t sr[kTN];
#pragma unroll
        for (int q = 0; q < kTN / 32; ++q) ptx::tmem_ld32(t_s + 32 * q, sr + 32 * q);
        ptx::tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int q = 0; q < kTN; ++q)
            if (q >= lim) sr[q] = __float_as_uint(-INFINITY);
        }
        // Factor of each 16 keys; held off 0 so that -inf stays -inf (scores
        // times 1e-37 vanish next to any maximum).
        float f[8];
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          f[g] = fmaxf(c * __shfl_sync(0xffffffffu, ks, g), 1e-37f);
          const uint32_t* x = sr + 16 * g;
          float a = ptx::fmax3(__uint_as_float(x[0]), __uint_as_float(x[1]),
                               __uint_as_float(x[2]));
          float b = ptx::fmax3(__uint_as_float(x[3]), __uint_as_float(x[4]),
                               __uint_as_float(x[5]));
          a = ptx::fmax3(a, __uint_as_float(x[6]), __uint_as_float(x[7]));
          b = ptx::fmax3(b, __uint_as_float(x[8]), __uint_as_float(x[9]));
          a = ptx::fmax3(a, __uint_as_float(x[10]), __uint_as_float(x[11]));
          b = ptx::fmax3(b, __uint_as_float(x[12]), __uint_as_float(x[13]));
          a = ptx::fmax3(a, __uint_as_float(x[14]), __uint_as_float(x[15]));
          mx = fmaxf(mx, fmaxf(a, b) * f[g]);
        }
        float m_new = m_run;
        if (__any_sync(0xffffffffu, mx > m_run + kTau)) m_new = fmaxf(m_run, mx);
        const float alpha = (m_new == -INFINITY) ? 1.f : ptx::ex2(m_run - m_new);
        const float neg_m = (m_new == -INFINITY) ? 0.f : kShift - m_new;
        float sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kTN / 32; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = 32 * q + 2 * e;
            float x0, x1;
            ptx::ffma2(x0, x1, __uint_as_float(sr[k]),
                       __uint_as_float(sr[k + 1]), f[k / 16], neg_m);
            const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
            if (e & 1)
              ptx::fadd2(sm[2], sm[3], p0, p1);
            else
              ptx::fadd2(sm[0], sm[1], p0, p1);
            pk[e] = ptx::pack2<false>(p0, p1);
          }
          ptx::tmem_st16(t_s + 16 * q, pk);
        }
        if (j > 0 && __any_sync(0xffffffffu, m_new != m_run)) {
          // O *= alpha (the PV before was issued before this S, whose commit
          // has been awaited).
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            ptx::tmem_ld32(t_o + 32 * q, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            ptx::tmem_st32(t_o + 32 * q, o);
          }
        }
        l_run *= alpha;
        ptx::tmem_wait_st();
        l_run += (sm[0] + sm[1]) + (sm[2] + sm[3]);
        m_run = m_new;
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar_p + 8 * t);
      }
      if (!ok) break;
      // The next unit's Q while this one's last products run.
      volatile Record* next = get_unit(k + 1);
      if (!ok) break;
      if (next != nullptr && next->n[t] > 0) c_next = stage_q(next);
      if (n > 0) {
        ok = wait(bar_o + 8 * t, o_uses, 4);
        if (!ok) break;
        ++o_uses;
        ptx::tc_fence_after();
      }
      const float unit = rec->v_unit;
      const int slot = rec->slot;
      const int row_u = rec->row0 + t * kTM + r;  // row of the K/V head
      const bool row_ok = row_u < rec->n_new * p.group;
      // O leaves as the average that it is: a sum of many large V could pass
      // fp32's largest.
      float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      if (unit >= kSmallUnit || n == 0) {
        inv *= unit;
      } else {
        // The factor would be a subnormal number: the average first.
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          ptx::tmem_ld32(t_o + 32 * q, o);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
          ptx::tmem_st32(t_o + 32 * q, o);
        }
        ptx::tmem_wait_st();
        inv = unit;
      }
      if (slot < 0) {
        const long long row =
            row_ok ? q_row_index(p, rec->b, rec->h, row_u) : 0;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) +
                                              row * D);
        // (O is 16-byte aligned, its rows whole 32-byte sectors from there.)
        const bool wide = reinterpret_cast<uintptr_t>(p.o) % 32 == 0;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (n > 0) {
            ptx::tmem_ld32(t_o + 32 * q, o);
            ptx::tmem_wait_ld();
          } else {  // no row of the tile sees a token
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (row_ok) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                // A row that sees nothing: 0, whatever its accumulator holds.
                const float a = __uint_as_float(o[16 * v + 2 * e]);
                const float b = __uint_as_float(o[16 * v + 2 * e + 1]);
                x[e] = l_run == 0.f ? 0u : ptx::pack2<kBF16>(a * inv, b * inv);
              }
              store_row(dst + 4 * q + 2 * v, x, wide);
            }
          }
        }
        if (row_ok) {
          const float lse2 = l_run == 0.f
                                 ? -INFINITY
                                 : (m_run == -INFINITY ? kNone : m_run) +
                                       log2f(l_run) - kShift;
          if (p.lse != nullptr) p.lse[row] = lse2 * 0.69314718055994531f;
          if (p.lse2 != nullptr)
            p.lse2[(static_cast<long long>(rec->b) * p.Hkv + rec->h) *
                       p.row_blocks * kUnitRows + row_u] = lse2;
        }
      } else {
        const long long at =
            static_cast<long long>(slot) * kUnitRows + t * kTM + r;
        float4* dst = reinterpret_cast<float4*>(p.part_o) + at * (D / 4);
        if (n > 0) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            ptx::tmem_ld32(t_o + 32 * q, o);
            ptx::tmem_wait_ld();
            if (row_ok) {
#pragma unroll
              for (int v = 0; v < 4; ++v) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  o[8 * v + e] =
                      __float_as_uint(__uint_as_float(o[8 * v + e]) * inv);
                store32(dst + 8 * q + 2 * v, o + 8 * v);
              }
            }
          }
        }
        if (row_ok)
          p.part_ml[at] =
              make_float2(m_run == -INFINITY ? kNone : m_run, l_run);
      }
      ptx::tc_fence_before();
      release_unit(k);
      rec = next;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ merge
// Joins the parts of the units that more than one CTA worked on: for each
// CTA's unit that went on behind it, a warp per row.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 32;
constexpr int kMergeParts = kUnitRows / kMergeRows;  // CTAs per unit
// log2 of the most parts, one per SM: their sum times V stays within fp32.
constexpr float kSlack = 8.f;

template <int D, bool kBF16>
__global__ void __launch_bounds__(kMergeThreads)
    kv8_prefill_merge_kernel(const FwdParams p) {
  constexpr int kCols = D / 4;  // float4 columns
  const int lane = threadIdx.x % 32;
  const int cta = blockIdx.x / kMergeParts;
  const int i = (blockIdx.x - cta * kMergeParts) * kMergeRows +
                threadIdx.x / 32;  // row of the unit
  start_after_previous();
  const int4 split = p.split[cta];
  const int b = split.x, h = split.y, parts = split.w;
  if (parts == 0) return;
  const int r = split.z * kUnitRows + i;
  if (r >= seq_new(p, b) * p.group) return;
  // Part s lies in slot 2 cta + 1 (s = 0) or 2 (cta + s).
  const long long at0 = (2LL * cta + 1) * kUnitRows + i;
  const long long at = 2LL * cta * kUnitRows + i;
  const int col = lane % kCols;
  // A part's weight: its LSE in log2 units (-inf: sees nothing).
  auto weight = [&](int s) {
    const float2 ml = p.part_ml[s == 0 ? at0 : at + 2LL * s * kUnitRows];
    return ml.x + __log2f(ml.y);
  };
  float mx = kNone;
  for (int s = lane; s < parts; s += 32) mx = fmaxf(mx, weight(s));
#pragma unroll
  for (int k = 16; k > 0; k /= 2)
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < parts; s0 += 32) {
    // Lane s: factor of part s0 + s.  (A part that sees nothing has the factor
    // 0 and no O.)
    const float f_all =
        s0 + lane < parts ? ptx::ex2((weight(s0 + lane) - mx) - kSlack) : 0.f;
    const int n = min(32, parts - s0);
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float f = __shfl_sync(0xffffffffu, f_all, s);
      // (Read in any case, so that the loads need not wait for f.)
      float4 y = reinterpret_cast<const float4*>(
          p.part_o)[(s0 + s == 0 ? at0 : at + 2LL * (s0 + s) * kUnitRows) *
                        kCols + col];
      if (f == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
      sum += f;
      acc.x += y.x * f;
      acc.y += y.y * f;
      acc.z += y.z * f;
      acc.w += y.w * f;
    }
  }
  const long long row = q_row_index(p, b, h, r);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (lane < kCols) {
    uint2 out;
    out.x = ptx::pack2<kBF16>(acc.x * inv, acc.y * inv);
    out.y = ptx::pack2<kBF16>(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D)[col] = out;
  }
  if (lane == 0) {
    const float lse2 =
        sum == 0.f ? -INFINITY : mx + log2f(sum) + (kSlack - kShift);
    if (p.lse != nullptr) p.lse[row] = lse2 * 0.69314718055994531f;
    if (p.lse2 != nullptr)
      p.lse2[(static_cast<long long>(b) * p.Hkv + h) * p.row_blocks *
                 kUnitRows + r] = lse2;
  }
}

// Whole units, each on one CTA and without a merge, or the list cut evenly:
// the shorter of the two in steps, for units as long as the cache's capacity
// (lengths are not known here).  Whole units take full rounds over the CTAs;
// cut ones another part's kOver and the merge, kOver steps too (about 7 us).
// Cut against whole, us, D = 128, 64 rows a head: 512 tokens of 2 heads 13.6
// against 11.8, of 128 22.8 against 14.2; 1024 of 2 13.7 against 17.4, of 128
// 29.4 against 20.4, of 512 79 against 68; 2048 of 32 22.0 against 30.0, of
// 128 39.7 against 31.8; 8 x 2048 rows of 8 heads over 4096 tokens 234 against
// 253.
bool whole_units(const FwdParams& p) {
  const long long units =
      static_cast<long long>(p.B) * p.Hkv * p.row_blocks;
  const long long each = (p.capacity - 1) / kTN + 1 + kOver;
  const long long rounds = (units + p.grid - 1) / p.grid;
  return rounds * each * p.grid <= units * each + 2LL * kOver * p.grid;
}

template <int D, bool kBF16>
cudaError_t launch(FwdParams p, cudaStream_t stream) {
  p.whole = whole_units(p);
  constexpr int kBytes = Smem<D>::kBytes + 1024;
  cudaError_t err = cudaFuncSetAttribute(
      kv8_prefill_kernel<D, kBF16>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (err != cudaSuccess) return err;
  err = launch_pdl(kv8_prefill_kernel<D, kBF16>, p.grid, kThreads, kBytes,
                   stream, p);
  if (err != cudaSuccess || p.whole) return err;
  return launch_pdl(kv8_prefill_merge_kernel<D, kBF16>,
                    static_cast<long long>(p.grid) * kMergeParts,
                    kMergeThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_prefill(int D, bool bf16, const FwdParams& p,
                           cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return bf16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace kv8
}  // namespace attn
