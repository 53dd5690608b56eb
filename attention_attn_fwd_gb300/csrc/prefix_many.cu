// Attention of many query rows over a shared prefix, and over the sequences'
// own keys where a K/V head has too many query rows for the few-row work (more
// than 16, or 8 of few sequences and heads: see Mode).
//
// The prefix's keys are the same for every sequence, so its query rows are
// packed across the batch: a 128-row Q tile holds the rows of as many
// sequences as fit, and two of them make a unit, which streams the prefix's
// 128-key tiles once.  With B sequences the prefix is read once instead of B
// times, and a decoding step's few rows fill the tensor cores' tiles.  Units
// of one sequence's rows take its own keys; where those rows fill a tile
// themselves (kJoint) its list of key tiles is the prefix's and then its own,
// and one pass makes the result.
//
// S = Q K^T and O += P V run as tcgen05 MMAs with fp32 accumulators in TMEM, K
// and V by tensor-map copies into a ring of 128-byte-swizzled tiles.  A tile
// that lengths end in is copied in boxes of 16 rows, its P V has as many 16-key
// steps, and a warp clears V's rows between the length and the last step's end
// (what lies there was never written and may be NaN; P is 0 there). P is
// rounded to the inputs' type, the tensor cores' operand (off by 2^-11 relative
// at most in fp16, 2^-8 in bf16, as O itself) and held times 2^kShift: in fp16,
// whose numbers end at 65504, so that weights stay normal down to 2^-21 of the
// row's largest; in bf16, whose V may come near fp32's largest number, so that
// sums of P V do not pass it (over 2^16 keys a part, 2^24 of like weights); a
// product is then off by 2^-150 at most, 2^-126 of O, which values of V below
// 2^-100 feel.  The row sums take P unrounded.
//
// The key tiles of all units form one list, with some empty places before each
// unit's, cut into equal consecutive shares, one per CTA: lengths come from
// device memory and the cut follows them.  A unit's parts are joined by the
// merge kernels (prefix_merge.cu).
//
// A tile is worked on in steps of 64 keys, two score buffers a Q tile, so that
// the tensor cores make one step's scores while the softmax works on the other:
// about 3000 clocks a tile of keys by 256 rows, D = 128 (1.5 us; 1.66 where a
// call is long enough for the power limit to lower the clock), of which the
// products' shared memory reads take 2560 (a 64-key product of scores reads 6 KB
// in the time of 4).  Steps of 128 keys took 1.6 to 1.75 us here: one score
// buffer is all that tensor memory holds of them beside O.
//
// What bounds it: those products, where rows are many and keys too; 8 prompts'
// chunks of 512 tokens, 32 heads, take 36 us and 1.66 for each of a CTA's key
// tiles: 205 to 215 us behind 3584 (103 tiles, 1.20 to 1.25 PFLOP/s), 391 behind
// 7680.  (Of the 36, about 8 are the start, 9 changes of units, 6 the join.)  The
// keys' bytes, the start (about 8 us: launch, lengths, cold instructions) and the
// parts' way through memory (128 KB a CTA) in a decoding step (64 sequences
// behind 8192 tokens: 44 to 46 us for 171 MB with the merge).
//
// Roles (384 threads): warps 0 and 2 MMA issue of Q tile 0 / 1, warp 1 tile
// copies, warp 3 walks the share, publishes its units in shared memory, copies
// their query rows and clears the ends of V, warps 4-7 / 8-11 softmax and
// output of Q tile 0 / 1.  (One warp for both tiles' products fell behind the
// tensor cores: 300 us where two took 205.)  Every wait is bounded as in the
// forward kernel.  Before a CTA ends, also after a wait that ran out in any of
// its roles, each role has seen what it started land: the copies in shared
// memory, the products in tensor memory, which is freed behind them.
//
// A Q tile is one copy by a tensor map whose box is (heads of the group,
// tokens, sequences), asked for as soon as the last S of the unit before is
// done. (Gathered by the softmax threads, a row each, it took them 3 to 5 us
// between two units; by one warp's 16-byte copies 2.5 to 4.)
#include "attn_sync.cuh"
#include "prefix_common.cuh"
#include "prefix_few.cuh"

namespace attn {
namespace prefix {
namespace {

using kv8::kNone;

constexpr int kThreads = 384;
constexpr int kHalf = kTN / 2;  // keys of a step
constexpr float kTau = 8.f;  // lazy rescale threshold (log2 units)
// Registers: the launch gives every thread 168; the shares of the three
// warpgroups add up to 3 * 168.
constexpr int kRegsControl = 72;
constexpr int kRegsSoftmax = 216;
static_assert(kRegsControl + 2 * kRegsSoftmax <= 3 * 168,
              "register split exceeds the launch allocation");

constexpr int kUnits = 4;  // published units held at a time
// Empty places of the list before a unit's key tiles, for what a part of a unit
// takes besides them.  64 sequences behind 8192 tokens, one new token each:
// 44.0 us, with 2 47.2, without 48.9; 32 behind 65531: 51.3, 52.9 and 57.5; but 8
// behind 4096, whose parts are short, 18.2, 18.3 and 17.6.
// None where a sequence's rows meet its own keys alone (kPacked), whose Q tile
// may be the other one than the unit's before, and whose key tiles take less
// time (32 sequences, 24 rows, 700 own keys behind 8192: 67 us; 75 with 4).
constexpr int kOver = 4;

// Tile maps: keys and values of the prefix and the sequences, whole tiles and
// boxes of their last ones; and the query rows.
struct Maps {
  CUtensorMap m[8];  // 4 * own + 2 * tail + (V)
  CUtensorMap q;
};

// Where a unit's part goes, other than a slot (>= 0).
constexpr int kFinal = -2, kBase = -1;

// A unit's part as the roles need it.
struct Record {
  int n_kv;       // key tiles of the part; 0: no more units
  int j0;         // first of them
  int np, plen;   // tiles and keys of the prefix in the unit's list
  int b, h, len, n_new;  // b < 0: rows of all sequences
  int tile0;      // first Q tile (-1: there is but tile 0, and it comes second)
  int dest;
  int n[2];       // key tiles each Q tile sees
};

template <int D>
struct Smem {
  static constexpr int kBox = kTN * 128;             // 128 rows x 128 bytes
  static constexpr int kTile = kBox * (D / 64);
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTile;
  static constexpr int kBars = kRing + kSlots * kTile;
  // kv_full, kv_empty [slots], unit_full, unit_empty, q[2], q_free[2],
  // s[2][2], p[2][2], pv[2], o[2], end, cleared, drain[2]
  static constexpr int kNumBars = 2 * kSlots + 2 * kUnits + 20;
  static constexpr int kMisc = kBars + 8 * kNumBars;  // TMEM base, abort
  static constexpr int kRecords = kMisc + 8;
  static constexpr int kBytes = kRecords + kUnits * sizeof(Record);
  static_assert(kBytes + 1024 <= 227 * 1024, "shared memory per CTA");
  static_assert(kFewWarps * kFewRing <= kBytes, "rings of the few rows");
};

// Valid keys of tile j of a unit's list, and whether it is the sequence's own.
__device__ __forceinline__ int tile_keys(int j, int np, int plen, int len,
                                         bool* own) {
  *own = j >= np;
  return *own ? min(kTN, len - (j - np) * kTN) : min(kTN, plen - j * kTN);
}

// ------------------------------------------------------------- the list
__device__ __forceinline__ int over(const PrefixParams& p, int i) {
  return p.mode == kPacked && i >= p.pack_blocks ? 0 : kOver;
}
__device__ __forceinline__ int places(const PrefixParams& p, int i,
                                      int steps) {
  return steps == 0 ? 0 : steps + over(p, i);
}

__device__ __forceinline__ kv8::Cut make_cut(int ctas, int total) {
  kv8::Cut c;
  c.n = max(1, min(ctas, total));
  c.q = total / c.n;
  c.rest = total - c.q * c.n;
  return c;
}

// kFew: CTAs that take the prefix, of those of the launch; the others take the
// sequences' own keys.  In proportion to the time that either takes an SM: a
// unit's key tile (256 rows) as long as 32 of the few rows' tiles where the
// prefix is 6 tiles a CTA (of all) or less, as 20 from 18 on, whose stream then
// keeps the memory busy and the own tiles waiting, and in even steps between.
// At 32 and at 20, us: 64 sequences, 8 K/V heads, 700 own keys behind 9472 tokens
// (4 a CTA) 52.7 and 58.6, behind 18944 (8) 58.5 and 64.0 (as it is 57.2), behind
// 28416 65.5 and 68.8 (64.0), behind 37888 (16) 73.4 and 73.5 (72.1), behind
// 85248 111 and 106; 24 sequences of 12 rows behind 9216 (8) 41.6 and 42.1, behind
// 41472 (34) 109 and 84.  (All at 26: 54.2, 59.3, 64.7, 70.5, 104, 39.9, 91.)  What
// is left over goes to the own keys: rounded to the nearest, 32 sequences of one
// own token behind 65536 took 61 us of 49, all own keys meeting one CTA.
__device__ __forceinline__ int prefix_ctas(const PrefixParams& p, int np,
                                           int few) {
  if (few == 0) return p.grid;
  if (np == 0) return 0;
  const float tiles = static_cast<float>(p.pack_blocks * p.Hkv) *
                      static_cast<float>(places(p, 0, np));
  const float far = 38.f * p.grid - tiles;  // 32 at 6 tiles a CTA, 20 at 18
  const float many = tiles * fmaxf(20.f * p.grid, fminf(32.f * p.grid, far));
  const int n = static_cast<int>(
      p.grid * (many / (many + static_cast<float>(few) * p.grid)));
  return max(1, min(n, p.grid - 1));
}

// A unit, or the part of one, that a CTA works on: [j0, j1) of its `steps` key
// tiles.  Units are numbered (i, h), h fastest: i < pack_blocks rows of all
// sequences, then (b, block).
struct Unit {
  int i, b, u, h;
  int len, n_new, steps;
  int j0, j1;
};

__device__ __forceinline__ int all_pairs(const PrefixParams& p) {
  return p.pack_blocks + p.B * p.row_blocks;
}

__device__ __forceinline__ int pair_steps(const PrefixParams& p, int np, int i,
                                          int* len, int* n_new) {
  if (i < p.pack_blocks) {
    *len = *n_new = 0;
    return np;
  }
  const int b = fast_div(i - p.pack_blocks, p.fd_blocks);
  const int u = i - p.pack_blocks - b * p.row_blocks;
  *len = kv8::seq_len(p, b);
  *n_new = kv8::seq_new(p, b);
  const int r0 = u * 2 * p.tile_rows;
  if (r0 >= *n_new * p.group) return 0;
  return tiles_seen(p, *len, *n_new, r0, r0 + 2 * p.tile_rows) +
         (p.mode == kJoint ? np : 0);
}

// Walks a CTA's share.  take() and next() are warp-collective and return
// whether there is a unit.
struct Walk {
  Unit w;
  int np;
  int left;      // places of the share behind this unit's part
  int cta;
  kv8::Cut cut;

  __device__ __forceinline__ void set_pair(const PrefixParams& p, int i) {
    w.i = i;
    if (i < p.pack_blocks) {
      w.b = -1;
      w.u = i;
    } else {
      w.b = fast_div(i - p.pack_blocks, p.fd_blocks);
      w.u = i - p.pack_blocks - w.b * p.row_blocks;
    }
  }

  // A share of `count` places that begins at place `off` of unit w.
  __device__ __forceinline__ bool start_at(const PrefixParams& p, int off,
                                           int count) {
    const int at = off - over(p, w.i);  // tiles before it (negative: places)
    w.j0 = max(0, at);
    w.j1 = min(w.steps, at + count);
    left = count - (w.j1 - at);
    return w.j1 > w.j0;
  }

  // The share of CTA cta_ of `ctas`.
  __device__ __forceinline__ bool take(const PrefixParams& p, int cta_,
                                       int ctas, int np_, int lane) {
    cta = cta_;
    np = np_;
    const int pairs = all_pairs(p);
    if (p.mode == kFew) {  // units alike
      const int each = places(p, 0, np);
      const int total = pairs * p.Hkv * each;
      if (total == 0) return false;
      cut = make_cut(ctas, total);
      if (cta >= cut.n) return false;
      const int x = cut.first(cta), count = cut.first(cta + 1) - x;
      const int unit = x / each, i = fast_div(unit, p.fd_hkv);
      set_pair(p, i);
      w.h = unit - i * p.Hkv;
      w.len = w.n_new = 0;
      w.steps = np;
      return start_at(p, x - unit * each, count);
    }
    int total = 0;
    for (int i = lane; i < pairs; i += 32) {
      int len, n_new;
      total += places(p, i, pair_steps(p, np, i, &len, &n_new));
    }
#pragma unroll
    for (int s = 16; s > 0; s /= 2)
      total += __shfl_xor_sync(0xffffffffu, total, s);
    total *= p.Hkv;
    if (total == 0) return false;
    cut = make_cut(ctas, total);
    if (cta >= cut.n) return false;
    const int x = cut.first(cta);
    const int count = cut.first(cta + 1) - x;
    int base = 0;
    for (int i0 = 0; i0 < pairs; i0 += 32) {
      const int i = i0 + lane;
      int len = 0, n_new = 0, steps = 0;
      if (i < pairs) steps = pair_steps(p, np, i, &len, &n_new);
      const int t = places(p, i, steps) * p.Hkv;
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
        const int each = places(p, w.i, w.steps);
        w.h = off / each;
        return start_at(p, off - w.h * each, count);
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }

  __device__ __forceinline__ bool next(const PrefixParams& p) {
    if (left <= 0) return false;
    if (++w.h == p.Hkv) {
      w.h = 0;
      int i = w.i;
      do {  // some later unit has steps: the share is not at its end
        ++i;
        w.steps = pair_steps(p, np, i, &w.len, &w.n_new);
      } while (w.steps == 0);
      set_pair(p, i);
    }
    if (left <= over(p, w.i)) return false;
    w.j0 = 0;
    w.j1 = min(w.steps, left - over(p, w.i));
    left -= places(p, w.i, w.j1);
    return true;
  }

  // The CTA that has the unit's last step.
  __device__ __forceinline__ int last_cta() const {
    return cut.owner(cut.first(cta + 1) - 1 - left - w.j1 + w.steps);
  }
};

__device__ __forceinline__ void fill_record(const PrefixParams& p,
                                            const Walk& walk, int plen,
                                            int swap, volatile Record* rec) {
  const Unit& w = walk.w;
  rec->n_kv = w.j1 - w.j0;
  rec->j0 = w.j0;
  const int np = w.b < 0 || p.mode == kJoint ? walk.np : 0;
  rec->np = np;
  rec->plen = plen;
  rec->b = w.b;
  rec->h = w.h;
  rec->len = w.len;
  rec->n_new = w.n_new;
  rec->tile0 = 2 * w.u - swap;
  const bool whole = w.j0 == 0 && w.j1 == w.steps;
  if (p.mode == kJoint)
    rec->dest = whole ? kFinal : walk.cta + (w.j0 == 0 ? p.grid : 0);
  else
    rec->dest = w.j0 == 0 ? kBase : walk.cta;
  for (int t = 0; t < 2; ++t) {
    const int tile = 2 * w.u - swap + t, r0 = tile * p.tile_rows;
    int hi = 0;
    if (w.b < 0) {
      if (tile * p.tile_seqs < p.B) hi = np;
    } else if (tile >= 0 && r0 < w.n_new * p.group) {
      hi = np + tiles_seen(p, w.len, w.n_new, r0, r0 + p.tile_rows);
    }
    rec->n[t] = max(0, min(hi, w.j1) - w.j0);
  }
}

// kJoint: rows of units without steps see nothing: the warp writes their O and
// LSE, each CTA its share of the units.  (Elsewhere the merge does.)
template <int D>
__device__ __forceinline__ void write_unseen(const PrefixParams& p, int lane) {
  if (p.mode != kJoint) return;
  const int np = prefix_tiles(p);
  for (int i = blockIdx.x; i < p.B * p.row_blocks; i += p.grid) {
    int len, n_new;
    if (pair_steps(p, np, i, &len, &n_new) > 0) continue;
    const int b = fast_div(i, p.fd_blocks);
    const int r0 = (i - b * p.row_blocks) * 2 * p.tile_rows;
    const int n = min(2 * p.tile_rows, n_new * p.group - r0);
    for (int j = lane; j < n * p.Hkv; j += 32) {
      const int h = j / n, r = r0 + j - h * n;
      const long long row = q_row_index(p, b, h, r);
      uint4* dst = reinterpret_cast<uint4*>(p.o + row * D);
      for (int k = 0; k < D / 8; ++k) dst[k] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr) p.lse[row] = -INFINITY;
    }
  }
}

// Row i of tile t of a unit: its sequence (-1: none) and row of the K/V head
// there.
__device__ __forceinline__ int row_of(const PrefixParams& p,
                                      volatile Record* rec, int t, int i,
                                      int* row) {
  const int tile = rec->tile0 + t;
  if (rec->b >= 0) {
    *row = tile * p.tile_rows + i;
    return tile >= 0 && i < p.tile_rows && *row < rec->n_new * p.group
               ? rec->b
               : -1;
  }
  const int s = fast_div(i, p.fd_rows);  // sequence within the tile
  const int b = tile * p.tile_seqs + s;
  *row = i - s * p.rows;
  if (s >= p.tile_seqs || b >= p.B) return -1;
  return *row < kv8::seq_new(p, b) * p.group ? b : -1;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m,
                                            uint32_t bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::"
      "complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}

// One 32-byte sector: a thread's row stores then fill sectors whole.
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
// S = Q K^T of D / 16 steps and its commit to `bar`, by one elected lane: one
// election for all of them (an election an instruction, and descriptors made
// between them, kept the issuing warp behind the tensor cores).  Descriptors as
// (lo, hi) words; a step's operands lie 32 bytes on, every fourth box by box.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a, uint32_t b,
                                             uint32_t hi, uint32_t idesc,
                                             uint32_t bar) {
#define ATTN_STEP(off, p)                                                   \
  "add.u32 la, %1, " off ";\n\tadd.u32 lb, %2, " off ";\n\t"              \
  "mov.b64 da, {la, %3};\n\tmov.b64 db, {lb, %3};\n\t"                    \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " p ";\n\t"
#define ATTN_BEGIN                                                          \
  "{\n\t.reg .pred e, no, yes;\n\t.reg .b64 da, db;\n\t"                 \
  ".reg .b32 la, lb;\n\t"                                                  \
  "setp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"                   \
  "elect.sync _|e, 0xffffffff;\n\t"
#define ATTN_END                                                            \
  "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster."   \
  "b64 [%5];\n\t}"
  if constexpr (D == 128) {
    asm volatile(ATTN_BEGIN ATTN_STEP("0", "no") ATTN_STEP("2", "yes")
                     ATTN_STEP("4", "yes") ATTN_STEP("6", "yes")
                         ATTN_STEP("1024", "yes") ATTN_STEP("1026", "yes")
                             ATTN_STEP("1028", "yes")
                                 ATTN_STEP("1030", "yes") ATTN_END ::"r"(d),
                 "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(bar)
                 : "memory");
  } else {
    asm volatile(ATTN_BEGIN ATTN_STEP("0", "no") ATTN_STEP("2", "yes")
                     ATTN_STEP("4", "yes") ATTN_STEP("6", "yes")
                         ATTN_END ::"r"(d),
                 "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(bar)
                 : "memory");
  }
#undef ATTN_STEP
#undef ATTN_BEGIN
#undef ATTN_END
}

// O (+)= P V of half a tile, four steps of 16 keys, and a commit to `bar`: P in
// tensor memory from `a` on, 8 columns a step, V 2 KB on.
__device__ __forceinline__ void issue_output(uint32_t d, uint32_t a,
                                             uint32_t b, uint32_t hi,
                                             uint32_t idesc, uint32_t acc,
                                             uint32_t bar) {
#define ATTN_STEP(at, off, p)                                               \
  "add.u32 ta, %1, " at ";\n\tadd.u32 lb, %2, " off ";\n\t"              \
  "mov.b64 db, {lb, %3};\n\t"                                              \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, " p ";\n\t"
  asm volatile(
      "{\n\t.reg .pred e, acc, yes;\n\t.reg .b64 db;\n\t"
      ".reg .b32 ta, lb;\n\t"
      "setp.ne.b32 acc, %5, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t" ATTN_STEP("0", "0", "acc")
          ATTN_STEP("8", "128", "yes") ATTN_STEP("16", "256", "yes")
              ATTN_STEP("24", "384", "yes")
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster."
      "b64 [%6];\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(bar)
      : "memory");
#undef ATTN_STEP
}

// NT: 8-row groups of the few-row work (0: not kFew).
template <int D, bool kBF16, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_many_kernel(const __grid_constant__ Maps maps,
                       const __grid_constant__ PrefixParams p) {
  using L = Smem<D>;
  constexpr int kOCol = 2 * kTN;  // TMEM: S0, S1, then O0, O1
  constexpr float kShift = kBF16 ? -24.f : 7.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_base = ptx::smem_u32(smem);
  const uint32_t bar_full = s_base + L::kBars;           // [kSlots]
  const uint32_t bar_empty = bar_full + 8 * L::kSlots;   // [kSlots]
  const uint32_t bar_unit = bar_empty + 8 * L::kSlots;   // [kUnits]
  const uint32_t bar_ufree = bar_unit + 8 * kUnits;      // [kUnits]
  const uint32_t bar_q = bar_ufree + 8 * kUnits;         // [2]
  const uint32_t bar_qfree = bar_q + 16;                 // [2]
  const uint32_t bar_s = bar_qfree + 16;                 // [tile][buffer]
  const uint32_t bar_p = bar_s + 32;                     // [tile][buffer]
  const uint32_t bar_pv = bar_p + 32;                    // [2]
  const uint32_t bar_o = bar_pv + 16;                    // [2]
  const uint32_t bar_end = bar_o + 16;                   // [1]
  const uint32_t bar_cleared = bar_end + 8;              // [1]
  const uint32_t bar_drain = bar_end + 16;               // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc + 4);
  volatile Record* records = reinterpret_cast<Record*>(smem + L::kRecords);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x < L::kNumBars) {
    const uint32_t bar = s_base + L::kBars + 8 * threadIdx.x;
    // Tiles used, and ends of V asked for: one arrival per issuing warp (2);
    // units read: one per warp of the other roles (11); P: one per softmax
    // thread of the tile.
    uint32_t count = 1;
    if ((bar >= bar_empty && bar < bar_unit) || bar == bar_end) count = 2;
    if (bar >= bar_ufree && bar < bar_q) count = 11;
    if (bar >= bar_p && bar < bar_pv) count = kTM;
    // (Self-test: an arrival more than comes.)
    const int cta = static_cast<int>(blockIdx.x);
    if ((cta == p.hold_keys && bar == bar_full) ||
        (cta == p.hold_rows && bar >= bar_q && bar < bar_qfree))
      count = 2;
    ptx::mbar_init(bar, count);
    if (threadIdx.x == 0) *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 41)
    ptx::prefetch_tensormap(threadIdx.x == 40 ? &maps.q
                                              : &maps.m[threadIdx.x - 32]);
  __syncthreads();
  ptx::griddep_wait();
  // (The merge kernel behind takes no tensor memory, and lets no other kernel
  // start before it has waited for this one.)
  ptx::griddep_launch_dependents();
  FewLens few_lens;
  if constexpr (NT > 0) few_lens.load(p, lane);
  const int plen = prefix_len(p), np = (plen + kTN - 1) / kTN;
  int ctas = p.grid;
  if constexpr (NT > 0) {
    const int few = few_total<D>(p, few_lens, lane);
    ctas = prefix_ctas(p, np, few);
    const int cta = static_cast<int>(blockIdx.x) - ctas;
    if (cta >= 0) {
      if (warp < 4) {
        ptx::setmaxnreg_dec<kRegsControl>();
      } else {
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        few_share<D, NT, kBF16>(p, cta * kFewWarps + warp - 4,
                                (p.grid - ctas) * kFewWarps, few, lane,
                                s_base + (warp - 4) * kFewRing);
      }
      return;
    }
  }
  // Tensor memory is taken behind the wait for the kernel ahead (which may
  // still have to take its own); the warps that use it meet here, the others
  // go ahead.
  uint32_t tmem = 0;
  if (warp == 0 || warp == 2 || warp >= 4) {
    if (warp == 0) {
      ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
      ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    ptx::named_barrier_sync(1, kThreads - 64);
    ptx::tc_fence_after();
    tmem = *tmem_slot;
  }

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
    if (warp == 3) {
      // --------- units of the share, their query rows, ends of V's last tiles
      Walk walk;
      bool more =
          walk.take(p, static_cast<int>(blockIdx.x), ctas, np, lane);
      int4 split = make_int4(0, 0, 0, 0);
      int published = 0;
      // A sequence's rows that fill one Q tile at most take either in turn, so
      // that a unit's first steps go along with the last of the unit before.
      const bool turns = p.rows <= p.tile_rows;
      int swap = 1;
      // Units are published one ahead of the one at hand (all roles can end
      // every unit before that without this warp, so that the wait ends).
      auto publish = [&] {
        const int k = published++;
        if (k >= kUnits)
          ok = wait(bar_ufree + 8 * (k % kUnits), k / kUnits - 1, 1);
        if (!ok) return;
        swap = turns && more && walk.w.b >= 0 ? swap ^ 1 : 0;
        if (lane == 0) {
          volatile Record* rec = records + k % kUnits;
          if (more)
            fill_record(p, walk, plen, swap, rec);
          else
            rec->n_kv = 0;
          ptx::mbar_arrive(bar_unit + 8 * (k % kUnits));
        }
        __syncwarp();
        if (!more) return;
        const Unit& w = walk.w;
        if (w.j0 == 0) {
          const int parts =
              w.j1 < w.steps ? walk.last_cta() - walk.cta + 1 : 1;
          if (p.mode == kJoint) {
            if (parts > 1) split = make_int4(w.b, w.h, w.u, parts);
          } else if (lane == 0) {
            p.info[static_cast<long long>(w.i) * p.Hkv + w.h] =
                make_int2(walk.cta, parts);
          }
        }
        more = walk.next(p);
      };
      publish();
      // The ends in step with the MMA issuers, which ask for each when it has
      // arrived (a warp that looked at some phases only of the ring's barriers
      // could take one for another).
      int slot_v = 1;  // V tiles of the stream are odd
      int ends = 0, q_uses[2] = {0, 0};
      const int q_tokens = fast_div(p.tile_rows, p.fd_group);
      const uint32_t q_bytes =
          (p.mode == kJoint ? p.tile_rows : p.tile_seqs * p.rows) * D * 2;
      auto load_q = [&](int k) {
        volatile Record* rec = records + k % kUnits;
        const int n0 = rec->n[0], n1 = rec->n[1];
        const int b = rec->b, h = rec->h, tile0 = rec->tile0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (t ? n1 : n0) == 0) continue;
          if (q_uses[t] > 0) ok = wait(bar_qfree + 8 * t, q_uses[t] - 1, 5);
          if (!ok) break;
          ++q_uses[t];
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar_q + 8 * t, q_bytes);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(s_base + L::kQ + t * L::kTile + c * L::kBox, &maps.q,
                          bar_q + 8 * t, c * 64, h * p.group,
                          b < 0 ? 0 : (tile0 + t) * q_tokens,
                          b < 0 ? (tile0 + t) * p.tile_seqs : b);
          }
        }
      };
      int loaded = 0;  // units whose query rows are asked for
      for (int k = 0; ok; ++k) {
        volatile Record* rec = records + k % kUnits;
        const int n = rec->n_kv;
        if (n == 0) break;
        const int j0 = rec->j0, unit_np = rec->np, len = rec->len;
        if (loaded == k) {
          load_q(k);
          ++loaded;
        }
        if (!ok) break;
        publish();
        if (!ok) break;
        // The next unit's, where they take the other tile (which the unit
        // before this one had: all its ends are cleared).
        volatile Record* next = records + (k + 1) % kUnits;
        if (turns && rec->b >= 0 && next->n_kv > 0) {
          load_q(k + 1);
          ++loaded;
          if (!ok) break;
        }
        for (int j = 0; j < n; ++j) {
          bool own;
          const int valid = tile_keys(j0 + j, unit_np, plen, len, &own);
          const int slot = slot_v;
          slot_v += 2;
          if (slot_v >= L::kSlots) slot_v -= L::kSlots;
          if (valid % 16 == 0) continue;
          ok = wait(bar_end, ends++, 5);
          if (!ok) break;
          const uint32_t at = s_base + L::kRing + slot * L::kTile;
          const int rows = 16 - valid % 16;
          for (int i = lane; i < rows * (D / 8); i += 32) {
            const int c = i % 8, x = i / 8;
            const int box = x / rows, r = valid + x - box * rows;
            ptx::st_shared_v4(at + box * L::kBox + r * 128 + c * 16, 0u, 0u,
                              0u, 0u);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar_cleared);
        }
      }
      // The copies in flight land before the CTA ends, whoever gave up.
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (q_uses[t] > 0)
          drain_wait(bar_q + 8 * t, (q_uses[t] - 1) & 1, p);
      __syncwarp();
      if (lane == 0 && p.mode == kJoint) p.split[blockIdx.x] = split;
      write_unseen<D>(p, lane);
    } else if (warp == 1) {
      // -------------------------------------------------------- tile copies
      int it = 0;
      for (int k = 0; ok; ++k) {
        volatile Record* rec = get_unit(k);
        if (rec == nullptr) break;
        const int n = rec->n_kv, j0 = rec->j0, np = rec->np;
        const int plen = rec->plen, len = rec->len, h = rec->h;
        const int own_plane = rec->b * p.Hkv + h;
        release_unit(k);
        for (int j = 0; j < n && ok; ++j) {
          bool own;
          const int valid = tile_keys(j0 + j, np, plen, len, &own);
          const int row = (own ? j0 + j - np : j0 + j) * kTN;
          const int plane = own ? own_plane : h;
          const bool tail = valid <= kTN - kTailRows;
          const int rows =
              tail ? (valid + kTailRows - 1) / kTailRows * kTailRows : kTN;
          const int step = tail ? kTailRows : kTN;
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = it % L::kSlots, use = it / L::kSlots;
            if (use > 0) ok = wait(bar_empty + 8 * slot, use - 1, 1);
            if (!ok) break;
            if (lane == 0) {
              const uint32_t bar = bar_full + 8 * slot;
              const uint32_t dst = s_base + L::kRing + slot * L::kTile;
              const CUtensorMap* m =
                  &maps.m[(own ? 4 : 0) + (tail ? 2 : 0) + kv];
              ptx::mbar_arrive_expect_tx(bar, rows * D * 2);
              for (int r = 0; r < rows; r += step)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  ptx::tma_load_3d(dst + c * L::kBox + r * 128, m, bar, c * 64,
                                   row + r, plane);
            }
            ++it;
          }
        }
      }
      // The copies in flight land before the CTA ends, whoever gave up.
      for (int i = max(0, it - L::kSlots); i < it; ++i)
        drain_wait(bar_full + 8 * (i % L::kSlots), (i / L::kSlots) & 1, p);
      __syncwarp();
    } else {
      // ----------------------------------------- MMA issue, a warp a Q tile
      const int t = warp / 2;
      const uint32_t idesc_qk =
          ptx::idesc_f16(kBF16, kTM, kHalf, false, p.negate != 0);
      const uint32_t idesc_pv = ptx::idesc_f16(kBF16, kTM, D, true, false);
      constexpr uint32_t kHi = ptx::sdesc_hi_sw128(1024);
      const uint32_t q_lo = ptx::sdesc_lo(s_base + L::kQ, 16);
      const uint32_t k_lo = ptx::sdesc_lo(s_base + L::kRing, 16);
      const uint32_t v_lo = ptx::sdesc_lo(s_base + L::kRing, L::kBox);
      constexpr uint32_t kTile16 = L::kTile >> 4;
      constexpr uint32_t kHalf16 = (kHalf * 128) >> 4;  // half a tile's rows on
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);  // uniform
      // The ring's tile that S, and that O, takes next (K_0, V_0, K_1, ...).
      int slot_k = 0, phase_k = 0, slot_v = 1, phase_v = 0;
      int s_count = 0, o_count = 0;  // steps issued
      int q_uses = 0;
      int ends = 0;  // tiles cleared behind their last key
      bool issued = false;
      auto two_on = [&](int& slot, int& phase) {
        slot += 2;
        if (slot >= L::kSlots) {
          slot -= L::kSlots;
          phase ^= 1;
        }
      };
      for (int k = 0; ok; ++k) {
        ok = wait(bar_unit + 8 * (k % kUnits), k / kUnits, 1);
        if (!ok) break;
        // Through a warp reduction the counts are warp-uniform to the
        // compiler, and with them the ring position: descriptors then stay in
        // uniform registers (else every MMA moves them there first).
        volatile Record* rec = records + k % kUnits;
        const int n = __reduce_max_sync(0xffffffffu, rec->n[t]);
        const int n_kv = __reduce_max_sync(0xffffffffu, rec->n_kv);
        const int j0 = __reduce_max_sync(0xffffffffu, rec->j0);
        const int np = __reduce_max_sync(0xffffffffu, rec->np);
        const int plen = __reduce_max_sync(0xffffffffu, rec->plen);
        const int len = __reduce_max_sync(0xffffffffu, rec->len);
        if (n_kv == 0) break;
        release_unit(k);
        // Tiles that lengths end in: the prefix's last and the own last one.
        const int end_p = np - 1 - j0, keys_p = plen - (np - 1) * kTN;
        const int end_own = np + (len - 1) / kTN - j0;
        const int keys_own = (len - 1) % kTN + 1;
        auto valid_of = [&](int j) {
          return j == end_p ? keys_p : j == end_own ? keys_own : kTN;
        };
        // Next steps of S and of O: tile and half.
        int jk = 0, hk = 0, jv = 0, hv = 0;
        auto scores = [&] {
          const bool last_half = valid_of(jk) <= kHalf * (hk + 1);
          if (hk == 0) {
            ok = wait(bar_full + 8 * slot_k, phase_k, 2);
            if (!ok) return;
          }
          if (jk < n) {
            if (jk == 0 && hk == 0) {
              ok = wait(bar_q + 8 * t, q_uses++, 2);
              if (!ok) return;
            }
            ptx::tc_fence_after();
            const int buf = s_count++ & 1;
            issue_scores<D>(tm + t * kTN + buf * kHalf, q_lo + t * kTile16,
                            k_lo + slot_k * kTile16 + hk * kHalf16, kHi,
                            idesc_qk, bar_s + 16 * t + 8 * buf);
            issued = true;
            // Behind the tile's last S its query rows make room.
            if (last_half && jk == n - 1)
              ptx::tc_commit_elect(bar_qfree + 8 * t);
          }
          hk = last_half ? 0 : 1;
          if (last_half) {
            ptx::tc_commit_elect(bar_empty + 8 * slot_k);
            two_on(slot_k, phase_k);
            ++jk;
          }
        };
        scores();
        while (ok && jv < n_kv) {
          // The next step's S is made while the softmax works on this one's.
          if (jk < n_kv) scores();
          if (!ok) break;
          const int valid = valid_of(jv);
          const bool last_half = valid <= kHalf * (hv + 1);
          bool clear = false;
          if (hv == 0) {
            ok = wait(bar_full + 8 * slot_v, phase_v, 2);
            if (!ok) break;
            clear = valid % 16 != 0;
            if (clear && lane == 0) ptx::mbar_arrive(bar_end);
          }
          if (clear) {
            ok = wait(bar_cleared, ends++, 2);
            if (!ok) break;
          }
          if (jv < n) {
            const int steps = (min(kHalf, valid - hv * kHalf) + 15) / 16;
            const int buf = o_count & 1;
            ok = wait(bar_p + 16 * t + 8 * buf, o_count >> 1, 2);
            if (!ok) break;
            ++o_count;
            ptx::tc_fence_after();
            const uint32_t d = tm + kOCol + t * D;
            const uint32_t a = tm + t * kTN + buf * kHalf;
            const uint32_t b = v_lo + slot_v * kTile16 + hv * kHalf16;
            const bool acc = jv > 0 || hv > 0;
            if (steps == kHalf / 16) {
              issue_output(d, a, b, kHi, idesc_pv, acc ? 1u : 0u,
                           bar_pv + 8 * t);
            } else {
#pragma unroll 1
              for (int kk = 0; kk < steps; ++kk)
                ptx::mma_ts_elect(d, a + kk * 8, b + ((kk * 16 * 128) >> 4),
                                  kHi, idesc_pv, (acc || kk > 0) ? 1u : 0u);
              ptx::tc_commit_elect(bar_pv + 8 * t);
            }
            if (last_half && jv == n - 1) ptx::tc_commit_elect(bar_o + 8 * t);
          }
          hv = last_half ? 0 : 1;
          if (last_half) {
            ptx::tc_commit_elect(bar_empty + 8 * slot_v);
            two_on(slot_v, phase_v);
            ++jv;
          }
        }
      }
      // The products issued end before TMEM is freed, whoever gave up.
      if (issued) {
        ptx::tc_commit_elect(bar_drain + 8 * t);
        drain_wait(bar_drain + 8 * t, 0, p);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------ softmax, correction, epilogue
    ptx::setmaxnreg_inc<kRegsSoftmax>();
    const int t = warp / 4 - 1;
    const int r = threadIdx.x % kTM;  // row within the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t t_scores = tmem + lane_off + t * kTN;
    const uint32_t t_o = tmem + lane_off + kOCol + t * D;
    // Factor of the scores, held off 0 so that -inf stays -inf (scores times
    // 1e-37 vanish next to any maximum).
    const float c = fmaxf(p.scale_log2, 1e-37f);
    int count = 0, o_uses = 0;  // steps and units done
    // Before the first scores a step is made of whatever O's columns hold, to
    // no effect but that its instructions have been fetched (2.5 us of the
    // first real step otherwise; the first products overwrite O).
    bool dry = true;
    for (int k = 0; ok; ++k) {
      volatile Record* rec = get_unit(k);
      if (rec == nullptr) break;
      const int n = rec->n[t];
      // Keys left from the tile at hand on: of the prefix (none behind its
      // tiles) and own ones, of which this row does not see the last `hidden`.
      int left = 0, left_own, hidden = 0;
      // A warp without rows keeps in step but computes nothing: its P are
      // whatever S left there, which reaches its own rows of O only.  Beside
      // rows, those of no row (made of what shared memory held) have no say in
      // when the warp rescales.
      bool live, row_here;
      {
        const int j0 = rec->j0, np = rec->np, len = rec->len;
        int row;
        row_here = row_of(p, rec, t, r, &row) >= 0;
        live = __any_sync(0xffffffffu, row_here);
        if (rec->b >= 0 && row_here)
          hidden = len - row_end(p, len, rec->n_new, row);
        if (np > 0) left = rec->plen - j0 * kTN;
        left_own = len - (j0 - np) * kTN;
      }
      float m_run = -INFINITY, l_run = 0.f;
      bool first = true;
      int half = 0;
      for (int j = 0; j < n;) {
        const int keys = left > 0 ? left : left_own;
        const int lim = (left > 0 ? left : left_own - hidden) - half * kHalf;
        const int buf = count & 1;
        if (!dry) {
          ok = wait(bar_s + 16 * t + 8 * buf, count >> 1, 4);
          if (!ok) break;
          ptx::tc_fence_after();
        }
        if (live) {
          const bool masked = __any_sync(0xffffffffu, lim < kHalf);
          const uint32_t t_s = dry ? t_o : t_scores + buf * kHalf;
          uint32_t sr[kHalf];
#pragma unroll
          for (int q = 0; q < kHalf / 32; ++q)
            ptx::tmem_ld32(t_s + 32 * q, sr + 32 * q);
          ptx::tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int q = 0; q < kHalf; ++q)
              if (q >= lim) sr[q] = __float_as_uint(-INFINITY);
          }
          float mx4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx4[e] = fmaxf(__uint_as_float(sr[e]), __uint_as_float(sr[e + 4]));
#pragma unroll
          for (int q = 8; q < kHalf; q += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx4[e] = ptx::fmax3(mx4[e], __uint_as_float(sr[q + e]),
                                  __uint_as_float(sr[q + 4 + e]));
          const float mx =
              fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * c;
          float m_new = m_run;
          if (__any_sync(0xffffffffu, row_here && mx > m_run + kTau))
            m_new = fmaxf(m_run, mx);
          const float alpha =
              (m_new == -INFINITY) ? 1.f : ptx::ex2(m_run - m_new);
          const float neg_m = (m_new == -INFINITY) ? 0.f : kShift - m_new;
          float sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < kHalf / 32; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i = 32 * q + 2 * e;
              float x0, x1;
              ptx::ffma2(x0, x1, __uint_as_float(sr[i]),
                         __uint_as_float(sr[i + 1]), c, neg_m);
              const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              if (e & 1)
                ptx::fadd2(sm[2], sm[3], p0, p1);
              else
                ptx::fadd2(sm[0], sm[1], p0, p1);
              pk[e] = ptx::pack2<kBF16>(p0, p1);
            }
            ptx::tmem_st16(t_s + 16 * q, pk);
          }
          if (!first && !dry && __any_sync(0xffffffffu, m_new != m_run)) {
            // O *= alpha, behind the products of the step before.  (Those of
            // the one before that are done, as this step's S came after them:
            // the barrier's phase is that step's or the next.)
            ok = wait(bar_pv + 8 * t, count - 1, 4);
            if (!ok) break;
            ptx::tc_fence_after();
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
          l_run = l_run * alpha + ((sm[0] + sm[1]) + (sm[2] + sm[3]));
          ptx::tmem_wait_st();
          m_run = m_new;
        }
        if (dry) {
          dry = false;
          m_run = -INFINITY;
          l_run = 0.f;
          continue;
        }
        first = false;
        ++count;
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar_p + 16 * t + 8 * buf);
        if (half == 0 && keys > kHalf) {
          half = 1;
        } else {
          half = 0;
          left -= kTN;
          left_own -= kTN;
          ++j;
        }
      }
      if (!ok) break;
      if (n > 0) {
        ok = wait(bar_o + 8 * t, o_uses, 4);
        if (!ok) break;
        ++o_uses;
        ptx::tc_fence_after();
      }
      const int dest = rec->dest, h = rec->h;
      int row;
      const int b = row_of(p, rec, t, r, &row);
      const bool row_ok = b >= 0;
      // O leaves as the average that it is.  A row that sees nothing: 0,
      // whatever its accumulator holds.
      const bool seen = l_run != 0.f;
      const float inv = seen ? 1.f / l_run : 0.f;
      const float lse2 =
          seen ? (m_run == -INFINITY ? kNone : m_run) + log2f(l_run) - kShift
               : -INFINITY;
      if (dest == kFinal) {
        const long long at = row_ok ? q_row_index(p, b, h, row) : 0;
        uint4* dst = reinterpret_cast<uint4*>(p.o + at * D);
        // (O is 16-byte aligned, its rows whole 32-byte sectors from there.)
        const bool wide = reinterpret_cast<uintptr_t>(p.o) % 32 == 0;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (n > 0) {
            ptx::tmem_ld32(t_o + 32 * q, o);
            ptx::tmem_wait_ld();
          }
          if (row_ok) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[e] = !seen ? 0u
                             : ptx::pack2<kBF16>(
                                   __uint_as_float(o[16 * v + 2 * e]) * inv,
                                   __uint_as_float(o[16 * v + 2 * e + 1]) *
                                       inv);
              store_row(dst + 4 * q + 2 * v, x, wide);
            }
          }
        }
        if (row_ok && p.lse != nullptr) p.lse[at] = lse2 * 0.69314718055994531f;
      } else {
        // Rows of a unit over the prefix lie packed, a sequence's own behind.
        long long at;
        float *dst_o = p.slot_o, *dst_lse2 = p.slot_lse2;
        if (dest == kBase) {
          dst_o = p.base_o;
          dst_lse2 = p.base_lse2;
          const long long all = static_cast<long long>(p.B) * p.rows;
          at = rec->b < 0 ? h * all + static_cast<long long>(b) * p.rows
                          : p.Hkv * all +
                                (static_cast<long long>(b) * p.Hkv + h) *
                                    p.rows;
          at += row;
        } else {
          at = static_cast<long long>(dest) * kUnitRows +
               ((rec->tile0 + t) & 1) * kTM + r;
        }
        if (n > 0) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            ptx::tmem_ld32(t_o + 32 * q, o);
            ptx::tmem_wait_ld();
            if (row_ok && seen) {
              float4* dst = reinterpret_cast<float4*>(dst_o) + at * (D / 4);
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
        if (row_ok) dst_lse2[at] = lse2;
      }
      ptx::tc_fence_before();
      release_unit(k);
    }
    if (!ok) ptx::tmem_wait_st();  // of a step that was given up
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kBF16, int NT>
cudaError_t launch(const PrefixParams& p, const CUtensorMap* maps,
                   cudaStream_t stream) {
  constexpr int kBytes = Smem<D>::kBytes + 1024;
  const cudaError_t err = cudaFuncSetAttribute(
      prefix_many_kernel<D, kBF16, NT>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (err != cudaSuccess) return err;
  Maps m;
  for (int i = 0; i < 8; ++i) m.m[i] = maps[i];
  m.q = maps[8];
  return kv8::launch_pdl(prefix_many_kernel<D, kBF16, NT>, p.grid, kThreads,
                         kBytes, stream, m, p);
}

template <int D, bool kBF16>
cudaError_t launch_dt(const PrefixParams& p, const CUtensorMap* maps,
                      cudaStream_t stream) {
  if (p.mode != kFew) return launch<D, kBF16, 0>(p, maps, stream);
  return few_rows(p.rows) == 8 ? launch<D, kBF16, 1>(p, maps, stream)
                               : launch<D, kBF16, 2>(p, maps, stream);
}

}  // namespace

cudaError_t launch_many(int D, bool bf16, const PrefixParams& p,
                        const CUtensorMap* maps, cudaStream_t stream) {
  if (D == 64)
    return bf16 ? launch_dt<64, true>(p, maps, stream)
                : launch_dt<64, false>(p, maps, stream);
  return bf16 ? launch_dt<128, true>(p, maps, stream)
              : launch_dt<128, false>(p, maps, stream);
}

}  // namespace prefix
}  // namespace attn
