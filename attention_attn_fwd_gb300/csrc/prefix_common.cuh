// Parameters of the attention of a batch whose sequences share a prefix, and
// the layout of its partial results.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "fast_div.h"
#include "kv8_common.cuh"

namespace attn {
namespace prefix {

constexpr int kTM = 128;             // rows of a Q tile
constexpr int kTN = 128;             // keys of a tile
constexpr int kUnitRows = 2 * kTM;   // rows of a unit's two tiles
constexpr int kTailRows = 16;        // rows of a copy of a last tile
constexpr int kFewWarps = 8;         // of a block that works on few rows

// How the query rows meet the keys (R rows of a K/V head per sequence, row r =
// token r / group, head r % group):
//   kFew    R <= 16 (8 for few sequences and heads): units of two Q tiles, each
//           the rows of as many sequences as it holds, over the prefix; the
//           sequences' own keys by thread blocks set aside for them
//           (prefix_few.cuh);
//   kPacked R <= 128, several sequences: such units over the prefix, and units
//           of each sequence over its own keys;
//   kJoint  units of each sequence over the prefix and its own keys in turn.
// 8 K/V heads of 128, 700 own keys behind 8192: 32 sequences of 4, 8 and 16
// rows take 34, 40 and 46 us by kFew, 48, 53 and 61 by kPacked; 4 sequences 21,
// 22 and 26, by kPacked 22, 22 and 22 (2 sequences of 12 rows: 24.6 and 19.8).
// 24, 64 and 128 rows take 67, 95 and 144 by kPacked, 194, 195 and 197 by kJoint
// (4 sequences: 23, 28 and 35; 40, 41 and 44).  More rows fill a Q tile without
// others'.
enum Mode { kFew = 0, kPacked = 1, kJoint = 2 };

struct PrefixParams {
  const uint16_t* k;      // own keys and values [B, Hkv, capacity, D]
  const uint16_t* v;
  const int* plen;        // [1]
  const int* lens;        // [B]
  const int* new_lens;    // [B] or nullptr
  const uint16_t* q;
  uint16_t* o;
  float* lse;             // or nullptr
  int B, Hq, Hkv, Sq, prefix_capacity, capacity;
  int group, rows;        // query heads per K/V head; R
  int mode, causal;
  int pack_blocks;        // units of a head over the prefix (0: kJoint)
  int row_blocks;         // units of a (sequence, head) (0: kFew)
  int tile_seqs;          // sequences of a Q tile over the prefix
  int tile_rows;          // rows of a sequence's Q tile: whole tokens
  float scale_log2;       // |scale| * log2(e)
  int negate;             // scale < 0
  // Parts of a row, each the average that it is, and their LSEs in log2 units
  // (-inf: sees nothing).  The part of a unit that has its first key lies by
  // row (kFew and kPacked: [Hkv, B * R] over the prefix, then [B, Hkv, R]; in
  // kJoint in slot grid + CTA), every other one in its CTA's slot.
  float* base_o;          // [rows, D]
  float* base_lse2;
  float* slot_o;          // [slots, 256, D]
  float* slot_lse2;
  int2* info;             // [units]: first CTA and number of parts
  int4* split;            // kJoint [grid]: b, h, block, parts (0: none)
  // Own keys of few rows: slot warp + segment.
  float* few_o;           // [slots, 8 or 16, D]
  float* few_lse2;
  int2* own_info;         // [B, Hkv]: first warp and number of parts
  int grid;               // CTAs of the launch
  // Self-test of the bounded waits: a CTA whose first key tile, or first query
  // rows, never count as there (-1: none).
  int hold_keys, hold_rows;
  FastDiv fd_group, fd_rows, fd_blocks, fd_tile_seqs, fd_hkv;
  unsigned long long timeout_ns;
  unsigned int* status;
};

__device__ __forceinline__ int prefix_len(const PrefixParams& p) {
  return kv8::clamp_len(*p.plen, p.prefix_capacity, p.status);
}
__device__ __forceinline__ int prefix_tiles(const PrefixParams& p) {
  return (prefix_len(p) + kTN - 1) / kTN;
}
// Query row r of K/V head h of sequence b, in Q, O and LSE.
__device__ __forceinline__ long long q_row_index(const PrefixParams& p, int b,
                                                 int h, int r) {
  const int tok = fast_div(r, p.fd_group), hd = r - tok * p.group;
  return (static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq + tok;
}

// The few-row work's tiles: 4 KB of keys; and empty places before a segment (64
// sequences behind 8192 tokens, 256 behind 2048, 32 behind 65531: 43, 44 and 51
// us; with 2 44, 44 and 52, and 32 sequences of one own token behind 65536 60
// for 49; with 5 45, 44 and 52).
template <int D>
__host__ __device__ constexpr int few_keys() {
  return 2048 / D;
}
constexpr int kFewOver = 4;

// Own tokens that row r of a sequence sees.
__device__ __forceinline__ int row_end(const PrefixParams& p, int len,
                                       int n_new, int r) {
  if (!p.causal) return len;
  return min(len, max(0, len - n_new + fast_div(r, p.fd_group) + 1));
}

// Own key tiles that rows [r0, r1) of a sequence with n_new tokens see.
__device__ __forceinline__ int tiles_seen(const PrefixParams& p, int len,
                                          int n_new, int r0, int r1) {
  const int last = min(r1, n_new * p.group) - 1;
  if (last < r0) return 0;
  return (row_end(p, len, n_new, last) + kTN - 1) / kTN;
}

cudaError_t launch_many(int D, bool bf16, const PrefixParams& p,
                        const CUtensorMap* maps, cudaStream_t stream);
cudaError_t launch_merge(int D, bool bf16, const PrefixParams& p,
                         cudaStream_t stream);

// Rows that the few-row work is compiled for.
__host__ __device__ constexpr int few_rows(int rows) {
  return rows <= 8 ? 8 : 16;
}

}  // namespace prefix
}  // namespace attn
