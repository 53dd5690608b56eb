// Parameters of the attention of a batch whose sequences share a prefix, and
// the layout of its partial results.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kv8_common.cuh"

namespace attn {
namespace prefix {

constexpr int kTM = 128;             // rows of a Q tile
constexpr int kTN = 128;             // keys of a tile
constexpr int kUnitRows = 2 * kTM;   // rows of a unit
constexpr int kTailRows = 16;        // rows of a copy of a last tile
constexpr int kFewWarps = 4;

// How the query rows meet the keys (R rows of a K/V head per sequence, row r =
// token r / group, head r % group):
//   kFew    R <= 16: units of 256 rows of all sequences over the prefix, the
//           sequences' own keys by the few-row kernel;
//   kPacked such units over the prefix, and units of each sequence over its
//           own keys;
//   kJoint  units of each sequence over the prefix and its own keys in turn.
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
  // Own keys of few rows: slot CTA + segment.
  float* few_o;           // [slots, 8 or 16, D]
  float* few_lse2;
  int grid;               // CTAs that the list at hand is cut for
  int many_grid, few_grid;
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
  const int tok = r / p.group, hd = r - tok * p.group;
  return (static_cast<long long>(b) * p.Hq + h * p.group + hd) * p.Sq + tok;
}

// The few-row kernel's tiles: 4 KB of keys; and empty places before a segment.
template <int D>
__host__ __device__ constexpr int few_keys() {
  return 2048 / D;
}
constexpr int kFewOver = 6;

// Own key tiles that rows [r0, r1) of a sequence with n_new tokens see.
__device__ __forceinline__ int tiles_seen(const PrefixParams& p, int len,
                                          int n_new, int r0, int r1) {
  const int last = min(r1, n_new * p.group) - 1;
  if (last < r0) return 0;
  return (kv8::row_end(p, len, n_new, last) + kTN - 1) / kTN;
}

cudaError_t launch_many(int D, bool bf16, const PrefixParams& p,
                        const CUtensorMap* maps, cudaStream_t stream);
cudaError_t launch_few(int D, bool bf16, const PrefixParams& p,
                       cudaStream_t stream);
cudaError_t launch_merge(int D, bool bf16, const PrefixParams& p,
                         cudaStream_t stream);

// CTAs of the few-row kernel that an SM holds, and rows it works on.
__host__ __device__ constexpr int few_ctas(int D, int rows) {
  return 2;
}
__host__ __device__ constexpr int few_rows(int rows) {
  return rows <= 8 ? 8 : 16;
}

}  // namespace prefix
}  // namespace attn
