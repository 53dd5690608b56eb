// Index arithmetic of the 8-bit cache's kernels whose operands may add up to
// more than 32 bits hold although each is a token count (below 2^31 - 2^16),
// as plain C++ that runs on host and device alike.
#pragma once

#ifdef __CUDACC__
#define ATTN_KV8_INDEX __host__ __device__ __forceinline__
#else
#define ATTN_KV8_INDEX inline
#endif

namespace attn {
namespace kv8 {

// The u-th block of `block` tokens from the one that holds token `start`, or
// -1 where it lies behind the last of len > 0 tokens.  (The grid has as many
// blocks as Sq tokens can touch; a sequence with fewer new ones is past its
// end long before, by up to Sq tokens: the block's number is compared, not
// its first token's place.)
ATTN_KV8_INDEX int append_block(int start, int len, int block, int u) {
  const int blk = start / block + u;
  return blk <= (len - 1) / block ? blk : -1;
}

// Rounds of `step` places that cover n >= 0 of them.  (Into another cache a
// round has as many places as that cache: n + step passes 2^31 from half of
// the largest capacity on.)
ATTN_KV8_INDEX int round_count(int n, int step) {
  return n / step + (n % step != 0 ? 1 : 0);
}

// The first place behind n kept ones that a thread clears, with `rank`
// thread blocks before its own: n and a quarter of the capacity at most.
ATTN_KV8_INDEX long long cleared_place(int n, int rank, int threads,
                                       int thread) {
  return static_cast<long long>(n) + static_cast<long long>(rank) * threads +
         thread;
}

}  // namespace kv8
}  // namespace attn
