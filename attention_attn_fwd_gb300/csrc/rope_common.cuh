// Parameters shared by the kernels that norm and rotate queries and keys, and
// by their C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "fast_div.h"

namespace attn {
namespace rope {

constexpr int kThreads = 128;

struct RopeParams {
  // Rotation: angle of pair i = position on axis axis[i] times phase[i], in
  // units of 2^-64 of a turn.
  const unsigned long long* phase;  // [rot / 2]
  const unsigned char* axis;        // [rot / 2], or nullptr (axis 0)
  const int* pos;                   // [axes, B, S], or nullptr: counted
  const int* offset;                // first position counted from, or nullptr
  const int* lens;                  // cache lengths [B], or nullptr
  const int* new_lens;              // [B], or nullptr
  // Forward: Q, K, V as the projections give them, and their places.
  // Backward: x Q and K again, y the gradients of what the forward wrote, dx
  // those of what it read.
  const uint16_t* x[3];
  uint16_t* y[3];
  uint16_t* dx[3];
  long long x_b[3], x_s[3], x_h[3];     // strides in elements
  long long dx_b[3], dx_s[3], dx_h[3];
  const void* w[2];                 // norm weights, or nullptr: no norm
  float* dw[2];
  float* part;                      // backward: [CTAs, D]
  unsigned int* status;
  int B, S, tokens;                 // tokens: B * S
  int Hq, Hkv, heads;               // heads: of Q, K and (if given) V
  int head_block;                   // heads of a group of lanes, all of a kind
  int q_blocks, kv_blocks, blocks;  // blocks of heads: Q's, K's, all
  FastDiv fd_blocks;
  int capacity;                     // rows of a head of y[1] and y[2]
  int rot, w_f32;
  float eps;
};

// bf16, pairs (2i, 2i + 1) instead of (i, i + rot / 2).
cudaError_t launch_rope(int D, bool bf16, bool interleaved,
                        const RopeParams& p, int sms, cudaStream_t stream);
cudaError_t launch_rope_bwd(int D, bool bf16, bool interleaved,
                            const RopeParams& p, int sms, cudaStream_t stream);
// CTAs of a backward launch at most (each leaves a row of partial sums).
constexpr int bwd_ctas(int sms) { return 6 * sms; }

}  // namespace rope
}  // namespace attn
