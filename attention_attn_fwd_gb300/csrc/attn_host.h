// Host helpers of the C ABI shared by its translation units.
#pragma once

#include <cstddef>

#include <cuda.h>

namespace attn {

// Status-word bit 1: a kernel met a length outside its range and clamped it.
constexpr unsigned int kStatusBadLength = 2u;

// Address of the device status word on `dev` (nullptr on failure).
unsigned int* device_status_word(int dev);
// Streaming multiprocessors of `dev` (0 on failure).
int device_sms(int dev);
// Limit of every bounded kernel wait, in nanoseconds.
unsigned long long wait_timeout_ns();
// Device or managed memory of `dev`.
bool on_device(const void* p, int dev);
// Whether two byte ranges share a byte.
bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb);

// Map of a [planes, rows, D] tensor of 16-bit elements for copies of box_rows
// rows by one 128-byte segment, 128-byte swizzled (false: it could not be
// made).
bool make_tile_map(CUtensorMap* m, const void* base, bool bf16, int D,
                   int rows, long long planes, int box_rows);

// Map of a [B, H, S, D] tensor of 16-bit elements for copies whose rows lie in
// the order (sequence, token, head): of box_b, box_s and box_h of these, by one
// 128-byte segment, 128-byte swizzled.
bool make_rows_map(CUtensorMap* m, const void* base, bool bf16, int D, int S,
                   int H, int B, int box_h, int box_s, int box_b);

}  // namespace attn
