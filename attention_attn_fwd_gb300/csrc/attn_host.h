// Host helpers of the C ABI shared by its translation units.
#pragma once

#include <cstddef>

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

}  // namespace attn
