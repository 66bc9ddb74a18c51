// Which keys a row sees through a sliding window with first tokens that stay visible.
#pragma once
#include <cuda_runtime.h>

namespace dg {

namespace {

constexpr float kLn2 = 0.69314718055994531f;

// The 64 keys from slot key0 on that a row at slot `at` sees: those up to itself that
// are less than `window` slots behind it, or below slot `sinks`.
__device__ __forceinline__ unsigned long long window_bits(int at, int key0, int window, int sinks) {
  const int up = at + 1 - key0, low = max(0, at - window + 1) - key0, sink = sinks - key0;
  if (up <= 0) return 0ull;
  unsigned long long v = low <= 0 ? ~0ull : low >= 64 ? 0ull : ~0ull << low;
  if (sink > 0) v |= sink >= 64 ? ~0ull : (1ull << sink) - 1;
  return up >= 64 ? v : v & ((1ull << up) - 1);
}

}  // namespace

}  // namespace dg
