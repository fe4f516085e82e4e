// share_split.h -- how many clusters of four SMs the shared prefixes of a call get beside the kernel for few rows.
// Arithmetic alone, for the plan on the device and for a test on the host.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define KV8_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KV8_HOST_DEVICE inline
#endif

namespace kv8 {

// Cycles that the prefixes' kernel and the join take besides its units (figures beside NARROW, chunk_work.cuh), and the
// kernel for few rows.
constexpr int START = 16000, START_WIDE = 40000, JOIN_MORE = 4000;

// What a call takes where the prefixes have t clusters (t < 64): its cycles, and t in the last six bits, so that the
// least of them names its t.  `wide`: the prefixes' cycles on one cluster; `narrow`: what lies behind them, on one SM.
// (Estimates: f32 does, and its divisions are the cheaper ones.)
KV8_HOST_DEVICE int64_t split_cost(float wide, float narrow, int t, int sms) {
  const float x = wide / (float)t + START_WIDE, y = narrow / (float)(sms - 4 * t) + START;
  return (int64_t)((x < y ? y : x) + JOIN_MORE) * 64 + t;
}

// The clusters, by the least cost (INT64_MAX: the device holds no two clusters at once, and one of them is the others'
// SMs) and the cycles with nothing shared; 0 shares nothing, and `always` shares wherever it can be.
KV8_HOST_DEVICE int split_taken(int64_t least, int64_t apart, bool always) {
  if (least == INT64_MAX) return 0;
  return always || least / 64 < apart ? (int)(least % 64) : 0;
}

}  // namespace kv8
