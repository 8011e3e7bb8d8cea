// Device helpers of the serving kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dequant.h"

namespace gq {

// 16-bit storage to float32 and back (round to nearest even).
template <int BF16>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, (uint32_t)v << 16);
  else return (float)__builtin_bit_cast(_Float16, v);
}
template <int BF16>
__device__ __forceinline__ uint16_t from_f32(float v) {
  if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// First b in [0, batch) with edge(b + 1) > row, for a wave-uniform row and edges that ascend
// (batch - 1 when there is none): each step reads 64 edges at once, one a lane, so up to 64
// sequences take one step and up to 4096 take two.
template <typename Edge>
__device__ __forceinline__ int find_sequence(int batch, int64_t row, Edge edge) {
  int lo = 0, n = batch;
  const int lane = threadIdx.x & 63;
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int at = (lane + 1) * step;               // sequences [lo, lo + at) end at or before row?
    const bool past = at < n && edge(lo + at) <= row;
    const int c = __builtin_popcountll(__ballot(past));
    lo += c * step;
    n = n - c * step < step ? n - c * step : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Sum over a wave, and the sum of a lane and all before it.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(v, d);
    if (lane >= d) v += other;
  }
  return v;
}
__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return __builtin_amdgcn_readfirstlane(v);
}

}  // namespace gq
