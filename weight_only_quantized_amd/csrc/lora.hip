// Low-rank adapters of many requests beside a shared projection.
//
// Mathematics: low[m] = A_i x[m] (rank values), out[m] = y[m] + scale_i * B_i low[m], i = ids[m].
// Two launches: one wave for each row and rank value sums over K; one thread for each output sums
// over the rank.  low stays in float32 in the workspace.
#include <hip/hip_runtime.h>

#include "serving.h"
#include "serving_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256;

template <int BF16>
__global__ void __launch_bounds__(kThreads) lora_low_kernel(LoraCall c, float* low) {
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t row = wave / c.bank.rank;
  const int r = (int)(wave % c.bank.rank), lane = threadIdx.x & 63;
  if (row >= c.M) return;
  const int id = c.ids[row], K = c.bank.in_features;
  if (id < 0 || id >= c.bank.adapters) return;
  const uint16_t* x = c.x + row * K;
  const uint16_t* w = (const uint16_t*)c.bank.a + ((int64_t)id * c.bank.rank + r) * K;
  float s = 0.0f;
  for (int k = lane; k < K; k += 64) s += to_f32<BF16>(x[k]) * to_f32<BF16>(w[k]);
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if (lane == 0) low[row * c.bank.rank + r] = s * c.bank.scale[id];
}

template <int BF16>
__global__ void __launch_bounds__(kThreads) lora_up_kernel(LoraCall c, const float* low, int64_t blocks_per_row) {
  const int64_t row = blockIdx.x / blocks_per_row;
  const int64_t n = blockIdx.x % blocks_per_row * kThreads + threadIdx.x;
  const int N = c.bank.out_features, rank = c.bank.rank;
  if (n >= N) return;
  const int id = c.ids[row];
  float s = to_f32<BF16>(c.y[row * N + n]);
  if (id >= 0 && id < c.bank.adapters) {
    const uint16_t* w = (const uint16_t*)c.bank.b + ((int64_t)id * N + n) * rank;
    float d = 0.0f;
    for (int r = 0; r < rank; ++r) d += low[row * rank + r] * to_f32<BF16>(w[r]);
    s += d;
  }
  c.out[row * N + n] = from_f32<BF16>(s);
}

}  // namespace

size_t lora_ws_bytes(const gptq_lora_bank& bank, int64_t M) { return ((size_t)M * bank.rank * 4 + 255) / 256 * 256; }

hipError_t launch_lora(const LoraCall& c, hipStream_t s) {
  float* low = (float*)c.ws;
  const int64_t waves = c.M * c.bank.rank, per_row = (c.bank.out_features + kThreads - 1) / kThreads;
  const int64_t blocks = (waves + kThreads / 64 - 1) / (kThreads / 64);
  if (blocks > 0x7fffffff || c.M * per_row > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (c.bank.dtype == GPTQ_BF16) {
    lora_low_kernel<1><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(c, low);
    lora_up_kernel<1><<<dim3((uint32_t)(c.M * per_row)), dim3(kThreads), 0, s>>>(c, low, per_row);
  } else {
    lora_low_kernel<0><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(c, low);
    lora_up_kernel<0><<<dim3((uint32_t)(c.M * per_row)), dim3(kThreads), 0, s>>>(c, low, per_row);
  }
  return hipGetLastError();
}

}  // namespace gq
