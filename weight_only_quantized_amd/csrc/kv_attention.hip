// Attention over the paged 8-bit cache.
//
// Mathematics: for a query q and its visible tokens j, s_j = scale * k_scale(page_j) * sum_d q_d kc_jd and
// out_d = sum_j p_j v_scale(page_j) vc_jd / sum_j p_j with p_j = exp(s_j - max_j s_j), in one pass over
// the tokens with the running maximum m and sum l: a new maximum scales what was summed by exp(m - m').
//
// One workgroup for each query row and head; DIM / 8 lanes hold a key, so a wave takes 512 / DIM
// tokens at a time, and every such group of lanes keeps its own maximum, sum and output until the
// end, when they are joined.
#include <hip/hip_runtime.h>

#include "serving.h"
#include "serving_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void codes8(const int8_t* at, float* x) {
  const uint2 w = *(const uint2*)at;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
}

template <int BF16, int DIM>
__global__ void __launch_bounds__(kThreads) kv_attention_row_kernel(KvAttentionCall a, int page_shift) {
  constexpr int kLanes = DIM / 8, kGroups = kThreads / kLanes;
  __shared__ float part[kGroups][DIM + 2];
  const gptq_kv_batch& b = a.b;
  const int head = blockIdx.x % a.a.q_heads;
  const int64_t row = blockIdx.x / a.a.q_heads;
  const int kv_head = head / (a.a.q_heads / a.c.kv_heads);
  const int seq = find_sequence(b.batch, row, [&](int i) { return (int64_t)b.cu[i]; });
  const int64_t place = row - b.cu[seq], n = (int64_t)b.cu[seq + 1] - b.cu[seq];
  const int64_t qpos = (int64_t)b.at[seq] - n + place;
  int64_t end = b.at[seq];
  if (a.a.causal && qpos + 1 < end) end = qpos + 1;
  const int64_t room = (int64_t)b.table_width << page_shift;
  if (end > room) end = room;
  if (place < 0 || place >= b.max_rows) end = 0;
  int64_t begin = a.a.window > 0 && qpos - a.a.window + 1 > 0 ? qpos - a.a.window + 1 : 0;

  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  float q[8], acc[8], m = -__builtin_inff(), l = 0.0f;
  const uint16_t* qp = a.q + row * a.a.q_stride + head * DIM + lane * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = to_f32<BF16>(qp[e]) * a.a.scale;
    acc[e] = 0.0f;
  }
  for (int64_t j = begin + group; j < end; j += kGroups) {
    const int64_t page = b.page_table[(int64_t)seq * b.table_width + (j >> page_shift)];
    if (page < 0 || page >= a.c.num_pages) continue;
    const int64_t unit = page * a.c.kv_heads + kv_head;
    const int64_t at = ((unit << page_shift) + (j & ((1 << page_shift) - 1))) * DIM + lane * 8;
    float k[8], v[8], s = 0.0f;
    codes8(a.c.k_codes + at, k);
    codes8(a.c.v_codes + at, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += q[e] * k[e];
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) s += __shfl_xor(s, d);
    s *= a.c.k_scale[unit];
    const float top = __builtin_fmaxf(m, s);
    const float keep = __expf(m - top), p = __expf(s - top);
    const float pv = p * a.c.v_scale[unit];
    l = l * keep + p;
    m = top;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = acc[e] * keep + pv * v[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[group][lane * 8 + e] = acc[e];
  if (lane == 0) {
    part[group][DIM] = m;
    part[group][DIM + 1] = l;
  }
  __syncthreads();
  if (threadIdx.x >= DIM) return;
  float top = -__builtin_inff();
  for (int g = 0; g < kGroups; ++g) top = __builtin_fmaxf(top, part[g][DIM]);
  float sum = 0.0f, o = 0.0f;
  for (int g = 0; g < kGroups; ++g) {
    if (part[g][DIM + 1] == 0.0f) continue;   // saw nothing
    const float w = __expf(part[g][DIM] - top);
    sum += w * part[g][DIM + 1];
    o += w * part[g][threadIdx.x];
  }
  a.out[row * a.a.out_stride + head * DIM + threadIdx.x] = from_f32<BF16>(sum != 0.0f ? o / sum : 0.0f);
}

}  // namespace

static bool few_rows(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  return (int64_t)b.max_rows * (a.q_heads / c.kv_heads) <= 64;
}

size_t kv_attention_ws_bytes(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  return few_rows(c, b, a) ? kv_decode_ws_bytes(c, b, a) : 0;
}

hipError_t launch_kv_attention(const KvAttentionCall& a, hipStream_t s) {
  if (few_rows(a.c, a.b, a.a)) return launch_kv_decode(a, s);
  const int page_shift = __builtin_ctz(a.c.page_size);
  const int64_t blocks = a.b.rows * a.a.q_heads;
  if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)blocks), block(kThreads);
  const bool bf16 = a.a.dtype == GPTQ_BF16;
  if (a.c.head_dim == 128) {
    if (bf16) kv_attention_row_kernel<1, 128><<<grid, block, 0, s>>>(a, page_shift);
    else kv_attention_row_kernel<0, 128><<<grid, block, 0, s>>>(a, page_shift);
  } else {
    if (bf16) kv_attention_row_kernel<1, 64><<<grid, block, 0, s>>>(a, page_shift);
    else kv_attention_row_kernel<0, 64><<<grid, block, 0, s>>>(a, page_shift);
  }
  return hipGetLastError();
}

}  // namespace gq
