// Library-internal declarations of the serving operators: the validated calls as the launchers see
// them, and the device helpers that the paged-cache kernels share.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gptq_mi355x.h"

namespace gq {

// True when device `dev` is a gfx950 (api.cpp; looked up once per device).
bool is_gfx950_device(int dev);

struct KvAppendCall {
  gptq_kv_cache c;
  gptq_kv_batch b;
  const uint16_t *k, *v, *q;     // q NULL: no queries to rotate
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  uint16_t* q_out;
  int32_t q_heads, bf16;
  gptq_rope rope;                // dim 0: no rotation
};
hipError_t launch_kv_append(const KvAppendCall& a, hipStream_t s);
hipError_t launch_kv_read(const gptq_kv_cache& c, const gptq_kv_batch& b, void* k_out, void* v_out, int dtype,
                          hipStream_t s);

struct KvAttentionCall {
  gptq_kv_cache c;
  gptq_kv_batch b;
  gptq_attention a;
  const uint16_t* q;
  uint16_t* out;
  void* ws;
};
// Tokens that the rows of one sequence can see, at most.
inline int64_t kv_span(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const int64_t room = (int64_t)b.table_width * c.page_size, span = a.max_kv < room ? a.max_kv : room;
  const int64_t windowed = (int64_t)a.window + b.max_rows;
  return a.causal && a.window > 0 && windowed < span ? windowed : span;
}
// Few rows a sequence (kv_decode.hip): split over the keys, joined by a second launch.
size_t kv_decode_ws_bytes(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a);
hipError_t launch_kv_decode(const KvAttentionCall& a, hipStream_t s);
// Many rows a sequence (kv_prefill.hip).
hipError_t launch_kv_prefill(const KvAttentionCall& a, hipStream_t s);

struct LoraCall {
  gptq_lora_bank bank;
  const uint16_t *x, *y;
  const int32_t* ids;
  int64_t M;
  uint16_t* out;
  void* ws;
};
size_t lora_ws_bytes(const gptq_lora_bank& bank, int64_t M);
hipError_t launch_lora(const LoraCall& a, hipStream_t s);

}  // namespace gq
