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

// Whether a launch can number its threads.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= 0x7fffffff && blocks * threads <= 0xffffffffLL; }

struct KvAppendCall {
  gptq_kv_cache c;
  gptq_kv_batch b;
  const uint16_t *k, *v, *q;     // q NULL: no queries to rotate
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  uint16_t* q_out;
  int32_t q_heads, bf16;
  gptq_rope rope;                // dim 0: no rotation
};
bool kv_append_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, int q_heads);
hipError_t launch_kv_append(const KvAppendCall& a, hipStream_t s);
bool kv_read_fits(const gptq_kv_cache& c, const gptq_kv_batch& b);
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
// Whether units of 16 (row, head) columns are few and short enough for a workgroup each (kv_decode.hip).
inline bool kv_local(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const int64_t columns = (int64_t)b.max_rows * (a.q_heads / c.kv_heads);
  const int64_t units = (int64_t)b.batch * c.kv_heads * ((columns + 15) / 16);
  // A CU alone takes in some 50 GB/s, so short units only; fewer than 64 leave most of the card idle in
  // exchange for the second launch (4.6 us of the device, 2.7 of the host).  Us on the device, local
  // against split, 8 kv heads of 128, codes not in the caches: 1 sequence of 128 tokens 6.4 / 9.3, 256: 7.8 /
  // 9.4, 512: 10.1 / 10.2, 777: 11.9 / 11.8, 1024: 12.3 / 10.8, 2048: 17.2 / 11.4 (in the caches 512: 8.8 / 9.3,
  // 777: 11.2 / 10.2, 1024: 11.0 / 9.1; a call among others, the host's launches counted, 777: 11.6 to 12.0 /
  // 11.9, 1000: 11.5 to 12.5 / 11.7); 16 sequences of 512: 11.1 / 15.8, 1024: 13.8 / 19.3, 2048: 21.5 / 23.9,
  // 4096: 35.2 / 33.2; 64 sequences of 512: 23.3 / 21.2 (two workgroups for each CU take turns).  Heads of 64
  // leave room for two workgroups on a CU; 384 of them, 700 tokens: 14.7 / 17.3, 1000: 17.5 / 19.8, 2000: 26.5 /
  // 26.8.  Several units for a sequence and kv head, local against what else would run, 4 query heads each: 1
  // sequence of 16 rows, 777 tokens 12.7 / 17.2; 4 of 8 rows 12.7 / 22.8; 8 of 16 rows, 1500 tokens 21.6 / 31.9;
  // one of 64 rows, 1500 tokens 17.2 / 34.0; one prompt of 64 7.1 / 9.2; 400 units, heads of 64, a prompt of 200:
  // 9.8 / 8.8.
  const int64_t most = units < 64 ? 256 << 10 : units <= 256 ? 512 << 10 : 160 << 10;
  return units <= (columns <= 16 ? 256 * 128 / c.head_dim : 256) && (kv_span(c, b, a) + 46) / 32 * 64 * c.head_dim <= most;
}
// Few rows a sequence (kv_decode.hip): split over the keys, joined by a second launch.
bool kv_decode_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a);
size_t kv_decode_ws_bytes(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a);
hipError_t launch_kv_decode(const KvAttentionCall& a, hipStream_t s);
// Many rows a sequence (kv_prefill.hip).
bool kv_prefill_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a);
hipError_t launch_kv_prefill(const KvAttentionCall& a, hipStream_t s);

struct LoraCall {
  gptq_lora_bank bank;
  const uint16_t *x, *y;
  const int32_t* ids;
  int64_t M;
  uint16_t* out;
  void* ws;
};
bool lora_fits(const gptq_lora_bank& bank, int64_t M);
size_t lora_ws_bytes(const gptq_lora_bank& bank, int64_t M);
hipError_t launch_lora(const LoraCall& a, hipStream_t s);

}  // namespace gq
