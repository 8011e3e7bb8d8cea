// Device helpers of attention over the paged 8-bit cache.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serving.h"
#include "serving_dev.h"

namespace gq {

// A column's weights are powers of two relative to a top that moves only when one would pass
// 2^kGrow; it then moves to kAbove below the largest.  Both keep weights inside float16's normal
// range (2^-14 .. 2^16) down to 2^-20 of the largest.
constexpr float kGrow = 14.0f, kAbove = 6.0f;
constexpr float kNoTop = -1e30f;          // finite, so that hidden tokens (-inf) never meet -inf
constexpr float kLog2e = 1.44269504088896f;

// Rows of a sequence in a batch; a sequence whose rows leave the packed tensors has none.  Rows and
// tokens count in 32 bits (at most 2^24 rows and 2^30 tokens of table are taken).
struct SeqRows {
  int row0;
  int rows;      // handled: at most max_rows
  int length;    // tokens in the cache
  int before;    // position of row 0: negative when there are more rows than tokens
};
__device__ __forceinline__ SeqRows sequence_rows(const gptq_kv_batch& b, int seq) {
  const int r0 = b.cu[seq], r1 = b.cu[seq + 1], at = b.at[seq], length = at > 0 ? at : 0;
  const bool good = r0 >= 0 && r1 > r0 && r1 <= b.rows;
  const int n = good ? r1 - r0 : 0;
  return SeqRows{r0, n < b.max_rows ? n : b.max_rows, length, length - n};
}

// Tokens past the table's width or the stated largest length are absent.
__device__ __forceinline__ int key_room(const gptq_kv_batch& b, const gptq_attention& a, int page_shift) {
  const int room = b.table_width << page_shift;
  return a.max_kv < room ? a.max_kv : room;
}

// Tokens [begin, end) that row `row` sees; begin <= end.
struct KeyRange {
  int begin, end;
};
__device__ __forceinline__ KeyRange key_range(const SeqRows& s, int row, const gptq_attention& a, int room) {
  const int at = s.before + row;
  int end = s.length < room ? s.length : room;
  if (a.causal && at + 1 < end) end = at + 1;
  if (end < 0) end = 0;
  int begin = a.window > 0 && at >= a.window ? at - a.window + 1 : 0;
  if (begin > end) begin = end;
  return KeyRange{begin, end};
}

// The page of a tile of 16 tokens, one a lane, and its scales for one kv head, in parts for callers that
// have other loads to send between them: the page (-1: absent), and its scales (page 0's for an absent tile;
// `marked` makes them 0 and -1).  No branches.
struct TilePage {
  int page;
  float k_scale, v_scale;
};
__device__ __forceinline__ int tile_page_id(const gptq_kv_cache& c, const gptq_kv_batch& b, int seq, int pos, bool wanted,
                                            int page_shift) {
  const int j = pos >> page_shift;
  const bool in = wanted && pos >= 0 && j < b.table_width;
  const int page = b.page_table[(int64_t)seq * b.table_width + (in ? j : 0)];
  return in && page >= 0 && page < c.num_pages ? page : -1;
}
__device__ __forceinline__ TilePage tile_scales(const gptq_kv_cache& c, int page, int kv_head) {
  const int64_t unit = (int64_t)(page < 0 ? 0 : page) * c.kv_heads + kv_head;
  return TilePage{page, c.k_scale[unit], c.v_scale[unit]};
}
__device__ __forceinline__ TilePage marked(const TilePage& t) {
  return TilePage{t.page, t.page < 0 ? 0.0f : t.k_scale, t.page < 0 ? -1.0f : t.v_scale};
}
// Bytes before a tile's codes (page 0's for an absent tile, which is safe to read).
__device__ __forceinline__ uint64_t tile_base(const gptq_kv_cache& c, int page, int kv_head, int pos, int page_shift) {
  const uint64_t unit = (uint64_t)(page < 0 ? 0 : page) * (uint32_t)c.kv_heads + (uint32_t)kv_head;
  return ((unit << page_shift) + (uint32_t)(pos & ((1 << page_shift) - 1))) * (uint32_t)c.head_dim;
}
__device__ __forceinline__ float lane_f32(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// Sums of probabilities are kept times 2^ref: a weight 2^(t + log v) stands for the probability
// 2^(t + log v) 2^(ref - log v).  float32 holds such sums for value scales of 2^(ref - 80) (2^80, weights
// of 2^14 and 2^30 tokens make 2^124) up to 2^(ref + 118).  ref lies 19 below the first value scale that is
// not zero (of marked tiles, one a lane), so that scales within 2^99 of that one keep their bits, and between
// -79 and 41, so that those of 2^-39 .. 2^39 always do (all up to 2^39 after zeros alone).
__device__ __forceinline__ float scale_reference(float v_scale) {
  const uint64_t some = __ballot(v_scale > 0.0f);
  const int bits = __builtin_amdgcn_readlane(__builtin_bit_cast(int, v_scale), some ? __builtin_ctzll(some) : 0);
  int e = some ? (bits >> 23) - 126 : -60;
  e = e < -60 ? -60 : e > 60 ? 60 : e;
  return (float)(e - 19);
}
// log2 of a value scale (subnormal ones too; zero and what lies below the range count as its end), and 2^ref
// over the scale by the same logarithm, so that both cancel; -inf and 0 when the tile is absent.
__device__ __forceinline__ float scale_log(float v_scale, float ref) {
  const float log = __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(v_scale)) + (float)__builtin_amdgcn_frexp_expf(v_scale);
  return v_scale < 0.0f ? -__builtin_inff() : __builtin_fmaxf(log, ref - 80.0f);
}
__device__ __forceinline__ float scale_inv(float v_log, float ref) {
  return v_log > -1e30f ? __builtin_amdgcn_exp2f(ref - v_log) : 0.0f;
}
// Codes to float16, exactly: byte b becomes 0x64'(b ^ 0x80) = 1024 + (code + 128), minus 1152.
__device__ __forceinline__ uint32_t less_1152(uint32_t w) {
  const f16x2 v = __builtin_bit_cast(f16x2, w) + f16x2{(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(uint32_t, v);
}
// eight codes next to each other
__device__ __forceinline__ u32x4 codes_f16(uint32_t a, uint32_t b) {
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  return u32x4{less_1152(__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)),
               less_1152(__builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)),
               less_1152(__builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)),
               less_1152(__builtin_amdgcn_perm(0x64646464u, b, 0x04030402u))};
}
// byte `byte` (0 .. 3) of two words: the codes of two tokens
__device__ __forceinline__ uint32_t pair_f16(uint32_t first, uint32_t second, int byte) {
  const uint32_t sel = 0x0c000c00u | (uint32_t)(4 + byte) << 16 | (uint32_t)byte;
  return less_1152(__builtin_amdgcn_perm(second, first, sel) ^ 0x64806480u);
}

// A query row's float16 operands, N of eight values (load_query: at at[offset(i)]), from lanes that together
// hold the row (xor `mask0`, `mask1` reach the others); returns the power of two that was taken out.
// float16 rows are exact as they are; bfloat16 rows are scaled so that the largest magnitude is in
// [2^14, 2^15), where float16 holds their 8 bits exactly down to 2^-29 of it.
template <int BF16, int N>
__device__ __forceinline__ float query_f16(const u32x4 (&w)[N], f16x8* q, int mask0, int mask1) {
  if constexpr (!BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __builtin_bit_cast(f16x8, w[i]);
    return 1.0f;
  } else {
    uint32_t most = 0;                        // magnitudes compare as integers
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[i][e] << 16 & 0x7fff0000u, hi = w[i][e] & 0x7fff0000u;
        most = most > lo ? most : lo;
        most = most > hi ? most : hi;
      }
    uint32_t other = __shfl_xor((int)most, mask0);
    most = most > other ? most : other;
    if (mask1) {
      other = __shfl_xor((int)most, mask1);
      most = most > other ? most : other;
    }
    int e = (int)(most >> 23) - 127;          // -127: zero or subnormal, 128: not finite
    e = e < -112 ? -112 : e;
    const float down = __builtin_ldexpf(1.0f, 14 - e);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[i][2 * k] = (_Float16)(__builtin_bit_cast(float, w[i][k] << 16) * down);
        q[i][2 * k + 1] = (_Float16)(__builtin_bit_cast(float, w[i][k] & 0xffff0000u) * down);
      }
    return __builtin_ldexpf(1.0f, e - 14);
  }
}
template <int BF16, int N, typename Offset>
__device__ __forceinline__ float load_query(const uint16_t* at, Offset offset, f16x8* q, int mask0, int mask1) {
  u32x4 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = *(const u32x4*)(at + offset(i));
  return query_f16<BF16, N>(w, q, mask0, mask1);
}

}  // namespace gq
