// Attention over the paged 8-bit cache for many query rows a sequence (prompts and their chunks).
//
// Mathematics as in kv_decode.hip: weights are powers of two relative to a column's top that moves
// only when a weight would pass 2^14, the value scale rides in the exponent, operands are float16
// (codes and queries exact, weights rounded once to 11 bits, of the size of a float16 output's own rounding;
// the rest of them in products of its own would cost 8192 tokens 788 us instead of 565, chunks of five
// prompts 202 instead of 155), sums float32.
//
// What bounds it: instruction issue, the matrix cores' and the vector units' together (a weight costs
// a fused multiply-add, a maximum, an exponential, a sum and a conversion; a code four operations to
// become float16).  One workgroup takes 32 (row, head) columns a wave of one sequence and kv head, the
// heads that share keys side by side, so one conversion of a tile's codes serves them all; each
// wave holds its columns' queries and outputs in registers (v_mfma_f32_32x32x16_f16, rows = tokens or
// output values, columns = queries, so a weight never leaves its lane).  A step takes 64 tokens:
// the waves turn their shares into float16 and put them into LDS, keys two steps ahead and values
// one, while the products of the next tile's scores run under this tile's exponentials and the
// products with the values under the next tile's exponents.  One barrier a step.
//
// Measured: one prompt of 8192 tokens, 32 query heads of 128 on 8 kv heads: 540 to 577 us, 953 to 1018 TFLOP/s of
// the 1275 that a large float16 product reaches; chunks of five prompts (115 GFLOP): 142 to 155 us.  The matrix
// cores are busy 47 % of the time, the vector units 57 %, LDS 35 %; waves wait for their turn to issue 28 % and
// for memory, LDS or the barrier 28 %.  An earlier form (594 us) took 317 us without reads of operands, with
// them 484 without staging, barrier and the test for hidden tokens, which cost 90, 30 and 38.  A wave with
// twice the columns (half the operand reads, one wave a SIMD): 667.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kv_dev.h"

namespace gq {
namespace {

constexpr int kTile = 64;                 // tokens of a step
typedef float f32x16 __attribute__((ext_vector_type(16)));

// First column slot of sequence b: its rows' columns / width, and one for each sequence before.
__device__ __forceinline__ int64_t slot_edge(const gptq_kv_batch& b, int seq, int group, int width) {
  return (int64_t)b.cu[seq] * group / width + seq;
}

template <int BF16, int DIM, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 2) kv_prefill_kernel(KvAttentionCall a, int slots, int page_shift) {
  constexpr int KS = DIM / 16;            // 16-value steps of a score
  constexpr int DT = DIM / 32;            // 32-value tiles of an output
  constexpr int kWidth = 32 * WAVES;      // columns
  // a wave's share of a tile: kShare tokens' keys in KL 16-byte loads a lane; the values of the quads of
  // tokens that it takes, VB bytes of four rows a lane
  constexpr int kShare = kTile / WAVES, KL = kShare * DIM / 1024;
  constexpr int VB = DIM * kShare / 256, VW = VB / 4, kGroups = DIM / VB;
  static_assert(KL >= 1 && VW >= 1 && kGroups * VB == DIM, "");
  // LDS rows of 16-byte chunks, one chunk longer than their data: eight rows' chunks cover all banks.
  // keys: token by value; values: value by token, row kGroups e + v holds value VB v + e
  constexpr int kKeyPitch = DIM / 8 + 1, kValuePitch = kTile / 8 + 1;
  __shared__ __align__(16) u32x4 keys[2][kTile * kKeyPitch];
  __shared__ __align__(16) u32x4 values[2][DIM * kValuePitch];
  // [tile & 3][key scale, log2 value scale, inverse][16 tokens]; 64 more where lanes write that have nothing
  // to write (a branch would cut the step: 8192 tokens 597 -> 590 us)
  __shared__ __align__(16) float scales[48 + 64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col32 = lane & 31, half = lane >> 5;
  const int kv_head = blockIdx.x % a.c.kv_heads;
  const int slot = slots - 1 - (int)(blockIdx.x / a.c.kv_heads);       // later rows see more: first
  const int group = a.a.q_heads / a.c.kv_heads;
  const int seq = find_sequence(a.b.batch, slot, [&](int i) { return slot_edge(a.b, i, group, kWidth); });
  const SeqRows s = sequence_rows(a.b, seq);
  const int columns = s.rows * group;
  const int64_t nth = slot - slot_edge(a.b, seq, group, kWidth);
  if (nth < 0 || nth * kWidth >= columns) return;
  const int first_col = (int)nth * kWidth;
  const int room = key_room(a.b, a.a, page_shift);
  const int last_col = first_col + kWidth < columns ? first_col + kWidth - 1 : columns - 1;
  const int lo = key_range(s, first_col / group, a.a, room).begin & ~15;
  const int hi = key_range(s, last_col / group, a.a, room).end;
  const int steps = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;

  // this lane's column (columns past the last repeat it)
  const int wave_col = first_col + wave * 32;
  const int col = wave_col + col32 < columns ? wave_col + col32 : columns - 1;
  const int row = col / group, head = kv_head * group + col % group;
  f16x8 q[KS];
  const float q_scale =
      load_query<BF16, KS>(a.q + (int64_t)(s.row0 + row) * a.a.q_stride + head * DIM + half * 8,
                           [](int i) { return i * 16; }, q, 32, 0) * (a.a.scale * kLog2e);
  float top = kNoTop, total = 0.0f;
  // tokens that all of the wave's columns see
  const int wave_last = wave_col + 32 <= columns ? wave_col + 31 : columns - 1;
  const int inner_lo = key_range(s, wave_last / group, a.a, room).begin;
  const int inner_hi = key_range(s, (wave_col < columns ? wave_col : columns - 1) / group, a.a, room).end;

  // staging: a wave's tokens lie in the 16 from 16 * part on; lane u of page, k_scale
  // and v_log holds tokens [16 u, 16 u + 16) of a run of 16 tiles (log2 of the value scale once a run: its
  // few instructions in every step cost 8192 tokens 558 us instead of 555)
  constexpr int kSplit = 16 / kShare;     // waves that share 16 tokens
  const int part = wave / kSplit, in_part = wave % kSplit;
  auto pages_of = [&](int run) {
    const int pos = lo + run * 1024 + lane * 16;
    return marked(tile_scales(a.c, tile_page_id(a.c, a.b, seq, pos, pos < hi, page_shift), kv_head));
  };
  TilePage next_pages = pages_of(0);
  const float ref = scale_reference(next_pages.v_scale);
  int page = next_pages.page;
  float k_scale = next_pages.k_scale, v_log = scale_log(next_pages.v_scale, ref);
  next_pages = pages_of(1);
  // keys: a row by neighbouring lanes (lanes that each read their own row cost the address unit a
  // cycle a lane); the piece of 16 codes in k_codes[p] is of row key_row + p * 1024 / DIM
  constexpr int kPieces = DIM / 16;
  const int key_row = in_part * kShare + lane / kPieces, key_piece = lane % kPieces;
  const uint32_t k_off = in_part * kShare * DIM + lane * 16;
  // values: tokens 4 v_quad .. + 3 of the 16 (quads q and q + 2 are halves of a chunk: sixteen lanes that
  // write together take eight groups of both), values VB v_group .. + VB - 1
  const int v_quad = kSplit == 1 ? (lane >> 5 & 1) | (lane >> 3 & 1) << 1 : in_part | (lane >> 3 & 1) << 1;
  const int v_group = kSplit == 1 ? (lane & 7) | (lane >> 4 & 1) << 3 : (lane & 7) | (lane >> 4 & 3) << 3;
  const uint32_t v_off = v_quad * 4 * DIM + v_group * VB;
  u32x4 k_codes[KL];
  uint32_t v_codes[4][VW];
  uint64_t k_base = 0;                    // of the tile in k_codes; its scales
  float st_k = 0.0f, st_log = 0.0f;
  auto turn_pages = [&](int j) {          // before tile j's keys are loaded
    if (!(j & 15)) {
      page = next_pages.page;
      k_scale = next_pages.k_scale;
      v_log = scale_log(next_pages.v_scale, ref);
      next_pages = pages_of((j >> 4) + 1);
    }
  };
  auto load_keys = [&](int j) {
    const int u = (j & 15) * 4 + part;
    k_base = tile_base(a.c, __builtin_amdgcn_readlane(page, u), kv_head, lo + j * kTile + part * 16, page_shift);
    st_k = lane_f32(k_scale, u);
    st_log = lane_f32(v_log, u);
    const int8_t* kb = a.c.k_codes + k_base;
#pragma unroll
    for (int p = 0; p < KL; ++p) k_codes[p] = *(const u32x4*)(kb + k_off + p * 1024);
  };
  auto load_values = [&](uint64_t base) {
    const int8_t* vb = a.c.v_codes + base;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t* at = (const uint32_t*)(vb + v_off + e * DIM);
      if constexpr (VW == 2) {
        const uint2 two = *(const uint2*)at;
        v_codes[e][0] = two.x;
        v_codes[e][VW - 1] = two.y;
      } else {
        v_codes[e][0] = at[0];
      }
    }
  };
  auto store_scales = [&](int j) {        // of the tile in k_codes
    const float inverse = scale_inv(st_log, ref);
    float one = st_k;
    one = lane == 1 ? st_log : one;
    one = lane == 2 ? inverse : one;
    const int to = lane < 3 && in_part == 0 ? (j & 3) * 12 + lane * 4 + part : 48 + lane;
    scales[to] = one;
  };
  auto store_key = [&](int j, int p) {
    u32x4* to = keys[j & 1] + (part * 16 + key_row + p * (1024 / DIM)) * kKeyPitch + key_piece * 2;
    to[0] = codes_f16(k_codes[p][0], k_codes[p][1]);
    to[1] = codes_f16(k_codes[p][2], k_codes[p][3]);
  };
  const int v_chunk = 2 * part + (v_quad & 1);
  auto store_value = [&](int j, int e) {
    const uint2 w{pair_f16(v_codes[0][e >> 2], v_codes[1][e >> 2], e & 3), pair_f16(v_codes[2][e >> 2], v_codes[3][e >> 2], e & 3)};
    ((uint2*)(values[j & 1] + (kGroups * e + v_group) * kValuePitch + v_chunk))[v_quad >> 1] = w;
  };

  f32x16 acc[DT], dot[2];
#pragma unroll
  for (int t = 0; t < DT; ++t) acc[t] = f32x16{};

  // operand of micro-step m of a tile's scores (tokens 32 (m / KS) .., values 16 (m % KS) ..); element e
  // of the result is token 32 (m / KS) + 8 (e / 4) + 4 half + e % 4
  auto key_at = [&](int j, int m) {
    return keys[j & 1][(m / KS * 32 + col32) * kKeyPitch + 2 * (m % KS) + half];
  };
  // operand of micro-step m of the output (value rows 32 (m / 4) .., tokens 16 (m % 4) ..)
  auto value_at = [&](int j, int m) {
    return values[j & 1][(m / 4 * 32 + col32) * kValuePitch + 2 * (m % 4) + half];
  };
  auto score_step = [&](int m, u32x4 key) {
    dot[m / KS] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, key), q[m % KS],
                                                         m % KS ? dot[m / KS] : f32x16{}, 0, 0, 0);
  };
  auto score = [&](int j) {
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m) score_step(m, key_at(j, m));
  };
  float x[2][16], most;
  auto scale4 = [&](int j, int field) { return *(const f32x4*)(scales + (j & 3) * 12 + field * 4); };
  // settles x of tile j, from its scores: hidden tokens, and a top that has to move
  auto settle = [&](int j) {
    const int pos = lo + j * kTile;
    const bool edge = pos < inner_lo || pos + kTile > inner_hi;
    if (__builtin_expect(!edge && !__any(most > kGrow), 1)) return;
    const KeyRange r = key_range(s, row, a.a, room);
    float m = -__builtin_inff();
    const f32x4 ks = scale4(j, 0), log = scale4(j, 1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float by = q_scale * ks[u];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = pos + u * 16 + (e >> 2) * 8 + half * 4 + (e & 3);
        const float v = __builtin_fmaf(dot[u >> 1][(u & 1) * 8 + e], by, log[u]);
        x[u >> 1][(u & 1) * 8 + e] = p < r.begin || p >= r.end ? -__builtin_inff() : v;
        m = __builtin_fmaxf(m, x[u >> 1][(u & 1) * 8 + e]);
      }
    }
    m = __builtin_fmaxf(m, __shfl_xor(m, 32));                       // the two lanes of a column agree
    if (m - top > kGrow) {
      const float moved = m - kAbove, keep = __builtin_amdgcn_exp2f(top - moved);
      top = moved;
      total *= keep;
#pragma unroll
      for (int t = 0; t < DT; ++t) acc[t] *= keep;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[h][e] -= top;
  };

  // Step i: LDS holds keys of tile i + 1 and values of tile i, registers the keys of tile i + 2 and the
  // values of tile i + 1, x tile i's exponents, inv its inverse scales.  Micro-steps of one operand keep
  // the vector work between the matrix instructions; a fence after each keeps the order.  Nothing is read
  // from LDS shortly before its use: operands run through a ring, kAhead ahead and over the middle of the
  // step.  Scores stay until the next step, which settles them (test for hidden tokens and tops) while its
  // first operands are on their way (8192 tokens: 594 -> 570 us; a window of 1000 over 4096: 98 -> 89).
  f32x4 inv;
  auto step = [&](int i, auto more) {
    constexpr bool kMore = decltype(more)::value;
    constexpr int kAhead = WAVES == 4 && DIM == 128 ? 2 : 3, kKeys = kMore ? 2 * KS : 0, kOut = 4 * DT;
    constexpr int kPer = 32 / (2 * KS);           // weights of a micro-step
    u32x4 ring[kAhead];
    auto operand = [&](int n) { return n < kKeys ? key_at(i + 1, n) : value_at(i, n - kKeys); };
    f16x8 w[4];
    f32x4 ks, log;
#pragma unroll
    for (int m = 0; m < kAhead; ++m) ring[m] = operand(m);
    // waves of this phase before those of the next (us: five chunks 155.6 -> 151.6, heads of 64 110 -> 107.7,
    // one of 2048 57.1 -> 58.6)
    __builtin_amdgcn_s_setprio(1);
    settle(i);                                    // while these are on their way
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m) {
      if constexpr (kMore) {
        score_step(m, ring[m % kAhead]);
        ring[m % kAhead] = operand(m + kAhead);
      }
      const int u = m * kPer / 8;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = m * kPer % 8 + k;
        const float p = __builtin_amdgcn_exp2f(x[u >> 1][(u & 1) * 8 + e]);
        total = __builtin_fmaf(p, inv[u], total);    // in 32 bits: small against the top may be large here
        w[u][e] = (_Float16)p;
      }
      asm volatile("" : "+v"(total));                // here, not after the step
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    if constexpr (kMore) {
      most = -__builtin_inff();
      ks = scale4(i + 1, 0);
      log = scale4(i + 1, 1);
      inv = scale4(i + 1, 2);
    }
    constexpr int kPerOut = 32 / kOut;
    float by, plus;
#pragma unroll
    for (int m = 0; m < kOut; ++m) {
      constexpr int kFrom = kKeys;
      acc[m / 4] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, ring[(kFrom + m) % kAhead]), w[m % 4],
                                                          acc[m / 4], 0, 0, 0);
      if (m + kAhead < kOut) ring[(kFrom + m) % kAhead] = operand(kFrom + m + kAhead);
      if constexpr (kMore) {
        const int u = m * kPerOut / 8;
        if (m * kPerOut % 8 == 0) {
          by = q_scale * ks[u];
          plus = log[u] - top;
        }
#pragma unroll
        for (int k = 0; k < kPerOut; ++k) {
          const int e = (u & 1) * 8 + m * kPerOut % 8 + k;
          x[u >> 1][e] = __builtin_fmaf(dot[u >> 1][e], by, plus);
          most = __builtin_fmaxf(most, x[u >> 1][e]);
        }
        if (m < VB) store_value(i + 1, m);
        else if (m < VB + KL) store_key(i + 2, m - VB);
        else if (m == VB + KL) {
          load_values(k_base);
          load_keys(i + 3);
        } else if (m == VB + KL + 1) {
          store_scales(i + 3);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (steps > 0) {
    load_keys(0);
    load_values(k_base);
    store_scales(0);
#pragma unroll
    for (int p = 0; p < KL; ++p) store_key(0, p);
    load_keys(1);
#pragma unroll
    for (int e = 0; e < VB; ++e) store_value(0, e);
    load_values(k_base);
    store_scales(1);
#pragma unroll
    for (int p = 0; p < KL; ++p) store_key(1, p);
    load_keys(2);
    store_scales(2);
    __syncthreads();
    score(0);
    most = __builtin_inff();               // the first tile always settles
    inv = scale4(0, 2);
  }
  for (int i = 0; i + 1 < steps; ++i) {
    turn_pages(i + 3);
    __syncthreads();
    step(i, std::true_type{});
  }
  if (steps > 0) {
    __syncthreads();
    step(steps - 1, std::false_type{});
  }

  const float sum = total + __shfl_xor(total, 32);
  if (wave_col + col32 >= columns) return;
  const float norm = sum != 0.0f ? 1.0f / sum : 0.0f, back = __builtin_amdgcn_exp2f(ref);
  uint16_t* to = a.out + (int64_t)(s.row0 + row) * a.a.out_stride + head * DIM;
  // element e of tile t is LDS row 32 t + 8 (e / 4) + 4 half + e % 4, which is value VB (row % kGroups) +
  // row / kGroups: of one e the tiles (and, with 16 groups, element e + 8) are values next to each other
  constexpr int kBoth = kGroups == 16 ? 2 : 1;
#pragma unroll
  for (int e = 0; e < 16 / kBoth; ++e) {
    uint32_t o[VB / 2];
#pragma unroll
    for (int t = 0; t < VB / 2; ++t) {
      const float v0 = kBoth == 2 ? acc[t][e] : acc[2 * t % DT][e], v1 = kBoth == 2 ? acc[t % DT][(e + 8) % 16] : acc[(2 * t + 1) % DT][e];
      o[t] = (uint32_t)from_f32<BF16>(v0 * norm * back) | (uint32_t)from_f32<BF16>(v1 * norm * back) << 16;
    }
    __builtin_memcpy(__builtin_assume_aligned(to + VB * (8 * (e >> 2) + 4 * half + (e & 3)), VB * 2), o, VB * 2);
  }
}

int64_t column_slots(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a, int waves) {
  return b.rows * (a.q_heads / c.kv_heads) / (32 * waves) + b.batch;
}

template <int BF16, int DIM, int WAVES>
hipError_t launch_waves(const KvAttentionCall& a, int page_shift, hipStream_t s) {
  const int64_t slots = column_slots(a.c, a.b, a.a, WAVES), blocks = slots * a.c.kv_heads;
  kv_prefill_kernel<BF16, DIM, WAVES><<<dim3((uint32_t)blocks), dim3(64 * WAVES), 0, s>>>(a, (int)slots, page_shift);
  return hipGetLastError();
}

// Waves of a workgroup (heads of 128).  Eight share the conversion of a tile: with two workgroups for every CU
// or more (us, 8 waves / 4, 32 heads: 8192 tokens 561 / 609, 4096: 152 / 167); the smaller workgroups fill the
// card better before (3000 tokens 96 / 95, 2048: 64 / 60).
int waves_of(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  return c.head_dim == 128 && b.rows * a.q_heads >= 256 * 512 ? 8 : 4;
}

}  // namespace

bool kv_prefill_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const int waves = waves_of(c, b, a);
  return grid_fits(column_slots(c, b, a, waves) * c.kv_heads, 64 * waves);
}

hipError_t launch_kv_prefill(const KvAttentionCall& a, hipStream_t s) {
  const int page_shift = __builtin_ctz(a.c.page_size);
  const bool bf16 = a.a.dtype == GPTQ_BF16;
  if (a.c.head_dim == 64) return bf16 ? launch_waves<1, 64, 4>(a, page_shift, s) : launch_waves<0, 64, 4>(a, page_shift, s);
  if (waves_of(a.c, a.b, a.a) == 8)
    return bf16 ? launch_waves<1, 128, 8>(a, page_shift, s) : launch_waves<0, 128, 8>(a, page_shift, s);
  return bf16 ? launch_waves<1, 128, 4>(a, page_shift, s) : launch_waves<0, 128, 4>(a, page_shift, s);
}

}  // namespace gq
