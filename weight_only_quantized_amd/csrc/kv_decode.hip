// Attention over the paged 8-bit cache with the keys split over the card: single tokens, drafts, and pieces
// of prompts that are short for the tokens they see.
//
// Mathematics.  For the queries c of one sequence and kv head and its visible tokens j,
//     t_cj = log2(e) scale k_scale(j) <q_c, kc_j> + log2 v_scale(j),    w_cj = 2^(t_cj - m_c),
//     out_c = 2^r sum_j w_cj vc_j / sum_j w_cj 2^r / v_scale(j),
// in one pass: the value scale rides in the exponent, so every weight that multiplies codes is
// relative to the column's largest contribution, whatever the pages' scales are, and the sum of
// probabilities takes the scale out again (2^r is about as large and keeps it in float32).  m_c only
// moves when a weight would pass 2^14 (then what was summed is scaled by 2^(m - m')), so the usual step
// has no cross-lane work.
//
// What bounds it: the cache's bytes.  MFMA operands are float16: codes are exact integers (the byte
// is spliced under an exponent that makes one unit 1, then the offset is subtracted), q is exact
// after a power-of-two scaling of its row.  A weight is the one rounding below 32 bits.  Units of up to
// eight columns use half of a matrix instruction's sixteen: there each column stands twice, once with its
// weights' first 11 bits and once with the rest of them, and the two sums are joined at the end: 21 bits,
// down to 2^-31 of the largest weight, for one fused multiply-add a weight (us, 11 bits / 21: one token 11.25 /
// 11.5, 64 sequences 48.4 / 48.8).  Units of up to sixteen take a second instruction for the rest (one token
// with 16 heads a kv head 12.05 / 12.25, 64 sequences of 3 drafts 95.0 / 95.2).  Wider units keep 11 bits down
// to 2^-20 of the largest weight, an error of the size of a float16 output's own rounding: they are bound by
// instructions (500 rows over 9000 tokens would take 170 us instead of 147).
//
// Split.  The work is cut into steps of 32 tokens of a unit: up to 32 (row, head) columns of one
// sequence and kv head.  All units' steps in order are dealt to as many waves as the card holds at
// once, the same number to each: sequences of any lengths fill it evenly, and no wave waits for
// another.  Units that cross waves leave unnormalised sums that a second launch joins in order.  Short
// units go to a workgroup each instead when there are few (it joins its waves' sums itself), to a wave
// each when there are many.
// Products are computed as rows = tokens, columns = queries (v_mfma_f32_16x16x32_f16), which leaves
// each lane with the weights of just those tokens whose values it holds as the second product's
// operand: values go from memory to the matrix cores without LDS.
//
// Measured (the device's time, both launches): 64 sequences of up to 4096 tokens, 8 kv heads of 128, 221
// MB: 44.5 + 5.0 us, 5.0 TB/s in the first launch; waves start their loads after 2 to 5 us and stream
// at 6.8 TB/s (a plain read of as many bytes: 6.85) until the first ends, 7 us before the last.  6
// sequences of up to 70001, 64 query heads, 325 MB: 59.6 + 6.3 us, 5.5 TB/s.  24 sequences, 5 rows each,
// a window of 2000, 16 heads of 64, 60 MB: 19.0 + 4.1 us, no unit at its limit.  1 sequence of 777 tokens, one
// launch: 11.4 us, of which a wave waits 47 % for results and 18 % for its turn to issue.  500 rows over 9000
// tokens: 141 + 10.6 us, vector units 61 % (each unit converts all codes).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "bufmem.h"
#include "kv_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kLocalWaves = 8;                     // of a workgroup that takes a whole unit: what its registers fit
constexpr int kStep = 32;                          // tokens of a step: two tiles of 16
constexpr int kMaxRun = 64 * 16;                   // a wave holds the pages of its tiles one a lane

struct DecodePlan {
  int col_tiles;    // 16-column tiles of a unit: 1 or 2
  int col_groups;   // units of a sequence and kv head, at most
  int waves, wave_bits;    // when split a power of two
  int units;        // batch * kv_heads * col_groups, at most 2^31 - 1 (kv_decode_fits refuses so many)
  int64_t steps;    // of a unit, at most
  int width;        // columns of a part: those that a unit can have
  int local;        // a workgroup of kLocalWaves takes a unit and joins it
  int split;        // units may cross waves: they leave parts; else (nor local) a wave takes a unit
  int many_parts;   // few or very long units, of some 32 parts or more: a workgroup joins them, else a wave
};

// A unit's parts, in the workspace: slots `first` to `last`, one a wave.  Wave w leaves its part of
// unit u in slot w + u, which no other pair shares since both only ascend.
struct UnitParts {
  int first, last;
};
__host__ __device__ inline size_t parts_offset(const DecodePlan& p) { return ((size_t)p.units * sizeof(UnitParts) + 255) / 256 * 256; }

// Tokens [lo, hi) that some row of a sequence sees, lo at 16, in `steps`; `groups` units of them for
// each kv head.  A sequence with rows has a step even if they see nothing (it writes zeros).
struct SeqWork {
  SeqRows s;
  int lo, hi, steps, groups;
};
template <int CT>
__device__ __forceinline__ SeqWork sequence_work(const KvAttentionCall& a, const SeqRows& s, int room) {
  SeqWork w;
  w.s = s;
  w.lo = w.hi = w.steps = w.groups = 0;
  if (w.s.rows == 0) return w;
  w.lo = key_range(w.s, 0, a.a, room).begin & ~15;
  w.hi = key_range(w.s, w.s.rows - 1, a.a, room).end;
  w.steps = w.hi > w.lo ? (w.hi - w.lo + kStep - 1) / kStep : 1;
  w.groups = (w.s.rows * (a.a.q_heads / a.c.kv_heads) + 16 * CT - 1) / (16 * CT);
  return w;
}

// Codes that few units read are not kept in the caches (64 sequences: 50.5 -> 45.0 us; one of 777 tokens 12.9 ->
// 11.9).  Where a sequence and kv head have more columns, other units read them again (a workgroup a unit, not
// kept / kept: 2 units of 16 columns, 4 sequences of 777 tokens 13.6 / 13.9 us; 4 units, 1 of 777 13.8 / 12.9; 16
// units, 1 of 800 15.2 / 13.5).
template <bool ONCE, typename T>
__device__ __forceinline__ T load_once(const T* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  else return *p;
}

// The kernel's first argument, read again: keeping all of it in scalar registers over the loop on
// units takes more than there are.
__device__ __forceinline__ KvAttentionCall call_again() {
  auto p = (const __attribute__((address_space(4))) KvAttentionCall*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const KvAttentionCall*)p;
}

// 2^ref o / sum, four values; zeros where nothing was seen.
template <int BF16>
__device__ __forceinline__ void store_joined(uint16_t* to, f32x4 o, float sum, float ref) {
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f, back = __builtin_amdgcn_exp2f(ref);
  o = o * inv * back;
  uint2 w;
  w.x = (uint32_t)from_f32<BF16>(o[0]) | (uint32_t)from_f32<BF16>(o[1]) << 16;
  w.y = (uint32_t)from_f32<BF16>(o[2]) | (uint32_t)from_f32<BF16>(o[3]) << 16;
  *(uint2*)to = w;
}

// A weight's bits in the second product: the first 11, rounded; those and the rest of them in the other eight
// columns of one matrix instruction; or in a second one.
enum { kFirstBits, kInPairs, kTwice };
template <int BF16, int DIM, int CT, bool LOCAL, bool ONCE, int BITS>
__global__ void __launch_bounds__(LOCAL ? 64 * kLocalWaves : kThreads, LOCAL && DIM == 64 ? 4 : 2)
    kv_decode_kernel(KvAttentionCall call, DecodePlan plan, int page_shift) {
  constexpr int kWaves = LOCAL ? kLocalWaves : gq::kWaves;
  constexpr int KL = DIM / 64;      // 16-byte loads of a lane for a tile's keys
  constexpr int VB = DIM / 16;      // bytes of a value row that a lane holds, one for each output tile
  constexpr int VW = VB / 4;
  constexpr int kPitch = DIM + 4;   // of a column's sums in memory
  // a wave's keys of a step: memory is read a row by neighbouring lanes (lanes that each read their
  // own row cost the address unit a cycle a lane), the product wants a row a lane.  16-byte pieces
  // of row r are stored at piece ^ kTurn(r): eight rows' pieces cover all banks.
  __shared__ __align__(16) u32x4 key_rows[kWaves][2][16 * (DIM / 16)];
  __shared__ __align__(16) float sums[LOCAL ? kWaves : 1][LOCAL ? 16 : 1][kPitch];       // of the waves' columns

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col16 = lane & 15, quad = lane >> 4;
  const int room = key_room(call.b, call.a, page_shift);
  const int group = call.a.q_heads / call.c.kv_heads;
  constexpr bool kPaired = BITS == kInPairs;
  static_assert(BITS == kFirstBits || CT == 1, "");
  const float less = col16 >= 8 ? -1.0f : 0.0f;    // columns from 8 on: what is left of a weight, negative

  // this wave's share of all steps (LOCAL: of its unit's), and the sequence where they
  // start: a scan over 64 sequences at a time, one a lane
  const int wave_id = blockIdx.x * kWaves + wave;
  SeqRows held;                                   // of sequence q + lane
  int seq = 0, skipped = 0;                       // the sequence, and its steps that come before
  int dealt = 0, full = 0;                        // its steps; of LOCAL's first waves
  const bool one_scan = !LOCAL && plan.split && call.b.batch <= 64;       // then `held` stays
  if constexpr (LOCAL) {
    const int unit = blockIdx.x % (call.c.kv_heads * plan.col_groups);
    seq = blockIdx.x / (call.c.kv_heads * plan.col_groups);
    const SeqWork work = sequence_work<CT>(call, sequence_rows(call.b, seq), room);
    if (unit >= work.groups * call.c.kv_heads) return;                       // of the whole workgroup
    full = (work.steps + kWaves - 1) / kWaves;
    skipped = unit * work.steps + wave * full;
    dealt = work.steps - wave * full < full ? work.steps - wave * full : full;
  } else if (!plan.split) {
    const int per_sequence = call.c.kv_heads * plan.col_groups, unit = wave_id % per_sequence;
    seq = wave_id / per_sequence;
    if (seq >= call.b.batch) return;
    const SeqWork work = sequence_work<CT>(call, sequence_rows(call.b, seq), room);
    if (unit >= work.groups * call.c.kv_heads) return;
    skipped = unit * work.steps;
    dealt = work.steps;
  } else {
  auto steps_of = [&](int q) {
    held = q < call.b.batch ? sequence_rows(call.b, q) : SeqRows{0, 0, 0, 0};
    const SeqWork w = sequence_work<CT>(call, held, room);
    return w.steps * w.groups * call.c.kv_heads;
  };
  int all = 0, mine = 0, upto = 0;
  if (one_scan) {
    mine = steps_of(lane);
    upto = wave_scan(mine);
    all = __builtin_amdgcn_readlane(upto, 63);
  } else {
    for (int q = 0; q < call.b.batch; q += 64) all += wave_sum(steps_of(q + lane));
  }
  // shares differ by one step, the longer ones everywhere; no wave without a step between two that have one
  const int dealers = all < plan.waves ? all : plan.waves;
  if (wave_id >= dealers) return;
  const int pos0 = dealers < plan.waves ? wave_id : (int)((int64_t)all * wave_id >> plan.wave_bits);
  dealt = (dealers < plan.waves ? wave_id + 1 : (int)((int64_t)all * (wave_id + 1) >> plan.wave_bits)) - pos0;
  for (int q = 0, before = 0; q < call.b.batch; q += 64) {
    if (!one_scan) {
      mine = steps_of(q + lane);
      upto = before + wave_scan(mine);            // steps up to and with this lane's sequence
    }
    const uint64_t past = __ballot(upto <= pos0);
    if (past != ~0ull) {
      const int at = __builtin_popcountll(past);
      seq = q + at;
      skipped = pos0 - __builtin_amdgcn_readlane(upto - mine, at);
      break;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  }
  auto rows_of = [&](int q) {
    if (!one_scan) return sequence_rows(call.b, q);
    return SeqRows{__builtin_amdgcn_readlane(held.row0, q), __builtin_amdgcn_readlane(held.rows, q),
                   __builtin_amdgcn_readlane(held.length, q), __builtin_amdgcn_readlane(held.before, q)};
  };
  int left = dealt;

  while (left > 0 && seq < call.b.batch) {
  const KvAttentionCall a = call_again();
  const SeqWork work = sequence_work<CT>(a, rows_of(seq), room);
  const SeqRows s = work.s;
  if (skipped >= work.steps * work.groups * a.c.kv_heads) {   // the next sequence (without rows: no steps)
    skipped = 0;
    ++seq;
    continue;
  }
  const int unit = skipped / work.steps, step0 = skipped % work.steps;
  const int kv_head = unit / work.groups, first_col = unit % work.groups * (16 * CT), columns = s.rows * group;
  const int steps = work.steps - step0 < left ? work.steps - step0 : left;
  const bool alone = steps == work.steps;        // the unit is all here
  const int unit_id = (seq * a.c.kv_heads + kv_head) * plan.col_groups + unit % work.groups;
  if (!LOCAL && plan.split && lane == 0) {
    if (step0 == 0) ((UnitParts*)a.ws)[unit_id].first = wave_id + unit_id;
    if (step0 + steps == work.steps) ((UnitParts*)a.ws)[unit_id].last = wave_id + unit_id;
  }
  const int run0 = work.lo + step0 * kStep;
  const int run1 = work.hi < run0 + steps * kStep ? work.hi : run0 + steps * kStep;
  const int last_col = first_col + 16 * CT < columns ? first_col + 16 * CT - 1 : columns - 1;

  // this lane's columns: visible tokens and the query (columns past the last repeat it)
  int begin[CT], end[CT];
  float q_scale[CT], top[CT], total[CT];
  f16x8 q[CT][2 * KL];
  u32x4 query[CT][2 * KL];
  auto page_id = [&](int base) {                  // 16 tokens a lane
    const int my_pos = base + lane * 16;
    return tile_page_id(a.c, a.b, seq, my_pos, my_pos < run1, page_shift);
  };
  int page = page_id(run0);                       // on its way with the query
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    int c = first_col + ct * 16 + (kPaired ? col16 & 7 : col16);
    c = c < columns ? c : columns - 1;
    const int row = c / group, head = kv_head * group + c % group;
    const KeyRange r = key_range(s, row, a.a, room);
    begin[ct] = r.begin;
    end[ct] = r.end;
    const uint16_t* at = a.q + (int64_t)(s.row0 + row) * a.a.q_stride + head * DIM + quad * 16;
#pragma unroll
    for (int i = 0; i < 2 * KL; ++i) query[ct][i] = *(const u32x4*)(at + (i >> 1) * 64 + (i & 1) * 8);
    top[ct] = kNoTop;
    total[ct] = 0.0f;
  }
  // all columns see these tokens
  const int inner_lo = key_range(s, last_col / group, a.a, room).begin;
  const int inner_hi = key_range(s, first_col / group, a.a, room).end;

  f32x4 acc[CT][VB];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int t = 0; t < VB; ++t) acc[ct][t] = f32x4{0, 0, 0, 0};

  struct Step {
    u32x4 k[2][KL];
    uint32_t v[2][4][VW];
  };
  // up to 32 steps at a time, from token `base` on: their pages, 16 tokens a lane
  int base = run0;
  TilePage pages;
  float my_log, my_inv;
  const uint32_t k_off = lane * 16, v_off = quad * 4 * DIM + col16 * VB;
  // Keys and values of a step are loaded again, for two steps ahead, as soon as they are used: up to two
  // steps of a wave are on their way (steps past the last are absent tiles: they read page 0).
  auto step_base = [&](int i, int t) {
    return tile_base(a.c, __builtin_amdgcn_readlane(pages.page, (2 * i + t) & 63), kv_head,
                     base + i * kStep + t * 16, page_shift);
  };
  auto load_keys = [&](Step& d, int i) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int8_t* kb = a.c.k_codes + step_base(i, t);
#pragma unroll
      for (int j = 0; j < KL; ++j) d.k[t][j] = load_once<ONCE>((const u32x4*)(kb + k_off + j * 1024));
    }
  };
  constexpr int kPieces = DIM / 16;               // of a key row
  auto turn = [](int row) { return DIM == 128 ? row & 7 : row >> 1 & 3; };
  const int put_row = lane / kPieces, put_at = put_row * kPieces + (lane % kPieces ^ turn(put_row));
  const int get_at = col16 * kPieces + (quad ^ turn(col16));      // piece quad; piece 4 + quad is at ^ 4
  auto load_values = [&](Step& d, int i) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int8_t* vb = a.c.v_codes + step_base(i, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (VW == 2) {
          const u32x2 w = load_once<ONCE>((const u32x2*)(vb + v_off + e * DIM));
          d.v[t][e][0] = w[0];
          d.v[t][e][VW - 1] = w[1];
        } else {
          d.v[t][e][0] = load_once<ONCE>((const uint32_t*)(vb + v_off + e * DIM));
        }
      }
    }
  };
  auto compute = [&](Step& d, int i, auto more) {
    const int pos = base + i * kStep;
    f32x4 dot[2][CT];
    float ks[2], lv[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < KL; ++j) key_rows[wave][t][put_at + j * 64] = d.k[t][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");        // the wave's LDS accesses stay in order
    if constexpr (decltype(more)::value) load_keys(d, i + 2);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) dot[t][ct] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        const u32x4 k = key_rows[wave][t][get_at ^ (j * 4)];
        const f16x8 k0 = __builtin_bit_cast(f16x8, codes_f16(k[0], k[1]));
        const f16x8 k1 = __builtin_bit_cast(f16x8, codes_f16(k[2], k[3]));
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          dot[t][ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[ct][2 * j], dot[t][ct], 0, 0, 0);
          dot[t][ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[ct][2 * j + 1], dot[t][ct], 0, 0, 0);
        }
      }
      ks[t] = lane_f32(pages.k_scale, 2 * i + t);
      lv[t] = lane_f32(my_log, 2 * i + t);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // x = the exponents of the weights relative to the columns' tops
    float x[CT][2][4], most = -__builtin_inff();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float by = q_scale[ct] * ks[t], plus = lv[t] - top[ct];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[ct][t][e] = __builtin_fmaf(dot[t][ct][e], by, plus);
          most = __builtin_fmaxf(most, x[ct][t][e]);
        }
      }
    // seldom: some column does not see the whole step, or a top has to move
    if (__builtin_expect(pos < inner_lo || pos + kStep > inner_hi || __any(most > kGrow), 0)) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float m = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = pos + t * 16 + quad * 4 + e;
            const float v = __builtin_fmaf(dot[t][ct][e], q_scale[ct] * ks[t], lv[t]);
            x[ct][t][e] = p < begin[ct] || p >= end[ct] ? -__builtin_inff() : v;
            m = __builtin_fmaxf(m, x[ct][t][e]);
          }
        m = __builtin_fmaxf(m, __shfl_xor(m, 16));
        m = __builtin_fmaxf(m, __shfl_xor(m, 32));                  // the four lanes of a column agree
        const bool moves = m - top[ct] > kGrow;
        const float to = moves ? m - kAbove : top[ct], keep = moves ? __builtin_amdgcn_exp2f(top[ct] - to) : 1.0f;
        top[ct] = to;
        total[ct] *= keep;
#pragma unroll
        for (int t = 0; t < VB; ++t) acc[ct][t] *= keep;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[ct][t][e] -= to;
      }
    }
    f16x8 w[CT], rest;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float rv = lane_f32(my_inv, 2 * i + t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(x[ct][t][e]);
          total[ct] = __builtin_fmaf(p, rv, total[ct]);
          const float first = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, p) & 0xffffe000u);
          w[ct][t * 4 + e] = (_Float16)(BITS == kFirstBits ? p : kPaired ? __builtin_fmaf(p, less, first) : first);
          if constexpr (BITS == kTwice) rest[t * 4 + e] = (_Float16)(p - first);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < VB; ++t) {
      const u32x4 v{pair_f16(d.v[0][0][t >> 2], d.v[0][1][t >> 2], t & 3), pair_f16(d.v[0][2][t >> 2], d.v[0][3][t >> 2], t & 3),
                    pair_f16(d.v[1][0][t >> 2], d.v[1][1][t >> 2], t & 3), pair_f16(d.v[1][2][t >> 2], d.v[1][3][t >> 2], t & 3)};
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        acc[ct][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), w[ct], acc[ct][t], 0, 0, 0);
      if constexpr (BITS == kTwice) acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), rest, acc[0][t], 0, 0, 0);
    }
    if constexpr (decltype(more)::value) load_values(d, i + 2);
  };

  Step even, odd;
  // a run's scales and first steps, in the order of the steps: a wait for one load waits for all before it
  auto start_run = [&] {
    pages = tile_scales(a.c, page, kv_head);
    __builtin_amdgcn_sched_barrier(0);
    load_keys(even, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_values(even, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_keys(odd, 1);
    __builtin_amdgcn_sched_barrier(0);
    load_values(odd, 1);
    __builtin_amdgcn_sched_barrier(0);
  };
  start_run();
  const float ref = scale_reference(marked(pages).v_scale);        // of this part
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) q_scale[ct] = query_f16<BF16, 2 * KL>(query[ct], q[ct], 16, 32) * (a.a.scale * kLog2e);
  for (;;) {
    const TilePage there = marked(pages);
    pages = there;
    my_log = scale_log(there.v_scale, ref);
    my_inv = scale_inv(my_log, ref);
    const int n = run1 - base < kMaxRun ? (run1 - base + kStep - 1) / kStep : kMaxRun / kStep;
    if constexpr (CT == 1) {               // pairs, so that every wait in the loop is for what it needs
      int i = 0;
      for (; i + 1 < n; i += 2) {
        // the older of a SIMD's waves would run ahead and leave the others alone at the end (64 sequences:
        // ends spread over 28 .. 43 us, now 31 .. 38): the more a wave has left, the earlier its turn
        const int togo = (left - i) * 8;
        if (togo > dealt * 4) __builtin_amdgcn_s_setprio(3);
        else if (togo > dealt * 2) __builtin_amdgcn_s_setprio(2);
        else if (togo > dealt) __builtin_amdgcn_s_setprio(1);
        else __builtin_amdgcn_s_setprio(0);
        compute(even, i, std::true_type{});
        compute(odd, i + 1, std::true_type{});
      }
      if (i < n) compute(even, i, std::false_type{});
    } else {                               // (two column tiles have no registers for the last step's copy)
      for (int i = 0; i < n; i += 2) {
        compute(even, i, std::true_type{});
        if (i + 1 < n) compute(odd, i + 1, std::true_type{});
      }
    }
    base += kMaxRun;
    if (base >= run1) break;
    page = page_id(base);
    start_run();
  }

  // output tile t of lane (col16, quad) holds values VB (4 quad + e) + t
  const KvAttentionCall e_call = call_again();
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    float sum = total[ct];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if constexpr (kPaired) {                                 // less the sums of what was left, in the lane eight on
#pragma unroll
      for (int t = 0; t < VB; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mine = acc[ct][t][e];
          acc[ct][t][e] = mine - __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, mine), 0x128, 15, 15,
                                                                                    true));      // row_ror:8
        }
      if (col16 >= 8) continue;
    }
    const int c = first_col + ct * 16 + col16;
    if (c >= columns) continue;
    if (alone) {
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f, back = __builtin_amdgcn_exp2f(ref);
      uint16_t* to = e_call.out + (int64_t)(s.row0 + c / group) * e_call.a.out_stride + (kv_head * group + c % group) * DIM;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t o[VB / 2];
#pragma unroll
        for (int t = 0; t < VB; t += 2)
          o[t / 2] = (uint32_t)from_f32<BF16>(acc[ct][t][e] * inv * back) | (uint32_t)from_f32<BF16>(acc[ct][t + 1][e] * inv * back) << 16;
        __builtin_memcpy(__builtin_assume_aligned(to + VB * (4 * quad + e), VB * 2), o, VB * 2);
      }
    } else {
      float* to = LOCAL ? sums[wave][col16]
                        : (float*)((uint8_t*)e_call.ws + parts_offset(plan)) +
                              ((int64_t)(wave_id + unit_id) * plan.width + ct * 16 + col16) * kPitch;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int t = 0; t < VB; t += 4)
          *(f32x4*)(to + VB * (4 * quad + e) + t) =
              f32x4{acc[ct][t][e], acc[ct][t + 1][e], acc[ct][t + 2][e], acc[ct][t + 3][e]};
      if (quad == 0) {
        to[DIM] = top[ct];
        to[DIM + 1] = sum;
        to[DIM + 2] = ref;
      }
    }
  }
  left -= steps;
  skipped += steps;
  }
  if constexpr (LOCAL) {
    // the waves' sums joined in order, four values of a column a thread
    const KvAttentionCall a = call_again();
    __syncthreads();
    const SeqWork work = sequence_work<CT>(a, sequence_rows(a.b, seq), room);
    const int count = (work.steps + full - 1) / full, unit = blockIdx.x % (a.c.kv_heads * plan.col_groups);
    const int kv_head = unit / work.groups, first_col = unit % work.groups * 16;
    const int c = first_col + threadIdx.x / (DIM / 4), d = threadIdx.x % (DIM / 4) * 4;
    if (count <= 1 || threadIdx.x >= 16 * (DIM / 4) || c >= work.s.rows * group) return;
    float most = kNoTop, all = 0.0f;
    f32x4 o{0, 0, 0, 0};
    for (int w = 0; w < count; ++w) most = __builtin_fmaxf(most, sums[w][c - first_col][DIM]);
    const float ref = sums[0][c - first_col][DIM + 2];
    for (int w = 0; w < count; ++w) {
      const float* from = sums[w][c - first_col];
      const float in = from[DIM] - most;
      all = __builtin_fmaf(from[DIM + 1], __builtin_amdgcn_exp2f(in + (ref - from[DIM + 2])), all);
      o += *(const f32x4*)(from + d) * __builtin_amdgcn_exp2f(in);
    }
    store_joined<BF16>(a.out + (int64_t)(work.s.row0 + c / group) * a.a.out_stride + (kv_head * group + c % group) * DIM + d, o, all, ref);
  }
}

// out = a unit's parts joined in order (those in more than one part only): THREADS for a row and
// head, DIM / 4 of them hold a part, the groups take parts in turn and join at the end.
template <int BF16, int DIM, int THREADS>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(KvAttentionCall a, DecodePlan plan) {
  constexpr int kPitch = DIM + 4, kLanes = DIM / 4, kGroups = THREADS / kLanes;
  __shared__ __align__(16) float sums[THREADS == kThreads ? kWaves : 1][kPitch];
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / THREADS;
  const int64_t row = item / a.a.q_heads;
  if (row >= a.b.rows) return;
  const int head = (int)(item % a.a.q_heads), group = a.a.q_heads / a.c.kv_heads;
  const int seq = find_sequence(a.b.batch, row, [&](int i) { return (int64_t)a.b.cu[i]; });
  const SeqRows s = sequence_rows(a.b, seq);
  const int place = (int)row - s.row0;
  if (place < 0 || place >= s.rows) return;
  const int width = 16 * plan.col_tiles, c = place * group + head % group;
  const UnitParts parts = ((const UnitParts*)a.ws)[(seq * a.c.kv_heads + head / group) * plan.col_groups + c / width];
  const int count = parts.last - parts.first + 1;
  if (count <= 1) return;
  const float* part = (const float*)((const uint8_t*)a.ws + parts_offset(plan)) +
                      ((int64_t)parts.first * plan.width + c % width) * kPitch;
  const int thread = threadIdx.x % THREADS, in_part = thread % kLanes;
  const float ref = part[DIM + 2];               // sums are joined relative to the first part's
  float most = kNoTop, all = 0.0f;
  f32x4 o{0, 0, 0, 0};
  auto join = [&](float top, float sum, float more, f32x4 v) {          // sum: times 2^more
    const float now = __builtin_fmaxf(most, top);
    const float keep = __builtin_amdgcn_exp2f(most - now), in = __builtin_amdgcn_exp2f(top - now);
    all = all * keep + sum * __builtin_amdgcn_exp2f(top - now + more);
    o = o * keep + v * in;
    most = now;
  };
#pragma unroll 4
  for (int i = thread / kLanes; i < count; i += kGroups) {
    const float* from = part + (int64_t)i * plan.width * kPitch;
    join(from[DIM], from[DIM + 1], ref - from[DIM + 2], *(const f32x4*)(from + in_part * 4));
  }
#pragma unroll
  for (int d = kLanes; d < 64; d <<= 1)
    join(__shfl_xor(most, d), __shfl_xor(all, d), 0.0f,
         f32x4{__shfl_xor(o[0], d), __shfl_xor(o[1], d), __shfl_xor(o[2], d), __shfl_xor(o[3], d)});
  if constexpr (THREADS == kThreads) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < kLanes) *(f32x4*)&sums[wave][in_part * 4] = o;
    if ((threadIdx.x & 63) == 0) {
      sums[wave][DIM] = most;
      sums[wave][DIM + 1] = all;
    }
    __syncthreads();
    if (threadIdx.x < kLanes)
#pragma unroll
      for (int w = 1; w < kWaves; ++w) join(sums[w][DIM], sums[w][DIM + 1], 0.0f, *(const f32x4*)&sums[w][in_part * 4]);
  }
  if (thread >= kLanes) return;
  store_joined<BF16>(a.out + row * a.a.out_stride + head * DIM + in_part * 4, o, all, ref);
}

// Two waves a SIMD (256 CUs), or as many as there can be steps: measured with 1, 1.5, 3 and 4 as well (221
// MB: 54, 51, 48 and 49 us against 47.8), three steps of a wave on their way instead of two: no change.
DecodePlan plan_of(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  DecodePlan p;
  const int64_t columns = (int64_t)b.max_rows * (a.q_heads / c.kv_heads);
  p.local = kv_local(c, b, a);
  p.col_tiles = columns <= 16 || p.local ? 1 : 2;
  p.width = (int)(columns < 16 * p.col_tiles ? columns : 16 * p.col_tiles);
  p.col_groups = (int)((columns + 16 * p.col_tiles - 1) / (16 * p.col_tiles));
  const int64_t steps = p.steps = (kv_span(c, b, a) + 15 + kStep - 1) / kStep;      // a range starts at 16: up to 15 more
  const int64_t all = (int64_t)b.batch * c.kv_heads * p.col_groups, units = all < 0x7fffffff ? all : 0x7fffffff;
  const int64_t fit = 256 * kWaves * 2;
  // Many short units: a wave takes a whole one, so that nothing is joined and no wave looks for its share.
  // Us, a wave a unit / split, 8 kv heads of 128, sequences of very different lengths up to: 64 of 128 8.7 /
  // 10.3, 512: 18.8 / 18.2; 128 of 64: 7.5 / 14.1, 1000: 32.9 / 32.9; 256 of 256: 18.3 / 31.7, 1500: 70 / 72,
  // 2000: 95 / 83; 16 heads of 64: 64 of 500 14.7 / 16.2, 1000: 24.3 / 20.9.
  const bool whole = steps <= 48 && steps * 32 * 128 <= units * c.head_dim;
  p.split = !p.local && steps > 1 && !whole;
  p.units = (int)units;
  p.many_parts = steps > 1024 || units < fit / 32;
  p.wave_bits = 0;
  while (1 << p.wave_bits < fit && 1 << p.wave_bits < units * steps) ++p.wave_bits;
  p.waves = p.split ? 1 << p.wave_bits : p.units;
  return p;
}

int64_t kernel_blocks(const DecodePlan& p) { return p.local ? p.units : ((int64_t)p.waves + kWaves - 1) / kWaves; }
int64_t join_blocks(const DecodePlan& p, const gptq_kv_batch& b, const gptq_attention& a) {
  return p.many_parts ? b.rows * a.q_heads : (b.rows * a.q_heads + kWaves - 1) / kWaves;
}

}  // namespace

bool kv_decode_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const DecodePlan p = plan_of(c, b, a);
  if (p.units == 0x7fffffff || !grid_fits(kernel_blocks(p), p.local ? 64 * kLocalWaves : kThreads)) return false;
  // a split call's waves count the steps of all units in 32 bits
  return !p.split || (p.steps * p.units <= 0x7fffffff && grid_fits(join_blocks(p, b, a), kThreads));
}

size_t kv_decode_ws_bytes(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const DecodePlan p = plan_of(c, b, a);
  return p.split ? parts_offset(p) + ((size_t)p.units + p.waves) * p.width * (c.head_dim + 4) * 4 : 0;
}

template <int BF16, int DIM>
static hipError_t launch_dim(const KvAttentionCall& a, const DecodePlan& p, int page_shift, hipStream_t s) {
  const dim3 grid((uint32_t)kernel_blocks(p)), block(kThreads), joins((uint32_t)join_blocks(p, a.b, a.a));
  const dim3 local(64 * kLocalWaves);
#define GQ_DECODE(CT, LOCAL, ONCE, BITS) \
  kv_decode_kernel<BF16, DIM, CT, LOCAL, ONCE, BITS><<<grid, LOCAL ? local : block, 0, s>>>(a, p, page_shift)
  if (p.local) {
    if (p.width <= 8) GQ_DECODE(1, true, true, kInPairs);
    else if (p.col_groups == 1) GQ_DECODE(1, true, true, kTwice);
    else if (p.col_groups == 2) GQ_DECODE(1, true, true, kFirstBits);
    else GQ_DECODE(1, true, false, kFirstBits);
  } else if (p.col_tiles == 1) {
    if (p.width <= 8) GQ_DECODE(1, false, true, kInPairs);
    else GQ_DECODE(1, false, true, kTwice);
  } else {
    GQ_DECODE(2, false, false, kFirstBits);
  }
#undef GQ_DECODE
  if (p.split && p.many_parts) kv_join_kernel<BF16, DIM, kThreads><<<joins, block, 0, s>>>(a, p);
  else if (p.split) kv_join_kernel<BF16, DIM, 64><<<joins, block, 0, s>>>(a, p);
  return hipGetLastError();
}

hipError_t launch_kv_decode(const KvAttentionCall& a, hipStream_t s) {
  const DecodePlan p = plan_of(a.c, a.b, a.a);
  const int page_shift = __builtin_ctz(a.c.page_size);
  if (a.c.head_dim == 128)
    return a.a.dtype == GPTQ_BF16 ? launch_dim<1, 128>(a, p, page_shift, s) : launch_dim<0, 128>(a, p, page_shift, s);
  return a.a.dtype == GPTQ_BF16 ? launch_dim<1, 64>(a, p, page_shift, s) : launch_dim<0, 64>(a, p, page_shift, s);
}

}  // namespace gq
