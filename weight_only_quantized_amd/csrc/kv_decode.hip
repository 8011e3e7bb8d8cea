// Attention over the paged 8-bit cache for few query rows a sequence (single tokens, drafts).
//
// Mathematics.  For the queries c of one sequence and kv head and its visible tokens j,
//     t_cj = log2(e) scale k_scale(j) <q_c, kc_j> + log2 v_scale(j),    w_cj = 2^(t_cj - m_c),
//     out_c = sum_j w_cj vc_j / sum_j w_cj / v_scale(j),
// in one pass: the value scale rides in the exponent, so every weight that multiplies codes is
// relative to the column's largest contribution, whatever the pages' scales are, and the sum of
// probabilities takes the scale out again.  m_c only moves when a weight would pass 2^14 (then what
// was summed is scaled by 2^(m - m')), so the usual step has no cross-lane work.
//
// What bounds it: the cache's bytes.  MFMA operands are float16: codes are exact integers (the byte
// is spliced under an exponent that makes one unit 1, then the offset is subtracted), q is exact
// after a power-of-two scaling of its row, and a weight keeps 11 bits down to 2^-20 of the largest
// one: the one rounding below 32 bits, of the size of the output's own.
//
// Split.  One workgroup takes up to 32 (row, head) columns of one sequence and kv head over a run of
// tokens; its four waves take 32 tokens each in turn and join at the end through LDS.  Long runs
// are split over workgroups whose unnormalised sums a second launch joins in order.  Products are
// computed as rows = tokens, columns = queries (v_mfma_f32_16x16x32_f16), which leaves each lane
// with the weights of just those tokens whose values it holds as the second product's operand:
// codes go from memory to the matrix cores without LDS.
#include <hip/hip_runtime.h>

#include "kv_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kStep = 32;                          // tokens of a wave's step: two tiles of 16
constexpr int kStride = kStep * kWaves;            // tokens of a workgroup's step
constexpr int kMaxRun = 64 / 2 * kStride;          // a wave holds its tiles' pages one a lane

struct DecodePlan {
  int col_tiles;    // 16-column tiles of a workgroup: 1 or 2
  int col_groups;   // workgroups for a sequence and kv head's columns
  int splits;       // runs of `run` tokens
  int run;
};

// Tokens [lo, hi) that some column of a column group sees; lo at a tile.
struct GroupRange {
  int columns;             // of the sequence and kv head
  int64_t lo, hi;
  KeyRange first, last;    // of the group's first and last row
};
__device__ __forceinline__ GroupRange group_range(const SeqRows& s, const KvAttentionCall& a, const DecodePlan& plan,
                                                  int first_col, int page_shift) {
  const int group = a.a.q_heads / a.c.kv_heads;
  GroupRange r;
  r.columns = s.rows * group;
  const int width = 16 * plan.col_tiles;
  const int last_col = first_col + width < r.columns ? first_col + width - 1 : r.columns - 1;
  const int64_t room = key_room(a.b, a.a, page_shift);
  r.first = key_range(s, first_col / group, a.a, room);
  r.last = key_range(s, last_col / group, a.a, room);
  r.lo = r.first.begin & ~(int64_t)15;
  r.hi = r.last.end;
  const int64_t most = r.lo + (int64_t)plan.run * plan.splits;      // never past what was planned
  r.hi = r.hi < most ? r.hi : most;
  return r;
}

template <int BF16, int DIM, int CT>
__global__ void __launch_bounds__(kThreads, CT == 1 ? 3 : 2)
    kv_decode_kernel(KvAttentionCall a, DecodePlan plan, int page_shift) {
  constexpr int KL = DIM / 64;      // 16-byte loads of a lane for a tile's keys
  constexpr int VB = DIM / 16;      // bytes of a value row that a lane holds, one for each output tile
  constexpr int VW = VB / 4;
  constexpr int kPitch = DIM + 4;   // of a column's sums in LDS and memory
  __shared__ __align__(16) float sums[kWaves][16][kPitch];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col16 = lane & 15, quad = lane >> 4;
  int id = blockIdx.x;
  const int kv_head = id % a.c.kv_heads;
  id /= a.c.kv_heads;
  const int first_col = id % plan.col_groups * (16 * CT);
  id /= plan.col_groups;
  const int seq = id % a.b.batch, split = id / a.b.batch;

  const SeqRows s = sequence_rows(a.b, seq);
  const int group = a.a.q_heads / a.c.kv_heads;
  if (first_col >= s.rows * group) return;
  const GroupRange g = group_range(s, a, plan, first_col, page_shift);
  const int64_t run0 = g.lo + (int64_t)split * plan.run;
  if (split > 0 && run0 >= g.hi) return;
  const int64_t run1 = g.hi < run0 + plan.run ? g.hi : run0 + plan.run;
  const bool alone = g.lo + plan.run >= g.hi;      // no other run of these columns has tokens
  const int64_t room = key_room(a.b, a.a, page_shift);

  // the wave's tiles, one a lane
  const int steps = run1 > run0 ? (int)((run1 - run0 + kStride - 1) / kStride) : 0;
  const int64_t my_pos = run0 + ((lane >> 1) * kWaves + wave) * kStep + (lane & 1) * 16;
  const TilePage mine = tile_page(a.c, a.b, seq, kv_head, my_pos, my_pos < run1, page_shift);
  const float my_log = scale_log(mine.v_scale), my_inv = scale_inv(my_log);

  // this lane's columns: visible tokens and the query (columns past the last repeat it)
  int begin[CT], end[CT];
  float q_scale[CT], top[CT], total[CT];
  f16x8 q[CT][2 * KL];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    int c = first_col + ct * 16 + col16;
    c = c < g.columns ? c : g.columns - 1;
    const int row = c / group, head = kv_head * group + c % group;
    const KeyRange r = key_range(s, row, a.a, room);
    begin[ct] = (int)r.begin;
    end[ct] = (int)r.end;
    const uint16_t* at = a.q + (s.row0 + row) * a.a.q_stride + head * DIM + quad * 16;
    q_scale[ct] = load_query<BF16, 2 * KL>(at, [](int i) { return (i >> 1) * 64 + (i & 1) * 8; }, q[ct], 16, 32) *
                  (a.a.scale * kLog2e);
    top[ct] = kNoTop;
    total[ct] = 0.0f;
  }
  const int inner_lo = (int)g.last.begin, inner_hi = (int)g.first.end;   // all columns see these tokens

  f32x4 acc[CT][VB];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int t = 0; t < VB; ++t) acc[ct][t] = f32x4{0, 0, 0, 0};

  struct Step {
    u32x4 k[2][KL];
    uint32_t v[2][4][VW];
  };
  const uint32_t k_off = col16 * DIM + quad * 16, v_off = quad * 4 * DIM + col16 * VB;
  auto load = [&](Step& d, int i) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint64_t base = tile_base(a.c, __builtin_amdgcn_readlane(mine.page, 2 * i + t), kv_head,
                                      (int)run0 + (i * kWaves + wave) * kStep + t * 16, page_shift);
      const int8_t *kb = a.c.k_codes + base, *vb = a.c.v_codes + base;
#pragma unroll
      for (int j = 0; j < KL; ++j) d.k[t][j] = *(const u32x4*)(kb + k_off + j * 64);
#pragma unroll
      for (int e = 0; e < 4; ++e) __builtin_memcpy(d.v[t][e], __builtin_assume_aligned(vb + v_off + e * DIM, VB), VB);
    }
  };
  auto compute = [&](const Step& d, int i) {
    const int pos = (int)run0 + (i * kWaves + wave) * kStep;
    f32x4 dot[2][CT];
    float ks[2], lv[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) dot[t][ct] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        const f16x8 k0 = __builtin_bit_cast(f16x8, codes_f16(d.k[t][j][0], d.k[t][j][1]));
        const f16x8 k1 = __builtin_bit_cast(f16x8, codes_f16(d.k[t][j][2], d.k[t][j][3]));
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          dot[t][ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[ct][2 * j], dot[t][ct], 0, 0, 0);
          dot[t][ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[ct][2 * j + 1], dot[t][ct], 0, 0, 0);
        }
      }
      ks[t] = lane_f32(mine.k_scale, 2 * i + t);
      lv[t] = lane_f32(my_log, 2 * i + t);
    }
    const bool edge = pos < inner_lo || pos + kStep > inner_hi;     // some column does not see the whole step
    float x[2][4];
    // x = the exponents of column tile ct's weights relative to `from`; returns the largest
    auto exponents = [&](int ct, float from) {
      float most = -__builtin_inff();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[t][e] = __builtin_fmaf(dot[t][ct][e], q_scale[ct] * ks[t], lv[t] - from);
          if (edge) {
            const int p = pos + t * 16 + quad * 4 + e;
            if (p < begin[ct] || p >= end[ct]) x[t][e] = -__builtin_inff();
          }
          most = __builtin_fmaxf(most, x[t][e]);
        }
      return most;
    };
    f16x8 w[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (__any(exponents(ct, top[ct]) > kGrow)) {
        float most = exponents(ct, 0.0f);
        most = __builtin_fmaxf(most, __shfl_xor(most, 16));
        most = __builtin_fmaxf(most, __shfl_xor(most, 32));         // the four lanes of a column agree
        if (most - top[ct] > kGrow) {
          const float moved = most - kAbove, keep = __builtin_amdgcn_exp2f(top[ct] - moved);
          top[ct] = moved;
          total[ct] *= keep;
#pragma unroll
          for (int t = 0; t < VB; ++t) acc[ct][t] *= keep;
        }
        (void)exponents(ct, top[ct]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float rv = lane_f32(my_inv, 2 * i + t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(x[t][e]);
          total[ct] = __builtin_fmaf(p, rv, total[ct]);
          w[ct][t * 4 + e] = (_Float16)p;
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
    }
  };

  Step even, odd;
  if (steps > 0) load(even, 0);
  for (int i = 0; i < steps; i += 2) {
    if (i + 1 < steps) load(odd, i + 1);
    compute(even, i);
    if (i + 1 < steps) {
      if (i + 2 < steps) load(even, i + 2);
      compute(odd, i + 1);
    }
  }

  // join the four waves, one column tile at a time: output tile t of lane (col16, quad) holds values
  // VB * (4 quad + e) + t
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    if (ct) __syncthreads();
    float sum = total[ct];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    float* mine_sums = sums[wave][col16];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int t = 0; t < VB; t += 4)
        *(f32x4*)(mine_sums + VB * (4 * quad + e) + t) =
            f32x4{acc[ct][t][e], acc[ct][t + 1][e], acc[ct][t + 2][e], acc[ct][t + 3][e]};
    if (quad == 0) {
      mine_sums[DIM] = top[ct];
      mine_sums[DIM + 1] = sum;
    }
    __syncthreads();
    constexpr int kPer = DIM / 16;                 // values of a thread: 16 threads a column
    const int c = first_col + ct * 16 + (int)(threadIdx.x >> 4), d0 = (threadIdx.x & 15) * kPer;
    if (c < g.columns) {
      float most = kNoTop, all = 0.0f, o[kPer];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) most = __builtin_fmaxf(most, sums[w][threadIdx.x >> 4][DIM]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* from = sums[w][threadIdx.x >> 4];
        const float keep = __builtin_amdgcn_exp2f(from[DIM] - most);
        all = __builtin_fmaf(from[DIM + 1], keep, all);
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = __builtin_fmaf(from[d0 + e], keep, o[e]);
      }
      const int64_t row = s.row0 + c / group;
      const int head = kv_head * group + c % group;
      if (alone) {
        const float inv = all != 0.0f ? 1.0f / all : 0.0f;
        uint16_t* to = a.out + row * a.a.out_stride + head * DIM + d0;
        uint32_t packed[kPer / 2];
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e)
          packed[e] = (uint32_t)from_f32<BF16>(o[2 * e] * inv) | (uint32_t)from_f32<BF16>(o[2 * e + 1] * inv) << 16;
        __builtin_memcpy(__builtin_assume_aligned(to, kPer * 2), packed, kPer * 2);
      } else {
        float* to = (float*)a.ws + ((row * a.a.q_heads + head) * plan.splits + split) * kPitch;
#pragma unroll
        for (int e = 0; e < kPer; e += 4) *(f32x4*)(to + d0 + e) = f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]};
        if (d0 == 0) {
          to[DIM] = most;
          to[DIM + 1] = all;
        }
      }
    }
  }
}

// out = the runs' sums joined in order, one wave for a row and head (those that were split only).
template <int BF16, int DIM>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(KvAttentionCall a, DecodePlan plan, int page_shift) {
  constexpr int kPitch = DIM + 4, kPer = DIM / 64;
  const int64_t wave = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int64_t row = wave / a.a.q_heads;
  if (row >= a.b.rows) return;
  const int head = (int)(wave % a.a.q_heads), group = a.a.q_heads / a.c.kv_heads;
  const int seq = find_sequence(a.b.batch, row, [&](int i) { return (int64_t)a.b.cu[i]; });
  const SeqRows s = sequence_rows(a.b, seq);
  const int64_t place = row - s.row0;
  if (place < 0 || place >= s.rows) return;
  const int width = 16 * plan.col_tiles, c = (int)place * group + head % group;
  const GroupRange g = group_range(s, a, plan, c / width * width, page_shift);
  const int64_t runs = (g.hi - g.lo + plan.run - 1) / plan.run;
  if (runs <= 1) return;
  const float* part = (const float*)a.ws + (row * a.a.q_heads + head) * plan.splits * kPitch;
  float most = kNoTop;
  for (int i = lane; i < runs; i += 64) most = __builtin_fmaxf(most, part[(int64_t)i * kPitch + DIM]);
#pragma unroll
  for (int d = 32; d; d >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, d));
  float all = 0.0f, o[kPer] = {};
#pragma unroll 4
  for (int i = 0; i < runs; ++i) {
    const float* from = part + (int64_t)i * kPitch;
    const float keep = __builtin_amdgcn_exp2f(from[DIM] - most);
    all = __builtin_fmaf(from[DIM + 1], keep, all);
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = __builtin_fmaf(from[lane * kPer + e], keep, o[e]);
  }
  const float inv = all != 0.0f ? 1.0f / all : 0.0f;
  uint16_t* to = a.out + row * a.a.out_stride + head * DIM + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; ++e) to[e] = from_f32<BF16>(o[e] * inv);
}

// Runs: enough workgroups to fill the card (256 CUs, three workgroups each) a few times over, but no
// run shorter than a workgroup's step.
DecodePlan plan_of(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  DecodePlan p;
  const int64_t columns = (int64_t)b.max_rows * (a.q_heads / c.kv_heads);
  p.col_tiles = columns <= 16 ? 1 : 2;
  p.col_groups = (int)((columns + 16 * p.col_tiles - 1) / (16 * p.col_tiles));
  const int64_t room = (int64_t)b.table_width * c.page_size;
  int64_t span = a.max_kv < room ? a.max_kv : room;
  if (a.window > 0 && (int64_t)a.window + b.max_rows + 16 < span) span = (int64_t)a.window + b.max_rows + 16;
  if (span < 1) span = 1;
  const int64_t units = (int64_t)b.batch * c.kv_heads * p.col_groups;
  const int64_t steps = (span + kStride - 1) / kStride;
  int64_t want = (2048 + units - 1) / units;
  if (want > steps) want = steps;
  int64_t per = (steps + want - 1) / want;
  if (per > kMaxRun / kStride) per = kMaxRun / kStride;
  p.run = (int)per * kStride;
  p.splits = (int)((span + 15 + p.run - 1) / p.run);          // a range starts at a tile: up to 15 more
  return p;
}

}  // namespace

size_t kv_decode_ws_bytes(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const DecodePlan p = plan_of(c, b, a);
  if (p.splits == 1) return 0;
  return ((size_t)b.rows * a.q_heads * p.splits * (c.head_dim + 4) * 4 + 255) / 256 * 256;
}

template <int BF16, int DIM>
static hipError_t launch_dim(const KvAttentionCall& a, const DecodePlan& p, int page_shift, hipStream_t s) {
  const int64_t blocks = (int64_t)a.b.batch * a.c.kv_heads * p.col_groups * p.splits;
  const int64_t joins = (a.b.rows * a.a.q_heads + kWaves - 1) / kWaves;
  if (blocks > 0x7fffffff || joins > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (p.col_tiles == 1) kv_decode_kernel<BF16, DIM, 1><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(a, p, page_shift);
  else kv_decode_kernel<BF16, DIM, 2><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(a, p, page_shift);
  if (p.splits > 1) kv_join_kernel<BF16, DIM><<<dim3((uint32_t)joins), dim3(kThreads), 0, s>>>(a, p, page_shift);
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
