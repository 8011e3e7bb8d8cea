// Low-rank adapters of many requests beside a shared projection.
//
// Mathematics: low[m] = scale_i A_i x[m] (rank values), out[m] = y[m] + B_i low[m], i = ids[m]: two
// launches, since every output needs the whole sum over K.
//
// What bounds it: bytes.  Single tokens of many requests read A_i and B_i of every adapter in use
// once; prompts read x and y and write out.  Both products run on v_mfma_f32_16x16x32 with columns =
// rows of x, straight from memory to registers: rows of A_i (or B_i) are the other operand, and the
// inner index is permuted alike on both sides so that a lane reads 32 bytes and four lanes a whole
// 128-byte line.
//
// Rows in any order: a workgroup takes 16 to 64 neighbouring rows and goes through the adapters that
// occur among them, keeping each product for its own adapter's rows (so no row meets another's
// values, not even times zero).  With few rows the adapters of a tile go to several workgroups.
//
// Sums over K are split over the waves and, with few rows, over workgroups; the parts are added in
// order by the second launch, which then takes low as two 16-bit numbers (value and remainder,
// float16 after a power-of-two scaling of the row): 16 bits or more for one more product.
#include <hip/hip_runtime.h>

#include "bufmem.h"
#include "serving.h"
#include "serving_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256, kWaves = 4;

struct LoraPlan {
  int low_tiles, low_rows;     // row tiles of the first launch, of 16 or 32 rows
  int up_tiles, up_rows;       // of the second, of 16, 32 or 64 rows
  int turns;                   // workgroups that share a tile's adapters
  int slices, wave_k;          // parts of K, each four waves of wave_k
  int blocks_n, per_n;         // workgroups over N, each per_n times 256 outputs
};

// Adapter of each row of a tile, one a lane (-1: none, or past the last row).
__device__ __forceinline__ int lane_id(const LoraCall& c, int64_t row0, int rows, int lane) {
  const int64_t row = row0 + lane;
  if (lane >= rows || row >= c.M) return -1;
  const int id = c.ids[row];
  return id >= 0 && id < c.bank.adapters ? id : -1;
}

// Calls f(adapter) for the adapters among `id`, in the order of their first rows: every turns-th
// one, starting at `turn`.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int turn, int turns, F f) {
  uint64_t left = __ballot(id >= 0);
  int nth = 0;
  while (left) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    left &= ~__ballot(id == a);
    if (nth % turns == turn) f(a);
    ++nth;
  }
}

// low: part[slice][row][rank] = the slice's share of A_i x.
template <int BF16, int RT, int CT>   // rank tiles and row tiles of 16
__global__ void __launch_bounds__(kThreads, 2) lora_low_kernel(LoraCall c, LoraPlan p) {
  constexpr int kRows = 16 * CT, kPitch = RT * 16 + 4;
  __shared__ __align__(16) float sums[kWaves][kRows][kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  int id = blockIdx.x;
  const int slice = id % p.slices;
  id /= p.slices;
  const int turn = id % p.turns;
  const int64_t row0 = (int64_t)(id / p.turns) * kRows;
  const int K = c.bank.in_features, rank = c.bank.rank;
  const int my_id = lane_id(c, row0, kRows, lane);
  const int k0 = (slice * kWaves + wave) * p.wave_k;
  const int k1 = k0 + p.wave_k < K ? k0 + p.wave_k : K;
  // rows and ranks past the last, and inputs past the slice, lie past the resources: they read as 0
  const int rows = c.M - row0 < kRows ? (int)(c.M - row0) : kRows;
  const rsrc_t x_rsrc = make_rsrc(c.x + row0 * K, (uint32_t)rows * K * 2);
  const uint32_t voff = (uint32_t)(col * K + quad * 16) * 2;
  float* part = (float*)c.ws + (int64_t)slice * c.M * rank;

  each_adapter(my_id, turn, p.turns, [&](int a) {
    const rsrc_t a_rsrc = make_rsrc((const uint16_t*)c.bank.a + (int64_t)a * rank * K, (uint32_t)rank * K * 2);
    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
    constexpr int kDeep = RT * CT <= 2 ? 4 : RT <= 4 ? 2 : 1;      // 64-value steps whose loads are in flight
    for (int k = k0; k < k1; k += 64 * kDeep) {
      u32x4 xs[kDeep][CT][2], ws[kDeep][RT][2];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const uint32_t at = k + d * 64 + quad * 16 < k1 ? voff + (uint32_t)(k + d * 64) * 2 : kOob;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int t = 0; t < CT; ++t) xs[d][t][h] = load_b128(x_rsrc, at + 16 * h + (uint32_t)(t * 16 * K) * 2, 0);
#pragma unroll
          for (int t = 0; t < RT; ++t) ws[d][t][h] = load_b128(a_rsrc, at + 16 * h + (uint32_t)(t * 16 * K) * 2, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < kDeep; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[r][t] = mfma16<BF16>(ws[d][r][h], xs[d][t][h], acc[r][t]);
    }
    __syncthreads();                                   // the last adapter's sums are read
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CT; ++t) *(f32x4*)&sums[wave][t * 16 + col][r * 16 + quad * 4] = acc[r][t];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * RT * 16; i += kThreads) {
      const int row = i / (RT * 16), r = i % (RT * 16);
      if (__shfl(my_id, row) != a || r >= rank) continue;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) s += sums[v][row][r];
      part[(row0 + row) * rank + r] = s;
    }
  });
}

// out = y + B_i low.
template <int BF16, int KS, int CT>   // 32-value steps of the rank, row tiles of 16
__global__ void __launch_bounds__(kThreads, 2) lora_up_kernel(LoraCall c, LoraPlan p) {
  constexpr int kRows = 16 * CT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  int id = blockIdx.x;
  const int block_n = id % p.blocks_n;
  id /= p.blocks_n;
  const int turn = id % p.turns;
  const int64_t row0 = (int64_t)(id / p.turns) * kRows;
  const int N = c.bank.out_features, rank = c.bank.rank;
  const int my_id = lane_id(c, row0, kRows, lane);
  const int n_first = block_n * p.per_n * 256 + wave * 64;
  int ids[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) ids[t] = __shfl(my_id, t * 16 + col);

  each_adapter(my_id, turn, p.turns, [&](int a) {
    // low of the adapter's rows (zeros elsewhere), added over the slices in order
    u32x4 high[CT][KS], rest[CT][KS];
    float back[CT];
    const float scale = c.bank.scale[a];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      float low[KS][8];
      float most = 0.0f;
      const float* from = (const float*)c.ws + (row0 + t * 16 + col) * rank + quad * 8;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        f32x4 s0{0, 0, 0, 0}, s1{0, 0, 0, 0};
        if (ids[t] == a && k * 32 + quad * 8 < rank) {
#pragma unroll 4
          for (int s = 0; s < p.slices; ++s) {
            const float* at = from + (int64_t)s * c.M * rank + k * 32;
            s0 += *(const f32x4*)at;
            s1 += *(const f32x4*)(at + 4);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          low[k][e] = s0[e] * scale;
          low[k][4 + e] = s1[e] * scale;
          most = __builtin_fmaxf(most, __builtin_fmaxf(__builtin_fabsf(low[k][e]), __builtin_fabsf(low[k][4 + e])));
        }
      }
      back[t] = 1.0f;
      float down = 1.0f;
      if constexpr (!BF16) {                           // the row's largest magnitude into [2^13, 2^14)
        most = __builtin_fmaxf(most, __shfl_xor(most, 16));
        most = __builtin_fmaxf(most, __shfl_xor(most, 32));
        int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127 - 13;
        e = e < -120 ? -120 : e > 114 ? 114 : e;
        down = __builtin_ldexpf(1.0f, -e);
        back[t] = __builtin_ldexpf(1.0f, e);
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v0 = low[k][2 * e] * down, v1 = low[k][2 * e + 1] * down;
          const uint16_t h0 = from_f32<BF16>(v0), h1 = from_f32<BF16>(v1);
          high[t][k][e] = (uint32_t)h0 | (uint32_t)h1 << 16;
          rest[t][k][e] = (uint32_t)from_f32<BF16>(v0 - to_f32<BF16>(h0)) |
                          (uint32_t)from_f32<BF16>(v1 - to_f32<BF16>(h1)) << 16;
        }
    }
    const rsrc_t b_rsrc = make_rsrc((const uint16_t*)c.bank.b + (int64_t)a * N * rank, (uint32_t)N * rank * 2);
    for (int i = 0; i < p.per_n; ++i) {
      const int n0 = n_first + i * 256;
      if (n0 >= N) break;
      // a lane's outputs are n0 + 16 quad .. + 15: row 4 q + e of tile t is output n0 + 16 q + 4 t + e
      const int n = n0 + quad * 16;
      f32x4 acc[4][CT];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t at = (uint32_t)((col >> 2) * 16 + t * 4 + (col & 3)) * rank * 2;   // past N: past the resource
        u32x4 w[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int r = k * 32 + quad * 8;
          w[k] = load_b128(b_rsrc, r < rank ? at + r * 2 : kOob, (uint32_t)n0 * rank * 2);
        }
#pragma unroll
        for (int m = 0; m < CT; ++m) {
          acc[t][m] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KS; ++k) acc[t][m] = mfma16<BF16>(w[k], high[m][k], acc[t][m]);
#pragma unroll
          for (int k = 0; k < KS; ++k) acc[t][m] = mfma16<BF16>(w[k], rest[m][k], acc[t][m]);
        }
      }
      if (n >= N) continue;
#pragma unroll
      for (int m = 0; m < CT; ++m) {
        if (ids[m] != a) continue;
        const int64_t at = (row0 + m * 16 + col) * N + n;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 in = *(const u32x4*)(c.y + at + 8 * h);
          u32x4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x4& v = acc[2 * h + (e >> 1)][m];
            o[e] = (uint32_t)from_f32<BF16>(__builtin_fmaf(v[2 * (e & 1)], back[m], to_f32<BF16>((uint16_t)in[e]))) |
                   (uint32_t)from_f32<BF16>(__builtin_fmaf(v[2 * (e & 1) + 1], back[m], to_f32<BF16>((uint16_t)(in[e] >> 16)))) << 16;
          }
          *(u32x4*)(c.out + at + 8 * h) = o;
        }
      }
    }
  });
  // rows without an adapter
  if (turn != 0 || c.out == c.y) return;
#pragma unroll
  for (int m = 0; m < CT; ++m) {
    const int64_t row = row0 + m * 16 + col;
    if (ids[m] >= 0 || row >= c.M) continue;
    for (int i = 0; i < p.per_n; ++i) {
      const int n = n_first + i * 256 + quad * 16;
      if (n >= N) break;
      *(u32x4*)(c.out + row * N + n) = *(const u32x4*)(c.y + row * N + n);
      *(u32x4*)(c.out + row * N + n + 8) = *(const u32x4*)(c.y + row * N + n + 8);
    }
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

LoraPlan plan_of(const gptq_lora_bank& bank, int64_t M) {
  LoraPlan p;
  const bool few = M <= 128;
  p.low_rows = few ? 16 : 32;
  p.up_rows = few ? 16 : bank.rank > 64 ? 32 : 64;
  p.low_tiles = (int)div_up(M, p.low_rows);
  p.up_tiles = (int)div_up(M, p.up_rows);
  int64_t turns = few ? (M < 16 ? M : 16) : 1;
  if (turns > bank.adapters) turns = bank.adapters;
  p.turns = (int)turns;
  // K: enough workgroups to fill the card, slices of at least one 64-value step a wave
  const int64_t units = p.low_tiles * turns, steps = div_up(bank.in_features, 64 * kWaves);
  int64_t slices = div_up(512, units);
  if (slices > 16) slices = 16;
  if (slices > steps) slices = steps;
  p.wave_k = (int)(div_up(steps, slices) * 64);
  p.slices = (int)div_up(bank.in_features, (int64_t)p.wave_k * kWaves);
  const int64_t blocks = div_up(bank.out_features, 256);
  int64_t per = p.up_tiles * turns * blocks / 1024;
  p.per_n = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
  if (few) p.per_n = 1;
  p.blocks_n = (int)div_up(blocks, p.per_n);
  return p;
}

template <int BF16, int RT>
void launch_low(const LoraCall& c, const LoraPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.low_tiles * p.turns * p.slices)), block(kThreads);
  if (p.low_rows == 16) lora_low_kernel<BF16, RT, 1><<<grid, block, 0, s>>>(c, p);
  else lora_low_kernel<BF16, RT, 2><<<grid, block, 0, s>>>(c, p);
}

template <int BF16, int KS>
void launch_up(const LoraCall& c, const LoraPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.up_tiles * p.turns * p.blocks_n)), block(kThreads);
  if (p.up_rows == 16) lora_up_kernel<BF16, KS, 1><<<grid, block, 0, s>>>(c, p);
  else if (KS == 4) lora_up_kernel<BF16, KS, 2><<<grid, block, 0, s>>>(c, p);
  else lora_up_kernel<BF16, KS, KS == 4 ? 2 : 4><<<grid, block, 0, s>>>(c, p);
}

template <int BF16>
hipError_t launch_type(const LoraCall& c, hipStream_t s) {
  const LoraPlan p = plan_of(c.bank, c.M);
  if ((int64_t)p.low_tiles * p.turns * p.slices > 0x7fffffff || (int64_t)p.up_tiles * p.turns * p.blocks_n > 0x7fffffff)
    return hipErrorInvalidConfiguration;
  const int rank = c.bank.rank;
  if (rank <= 16) launch_low<BF16, 1>(c, p, s);
  else if (rank <= 32) launch_low<BF16, 2>(c, p, s);
  else if (rank <= 64) launch_low<BF16, 4>(c, p, s);
  else launch_low<BF16, 8>(c, p, s);
  if (rank <= 32) launch_up<BF16, 1>(c, p, s);
  else if (rank <= 64) launch_up<BF16, 2>(c, p, s);
  else launch_up<BF16, 4>(c, p, s);
  return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(const gptq_lora_bank& bank, int64_t M) {
  return ((size_t)plan_of(bank, M).slices * M * bank.rank * 4 + 255) / 256 * 256;
}

hipError_t launch_lora(const LoraCall& c, hipStream_t s) {
  return c.bank.dtype == GPTQ_BF16 ? launch_type<1>(c, s) : launch_type<0>(c, s);
}

}  // namespace gq
