// Low-rank adapters of many requests beside a shared projection.
//
// Mathematics: low[m] = scale_i A_i x[m] (rank values), out[m] = y[m] + B_i low[m], i = ids[m]: two
// launches, since every output needs the whole sum over K.  Where there is little of both, one launch
// whose workgroups each compute all of low is quicker.
//
// What bounds it: bytes.  Single tokens of many requests read A_i and B_i of every adapter in use
// once; prompts read x and y and write out.  Both products run on v_mfma_f32_16x16x32 with columns =
// rows of x, straight from memory to registers: rows of A_i (or B_i) are the other operand.
//
// Rows in any order.  Up to 1024 rows (tokens of many requests): a workgroup takes up to sixteen rows
// of one adapter, gathered from wherever they stand among 128.  More (prompts): a wave or workgroup takes
// 32 or 64 neighbouring rows and goes through the adapters that occur among them, keeping each product
// for its own adapter's rows (so no row meets another's values, not even times zero).
//
// Sums over K are split: with few rows over the waves of a workgroup and over workgroups, whose
// parts the second launch adds in order; with many rows over workgroups only, whose waves take
// different rows and meet in the first-level cache over A_i, and a small launch in between adds the
// parts once.  low goes into the second product as two 16-bit numbers (value and remainder, float16
// after a power-of-two scaling of the row, its remainder times 2^11): 16 bits or more of each value that is
// 2^-33 of its row's largest or more, for one more product.
//
// Measured (the device's time): 1 row, rank 16, 4096 x 14336, one launch: 7.8 us, most of it two trips to
// memory and the pass over A_i.  61 rows of 48 adapters, rank 32, 8192 x 28672 (86 MB): 7.0 + 15.9 us, 4.3
// TB/s in the second launch.  4001 rows in 9 runs, rank 64, 4096 x 14336 (271 MB): 12.5 + 4.7 + 58.5 us, 3.9
// TB/s of y and out against 4.9 of a copy.
#include <hip/hip_runtime.h>

#include "bufmem.h"
#include "serving.h"
#include "serving_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256, kWaves = 4;

constexpr int kManyRows = 32;  // rows of a wave of the first launch when there are many

struct LoraPlan {
  bool few;                    // few rows: adapters of a tile over workgroups, low added by its readers
  int groups;                  // few: groups of a chunk's rows, at most
  int low_tiles;               // tiles of the first launch: groups, or 4 * kManyRows rows
  int up_tiles;                // of the second: groups, or 32 or 64 rows
  bool here;                   // few and small: one launch, each workgroup computes low itself
  int slices, slice_k;         // parts of K
  int blocks_n, per_n;         // workgroups over N, each per_n times 256 outputs
  size_t part_bytes;           // of the parts; then low's two numbers and the rows' powers of two
};

// Adapter of each row of a tile, one a lane (-1: none, or past the last row).
__device__ __forceinline__ int lane_id(const LoraCall& c, int64_t row0, int rows, int lane) {
  const int64_t row = row0 + lane;
  if (lane >= rows || row >= c.M) return -1;
  const int id = c.ids[row];
  return id >= 0 && id < c.bank.adapters ? id : -1;
}

// Calls f(adapter) for the adapters among `id`, in the order of their first rows.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, F f) {
  uint64_t left = __ballot(id >= 0);
  while (left) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    left &= ~__ballot(id == a);
    f(a);
  }
}

// Few rows, in chunks of kChunk: up to sixteen rows of one adapter, which need not be neighbours, make a
// group.  (Chunks of 256 read an adapter less often, but looking for groups among so many, and the code
// for it, cost all calls: rank 64, 4096 x 14336, us with 128 / 256: 4 rows 11.3 / 12.1, 256 in runs 19.5 /
// 19.9, 256 of 48 adapters 47 / 38.)
constexpr int kChunk = 128;
struct RowGroup {
  int adapter;    // -1: there is no such group
  int row;        // within the chunk, of place lane & 15, -1: none
};
// Group `nth` of rows [row0, row0 + rows), in the order of the rows that open one: the 1st, 17th, .. of each
// adapter's.  rows <= 64 PARTS.
template <int PARTS>
__device__ __forceinline__ RowGroup group_among(const LoraCall& c, int64_t row0, int rows, int lane, int nth) {
  int id[PARTS];
#pragma unroll
  for (int h = 0; h < PARTS; ++h) id[h] = lane_id(c, row0 + h * 64, rows - h * 64, lane);
  // same[h][g]: rows 64 g + .. that have the adapter of this lane's row 64 h + lane
  const uint64_t below = (1ull << lane) - 1;
  uint64_t same[PARTS][PARTS];
#pragma unroll
  for (int h = 0; h < PARTS; ++h)
#pragma unroll
    for (int g = 0; g <= h; ++g) same[h][g] = __ballot(id[g] >= 0);
  for (int bit = 0; (c.bank.adapters - 1) >> bit; ++bit)
#pragma unroll
    for (int g = 0; g < PARTS; ++g) {
      const uint64_t set = __ballot(id[g] >> bit & 1);
#pragma unroll
      for (int h = g; h < PARTS; ++h) same[h][g] &= id[h] >> bit & 1 ? set : ~set;
    }
  int rank[PARTS], opened = 0, a = -1, first = 0;
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    rank[h] = __builtin_popcountll(same[h][h] & below);
#pragma unroll
    for (int g = 0; g < h; ++g) rank[h] += __builtin_popcountll(same[h][g]);
    const bool opens = id[h] >= 0 && rank[h] % 16 == 0;
    const uint64_t open = __ballot(opens), it = __ballot(opens && opened + __builtin_popcountll(open & below) == nth);
    opened += __builtin_popcountll(open);
    if (it) {
      a = __builtin_amdgcn_readlane(id[h], __builtin_ctzll(it));
      first = __builtin_amdgcn_readlane(rank[h], __builtin_ctzll(it));
    }
  }
  if (a < 0) return RowGroup{-1, -1};
  // each row's lane sends it to the lane of its place (others to lane 63, which nobody reads)
  int row = -1, before = 0;
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    const bool mine = id[h] == a && rank[h] >= first && rank[h] < first + 16;
    const int from = __builtin_amdgcn_ds_permute((mine ? rank[h] - first : 63) * 4, h * 64 + lane);
    const int n = __builtin_popcountll(__ballot(mine));
    row = lane >= before && lane < before + n ? from : row;
    before += n;
  }
  return RowGroup{a, __shfl(row, lane & 15)};
}
__device__ __forceinline__ RowGroup row_group(const LoraCall& c, int64_t row0, int rows, int lane, int nth) {
  if (rows > 64) return group_among<2>(c, row0, rows, lane, nth);
  if (rows > 16) return group_among<1>(c, row0, rows, lane, nth);
  // a row's place is its number
  const int id = lane_id(c, row0, rows, lane);
  for (uint64_t left = __ballot(id >= 0); left; --nth) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    if (nth == 0) return RowGroup{a, __shfl(id, lane & 15) == a ? lane & 15 : -1};
    left &= ~__ballot(id == a);
  }
  return RowGroup{-1, -1};
}

// Memory is read a row by neighbouring lanes, 64 inputs (128 bytes) by eight of them: lanes that each
// read their own row cost the address unit a cycle a lane.  The products want a row a lane: rows pass
// through the wave's own LDS, 16-byte piece p of row r stored at p ^ (r & 7), so that eight rows'
// pieces cover all banks.
template <int RT, int CT>
constexpr int kStage = (RT + CT) * 16 * 8;         // 16-byte pieces of a wave's x rows, then A rows

// acc = A_i x over inputs [k0, k1) for CT tiles of 16 rows: ranks 16 r + 4 quad + e of row 16 t + col.
// x_at[n]: bytes before this lane's piece of row 8 n + lane / 8 (kOob: none; it stays past every resource).  Absent rows, ranks past the
// last and inputs past k1 read as 0.
template <int BF16, int RT, int CT>
__device__ __forceinline__ void low_product(rsrc_t x_rsrc, const uint32_t (&x_at)[2 * CT], rsrc_t a_rsrc, int K, int k0, int k1,
                                            int lane, u32x4* stage, f32x4 (&acc)[RT][CT]) {
  const int col = lane & 15, quad = lane >> 4, piece = lane & 7;
  const uint32_t voff = (uint32_t)((lane >> 3) * K + piece * 8) * 2, next = (uint32_t)(8 * K) * 2;
  const int put = (lane >> 3) * 8 + (piece ^ (lane >> 3)), get = col * 8 + (quad ^ (col & 7));
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < CT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
  constexpr int kDeep = RT + CT <= 3 ? 4 : RT + CT <= 6 ? 2 : 1;   // steps of 64 whose loads are in flight
  u32x4 xs[kDeep][2 * CT], ws[kDeep][2 * RT];
  auto load = [&](int d, int k) {
    const bool in = k + piece * 8 < k1;
    const uint32_t at = in ? voff + (uint32_t)k * 2 : kOob;
#pragma unroll
    for (int n = 0; n < 2 * CT; ++n) xs[d][n] = load_b128(x_rsrc, in ? x_at[n] + (uint32_t)k * 2 : kOob, 0);
#pragma unroll
    for (int n = 0; n < 2 * RT; ++n) ws[d][n] = load_b128(a_rsrc, at + n * next, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // where registers allow, a step's operands are read while the step before is multiplied (first: zeros)
  constexpr bool kLate = RT + CT <= 3;
  u32x4 xr[2][CT], wr[2][RT];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int t = 0; t < CT; ++t) xr[h][t] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < RT; ++r) wr[h][r] = u32x4{0, 0, 0, 0};
  }
  auto multiply = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[r][t] = mfma16<BF16>(wr[h][r], xr[h][t], acc[r][t]);
  };
#pragma unroll
  for (int d = 0; d < kDeep; ++d) load(d, k0 + d * 64);
  for (int k = k0; k < k1; k += 64 * kDeep)
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
#pragma unroll
      for (int n = 0; n < 2 * CT; ++n) stage[put + n * 64] = xs[d][n];
#pragma unroll
      for (int n = 0; n < 2 * RT; ++n) stage[CT * 128 + put + n * 64] = ws[d][n];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");       // the wave's LDS accesses stay in order
      load(d, k + (d + kDeep) * 64);
      u32x4 xn[2][CT], wn[2][RT];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < CT; ++t) xn[h][t] = stage[t * 128 + (get ^ h * 4)];
#pragma unroll
        for (int r = 0; r < RT; ++r) wn[h][r] = stage[CT * 128 + r * 128 + (get ^ h * 4)];
      }
      if constexpr (kLate) multiply();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < CT; ++t) xr[h][t] = xn[h][t];
#pragma unroll
        for (int r = 0; r < RT; ++r) wr[h][r] = wn[h][r];
      }
      if constexpr (!kLate) multiply();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  if constexpr (kLate) multiply();
}

__device__ __forceinline__ rsrc_t adapter_a(const LoraCall& c, int a) {
  const int64_t n = (int64_t)c.bank.rank * c.bank.in_features;
  return make_rsrc((const uint16_t*)c.bank.a + a * n, (uint32_t)n * 2);
}

// x offsets of a lane's two rows (low_product) from the row of lane & 15.
struct RowOffsets {
  uint32_t at[2];
};
__device__ __forceinline__ RowOffsets row_offsets(int my_row, int lane, int K) {
  RowOffsets o;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int row = __shfl(my_row, n * 8 + (lane >> 3));
    o.at[n] = row < 0 ? kOob : (uint32_t)(row * K + (lane & 7) * 8) * 2;
  }
  return o;
}

// Few rows: part[slice][row][rank] = the slice's share of A_i x, the slice's K over the four waves.
template <int BF16, int RT>   // rank tiles of 16
__global__ void __launch_bounds__(kThreads, 2) lora_low_kernel(LoraCall c, LoraPlan p) {
  constexpr int kPitch = RT * 16 + 4;
  __shared__ u32x4 stage[kWaves][kStage<RT, 1>];
  float (*const sums)[16][kPitch] = (float (*)[16][kPitch])stage;     // of the waves, in the same place
  static_assert(sizeof(float) * kWaves * 16 * kPitch <= sizeof(stage), "");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = blockIdx.x % p.slices;
  const int K = c.bank.in_features, rank = c.bank.rank;
  const int k0 = slice * p.slice_k + wave * (p.slice_k / kWaves);
  const int k1 = k0 + p.slice_k / kWaves < K ? k0 + p.slice_k / kWaves : K;
  const int tile_id = blockIdx.x / p.slices;
  const int chunk = c.M <= kChunk ? 0 : tile_id / p.groups;
  const int64_t row0 = (int64_t)chunk * kChunk;
  const int rows = c.M - row0 < kChunk ? (int)(c.M - row0) : kChunk;
  const rsrc_t x_rsrc = make_rsrc(c.x + row0 * K, (uint32_t)rows * K * 2);
  float* part = (float*)c.ws + ((int64_t)slice * c.M + row0) * rank;
  const RowGroup g = row_group(c, row0, rows, lane, tile_id - chunk * p.groups);
  if (g.adapter < 0) return;
  f32x4 acc[RT][1];
  low_product<BF16>(x_rsrc, row_offsets(g.row, lane, K).at, adapter_a(c, g.adapter), K, k0, k1, lane, stage[wave], acc);
  __syncthreads();                                     // all waves have read their rows
#pragma unroll
  for (int r = 0; r < RT; ++r) *(f32x4*)&sums[wave][lane & 15][r * 16 + (lane >> 4) * 4] = acc[r][0];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RT * 16; i += kThreads) {
    const int at = i / (RT * 16), r = i % (RT * 16), row = __shfl(g.row, at);
    if (row < 0 || r >= rank) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) s += sums[v][at][r];
    part[(int64_t)row * rank + r] = s;
  }
}

// Many rows: the same, each wave its own kManyRows rows over all of the slice.
template <int BF16, int RT>
__global__ void __launch_bounds__(kThreads, 2) lora_low_rows_kernel(LoraCall c, LoraPlan p) {
  constexpr int CT = kManyRows / 16;
  __shared__ u32x4 stage[kWaves][kStage<RT, CT>];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = blockIdx.x % p.slices;
  const int64_t row0 = ((int64_t)(blockIdx.x / p.slices) * kWaves + wave) * kManyRows;
  if (row0 >= c.M) return;
  const int K = c.bank.in_features, rank = c.bank.rank;
  const int my_id = lane_id(c, row0, kManyRows, lane);
  const int k0 = slice * p.slice_k, k1 = k0 + p.slice_k < K ? k0 + p.slice_k : K;
  const int rows = c.M - row0 < kManyRows ? (int)(c.M - row0) : kManyRows;
  const rsrc_t x_rsrc = make_rsrc(c.x + row0 * K, (uint32_t)rows * K * 2);
  float* part = (float*)c.ws + ((int64_t)slice * c.M + row0) * rank;
  uint32_t x_at[2 * CT];
#pragma unroll
  for (int n = 0; n < 2 * CT; ++n) x_at[n] = (uint32_t)((n * 8 + (lane >> 3)) * K + (lane & 7) * 8) * 2;
  each_adapter(my_id, [&](int a) {
    f32x4 acc[RT][CT];
    low_product<BF16>(x_rsrc, x_at, adapter_a(c, a), K, k0, k1, lane, stage[wave], acc);
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const int row = t * 16 + (lane & 15);
      const bool mine = __shfl(my_id, row) == a;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int at = r * 16 + (lane >> 4) * 4;
        if (mine && at < rank) *(f32x4*)(part + row * rank + at) = acc[r][t];
      }
    }
  });
}

// low of eight ranks: the slices' parts in order, times the adapter's scale.
__device__ __forceinline__ void add_parts(const float* from, int slices, int64_t apart, float scale, float* low) {
  f32x4 s0{0, 0, 0, 0}, s1{0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < slices; ++s) {
    s0 += *(const f32x4*)(from + s * apart);
    s1 += *(const f32x4*)(from + s * apart + 4);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    low[e] = s0[e] * scale;
    low[4 + e] = s1[e] * scale;
  }
}
__device__ __forceinline__ float largest8(const float* v) {
  float most = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) most = __builtin_fmaxf(most, __builtin_fabsf(v[e]));
  return most;
}
// The power of two that takes a float16 row's largest magnitude into [2^13, 2^14).
__device__ __forceinline__ int row_exponent(float most) {
  const int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127 - 13;
  return e < -120 ? -120 : e > 114 ? 114 : e;
}
// low * down as value and remainder (0 beside an infinity).  float16's remainder is held times 2^11: a value
// far below its row's largest is subnormal there, and what it lacks would be too small to hold.
template <int BF16>
constexpr float kRestUp = BF16 ? 1.0f : 0x1p11f;
template <int BF16>
__device__ __forceinline__ void split8(const float* low, float down, u32x4* high, u32x4* rest) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v0 = low[2 * e] * down, v1 = low[2 * e + 1] * down;
    const uint16_t h0 = from_f32<BF16>(v0), h1 = from_f32<BF16>(v1);
    (*high)[e] = (uint32_t)h0 | (uint32_t)h1 << 16;
    const float r0 = (v0 - to_f32<BF16>(h0)) * kRestUp<BF16>, r1 = (v1 - to_f32<BF16>(h1)) * kRestUp<BF16>;
    constexpr uint32_t kInf = BF16 ? 0x7f80 : 0x7c00;
    (*rest)[e] = ((h0 & 0x7fffu) == kInf ? 0u : (uint32_t)from_f32<BF16>(r0)) |
                 ((h1 & 0x7fffu) == kInf ? 0u : (uint32_t)from_f32<BF16>(r1)) << 16;
  }
}

// Many rows, between the products: low's two numbers of each row with an adapter, sixteen lanes a
// row, eight ranks a lane.
template <int BF16>
__global__ void __launch_bounds__(kThreads) lora_join_kernel(LoraCall c, LoraPlan p) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  const int r = (threadIdx.x & 15) * 8, rank = c.bank.rank;
  const int id = row < c.M ? c.ids[row] : -1;
  const bool used = id >= 0 && id < c.bank.adapters;
  float low[8] = {};
  if (used && r < rank) add_parts((const float*)c.ws + row * rank + r, p.slices, c.M * rank, c.bank.scale[id], low);
  float down = 1.0f;
  uint16_t* lows = (uint16_t*)((uint8_t*)c.ws + p.part_bytes);
  if constexpr (!BF16) {
    float most = largest8(low);
#pragma unroll
    for (int d = 8; d; d >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, d));
    const int e = row_exponent(most);
    down = __builtin_ldexpf(1.0f, -e);
    if (used && r == 0) ((float*)(lows + 2 * c.M * rank))[row] = __builtin_ldexpf(1.0f, e);
  }
  if (!used || r >= rank) return;
  u32x4 high, rest;
  split8<BF16>(low, down, &high, &rest);
  *(u32x4*)(lows + row * rank + r) = high;
  *(u32x4*)(lows + (c.M + row) * rank + r) = rest;
}

// out = y + B_i low.  The waves of a workgroup share low (two 16-bit numbers, in LDS) and take 64
// outputs each of a run of 256.  B_i's 64 rows are one piece of memory, y and out 128 bytes of a row for
// eight lanes: B_i and the products pass through the wave's own LDS between that order and the matrix
// operands'.
enum { kLowParts, kLowJoined, kLowHere };            // low: the slices' parts, two numbers, not yet computed
template <int BF16, int KS, int CT, int LOW>         // 32-value steps of the rank, row tiles of 16
__global__ void __launch_bounds__(kThreads, KS == 4 ? 1 : 2) lora_up_kernel(LoraCall c, LoraPlan p) {
  constexpr int kRows = 16 * CT, kPitch = KS * 4 + 1;      // 16-byte pieces of a row: no two of eight rows on a bank
  constexpr int kTilePitch = 64 + 4;                       // floats of a row of 64 outputs
  constexpr int kAux = LOW == kLowJoined ? kAuxStream : 0;            // many rows of y and out pass the caches by (61.4 -> 59.4 us)
  constexpr int kOwn = 64 * kPitch > 16 * kTilePitch / 4 ? 64 * kPitch : 16 * kTilePitch / 4;
  __shared__ __align__(16) u32x4 lows[2][kRows * kPitch];  // value, remainder
  __shared__ float scaled[kRows];                          // the power of two that a row was scaled by
  __shared__ __align__(16) u32x4 own[kWaves][kOwn];        // a wave's B rows, then its 16 x 64 products
  constexpr int kRanks = 2 * KS, kSumPitch = kRanks * 16 + 4;          // rank tiles of low computed here
  __shared__ u32x4 stage[LOW == kLowHere ? kWaves : 1][LOW == kLowHere ? kStage<kRanks, 1> : 1];
  float (*const sums)[16][kSumPitch] = (float (*)[16][kSumPitch])stage;
  static_assert(LOW != kLowHere || (CT == 1 && sizeof(float) * kWaves * 16 * kSumPitch <= sizeof(stage)), "");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4, piece = lane & 7;
  constexpr bool kFew = LOW != kLowJoined;                 // one tile of an adapter's rows, else neighbouring rows
  static_assert(!kFew || CT == 1, "");
  const int block_n = blockIdx.x % p.blocks_n, tile_id = blockIdx.x / p.blocks_n;
  const int chunk = !kFew || c.M <= kChunk ? 0 : tile_id / p.groups, nth = tile_id - chunk * p.groups;
  const int64_t row0 = kFew ? (int64_t)chunk * kChunk : (int64_t)tile_id * kRows;
  const int N = c.bank.out_features, rank = c.bank.rank, pieces = rank / 8;
  const int my_id = kFew ? -1 : lane_id(c, row0, kRows, lane);
  const int n_first = block_n * p.per_n * 256 + wave * 64;
  const int rows = c.M - row0 < (kFew ? kChunk : kRows) ? (int)(c.M - row0) : kFew ? kChunk : kRows;
  const rsrc_t y_rsrc = make_rsrc(c.y + row0 * N, (uint32_t)rows * N * 2);
  const rsrc_t out_rsrc = make_rsrc(c.out + row0 * N, (uint32_t)rows * N * 2);
  u32x4* const b_rows = own[wave];
  float* const tile = (float*)own[wave];
  // B: this lane's pieces of the 64 rows, in memory's order (past them: zeros into a row's spare piece)
  int put[KS * 4];
#pragma unroll
  for (int j = 0; j < KS * 4; ++j)
    put[j] = j < pieces ? (j * 64 + lane) / pieces * kPitch + (j * 64 + lane) % pieces : kPitch - 1;
  // y and out: a lane's rows are 16 m + 8 s + lane / 8 of the tile
  int ids[CT][2];
#pragma unroll
  for (int m = 0; m < CT; ++m)
#pragma unroll
    for (int s = 0; s < 2; ++s) ids[m][s] = kFew ? -1 : __shfl(my_id, m * 16 + s * 8 + (lane >> 3));

  [[maybe_unused]] bool first = true;
  auto adapter_rows = [&](int a, int my_row) {             // my_row (few): the row of lane & 15, -1: none
    int my_rows[CT][2];                                    // this lane's, -1: not the adapter's
#pragma unroll
    for (int m = 0; m < CT; ++m)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        my_rows[m][s] = kFew ? __shfl(my_row, s * 8 + (lane >> 3)) : ids[m][s] == a ? m * 16 + s * 8 + (lane >> 3) : -1;
    const rsrc_t b_rsrc = make_rsrc((const uint16_t*)c.bank.b + (int64_t)a * N * rank, (uint32_t)N * rank * 2);
    // past N, and in rows of other adapters: past the resource, read as 0 and not written
    u32x4 b_in[KS * 4], in[CT][2];
    uint32_t at[CT][2];
    auto load = [&](int n0) {
#pragma unroll
      for (int j = 0; j < KS * 4; ++j)
        b_in[j] = load_b128(b_rsrc, j < pieces ? (uint32_t)(j * 64 + lane) * 16 : kOob, (uint32_t)n0 * rank * 2);
#pragma unroll
      for (int m = 0; m < CT; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          at[m][s] = my_rows[m][s] >= 0 && n0 + piece * 8 < N ? (uint32_t)(my_rows[m][s] * N + n0 + piece * 8) * 2 : kOob;
          in[m][s] = __builtin_amdgcn_raw_buffer_load_b128(y_rsrc, at[m][s], 0, kAux);
        }
      __builtin_amdgcn_sched_barrier(0);
    };
    if (n_first < N) load(n_first);                    // on its way while low is added up

    if (!kFew && !first) __syncthreads();
    first = false;
    if constexpr (LOW == kLowHere) {
      // each wave its part of K
      const int K = c.bank.in_features, k0 = wave * p.slice_k, k1 = k0 + p.slice_k < K ? k0 + p.slice_k : K;
      f32x4 acc[kRanks][1];
      low_product<BF16>(make_rsrc(c.x + row0 * K, (uint32_t)rows * K * 2), row_offsets(my_row, lane, K).at, adapter_a(c, a), K, k0, k1, lane,
                        stage[wave], acc);
      __syncthreads();                                   // all waves have read their rows
#pragma unroll
      for (int r = 0; r < kRanks; ++r) *(f32x4*)&sums[wave][col][r * 16 + quad * 4] = acc[r][0];
      __syncthreads();
    }
    if constexpr (LOW == kLowJoined) {
      // rows of other adapters hold zeros
      const uint16_t* from = (const uint16_t*)((const uint8_t*)c.ws + p.part_bytes);
      for (int i = threadIdx.x; i < kRows * KS * 4; i += kThreads) {
        const int row = i / (KS * 4), r = i % (KS * 4) * 8;
        const bool mine = __shfl(my_id, row) == a && r < rank;
        const int64_t of = (row0 + row) * rank + r;
        lows[0][row * kPitch + r / 8] = mine ? *(const u32x4*)(from + of) : u32x4{0, 0, 0, 0};
        lows[1][row * kPitch + r / 8] = mine ? *(const u32x4*)(from + of + c.M * rank) : u32x4{0, 0, 0, 0};
        if (!BF16 && r == 0) scaled[row] = mine ? ((const float*)(from + 2 * c.M * rank))[row0 + row] : 1.0f;
      }
    } else {
      if (wave == 0) {
        float low[KS][8], most = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) low[k][e] = 0.0f;
          if (my_row >= 0 && k * 32 + quad * 8 < rank) {
            if constexpr (LOW == kLowHere)
              add_parts(&sums[0][col][k * 32 + quad * 8], kWaves, 16 * kSumPitch, c.bank.scale[a], low[k]);
            else
              add_parts((const float*)c.ws + (row0 + my_row) * rank + k * 32 + quad * 8, p.slices, c.M * rank,
                        c.bank.scale[a], low[k]);
          }
          most = __builtin_fmaxf(most, largest8(low[k]));
        }
        float down = 1.0f;
        if constexpr (!BF16) {
          most = __builtin_fmaxf(most, __shfl_xor(most, 16));
          most = __builtin_fmaxf(most, __shfl_xor(most, 32));
          const int e = row_exponent(most);
          down = __builtin_ldexpf(1.0f, -e);
          if (quad == 0) scaled[col] = __builtin_ldexpf(1.0f, e);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int to = col * kPitch + k * 4 + quad;
          split8<BF16>(low[k], down, &lows[0][to], &lows[1][to]);
        }
      }
    }
    __syncthreads();

    for (int i = 0; i < p.per_n && n_first + i * 256 < N; ++i) {
#pragma unroll
      for (int j = 0; j < KS * 4; ++j)
        b_rows[put[j]] = b_in[j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");       // the wave's LDS accesses stay in order
      u32x4 w[4][KS];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          w[t][k] = b_rows[(t * 16 + col) * kPitch + k * 4 + quad];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[t][k][e] = k * 4 + quad < pieces ? w[t][k][e] : 0u;
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int m = 0; m < CT; ++m) {
        f32x4 acc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int part = 1; part >= 0; --part) {            // the remainders first
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const u32x4 low = lows[part][(m * 16 + col) * kPitch + k * 4 + quad];
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = mfma16<BF16>(w[t][k], low, acc[t]);
          }
          if (!BF16 && part == 1)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] *= 1.0f / kRestUp<BF16>;
        }
        const float back = BF16 ? 1.0f : scaled[m * 16 + col];
#pragma unroll
        for (int t = 0; t < 4; ++t) *(f32x4*)(tile + col * kTilePitch + t * 16 + quad * 4) = BF16 ? acc[t] : acc[t] * back;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float* d = tile + (s * 8 + (lane >> 3)) * kTilePitch + piece * 8;
          const f32x4 d0 = *(const f32x4*)d, d1 = *(const f32x4*)(d + 4);
          u32x4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x4& v = e < 2 ? d0 : d1;
            const uint32_t y2 = in[m][s][e];
            o[e] = (uint32_t)from_f32<BF16>(to_f32<BF16>((uint16_t)y2) + v[2 * (e & 1)]) |
                   (uint32_t)from_f32<BF16>(to_f32<BF16>((uint16_t)(y2 >> 16)) + v[2 * (e & 1) + 1]) << 16;
          }
          __builtin_amdgcn_raw_buffer_store_b128(o, out_rsrc, at[m][s], 0, kAux);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      if (i + 1 < p.per_n && n_first + (i + 1) * 256 < N) load(n_first + (i + 1) * 256);
    }
  };
  if constexpr (kFew) {
    const RowGroup g = row_group(c, row0, rows, lane, nth);
    if (g.adapter >= 0) adapter_rows(g.adapter, g.row);
  } else {
    each_adapter(my_id, [&](int a) { adapter_rows(a, -1); });
  }

  // rows without an adapter, eight at a time
  if (c.out == c.y) return;
  for (int j = kFew ? nth : 0; j * 8 < rows; j += kFew ? p.groups : 1) {
    const int r = j * 8 + (lane >> 3);
    const int id = kFew ? r < rows ? c.ids[row0 + r] : -1 : __shfl(my_id, r);
    if ((id >= 0 && id < c.bank.adapters) || r >= rows) continue;
    for (int i = 0; i < p.per_n; ++i) {
      const int n = n_first + i * 256 + piece * 8;
      if (n >= N) break;
      *(u32x4*)(c.out + (row0 + r) * N + n) = *(const u32x4*)(c.y + (row0 + r) * N + n);
    }
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

LoraPlan plan_of(const gptq_lora_bank& bank, int64_t M) {
  LoraPlan p;
  // Few: every adapter of a chunk is read once for each sixteen of its rows, in whatever order they come.
  // Many: a tile goes through the adapters among its rows, good for long runs only.  Us, few / many, rank
  // 64, 4096 x 14336: 129 rows, 48 adapters 36 / 219, 6 in runs 17 / 28; 1024 rows 127 / 374, 32 / 33; 2048
  // rows 241 / 631, 66 / 49; 4001 rows 453 / 1092, 102 / 71: over 1024 rows are taken to be prompts.
  p.few = M <= 1024;
  // groups of a chunk, at most: each row may open one, and each adapter has one that is not full
  const int64_t chunk = M < kChunk ? M : kChunk, most = chunk / 16 + bank.adapters;
  p.groups = (int)(chunk < most ? chunk : most);
  const int64_t groups = div_up(M, kChunk) * p.groups;
  p.low_tiles = (int)(p.few ? groups : div_up(M, kWaves * kManyRows));
  p.up_tiles = (int)(p.few ? groups : div_up(M, bank.rank > 64 ? 32 : 64));
  // K: enough workgroups to fill the card, slices of at least 64 values a wave
  const int64_t units = p.low_tiles, step = p.few ? 64 * kWaves : 64, steps = div_up(bank.in_features, step);
  int64_t slices = div_up(256, units);
  // many: twice as many while the parts stay few (8192 rows, rank 128, K = 14336: 113 -> 91 us, 4001 rows and
  // 16 parts instead of 8: 75.4 -> 76.3)
  const int64_t more = div_up(512, units) < 8 ? div_up(512, units) : 8;
  if (!p.few && slices < more) slices = more;
  if (slices > 16) slices = 16;
  if (slices > steps) slices = steps;
  p.slice_k = (int)(div_up(steps, slices) * step);
  p.slices = (int)div_up(bank.in_features, p.slice_k);
  const int64_t blocks = div_up(bank.out_features, 256);
  // few: all workgroups on the card at once; many: about 1536 of them, 768 when only one fits a CU (rank 128,
  // us with 768 / 1536: 2048 rows of 14336 outputs 74.5 / 79.3, 4001: 125 / 124, 4001 of 4096: 53 / 63)
  const int64_t fit = bank.rank <= 32 ? 1024 : bank.rank <= 64 ? 768 : 512;
  int64_t per = p.few ? div_up(p.up_tiles * blocks, fit) : p.up_tiles * blocks / (bank.rank > 64 ? 768 : 1536);
  p.per_n = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
  p.blocks_n = (int)div_up(blocks, p.per_n);
  p.per_n = (int)div_up(blocks, p.blocks_n);         // no workgroup with a short remainder
  // One launch while its workgroups have a CU each and A_i is small, since each reads all of it.  Us on the
  // device, one launch against two, rank 8, 1 row: K = 1024 4.9 / 6.8, 4096 7.1 / 8.0, 5120 7.8 / 7.6, 6144
  // 8.6 / 7.8 (the second launch costs the host 2.7 more); K = 4096, N = 14336, 4 rows (224 workgroups)
  // 7.4 / 8.2, 8 rows (448) 11.5 / 8.6.  Eight waves that share K instead of four: 7.9 at K = 4096.
  p.here = p.few && bank.rank <= 32 && bank.in_features <= 5120 && groups * p.blocks_n <= 256;
  if (p.here) p.slice_k = (int)(div_up(div_up(bank.in_features, 64), kWaves) * 64);
  p.part_bytes = p.here ? 0 : (size_t)div_up((int64_t)p.slices * M * bank.rank * 4, 256) * 256;
  return p;
}

template <int BF16, int RT>
void launch_low(const LoraCall& c, const LoraPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.low_tiles * p.slices)), block(kThreads);
  if (p.few) lora_low_kernel<BF16, RT><<<grid, block, 0, s>>>(c, p);
  else lora_low_rows_kernel<BF16, RT><<<grid, block, 0, s>>>(c, p);
}

template <int BF16, int KS>
void launch_up(const LoraCall& c, const LoraPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.up_tiles * p.blocks_n)), block(kThreads);
  if (p.here) {
    if constexpr (KS == 1) lora_up_kernel<BF16, KS, 1, kLowHere><<<grid, block, 0, s>>>(c, p);
  } else if (p.few) {
    lora_up_kernel<BF16, KS, 1, kLowParts><<<grid, block, 0, s>>>(c, p);
  } else {
    lora_join_kernel<BF16><<<dim3((uint32_t)div_up(c.M, kThreads / 16)), block, 0, s>>>(c, p);
    lora_up_kernel<BF16, KS, KS == 4 ? 2 : 4, kLowJoined><<<grid, block, 0, s>>>(c, p);
  }
}

template <int BF16>
hipError_t launch_type(const LoraCall& c, hipStream_t s) {
  const LoraPlan p = plan_of(c.bank, c.M);
  const int rank = c.bank.rank;
  if (p.here) ;
  else if (rank <= 16) launch_low<BF16, 1>(c, p, s);
  else if (rank <= 32) launch_low<BF16, 2>(c, p, s);
  else if (rank <= 64) launch_low<BF16, 4>(c, p, s);
  else launch_low<BF16, 8>(c, p, s);
  if (rank <= 32) launch_up<BF16, 1>(c, p, s);
  else if (rank <= 64) launch_up<BF16, 2>(c, p, s);
  else launch_up<BF16, 4>(c, p, s);
  return hipGetLastError();
}

}  // namespace

bool lora_fits(const gptq_lora_bank& bank, int64_t M) {
  const LoraPlan p = plan_of(bank, M);
  return grid_fits((int64_t)p.low_tiles * p.slices, kThreads) && grid_fits((int64_t)p.up_tiles * p.blocks_n, kThreads);
}

size_t lora_ws_bytes(const gptq_lora_bank& bank, int64_t M) {
  const LoraPlan p = plan_of(bank, M);
  return p.few ? p.part_bytes : (p.part_bytes + (size_t)M * bank.rank * 4 + (size_t)M * 4 + 255) / 256 * 256;
}

hipError_t launch_lora(const LoraCall& c, hipStream_t s) {
  return c.bank.dtype == GPTQ_BF16 ? launch_type<1>(c, s) : launch_type<0>(c, s);
}

}  // namespace gq
