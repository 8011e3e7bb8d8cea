// Products with packed 4-bit weights for many rows: y = x W^T, or act(x Wg^T) * (x Wu^T).
//
// Four waves share a tile of 64 FR rows by 64 FC packed outputs (a gated pair: 32 FC outputs), each FR x FC
// products of 32 x 32, weights as the first operand.  A step takes 128 bytes of each row of x: 256 inputs in the
// format (four v_mfma_scale_f32_32x32x64_f8f6f4 for each product, both sides' scales in the instruction) or 64
// in 16 bits (four 32x32x16 products; weights become the same type in registers: exactly in bfloat16, in float16 down
// to 2^-36 of the output's largest scale, kF16Top in mx_dev.h).  Both operands come through LDS, filled by
// buffer_load ... lds under the steps before; a part of a step (a quarter) is multiplied from registers while the next
// part's operands are read.
//
// LDS: rows of x are 128 bytes, piece p (16 bytes) of row r at place p ^ (r / 2 & 7), so that sixteen rows' pieces of
// one number lie on all banks; weights keep their packed order (mx.h), in which sixteen lanes read a run of 256.
//
// What bounds the largest tiles (256 x 256, one workgroup a CU, 512 registers a lane): matrix cores are busy 55 % of
// the time at the 1.8 GHz that the card keeps under this load, waves wait 16 % of it for loads or the barrier and 34 %
// for their turn to issue, mostly behind a product (in 16 bits 58, 13 and 44; gated codes 47, 13 and 34).  4096 rows in codes,
// 8192 -> 28672: 447 us, 4.3 PFLOP/s; 2003 gated rows, 8192 -> 14336: 234 to 240 us, 4.0; 2048 in bfloat16, 4096 -> 14336: 182 to
// 186 us, 1.3 (a library product with bfloat16 weights of that shape: 173 us, of 8192 x 8192 x 8192 at most 1.62 PFLOP/s).
// Copies that left parts out, when the first took 474 us: without loads 333, without reads from LDS 433, without
// both 292; loads alone 287 of them (L2 to LDS at 14 TB/s), and 194 with all of them in L1.
// Small tiles are bound by the way of a step's operands: 0.36 us a step of 64 x 64, with two steps to a barrier (0.5 with one).
#include <type_traits>
#include <utility>

#include "mx_dev.h"
#include "serving.h"

namespace gq {
namespace {

constexpr int kWaves = 4, kTiledThreads = 64 * kWaves;
constexpr int kXRow = 128;                // bytes of a row of x in a step

template <int X, int FR, int FC>
struct Shape {
  // A workgroup alone on its CU goes through several tiles, without a pause between them.
  static constexpr bool kLong = FR * FC >= 16;
  // Small tiles are bound by the way of their operands: two steps to a buffer, a barrier every other step.
  static constexpr int kSub = FR * FC == 1 ? 2 : 1;
  static constexpr int kRows = 64 * FR, kOuts = 64 * FC, kTiles = kOuts / 16;
  static constexpr int kInputs = X == kMxCodes ? 256 : 64;              // of a step
  static constexpr int kTileStep = X == kMxCodes ? kMxTileBytes : kMxTileBytes / 4;      // bytes of a tile's codes in a step
  static constexpr int kXBytes = kRows * kXRow, kWBytes = kTiles * kTileStep < 4096 ? 4096 : kTiles * kTileStep;
  static constexpr int kWAt = kXBytes, kBytes = kWAt + kWBytes;
  // scales of four steps: of x, [step][odd blocks][row] words; of weights, [stage][tile] of four stages or one
  static constexpr int kXsBytes = X == kMxCodes ? kRows * 32 : 16, kWsStage = kTiles * 128;
  static constexpr int kWsLoads = ((X == kMxCodes ? 4 : 1) * kWsStage + 1023) / 1024;    // of 1 KB, shared by the waves
};

template <int I> using Int = std::integral_constant<int, I>;
// body(Int<0>) .. body(Int<N - 1>): matrix instructions name their scale bytes by constants.
template <int... I, typename Body>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, Body&& body) { (body(Int<I>{}), ...); }
template <int N, typename Body>
__device__ __forceinline__ void each(Body&& body) { each_of(std::make_integer_sequence<int, N>{}, body); }

// Where tile `id` of a call lies.
struct Place {
  int m0, rows;                           // first row, rows
  int tile0, tiles;                       // first packed tile, packed tiles
};

// Workgroups go round the eight XCDs: each takes one run of tiles, and a run goes down eight rows of tiles
// before the next column, so that the workgroups of one L2 share rows of x and weights.
template <typename S>
__device__ __forceinline__ Place place_of(const MxGemmCall& a, int id, int row_tiles, int col_tiles) {
  const int total = row_tiles * col_tiles, share = total >> 3, more = total & 7, xcd = id & 7;
  const int at = xcd * share + (xcd < more ? xcd : more) + (id >> 3);
  const int band = at / (8 * col_tiles), in_band = at - band * 8 * col_tiles;
  const int high = row_tiles - band * 8 < 8 ? row_tiles - band * 8 : 8;
  Place p;
  p.m0 = (band * 8 + in_band % high) * S::kRows;
  p.rows = (int)a.M - p.m0 < S::kRows ? (int)a.M - p.m0 : S::kRows;
  p.tile0 = in_band / high * S::kTiles;
  p.tiles = a.lay.tiles - p.tile0 < S::kTiles ? a.lay.tiles - p.tile0 : S::kTiles;
  return p;
}

template <int X, int FR, int FC, int SIDES>
__global__ void __launch_bounds__(kTiledThreads, 1) mx_tiled_kernel(MxGemmCall a, int row_tiles, int col_tiles) {
  using S = Shape<X, FR, FC>;
  // separate arrays: the compiler then knows that reads of one do not wait for loads into another
  __shared__ __align__(1024) uint8_t buf0[S::kSub * S::kBytes];
  __shared__ __align__(1024) uint8_t buf1[S::kSub * S::kBytes];
  __shared__ __align__(1024) uint8_t w_scales[2][S::kWsLoads * 1024];   // of four steps and the next four
  __shared__ __align__(1024) uint8_t x_scales[2][S::kXsBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  const int wave_m = wave & 1, wave_n = wave >> 1;
  const uint32_t x_bytes = (uint32_t)a.x_bytes, xs_bytes = (uint32_t)a.x_scale_stride, tile_bytes = (uint32_t)a.lay.stages * kMxTileBytes;
  const int blocks = a.K / 32, real = (a.K + S::kInputs - 1) / S::kInputs;
  // a workgroup of several tiles takes whole groups of four steps (inputs past K count as zeros)
  const int steps = S::kLong ? (real + 3) & ~3 : real;

  // ---- loads
  constexpr int kXLoads = S::kXBytes / (1024 * kWaves), kLoads = kXLoads + S::kWBytes / (1024 * kWaves);
  static_assert(kXLoads % 2 == 0, "pieces");
  typedef __attribute__((address_space(3))) void* lds_ptr;
  const uint32_t x_piece = ((lane & 7) ^ (lane >> 4)) * 16;
  const uint32_t x_at = (uint32_t)(wave * kXLoads * 8 + lane / 8) * x_bytes;
  // Loads of step `step` of a tile: resources, and lane offsets of its rows' pieces.  Only lane offsets are
  // checked against a resource's size: rows past `rows` and tiles past `tiles` lie behind it, and so do blocks past K.
  struct Source {
    const uint8_t *x, *w;
    uint32_t x_size, w_size, w_base, at[2];
    int wave;                             // as a value that no address is computed from ahead of the loop
  };
  auto source_of = [&](const Place& p, int step) {
    Source f;
    int stage = X == kMxCodes ? step : step >> 2;
    if (S::kLong && stage >= a.lay.stages) stage = a.lay.stages - 1;    // times zeros
    f.x = a.x + (uint64_t)p.m0 * x_bytes;
    f.x_size = (uint32_t)p.rows * x_bytes;
    f.w = a.packed + (size_t)p.tile0 * tile_bytes;
    f.w_size = (uint32_t)p.tiles * tile_bytes;
    f.w_base = (uint32_t)stage * kMxTileBytes + (X == kMxCodes ? 0 : (step & 3) * S::kTileStep);
    f.wave = wave;
    asm("" : "+s"(f.wave));
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const uint32_t piece = x_piece ^ odd * 64;
      const int block = X == kMxCodes ? step * 8 + (int)(piece >> 4) : step * 2 + (int)(piece >> 6);
      f.at[odd] = block < blocks ? x_at + piece : kOob;
    }
    return f;
  };
  auto issue = [&](auto I, const Source& f, int step, uint8_t* buf) {
    constexpr int i = decltype(I)::value;
    if constexpr (i < kXLoads) {
      // eight rows, 16 bytes a lane; the places of odd loads' pieces lie xor 4
      const uint32_t at = f.at[i & 1] + i * 8 * x_bytes, base = (uint32_t)step * kXRow;
      const rsrc_t rsrc = make_rsrc(f.x, f.x_size);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(buf + (f.wave * kXLoads + i) * 1024), 16, at, base, 0, 0);
    } else {
      const int first = ((i - kXLoads) * kWaves + f.wave) * 1024;       // byte of the step's weights
      // 16-bit x: a quarter of each tile, two tiles a load
      const uint32_t at = (X == kMxCodes ? lane * 16 : half * tile_bytes + l32 * 16) +
                          (uint32_t)(first / S::kTileStep) * tile_bytes + first % S::kTileStep;
      const uint32_t base = f.w_base;
      const rsrc_t rsrc = make_rsrc(f.w, f.w_size);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(buf + S::kWAt + first), 16, at, base, 0, 0);
    }
  };
  // Scales of four steps.  Weights: load n, of all waves, fills bytes 1024 n .. of them.
  auto issue_ws = [&](int n, const Place& p, int group, uint8_t* to) {
    n %= S::kWsLoads;                     // small tiles: some load the same bytes
    const int byte = n * 1024 + lane * 16, rest = byte % S::kWsStage;
    // stages past the last repeat it (times zeros), tiles past the last too (not stored)
    const int first = X == kMxCodes ? group * 4 : group, last = a.lay.stages - 1 - first;
    int stage = X == kMxCodes ? byte / S::kWsStage : 0;
    stage = stage < last ? stage : last;
    const int tile = rest / 128 < p.tiles ? rest / 128 : p.tiles - 1;
    const rsrc_t rsrc = make_rsrc(a.packed + a.lay.scales_at + ((size_t)p.tile0 * a.lay.stages + first) * 128, 0x7fffffffu);
    const uint32_t at = (uint32_t)(tile * a.lay.stages + stage) * 128 + rest % 128;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(to + n * 1024), 16, at, 0, 0, 0);
  };
  // Rows of x: through registers, since a lane's products take every other byte.  Sixteen bytes (two steps) of a row a
  // lane, half of the tile's at a time; a byte past the row's blocks may be anything and becomes 0.
  u32x4 xs_in;
  auto load_xs = [&](int part, const Place& p, int group) {
    const int unit = (part * kTiledThreads + tid) % (S::kRows * 2), row = unit >> 1 < p.rows ? unit >> 1 : p.rows - 1;
    const rsrc_t rsrc = make_rsrc(a.x_scales + (uint64_t)p.m0 * xs_bytes, (uint32_t)p.rows * xs_bytes);
    xs_in = load_b128(rsrc, (uint32_t)row * xs_bytes + (uint32_t)group * 32 + (unit & 1) * 16, 0);
  };
  uint32_t xs_keep[4];
  auto keep_xs = [&](auto K, int part, int group) {      // mask of word K of the lane's four
    constexpr int k = decltype(K)::value;
    const int unit = (part * kTiledThreads + tid) % (S::kRows * 2), left = blocks - group * 32 - (unit & 1) * 16 - 4 * k;
    const int keep = left < 0 ? 0 : left > 4 ? 4 : left;
    xs_keep[k] = (uint32_t)((1ull << (8 * keep)) - 1);
  };
  auto store_xs = [&](int part, uint8_t* to) {
    const int unit = (part * kTiledThreads + tid) % (S::kRows * 2);
    uint32_t* at = (uint32_t*)to + (unit & 1) * 4 * S::kRows + (unit >> 1);
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const uint32_t lo = xs_in[k] & xs_keep[k], hi = xs_in[k + 1] & xs_keep[k + 1];
      at[k * S::kRows] = __builtin_amdgcn_perm(hi, lo, 0x06040200);
      at[(k + 1) * S::kRows] = __builtin_amdgcn_perm(hi, lo, 0x07050301);
    }
  };

  // ---- products
  f32x16 acc[FC][FR];
  const int x_row = wave_m * FR * 32 + l32;
  uint32_t x_read[4];                     // this lane's piece in part j of a step: 2 j + half, or 4 half + j
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int piece = X == kMxCodes ? 2 * j + half : 4 * half + j;
    x_read[j] = x_row * kXRow + ((piece ^ (x_row >> 1 & 7)) * 16);
  }
  const uint32_t w_read = S::kWAt + (wave_n * FC * 2 + (l32 >> 4)) * S::kTileStep + half * 256 + (lane & 15) * 16;
  const uint32_t ws_read = (wave_n * FC * 2 + (l32 >> 4)) * 128 + half * 64 + (lane & 15) * 4;
  const uint32_t xs_read = half * 4 * S::kRows + x_row * 4;

  // Operands of part j lie in x[j & 1], and in w[j & 1] (codes) or, for all four parts of step t, in w[t & 1].
  u32x4 x[2][FR], w[2][FC];
  uint32_t ws[2][FC], xs[2][FR];          // by step & 1
  float w_scale[FC];
  int lift[FC] = {};                      // added to a scale byte (float16 activations)

  // Read I for part J: of the same step from `buf`, or, before a step's first part, of step parity T.
  constexpr int kReads = FR + (X == kMxCodes ? FC : 0), kFirstReads = FR + FC;
  auto read = [&](auto I, auto J, auto T, const uint8_t* buf) {
    constexpr int i = decltype(I)::value, j = decltype(J)::value, t = decltype(T)::value;
    if constexpr (i < FR) x[j & 1][i] = *(const u32x4*)(buf + x_read[j] + i * 32 * kXRow);
    else if constexpr (X == kMxCodes) w[j & 1][i - FR] = *(const u32x4*)(buf + w_read + (i - FR) * 4096 + j * 512);
    else w[t][i - FR] = *(const u32x4*)(buf + w_read + (i - FR) * 2 * S::kTileStep);
  };
  auto read_scales = [&](auto T, int step, int side) {
    constexpr int t = decltype(T)::value;
#pragma unroll
    for (int c = 0; c < FC; ++c)
      ws[t][c] = *(const uint32_t*)(w_scales[side] + (X == kMxCodes ? (step & 3) * S::kWsStage : 0) + ws_read + c * 256);
    if constexpr (X == kMxCodes) {
#pragma unroll
      for (int r = 0; r < FR; ++r) xs[t][r] = *(const uint32_t*)(x_scales[side] + (step & 3) * 8 * S::kRows + xs_read + r * 128);
    }
  };
  // Scales of a step as its conversions take them.
  auto settle = [&](auto T, int step) {
    constexpr int t = decltype(T)::value;
    if constexpr (X != kMxCodes) {
#pragma unroll
      for (int c = 0; c < FC; ++c) {
        int v = (int)(ws[t][c] >> (8 * (step & 3)) & 255);
        if constexpr (X == kMxF16) v = v + lift[c] > 0 ? v + lift[c] : 0;
        w_scale[c] = scale_of(v);
      }
    }
  };

  // A turn multiplies step `step` (in buffer `here`, parity T) and prepares what follows it:
  enum { kLoad, kNoLoad, kInside };
  struct Next {
    Place two, group;                     // tiles of the steps that follow the other buffer's, and of the next four steps' scales
    int two_step[S::kSub], group_at;      // their places in them
    int one_side, group_side;             // where the next step's scales lie, and the next four steps' go
  };
  // Part J: FC x FR products, and the reads for the next part (after part 3: for the next step, from `from`) and the
  // loads beside them.  Where a wave is alone on its SIMD each product is followed by its share, in this
  // order, reads early, so that they are back by the next part (4096 rows in codes, 8192 -> 28672: 605 us in the compiler's
  // order, 474 so).  Else other waves cover for it, and all reads and loads go first (tiles of 128, the same call:
  // 622 us spread, 587 so).
  auto part = [&](auto J, auto T, auto L, const uint8_t* from, uint8_t* fill, int step, const Next& n) {
    constexpr int j = decltype(J)::value, t = decltype(T)::value;
    constexpr int products = FC * FR, reads = j == 3 ? kFirstReads : kReads, loads = j == 3 && decltype(L)::value == kLoad ? S::kSub * kLoads : 0;
    Source from_memory[S::kSub];
    if constexpr (loads > 0) {
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) from_memory[i] = source_of(n.two, n.two_step[i]);
    }
    u32x4 v;
    auto product = [&](auto P) {
      constexpr int p = decltype(P)::value, c = p / FR, r = p % FR;
      if constexpr (X == kMxCodes) {
        const u32x4 a4 = w[j & 1][c], b4 = x[j & 1][r];
        const i32x8 wa = {(int)a4[0], (int)a4[1], (int)a4[2], (int)a4[3], 0, 0, 0, 0};
        const i32x8 xb = {(int)b4[0], (int)b4[1], (int)b4[2], (int)b4[3], 0, 0, 0, 0};
        acc[c][r] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wa, xb, acc[c][r], kFp4, kFp4, j, (int)ws[t][c], j,
                                                                    (int)xs[t][r]);
      } else {
        if constexpr (r == 0) v = mx_values<X == kMxBf16>(w[t][c][j], w_scale[c]);
        if constexpr (X == kMxBf16)
          acc[c][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, x[j & 1][r]),
                                                              acc[c][r], 0, 0, 0);
        else
          acc[c][r] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, v), __builtin_bit_cast(f16x8, x[j & 1][r]),
                                                             acc[c][r], 0, 0, 0);
      }
    };
    // What goes beside product P of `places`.  Scales: of the next step before any load is under way (the compiler has LDS
    // writes, and some reads, wait for those); of the next four steps over these, without a branch (the compiler
    // moves products past one).
    auto beside = [&](auto P, auto Places) {
      constexpr int p = decltype(P)::value, places = decltype(Places)::value;
      if constexpr (j == 3 && p == 0) {
        read_scales(Int<t ^ 1>{}, step + 1, n.one_side);
        if constexpr (X == kMxCodes && S::kSub == 1 && t == 0) store_xs(step >> 1 & 1, x_scales[n.group_side]);
        if constexpr (X == kMxCodes && S::kSub == 2 && t == 1)
          if (!(step & 2)) store_xs(0, x_scales[n.group_side]);
      }
      if constexpr (j == 0 && p == places - 1) {
        if constexpr (X == kMxCodes && S::kSub == 1 && t == 0) load_xs(step >> 1 & 1, n.group, n.group_at);
        if constexpr (X == kMxCodes && S::kSub == 2 && t == 0)
          if (!(step & 2)) load_xs(0, n.group, n.group_at);
        issue_ws(t * kWaves + wave, n.group, n.group_at, w_scales[n.group_side]);
      }
      if constexpr (X == kMxCodes && j == 1 && t == 0) {
        constexpr int k0 = 4 * p / places, k1 = 4 * (p + 1) / places;
        each<k1 - k0>([&](auto K) { keep_xs(Int<k0 + decltype(K)::value>{}, S::kSub == 1 ? step >> 1 & 1 : 0, n.group_at); });
      }
      constexpr int soon = places > 8 ? places * 5 / 8 : places;
      constexpr int read0 = p < soon ? reads * p / soon : reads, read1 = p < soon ? reads * (p + 1) / soon : reads;
      each<read1 - read0>([&](auto K) {
        read(Int<read0 + decltype(K)::value>{}, Int<(j + 1) & 3>{}, Int<j == 3 ? t ^ 1 : t>{}, from);
      });
      constexpr int issue0 = loads * p / places, issue1 = loads * (p + 1) / places;
      each<issue1 - issue0>([&](auto K) {
        constexpr int i = issue0 + decltype(K)::value, sub = i / kLoads;
        issue(Int<i % kLoads>{}, from_memory[sub], n.two_step[sub], fill + sub * S::kBytes);
      });
    };
    if constexpr (S::kLong) {
      each<products>([&](auto P) {
        product(P);
        beside(P, Int<products>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      beside(Int<0>{}, Int<1>{});
      __builtin_amdgcn_sched_barrier(0);
      each<products>([&](auto P) { product(P); });
    }
  };
  // The last part of a buffer's last step runs behind the barrier, from registers: there every wave has read the rest of
  // the buffer and has its own loads of the other one in LDS (a full wait: a count of loads into LDS that may stay
  // in flight is not a sound wait on this card).  So the next step's operands arrive under part 3, and this buffer
  // (`fill`) takes the steps after the other one's.  L: kLoad; kNoLoad: the results go through the buffer first;
  // kInside: not a buffer's last step.
  auto turn = [&](auto T, auto L, int step, const uint8_t* here, const uint8_t* next, uint8_t* fill, const Next& n) {
    settle(T, step);
    part(Int<0>{}, T, L, here, nullptr, step, n);
    part(Int<1>{}, T, L, here, nullptr, step, n);
    part(Int<2>{}, T, L, here, nullptr, step, n);
    if constexpr (decltype(L)::value != kInside) {
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
    part(Int<3>{}, T, L, next, fill, step, n);
  };

  const int total = row_tiles * col_tiles;
  Place here = place_of<S>(a, blockIdx.x, row_tiles, col_tiles);
  auto fill_buffer = [&](const Place& p, int step, uint8_t* buf) {
    each<S::kSub>([&](auto I) {
      constexpr int sub = decltype(I)::value;
      const int at = step + sub < steps ? step + sub : steps - 1;
      const Source f = source_of(p, at);
      each<kLoads>([&](auto K) { issue(K, f, at, buf + sub * S::kBytes); });
    });
  };
  fill_buffer(here, 0, buf0);
  for (int n = wave; n < S::kWsLoads; n += kWaves) issue_ws(n, here, 0, w_scales[0]);
  if constexpr (X == kMxCodes) {
    for (int part = 0; part < 2; ++part) {
      load_xs(part, here, 0);
      each<4>([&](auto K) { keep_xs(K, part, 0); });
      store_xs(part, x_scales[0]);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  read_scales(Int<0>{}, 0, 0);
  each<kFirstReads>([&](auto I) { read(I, Int<0>{}, Int<0>{}, buf0); });
  fill_buffer(here, S::kSub, buf1);

  int round = 0;                          // groups of four steps so far: the parity of their scales
  for (int id = blockIdx.x;;) {
    // (Past the last step, and after the last tile, loads repeat some: nothing reads them.)
    const int next_id = id + gridDim.x;
    const Place after = next_id < total ? place_of<S>(a, next_id, row_tiles, col_tiles) : here;
    if constexpr (X == kMxF16) {
#pragma unroll
      for (int c = 0; c < FC; ++c) {
        const int tile = (wave_n * FC + c) * 2 + (l32 >> 4);
        lift[c] = 127 + kF16Top - a.packed[a.lay.tops_at + (size_t)(here.tile0 + (tile < here.tiles ? tile : 0)) * 16 + (lane & 15)];
      }
    }
#pragma unroll
    for (int c = 0; c < FC; ++c)
#pragma unroll
      for (int r = 0; r < FR; ++r) {
        acc[c][r] = f32x16{};
        if constexpr (S::kLong) asm("" : "+a"(acc[c][r]));
      }
    auto next_of = [&](int step) {
      Next n;
      const bool last_two = step + 2 >= steps, last_four = (step | 3) + 1 >= steps;
      n.two = S::kLong && last_two ? after : here;
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) {
        const int at = step + 1 + S::kSub + i;
        n.two_step[i] = at < steps ? at : S::kLong ? at - steps : steps - 1;
      }
      n.group = S::kLong && last_four ? after : here;
      n.group_at = last_four && S::kLong ? 0 : (step >> 2) + 1;
      n.group_side = (round + (step >> 2) + 1) & 1;
      n.one_side = (round + ((step + 1) >> 2)) & 1;
      return n;
    };
    int step = 0;
    auto pair = [&](auto L) {
      turn(Int<0>{}, Int<kLoad>{}, step, buf0, buf1, buf0, next_of(step));
      turn(Int<1>{}, L, step + 1, buf1, buf0, buf1, next_of(step + 1));
      step += 2;
    };
    if constexpr (S::kLong) {
      do pair(Int<kLoad>{});
      while (step + 2 < steps);
      pair(Int<kNoLoad>{});
#pragma unroll
      for (int c = 0; c < FC; ++c)
#pragma unroll
        for (int r = 0; r < FR; ++r) asm("" : "+a"(acc[c][r]));
    } else if constexpr (S::kSub == 2) {
      auto first = [&](const uint8_t* buf) {
        turn(Int<0>{}, Int<kInside>{}, step, buf, buf + S::kBytes, nullptr, next_of(step));
        ++step;
      };
      auto second = [&](uint8_t* buf, const uint8_t* other) {
        turn(Int<1>{}, Int<kLoad>{}, step, buf + S::kBytes, other, buf, next_of(step));
        ++step;
      };
      while (step + 3 < steps) {
        first(buf0);
        second(buf0, buf1);
        first(buf1);
        second(buf1, buf0);
      }
      if (step < steps) first(buf0);
      if (step < steps) second(buf0, buf1);
      if (step < steps) first(buf1);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    } else {
      while (step + 1 < steps) pair(Int<kLoad>{});
      if (step < steps) turn(Int<0>{}, Int<kLoad>{}, step, buf0, buf1, buf0, next_of(step));
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
    round += steps >> 2;

    // ---- results: register q of a product is output 8 (q / 4) + 4 half + q % 4 of row l32.
    // Four outputs of product (c, r), from register 4 Q on (of a pair: with the up side's, eight registers on).
    auto four = [&](int c, int r, int q, const float (&factor)[SIDES][4]) {
      uint16_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float g = acc[c][r][q + e] * factor[0][e];
        if constexpr (SIDES == 2) g = mx_gate(g, acc[c][r][(q + e + 8) & 15] * factor[SIDES - 1][e], a.act);
        v[e] = mx_round(g, a.y_bf16);
      }
      return u32x2{(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16};
    };
    auto factors = [&](int c, int q, float (&factor)[SIDES][4]) {
#pragma unroll
      for (int i = 0; i < SIDES; ++i) {
        uint32_t tops = 0;
        if constexpr (X == kMxF16) {
          const int t = (wave_n * FC + c) * 2 + (SIDES == 2 ? i : q >> 3);
          tops = *(const uint32_t*)(a.packed + a.lay.tops_at + (size_t)(here.tile0 + (t < here.tiles ? t : 0)) * 16 + (2 * q & 15) + 4 * half);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) factor[i][e] = X == kMxF16 ? mx_row_factor(tops >> (8 * e) & 255) : 1.0f;
      }
    };
    // A wave turns its own part in LDS (buf1, which nobody reads now), so that rows go out in runs of up to 128 bytes,
    // past the caches: with runs of 32 bytes, straight from registers, 4096 x 28672 results took 100 us of 490, so 40.
    constexpr int kGroup = FC < 2 * SIDES ? FC : 2 * SIDES;             // products side by side in a pass
    constexpr int kWide = 32 * kGroup / SIDES, kPitch = kWide * 2 + 16; // outputs of a pass, bytes of its rows
    constexpr int kHigh = FR >= 2 && 4 * 64 * kPitch <= S::kSub * S::kBytes ? 2 : 1;     // products one below the other
    static_assert(4 * kHigh * 32 * kPitch <= S::kSub * S::kBytes && FC % kGroup == 0 && FR % kHigh == 0, "four waves share a buffer");
    uint8_t* mine = buf1 + wave * (kHigh * 32 * kPitch);
#pragma unroll
    for (int c0 = 0; c0 < FC; c0 += kGroup)
#pragma unroll
      for (int r0 = 0; r0 < FR; r0 += kHigh) {
#pragma unroll
        for (int c = 0; c < kGroup; ++c)
#pragma unroll
          for (int q = 0; q < 16 / SIDES; q += 4) {
            float factor[SIDES][4];
            factors(c0 + c, q, factor);
#pragma unroll
            for (int r = 0; r < kHigh; ++r)
              *(u32x2*)(mine + (r * 32 + l32) * kPitch + (c * 32 / SIDES + 2 * q + 4 * half) * 2) = four(c0 + c, r0 + r, q, factor);
          }
        __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0): the wave's own writes
        __builtin_amdgcn_wave_barrier();
        const int n0 = (here.tile0 + (wave_n * FC + c0) * 2) / SIDES * 16, row0 = wave_m * FR * 32 + r0 * 32;
        constexpr int kLanes = kWide / 8;                // of a row, 16 bytes each
        if (a.N % 8 == 0) {
#pragma unroll 4
          for (int i = 0; i < kHigh * 32; i += 64 / kLanes) {
            const int row = i + lane / kLanes, n = n0 + lane % kLanes * 8;
            const u32x4 v = *(const u32x4*)(mine + row * kPitch + lane % kLanes * 16);
            if (row0 + row < here.rows && n < a.N)
              __builtin_nontemporal_store(v, (u32x4*)(a.y + (int64_t)(here.m0 + row0 + row) * a.N + n));
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kHigh * 32; i += 64 / kLanes) {
            const int row = i + lane / kLanes, n = n0 + lane % kLanes * 8;
            const uint16_t* v = (const uint16_t*)(mine + row * kPitch + lane % kLanes * 16);
            uint16_t* y = a.y + (int64_t)(here.m0 + row0 + row) * a.N + n;
            const int left = row0 + row < here.rows ? a.N - n : 0;
            if (left >= 8) *(u32x4_at2*)y = *(const u32x4*)v;
#pragma unroll
            for (int e = 0; e < 7; ++e)
              if (left < 8 && e < left) y[e] = v[e];
          }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        __builtin_amdgcn_wave_barrier();
      }
    if (!S::kLong || next_id >= total) break;
    id = next_id;
    here = after;
    __syncthreads();
    fill_buffer(here, 1, buf1);
  }
  __builtin_amdgcn_s_waitcnt(0);          // no load into LDS outlives the workgroup
}

template <int X, int FR, int FC, int SIDES>
hipError_t run(const MxGemmCall& c, hipStream_t s) {
  using S = Shape<X, FR, FC>;
  const int64_t row_tiles = (c.M + S::kRows - 1) / S::kRows;
  const int col_tiles = (c.lay.tiles + S::kTiles - 1) / S::kTiles;
  int64_t groups = row_tiles * col_tiles;
  if (S::kLong && groups > kMxCus) groups = kMxCus;
  mx_tiled_kernel<X, FR, FC, SIDES><<<(unsigned)groups, kTiledThreads, 0, s>>>(c, (int)row_tiles, col_tiles);
  return hipGetLastError();
}

// Microseconds of a step of a tile when the card is full (`full`, for each tile of a CU), and at least (`least`: a step's
// loads and its barrier), measured: tiles of 256, 128 and 64 rows and outputs.
struct Cost { double full, least; };
constexpr Cost kCodesCost[3] = {{1.95, 1.8}, {0.65, 0.8}, {0.27, 0.36}}, k16Cost[3] = {{1.46, 1.4}, {0.43, 0.5}, {0.165, 0.33}};

// Large tiles load each operand least often, small ones fill the card and its last round.  The estimate for each
// size ranks as measured, us for 256 / 128 / 64: 4096 rows in codes, 8192 -> 28672: 439 / 587 / 979; 1301 rows, 4160 -> 4001: 48 /
// 28 / 34; 257 rows, 4096 -> 4096: 29 / 14 / 11; 512 rows, 8192 -> 8192: 56 / 28 / 38, in 16 bits - / 72 / 89.
int size_of(const MxGemmCall& c, double* us) {
  const bool codes = c.x_kind == kMxCodes;
  const int64_t steps = (c.K + (codes ? 255 : 63)) / (codes ? 256 : 64);
  int best = 0;
  for (int i = 0; i < 3; ++i) {
    const int64_t side = 256 >> i, tiles = (c.M + side - 1) / side * ((c.lay.tiles + side / 16 - 1) / (side / 16));
    const Cost& cost = (codes ? kCodesCost : k16Cost)[i];
    const double full = (double)((tiles + kMxCus - 1) / kMxCus) * cost.full;
    const double t = 3.0 + (double)steps * (full > cost.least ? full : cost.least);
    if (i == 0 || t < *us) best = i, *us = t;
  }
  return best;
}

template <int X, int SIDES>
hipError_t run_size(const MxGemmCall& c, hipStream_t s) {
  double us;
  switch (size_of(c, &us)) {
    case 0: return run<X, 4, 4, SIDES>(c, s);
    case 1: return run<X, 2, 2, SIDES>(c, s);
    default: return run<X, 1, 1, SIDES>(c, s);
  }
}

template <int X>
hipError_t run_sides(const MxGemmCall& c, hipStream_t s) {
  return c.lay.sides == 2 ? run_size<X, 2>(c, s) : run_size<X, 1>(c, s);
}

}  // namespace

double mx_tiled_us(const MxGemmCall& c) {
  double us;
  size_of(c, &us);
  return us;
}

bool mx_tiled_fits(const MxGemmCall& c) { return grid_fits((c.M + 63) / 64 * ((c.lay.tiles + 3) / 4), kTiledThreads); }

hipError_t launch_mx_tiled(const MxGemmCall& c, hipStream_t s) {
  if (c.x_kind == kMxCodes) return run_sides<kMxCodes>(c, s);
  return c.x_kind == kMxF16 ? run_sides<kMxF16>(c, s) : run_sides<kMxBf16>(c, s);
}

}  // namespace gq
