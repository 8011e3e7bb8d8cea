// Products with packed 4-bit weights for few rows: y = x W^T, or act(x Wg^T) * (x Wu^T).
//
// Bound by the weights' bytes, and beyond a few rows by the reads of x, which every workgroup makes for
// itself.  A wave multiplies CT tiles of 16 packed outputs with up to 64 rows: weights go from memory to
// registers once, in 1 KB runs, as the first operand of a 16 x 16 matrix instruction, rows of x are
// the second.  The waves of a workgroup share the inputs, in chunks of 128, and their sums are
// added in LDS in a fixed order, so a call's bits do not depend on timing.  Activations in the format go to
// v_mfma_scale_f32_16x16x128_f8f6f4 with both sides' scales; 16-bit ones to 16x16x32 products with the
// weights turned into the same type in registers: exact in bfloat16, in float16 down to 2^-36 of the output's largest
// scale (kF16Top, mx_dev.h).
//
// Measured, calls among others from Python: one row, 4096 -> 14336: 7.5 us, 4.2 TB/s (6.8 in codes), the pair of a gated block
// 11.9, 5.2 TB/s (10.9 in codes); 16 rows in 16 bits, 8192 -> 28672: 29.7 us, 4.2 TB/s; 61 in codes, 8192 -> 8192: 11.2.  In the
// comments below both sides of a choice are of one run, made when it was taken.
#include "mx_dev.h"
#include "serving.h"

namespace gq {
namespace {

constexpr int kSkinnyWaves = 8;

// Four registers of lane group g (16 lanes) hold words 0..3 of block g; after it register p holds word g of block p.
__device__ __forceinline__ u32x4 turned(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// MT tiles of 16 rows by CT tiles of 16 packed outputs (a gated pair: two) a wave, DEPTH chunks of it in flight.
template <int X, int MT, int CT, int SIDES, int DEPTH, int BOUND, bool STAGE>
__global__ void __launch_bounds__(BOUND) mx_skinny_kernel(MxGemmCall a, int groups) {
  constexpr int waves = kSkinnyWaves;
  constexpr int kFit = 64 / (waves * SIDES * MT), kOutTiles = CT / SIDES;        // output tiles joined at once, in 64 KB
  constexpr int kBatch = kFit < 1 ? 1 : kFit < kOutTiles ? kFit : kOutTiles, kBatchTiles = kBatch * SIDES;
  constexpr int kSums = waves * kBatchTiles * MT * 64, XL = X == kMxCodes ? 1 : 4, kStaged = STAGE ? waves * XL * 64 : 0;
  __shared__ f32x4 sums[kSums > kStaged ? kSums : kStaged];                      // [wave][output tile][row tile][lane]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int tile0 = blockIdx.x % groups * CT, last = a.lay.tiles - 1 - tile0;
  const int64_t m0 = (int64_t)(blockIdx.x / groups) * (MT * 16);
  const int rows = a.M - m0 < MT * 16 ? (int)(a.M - m0) : MT * 16, blocks = a.K / 32;
  const int chunks = (blocks + 3) / 4;

  // Up to four tiles a base each (one gated row, 4096 -> 14336: 12.4 us, from one base 13.6); more would not fit the scalar registers,
  // and a tile's place goes into the offset.
  constexpr bool kOneBase = CT > 4;
  constexpr int kBases = kOneBase ? 1 : CT;
  const uint32_t w_size = (uint32_t)a.lay.stages * kMxTileBytes, s_size = (uint32_t)a.lay.stages * 128;
  const uint32_t held = !kOneBase ? 1 : last + 1 < CT ? last + 1 : CT;           // tiles of a base
  rsrc_t w_rsrc[kBases], s_rsrc[kBases];
#pragma unroll
  for (int i = 0; i < kBases; ++i) {
    const size_t tile = tile0 + (i < last ? i : last);   // past the last: not stored
    w_rsrc[i] = make_rsrc(a.packed + tile * w_size, held * w_size);
    s_rsrc[i] = make_rsrc(a.packed + a.lay.scales_at + tile * s_size, held * s_size);
  }
  // Added to a scale byte (float16 activations): kLift less its row's largest; of more than four tiles those share registers.
  constexpr int kLift = 127 + kF16Top;
  int lift[kOneBase ? 1 : CT] = {};
  uint32_t tops[kOneBase ? (CT + 3) / 4 : 1] = {};
  if constexpr (X == kMxF16) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int top = a.packed[a.lay.tops_at + (size_t)(tile0 + (i < last ? i : last)) * 16 + r];
      if constexpr (kOneBase) tops[i / 4] |= (uint32_t)top << (8 * (i % 4));
      else lift[i] = kLift - top;
    }
  }
  const rsrc_t x_rsrc = make_rsrc(a.x + m0 * a.x_bytes, (uint32_t)(rows * a.x_bytes));
  const rsrc_t xs_rsrc = X == kMxCodes ? make_rsrc(a.x_scales + m0 * a.x_scale_stride, (uint32_t)(rows * a.x_scale_stride))
                                       : x_rsrc;
  constexpr int WS = X == kMxCodes ? 1 : 2;

  // Chunk q is blocks 4 q .. 4 q + 3.  Codes: lane group g multiplies block g of it, whole.  16 bits: product p takes block
  // p, a quarter of it each group, so that a load of x reads runs of 64 bytes.  A wave takes DEPTH chunks
  // at once: of many rows neighbouring ones, whose scales it reads together (61 rows in codes, 8192 -> 8192: 17.9 -> 13.0 us),
  // of up to 16 rows every eighth, so that the waves read side by side (one row, 4096 -> 14336: 8.2 us against 9.6).
  constexpr bool kNear = MT > 1;
  constexpr int kStep = kNear ? 1 : waves, kStages = kNear ? (DEPTH + 1) / 2 : DEPTH;
  // STAGE: neighbouring lanes read neighbouring pieces of a row, and a wave turns them in LDS (piece j of row r at a place
  // such that sixteen rows' pieces of one number lie on all banks).  Straight from memory a load takes 16 bytes of each of
  // sixteen rows, a cache access for every lane: 48 gated rows in 16 bits, 4096 -> 14336: 30.4 us against 24.5; 32 rows, 4096 -> 4096:
  // 10.4 against 7.5; of up to 8 rows, or 16 in codes, there is little to gain (16 in codes, 4096 -> 14336: 7.5 against 7.8).
  u32x4* staged = (u32x4*)sums + wave * XL * 64;
  const auto place = [](int row, int piece) {
    return X == kMxCodes ? row * 4 + (piece ^ (row >> 2 & 3)) : row * 16 + (piece ^ row);
  };
  f32x4 acc[CT][MT] = {};
  u32x4 w[DEPTH][CT], x[DEPTH][MT][XL];
  uint32_t ws[kStages][CT][WS], xs[MT][DEPTH];
  // (Loads of the next chunks under the products of these take registers that resident waves use better: one row, 4096 ->
  // 14336, 11.9 us against 8.1.)
  for (int q0 = kNear ? wave * DEPTH : wave; q0 < chunks; q0 += waves * DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int q = q0 + d * kStep, c = q & 1, stage = kNear ? d / 2 : d;
      const bool in = q < chunks;         // past the last all reads as zeros
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        const int base = kOneBase ? 0 : i;
        const uint32_t tile = !kOneBase ? 0 : i < last ? i : last;
        w[d][i] = load_b128(w_rsrc[base], in ? (uint32_t)(c * 1024 + lane * 16) : kOob, tile * w_size + (uint32_t)(q >> 1) * kMxTileBytes);
        if (!kNear || d % 2 == 0) {
#pragma unroll
          for (int h = 0; h < WS; ++h)
            ws[stage][i][h] = load_b32(s_rsrc[base], in ? (uint32_t)((WS == 1 ? g & 1 : h) * 64 + r * 4) : kOob,
                                       tile * s_size + (uint32_t)(q >> 1) * 128);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int p = 0; p < XL; ++p) {
          const int row = m * 16 + (!STAGE ? r : X == kMxCodes ? lane >> 2 : 4 * p + g);
          const int piece = X == kMxCodes ? (STAGE ? lane & 3 : g) : STAGE ? r : 4 * p + g;
          const bool there = 4 * q + (X == kMxCodes ? piece : piece >> 2) < blocks && row < rows;
          x[d][m][p] = load_b128(x_rsrc, there ? (uint32_t)(row * a.x_bytes) + (uint32_t)(q * XL * 64 + piece * 16) : kOob, 0);
        }
      }
    }
    if constexpr (X == kMxCodes) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + r;
        const uint32_t at = row < rows ? (uint32_t)(row * a.x_scale_stride) + (uint32_t)q0 * 4 : kOob;
        if constexpr (kNear) {
          load_words<DEPTH, 0>(xs_rsrc, at, 0, xs[m]);
        } else {
#pragma unroll
          for (int d = 0; d < DEPTH; ++d) xs[m][d] = load_b32(xs_rsrc, at + d * waves * 4, 0);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int q = q0 + d * kStep, c = q & 1, stage = kNear ? d / 2 : d;
      if constexpr (STAGE) {
        // rows' pieces as they were loaded, to where their products take them; a wave's LDS accesses stay in order
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int p = 0; p < XL; ++p) {
            const int row = X == kMxCodes ? lane >> 2 : 4 * p + g, piece = X == kMxCodes ? lane & 3 : r;
            staged[place(row, piece)] = x[d][m][p];
          }
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int p = 0; p < XL; ++p) x[d][m][p] = staged[place(r, X == kMxCodes ? g : 4 * p + g)];
          __builtin_amdgcn_wave_barrier();
        }
      }
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        // byte j of word h is the scale of the stage's block 2 j + h
        if constexpr (X == kMxCodes) {
          const uint32_t byte = ws[stage][i][0] >> (16 * c + 8 * (g >> 1)) & 255;
          const u32x4 u = w[d][i];
          const i32x8 wa = {(int)u[0], (int)u[1], (int)u[2], (int)u[3], 0, 0, 0, 0};
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const u32x4 v = x[d][m][0];
            const i32x8 xb = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
            // a byte past the row's blocks may be anything
            const uint32_t x_byte = 4 * q + g < blocks ? xs[m][d] >> (8 * g) & 255 : 0;
            acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, acc[i][m], kFp4, kFp4, 0, (int)byte, 0,
                                                                         (int)x_byte);
          }
        } else {
          const u32x4 u = turned(w[d][i]);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            int s = (int)(ws[stage][i][p & 1] >> (16 * c + 8 * (p >> 1)) & 255);
            if constexpr (X == kMxF16) {
              if constexpr (kOneBase) s += kLift - (int)(tops[i / 4] >> (8 * (i % 4)) & 255);
              else s += lift[i];
              s = s > 0 ? s : 0;
            }
            const u32x4 wa = mx_values<X == kMxBf16>(u[p], scale_of(s));
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[i][m] = mfma16<X == kMxBf16>(wa, x[d][m][p], acc[i][m]);
          }
        }
      }
    }
  }
  // lane l of a product holds outputs 4 (l / 16) .. + 3 of row l % 16
#pragma unroll
  for (int first = 0; first < kOutTiles; first += kBatch) {
    if (STAGE || first > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < kBatchTiles; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        if (first * SIDES + i < CT) sums[((wave * kBatchTiles + i) * MT + m) * 64 + lane] = acc[first * SIDES + i][m];
    __syncthreads();
    for (int q = threadIdx.x; q < kBatch * MT * 64; q += waves * 64) {
      const int l = q & 63, m = (q >> 6) % MT, out = (q >> 6) / MT;
      const int row = m * 16 + (l & 15), o = 4 * (l >> 4), tile = tile0 + (first + out) * SIDES;
      if (row >= rows || tile >= a.lay.tiles || first + out >= kOutTiles) continue;
      f32x4 t[SIDES];
#pragma unroll
      for (int i = 0; i < SIDES; ++i) {
        const int at = ((out * SIDES + i) * MT + m) * 64 + l;
        t[i] = sums[at];
#pragma unroll
        for (int k = 1; k < waves; ++k) t[i] += sums[k * kBatchTiles * MT * 64 + at];
        if constexpr (X == kMxF16) {
          const uint32_t tops = *(const uint32_t*)(a.packed + a.lay.tops_at + (size_t)(tile + i) * 16 + o);
#pragma unroll
          for (int e = 0; e < 4; ++e) t[i][e] *= mx_row_factor(tops >> (8 * e) & 255);
        }
      }
      uint16_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (SIDES == 2) t[0][e] = mx_gate(t[0][e], t[1][e], a.act);
        v[e] = mx_round(t[0][e], a.y_bf16);
      }
      const int n = tile / SIDES * 16 + o;
      uint16_t* y = a.y + (m0 + row) * a.N + n;
      if (n + 4 <= a.N) {
        *(u32x2_at2*)y = u32x2{(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) y[e] = v[e];
      }
    }
  }
}

template <int X, int MT, int CT, int SIDES, bool STAGE = (MT > 1 || (X != kMxCodes && CT >= 4))>
hipError_t run(const MxGemmCall& c, hipStream_t s) {
  // Registers: 4 CT MT of sums, and DEPTH times the operands.  Fewer chunks at once leave room for a second workgroup on a CU,
  // but for few tiles of codes.  Us with 190 / 120 here: 16 rows in 16 bits, 8192 -> 28672: 39 / 30; 32, 14336 -> 4096: 17.6 / 15.1; 64 gated
  // rows in codes, 4096 -> 14336: 19.0 / 17.7; 61 rows in codes, 8192 -> 8192 (CT 2): 11.7 / 12.7.
  constexpr int kChunk = X == kMxCodes ? 5 * CT + 5 * MT : 6 * CT + 16 * MT;
  constexpr int kFree = (STAGE && !(X == kMxCodes && CT <= 2) ? 120 : 190) - 4 * CT * MT;
  constexpr int DEPTH = kFree >= 4 * kChunk ? 4 : kFree >= 2 * kChunk ? 2 : 1;
  constexpr int BOUND = MT == 1 && CT <= 2 ? 1024 : 512;
  const int groups = (c.lay.tiles + CT - 1) / CT;
  const int64_t row_blocks = (c.M + MT * 16 - 1) / (MT * 16);
  mx_skinny_kernel<X, MT, CT, SIDES, DEPTH, BOUND, STAGE><<<(unsigned)(groups * row_blocks), kSkinnyWaves * 64, 0, s>>>(c, groups);
  return hipGetLastError();
}

// More tiles a wave read x less often (every workgroup reads all of it), fewer fill the card: as many as leave 200
// workgroups.  Us for 1 / 2 / 4: 16 rows in 16 bits, 8192 -> 28672: 62 / 44 / 34; 61 in codes, 8192 -> 8192: 31 / 18 / 26; 48 gated, 4096 ->
// 14336: - / 49 / 31.  Up to 8 rows x is little, and more workgroups are better: one row, 4096 -> 14336: 8.5 / 8.2 / 9.1; 4 in codes,
// 8192 -> 8192: 7.7 / 8.0 / 9.0.  Eight for 33 to 48 rows in 16 bits, us for 4 / 8: 48, 8192 -> 28672: 46.9 / 38.0, 14336 -> 28672: 75 / 58;
// 40 gated, 4096 -> 14336: 22.5 / 22.3.  For 32 rows 4 is better (gated, 4096 -> 14336: 16.6 / 20.3), for more the sums leave no registers.
int tiles_a_wave(const MxGemmCall& c) {
  if (c.M > 32 && c.M <= 48 && c.x_kind != kMxCodes && c.lay.tiles >= 8 * 200) return 8;
  if (c.M > 8 && c.lay.tiles >= 4 * 200) return 4;
  return c.lay.sides == 2 || c.lay.tiles >= 2 * (c.M > 8 ? 200 : 400) ? 2 : 1;
}

template <int X, int MT, int SIDES>
hipError_t run_tiles(const MxGemmCall& c, hipStream_t s) {
  switch (tiles_a_wave(c)) {
    case 8:
      if constexpr (X != kMxCodes && MT == 3) return run<X, MT, 8, SIDES>(c, s);
    case 4: return run<X, MT, 4, SIDES>(c, s);
    case 2: return run<X, MT, 2, SIDES>(c, s);
    default: return run<X, MT, SIDES, SIDES>(c, s);
  }
}

template <int X, int SIDES>
hipError_t run_rows(const MxGemmCall& c, hipStream_t s) {
  if (c.M <= 16) return run_tiles<X, 1, SIDES>(c, s);
  if (c.M <= 32) return run_tiles<X, 2, SIDES>(c, s);
  if (c.M <= 48) return run_tiles<X, 3, SIDES>(c, s);
  return run_tiles<X, 4, SIDES>(c, s);
}

template <int X>
hipError_t run_sides(const MxGemmCall& c, hipStream_t s) {
  return c.lay.sides == 2 ? run_rows<X, 2>(c, s) : run_rows<X, 1>(c, s);
}

}  // namespace

// Rounds of workgroups over the card, of chunks over a workgroup's waves, and what a chunk takes (measured, 64 rows).
double mx_skinny_us(const MxGemmCall& c) {
  const int ct = tiles_a_wave(c), chunks = (c.K + 127) / 128;
  const int64_t groups = (c.M + 63) / 64 * ((c.lay.tiles + ct - 1) / ct);
  const double chunk = c.x_kind == kMxCodes ? 0.5 + 0.33 * ct : 1.1 + 0.5 * ct;
  return 3.0 + (double)((groups + kMxCus - 1) / kMxCus) * ((chunks + kSkinnyWaves - 1) / kSkinnyWaves) * chunk;
}

bool mx_skinny_fits(const MxGemmCall& c) { return grid_fits((c.M + 15) / 16 * (c.lay.tiles / c.lay.sides), 512); }

hipError_t launch_mx_skinny(const MxGemmCall& c, hipStream_t s) {
  if (c.x_kind == kMxCodes) return run_sides<kMxCodes>(c, s);
  return c.x_kind == kMxF16 ? run_sides<kMxF16>(c, s) : run_sides<kMxBf16>(c, s);
}

}  // namespace gq
