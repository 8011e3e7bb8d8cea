// Products with packed 4-bit weights for few rows: y = x W^T, or act(x Wg^T) * (x Wu^T).
//
// Bound by the weights' bytes.  A wave multiplies a tile of 16 outputs (a gated pair: two) with up to
// 64 rows, straight from global memory to registers: weights are the first operand of a 16 x 16
// matrix instruction, read once in 1 KB runs, rows of x the second.  The waves of a workgroup take
// the chunks of 128 inputs in turn and their sums are added in LDS in a fixed order, so a call's
// bits do not depend on timing.  Activations in the format go to v_mfma_scale_f32_16x16x128_f8f6f4 with both
// sides' scales; 16-bit ones to 16x16x32 products with the weights turned into the same type in
// registers, which is exact (mx_dev.h).
#include "mx_dev.h"
#include "serving.h"

namespace gq {
namespace {

// Which block of its stage lane group g (16 lanes) multiplies in chunk c (0 or 1) of it: any order serves
// as long as both operands agree, and this one takes both bytes from one scale word of each operand.
__device__ __forceinline__ int chunk_block(int g, int c) { return (g & 1) + 4 * (g >> 1) + 2 * c; }

// Inputs in flight: DEPTH chunks a wave.
template <int X, int MT, int SIDES, int DEPTH>
__global__ void __launch_bounds__(1024) mx_skinny_kernel(MxGemmCall a, int groups) {
  extern __shared__ __align__(16) uint8_t smem[];
  f32x4* sums = (f32x4*)smem;             // [wave][side][row tile][lane]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int column = blockIdx.x % groups;                // tile of 16 outputs
  const int64_t m0 = (int64_t)(blockIdx.x / groups) * (MT * 16);
  const int rows = a.M - m0 < MT * 16 ? (int)(a.M - m0) : MT * 16, blocks = a.K / 32;
  const int chunks = 2 * a.lay.stages - ((blocks & 7) == 1 || (blocks & 7) == 2);       // chunk 1 starts at block 2

  int lift[SIDES] = {};                   // added to a scale byte (float16 activations)
  if constexpr (X == kMxF16) {
#pragma unroll
    for (int i = 0; i < SIDES; ++i)
      lift[i] = 127 + kF16Top - a.packed[a.lay.tops_at + ((size_t)column * SIDES + i) * 16 + r];
  }
  const rsrc_t x_rsrc = make_rsrc(a.x + m0 * a.x_bytes, (uint32_t)(rows * a.x_bytes));
  const rsrc_t xs_rsrc = X == kMxCodes ? make_rsrc(a.x_scales + m0 * a.x_scale_stride, (uint32_t)(rows * a.x_scale_stride))
                                       : x_rsrc;
  constexpr int kBlockBytes = X == kMxCodes ? 16 : 64, XL = kBlockBytes / 16;

  f32x4 acc[SIDES][MT] = {};
  for (int base = wave; base < chunks; base += waves * DEPTH) {
    u32x4 w[DEPTH][SIDES], x[DEPTH][MT][XL];
    uint32_t ws[DEPTH][SIDES], xs[DEPTH][MT];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int q = base + d * waves, stage = q >> 1, block = chunk_block(g, q & 1);
      const bool in = stage * 8 + block < blocks;        // of x's row; packed weights hold whole stages
      // chunks past the last read as zeros
      const size_t tile = q < chunks ? (size_t)stage * a.lay.tiles + (size_t)column * SIDES : 0;
      const rsrc_t w_rsrc = make_rsrc(a.packed + tile * kMxTileBytes, q < chunks ? SIDES * kMxTileBytes : 0);
      const rsrc_t s_rsrc = make_rsrc(a.packed + a.lay.scales_at + tile * 128, q < chunks ? SIDES * 128 : 0);
#pragma unroll
      for (int i = 0; i < SIDES; ++i) {
        w[d][i] = load_b128(w_rsrc, (uint32_t)(block * 256 + r * 16) + i * kMxTileBytes, 0);
        ws[d][i] = load_b32(s_rsrc, (uint32_t)((g & 1) * 64 + r * 4) + i * 128, 0);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + r;
        const bool there = in && row < rows;
        const uint32_t at = (uint32_t)(row * a.x_bytes) + (uint32_t)(stage * 8 + block) * kBlockBytes;
#pragma unroll
        for (int p = 0; p < XL; ++p) x[d][m][p] = load_b128(x_rsrc, there ? at + p * 16 : kOob, 0);
        if constexpr (X == kMxCodes) {
          // the word that holds the block's byte; a block past K may share it, and is masked below
          const uint32_t word = (uint32_t)(row * a.x_scale_stride) + (uint32_t)(stage * 8 + 4 * (g >> 1));
          xs[d][m] = load_b32(xs_rsrc, there ? word : kOob, 0);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int c = (base + d * waves) & 1;
#pragma unroll
      for (int i = 0; i < SIDES; ++i) {
        const uint32_t byte = ws[d][i] >> (16 * (g >> 1) + 8 * c) & 255;
        if constexpr (X == kMxCodes) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const u32x4 u = w[d][i], v = x[d][m][0];
            const i32x8 wa = {(int)u[0], (int)u[1], (int)u[2], (int)u[3], 0, 0, 0, 0};
            const i32x8 xb = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
            const uint32_t x_byte = xs[d][m] >> (8 * (g & 1) + 16 * c) & 255;
            acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, acc[i][m], kFp4, kFp4, 0, (int)byte, 0,
                                                                         (int)x_byte);
          }
        } else {
          int s = (int)byte;
          if constexpr (X == kMxF16) s = s + lift[i] > 0 ? s + lift[i] : 0;
          const float scale = scale_of(s);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const u32x4 wa = mx_values<X == kMxBf16>(w[d][i][p], scale);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[i][m] = mfma16<X == kMxBf16>(wa, x[d][m][p], acc[i][m]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < SIDES; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[((wave * SIDES + i) * MT + m) * 64 + lane] = acc[i][m];
  __syncthreads();
  // lane l of a product holds outputs 4 (l / 16) .. + 3 of row l % 16
  for (int q = threadIdx.x; q < MT * 64; q += blockDim.x) {
    const int row = (q >> 6) * 16 + (q & 15), o = 4 * ((q & 63) >> 4);
    if (row >= rows) continue;
    f32x4 t[SIDES];
#pragma unroll
    for (int i = 0; i < SIDES; ++i) {
      t[i] = sums[i * MT * 64 + q];
      for (int k = 1; k < waves; ++k) t[i] += sums[(k * SIDES + i) * MT * 64 + q];
      if constexpr (X == kMxF16) {
        const uint32_t tops = *(const uint32_t*)(a.packed + a.lay.tops_at + ((size_t)column * SIDES + i) * 16 + o);
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
    const int n = column * 16 + o;
    uint16_t* y = a.y + (m0 + row) * a.N + n;
    if (a.N % 4 == 0 && n < a.N) {
      *(uint64_t*)y = (uint64_t)(v[0] | (uint32_t)v[1] << 16) | (uint64_t)(v[2] | (uint32_t)v[3] << 16) << 32;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) y[e] = v[e];
    }
  }
}

template <int X, int MT, int SIDES>
hipError_t run(const MxGemmCall& c, hipStream_t s) {
  constexpr int DEPTH = MT * SIDES * (X == kMxCodes ? 1 : 4) <= 4 ? 4 : MT * (X == kMxCodes ? 1 : 4) <= 4 ? 2 : 1;
  const int groups = c.lay.tiles / SIDES, waves = 8;
  const int64_t row_blocks = (c.M + MT * 16 - 1) / (MT * 16);
  const size_t lds = (size_t)waves * SIDES * MT * 64 * sizeof(f32x4);
  mx_skinny_kernel<X, MT, SIDES, DEPTH><<<(unsigned)(groups * row_blocks), waves * 64, lds, s>>>(c, groups);
  return hipGetLastError();
}

template <int X, int SIDES>
hipError_t run_rows(const MxGemmCall& c, hipStream_t s) {
  if (c.M <= 16) return run<X, 1, SIDES>(c, s);
  if (c.M <= 32) return run<X, 2, SIDES>(c, s);
  if (c.M <= 48) return run<X, 3, SIDES>(c, s);
  return run<X, 4, SIDES>(c, s);
}

template <int X>
hipError_t run_sides(const MxGemmCall& c, hipStream_t s) {
  return c.lay.sides == 2 ? run_rows<X, 2>(c, s) : run_rows<X, 1>(c, s);
}

}  // namespace

bool mx_skinny_fits(const MxGemmCall& c) { return grid_fits((c.M + 15) / 16 * (c.lay.tiles / c.lay.sides), 512); }

hipError_t launch_mx_skinny(const MxGemmCall& c, hipStream_t s) {
  if (c.x_kind == kMxCodes) return run_sides<kMxCodes>(c, s);
  return c.x_kind == kMxF16 ? run_sides<kMxF16>(c, s) : run_sides<kMxBf16>(c, s);
}

}  // namespace gq
