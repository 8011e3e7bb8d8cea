// Library-internal declarations of the operators on microscaled 4-bit floating point: the validated
// calls as the launchers see them, and the layout of packed weights.
//
// A block of the format is 32 consecutive inputs of one row: 16 bytes of codes and one scale byte.
// Packed weights are cut into tiles of 16 outputs (rows past N are zeros; of a gated pair, tile 2 i
// holds gate rows, tile 2 i + 1 the up rows of the same outputs) and stages of 256 inputs (inputs past
// K are zeros).  One stage of one tile is 2048 bytes, [block 0..7][row 0..15][16 bytes], so that each
// matrix instruction's operand is read 16 bytes a lane in runs of 256 bytes, whatever its shape:
// 16 x 16 x 128 takes four blocks of a tile, 32 x 32 x 64 two blocks of two tiles.  Its scales are 32
// words, [block & 1][row]: byte j of a word belongs to block 2 j + (block & 1), so the four
// 32 x 32 x 64 instructions of a stage name bytes 0..3 of one register.  A tile's stages follow
// one another: a wave that streams one reads on in memory (one row, 4096 -> 14336, when this was chosen: 7.7 us; 9.1 with all
// tiles' first stages first, where the kernel by tiles takes the same time).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gptq_mi355x.h"

namespace gq {

constexpr int kMxStage = 256;             // inputs of a stage
constexpr int kMxTileBytes = 2048;        // codes of one stage of one tile

struct MxPacked {
  int sides, tiles, stages;               // tiles of all sides
  size_t scales_at, tops_at, bytes;       // codes lie at 0
};
// The parts of N x K weights with `sides` 1 or 2 (gated).  tops: each row's largest scale byte below
// 255 over blocks that hold more than zeros, or 255 when the row has a NaN block.
inline MxPacked mx_packed(int N, int K, int sides) {
  MxPacked p{sides, sides * ((N + 15) / 16), (K + kMxStage - 1) / kMxStage, 0, 0, 0};
  const size_t pieces = (size_t)p.tiles * p.stages;
  p.scales_at = pieces * kMxTileBytes;
  p.tops_at = p.scales_at + pieces * 128;
  p.bytes = (p.tops_at + (size_t)p.tiles * 16 + 255) / 256 * 256;
  return p;
}

hipError_t launch_mx_quantize(const void* x, int64_t x_stride, int64_t rows, int K, int dtype, uint8_t* codes,
                              uint8_t* scales, int64_t scale_stride, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t scale_stride, int64_t rows, int K,
                                void* out, int dtype, hipStream_t s);
hipError_t launch_mx_pack(const gptq_mx_tensor* const side[2], int sides, int N, int K, void* packed, hipStream_t s);

enum MxInput { kMxCodes = 0, kMxF16 = 1, kMxBf16 = 2 };
struct MxGemmCall {
  const uint8_t* packed;
  MxPacked lay;
  int N, K, act;                          // act: gptq_mx_activation
  int x_kind;                             // MxInput
  const uint8_t* x;                       // rows x_bytes apart
  int64_t x_bytes;
  const uint8_t* x_scales;                // kMxCodes only
  int64_t x_scale_stride;
  int64_t M;
  uint16_t* y;                            // [M, N]
  int y_bf16;
};
constexpr int kMxCus = 256;               // compute units of the card

// The kernel that streams the weights for each 64 rows (mx_skinny.hip) takes calls of up to this many rows.  Us streamed / by tiles:
// in 16 bits 33 rows, 8192 -> 28672: 36 / 65, 4096 -> 14336 gated: 21 / 26; 64 rows, 8192 -> 28672: 54 / 67, 14336 -> 4096: 27 / 71, 4096 ->
// 4096: 11 / 22, 4096 -> 14336 gated: 25.7 / 26.2; in codes 33 rows, 14336 -> 4096: 9.5 / 22, 64 rows there 14.3 / 23.3, 8192 -> 8192: 11.7 /
// 14.9.  Many outputs in codes are the other way about and go streamed all the same: 33 rows, 8192 -> 28672: 32.6 / 30.1, 64 rows 43.2 /
// 32.8, 64 gated, 4096 -> 14336: 17.0 / 13.9 ...
constexpr int64_t kMxSkinnyRows = 64;
bool mx_skinny_fits(const MxGemmCall& c);
hipError_t launch_mx_skinny(const MxGemmCall& c, hipStream_t s);
// ... and longer ones that its estimate, in us, puts before the kernel by tiles (mx_tiled.hip): few outputs, or 16 bits and few
// rows.  The estimates count rounds and steps, no bytes: where the weights' bytes alone take longer (64 rows in codes, 8192 -> 28672: 20
// estimated by tiles, 32.8 measured) both are low.  Us by tiles / streamed: 128 rows in 16 bits, 4096 -> 4096: 22.5 / 16.7, 14336 -> 4096: 72 / 45, 4096 -> 14336 gated: 38 / 53; 256 rows,
// 4096 -> 512: 23 / 10, 4096 -> 4096: 23 / 28; in codes 128 rows, 4096 -> 4096: 8.6 / 10.8, 256 rows, 4096 -> 512: 7.7 / 6.5.
double mx_skinny_us(const MxGemmCall& c);
double mx_tiled_us(const MxGemmCall& c);
bool mx_tiled_fits(const MxGemmCall& c);
hipError_t launch_mx_tiled(const MxGemmCall& c, hipStream_t s);

}  // namespace gq
