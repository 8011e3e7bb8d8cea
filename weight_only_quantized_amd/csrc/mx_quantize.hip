// Rows of activations or weights to microscaled 4-bit floating point and back, and packed weights.
//
// Mathematics: a block's scale is 2^e, e = floor(log2 max|x|) - 2 (the largest exponent of an element),
// so the exponent field of the largest magnitude, less two, is the scale byte; an element is x 2^-e rounded
// to 0 .5 1 1.5 2 3 4 6, ties to the even code, anything past 6 to 6.  The card's conversion does the division
// and the rounding at once (checked against the definition for every 16-bit input), so each is rounded once.
//
// Bound by memory: 2 bytes in, 17/32 out for a 16-bit value.  A lane takes eight values (16 bytes of 16-bit
// ones), four neighbouring lanes a block: loads and stores of a wave are each one run, and a block's maximum
// takes two exchanges between neighbours.  2777 rows of 14336 float16 values: 20.5 us to quantize (4.9 TB/s of the 5.1 that
// a large copy reaches), 17.5 back (5.7, codes from the caches); one row of 4096: 2.0 each on the device, 7 and 6 on the host.
#include "mx_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 256 * 8;       // all of a card's threads; longer calls take turns

// Group G of eight values lies in row G / per_row at 8 (G % per_row).  Each turn moves on by a whole
// number of rows and a rest, so only a lane's place within the block's run needs a division, in 32 bits.
struct Walk {
  int64_t groups;                         // of all rows
  uint32_t per_row, step_rest;
  int64_t step, step_rows;
};

Walk walk_of(int64_t rows, int K, int blocks) {
  Walk w{};
  w.per_row = (uint32_t)K / 8;
  w.groups = rows * w.per_row;
  w.step = (int64_t)blocks * kThreads;
  w.step_rows = w.step / w.per_row;
  w.step_rest = (uint32_t)(w.step % w.per_row);
  return w;
}

int blocks_of(int64_t groups) {
  const int64_t n = (groups + kThreads - 1) / kThreads;
  return (int)(n < kMaxBlocks ? n : kMaxBlocks);
}

// body(row, first value) of each group of this thread.
template <typename Body>
__device__ __forceinline__ void each_group(const Walk& w, Body body) {
  int64_t first = (int64_t)blockIdx.x * kThreads, row = first / w.per_row;
  uint32_t rest = (uint32_t)(first - row * w.per_row);
  for (; first < w.groups; first += w.step) {
    const uint32_t at = rest + threadIdx.x, over = at / w.per_row;
    if (first + threadIdx.x < w.groups) body(row + over, (at - over * w.per_row) * 8);
    row += w.step_rows;
    rest += w.step_rest;
    if (rest >= w.per_row) {
      rest -= w.per_row;
      ++row;
    }
  }
}

// Bits of a value (by value: a bit cast of a vector's element in place takes the first one's).
__device__ __forceinline__ float as_f32(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t as_u32(float v) { return __builtin_bit_cast(uint32_t, v); }

// The largest magnitude among eight 16-bit values, as bits.
__device__ __forceinline__ uint32_t top16(u32x4 v) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = v[i] & 0x7fff, hi = (v[i] >> 16) & 0x7fff;
    most = most > lo ? most : lo;
    most = most > hi ? most : hi;
  }
  return most;
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const uint8_t* x, int64_t x_stride, Walk w, uint8_t* codes,
                                                            uint8_t* scales, int64_t scale_stride, int64_t code_stride) {
  each_group(w, [&](int64_t row, uint32_t k) {
    uint32_t most = 0;
    u32x4 v[DTYPE == GPTQ_F32 ? 2 : 1];
    if constexpr (DTYPE == GPTQ_F32) {
      const uint8_t* at = x + (row * x_stride + k) * 4;
      v[0] = *(const u32x4*)at;
      v[1] = *(const u32x4*)(at + 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = v[i >> 2][i & 3] & 0x7fffffff;
        most = most > m ? most : m;
      }
    } else {
      v[0] = *(const u32x4*)(x + (row * x_stride + k) * 2);
      most = top16(v[0]);
    }
    // magnitudes order as their bits do, infinities and NaN above all
    uint32_t other = __shfl_xor(most, 1);
    most = most > other ? most : other;
    other = __shfl_xor(most, 2);
    most = most > other ? most : other;
    int field;                            // of float32
    if constexpr (DTYPE == GPTQ_F32) field = (int)(most >> 23);
    else if constexpr (DTYPE == GPTQ_BF16) field = (int)(most >> 7);
    else field = (int)(__builtin_bit_cast(uint32_t, to_f32<0>((uint16_t)most)) >> 23);
    const int byte = field == 255 ? 255 : field > 2 ? field - 2 : 0;
    const float scale = scale_of(byte);
    uint32_t out = 0;
    if constexpr (DTYPE == GPTQ_F32) {
#define GQ_PAIR(i)                                                                                                                  \
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, as_f32(v[(i) / 2][2 * ((i) & 1)]), as_f32(v[(i) / 2][2 * ((i) & 1) + 1]), \
                                                 scale, i)
      GQ_PAIR(0); GQ_PAIR(1); GQ_PAIR(2); GQ_PAIR(3);
#undef GQ_PAIR
    } else if constexpr (DTYPE == GPTQ_BF16) {
#define GQ_PAIR(i) out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2, (uint32_t)v[0][i]), scale, i)
      GQ_PAIR(0); GQ_PAIR(1); GQ_PAIR(2); GQ_PAIR(3);
#undef GQ_PAIR
    } else {
#define GQ_PAIR(i) out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(out, __builtin_bit_cast(f16x2, (uint32_t)v[0][i]), scale, i)
      GQ_PAIR(0); GQ_PAIR(1); GQ_PAIR(2); GQ_PAIR(3);
#undef GQ_PAIR
    }
    *(uint32_t*)(codes + row * code_stride + k / 2) = byte == 255 ? 0u : out;
    if (!(k & 31)) scales[row * scale_stride + k / 32] = (uint8_t)byte;
  });
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t scale_stride,
                                                              int64_t code_stride, Walk w, uint8_t* out) {
  each_group(w, [&](int64_t row, uint32_t k) {
    const uint32_t c = *(const uint32_t*)(codes + row * code_stride + k / 2);
    const float scale = scale_of(scales[row * scale_stride + k / 32]);
    const int64_t at = row * (code_stride * 2) + k;
    if constexpr (DTYPE == GPTQ_F32) {
      u32x4 v[2];
#define GQ_PAIR(i)                                                                 \
  {                                                                                \
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, i);         \
    v[(i) / 2][2 * ((i) & 1)] = as_u32(p[0]);                                      \
    v[(i) / 2][2 * ((i) & 1) + 1] = as_u32(p[1]);                                  \
  }
      GQ_PAIR(0) GQ_PAIR(1) GQ_PAIR(2) GQ_PAIR(3)
#undef GQ_PAIR
      *(u32x4*)(out + at * 4) = v[0];
      *(u32x4*)(out + at * 4 + 16) = v[1];
    } else {
      *(u32x4*)(out + at * 2) = mx_values<DTYPE == GPTQ_BF16>(c, scale);
    }
  });
}

struct PackSide {
  const uint8_t *codes, *scales;
  int64_t scale_stride;
};

// One workgroup a tile (mx.h): runs once, when weights are loaded.  A block of nothing but 0 and -0 is packed with scale
// 0, which its values do not show: whatever its own was, it must not set the unit of its row's other weights (kF16Top).
__global__ void __launch_bounds__(kThreads) pack_kernel(PackSide a, PackSide b, int N, int K, MxPacked lay, uint8_t* out) {
  __shared__ int tops[kThreads];
  const int tile = blockIdx.x, side = tile % lay.sides, blocks = K / 32;
  const PackSide src = side ? b : a;
  uint8_t* codes = out + (size_t)tile * lay.stages * kMxTileBytes;
  uint8_t* scales = out + lay.scales_at + (size_t)tile * lay.stages * 128;
  const int row = threadIdx.x % 16;       // a thread's blocks are all of one row
  const int64_t n = (int64_t)(tile / lay.sides) * 16 + row;
  int top = 0, bad = 0;
  for (int i = threadIdx.x; i < lay.stages * 128; i += kThreads) {
    const int block = i / 16;
    u32x4 v = {0, 0, 0, 0};
    int s = 0;
    if (n < N && block < blocks) {
      v = *(const u32x4*)(src.codes + n * (K / 2) + (int64_t)block * 16);
      s = src.scales[n * src.scale_stride + block];
      if (s == 255) bad = 1;
      else if (!((v[0] | v[1] | v[2] | v[3]) & 0x77777777)) s = 0;
      else if (s > top) top = s;
    }
    *(u32x4*)(codes + (size_t)i * 16) = v;
    scales[(block / 8 * 32 + block % 2 * 16 + row) * 4 + block % 8 / 2] = (uint8_t)s;
  }
  tops[threadIdx.x] = bad ? 255 : top;
  __syncthreads();
  if (threadIdx.x < 16) {
    for (int i = threadIdx.x; i < kThreads; i += 16) top = tops[i] > top ? tops[i] : top;
    if (bad) top = 255;
    out[lay.tops_at + (size_t)tile * 16 + threadIdx.x] = (uint8_t)top;
  }
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int64_t x_stride, int64_t rows, int K, int dtype, uint8_t* codes,
                              uint8_t* scales, int64_t scale_stride, hipStream_t s) {
  const int blocks = blocks_of(rows * (K / 8));
  const Walk w = walk_of(rows, K, blocks);
  auto run = [&](auto kernel) {
    kernel<<<blocks, kThreads, 0, s>>>((const uint8_t*)x, x_stride, w, codes, scales, scale_stride, (int64_t)K / 2);
  };
  if (dtype == GPTQ_F32) run(quantize_kernel<GPTQ_F32>);
  else if (dtype == GPTQ_BF16) run(quantize_kernel<GPTQ_BF16>);
  else run(quantize_kernel<GPTQ_F16>);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t scale_stride, int64_t rows, int K,
                                void* out, int dtype, hipStream_t s) {
  const int blocks = blocks_of(rows * (K / 8));
  const Walk w = walk_of(rows, K, blocks);
  auto run = [&](auto kernel) {
    kernel<<<blocks, kThreads, 0, s>>>(codes, scales, scale_stride, (int64_t)K / 2, w, (uint8_t*)out);
  };
  if (dtype == GPTQ_F32) run(dequantize_kernel<GPTQ_F32>);
  else if (dtype == GPTQ_BF16) run(dequantize_kernel<GPTQ_BF16>);
  else run(dequantize_kernel<GPTQ_F16>);
  return hipGetLastError();
}

hipError_t launch_mx_pack(const gptq_mx_tensor* const side[2], int sides, int N, int K, void* packed, hipStream_t s) {
  PackSide p[2] = {};
  for (int i = 0; i < sides; ++i) p[i] = PackSide{side[i]->codes, side[i]->scales, side[i]->scale_stride};
  const MxPacked lay = mx_packed(N, K, sides);
  pack_kernel<<<lay.tiles, kThreads, 0, s>>>(p[0], p[1], N, K, lay, (uint8_t*)packed);
  return hipGetLastError();
}

}  // namespace gq
