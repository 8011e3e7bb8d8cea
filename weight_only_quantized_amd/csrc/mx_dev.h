// Device helpers of the microscaled products.
#pragma once
#include "bufmem.h"
#include "mx.h"
#include "serving_dev.h"

namespace gq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kFp4 = 4;                   // operand format of the scaled matrix instructions: e2m1

// A float16 operand holds 2^-24 .. 65504, a scale byte 2^-127 .. 2^127: weights of float16 activations
// are made relative to their row's largest scale, which goes to 2^13 (6 * 2^13 is in range), and the sum is
// multiplied back.  Exact for scales down to 2^-36 of the row's largest; below, rounded to 2^-24 of that unit.
constexpr int kF16Top = 13;

// float whose exponent field is `byte` (the conversions below read only that field: 2^(byte - 127), NaN for 255).
__device__ __forceinline__ float scale_of(int byte) { return __builtin_bit_cast(float, (uint32_t)byte << 23); }

// Eight codes as eight values times 2^(byte - 127) in float16 or bfloat16, rounded to nearest even.
template <int BF16>
__device__ __forceinline__ u32x4 mx_values(uint32_t codes, float scale) {
  u32x4 v;
  if constexpr (BF16) {
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  } else {
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3));
  }
  return v;
}

// What a row's sum is multiplied by (float16 activations; see kF16Top).
__device__ __forceinline__ float mx_row_factor(int top) {
  return top == 255 ? __builtin_nanf("") : ldexpf(1.0f, top - 127 - kF16Top);
}

// act(g) * u.  Both activations are g times a logistic function, whose exponential may overflow (what is
// below 2^-128 counts as 0) or vanish without harm: silu(g) = g / (1 + exp(-g)); gelu's tanh form 0.5 g (1 + tanh(t)) = g / (1 + exp(-2 t)),
// t = sqrt(2 / pi) (g + 0.044715 g^3), which keeps its digits for negative g, where 1 + tanh cancels.
__device__ __forceinline__ float mx_gate(float g, float u, int act) {
  constexpr float kLog2e = 1.4426950408889634f, kRoot = 0.7978845608028654f;
  const float t = act == GPTQ_MX_SILU ? g : 2.0f * kRoot * (g + 0.044715f * g * g * g);
  // The card's reciprocal gives 0 below 2^-126, where g times it is still in range: it is taken of a quarter of the sum.
  const float quarter = __builtin_fmaf(0.25f, __builtin_amdgcn_exp2f(-kLog2e * t), 0.25f);
  return g * (0.25f * __builtin_amdgcn_rcpf(quarter)) * u;
}

// Results of rows whose length is odd lie at any even address: vectors that say so.
typedef u32x4 __attribute__((aligned(2), may_alias)) u32x4_at2;
typedef u32x2 __attribute__((aligned(2), may_alias)) u32x2_at2;

__device__ __forceinline__ uint16_t mx_round(float v, int bf16) { return bf16 ? from_f32<1>(v) : from_f32<0>(v); }

}  // namespace gq
