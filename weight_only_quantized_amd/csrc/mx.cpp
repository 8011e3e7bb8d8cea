// Host side of the operators on microscaled 4-bit floating point: argument checks and dispatch.  All
// checks run before any device work.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"
#include "serving.h"

namespace gq {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxInputs = 1 << 20;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

bool is_16bit(int32_t dtype) { return dtype == GPTQ_F16 || dtype == GPTQ_BF16; }

gptq_status check_device() {
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e);
  return is_gfx950_device(dev) ? GPTQ_OK : GPTQ_E_DEVICE;
}

bool inputs_fit(int64_t K) { return K >= 32 && K <= kMaxInputs && K % 32 == 0; }
bool outputs_fit(int64_t N) { return N >= 1 && N <= (1 << 20); }

// A tensor's sizes; its pointers only where it has rows.
gptq_status check_tensor(const gptq_mx_tensor* t) {
  if (!t || t->reserved != 0) return GPTQ_E_INVALID_ARG;
  if (!inputs_fit(t->K) || t->rows < 0 || t->rows > kMaxRows) return GPTQ_E_SHAPE;
  if (t->scale_stride < t->K / 32 || t->scale_stride % 4 != 0 || t->scale_stride > (1 << 20)) return GPTQ_E_INVALID_ARG;
  if (t->rows == 0) return GPTQ_OK;
  if (!t->codes || !t->scales || !aligned(t->codes, 16) || !aligned(t->scales, 4)) return GPTQ_E_INVALID_ARG;
  return GPTQ_OK;
}

size_t code_bytes(const gptq_mx_tensor* t) { return (size_t)t->rows * (t->K / 2); }
size_t scale_bytes(const gptq_mx_tensor* t) { return (size_t)t->rows * t->scale_stride; }
bool overlaps_tensor(const gptq_mx_tensor* t, const void* p, size_t n) {
  return overlaps(p, n, t->codes, code_bytes(t)) || overlaps(p, n, t->scales, scale_bytes(t));
}

gptq_status check_weight(const gptq_mx_weight* w) {
  if (!w || w->reserved != 0 || w->activation < GPTQ_MX_PLAIN || w->activation > GPTQ_MX_GELU_TANH) return GPTQ_E_INVALID_ARG;
  if (!inputs_fit(w->K) || !outputs_fit(w->N)) return GPTQ_E_SHAPE;
  return w->packed && aligned(w->packed, 256) ? GPTQ_OK : GPTQ_E_INVALID_ARG;
}

gptq_status run_gemm(const gptq_mx_weight* w, MxGemmCall& c, void* stream) {
  c.packed = (const uint8_t*)w->packed;
  c.lay = mx_packed(w->N, w->K, w->activation == GPTQ_MX_PLAIN ? 1 : 2);
  c.N = w->N;
  c.K = w->K;
  c.act = w->activation;
  if (overlaps(c.y, (size_t)c.M * c.N * 2, c.packed, c.lay.bytes)) return GPTQ_E_INVALID_ARG;
  const bool few = c.M <= kMxSkinnyRows || (mx_skinny_fits(c) && mx_skinny_us(c) < mx_tiled_us(c));
  if (few ? !mx_skinny_fits(c) : !mx_tiled_fits(c)) return GPTQ_E_SHAPE;
  const gptq_status st = check_device();
  if (st != GPTQ_OK) return st;
  const hipError_t e = few ? launch_mx_skinny(c, (hipStream_t)stream) : launch_mx_tiled(c, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" {

gptq_status gptq_mx_quantize(const void* x, int64_t x_stride, int32_t dtype, const gptq_mx_tensor* out, void* stream) {
  gptq_status st = check_tensor(out);
  if (st != GPTQ_OK) return st;
  if (!is_16bit(dtype) && dtype != GPTQ_F32) return GPTQ_E_INVALID_ARG;
  if (out->rows == 0) return GPTQ_OK;
  const int size = dtype == GPTQ_F32 ? 4 : 2;
  if (!x || !aligned(x, 16) || x_stride < out->K || x_stride > (int64_t(1) << 32) || x_stride * size % 16 != 0)
    return GPTQ_E_INVALID_ARG;
  const size_t xb = ((size_t)(out->rows - 1) * x_stride + out->K) * size;
  if (overlaps_tensor(out, x, xb) || overlaps(out->codes, code_bytes(out), out->scales, scale_bytes(out)))
    return GPTQ_E_INVALID_ARG;
  if ((st = check_device()) != GPTQ_OK) return st;
  const hipError_t e = launch_mx_quantize(x, x_stride, out->rows, out->K, dtype, out->codes, out->scales,
                                          out->scale_stride, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

gptq_status gptq_mx_dequantize(const gptq_mx_tensor* x, void* out, int32_t dtype, void* stream) {
  gptq_status st = check_tensor(x);
  if (st != GPTQ_OK) return st;
  if (!is_16bit(dtype) && dtype != GPTQ_F32) return GPTQ_E_INVALID_ARG;
  if (x->rows == 0) return GPTQ_OK;
  if (!out || !aligned(out, 16) || overlaps_tensor(x, out, (size_t)x->rows * x->K * (dtype == GPTQ_F32 ? 4 : 2)))
    return GPTQ_E_INVALID_ARG;
  if ((st = check_device()) != GPTQ_OK) return st;
  const hipError_t e = launch_mx_dequantize(x->codes, x->scales, x->scale_stride, x->rows, x->K, out, dtype,
                                            (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

gptq_status gptq_mx_weight_bytes(int32_t N, int32_t K, int32_t gated, size_t* bytes) {
  if (!bytes || (gated != 0 && gated != 1)) return GPTQ_E_INVALID_ARG;
  if (!inputs_fit(K) || !outputs_fit(N)) return GPTQ_E_SHAPE;
  *bytes = mx_packed(N, K, gated + 1).bytes;
  return GPTQ_OK;
}

gptq_status gptq_mx_pack(const gptq_mx_tensor* weight, const gptq_mx_tensor* up, void* packed, void* stream) {
  gptq_status st = check_tensor(weight);
  if (st == GPTQ_OK && up) st = check_tensor(up);
  if (st != GPTQ_OK) return st;
  if (!outputs_fit(weight->rows)) return GPTQ_E_SHAPE;
  if (up && (up->rows != weight->rows || up->K != weight->K)) return GPTQ_E_INVALID_ARG;
  if (!packed || !aligned(packed, 256)) return GPTQ_E_INVALID_ARG;
  const gptq_mx_tensor* side[2] = {weight, up};
  const size_t bytes = mx_packed((int)weight->rows, weight->K, up ? 2 : 1).bytes;
  if (overlaps_tensor(weight, packed, bytes) || (up && overlaps_tensor(up, packed, bytes))) return GPTQ_E_INVALID_ARG;
  if ((st = check_device()) != GPTQ_OK) return st;
  const hipError_t e = launch_mx_pack(side, up ? 2 : 1, (int)weight->rows, weight->K, packed, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

gptq_status gptq_mx_gemm(const gptq_mx_weight* weight, const void* x, int64_t x_stride, int32_t dtype, int64_t M, void* y,
                         void* stream) {
  const gptq_status st = check_weight(weight);
  if (st != GPTQ_OK) return st;
  if (!is_16bit(dtype)) return GPTQ_E_INVALID_ARG;
  if (M < 0 || M > kMaxRows) return GPTQ_E_SHAPE;
  if (M == 0) return GPTQ_OK;
  if (!x || !y || !aligned(x, 16) || !aligned(y, 16)) return GPTQ_E_INVALID_ARG;
  if (x_stride < weight->K || x_stride % 8 != 0 || x_stride > (1 << 21)) return GPTQ_E_INVALID_ARG;
  if (overlaps(y, (size_t)M * weight->N * 2, x, ((size_t)(M - 1) * x_stride + weight->K) * 2)) return GPTQ_E_INVALID_ARG;
  MxGemmCall c{};
  c.x_kind = dtype == GPTQ_BF16 ? kMxBf16 : kMxF16;
  c.x = (const uint8_t*)x;
  c.x_bytes = x_stride * 2;
  c.M = M;
  c.y = (uint16_t*)y;
  c.y_bf16 = dtype == GPTQ_BF16;
  return run_gemm(weight, c, stream);
}

gptq_status gptq_mx_gemm_mx(const gptq_mx_weight* weight, const gptq_mx_tensor* x, void* y, int32_t y_dtype, void* stream) {
  gptq_status st = check_weight(weight);
  if (st == GPTQ_OK) st = check_tensor(x);
  if (st != GPTQ_OK) return st;
  if (!is_16bit(y_dtype) || x->K != weight->K) return GPTQ_E_INVALID_ARG;
  if (x->rows == 0) return GPTQ_OK;
  if (!y || !aligned(y, 16) || overlaps_tensor(x, y, (size_t)x->rows * weight->N * 2)) return GPTQ_E_INVALID_ARG;
  MxGemmCall c{};
  c.x_kind = kMxCodes;
  c.x = x->codes;
  c.x_bytes = x->K / 2;
  c.x_scales = x->scales;
  c.x_scale_stride = x->scale_stride;
  c.M = x->rows;
  c.y = (uint16_t*)y;
  c.y_bf16 = y_dtype == GPTQ_BF16;
  return run_gemm(weight, c, stream);
}

}  // extern "C"
