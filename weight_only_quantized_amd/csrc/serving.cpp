// Host side of the serving operators: argument checks and dispatch.  All checks run before any
// device work; what lives in device memory (tables, lengths, ids) is checked by the kernels.
#include <hip/hip_runtime.h>

#include <cmath>

#include "internal.h"
#include "serving.h"

namespace gq {
namespace {

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

gptq_status check_cache(const gptq_kv_cache* c) {
  if (!c || c->reserved != 0) return GPTQ_E_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return GPTQ_E_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return GPTQ_E_UNSUPPORTED;
  if (c->num_pages < 1 || c->num_pages > 0x7fffffff || c->kv_heads < 1 || c->kv_heads > 1024) return GPTQ_E_SHAPE;
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return GPTQ_E_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return GPTQ_E_INVALID_ARG;
  return GPTQ_OK;
}

// The batch's sizes; its pointers only where there are rows.
gptq_status check_batch(const gptq_kv_batch* b) {
  if (!b || b->reserved != 0) return GPTQ_E_INVALID_ARG;
  if (b->rows < 0 || b->rows > (int64_t(1) << 24) || b->batch < 0 || b->batch > (1 << 20)) return GPTQ_E_SHAPE;
  if (b->table_width < 1 || b->table_width > (1 << 22)) return GPTQ_E_SHAPE;
  if (b->max_rows < 0 || b->max_rows > b->rows) return GPTQ_E_SHAPE;
  if (b->rows == 0 || b->batch == 0) return GPTQ_OK;
  if (!b->page_table || !b->at || !b->cu) return GPTQ_E_INVALID_ARG;
  if (!aligned(b->page_table, 4) || !aligned(b->at, 4) || !aligned(b->cu, 4)) return GPTQ_E_INVALID_ARG;
  return GPTQ_OK;
}

// A packed tensor of `rows` rows of `width` 16-bit elements, `stride` apart.
gptq_status check_rows(const void* p, int64_t width, int64_t stride) {
  if (!p || !aligned(p, 16)) return GPTQ_E_INVALID_ARG;
  if (stride < width || stride % 8 != 0 || stride > (int64_t(1) << 32)) return GPTQ_E_INVALID_ARG;
  return GPTQ_OK;
}

size_t row_bytes(int64_t rows, int64_t width, int64_t stride) { return ((size_t)(rows - 1) * stride + width) * 2; }

// Whether two packed tensors share memory; rows of one fused tensor (equal strides) may interleave.
bool rows_overlap(const void* a, int64_t wa, int64_t sa, const void* b, int64_t wb, int64_t sb, int64_t rows) {
  if (!overlaps(a, row_bytes(rows, wa, sa), b, row_bytes(rows, wb, sb))) return false;
  if (sa != sb) return true;
  const int64_t apart = ((int64_t)((uintptr_t)b - (uintptr_t)a)) / 2;
  const int64_t d = (apart % sa + sa) % sa;            // b's column within a's rows
  return d < wa || d + wb > sa;
}

size_t code_bytes(const gptq_kv_cache* c) {
  return (size_t)c->num_pages * c->kv_heads * c->page_size * c->head_dim;
}

// Whether [p, p + n) overlaps any array of the cache.
bool overlaps_cache(const gptq_kv_cache* c, const void* p, size_t n) {
  const size_t scales = (size_t)c->num_pages * c->kv_heads * 4;
  return overlaps(p, n, c->k_codes, code_bytes(c)) || overlaps(p, n, c->v_codes, code_bytes(c)) ||
         overlaps(p, n, c->k_scale, scales) || overlaps(p, n, c->v_scale, scales);
}

// Whether [p, p + n) overlaps the batch's tables.
bool overlaps_tables(const gptq_kv_batch* b, const void* p, size_t n) {
  return overlaps(p, n, b->page_table, (size_t)b->batch * b->table_width * 4) || overlaps(p, n, b->at, (size_t)b->batch * 4) ||
         overlaps(p, n, b->cu, ((size_t)b->batch + 1) * 4);
}

gptq_status check_rope(const gptq_rope* r, int head_dim) {
  if (r->reserved != 0 || !r->cos || !r->sin || !aligned(r->cos, 16) || !aligned(r->sin, 16)) return GPTQ_E_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return GPTQ_E_INVALID_ARG;
  if (r->dim < 16 || r->dim > head_dim || r->dim % 16 != 0) return GPTQ_E_UNSUPPORTED;
  if (r->rows < 1 || r->rows > (1 << 24)) return GPTQ_E_SHAPE;
  return GPTQ_OK;
}

// Whether a call has nothing to attend for.
bool no_queries(const gptq_kv_batch& b) { return b.rows == 0 || b.batch == 0 || b.max_rows == 0; }

gptq_status check_attention(const gptq_kv_cache* c, const gptq_kv_batch* b, const gptq_attention* a) {
  gptq_status st = check_cache(c);
  if (st == GPTQ_OK) st = check_batch(b);
  if (st != GPTQ_OK) return st;
  if (!a || !is_16bit(a->dtype) || !std::isfinite(a->scale)) return GPTQ_E_INVALID_ARG;
  if ((a->causal != 0 && a->causal != 1) || a->window < 0 || a->max_kv < 0) return GPTQ_E_INVALID_ARG;
  if (a->q_heads < 1 || a->q_heads % c->kv_heads != 0 || a->q_heads / c->kv_heads > 64) return GPTQ_E_SHAPE;
  return GPTQ_OK;
}

// Whether the keys are split over the card (kv_decode.hip) or each workgroup goes through all that its
// columns see (kv_prefill.hip).  For U units of 32 (row, head) columns over n thousand tokens splitting takes
// about 25 + U n / 30 us (U n / 20 when the codes of several sequences do not fit the caches), going through
// 6 + 20 n while every workgroup has a CU: the first for less than 590 units, fewer for short ones.
// Us, split / not, 8 kv heads of 128, 32 query heads: 1 sequence of 64 rows (U = 64), 2500 tokens 35 / 56,
// 16000: 52 / 315; 300 rows (304), 2000: 46 / 47, 3000: 57 / 66; 350 rows (352), 60000: 578 / 1169; 540 rows
// (544), 60000: 884 / 1173; 560 rows (560), 16000: 283 / 318; 600 rows (600), 30000: 655 / 592, 60000: 1363 /
// 1173; 2 of 270 rows (544), 9000: 160 / 183; 4 of 64 rows (256), 16000: 139 / 320; 4 of 130 rows (544), 20000:
// 445 / 402 (taken wrongly); 16 of 32 rows (512), 2500: 71 / 60, 8000: 180 / 173, 16000: 336 / 334; 20 of 32
// rows (640), 30000: 929 / 824.  Few short units (kv_local) come before both.
bool few_rows(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const int64_t columns = (int64_t)b.max_rows * (a.q_heads / c.kv_heads);
  if (columns <= 16 || kv_local(c, b, a)) return true;
  const int64_t units = (int64_t)b.batch * c.kv_heads * ((columns + 31) / 32), span = kv_span(c, b, a);
  return units <= 24 || (units <= 590 && units * span <= 590 * (span - 500));
}

bool kv_attention_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  return few_rows(c, b, a) ? kv_decode_fits(c, b, a) : kv_prefill_fits(c, b, a);
}

size_t kv_attention_ws_bytes(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  return few_rows(c, b, a) ? kv_decode_ws_bytes(c, b, a) : 0;
}

gptq_status check_bank(const gptq_lora_bank* k, int64_t M) {
  if (!k || k->reserved != 0 || !is_16bit(k->dtype)) return GPTQ_E_INVALID_ARG;
  if (k->rank < 8 || k->rank > 128 || k->rank % 8 != 0) return GPTQ_E_UNSUPPORTED;
  if (k->adapters < 1 || k->adapters > 65536) return GPTQ_E_SHAPE;
  if (k->in_features < 32 || k->in_features > (1 << 20) || k->in_features % 32 != 0) return GPTQ_E_SHAPE;
  if (k->out_features < 32 || k->out_features > (1 << 20) || k->out_features % 32 != 0) return GPTQ_E_SHAPE;
  if (M < 0 || M > (int64_t(1) << 24)) return GPTQ_E_SHAPE;
  return GPTQ_OK;
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" {

gptq_status gptq_kv_append(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const void* q, int64_t q_stride, int32_t q_heads,
                           void* q_out, int64_t q_out_stride, int32_t dtype, const gptq_rope* rope, void* stream) {
  gptq_status st = check_cache(cache);
  if (st == GPTQ_OK) st = check_batch(batch);
  if (st != GPTQ_OK) return st;
  if (!is_16bit(dtype)) return GPTQ_E_INVALID_ARG;
  if (rope && (st = check_rope(rope, cache->head_dim)) != GPTQ_OK) return st;
  if (q && (!rope || !q_out)) return GPTQ_E_INVALID_ARG;
  if (q && (q_heads < 1 || q_heads > 65536)) return GPTQ_E_SHAPE;
  if (batch->rows == 0 || batch->batch == 0) return GPTQ_OK;
  const int64_t kv_width = (int64_t)cache->kv_heads * cache->head_dim, q_width = (int64_t)q_heads * cache->head_dim;
  if (!kv_append_fits(*cache, *batch, q ? q_heads : 0)) return GPTQ_E_SHAPE;
  if ((st = check_rows(k, kv_width, k_stride)) != GPTQ_OK) return st;
  if ((st = check_rows(v, kv_width, v_stride)) != GPTQ_OK) return st;
  const size_t kb = row_bytes(batch->rows, kv_width, k_stride), vb = row_bytes(batch->rows, kv_width, v_stride);
  if (overlaps_cache(cache, k, kb) || overlaps_cache(cache, v, vb)) return GPTQ_E_INVALID_ARG;
  if (q) {
    if ((st = check_rows(q, q_width, q_stride)) != GPTQ_OK) return st;
    if ((st = check_rows(q_out, q_width, q_out_stride)) != GPTQ_OK) return st;
    const size_t ob = row_bytes(batch->rows, q_width, q_out_stride);
    const int64_t rows = batch->rows;
    const bool in_place = q_out == q && q_out_stride == q_stride;
    if ((!in_place && rows_overlap(q, q_width, q_stride, q_out, q_width, q_out_stride, rows)) ||
        rows_overlap(k, kv_width, k_stride, q_out, q_width, q_out_stride, rows) ||
        rows_overlap(v, kv_width, v_stride, q_out, q_width, q_out_stride, rows))
      return GPTQ_E_INVALID_ARG;
    const size_t turns = (size_t)rope->rows * (rope->dim / 2) * 4;
    if (overlaps_cache(cache, q_out, ob) || overlaps_tables(batch, q_out, ob) || overlaps(q_out, ob, rope->cos, turns) ||
        overlaps(q_out, ob, rope->sin, turns))
      return GPTQ_E_INVALID_ARG;
  }
  if ((st = check_device()) != GPTQ_OK) return st;
  KvAppendCall a{};
  a.c = *cache;
  a.b = *batch;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.q = (const uint16_t*)q;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.q_out = (uint16_t*)q_out;
  a.q_heads = q ? q_heads : 0;
  a.bf16 = dtype == GPTQ_BF16;
  if (rope) a.rope = *rope;
  const hipError_t e = launch_kv_append(a, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

gptq_status gptq_kv_read(const gptq_kv_cache* cache, const gptq_kv_batch* batch, void* k_out, void* v_out, int32_t dtype,
                         void* stream) {
  gptq_status st = check_cache(cache);
  if (st == GPTQ_OK) st = check_batch(batch);
  if (st != GPTQ_OK) return st;
  if (!is_16bit(dtype) && dtype != GPTQ_F32) return GPTQ_E_INVALID_ARG;
  if (batch->rows == 0 || batch->batch == 0) return GPTQ_OK;
  if (!kv_read_fits(*cache, *batch)) return GPTQ_E_SHAPE;
  if (!k_out && !v_out) return GPTQ_E_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return GPTQ_E_INVALID_ARG;
  const size_t n = (size_t)batch->rows * cache->kv_heads * cache->head_dim * (dtype == GPTQ_F32 ? 4 : 2);
  if (overlaps(k_out, n, v_out, n) || overlaps_cache(cache, k_out, n) || overlaps_cache(cache, v_out, n) ||
      overlaps_tables(batch, k_out, n) || overlaps_tables(batch, v_out, n))
    return GPTQ_E_INVALID_ARG;
  if ((st = check_device()) != GPTQ_OK) return st;
  const hipError_t e = launch_kv_read(*cache, *batch, k_out, v_out, dtype, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

gptq_status gptq_kv_attention_workspace_size(const gptq_kv_cache* cache, const gptq_kv_batch* batch,
                                             const gptq_attention* call, size_t* bytes) {
  if (!bytes) return GPTQ_E_INVALID_ARG;
  const gptq_status st = check_attention(cache, batch, call);
  if (st != GPTQ_OK) return st;
  if (!no_queries(*batch) && !kv_attention_fits(*cache, *batch, *call)) return GPTQ_E_SHAPE;
  *bytes = no_queries(*batch) ? 0 : kv_attention_ws_bytes(*cache, *batch, *call);
  return GPTQ_OK;
}

gptq_status gptq_kv_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const gptq_attention* call,
                              const void* q, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  gptq_status st = check_attention(cache, batch, call);
  if (st != GPTQ_OK) return st;
  if (no_queries(*batch)) return GPTQ_OK;
  if (!kv_attention_fits(*cache, *batch, *call)) return GPTQ_E_SHAPE;
  const int64_t width = (int64_t)call->q_heads * cache->head_dim;
  if ((st = check_rows(q, width, call->q_stride)) != GPTQ_OK) return st;
  if ((st = check_rows(out, width, call->out_stride)) != GPTQ_OK) return st;
  const size_t qb = row_bytes(batch->rows, width, call->q_stride), ob = row_bytes(batch->rows, width, call->out_stride);
  if (rows_overlap(q, width, call->q_stride, out, width, call->out_stride, batch->rows) ||
      overlaps_cache(cache, out, ob) || overlaps_tables(batch, out, ob))
    return GPTQ_E_INVALID_ARG;
  const size_t need = kv_attention_ws_bytes(*cache, *batch, *call);
  if (need > 0) {
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return GPTQ_E_WORKSPACE;
    if (overlaps(workspace, need, q, qb) || overlaps(workspace, need, out, ob) || overlaps_cache(cache, workspace, need) ||
        overlaps_tables(batch, workspace, need))
      return GPTQ_E_INVALID_ARG;
  }
  if ((st = check_device()) != GPTQ_OK) return st;
  const KvAttentionCall a{*cache, *batch, *call, (const uint16_t*)q, (uint16_t*)out, workspace};
  const hipError_t e = few_rows(*cache, *batch, *call) ? launch_kv_decode(a, (hipStream_t)stream)
                                                       : launch_kv_prefill(a, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

gptq_status gptq_lora_workspace_size(const gptq_lora_bank* bank, int64_t M, size_t* bytes) {
  if (!bytes) return GPTQ_E_INVALID_ARG;
  const gptq_status st = check_bank(bank, M);
  if (st != GPTQ_OK) return st;
  if (M > 0 && !lora_fits(*bank, M)) return GPTQ_E_SHAPE;
  *bytes = M == 0 ? 0 : lora_ws_bytes(*bank, M);
  return GPTQ_OK;
}

gptq_status gptq_lora_add(const gptq_lora_bank* bank, const void* x, const void* y, const int32_t* ids, int64_t M,
                          void* out, void* workspace, size_t workspace_bytes, void* stream) {
  gptq_status st = check_bank(bank, M);
  if (st != GPTQ_OK) return st;
  if (!bank->a || !bank->b || !bank->scale || !aligned(bank->a, 16) || !aligned(bank->b, 16) || !aligned(bank->scale, 4))
    return GPTQ_E_INVALID_ARG;
  if (M == 0) return GPTQ_OK;
  if (!lora_fits(*bank, M)) return GPTQ_E_SHAPE;
  if (!x || !y || !out || !ids || !aligned(x, 16) || !aligned(y, 16) || !aligned(out, 16) || !aligned(ids, 4))
    return GPTQ_E_INVALID_ARG;
  const size_t xb = (size_t)M * bank->in_features * 2, yb = (size_t)M * bank->out_features * 2;
  const size_t ab = (size_t)bank->adapters * bank->rank * bank->in_features * 2;
  const size_t bb = (size_t)bank->adapters * bank->rank * bank->out_features * 2;
  if (overlaps(out, yb, x, xb) || (out != y && overlaps(out, yb, y, yb)) || overlaps(out, yb, bank->a, ab) ||
      overlaps(out, yb, bank->b, bb) || overlaps(out, yb, ids, (size_t)M * 4) ||
      overlaps(out, yb, bank->scale, (size_t)bank->adapters * 4))
    return GPTQ_E_INVALID_ARG;
  const size_t need = lora_ws_bytes(*bank, M);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return GPTQ_E_WORKSPACE;
  if (overlaps(workspace, need, x, xb) || overlaps(workspace, need, y, yb) || overlaps(workspace, need, out, yb) ||
      overlaps(workspace, need, bank->a, ab) || overlaps(workspace, need, bank->b, bb) ||
      overlaps(workspace, need, ids, (size_t)M * 4) || overlaps(workspace, need, bank->scale, (size_t)bank->adapters * 4))
    return GPTQ_E_INVALID_ARG;
  if ((st = check_device()) != GPTQ_OK) return st;
  const LoraCall c{*bank, (const uint16_t*)x, (const uint16_t*)y, ids, M, (uint16_t*)out, workspace};
  const hipError_t e = launch_lora(c, (hipStream_t)stream);
  return e == hipSuccess ? GPTQ_OK : hip_fail(e);
}

}  // extern "C"
