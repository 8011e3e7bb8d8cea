// Appending rotated keys and values to the paged 8-bit cache, and reading tokens back.
//
// Mathematics, for each page and head that gets tokens (gptq_mi355x.h, gptq_kv_append): the scale of
// the page is the largest |x| / 127 that it has seen, so appending is a maximum over the page's new
// values, a rescale of the codes already there when that maximum grew, and one rounding of the new
// values.  Products and differences of the rotation are rounded one by one (no fused multiply-add),
// so the codes do not depend on how a compiler contracts them.
//
// Split: one workgroup for each touched page, head and half (key or value), with all of the page's
// new values in registers between the maximum and the rounding, so every value is read once.  The
// queries' rotation runs in further workgroups of the same launch, one wave for each 512 values of
// a token.  Touched pages are numbered without a plan: sequence b gets the slots from
// cu[b] / page + 2 b on, which are never fewer than the pages that its rows touch.
//
// What bounds it: bytes (new rows in, rotated queries in and out, touched pages' codes out, their older
// codes in too); a token a request: the launch.  Measured (the device's time): 64 requests, one token each,
// 32 + 8 heads of 128: 5.0 us; 5011 tokens of 7 prompts, 64 + 8 heads, 96 MB: 22.1 us, 4.3 TB/s of the 4.9
// that a large copy reaches; reading 5 MB of codes back as 10 MB of float16: 5.5 us.
#include <hip/hip_runtime.h>

#include "serving.h"
#include "serving_dev.h"

namespace gq {
namespace {

constexpr int kThreads = 256;      // of a read; an append takes 1024 for pages of over 8192 values

// Index of the first page slot of sequence b (a call of at most one row a sequence: slot b).
__device__ __forceinline__ int64_t slot_edge(const gptq_kv_batch& b, int seq, int page_shift) {
  return ((int64_t)b.cu[seq] >> page_shift) + 2 * (int64_t)seq;
}

// Eight values at `at`.
template <int BF16>
__device__ __forceinline__ void load8(const uint16_t* at, float* x) {
  const u32x4 w = *(const u32x4*)at;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = to_f32<BF16>((uint16_t)w[i]);
    x[2 * i + 1] = to_f32<BF16>((uint16_t)(w[i] >> 16));
  }
}

// The eight values [d, d + 8) of a head at `head`, rotated at table row `pos`.
template <int BF16>
__device__ __forceinline__ void rotated8(const uint16_t* head, int d, int64_t pos, const gptq_rope& r, float* x) {
#pragma clang fp contract(off)
  load8<BF16>(head + d, x);
  if (d >= r.dim) return;
  const int half = r.dim >> 1;
  const int64_t row = pos < r.rows ? pos : r.rows - 1;
  if (r.interleaved) {
    const float* c = r.cos + row * half + (d >> 1);
    const float* s = r.sin + row * half + (d >> 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
    }
  } else {
    const bool low = d < half;
    const int i0 = low ? d : d - half;
    float y[8];
    load8<BF16>(head + (low ? d + half : d - half), y);
    const float* c = r.cos + row * half + i0;
    const float* s = r.sin + row * half + i0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = y[i] * s[i], own = x[i] * c[i];
      x[i] = low ? own - t : own + t;
    }
  }
}

// |x| of a finite value, else 0: infinities and NaN do not set a page's scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = __builtin_fabsf(x);
  return a < __builtin_inff() ? a : 0.0f;
}

// The code of a value: rint(x / unit) within [-127, 127], NaN (also 0 * inf) 0.
__device__ __forceinline__ int code_of(float x, float inverse) {
  const float c = __builtin_rintf(x * inverse);
  const float in = __builtin_fminf(__builtin_fmaxf(c, -127.0f), 127.0f);
  return c == c ? (int)in : 0;
}

template <int BF16, int CHUNKS, int DIM, int THREADS>
__device__ __forceinline__ void append_page(const KvAppendCall& a, int slot, int head, bool value, int page_shift,
                                            float* most_of_wave) {
  const gptq_kv_batch& b = a.b;
  const int page_size = 1 << page_shift;
  int seq, nth;
  if (b.max_rows == 1) {
    seq = slot;
    nth = 0;
  } else {
    seq = find_sequence(b.batch, slot, [&](int i) { return slot_edge(b, i, page_shift); });
    nth = (int)(slot - slot_edge(b, seq, page_shift));
  }
  const int64_t row0 = b.cu[seq], row1 = b.cu[seq + 1];
  int64_t rows = row1 - row0;
  if (rows > b.max_rows) rows = b.max_rows;
  const int64_t start = b.at[seq];
  if (rows <= 0 || row0 < 0 || row0 + rows > b.rows || start < 0 || nth < 0) return;
  const int64_t j = (start >> page_shift) + nth;
  const int64_t base = j << page_shift;                       // position of the page's first token
  if (base >= start + rows || j >= b.table_width) return;
  const int64_t page = b.page_table[(int64_t)seq * b.table_width + j];
  if (page < 0 || page >= a.c.num_pages) return;

  const uint16_t* src = value ? a.v : a.k;
  const int64_t stride = value ? a.v_stride : a.k_stride;
  const int64_t unit_at = page * a.c.kv_heads + head;
  float* scale = (value ? a.c.v_scale : a.c.k_scale) + unit_at;
  int8_t* codes = (value ? a.c.v_codes : a.c.k_codes) + unit_at * page_size * DIM;

  constexpr int kRow = DIM / 8;                               // chunks of eight values in a row
  float x[CHUNKS][8];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int chunk = i * THREADS + threadIdx.x;
    const int64_t pos = base + chunk / kRow;
    const bool fresh = chunk < page_size * kRow && pos >= start && pos < start + rows;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
    if (fresh) {
      const uint16_t* at = src + (row0 + pos - start) * stride + head * DIM;
      if (value) load8<BF16>(at + (chunk % kRow) * 8, x[i]);
      else rotated8<BF16>(at, (chunk % kRow) * 8, pos, a.rope, x[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) most = __builtin_fmaxf(most, finite_abs(x[i][e]));
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, d));
  if ((threadIdx.x & 63) == 0) most_of_wave[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) most = __builtin_fmaxf(most, most_of_wave[i]);
  const float had = base < start ? *scale : 0.0f;
  const float unit = __builtin_fmaxf(had, most * (1.0f / 127.0f));
  // below 2^-128 the inverse would be infinite: there the page's values, exactly, times 2^64
  const bool tiny = unit < 0x1p-100f;
  const float up = tiny ? 0x1p64f : 1.0f;
  const float inverse = unit > 0.0f ? 1.0f / (unit * up) : 0.0f;
  const float ratio = had * up * inverse;
  if (tiny) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= up;
  }
  __syncthreads();                                            // every thread has read the old scale
  if (threadIdx.x == 0) *scale = unit;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int chunk = i * THREADS + threadIdx.x;
    const int64_t pos = base + chunk / kRow;
    if (chunk >= page_size * kRow || pos >= start + rows) continue;
    uint2* at = (uint2*)(codes + chunk * 8);
    int c[8];
    if (pos >= start) {
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = code_of(x[i][e], inverse);
    } else {
      if (!(unit > had)) continue;
      const uint2 w = *at;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int old = (int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
        c[e] = (int)__builtin_rintf((float)old * ratio);
      }
    }
    uint2 w{0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) (e < 4 ? w.x : w.y) |= (uint32_t)(c[e] & 255) << (8 * (e & 3));
    *at = w;
  }
}

template <int BF16, int CHUNKS, int DIM, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(KvAppendCall a, int page_blocks, int slots, int page_shift,
                                                             int waves_per_row) {
  __shared__ float most_of_wave[THREADS / 64];
  if ((int)blockIdx.x < page_blocks) {
    const int block = blockIdx.x;
    const int slot = block / (2 * a.c.kv_heads), rest = block % (2 * a.c.kv_heads);
    append_page<BF16, CHUNKS, DIM, THREADS>(a, slot, rest >> 1, rest & 1, page_shift, most_of_wave);
    return;
  }
  // rotate the queries: one wave for 512 values of a token
  const int64_t wave = (int64_t)(blockIdx.x - page_blocks) * (THREADS / 64) + (threadIdx.x >> 6);
  const int64_t row = wave / waves_per_row;
  if (row >= a.b.rows) return;
  const int seq = find_sequence(a.b.batch, row, [&](int i) { return (int64_t)a.b.cu[i]; });
  const int chunk = (int)(wave % waves_per_row) * 64 + (threadIdx.x & 63);
  if (chunk >= a.q_heads * (DIM / 8)) return;
  int64_t pos = a.b.at[seq] + row - a.b.cu[seq];
  if (pos < 0) pos = 0;
  const int head = chunk / (DIM / 8), d = chunk % (DIM / 8) * 8;
  float x[8];
  rotated8<BF16>(a.q + row * a.q_stride + head * DIM, d, pos, a.rope, x);
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)from_f32<BF16>(x[2 * i]) | (uint32_t)from_f32<BF16>(x[2 * i + 1]) << 16;
  *(u32x4*)(a.q_out + row * a.q_out_stride + head * DIM + d) = w;
}

// One wave for 512 values of a token's keys or values.
template <int OUT>   // gptq_dtype
__global__ void __launch_bounds__(kThreads) kv_read_kernel(gptq_kv_cache c, gptq_kv_batch b, void* k_out, void* v_out,
                                                           int page_shift, int waves_per_row) {
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t row = wave / waves_per_row;
  if (row >= b.rows) return;
  const int seq = find_sequence(b.batch, row, [&](int i) { return (int64_t)b.cu[i]; });
  const int per_head = c.head_dim / 8;
  const int chunk = (int)(wave % waves_per_row) * 64 + (threadIdx.x & 63);
  if (chunk >= c.kv_heads * per_head) return;
  const int head = chunk / per_head, d = chunk % per_head * 8;
  const int64_t place = row - b.cu[seq], pos = b.at[seq] + place, j = pos >> page_shift;
  int64_t page = -1;
  if (pos >= 0 && place >= 0 && place < b.max_rows && j < b.table_width)
    page = b.page_table[(int64_t)seq * b.table_width + j];
  const bool there = page >= 0 && page < c.num_pages;
  const int64_t unit = there ? page * c.kv_heads + head : 0;
  const int64_t at = ((unit << page_shift) + (pos & ((1 << page_shift) - 1))) * c.head_dim + d;
  const int64_t to = (row * c.kv_heads + head) * c.head_dim + d;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    void* out = half ? v_out : k_out;
    if (!out) continue;
    uint2 w{0, 0};
    float s = 0.0f;
    if (there) {
      w = *(const uint2*)((half ? c.v_codes : c.k_codes) + at);
      s = (half ? c.v_scale : c.k_scale)[unit];
    }
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = there ? (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * s : 0.0f;
      asm("" : "+v"(x[e]));   // the value is the float32 product: keep it from a product rounded straight to float16
    }
    if constexpr (OUT == GPTQ_F32) {
      float4* o = (float4*)((float*)out + to);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = (uint32_t)from_f32<OUT == GPTQ_BF16>(x[2 * i]) | (uint32_t)from_f32<OUT == GPTQ_BF16>(x[2 * i + 1]) << 16;
      *(u32x4*)((uint16_t*)out + to) = o;
    }
  }
}

struct AppendGrid {
  int64_t slots, page_blocks, blocks;
  int chunks, threads, waves_per_row;
};
AppendGrid append_grid(const gptq_kv_cache& c, const gptq_kv_batch& b, int q_heads) {
  AppendGrid g;
  const int page_shift = __builtin_ctz(c.page_size);
  // slots of every sequence: its rows / page, rounded down, and two
  g.slots = b.max_rows == 1 ? b.batch : (b.rows >> page_shift) + 2 * (int64_t)b.batch;
  g.page_blocks = g.slots * c.kv_heads * 2;
  g.waves_per_row = (q_heads * (c.head_dim / 8) + 63) / 64;
  g.chunks = (c.head_dim / 8) << page_shift;
  g.threads = g.chunks > 1024 ? 1024 : 256;
  g.blocks = g.page_blocks + (b.rows * g.waves_per_row + g.threads / 64 - 1) / (g.threads / 64);
  return g;
}

template <int BF16, int DIM>
hipError_t launch_append_dim(const KvAppendCall& a, int page_shift, hipStream_t s) {
  const AppendGrid g = append_grid(a.c, a.b, a.q_heads);
  const int chunks = g.chunks;
#define GQ_APPEND(C, T)                                                                                            \
  kv_append_kernel<BF16, C, DIM, T><<<dim3((uint32_t)g.blocks), dim3(T), 0, s>>>(a, (int)g.page_blocks, (int)g.slots, \
                                                                                 page_shift, g.waves_per_row)
  if (g.threads == 1024) {
    if (chunks <= 2048) GQ_APPEND(2, 1024);
    else GQ_APPEND(4, 1024);
  } else if (chunks <= 256) {
    GQ_APPEND(1, 256);
  } else if (chunks <= 512) {
    GQ_APPEND(2, 256);
  } else {
    GQ_APPEND(4, 256);
  }
#undef GQ_APPEND
  return hipGetLastError();
}

int read_waves_per_row(const gptq_kv_cache& c) { return (c.kv_heads * (c.head_dim / 8) + 63) / 64; }
int64_t read_blocks(const gptq_kv_cache& c, const gptq_kv_batch& b) {
  return (b.rows * read_waves_per_row(c) + kThreads / 64 - 1) / (kThreads / 64);
}

}  // namespace

bool kv_append_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, int q_heads) {
  const AppendGrid g = append_grid(c, b, q_heads);
  return grid_fits(g.blocks, g.threads);
}

bool kv_read_fits(const gptq_kv_cache& c, const gptq_kv_batch& b) { return grid_fits(read_blocks(c, b), kThreads); }

hipError_t launch_kv_append(const KvAppendCall& a, hipStream_t s) {
  const int page_shift = __builtin_ctz(a.c.page_size);
  if (a.c.head_dim == 128)
    return a.bf16 ? launch_append_dim<1, 128>(a, page_shift, s) : launch_append_dim<0, 128>(a, page_shift, s);
  return a.bf16 ? launch_append_dim<1, 64>(a, page_shift, s) : launch_append_dim<0, 64>(a, page_shift, s);
}

hipError_t launch_kv_read(const gptq_kv_cache& c, const gptq_kv_batch& b, void* k_out, void* v_out, int dtype,
                          hipStream_t s) {
  const int page_shift = __builtin_ctz(c.page_size);
  const int waves_per_row = read_waves_per_row(c);
  const dim3 grid((uint32_t)read_blocks(c, b)), block(kThreads);
  if (dtype == GPTQ_F16) kv_read_kernel<GPTQ_F16><<<grid, block, 0, s>>>(c, b, k_out, v_out, page_shift, waves_per_row);
  else if (dtype == GPTQ_BF16) kv_read_kernel<GPTQ_BF16><<<grid, block, 0, s>>>(c, b, k_out, v_out, page_shift, waves_per_row);
  else kv_read_kernel<GPTQ_F32><<<grid, block, 0, s>>>(c, b, k_out, v_out, page_shift, waves_per_row);
  return hipGetLastError();
}

}  // namespace gq
