// What the kernels that write the paged 8-bit cache share.
#pragma once
#include <cuda_bf16.h>

#include "internal.h"
#include "rotation.cuh"

namespace gb300 {

namespace {

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  const int* table;
  const int* start;
  const int* lens;
  const int* tok_start;
  int64_t tokens, token_stride, row_tokens, page_stride, units;
  int num_pages, h_kv, page_size, max_pages, max_new, pages_per_seq;
};

// Two e4m3 codes of two fp32 values (round to nearest even, saturating; NaN
// stays NaN): lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two fp32 values of two e4m3 codes (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h2));
  return f;
}

// max(m, |both|) over the values that are finite
__device__ __forceinline__ float amax_finite(float m, uint32_t w) {
  const float2 f = widen_bf16x2(w);
  const float a = fabsf(f.x), b = fabsf(f.y);
  if (a < INFINITY) m = fmaxf(m, a);
  if (b < INFINITY) m = fmaxf(m, b);
  return m;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Exponent k of the smallest power of two with amax <= 448 * 2^k (448 = 1.75 *
// 2^8, so the exponent less 8, and one more above a mantissa of 1.75), no less
// than -126.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, -126);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

inline AppendArgs append_args(const attn_kv_append_params& p) {
  const attn_kv_cache& c = p.cache;
  AppendArgs a;
  a.k = static_cast<const __nv_bfloat16*>(p.k);
  a.v = static_cast<const __nv_bfloat16*>(p.v);
  a.kc = static_cast<uint8_t*>(c.k);
  a.vc = static_cast<uint8_t*>(c.v);
  a.ks = c.k_scale;
  a.vs = c.v_scale;
  a.table = p.page_table;
  a.start = p.start;
  a.lens = p.lens;
  a.tok_start = p.tok_start;
  a.tokens = p.tokens;
  a.token_stride = p.token_stride > 0 ? p.token_stride : c.h_kv * c.d;
  a.row_tokens = p.row_tokens;
  a.page_stride = c.page_stride > 0 ? c.page_stride : c.h_kv * c.page_size * c.d;
  a.num_pages = (int)c.num_pages;
  a.h_kv = (int)c.h_kv;
  a.page_size = (int)c.page_size;
  a.max_pages = (int)p.max_pages;
  a.max_new = (int)p.max_new;
  // most pages that max_new tokens in a row can touch
  int64_t pages = (p.max_new + c.page_size - 2) / c.page_size + 1;
  if (pages > p.max_pages) pages = p.max_pages;
  a.pages_per_seq = (int)pages;
  a.units = p.n * pages * 2 * c.h_kv;
  return a;
}

}  // namespace

}  // namespace gb300
