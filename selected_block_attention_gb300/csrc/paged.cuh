// Shared pieces of the paged-cache kernels: the view of a cache, page lookups and the
// conversions between e4m3, fp16, bf16 and fp32.
//
// A cache is two pools of pages, [num_pages, Hkv, P, D] (each (page, head) tile is one
// contiguous run of P rows), a table [B, width] naming each row's pages in order, and the
// rows' lengths.  An e4m3 pool has one fp32 scale per (page, head): value = code * scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "ptx.cuh"

namespace sba {

struct PagedView {
  uint8_t* k;  // pools, by bytes
  uint8_t* v;
  float* ks;  // [num_pages, Hkv] scales (e4m3), else null
  float* vs;
  const int* table;  // [B, width]
  const int* lens;   // [B] lengths, the call's own tokens included
  const int* cu;     // [B + 1] token offsets of the rows, or null: Qn tokens per row
  long long page_bytes;  // distance between pages
  int B, Qn, N;          // rows, tokens per row (cu == null), tokens in all
  int width, num_pages, p_shift, Hkv;
};

// The tokens of row b, clamped so that every index stays inside the call's arrays;
// *bad reports input that is not what the caller promised.
struct PagedRow {
  int t0, n, len;  // first token, number of tokens, length
};
__device__ __forceinline__ PagedRow paged_row(const PagedView& c, int b, bool* bad) {
  PagedRow r;
  const int len = c.lens[b];
  const long long room = (long long)c.width << c.p_shift;
  r.len = (int)min((long long)max(len, 0), room);
  *bad = len < 0 || len > room;
  if (c.cu == nullptr) {
    r.t0 = b * c.Qn;
    r.n = c.Qn;
  } else {
    const int a = c.cu[b], e = c.cu[b + 1];
    r.t0 = min(max(a, 0), c.N);
    const int t1 = min(max(e, r.t0), c.N);
    r.n = t1 - r.t0;
    *bad = *bad || a < 0 || e < a || e > c.N;
  }
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two_codes));
  return r;
}
// Both halves of a word of four codes.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
// Round to nearest (ties to even), magnitudes over 448 and infinities to 448, NaN kept.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t two) { return __uint_as_float(two & 0xFFFF0000u); }

}  // namespace sba
