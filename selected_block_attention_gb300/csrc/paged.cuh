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

// Every paged kernel is launched so that it may be set up while the kernel before it ends,
// and begins with this wait: nothing that kernel wrote is read earlier.
__device__ __forceinline__ void paged_wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A kernel with a second one behind it lets that one be set up as well.
__device__ __forceinline__ void paged_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class Params>
cudaError_t paged_launch(void (*kernel)(Params), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         const Params& p, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
// Raises a kernel's dynamic shared memory limit, once for each device that a thread uses.
template <class Kernel>
cudaError_t paged_allow_smem(Kernel kernel, size_t bytes, unsigned long long* devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && ((*devices >> dev) & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) *devices |= 1ull << dev;
  return e;
}

__device__ __forceinline__ void paged_cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void paged_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void paged_cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 paged_lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void paged_sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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
