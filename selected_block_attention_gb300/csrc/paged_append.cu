// New keys and values into a paged cache, keys and queries rotated by their positions on
// the way: paged_append_kernel.
//
// Row b's last n_b tokens are new; token i sits at pos = len_b - n_b + i, in page
// table[b, pos / P] at offset pos % P.  With x the token's key (or query) in fp32 and
// (c, s) = (cos, sin)[pos], dimension pairs (x0, x1) of the first `rot` dimensions become
// (x0 c - x1 s, x1 c + x0 s); the products and the sum are rounded one by one, so the
// result does not depend on how the compiler contracts them.  A bf16 cache stores the
// rounded result.  An e4m3 cache has one scale for each page and head, a power of two:
//
//   need  = the least 2^e >= amax / 448 over the call's finite values in that page
//   scale = need when the call writes the page's first slot, else max(old scale, need)
//   code  = e4m3(x / scale), to nearest
//
// When a page's scale grows, the codes that it already holds are taken to the new scale;
// since both are powers of two that moves their exponents and loses bits only of values
// that become subnormal, so a page filled token by token ends within half a subnormal
// step of the same page filled at once.
//
// Work unit: one page of one row, for one head of K, V or Q: its maximum is all that the
// scale needs, so a unit is one block (or one warp) and nothing waits for another.  The
// kernel is bound by memory: every input is read once and held in registers between the
// maximum and the store.
#include <string>

#include "paged.cuh"

namespace sba {

static __device__ unsigned g_err_append = 0;

namespace {

struct AppendParams {
  PagedView c;
  const __nv_bfloat16* k;  // [tokens, Hkv, D], k_tok elements between tokens
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;  // [tokens, Hq, D] or null
  __nv_bfloat16* q_out;
  const float* cosp;  // [max_pos, rot / 2] or null
  const float* sinp;
  long long k_tok, v_tok, q_tok, qo_tok;
  int Hq, rot, interleaved, max_pos;
  int units_per_row;  // pages a row's tokens can touch (cu == null)
};

// x[0..8) and y[0..8): the thread's two chunks of 8 dimensions.  Half-split pairs are
// (x[i], y[i]); neighbouring pairs lie inside each chunk.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float a2 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float b2 = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = a2;
  b = b2;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint4 w;
  w.x = pack_bf16x2(x[0], x[1]); w.y = pack_bf16x2(x[2], x[3]);
  w.z = pack_bf16x2(x[4], x[5]); w.w = pack_bf16x2(x[6], x[7]);
  *reinterpret_cast<uint4*>(p) = w;
}

// Least power of two s >= 2^-126 with 448 s >= amax (amax finite, >= 0).
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  e = max(e, -126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// kUnit threads work on one unit; a row (token) takes kD / 16 of them, each with two
// chunks of 8 dimensions; kPasses passes cover the unit's rows.
template <bool kF8, int kD, int kUnit, int kPasses>
__global__ void __launch_bounds__(kUnit == 32 ? 128 : 256)
paged_append_kernel(const AppendParams p) {
  constexpr int kRowThreads = kD / 16;
  constexpr int kRows = kUnit / kRowThreads;
  const PagedView& c = p.c;
  const int tid = kUnit == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int stream = kUnit == 32 ? blockIdx.y * 4 + (threadIdx.x >> 5) : blockIdx.y;
  const int streams = p.Hq + 2 * c.Hkv;
  const int P = 1 << c.p_shift;

  // ---- the unit: page number j of row b's new tokens
  int b, j;
  if (c.cu == nullptr) {
    b = blockIdx.x / p.units_per_row;
    j = blockIdx.x - b * p.units_per_row;
  } else {
    // Row b owns units from floor(cu[b] / P) + 2 b on: n tokens touch at most
    // floor(n / P) + 2 pages, and floor is superadditive, so rows never overlap.
    __shared__ int s_b;
    if (threadIdx.x == 0) s_b = -1;
    __syncthreads();
    const int u = blockIdx.x;
    for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
      const int lo = (min(max(c.cu[i], 0), c.N) >> c.p_shift) + 2 * i;
      const int hi = (min(max(c.cu[i + 1], 0), c.N) >> c.p_shift) + 2 * i + 2;
      if (u >= lo && u < hi) s_b = i;
    }
    __syncthreads();
    b = s_b;
    if (b < 0) return;
    j = u - (min(max(c.cu[b], 0), c.N) >> c.p_shift) - 2 * b;
  }
  if (stream >= streams) return;
  bool bad;
  const PagedRow r = paged_row(c, b, &bad);
  if (bad) {
    if (tid == 0) atomicOr(&g_err_append, (unsigned)kDevErrInput);
    return;
  }
  const int start = r.len - r.n;  // position of the row's first token; those left of 0 do not exist
  const int pj = (max(start, 0) >> c.p_shift) + j;
  const int p0 = max(max(start, 0), pj << c.p_shift);
  const int p1 = min(r.len, (pj + 1) << c.p_shift);
  const int m = p1 - p0;
  if (r.n == 0 || m <= 0) return;

  // ---- the stream: a query head, a key head or a value head
  const bool is_q = stream < p.Hq;
  const bool is_k = !is_q && stream < p.Hq + c.Hkv;
  const int h = is_q ? stream : (is_k ? stream - p.Hq : stream - p.Hq - c.Hkv);
  const __nv_bfloat16* src = is_q ? p.q : (is_k ? p.k : p.v);
  const long long tok = is_q ? p.q_tok : (is_k ? p.k_tok : p.v_tok);
  const int first = r.t0 + (p0 - start);  // token at position p0
  const int rot = (is_q || is_k) ? p.rot : 0;
  int page = 0;
  if (!is_q) {
    page = c.table[(long long)b * c.width + pj];
    if ((unsigned)page >= (unsigned)c.num_pages) {
      if (tid == 0) atomicOr(&g_err_append, (unsigned)kDevErrInput);
      return;
    }
  }

  const int rt = tid % kRowThreads, slot = tid / kRowThreads;
  // rotated dimensions first, a chunk with its partner; then the rest two by two
  int c0, c1;
  const bool turn = rt < rot / 16;
  if (turn && !p.interleaved) {
    c0 = rt;
    c1 = rt + rot / 16;
  } else {
    c0 = 2 * rt;
    c1 = 2 * rt + 1;
  }
  float x[kPasses][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = i * kRows + slot;
    if (row >= m) continue;
    const __nv_bfloat16* s = src + (long long)(first + row) * tok + (long long)h * kD;
    load8(s + 8 * c0, x[i]);
    load8(s + 8 * c1, x[i] + 8);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = i * kRows + slot;
    if (row >= m) continue;
    if (turn) {
      int pos = p0 + row;
      if (pos >= p.max_pos) {
        atomicOr(&g_err_append, (unsigned)kDevErrInput);
        pos = p.max_pos - 1;
      }
      // 8 angles: of pairs 8 c0 .. 8 c0 + 7 (half split) or of the 16 neighbours
      const float4* cp = reinterpret_cast<const float4*>(p.cosp + (long long)pos * (rot / 2) + 8 * rt);
      const float4* sp = reinterpret_cast<const float4*>(p.sinp + (long long)pos * (rot / 2) + 8 * rt);
      const float4 ca = __ldg(cp), cb = __ldg(cp + 1), sa = __ldg(sp), sb = __ldg(sp + 1);
      const float cs[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
      const float sn[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate_pair(x[i][2 * e], x[i][2 * e + 1], cs[e], sn[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate_pair(x[i][e], x[i][e + 8], cs[e], sn[e]);
      }
    }
    if (kF8 && !is_q) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = fabsf(x[i][e]);
        if (a <= 3.4028235e38f) amax = fmaxf(amax, a);  // infinities and NaN set no scale
      }
    }
  }

  if (is_q) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = i * kRows + slot;
      if (row >= m) continue;
      __nv_bfloat16* o = p.q_out + (long long)(first + row) * p.qo_tok + (long long)h * kD;
      store8(o + 8 * c0, x[i]);
      store8(o + 8 * c1, x[i] + 8);
    }
    return;
  }
  const int off = p0 & (P - 1);
  uint8_t* tile = (is_k ? c.k : c.v) + page * c.page_bytes + (long long)h * P * (kD * (kF8 ? 1 : 2));
  if constexpr (!kF8) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = i * kRows + slot;
      if (row >= m) continue;
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(tile) + (off + row) * kD;
      store8(o + 8 * c0, x[i]);
      store8(o + 8 * c1, x[i] + 8);
    }
    return;
  } else {
    float* scale_at = (is_k ? c.ks : c.vs) + (long long)page * c.Hkv + h;
    const float old = off > 0 ? *scale_at : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if constexpr (kUnit > 32) {
      __shared__ float s_max[kUnit / 32];
      if ((tid & 31) == 0) s_max[tid >> 5] = amax;
      __syncthreads();
      amax = s_max[0];
#pragma unroll
      for (int w = 1; w < kUnit / 32; ++w) amax = fmaxf(amax, s_max[w]);
    } else {
      __syncwarp();
    }
    const float need = pow2_scale(amax);
    const float scale = need > old ? need : old;
    const float inv = __frcp_rn(scale);
    if (scale != old) {
      if (tid == 0) *scale_at = scale;  // every thread has read the old one
      // codes that the page holds already, to the new scale
      for (int row = slot; row < off; row += kRows) {
        uint2* at = reinterpret_cast<uint2*>(tile + row * kD + 16 * rt);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint2 w = at[half];
          uint2 o;
          float f[8];
          uint32_t lo, hi;
          e4m3x4_to_f16x2(w.x, lo, hi);
          float2 t = __half22float2(*reinterpret_cast<__half2*>(&lo));
          f[0] = t.x; f[1] = t.y;
          t = __half22float2(*reinterpret_cast<__half2*>(&hi));
          f[2] = t.x; f[3] = t.y;
          e4m3x4_to_f16x2(w.y, lo, hi);
          t = __half22float2(*reinterpret_cast<__half2*>(&lo));
          f[4] = t.x; f[5] = t.y;
          t = __half22float2(*reinterpret_cast<__half2*>(&hi));
          f[6] = t.x; f[7] = t.y;
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(__fmul_rn(f[e], old), inv);
          o.x = f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]);
          o.y = f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]);
          at[half] = o;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = i * kRows + slot;
      if (row >= m) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) x[i][e] = __fmul_rn(x[i][e], inv);
      uint8_t* o = tile + (off + row) * kD;
      *reinterpret_cast<uint2*>(o + 8 * c0) =
          make_uint2(f32x4_to_e4m3x4(x[i][0], x[i][1], x[i][2], x[i][3]),
                     f32x4_to_e4m3x4(x[i][4], x[i][5], x[i][6], x[i][7]));
      *reinterpret_cast<uint2*>(o + 8 * c1) =
          make_uint2(f32x4_to_e4m3x4(x[i][8], x[i][9], x[i][10], x[i][11]),
                     f32x4_to_e4m3x4(x[i][12], x[i][13], x[i][14], x[i][15]));
    }
  }
}

template <bool kF8, int kD>
void launch_append(const AppendParams& p, cudaStream_t st) {
  const PagedView& c = p.c;
  const int streams = p.Hq + 2 * c.Hkv;
  constexpr int kWarpRows = 32 / (kD / 16);
  if (c.cu == nullptr && c.Qn <= kWarpRows) {
    // decode steps: a unit has at most kWarpRows tokens, one warp each
    dim3 grid((unsigned)c.B * p.units_per_row, (streams + 3) / 4);
    paged_append_kernel<kF8, kD, 32, 1><<<grid, 128, 0, st>>>(p);
    return;
  }
  const long long units = c.cu == nullptr ? (long long)c.B * p.units_per_row
                                          : ((long long)c.N >> c.p_shift) + 2LL * c.B;
  dim3 grid((unsigned)units, streams);
  constexpr int kRows = 256 / (kD / 16);
  const int passes = ((1 << c.p_shift) + kRows - 1) / kRows;
  if (passes == 1)
    paged_append_kernel<kF8, kD, 256, 1><<<grid, 256, 0, st>>>(p);
  else if (passes == 2)
    paged_append_kernel<kF8, kD, 256, 2><<<grid, 256, 0, st>>>(p);
  else
    paged_append_kernel<kF8, kD, 256, 4><<<grid, 256, 0, st>>>(p);
}

}  // namespace

unsigned read_and_clear_error_append(cudaStream_t, std::string* where) {
  unsigned w = 0, zero = 0;
  cudaMemcpyFromSymbol(&w, g_err_append, sizeof(w));
  if (w) {
    cudaMemcpyToSymbol(g_err_append, &zero, sizeof(zero));
    *where += " (paged append: a length, a page number or a position out of range)";
  }
  return w;
}

int launch_paged_append(const PagedView& c, int f8, int D, const void* k, long long k_tok,
                        const void* v, long long v_tok, const void* q, long long q_tok, void* q_out,
                        long long qo_tok, int Hq, const float* cosp, const float* sinp, int rot,
                        int max_pos, int interleaved, cudaStream_t stream) {
  AppendParams p;
  p.c = c;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.cosp = cosp;
  p.sinp = sinp;
  p.k_tok = k_tok; p.v_tok = v_tok; p.q_tok = q_tok; p.qo_tok = qo_tok;
  p.Hq = q ? Hq : 0;
  p.rot = cosp ? rot : 0;
  p.interleaved = interleaved;
  p.max_pos = max_pos;
  // n tokens in a row lie in at most floor((n - 2) / P) + 2 pages (n >= 2), one for n = 1
  p.units_per_row = c.Qn <= 1 ? 1 : ((c.Qn - 2) >> c.p_shift) + 2;
  if (D == 128)
    f8 ? launch_append<true, 128>(p, stream) : launch_append<false, 128>(p, stream);
  else
    f8 ? launch_append<true, 64>(p, stream) : launch_append<false, 64>(p, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_error(e, "paged append launch");
  return SBA_OK;
}

}  // namespace sba
