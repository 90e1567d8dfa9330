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
// scale needs, so a unit is one block (or one warp) and nothing waits for another.  Every
// input is read once and held in registers between the maximum and the store.
//
// What bounds it.  Prompts: bytes.  12 rows of up to 2600 tokens, 32 + 2 * 8 heads of 128,
// e4m3 pages of 64: 340 MB in 65.2 us (5.2 TB/s); the angles of a page's positions are
// kept over the heads (79 us when each head reads them again), and the next head's
// loads are under way (none: 81.7; a second head's as well: 66.4; a ring of cp.async in shared
// memory instead: 67.3).  One token a row: the chain of length, table,
// values, scale and store, 2.2 us for 8 rows and 2.8 for 256; a warp takes several heads
// because one head each needs four times the waves of blocks (5.7).
#include <algorithm>
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
  int heads;  // few tokens: heads of a warp
};

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float a2 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float b2 = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = a2;
  b = b2;
}
__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  unpack8(__ldg(reinterpret_cast<const uint4*>(p)), x);
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

// The unit's row, first token and positions [p0, p1); m = p1 - p0 <= 0: nothing to do.
struct Unit {
  int b, first, p0, m, page_slot;
};
__device__ __forceinline__ Unit unit_of(const PagedView& c, int b, int j, bool report) {
  Unit u;
  u.b = b;
  u.m = 0;
  u.first = u.p0 = u.page_slot = 0;
  bool bad;
  const PagedRow r = paged_row(c, b, &bad);
  if (bad) {
    if (report) atomicOr(&g_err_append, (unsigned)kDevErrInput);
    return u;
  }
  if (r.n == 0) return u;
  const int start = r.len - r.n;  // position of the row's first token; those left of 0 do not exist
  u.page_slot = (max(start, 0) >> c.p_shift) + j;
  u.p0 = max(max(start, 0), u.page_slot << c.p_shift);
  u.m = min(r.len, (u.page_slot + 1) << c.p_shift) - u.p0;
  u.first = r.t0 + (u.p0 - start);
  return u;
}
__device__ __forceinline__ int page_of(const PagedView& c, const Unit& u, bool report) {
  const int page = c.table[(long long)u.b * c.width + u.page_slot];
  if ((unsigned)page < (unsigned)c.num_pages) return page;
  if (report) atomicOr(&g_err_append, (unsigned)kDevErrInput);
  return -1;
}

// A head of the call's queries, keys or values.
struct Stream {
  const __nv_bfloat16* src;
  long long tok;
  int h;
  bool is_q, is_k;
};
template <int kD>
__device__ __forceinline__ Stream stream_of(const AppendParams& p, int s) {
  Stream t;
  t.is_q = s < p.Hq;
  t.is_k = !t.is_q && s < p.Hq + p.c.Hkv;
  t.h = t.is_q ? s : (t.is_k ? s - p.Hq : s - p.Hq - p.c.Hkv);
  t.src = (t.is_q ? p.q : (t.is_k ? p.k : p.v)) + (long long)t.h * kD;
  t.tok = t.is_q ? p.q_tok : (t.is_k ? p.k_tok : p.v_tok);
  return t;
}

// Chunks of 8 dimensions of the thread `rt` of a row: rotated ones first, a chunk with its
// partner; then the rest two by two.
__device__ __forceinline__ void chunks_of(int rt, int rot, int interleaved, int& c0, int& c1) {
  if (rt < rot / 16 && !interleaved) {
    c0 = rt;
    c1 = rt + rot / 16;
  } else {
    c0 = 2 * rt;
    c1 = 2 * rt + 1;
  }
}
__device__ __forceinline__ void load_angles(const AppendParams& p, int pos, int rt, float* cs, float* sn) {
  if (pos >= p.max_pos) {
    atomicOr(&g_err_append, (unsigned)kDevErrInput);
    pos = p.max_pos - 1;
  }
  // of pairs 8 rt .. 8 rt + 7
  const float4* cp = reinterpret_cast<const float4*>(p.cosp + (long long)pos * (p.rot / 2) + 8 * rt);
  const float4* sp = reinterpret_cast<const float4*>(p.sinp + (long long)pos * (p.rot / 2) + 8 * rt);
  *reinterpret_cast<float4*>(cs) = __ldg(cp);
  *reinterpret_cast<float4*>(cs + 4) = __ldg(cp + 1);
  *reinterpret_cast<float4*>(sn) = __ldg(sp);
  *reinterpret_cast<float4*>(sn + 4) = __ldg(sp + 1);
}
__device__ __forceinline__ void rotate16(float* x, const float* cs, const float* sn, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) rotate_pair(x[2 * e], x[2 * e + 1], cs[e], sn[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) rotate_pair(x[e], x[e + 8], cs[e], sn[e]);
  }
}
__device__ __forceinline__ float finite_max(const float* x, float top) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float a = fabsf(x[e]);
    if (a <= 3.4028235e38f) top = fmaxf(top, a);  // infinities and NaN set no scale
  }
  return top;
}
// 16 codes that a page holds, from scale `old` to 1 / `inv`.
__device__ __forceinline__ uint4 rescaled16(uint4 w, float old, float inv) {
  uint32_t* c = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16x2(c[i], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    c[i] = f32x4_to_e4m3x4(__fmul_rn(__fmul_rn(a.x, old), inv), __fmul_rn(__fmul_rn(a.y, old), inv),
                           __fmul_rn(__fmul_rn(b.x, old), inv), __fmul_rn(__fmul_rn(b.y, old), inv));
  }
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* row, int c0, int c1, float* x, float inv) {
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(x[e], inv);
  *reinterpret_cast<uint2*>(row + 8 * c0) =
      make_uint2(f32x4_to_e4m3x4(x[0], x[1], x[2], x[3]), f32x4_to_e4m3x4(x[4], x[5], x[6], x[7]));
  *reinterpret_cast<uint2*>(row + 8 * c1) =
      make_uint2(f32x4_to_e4m3x4(x[8], x[9], x[10], x[11]), f32x4_to_e4m3x4(x[12], x[13], x[14], x[15]));
}

// Few tokens of a page (at most kFew = 512 / kD), one warp, heads first .. min(first + kFew >>
// shift, end) - 1: a row of a head is kD / 16 threads, 16 dimensions each, and a head has
// 2^shift rows of threads.
template <bool kF8, int kD>
__device__ __forceinline__ void append_few(const AppendParams& p, const Unit& u, int first, int end, int shift) {
  constexpr int kRowThreads = kD / 16;
  constexpr int kFew = 32 / kRowThreads;
  const PagedView& c = p.c;
  const int lane = threadIdx.x & 31, rt = lane % kRowThreads;
  const int row = lane / kRowThreads & ((1 << shift) - 1), stream = first + (lane / kRowThreads >> shift);
  const Stream t = stream_of<kD>(p, min(stream, end - 1));
  const int rot = t.is_q || t.is_k ? p.rot : 0;
  const bool mine = row < u.m && stream < end;
  int c0, c1;
  chunks_of(rt, rot, p.interleaved, c0, c1);
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.f;
  if (mine) {
    const __nv_bfloat16* s = t.src + (long long)(u.first + row) * t.tok;
    load8(s + 8 * c0, x);
    load8(s + 8 * c1, x + 8);
  }
  const bool any_kv = min(first + (kFew >> shift), end) > p.Hq;
  const int page = any_kv ? page_of(c, u, lane == 0) : 0;
  if (page < 0) return;
  if (mine && rt < rot / 16) {
    float cs[8], sn[8];
    load_angles(p, u.p0 + row, rt, cs, sn);
    rotate16(x, cs, sn, p.interleaved);
  }
  const int P = 1 << c.p_shift, off = u.p0 & (P - 1);
  uint8_t* tile = (t.is_k ? c.k : c.v) + page * c.page_bytes + (long long)t.h * P * (kD * (kF8 ? 1 : 2));
  if ((t.is_q || !kF8) && mine) {
    __nv_bfloat16* o = t.is_q ? p.q_out + (long long)(u.first + row) * p.qo_tok + (long long)t.h * kD
                              : reinterpret_cast<__nv_bfloat16*>(tile) + (off + row) * kD;
    store8(o + 8 * c0, x);
    store8(o + 8 * c1, x + 8);
  }
  if constexpr (kF8) {
    const bool stores = !t.is_q && stream < end;  // this head's values are quantised
    if (!__any_sync(0xffffffffu, stores)) return;
    float* scale_at = (t.is_k ? c.ks : c.vs) + (long long)page * c.Hkv + t.h;
    const float old = stores && off > 0 ? *scale_at : 0.f;
    float amax = finite_max(x, 0.f);
#pragma unroll
    for (int d = (kRowThreads << shift) / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const float need = pow2_scale(amax);
    const float scale = need > old ? need : old;
    const float inv = __frcp_rn(scale);
    // Heads whose scale grows: the whole warp takes their codes along, one head after the
    // other, eight loads in flight.
    const bool grow = stores && scale != old;
    unsigned heads = __ballot_sync(0xffffffffu, grow && rt == 0 && row == 0);
    if (grow && rt == 0 && row == 0) *scale_at = scale;
    while (heads) {
      const int from = __ffs(heads) - 1;
      heads &= heads - 1;
      uint8_t* const at = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(tile), from));
      const float was = __shfl_sync(0xffffffffu, old, from), now = __shfl_sync(0xffffffffu, inv, from);
      const int n = off * (kD / 16);  // 16-byte pieces held already
      for (int i0 = 0; i0 < n; i0 += 256) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + j * 32 + lane < n) w[j] = reinterpret_cast<const uint4*>(at)[i0 + j * 32 + lane];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + j * 32 + lane < n) reinterpret_cast<uint4*>(at)[i0 + j * 32 + lane] = rescaled16(w[j], was, now);
      }
    }
    if (stores && mine) store_codes(tile + (off + row) * kD, c0, c1, x, inv);
  }
}

// The first and the last page of a row, where they get at most kFew tokens: all of a call's
// pages when no row has more.  kOne: every row has one.
template <bool kF8, int kD, bool kOne>
__global__ void __launch_bounds__(128, 6)  // 256 rows of 4 tokens: 8.3 us with 5 blocks an SM, 7.8 with 6, 12.0 with 8
paged_append_few_kernel(const AppendParams p) {
  constexpr int kFew = 512 / kD;
  const PagedView& c = p.c;
  paged_wait_before();
  const int heads = kOne ? kFew : p.heads, b = blockIdx.x;
  const int first = (blockIdx.y * 4 + (threadIdx.x >> 5)) * heads, end = min(first + heads, p.Hq + 2 * c.Hkv);
  if (first >= end) return;
  const bool report = (threadIdx.x & 31) == 0;
  const Unit u = unit_of(c, b, 0, report);
  if (u.m <= 0) return;
  if constexpr (kOne) {
    append_few<kF8, kD>(p, u, first, end, 0);
  } else {
    auto put = [&](const Unit& x) {
      const int shift = x.m > 4 ? 3 : x.m > 2 ? 2 : x.m - 1;
      for (int s = first; s < end; s += kFew >> shift) append_few<kF8, kD>(p, x, s, end, shift);
    };
    if (u.m <= kFew) put(u);
    const int last = ((c.lens[b] - 1) >> c.p_shift) - u.page_slot;
    if (last > 0) {
      const Unit v = unit_of(c, b, last, report);
      if (v.m > 0 && v.m <= kFew) put(v);
    }
  }
}

// Rows of a page that a thread takes.  e4m3: fewer warps meet at the barrier between a
// head's maximum and its codes (12 prompts as above: 65.1 us with two, 67.0 with one); bf16
// has no barrier (6 MB of prompts into pages of 16: 11.6 / 10.8 us).
template <bool kF8>
constexpr int append_passes = kF8 ? 2 : 1;

// The pages of a row that this kernel writes: `n` of them from the row's page `first` on.
// kBig: pages that get at most kFew tokens are paged_append_few_kernel's (those between a
// row's first and last are full).
struct RowPages {
  int first, n;
};
template <bool kBig, int kFew>
__device__ __forceinline__ RowPages row_pages(const PagedView& c, int b, bool* bad) {
  const PagedRow r = paged_row(c, b, bad);
  const int start = max(r.len - r.n, 0);
  RowPages w = {0, 0};
  if (*bad || r.n == 0 || r.len <= start) return w;
  const int p0 = start >> c.p_shift, p1 = (r.len - 1) >> c.p_shift;
  w.n = p1 - p0 + 1;
  if constexpr (kBig) {
    if (min(r.len, (p0 + 1) << c.p_shift) - start <= kFew) {
      w.first = 1;
      --w.n;
    }
    if (p1 > p0 && r.len - (p1 << c.p_shift) <= kFew) --w.n;
  }
  return w;
}

// a / b, b > 0; a is nearly always small enough for the short division.
__device__ __forceinline__ long long quotient(long long a, unsigned b) {
  return a >> 32 ? a / b : (unsigned)a / b;
}

// Any number of tokens.  All pages in order, `streams` heads each, form one line that is cut
// into equal runs, one for each block that is resident: no last wave with few blocks, and
// (few rows) no place for a page that a row might have had: blocks of 8 heads of each such
// page take 36.6 us for 256 rows of 8 tokens, 10.8 for 16 of 32, this one 30.5 and 9.0; long
// prompts alike.  In a page a block goes from head to head:
// the angles of its positions stay in registers, and a head's values are loaded while the
// one before is worked on.
template <bool kF8, int kD, bool kBig, bool kCounted>
__global__ void __launch_bounds__(kF8 ? 512 : 1024)
paged_append_kernel(const AppendParams p) {
  constexpr int kRowThreads = kD / 16;
  constexpr int kPasses = append_passes<kF8>, kFew = 512 / kD;
  const PagedView& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int streams = p.Hq + 2 * c.Hkv;
  __shared__ float s_max[2][32];
  __shared__ long long s_sum[32], s_off;
  __shared__ int s_row;
  paged_wait_before();

  // ---- this block's run of the line, and the row it begins in.  Few rows are counted; many
  // get the most pages that they could have: n tokens touch at most floor(n / P) + 2 (kBig:
  // fill floor(n / (kFew + 1))), and floor is superadditive, so that the row's part begins at
  // begin_of(row) and parts never overlap.
  auto begin_of = [&](int i) -> long long {
    if (c.cu == nullptr) return (long long)i * (((c.Qn - 1) >> c.p_shift) + 2);
    const int t = min(max(c.cu[i], 0), c.N);
    return kBig ? t / (kFew + 1) : (t >> c.p_shift) + 2LL * i;
  };
  long long cur, end, at;  // at: of the row's part of the line
  int b;
  if constexpr (kCounted) {
    const int chunk = (c.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * chunk, c.B), b1 = min(b0 + chunk, c.B);
    long long sum = 0;
    bool wrong = false;
    for (b = b0; b < b1; ++b) {
      bool x;
      sum += row_pages<kBig, kFew>(c, b, &x).n;
      wrong |= x;
    }
    if (wrong && blockIdx.x == 0) atomicOr(&g_err_append, (unsigned)kDevErrInput);
    long long pre = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, pre, d);
      if (lane >= d) pre += x;
    }
    if (lane == 31) s_sum[warp] = pre;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < warps; ++i) {
      if (i == warp) pre += total;
      total += s_sum[i];
    }
    pre -= sum;  // pages before this thread's rows
    const long long per = quotient(total * streams + gridDim.x - 1, gridDim.x);
    cur = blockIdx.x * per;
    end = min(cur + per, total * streams);
    if (cur >= end) return;
    b = b0;
    at = cur - pre * streams;
    if (at >= 0 && at < sum * streams) {
      for (; b + 1 < b1; ++b) {
        bool x;
        const long long n = (long long)row_pages<kBig, kFew>(c, b, &x).n * streams;
        if (at < n) break;
        at -= n;
      }
      s_row = b;
      s_off = at;
    }
    __syncthreads();
    b = s_row;
    at = s_off;
  } else {
    for (int i = blockIdx.x * blockDim.x + tid; i < c.B; i += gridDim.x * blockDim.x) {
      bool wrong;
      paged_row(c, i, &wrong);
      if (wrong) atomicOr(&g_err_append, (unsigned)kDevErrInput);
    }
    const long long total = c.cu == nullptr ? begin_of(c.B) : kBig ? c.N / (kFew + 1) : (c.N >> c.p_shift) + 2LL * c.B;
    const long long per = quotient(total * streams + gridDim.x - 1, gridDim.x);
    cur = blockIdx.x * per;
    end = min(cur + per, total * streams);
    if (cur >= end) return;
    // the last row that begins at or before this place: 32 probes a round
    const long long unit = quotient(cur, streams);
    b = 0;
    for (int range = c.B; range > 1;) {
      const int step = (range + 31) / 32, i = b + lane * step;
      const unsigned before = __ballot_sync(0xffffffffu, lane * step < range && begin_of(min(i, c.B - 1)) <= unit);
      const int hit = before ? 31 - __clz(before) : 0;
      b += hit * step;
      range = min(step, range - hit * step);
    }
    at = cur - begin_of(b) * streams;
    if (at < 0) {  // ahead of the first row's first token
      cur -= at;
      at = 0;
    }
  }

  const int rows = blockDim.x / kRowThreads;
  const int rt = tid % kRowThreads, slot = tid / kRowThreads;
  while (cur < end) {
    bool bad;
    const RowPages w = row_pages<kBig, kFew>(c, b, &bad);
    if (at >= (long long)w.n * streams) {
      // on to the next row with a page, 32 looked at together
      at = 0;
      unsigned some = 0;
      int i = b + 1;
      for (; i < c.B; i += 32) {
        some = __ballot_sync(0xffffffffu, i + lane < c.B && row_pages<kBig, kFew>(c, min(i + lane, c.B - 1), &bad).n > 0);
        if (some || (!kCounted && begin_of(i) * streams >= end)) break;
      }
      if (some == 0) return;
      b = i + __ffs(some) - 1;
      if constexpr (!kCounted) cur = max(cur, begin_of(b) * streams);
      continue;
    }
    const int j = (int)quotient(at, streams), s0 = (int)(at - (long long)j * streams);
    const int s_end = (int)min((long long)streams, s0 + (end - cur));
    cur += s_end - s0;
    at += s_end - s0;
    const Unit u = unit_of(c, b, w.first + j, false);
    const int P = 1 << c.p_shift, off = u.p0 & (P - 1);
    const int page = s_end > p.Hq ? page_of(c, u, tid == 0) : 0;
    if (page < 0) continue;

    bool mine[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) mine[i] = i * rows + slot < u.m;
    const bool turns = rt < p.rot / 16;
    float cs[kPasses][8], sn[kPasses][8];
    if (turns && s0 < p.Hq + c.Hkv) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (mine[i]) load_angles(p, u.p0 + i * rows + slot, rt, cs[i], sn[i]);
    }
    uint4 next[kPasses][2];
    auto fetch = [&](int stream) {
      const Stream t = stream_of<kD>(p, stream);
      int c0, c1;
      chunks_of(rt, t.is_q || t.is_k ? p.rot : 0, p.interleaved, c0, c1);
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (mine[i]) {
          const __nv_bfloat16* src = t.src + (long long)(u.first + i * rows + slot) * t.tok;
          next[i][0] = __ldg(reinterpret_cast<const uint4*>(src + 8 * c0));
          next[i][1] = __ldg(reinterpret_cast<const uint4*>(src + 8 * c1));
        }
    };
    fetch(s0);
    for (int s = s0; s < s_end; ++s) {
      const Stream t = stream_of<kD>(p, s);
      const int rot = t.is_q || t.is_k ? p.rot : 0;
      int c0, c1;
      chunks_of(rt, rot, p.interleaved, c0, c1);
      float x[kPasses][16];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        unpack8(next[i][0], x[i]);
        unpack8(next[i][1], x[i] + 8);
      }
      if (s + 1 < s_end) fetch(s + 1);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (mine[i]) {
          if (rt < rot / 16) rotate16(x[i], cs[i], sn[i], p.interleaved);
          if (kF8 && !t.is_q) amax = finite_max(x[i], amax);
        }
      uint8_t* tile = (t.is_k ? c.k : c.v) + page * c.page_bytes + (long long)t.h * P * (kD * (kF8 ? 1 : 2));
      if (t.is_q || !kF8) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          if (mine[i]) {
            const int row = i * rows + slot;
            __nv_bfloat16* o = t.is_q ? p.q_out + (long long)(u.first + row) * p.qo_tok + (long long)t.h * kD
                                      : reinterpret_cast<__nv_bfloat16*>(tile) + (off + row) * kD;
            store8(o + 8 * c0, x[i]);
            store8(o + 8 * c1, x[i] + 8);
          }
        continue;
      }
      float* scale_at = (t.is_k ? c.ks : c.vs) + (long long)page * c.Hkv + t.h;
      const float old = off > 0 ? *scale_at : 0.f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      float* most = s_max[s & 1];  // two in turn: a head's readers are behind the next barrier
      if ((tid & 31) == 0) most[tid >> 5] = amax;
      __syncthreads();
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, most[w]);
      const float need = pow2_scale(amax);
      const float scale = need > old ? need : old;
      const float inv = __frcp_rn(scale);
      if (scale != old) {
        if (tid == 0) *scale_at = scale;  // every thread has read the old one
        for (int i = slot; i < off; i += rows) {
          uint4* at = reinterpret_cast<uint4*>(tile + i * kD + 16 * rt);
          *at = rescaled16(*at, old, inv);
        }
      }
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (mine[i]) store_codes(tile + (off + i * rows + slot) * kD, c0, c1, x[i], inv);
    }
  }
}

template <bool kF8, int kD>
cudaError_t launch_append(AppendParams p, cudaStream_t st) {
  const PagedView& c = p.c;
  constexpr int kFew = 512 / kD;
  const int streams = p.Hq + 2 * c.Hkv;
  const bool few = c.cu == nullptr && c.Qn <= kFew;
  // Token counts only the device knows: pages with few tokens go to the kernel that is made
  // for them when the average row has few.  Rows of n tokens each, e4m3 D = 128 (kFew = 4),
  // 48 heads, us with one kernel / with two, all rows of 150 tokens (a page each, the inputs
  // of one call over and over): 256 rows n = 1: 30.2 / 5.3, 4: 29.4 / 10.6, 8: 30.5 / 34.1,
  // 16: 39.5 / 43.1; 16 rows n = 1: 5.5 / 4.7, 8: 5.6 / 7.2.  As chosen, with lengths spread
  // over the pages and three calls' inputs in turn: 256 rows n = 4: 12.0, 8: 41.5, 16: 49.8,
  // 32: 67.0 (floors 3.5, 7.0, 13.9, 27.9).
  const bool two = c.cu != nullptr && c.N <= (long long)kFew * c.B;
  if (few || two) {
    // a warp takes as many heads as it has threads for, going by the tokens of the average row
    const int rows = std::min(kFew, (int)((c.N + (long long)c.B - 1) / c.B));
    p.heads = kFew / (rows > 4 ? 8 : rows > 2 ? 4 : rows);
    const dim3 grid((unsigned)c.B, (streams + 4 * p.heads - 1) / (4 * p.heads));
    const cudaError_t e = few && c.Qn == 1 ? paged_launch(paged_append_few_kernel<kF8, kD, true>, grid, 128, 0, st, p)
                                           : paged_launch(paged_append_few_kernel<kF8, kD, false>, grid, 128, 0, st, p);
    if (e != cudaSuccess || few || c.N <= kFew) return e;
  }
  // blocks that are resident together: two of 256 threads on an SM (e4m3, 124 registers),
  // or 1024 threads (bf16)
  const int threads = (kD << c.p_shift) / (16 * append_passes<kF8>);
  const dim3 grid(152 * ((kF8 ? 512 : 1024) / threads));
  // Counting takes each block a pass over the rows: 4096 rows of one token, D = 64, pages of 16
  // (32 threads) 82 us, where the search takes 19.8; 1000 rows, D = 128 (64 threads) 14.3 / 11.3.
  const bool counted = c.B <= 4 * threads;
  auto* kernel = two ? (counted ? paged_append_kernel<kF8, kD, true, true> : paged_append_kernel<kF8, kD, true, false>)
                     : (counted ? paged_append_kernel<kF8, kD, false, true> : paged_append_kernel<kF8, kD, false, false>);
  return paged_launch(kernel, grid, threads, 0, st, p);
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
  cudaError_t e;
  if (D == 128)
    e = f8 ? launch_append<true, 128>(p, stream) : launch_append<false, 128>(p, stream);
  else
    e = f8 ? launch_append<true, 64>(p, stream) : launch_append<false, 64>(p, stream);
  if (e != cudaSuccess) return cuda_error(e, "paged append launch");
  return SBA_OK;
}

}  // namespace sba
