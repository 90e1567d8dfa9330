// One warp's walk over key tiles of a paged cache: 16 query rows, an online softmax.
//
// Rows are (query, head) pairs of one KV head, the 16 rows of an m16n8k16 MMA.  A tile is
// kTileKeys keys, whole 16-key subtiles of one page each, brought into shared memory with
// 16-byte cp.async through a ring of kPagedStages tiles per warp.
//
// e4m3 operands.  The tensor instruction takes fp16 pairs.  Codes become fp16 exactly
// (one conversion per pair); the query row is multiplied by a power of two that puts its
// largest element near 2^14, so its conversion drops only what lies 2^-38 below it; the
// page's key scale and the query's factor multiply the logit.  A page's value scale
// s = a 2^e (1 <= a < 2) multiplies the probability: with p = 2^(x - m) the kernel sums
// l += p in fp32 and feeds p s 2^(m - u + 8) to the MMA, where u is a running maximum of
// x + e over the keys, so the product stays below 2^15 whatever the pages' scales are, and
// what rounds to zero in fp16 lies 2^-33 below the largest contribution.  fp16 keeps 11
// bits of each probability; a bf16 cache uses bf16 probabilities (8 bits) and u = m, as the
// contiguous kernels do: the MMA takes both operands in one type, and fp16 has not the range
// of bf16 values.  Sums, maxima and o stay in fp32.
//
// Fragments.  The order of the contraction index is free, so the thread that holds
// elements (2c, 2c+1, 2c+8, 2c+9) of a 16-step takes four neighbouring bytes instead: its
// part of a key row is 16-byte chunks c and c + 4, its part of a value row is the run of
// kD / 8 dimensions from (kD / 8) g on, for the four keys that its probabilities belong
// to; two byte permutes per word put a pair of keys next to each other.  Output column n
// of MMA j is dimension (kD / 8) n + j.  Chunks are stored at chunk ^ f(row), which
// spreads both reads over all banks (f below).
#pragma once

#include <cooperative_groups.h>

#include <climits>

#include "paged.cuh"

namespace sba {

constexpr float kPagedLog2e = 1.4426950408889634f;
constexpr float kPagedLn2 = 0.6931471805599453f;
constexpr int kPagedStages = 2;

__device__ __forceinline__ uint2 paged_lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <bool kHalf>
__device__ __forceinline__ void paged_mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What the 16 rows may see and how their logits are formed.
struct PagedMask {
  int len;         // keys < len exist
  int wlo0, whi0;  // window of the thread's row g
  int wlo1, whi1;  // window of row g + 8
  int all_lo, all_hi;  // the part of the window that every row shares
  int num_sinks;       // keys < num_sinks are always visible
  const float* bias0;  // their biases for row g
  int bias_step;       // distance to those for row g + 8
};

// log2(e) cap tanh(y) with an error relative to the value: near zero the odd series (its
// next term is below 2^-26 of the sum at |y| = 0.25), elsewhere 1 - 2 / (1 + e^(2y)).
__device__ __forceinline__ float paged_capped(float y, float c1k) {
  const float e = ptx::ex2(y * (2.f * kPagedLog2e));
  float rc;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc) : "f"(1.f + e));
  const float far = fmaf(-2.f, rc, 1.f);
  const float y2 = y * y;
  float pl = fmaf(y2, 62.f / 2835.f, -17.f / 315.f);
  pl = fmaf(y2, pl, 2.f / 15.f);
  pl = fmaf(y2, pl, -1.f / 3.f);
  const float near = fmaf(y * y2, pl, y);
  return c1k * (fabsf(y) < 0.25f ? near : far);
}
// The same of two scores times f = 2 log2(e) scale / cap, the exponent of e^(2y), two at a time
// where the instructions are; the series has a term less and ends at |y| = 1/8 (next one 2^-22).
__device__ __forceinline__ void paged_capped2(float& x0, float& x1, float f, float c1k, float half_cap) {
  using namespace ptx;
  constexpr float k2 = 4.f * kPagedLog2e * kPagedLog2e;  // (exponent / y)^2
  const uint64_t w = mul_f32x2(pack_f32x2(x0, x1), pack_f32x2(f, f));
  float w0, w1, rc0, rc1, far0, far1, near0, near1;
  unpack_f32x2(w, w0, w1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc0) : "f"(1.f + ex2(w0)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc1) : "f"(1.f + ex2(w1)));
  unpack_f32x2(fma_f32x2(pack_f32x2(rc0, rc1), pack_f32x2(-2.f * c1k, -2.f * c1k), pack_f32x2(c1k, c1k)), far0, far1);
  const uint64_t u = mul_f32x2(w, w), z = mul_f32x2(w, pack_f32x2(half_cap, half_cap));
  constexpr float a = 2.f / 15.f / (k2 * k2), b = -1.f / 3.f / k2;
  unpack_f32x2(fma_f32x2(mul_f32x2(z, u), fma_f32x2(u, pack_f32x2(a, a), pack_f32x2(b, b)), z), near0, near1);
  constexpr float end = 2.f * kPagedLog2e / 8.f;
  x0 = fabsf(w0) < end ? near0 : far0;
  x1 = fabsf(w1) < end ? near1 : far1;
}

// kCap: there is a soft cap.
// kSinks: there are sinks (a call without them needs no part of their masks and addresses).
template <bool kF8, int kD, int kTileKeys, bool kHi, bool kCap, bool kSinks>
struct PagedWarp {
  static constexpr bool kCodes = kF8;
  static constexpr int kKeys = kTileKeys;
  static constexpr int kSub = kKeys / 16;
  static constexpr int kRowBytes = kD * (kF8 ? 1 : 2);
  static constexpr int kTileBytes = kKeys * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kWarpBytes = kPagedStages * kStageBytes;
  static constexpr int kChunks = kRowBytes / 16;   // 16-byte chunks per row
  static constexpr int kStep = 32 / kChunks;       // rows per warp-wide copy
  static constexpr int kCopies = kKeys / kStep;
  static constexpr int kNT = kD / 8;               // output columns / 8
  static constexpr int kKS = kD / 16;              // contraction steps of Q K^T
  static constexpr int kSmemRow = kD + 8;          // merge buffer row, floats
  static constexpr float kRaise = 8.f;             // m moves when a tile exceeds it by 2^8

  uint32_t qa[kKS][4];
  float o[kNT][4];
  float m0, m1, l0, l1;
  float u0, u1;    // e4m3: reference of the values' probabilities
  float r0, r1;    // logit factors of rows g, g + 8
  float c1k, half_cap;  // log2(e) cap, cap / 2
  int lane, g, c;
  uint32_t ring;
  const uint8_t* kbase;
  const uint8_t* vbase;
  const float* ks;
  const float* vs;
  const int* table;
  long long page_bytes;
  int p_shift, Hkv, num_pages;
  unsigned* err;

  // Byte offset of 16-byte chunk `ch` of row `row` inside a tile.
  static __device__ __forceinline__ uint32_t at(int row, int ch) {
    if constexpr (!kF8) return row * kRowBytes + ((ch ^ (row & 7)) << 4);
    if constexpr (kF8 && kD == 128) {
      const int f = (((row >> 1) & 3) << 1) ^ ((row & 1) << 2);
      return row * 128 + ((ch ^ f) << 4);
    }
    const int line = row >> 1;
    return line * 128 + (((((row & 1) << 2) + ch) ^ ((line & 3) << 1)) << 4);
  }

  __device__ __forceinline__ void init(const PagedView& v, int b, int h, uint32_t smem_ring, float scale,
                                       float cap, unsigned* e) {
    lane = threadIdx.x & 31;
    g = lane >> 2;
    c = lane & 3;
    ring = smem_ring;
    p_shift = v.p_shift;
    Hkv = v.Hkv;
    num_pages = v.num_pages;
    page_bytes = v.page_bytes;
    const long long head = ((long long)h << p_shift) * kRowBytes;
    kbase = v.k + head;
    vbase = v.v + head;
    ks = kF8 ? v.ks + h : nullptr;
    vs = kF8 ? v.vs + h : nullptr;
    table = v.table + (long long)b * v.width;
    err = e;
#pragma unroll
    for (int i = 0; i < kNT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = u0 = u1 = -INFINITY;
    l0 = l1 = 0.f;
    r0 = r1 = kCap ? scale * (2.f * kPagedLog2e / cap) : scale * kPagedLog2e;
    half_cap = 0.5f * cap;
    c1k = cap * kPagedLog2e;
  }

  // Query rows g and g + 8 (null: a row of zeros).
  __device__ __forceinline__ void load_q(const __nv_bfloat16* q0, const __nv_bfloat16* q1) {
    if constexpr (!kF8) {
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        const int d = s * 16 + 2 * c;
        qa[s][0] = q0 ? __ldg(reinterpret_cast<const unsigned*>(q0 + d)) : 0u;
        qa[s][2] = q0 ? __ldg(reinterpret_cast<const unsigned*>(q0 + d + 8)) : 0u;
        qa[s][1] = kHi && q1 ? __ldg(reinterpret_cast<const unsigned*>(q1 + d)) : 0u;
        qa[s][3] = kHi && q1 ? __ldg(reinterpret_cast<const unsigned*>(q1 + d + 8)) : 0u;
      }
    } else {
#pragma unroll
      for (int hi = 0; hi < (kHi ? 2 : 1); ++hi) {
        const __nv_bfloat16* q = hi ? q1 : q0;
        uint2 w[kKS];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < kKS; ++s) {
          const int d = 16 * (c + 4 * (s >> 2)) + 4 * (s & 3);
          w[s] = q ? __ldg(reinterpret_cast<const uint2*>(q + d)) : make_uint2(0u, 0u);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(w[s].x)), fabsf(bf16_hi(w[s].x))),
                                 fmaxf(fabsf(bf16_lo(w[s].y)), fabsf(bf16_hi(w[s].y)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // power of two f with top f in [2^14, 2^15); 1 for zero and non-finite rows.  Both
        // f and 1 / f stay normal numbers.
        const int ex = (int)((__float_as_uint(top) >> 23) & 255);
        const int fe = (ex == 0 || ex == 255) ? 127 : min(127 + 14 - (ex - 127), 253);
        const float f = __uint_as_float((uint32_t)fe << 23);
        const float inv = __uint_as_float((uint32_t)(254 - fe) << 23);
        if (hi) r1 *= inv; else r0 *= inv;
#pragma unroll
        for (int s = 0; s < kKS; ++s) {
          qa[s][hi] = pack_f16x2(bf16_lo(w[s].x) * f, bf16_hi(w[s].x) * f);
          qa[s][hi + 2] = pack_f16x2(bf16_lo(w[s].y) * f, bf16_hi(w[s].y) * f);
        }
      }
      if constexpr (!kHi) {
#pragma unroll
        for (int s = 0; s < kKS; ++s) qa[s][1] = qa[s][3] = 0u;
      }
    }
  }

  struct Pages { int page[kSub]; };
  struct Scales { float k[kSub], v[kSub]; };

  // The key read in place of `key`, of subtile s of the tile at key0: keys outside [cl, ch]
  // repeat its ends, as slots that no query sees may hold anything and 0 * NaN would reach the
  // output.  The sinks, all in the first subtile, lie left of cl where a window begins; that
  // subtile's keys between them and cl repeat the last sink, so that all stay in its page.
  __device__ __forceinline__ int read_for(int key, int s, int key0, int cl, int ch, int sinks) const {
    if (kSinks && s == 0 && key0 < sinks && key < cl) return min(min(key, sinks - 1), ch);
    return min(max(key, cl), ch);
  }
  // Page numbers of the tile's subtiles.
  __device__ __forceinline__ Pages fetch(int key0, int cl, int ch, int sinks) const {
    Pages p;
#pragma unroll
    for (int s = 0; s < kSub; ++s) p.page[s] = __ldg(table + (read_for(key0 + 16 * s, s, key0, cl, ch, sinks) >> p_shift));
    return p;
  }
  __device__ __forceinline__ void check(Pages& p) const {
#pragma unroll
    for (int s = 0; s < kSub; ++s)
      if ((unsigned)p.page[s] >= (unsigned)num_pages) {
        if (lane == 0) atomicOr(err, (unsigned)kDevErrInput);
        p.page[s] = 0;  // any page that exists: the row's result is undefined, the read is not
      }
  }
  __device__ __forceinline__ Scales scales(const Pages& p) const {
    Scales s;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      s.k[i] = kF8 ? __ldg(ks + (long long)p.page[i] * Hkv) : 1.f;
      s.v[i] = kF8 ? __ldg(vs + (long long)p.page[i] * Hkv) : 1.f;
    }
    return s;
  }
  // Starts the copies of the tile at key0.
  __device__ __forceinline__ void issue(int key0, int cl, int ch, int sinks, const Pages& p, int stage) const {
    const uint32_t kd = ring + stage * kStageBytes, vd = kd + kTileBytes;
    const int chunk = lane % kChunks, row0 = lane / kChunks;
    const int pmask = (1 << p_shift) - 1;
    const bool inside = key0 >= cl && key0 + kKeys - 1 <= ch;
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      const long long page_off = p.page[s] * page_bytes + chunk * 16;
      const uint8_t* kp = kbase + page_off;
      const uint8_t* vp = vbase + page_off;
#pragma unroll
      for (int i = 0; i < kCopies / kSub; ++i) {
        const int row = 16 * s + row0 + i * kStep;
        int key = key0 + row;
        if (!inside) key = read_for(key, s, key0, cl, ch, sinks);
        const int src = (key & pmask) * kRowBytes;
        paged_cp16(kd + at(row, chunk), kp + src);
        paged_cp16(vd + at(row, chunk), vp + src);
      }
    }
  }

  // Scores of the tile in `stage` into the softmax, its values into o.
  __device__ __forceinline__ void consume(int key0, const Scales& sl, int stage, const PagedMask& mk) {
    const uint32_t kt = ring + stage * kStageBytes, vt = kt + kTileBytes;
    float sc[kSub][2][4];
#pragma unroll
    for (int s = 0; s < kSub; ++s)
#pragma unroll
      for (int n = 0; n < 2; ++n) sc[s][n][0] = sc[s][n][1] = sc[s][n][2] = sc[s][n][3] = 0.f;
    if constexpr (kF8) {
      // four accumulators in turn: a step of one chain waits for nothing
#pragma unroll
      for (int s0 = 0; s0 < kSub; s0 += 2)
#pragma unroll
        for (int i = 0; i < kKS / 4; ++i) {
          uint4 w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = paged_lds16(kt + at(16 * (s0 + (x >> 1)) + 8 * (x & 1) + g, c + 4 * i));
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              e4m3x4_to_f16x2(k == 0 ? w[x].x : k == 1 ? w[x].y : k == 2 ? w[x].z : w[x].w, b0, b1);
              paged_mma<true>(sc[s0 + (x >> 1)][x & 1], qa[4 * i + k], b0, b1);
            }
        }
    } else {
      const int mi = lane >> 3, ri = lane & 7;
      const int row = (mi >> 1) * 8 + ri;
#pragma unroll
      for (int t = 0; t < kSub; ++t)
#pragma unroll
        for (int s = 0; s < kKS; ++s) {
          uint32_t b00, b01, b10, b11;
          ptx::ldsm_x4(kt + at(16 * t + row, 2 * s + (mi & 1)), b00, b01, b10, b11);
          paged_mma<false>(sc[t][0], qa[s], b00, b01);
          paged_mma<false>(sc[t][1], qa[s], b10, b11);
        }
    }

    // ---- logits (log2 units), masks, maxima
    float t0 = -INFINITY, t1 = -INFINITY;  // tile maxima of rows g, g + 8
    float d0 = -INFINITY, d1 = -INFINITY;  // e4m3: maxima of logit + value exponent
    float mant[kSub], expo[kSub];
    const bool plain = (!kSinks || key0 >= mk.num_sinks) && key0 >= mk.all_lo && key0 + kKeys - 1 <= mk.all_hi &&
                       key0 + kKeys <= mk.len;
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      const float f0 = kF8 ? r0 * sl.k[s] : r0, f1 = kF8 ? r1 * sl.k[s] : r1;
      if constexpr (kCap) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          paged_capped2(sc[s][n][0], sc[s][n][1], f0, c1k, half_cap);
          if constexpr (kHi) paged_capped2(sc[s][n][2], sc[s][n][3], f1, c1k, half_cap);
        }
      }
      float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x0 = kCap ? sc[s][n][e] : sc[s][n][e] * f0;
          float x1 = !kHi ? -INFINITY : kCap ? sc[s][n][2 + e] : sc[s][n][2 + e] * f1;
          if (!plain) {
            const int key = key0 + 16 * s + 8 * n + 2 * c + e;
            const bool sink = kSinks && key < mk.num_sinks;
            if (sink) {
              x0 = fmaf(mk.bias0[key], kPagedLog2e, x0);
              if constexpr (kHi) x1 = fmaf(mk.bias0[mk.bias_step + key], kPagedLog2e, x1);
            }
            const bool here = key < mk.len;
            x0 = here && ((key >= mk.wlo0 && key <= mk.whi0) || sink) ? x0 : -INFINITY;
            if constexpr (kHi) x1 = here && ((key >= mk.wlo1 && key <= mk.whi1) || sink) ? x1 : -INFINITY;
          }
          sc[s][n][e] = x0;
          a0 = fmaxf(a0, x0);
          if constexpr (kHi) {
            sc[s][n][2 + e] = x1;
            a1 = fmaxf(a1, x1);
          }
        }
      t0 = fmaxf(t0, a0);
      t1 = fmaxf(t1, a1);
      if constexpr (kF8) {
        // value scale = mant 2^expo (0 for a zero or subnormal one)
        const uint32_t bits = __float_as_uint(sl.v[s]);
        const uint32_t field = (bits >> 23) & 255u;
        expo[s] = (float)((int)field - 127);
        mant[s] = field == 0 ? 0.f : __uint_as_float((bits & 0x807FFFFFu) | 0x3F800000u);
        d0 = fmaxf(d0, a0 + expo[s]);
        d1 = fmaxf(d1, a1 + expo[s]);
      }
    }
    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
    if constexpr (kHi) {
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
    }
    if constexpr (kF8) {
      d0 = fmaxf(d0, __shfl_xor_sync(0xffffffffu, d0, 1));
      d0 = fmaxf(d0, __shfl_xor_sync(0xffffffffu, d0, 2));
      if constexpr (kHi) {
        d1 = fmaxf(d1, __shfl_xor_sync(0xffffffffu, d1, 1));
        d1 = fmaxf(d1, __shfl_xor_sync(0xffffffffu, d1, 2));
      }
    }
    // ---- references: moved only when a tile passes them clearly
    auto raise = [](float& ref, float top, float slack) -> float {
      const bool move = top > ref + slack || (ref == -INFINITY && top != -INFINITY);
      const float now = move ? top : ref;
      const float alpha = (move && ref != -INFINITY) ? ptx::ex2(ref - now) : 1.f;
      ref = now;
      return alpha;
    };
    const float am0 = raise(m0, t0, kRaise), am1 = kHi ? raise(m1, t1, kRaise) : 1.f;
    l0 *= am0;
    l1 *= am1;
    float ao0, ao1;
    if constexpr (kF8) {
      ao0 = raise(u0, d0, 6.f);
      ao1 = kHi ? raise(u1, d1, 6.f) : 1.f;
    } else {
      ao0 = am0;
      ao1 = am1;
    }
    if (__any_sync(0xffffffffu, ao0 != 1.f || ao1 != 1.f)) {
#pragma unroll
      for (int i = 0; i < kNT; ++i) {
        o[i][0] *= ao0; o[i][1] *= ao0;
        if constexpr (kHi) { o[i][2] *= ao1; o[i][3] *= ao1; }
      }
    }
    const float mm0 = m0 == -INFINITY ? 0.f : m0, mm1 = m1 == -INFINITY ? 0.f : m1;
    uint32_t pa[kSub][4];
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      float w0 = 1.f, w1 = 1.f;
      if constexpr (kF8) {
        // The exponent's limit only bites for keys whose weight is below 2^-110.
        w0 = m0 == -INFINITY ? 0.f : mant[s] * ptx::ex2(fminf(expo[s] + m0 - u0 + 8.f, 126.f));
        w1 = m1 == -INFINITY ? 0.f : mant[s] * ptx::ex2(fminf(expo[s] + m1 - u1 + 8.f, 126.f));
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p00 = ptx::ex2(sc[s][n][0] - mm0), p01 = ptx::ex2(sc[s][n][1] - mm0);
        l0 += p00 + p01;
        pa[s][2 * n] = kF8 ? pack_f16x2(p00 * w0, p01 * w0) : pack_bf16x2(p00, p01);
        if constexpr (kHi) {
          const float p10 = ptx::ex2(sc[s][n][2] - mm1), p11 = ptx::ex2(sc[s][n][3] - mm1);
          l1 += p10 + p11;
          pa[s][2 * n + 1] = kF8 ? pack_f16x2(p10 * w1, p11 * w1) : pack_bf16x2(p10, p11);
        } else {
          pa[s][2 * n + 1] = 0u;
        }
      }
    }
    // ---- values
    if constexpr (kF8) {
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        const int k0 = 16 * s + 2 * c;
        constexpr int kWords = kD / 32;  // words of a thread's run of kD / 8 bytes
        uint32_t w[4][kWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = k0 + (i & 1) + (i >> 1) * 8;
          if constexpr (kD == 128) {
            const uint4 v = paged_lds16(vt + at(row, g));
            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
          } else {
            const uint2 v = paged_lds8(vt + at(row, g >> 1) + (g & 1) * 8);
            w[i][0] = v.x; w[i][1] = v.y;
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t b0, b1, b2, b3;
          e4m3x4_to_f16x2(__byte_perm(w[0][j], w[1][j], 0x5140), b0, b2);
          e4m3x4_to_f16x2(__byte_perm(w[2][j], w[3][j], 0x5140), b1, b3);
          paged_mma<true>(o[4 * j], pa[s], b0, b1);
          paged_mma<true>(o[4 * j + 1], pa[s], b2, b3);
          e4m3x4_to_f16x2(__byte_perm(w[0][j], w[1][j], 0x7362), b0, b2);
          e4m3x4_to_f16x2(__byte_perm(w[2][j], w[3][j], 0x7362), b1, b3);
          paged_mma<true>(o[4 * j + 2], pa[s], b0, b1);
          paged_mma<true>(o[4 * j + 3], pa[s], b2, b3);
        }
      }
    } else {
      const int mi = lane >> 3, ri = lane & 7;
      const int row = (mi & 1) * 8 + ri;
#pragma unroll
      for (int t = 0; t < kSub; ++t)
#pragma unroll
        for (int dn = 0; dn < kNT; dn += 2) {
          uint32_t b00, b01, b10, b11;
          ptx::ldsm_x4_t(vt + at(16 * t + row, dn + (mi >> 1)), b00, b01, b10, b11);
          paged_mma<false>(o[dn], pa[t], b00, b01);
          paged_mma<false>(o[dn + 1], pa[t], b10, b11);
        }
    }
  }

  // Tiles first, first + step, ... below count; key_of(t) is tile t's first key and
  // lim_of(t, cl, ch) the keys that may be read for it.  queries() brings the query rows in
  // while the first tile is on its way.
  template <class KeyOf, class LimOf, class Queries>
  __device__ __forceinline__ void walk(int first, int step, int count, KeyOf key_of, LimOf lim_of, Queries queries,
                                       const PagedMask& mk) {
    if (first >= count) return;
    int cl, ch;
    int key = key_of(first);
    lim_of(first, cl, ch);
    Pages pg = fetch(key, cl, ch, mk.num_sinks);
    check(pg);
    issue(key, cl, ch, mk.num_sinks, pg, 0);
    paged_cp_commit();
    Scales sl = scales(pg);
    int nkey = 0, ncl = 0, nch = 0;
    if (first + step < count) {
      nkey = key_of(first + step);
      lim_of(first + step, ncl, nch);
      pg = fetch(nkey, ncl, nch, mk.num_sinks);
    }
    queries();
    int stage = 0;
    for (int t = first; t < count; t += step) {
      Scales sn = sl;
      const int this_key = key;
      if (t + step < count) {
        check(pg);
        issue(nkey, ncl, nch, mk.num_sinks, pg, stage ^ 1);
        sn = scales(pg);
        key = nkey;
        if (t + 2 * step < count) {
          nkey = key_of(t + 2 * step);
          lim_of(t + 2 * step, ncl, nch);
          pg = fetch(nkey, ncl, nch, mk.num_sinks);
        }
      }
      paged_cp_commit();
      paged_cp_wait<1>();
      __syncwarp();
      consume(this_key, sl, stage, mk);
      __syncwarp();
      stage ^= 1;
      sl = sn;
    }
    paged_cp_wait<0>();
  }

  // The warp's state into the merge buffer: o rows at so[(warp * 16 + row) * kSmemRow +
  // 8 j + n], (max, sum, exponent that multiplies o) at sm[(warp * 16 + row) * 3].
  __device__ __forceinline__ void park(float* so, float* sm, int warp) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    float* a = so + (warp * 16 + g) * kSmemRow + 2 * c;
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      *reinterpret_cast<float2*>(a + 8 * j) = make_float2(o[j][0], o[j][1]);
      if constexpr (kHi)
        *reinterpret_cast<float2*>(a + 8 * kSmemRow + 8 * j) = make_float2(o[j][2], o[j][3]);
    }
    if (c == 0) {
      float* s = sm + (warp * 16 + g) * 3;
      s[0] = m0; s[1] = l0; s[2] = kF8 ? u0 - 8.f : m0;
      if constexpr (kHi) { s[24] = m1; s[25] = l1; s[26] = kF8 ? u1 - 8.f : m1; }
    }
  }
};

// Merge of the CTA's warps for row r: each warp's weight, the common max, the sum.
template <int kWarps>
__device__ __forceinline__ void paged_merge_row(const float* sm, int r, float* w) {
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm[(i * 16 + r) * 3]);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const float* s = sm + (i * 16 + r) * 3;
    const bool some = s[1] != 0.f;  // a NaN sum has to reach the output
    w[i] = some ? ptx::ex2(s[2] - M) : 0.f;
    L += some ? ptx::ex2(s[0] - M) * s[1] : 0.f;
  }
  w[kWarps] = M;
  w[kWarps + 1] = L;
}
// Dimensions d0 .. d0 + 7 of row r over the CTA's warps with weights w.
template <class W, int kWarps>
__device__ __forceinline__ void paged_merge_dims(const float* so, const float* w, int r, int d0, float (&o)[8]) {
  // e4m3: dimension kNT n + j is at 8 j + n
  const int n = d0 / W::kNT, j0 = d0 % W::kNT;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const float* s = so + (i * 16 + r) * W::kSmemRow;
    if (w[i] == 0.f) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(w[i], s[W::kCodes ? 8 * (j0 + e) + n : d0 + e], o[e]);
  }
}
__device__ __forceinline__ void paged_store_row(__nv_bfloat16* at, const float (&o)[8], float f) {
  *reinterpret_cast<uint4*>(at) = make_uint4(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f),
                                             pack_bf16x2(o[4] * f, o[5] * f), pack_bf16x2(o[6] * f, o[7] * f));
}
// LSE of a row from its max (log2 units) and sum.
__device__ __forceinline__ float paged_lse(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L)) * kPagedLn2;
}

// Result of an item whose tiles the `split` CTAs of a cluster shared: the CTA's warps merge
// in shared memory, the CTAs through distributed shared memory.  Row r < rows goes to row
// row_of(r) of out and lse, o times factor_of(r, sum).
constexpr int kPagedMaxSplit = 8;  // CTAs of a cluster, at most (the portable limit)
template <class W, int kWarps, int kD>
constexpr int paged_finish_bytes() {
  return (kWarps * 16 * (W::kSmemRow + 3) + 16 * (kD + kWarps + 2)) * 4;
}
template <class W, int kWarps, int kD, class RowOf, class FactorOf>
__device__ __forceinline__ void paged_cluster_finish(W& w, uint8_t* smem, int split, int part, int rows, RowOf row_of,
                                                     FactorOf factor_of, __nv_bfloat16* out, float* lse) {
  constexpr int kThreads = kWarps * 32;
  static_assert(kWarps % 2 == 0, "(max, sum) of a row are read as 8 bytes");
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  float* so = reinterpret_cast<float*>(smem);    // [warps][16][kSmemRow]
  float* sm = so + kWarps * 16 * W::kSmemRow;    // [warps][16][3]
  float* sw = sm + kWarps * 16 * 3;              // [16][warps + 2]: weights, max, sum
  float* sp = sw + 16 * (kWarps + 2);            // [16][kD] the CTA's o
  __syncthreads();
  w.park(so, sm, tid >> 5);
  __syncthreads();
  if (tid < rows) paged_merge_row<kWarps>(sm, tid, sw + tid * (kWarps + 2));
  __syncthreads();
  for (int x = tid; x < rows * (kD / 8); x += kThreads) {
    const int r = x / (kD / 8), d0 = x % (kD / 8) * 8;
    const float* wt = sw + r * (kWarps + 2);
    float O[8];
    paged_merge_dims<W, kWarps>(so, wt, r, d0, O);
    if (split == 1) {
      paged_store_row(out + row_of(r) * kD + d0, O, factor_of(r, wt[kWarps + 1]));
      if (lse != nullptr && d0 == 0) lse[row_of(r)] = paged_lse(wt[kWarps], wt[kWarps + 1]);
    } else {
      float4* to = reinterpret_cast<float4*>(sp + r * kD + d0);
      to[0] = make_float4(O[0], O[1], O[2], O[3]);
      to[1] = make_float4(O[4], O[5], O[6], O[7]);
    }
  }
  if (split == 1) return;
  cluster.sync();
  for (int x = part * kThreads + tid; x < rows * (kD / 4); x += split * kThreads) {
    const int r = x / (kD / 4), col = x % (kD / 4) * 4;
    float2 ml[kPagedMaxSplit];
    float4 v[kPagedMaxSplit];
#pragma unroll
    for (int i = 0; i < kPagedMaxSplit; ++i) {
      if (i >= split) break;
      ml[i] = *reinterpret_cast<const float2*>(cluster.map_shared_rank(sw, i) + r * (kWarps + 2) + kWarps);
      v[i] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sp, i) + r * kD + col);
    }
    float M = -INFINITY, L = 0.f, O[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPagedMaxSplit; ++i)
      if (i < split) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int i = 0; i < kPagedMaxSplit; ++i) {
      if (i >= split || ml[i].y == 0.f) continue;
      const float f = ptx::ex2(ml[i].x - M);
      L = fmaf(f, ml[i].y, L);
      O[0] = fmaf(f, v[i].x, O[0]); O[1] = fmaf(f, v[i].y, O[1]);
      O[2] = fmaf(f, v[i].z, O[2]); O[3] = fmaf(f, v[i].w, O[3]);
    }
    const float f = factor_of(r, L);
    *reinterpret_cast<uint2*>(out + row_of(r) * kD + col) =
        make_uint2(pack_bf16x2(O[0] * f, O[1] * f), pack_bf16x2(O[2] * f, O[3] * f));
    if (lse != nullptr && col == 0) lse[row_of(r)] = paged_lse(M, L);
  }
  cluster.sync();  // no CTA leaves while others read its shared memory
}

}  // namespace sba
