// Gradients of attention over SparseMask block bounds, for sm_103a: dQ, dK, dV.
//
// The forward (blocksparse_attn.cu) is softmax attention of each row (token, query head) over
// the keys that the bounds and the token mask leave it.  With P = exp(scale q.k - LSE) on those
// keys and Delta = rowsum(dO * O):
//   dV = P^T dO,   dS = P * (dO V^T - Delta),   dQ = scale dS K,   dK = scale dS^T Q.
// The probabilities are computed again from q, k and the LSE; nothing of size T x T is stored.
//
// Two or three launches, on one stream:
//   1. prep: Delta and the LSE of every row, negated and laid out [B, Hq, T], so that a tile's
//      128 values are one run; for each key tile the query blocks whose bounds reach it (the
//      bounds of the forward, turned round: dK and dV sum exactly the pairs that the forward
//      used, whatever the positions are).
//   2. the products.  dK / dV: a work item is a tile of 128 keys of one KV head; its steps are the
//      (query block, query head) pairs that reach it.  With few such tiles, those of a part of the
//      heads.  dQ: a work item is a query block of 128 tokens of one query head; its steps are the
//      128-key tiles of its bounds.  A block takes items of dK / dV until there are none left, then
//      items of dQ; blocks that find none of the first kind begin with dQ at once.
//   3. merge, if the heads are in parts: their dK and dV added up.
// S and dP are computed in both (7 products for the 5 of the formulas).  The other way, one pass
// with dQ added up in memory, needs B T Hq D fp32 sums cleared, added to by every key tile and
// rounded at the end, some 2.7 GB beside 1.9 GB of inputs on a batch of 4 x 16384 tokens (32 heads over 8
// of 128), and its sums come in an order set by timing.  Here every sum is held in tensor memory by one CTA,
// in an order that the bounds fix, so results are the same from run to run.
//
// Both halves of the kernel keep one tile of S and one of dP (128 x 128 fp32 each) in tensor memory
// and are arranged so that the tensor core always has a product to do while the softmax warps work
// on the other tile.  In steady state, per step:
//   dK / dV:  dV(i)   S(i+1)   dK(i)   dP(i+1)      softmax warps: dS(i) | P(i+1)
//   dQ:       S(i+1)  dQ(i)    dP(i+1)              softmax warps: dS(i) | P(i+1)
// What bounds them is the tensor core: the seven products over whole tiles of one row of 8192 (16 heads
// over 4) take 519 us at the rate of a large library product in a burst and 577 at its sustained one, the
// kernels 570 to 630 with prep, by the GPU's clocks; of a batch of 4 x 16384 behind a window of 1024, 1855
// and 2066, the kernels 2430 to 2600, 160 of it prep's.  Heads of 64 have half the products and the same
// softmax: there the chain of waits through the issuing warp is as long (2 x 4096, 12 heads over 4, 500
// and 300 tokens in view: 42 us at that rate, 103 taken).  Exponentials left out, or a second tile of S
// for heads of 64, change nothing.
// dK / dV works on S^T = K Q^T and dP^T = V dO^T (lanes = keys), whose P^T and dS^T go back over
// their own columns in bf16 and are the A operands of dV += P^T dO and dK += dS^T Q straight from
// tensor memory.  dQ holds Q and dO of the item in tensor memory as A operands as well, and dS
// over dP.
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "common.cuh"
#include "ptx.cuh"
#include "sync.cuh"

namespace sba {

static __device__ DevError g_err_bsb = {0u, 0u, 0};

namespace {

using namespace ptx;

// warp_wait behind one probe: most waits here find their phase over, and the step's chain of them is
// what it takes longest for (8192 tokens: dK / dV 372 -> 350 us, dQ 272 -> 257).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const Abort& ab, unsigned role,
                                           unsigned bar_id, int item) {
  if (__all_sync(0xffffffffu, mbar_test_wait(smem_u32(bar), parity))) return true;
  return warp_wait(bar, parity, ab, role, bar_id, item);
}

constexpr int kM = 128;           // query rows, and keys, of a tile
constexpr int kSub = 64;          // keys of a tile of the bounds
constexpr int kCols = 32;         // columns of a tile that one softmax warpgroup takes
constexpr int kSoftWarps = 16;    // four warpgroups
constexpr int kThreads = 128 + 32 * kSoftWarps;  // warp 0 loader, warp 1 MMA issuer, warps 4-19 softmax
constexpr int kItemSlots = 3;
constexpr float kLog2e = 1.4426950408889634f;

enum Role : unsigned { kRoleLoader = 1, kRoleMma = 2, kRoleSoftmax = 3 };
enum BarId : unsigned {
  kBarItemFull = 1, kBarItemEmpty, kBarQFull, kBarQEmpty, kBarDoFull, kBarDoEmpty, kBarKFull,
  kBarKEmpty, kBarVFull, kBarVEmpty, kBarSFull, kBarSEmpty, kBarDpFull, kBarPFull, kBarDsFull,
  kBarAccFull, kBarAccEmpty, kBarRowFull, kBarRowEmpty
};

struct Params {
  const __nv_bfloat16* out;
  const __nv_bfloat16* dout;
  const float* lse;
  const int* q_pos;
  const int* q_seg;
  const int* kv_pos;
  const int* kv_seg;
  const int* lower;
  const int* upper;
  const int* lower_full;
  const int* upper_full;
  float* nlse;      // [B, Hq, T]  -LSE in log2 units; -inf for rows without a key
  float* ndelta;    // [B, Hq, T]  -Delta
  int4* reach;      // [B, nb]     query blocks [x, y) reach this key tile, z of them; w: which halves (bits)
  int4* q_cols;     // [B, T / 32] 32 queries' positions and segments (see Cols)
  int4* kv_cols;    // [B, T / 32] ... and keys'
  int* next;        // next item of dK / dV, of dQ
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* parts;     // [n_split, dK and dV, B T, Hkv, D] sums of a part of the query heads, or null
  int n_split;      // parts of a KV head's query heads, each an item's
  int B, T, Hq, Hkv, G, nb, nbkv, tpb, causal, window_left, window_right, pad_id;
  float scale, scale_log2;
  int n_items_dq, n_items_kv;
  long long wait_limit;
};

// Key range of query block qblk of row b in 64-key tiles: [lo, up) visited, [lof, upf) without a
// token mask (as the forward reads the bounds).
struct Range {
  int lo, up, lof, upf;
};
__device__ __forceinline__ Range block_range(const Params& p, int b, int qblk) {
  const long long row = (long long)b * p.nb + qblk;
  Range r{0, 0, 0, 0};
  const int lo = max(p.lower[row], 0), up = min(p.upper[row], p.nbkv);
  if (up > lo) {
    r.lo = lo * p.tpb;
    r.up = up * p.tpb;
    // full blocks only matter inside [lo, up): clamped so that the products stay in range
    r.lof = min(max(p.lower_full[row], 0), p.nbkv) * p.tpb;
    r.upf = min(max(p.upper_full[row], 0), p.nbkv) * p.tpb;
  }
  return r;
}

// ------------------------------------------------------------------ 1. prep
// Blocks [0, n_delta): 32 tokens x 8 heads each, 16 bytes a thread and row (D / 8 threads a row),
// transposed through shared memory.  The blocks behind them: a warp for each key tile's reach, and one
// for each 32 queries and each 32 keys.
constexpr int kPrepTok = 32, kPrepHeads = 8;
template <int D>
__global__ void __launch_bounds__(256) bsa_bwd_prep_kernel(const Params p, int n_delta, int tok_groups,
                                                           int head_groups) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && tid < 2) p.next[tid] = 0;
  if (static_cast<int>(blockIdx.x) < n_delta) {
    __shared__ float sd[kPrepHeads][kPrepTok + 1], sl[kPrepHeads][kPrepTok + 1];
    const int hg = blockIdx.x % head_groups;
    const int tg = blockIdx.x / head_groups % tok_groups, b = blockIdx.x / head_groups / tok_groups;
    const int t0 = tg * kPrepTok, h0 = hg * kPrepHeads;
    constexpr int kLanes = D / 8;               // threads of a row
    constexpr int kRows = 256 / kLanes;         // rows of a pass
    constexpr int kPasses = kPrepTok * kPrepHeads / kRows;
    const int sub = tid / kLanes, part = tid % kLanes;
    uint4 ov[kPasses / 2], dv[kPasses / 2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < kPasses / 2; ++i) {
        const int r = (half * (kPasses / 2) + i) * kRows + sub, h = h0 + r % kPrepHeads;
        if (h < p.Hq) {
          const long long o = (((long long)b * p.T + t0 + r / kPrepHeads) * p.Hq + h) * D + part * 8;
          ov[i] = *reinterpret_cast<const uint4*>(p.out + o);
          dv[i] = *reinterpret_cast<const uint4*>(p.dout + o);
        }
      }
#pragma unroll
      for (int i = 0; i < kPasses / 2; ++i) {
        const int r = (half * (kPasses / 2) + i) * kRows + sub;
        const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&ov[i]);
        const __nv_bfloat162* d2 = reinterpret_cast<const __nv_bfloat162*>(&dv[i]);
        float acc = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 a = __bfloat1622float2(o2[u]), c = __bfloat1622float2(d2[u]);
          acc = fmaf(a.x, c.x, fmaf(a.y, c.y, acc));
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (part == 0) sd[r % kPrepHeads][r / kPrepHeads] = -acc;
      }
    }
    {
      const int t = tid / kPrepHeads, h = tid % kPrepHeads;
      if (h0 + h < p.Hq) sl[h][t] = p.lse[((long long)b * p.T + t0 + t) * p.Hq + h0 + h];
    }
    __syncthreads();
    const int h = tid / kPrepTok, t = tid % kPrepTok;
    if (h0 + h < p.Hq) {
      const long long o = ((long long)b * p.Hq + h0 + h) * p.T + t0 + t;
      const float l = sl[h][t];
      p.ndelta[o] = sd[h][t];
      // a row without a key: 2^(s - inf) = 0 for every key
      p.nlse[o] = l == -INFINITY ? -INFINITY : -l * kLog2e;
    }
    return;
  }
  int item = (blockIdx.x - n_delta) * 8 + warp;
  if (item >= p.B * p.nb) {
    // the warps behind those: 32 tokens' positions and segments, of the queries and of the keys
    item -= p.B * p.nb;
    const int groups = p.B * p.nb * (kM / 32);
    if (item >= 2 * groups) return;
    const bool keys = item >= groups;
    if (keys) item -= groups;
    const int pos = (keys ? p.kv_pos : p.q_pos)[item * 32 + lane], seg = (keys ? p.kv_seg : p.q_seg)[item * 32 + lane];
    const int p0 = __shfl_sync(0xffffffffu, pos, 0), s0 = __shfl_sync(0xffffffffu, seg, 0);
    const int s1 = __shfl_sync(0xffffffffu, seg, 31);
    const unsigned first = __ballot_sync(0xffffffffu, seg == s0);
    const int n0 = __popc(first);
    const bool simple = (long long)pos == (long long)p0 + lane && (seg == s0 || seg == s1) &&
                        first == (n0 >= 32 ? 0xffffffffu : (1u << n0) - 1u);
    const bool all = __all_sync(0xffffffffu, simple);
    if (lane == 0) (keys ? p.kv_cols : p.q_cols)[item] = make_int4(p0, s0, s1, all ? n0 : -1);
    return;
  }
  const int b = item / p.nb, kt = item % p.nb;
  int first = INT_MAX, last = -1, n = 0, halves = 0;
  for (int q0 = 0; q0 < p.nb; q0 += 32) {
    const int qb = q0 + lane;
    bool hit = false;
    if (qb < p.nb) {
      const Range r = block_range(p, b, qb);
      hit = r.lo < 2 * kt + 2 && r.up > 2 * kt;
      halves |= (r.lo <= 2 * kt && r.up > 2 * kt ? 1 : 0) | (r.lo <= 2 * kt + 1 && r.up > 2 * kt + 1 ? 2 : 0);
    }
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (m != 0u) {
      if (first == INT_MAX) first = q0 + __ffs(m) - 1;
      last = q0 + 31 - __clz(m);
      n += __popc(m);
    }
  }
  halves = __reduce_or_sync(0xffffffffu, halves);
  if (lane == 0) p.reach[item] = make_int4(n ? first : 0, last + 1, n, halves);
}

// ------------------------------------------------------------------ shared pieces
// Swizzled tiles start on 1024-byte boundaries, and the budget has no room to move them there; the
// whole block leaves, and the call is reported as failed, if the shared memory does not begin on one.
__device__ __forceinline__ bool swizzle_aligned(const void* smem) {
  if ((smem_u32(smem) & 1023u) == 0u) return true;
  atomicOr(&g_err_bsb.flags, kDevErrTimeout);
  return false;
}

// Byte offset (16-byte units) of K step kk of a K-major 128-byte-swizzled tile of 128 rows.
constexpr int kPanel = kM * 128;  // 128 rows x 64 elements
__device__ __forceinline__ uint64_t kmajor(int kk) {
  return static_cast<uint64_t>(((kk / 4) * kPanel + (kk % 4) * 32) >> 4);
}
// ... of a tile read with its 128 rows as the K dimension (16 rows a step).
__device__ __forceinline__ uint64_t mnmajor(int kk) { return static_cast<uint64_t>((kk * 16 * 128) >> 4); }
// bf16 columns of K step kk of a 128-column operand that lies in four parts, each over the first
// 16 of a warpgroup's 32 fp32 columns.
__device__ __forceinline__ uint32_t part_cols(int kk) { return (kk / 2) * kCols + (kk % 2) * 8; }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h2);
}

// What prep says of 32 neighbouring tokens: x the first one's position, y and z the first and the
// last one's segment, w how many have segment y, or -1 if they are not at consecutive positions in
// one run of segment y and one of z.
using Cols = int4;

// Columns of a warp that a row may pair with, as bits: same segment as the row's and a position in
// [lo, hi] (none if lo > hi).  Consecutive positions in two runs of one segment each (a document
// boundary, the start of padding) or in one give every row one interval; others are tested one by
// one.
__device__ __forceinline__ uint32_t keep_bits(const Cols& c, const int* pos, const int* segs, int lane, int lo, int hi,
                                              int seg) {
  uint32_t w = 0u;
  if (c.w >= 0) {
    if (lo <= hi && (seg == c.y || seg == c.z)) {
      const int jlo = static_cast<int>(min(max((long long)lo - c.x, seg == c.y ? 0LL : (long long)c.w), 32LL));
      const int jhi = static_cast<int>(max(min((long long)hi - c.x, seg == c.y ? c.w - 1LL : 31LL), -1LL));
      if (jlo <= jhi) w = (jhi >= 31 ? 0xffffffffu : (2u << jhi) - 1u) & (0xffffffffu << jlo);
    }
  } else {
    const int cp = pos[lane], cs = segs[lane];
    for (int j = 0; j < 32; ++j) {
      const int pj = __shfl_sync(0xffffffffu, cp, j), sj = __shfl_sync(0xffffffffu, cs, j);
      w |= (sj == seg && pj >= lo && pj <= hi) ? 1u << j : 0u;
    }
  }
  return w;
}

// The positions [lo, hi] that a token at `pos` pairs with: as a query `before` positions back and
// `after` on (-1: all), as a key the other way round.  Positions are 32-bit, so the ends may be
// clamped to that range.
__device__ __forceinline__ void in_view(int pos, int before, int after, int& lo, int& hi) {
  lo = before < 0 ? INT_MIN : static_cast<int>(max((long long)pos - before, (long long)INT_MIN));
  hi = after < 0 ? INT_MAX : static_cast<int>(min((long long)pos + after, (long long)INT_MAX));
}

// A row's columns are kChunks chunks of 16 bytes, a lane holds a row: transposes chunks against lanes in
// groups of kChunks, so that afterwards v[i] is this lane's chunk of row i of its group and a store of
// the group fills one row (a lane storing its own row's chunks writes half a sector to each of 32 lines
// at a time: with D = 128 some 2000 cycles for a tile of dQ, of the 25000 of its item).
template <int kChunks>
__device__ __forceinline__ void swap_chunks(uint32_t (&v)[kChunks][4], int lane) {
#pragma unroll
  for (int s = 1; s < kChunks; s <<= 1) {
    const bool odd = (lane & s) != 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (c & s) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[c][j] : v[c | s][j], s);
        if (odd) v[c][j] = got; else v[c | s][j] = got;
      }
    }
  }
}

// N = 32 or 16 fp32 accumulator columns of the lane row, times f, as bf16.  `to`: this lane's row, the
// rows of neighbouring lanes `stride` elements apart.
template <int N>
__device__ __forceinline__ void store_cols(uint32_t a, float f, __nv_bfloat16* to, long long stride, int lane) {
  float x[N];
  if constexpr (N == 32) tmem_ld_32x32b_x32(a, x); else tmem_ld_32x32b_x16(a, x);
  constexpr int kChunks = N / 8;
  uint32_t v[kChunks][4];
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[c][j] = pack_bf16(x[c * 8 + 2 * j] * f, x[c * 8 + 2 * j + 1] * f);
  swap_chunks(v, lane);
  const int me = lane % kChunks;
  __nv_bfloat16* row0 = to - me * stride + me * 8;
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    *reinterpret_cast<uint4*>(row0 + i * stride) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
}

// The same columns in fp32, for the merge; 16 at a time, as the caller holds P meanwhile (all 32 at once
// spilled: 8192 tokens of 16 heads in two parts 600 -> 840 us).
template <int N>
__device__ __forceinline__ void store_part(uint32_t a, float* to, long long stride, int lane) {
  const int me = lane % 4;
  float* row0 = to - me * stride + me * 4;
#pragma unroll 1
  for (int c = 0; c < N; c += 16) {
    float x[16];
    tmem_ld_32x32b_x16(a + c, x);
    uint32_t v[4][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j / 4][j % 4] = __float_as_uint(x[j]);
    swap_chunks(v, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(row0 + i * stride + c) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
  }
}

// ------------------------------------------------------------------ 2. the products: dK / dV
// What the loader says of a step, in the row ring's slot; flags also beside the Q ring's stage.
// kIn, kIn + 1: the bounds take in the tile's first and second 64 keys; kFull, kFull + 1: without a
// token mask (bit numbers).
// kSame: the query block of the step before.  From bit 16 on: the item's part.
enum StepFlag : int { kFirst = 1, kLast = 2, kEnd = 8, kIn = 4, kFull = 6, kSame = 256 };
struct alignas(16) StepRow {
  float nlse[kM];
  float ndelta[kM];
  int4 what;  // flags, first query and first key as rows of [B T], KV head
};

template <int D>
struct KvCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = kPanels * kPanel;   // 128 rows of K, V, Q or dO
  // Heads of 64 leave room to load further ahead, above all the rows, which a step's exponentials begin
  // with (2 x 4096 tokens, 12 heads over 4: 107.5 -> 102.8 us; four stages and six rows no more).
  static constexpr int kQStages = 3, kDoStages = D == 64 ? 3 : 2, kRowSlots = D == 64 ? 4 : 2;
  static constexpr int kDpBars = 2;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTile;
  static constexpr int kOffQ = 2 * kTile;
  static constexpr int kOffDo = kOffQ + kQStages * kTile;
  static constexpr int kOffRows = kOffDo + kDoStages * kTile;
  static constexpr int kDataEnd = kOffRows + kRowSlots * static_cast<int>(sizeof(StepRow));
  static constexpr int kNumBars = 4 + kQStages + kDoStages + 2 * kRowSlots + kDpBars + 6;
  static constexpr int kSCol = 0, kDpCol = 128, kDvCol = 256, kDkCol = 256 + D;
  static constexpr uint32_t kIdescS = make_idesc(128, kM, 1u, false, false);
  static constexpr uint32_t kIdescAcc = make_idesc(128, D, 1u, false, true);
};

// Items: key tiles of windows of kGroupWindow (row, KV head, part of its query heads) groups, tile by
// tile across the window.  Under causal masking early key tiles have the most steps, so a window's
// longest items go out first; the window bounds the Q and dO that the items running at once read.
constexpr int kGroupWindow = 8;
__device__ __forceinline__ void kv_item(const Params& p, int item, int& b, int& hkv, int& part, int& kt) {
  const int per = kGroupWindow * p.nb, win = item / per, rem = item - win * per;
  const int wsz = min(kGroupWindow, p.B * p.Hkv * p.n_split - win * kGroupWindow);
  kt = rem / wsz;
  int g = win * kGroupWindow + rem % wsz;
  part = g % p.n_split;
  g /= p.n_split;
  hkv = g % p.Hkv;
  b = g / p.Hkv;
}

// dK and dV of a tile of keys set to zero by one warp.
template <int D, bool kSplit>
__device__ __forceinline__ void zero_rows(const Params& p, int part, int key0, int hkv, int lane) {
  constexpr int kChunks = D / (kSplit ? 4 : 8);  // of 16 bytes a row
#pragma unroll 1
  for (int i = lane; i < kM * kChunks; i += 32) {
    const long long row = (long long)(key0 + i / kChunks) * p.Hkv + hkv;
    const int c = i % kChunks;
    if constexpr (kSplit) {
      const long long rows = (long long)p.B * p.T * p.Hkv;
      reinterpret_cast<uint4*>(p.parts + (part * 2 * rows + row) * D)[c] = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint4*>(p.parts + ((part * 2 + 1) * rows + row) * D)[c] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      reinterpret_cast<uint4*>(p.dk + row * D)[c] = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint4*>(p.dv + row * D)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <int D>
struct KvBars {
  uint64_t *k_full, *k_empty, *v_full, *v_empty, *q_full, *do_full, *row_full, *row_empty, *s_full, *p_full;
  uint64_t *dp_full, *ds_full, *acc_full, *acc_empty, *mma_done;  // dp_full by turns
  __device__ __forceinline__ explicit KvBars(uint64_t* bb) {
    using C = KvCfg<D>;
    k_full = bb;     bb += 1;
    k_empty = bb;    bb += 1;
    v_full = bb;     bb += 1;
    v_empty = bb;    bb += 1;
    q_full = bb;     bb += C::kQStages;
    do_full = bb;    bb += C::kDoStages;
    row_full = bb;   bb += C::kRowSlots;
    row_empty = bb;  bb += C::kRowSlots;
    s_full = bb;     bb += 1;
    p_full = bb;     bb += 1;
    dp_full = bb;    bb += C::kDpBars;
    ds_full = bb;    bb += 1;
    acc_full = bb;   bb += 1;
    acc_empty = bb;  bb += 1;
    mma_done = bb;
  }
  __device__ __forceinline__ void init() const {
    using C = KvCfg<D>;
    mbar_init(k_full, 1); mbar_init(k_empty, 1); mbar_init(v_full, 1); mbar_init(v_empty, 1);
    for (int i = 0; i < C::kQStages; ++i) mbar_init(&q_full[i], 1);
    for (int i = 0; i < C::kDoStages; ++i) mbar_init(&do_full[i], 1);
    for (int i = 0; i < C::kRowSlots; ++i) { mbar_init(&row_full[i], 1); mbar_init(&row_empty[i], kSoftWarps); }
    mbar_init(s_full, 1); mbar_init(p_full, kSoftWarps);
    for (int i = 0; i < C::kDpBars; ++i) mbar_init(&dp_full[i], 1);
    mbar_init(ds_full, kSoftWarps);
    mbar_init(acc_full, 1); mbar_init(acc_empty, kSoftWarps); mbar_init(mma_done, 1);
  }
};

// Boxes of 128 tokens of a head and 64 columns, of K and V also of 64 tokens.
struct Maps {
  CUtensorMap q, d_out, k, k_half, v_half;
};

// 64 tokens from token0 on of a head to the first half of a tile, those from token1 on to the second.  A half
// outside the bounds is read as zeros, by a box that begins behind the last token: its keys take part in the
// products with weight 0, and 0 times what they hold, which behind a row's last tile is another sequence's,
// need not be 0.  Two boxes for whole tiles too: they cost nothing beside one of 128.
template <int kPanels>
__device__ __forceinline__ void load_halves(uint8_t* to, const CUtensorMap& map, uint64_t* bar, int head, int token0,
                                            int token1) {
  mbar_arrive_expect_tx(bar, kPanels * kPanel);
#pragma unroll
  for (int pn = 0; pn < kPanels; ++pn) {
    tma_load_3d(to + pn * kPanel, &map, bar, pn * 64, head, token0);
    tma_load_3d(to + pn * kPanel + kPanel / 2, &map, bar, pn * 64, head, token1);
  }
}

// What a block's warps share besides the barriers.
struct Block {
  uint8_t* smem;
  uint32_t tmem;
  volatile int* abort_flag;
  volatile int* step_flags;  // dK / dV: per Q stage
};

// Items of dK / dV until there are none left.  kSplit: an item's sums are a part's, and leave in fp32 for
// the merge kernel.
template <int D, bool kSplit>
__device__ __forceinline__ void dkdv_items(const Maps& maps, const Params& p, const Block& block, const KvBars<D>& bars) {
  using C = KvCfg<D>;
  uint64_t *const k_full = bars.k_full, *const k_empty = bars.k_empty, *const v_full = bars.v_full,
           *const v_empty = bars.v_empty, *const q_full = bars.q_full, *const do_full = bars.do_full,
           *const row_full = bars.row_full, *const row_empty = bars.row_empty, *const s_full = bars.s_full,
           *const p_full = bars.p_full, *const dp_full = bars.dp_full, *const ds_full = bars.ds_full,
           *const acc_full = bars.acc_full, *const acc_empty = bars.acc_empty, *const mma_done = bars.mma_done;
  uint8_t* const smem = block.smem;
  volatile int* const step_flags = block.step_flags;
  const uint32_t tmem = block.tmem, smem_base = smem_u32(smem);
  const Abort ab{block.abort_flag, &g_err_bsb, 5u, p.wait_limit};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto row_at = [&](int slot) -> StepRow& {
    return *reinterpret_cast<StepRow*>(smem + C::kOffRows + slot * sizeof(StepRow));
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ loader
    // Steps are counted through all items.  The issuing warp's order is dV(n), S(n + 1), dK(n), dP(n + 1):
    // once dP(n) is there, the stages of Q and dO that steps before n read are free.  Step n's loads wait
    // for dP(n + 1 - stages), Q's of heads of 128, with a stage more than dO, for nothing, as dO(n - 1) did.
    // dP takes barriers by turns, so that a wait cannot take one phase for another: on the barrier waited
    // for, the next phase needs a dO that is not loaded yet, and the one before was over when the loads of
    // the step before began.
    auto dp_there = [&](int n, int item) {
      return n < 0 || wait_phase(&dp_full[n % C::kDpBars], (n / C::kDpBars) & 1, ab, kRoleLoader, kBarDoEmpty, item);
    };
    constexpr bool kTogether = C::kQStages == C::kDoStages;
    static_assert(C::kDpBars >= C::kDoStages - 1 && C::kQStages - C::kDoStages <= 1, "the order above");
    int qs = 0, ds = 0, rs = 0, n_loaded = 0;
    uint32_t qph = 0, dph = 0, rph = 0, kph = 0, vph = 0;
    // stages loaded and the phase of their last load (bit sets), for the drain
    uint32_t q_out = 0u, q_last = 0u, d_out = 0u, d_last = 0u, r_out = 0u, r_last = 0u;
    bool k_out = false, v_out = false;
    bool ok = true;
    while (ok) {
      int item = 0;
      if (lane == 0) item = atomicAdd(&p.next[0], 1);
      item = __shfl_sync(0xffffffffu, item, 0);
      if (item >= p.n_items_kv) {
        // no more: say so in both rings
        if (!wait_phase(&row_empty[rs], rph ^ 1, ab, kRoleLoader, kBarRowEmpty, item)) break;
        if (lane == 0) {
          row_at(rs).what.x = kEnd;
          mbar_arrive(&row_full[rs]);
        }
        __syncwarp();
        if (lane == 0) {
          step_flags[qs] = kEnd;
          mbar_arrive(&q_full[qs]);
        }
        __syncwarp();
        q_out &= ~(1u << qs);  // the last loads there were taken, and their phases are over
        r_out &= ~(1u << rs);
        break;
      }
      int b, hkv, part, kt;
      kv_item(p, item, b, hkv, part, kt);
      const int4 reach = p.reach[b * p.nb + kt];
      const int heads = p.G / p.n_split, n_steps = reach.z * heads;
      const int key0 = b * p.T + kt * kM;
      if (n_steps == 0) {
        // No query sees these keys.  The zeros are written from here, as many such tiles may follow one
        // another: in the row ring they would wait for the softmax warps, these in finish() for the last
        // item's sums, the MMA warp before those for the next item's Q, and that for this warp.
        zero_rows<D, kSplit>(p, part, key0, hkv, lane);
        continue;
      }
      int step = 0;
      for (int q0 = reach.x; q0 < reach.y && ok; q0 += 32) {
        Range mine{0, 0, 0, 0};
        if (q0 + lane < reach.y) mine = block_range(p, b, q0 + lane);
        int views = 0;  // of this lane's query block: kIn and kFull bits
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ti = 2 * kt + i;
          const bool in = ti >= mine.lo && ti < mine.up;
          views |= (in ? 1 << (kIn + i) : 0) | (in && ti >= mine.lof && ti < mine.upf ? 1 << (kFull + i) : 0);
        }
        unsigned hits = __ballot_sync(0xffffffffu, views != 0);
        while (hits != 0u && ok && step < n_steps) {
          const int at = __ffs(hits) - 1;
          hits &= hits - 1u;
          const int seen = __shfl_sync(0xffffffffu, views, at);
          const int qblk = q0 + at;
          for (int g = 0; g < heads; ++g, ++step) {
            const int h = hkv * p.G + part * heads + g, tok0 = b * p.T + qblk * kM;
            const int flags = (step == 0 ? kFirst : 0) | (step == n_steps - 1 ? kLast : 0);
            // the step's row goes out first: the softmax warps look it up before they free the tiles that
            // its other loads wait for
            if (!wait_phase(&row_empty[rs], rph ^ 1, ab, kRoleLoader, kBarRowEmpty, item)) { ok = false; break; }
            if (lane == 0) {
              StepRow& w = row_at(rs);
              w.what = make_int4(flags | seen | (g > 0 ? kSame : 0) | part << 16, tok0, key0, hkv);
              const long long o = ((long long)b * p.Hq + h) * p.T + qblk * kM;
              mbar_arrive_expect_tx(&row_full[rs], 2 * kM * 4);
              bulk_load(w.nlse, p.nlse + o, kM * 4, &row_full[rs]);
              bulk_load(w.ndelta, p.ndelta + o, kM * 4, &row_full[rs]);
            }
            __syncwarp();
            r_out |= 1u << rs; r_last = (r_last & ~(1u << rs)) | (rph << rs);
            if (++rs == C::kRowSlots) { rs = 0; rph ^= 1; }
            if (step == 0) {
              if (!wait_phase(k_empty, kph ^ 1, ab, kRoleLoader, kBarKEmpty, item)) { ok = false; break; }
              if (lane == 0) {
                mbar_arrive_expect_tx(k_full, C::kTile);
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                  tma_load_3d(smem + C::kOffK + pn * kPanel, &maps.k, k_full, pn * 64, hkv, key0);
              }
              k_out = true; kph ^= 1;
            }
            if (kTogether && !dp_there(n_loaded + 1 - C::kDoStages, item)) { ok = false; break; }
            if (lane == 0) {
              step_flags[qs] = flags;
              mbar_arrive_expect_tx(&q_full[qs], C::kTile);
#pragma unroll
              for (int pn = 0; pn < C::kPanels; ++pn)
                tma_load_3d(smem + C::kOffQ + qs * C::kTile + pn * kPanel, &maps.q, &q_full[qs], pn * 64, h, tok0);
            }
            q_out |= 1u << qs; q_last = (q_last & ~(1u << qs)) | (qph << qs);
            if (++qs == C::kQStages) { qs = 0; qph ^= 1; }
            if (step == 0) {
              if (!wait_phase(v_empty, vph ^ 1, ab, kRoleLoader, kBarVEmpty, item)) { ok = false; break; }
              if (lane == 0)
                load_halves<C::kPanels>(smem + C::kOffV, maps.v_half, v_full, hkv, (reach.w & 1) ? key0 : p.B * p.T,
                                        (reach.w & 2) ? key0 + kSub : p.B * p.T);
              v_out = true; vph ^= 1;
            }
            if (!kTogether && n_loaded >= 2 && !dp_there(n_loaded - 1, item)) { ok = false; break; }
            ++n_loaded;
            if (lane == 0) {
              mbar_arrive_expect_tx(&do_full[ds], C::kTile);
#pragma unroll
              for (int pn = 0; pn < C::kPanels; ++pn)
                tma_load_3d(smem + C::kOffDo + ds * C::kTile + pn * kPanel, &maps.d_out, &do_full[ds], pn * 64, h, tok0);
            }
            d_out |= 1u << ds; d_last = (d_last & ~(1u << ds)) | (dph << ds);
            if (++ds == C::kDoStages) { ds = 0; dph ^= 1; }
          }
        }
      }
    }
    // every copy issued has landed before the CTA may end
    if (lane == 0) {
      if (k_out) drain_wait(k_full, kph ^ 1);
      if (v_out) drain_wait(v_full, vph ^ 1);
      for (int i = 0; i < C::kQStages; ++i)
        if ((q_out >> i) & 1u) drain_wait(&q_full[i], (q_last >> i) & 1u);
      for (int i = 0; i < C::kDoStages; ++i)
        if ((d_out >> i) & 1u) drain_wait(&do_full[i], (d_last >> i) & 1u);
      for (int i = 0; i < C::kRowSlots; ++i)
        if ((r_out >> i) & 1u) drain_wait(&row_full[i], (r_last >> i) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // Converged warp, one elected lane issues.  Products of one thread run in the order issued,
    // so S(i + 1) may overwrite the P(i) that dV(i) reads, and dP(i + 1) the dS(i) of dK(i).
    const uint32_t leader = elect_one();
    const uint64_t k_desc = make_sdesc(smem_base + C::kOffK, 16, 1024, kLayoutSW128);
    const uint64_t v_desc = make_sdesc(smem_base + C::kOffV, 16, 1024, kLayoutSW128);
    const uint64_t q_desc = make_sdesc(smem_base + C::kOffQ, 16, 1024, kLayoutSW128);
    const uint64_t do_desc = make_sdesc(smem_base + C::kOffDo, 16, 1024, kLayoutSW128);
    const uint64_t qmn_desc = make_sdesc(smem_base + C::kOffQ, kPanel, 1024, kLayoutSW128);
    const uint64_t domn_desc = make_sdesc(smem_base + C::kOffDo, kPanel, 1024, kLayoutSW128);
    auto off = [](int stage) { return static_cast<uint64_t>((stage * C::kTile) >> 4); };
    int qs = 0, ds = 0, dpt = 0;             // stages of the next S and dP, barrier of dP
    uint32_t qph = 0, dph = 0, kph = 0, vph = 0, pph = 0, dsph = 0, accph = 0;
    // S of the step in Q stage qs; its flags, or kEnd
    auto issue_s = [&](int& flags) -> bool {
      if (!wait_phase(&q_full[qs], qph, ab, kRoleMma, kBarQFull, -1)) return false;
      flags = step_flags[qs];
      if (flags & kEnd) return true;
      if (flags & kFirst) {
        if (!wait_phase(k_full, kph, ab, kRoleMma, kBarKFull, -1)) return false;
        kph ^= 1;
      }
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_f16_ss_by(leader, tmem + C::kSCol, k_desc + kmajor(kk), q_desc + off(qs) + kmajor(kk), C::kIdescS,
                      kk > 0 ? 1u : 0u);
      mma_commit_by(leader, s_full);
      if (flags & kLast) mma_commit_by(leader, k_empty);
      if (++qs == C::kQStages) { qs = 0; qph ^= 1; }
      return true;
    };
    auto issue_dp = [&](int flags) -> bool {
      if (flags & kFirst) {
        if (!wait_phase(v_full, vph, ab, kRoleMma, kBarVFull, -1)) return false;
        vph ^= 1;
      }
      if (!wait_phase(&do_full[ds], dph, ab, kRoleMma, kBarDoFull, -1)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_f16_ss_by(leader, tmem + C::kDpCol, v_desc + kmajor(kk), do_desc + off(ds) + kmajor(kk), C::kIdescS,
                      kk > 0 ? 1u : 0u);
      mma_commit_by(leader, &dp_full[dpt]);
      if (++dpt == C::kDpBars) dpt = 0;
      if (flags & kLast) mma_commit_by(leader, v_empty);
      if (++ds == C::kDoStages) { ds = 0; dph ^= 1; }
      return true;
    };
    int cur = kEnd, next = kEnd;
    bool ok = issue_s(cur) && ((cur & kEnd) || issue_dp(cur));
    int cq = 0, cd = 0;  // stages of the current step's Q and dO
    while (ok && !(cur & kEnd)) {
      // dV += P^T dO
      if (!wait_phase(p_full, pph, ab, kRoleMma, kBarPFull, -1)) break;
      pph ^= 1;
      if (cur & kFirst) {
        if (!wait_phase(acc_empty, accph ^ 1, ab, kRoleMma, kBarAccEmpty, -1)) break;
        accph ^= 1;
      }
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kM / 16; ++kk)
        mma_f16_ts_by(leader, tmem + C::kDvCol, tmem + C::kSCol + part_cols(kk), domn_desc + off(cd) + mnmajor(kk),
                      C::kIdescAcc, ((cur & kFirst) && kk == 0) ? 0u : 1u);
      if (++cd == C::kDoStages) cd = 0;
      if (!issue_s(next)) break;
      // dK += dS^T Q
      if (!wait_phase(ds_full, dsph, ab, kRoleMma, kBarDsFull, -1)) break;
      dsph ^= 1;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kM / 16; ++kk)
        mma_f16_ts_by(leader, tmem + C::kDkCol, tmem + C::kDpCol + part_cols(kk), qmn_desc + off(cq) + mnmajor(kk),
                      C::kIdescAcc, ((cur & kFirst) && kk == 0) ? 0u : 1u);
      if (++cq == C::kQStages) cq = 0;
      if (cur & kLast) mma_commit_by(leader, acc_full);
      if (!(next & kEnd) && !issue_dp(next)) break;
      cur = next;
    }
    // every tcgen05 operation of this thread has finished once mma_done fires
    mma_commit_by(leader, mma_done);
    drain_wait(mma_done, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax / epilogue
    // Lane = key.  Warpgroup w takes the tile's queries 32 w .. 32 w + 31, and of dK and dV the
    // columns D / 4 w .. in the epilogue.
    const int w = (warp - 4) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t s_col = tmem + lane_off + C::kSCol + w * kCols, dp_col = tmem + lane_off + C::kDpCol + w * kCols;
    int rs = 0, next_rs = 0;       // row slots of the step and of the one looked up
    uint32_t rph = 0, sph = 0, dpph = 0, accph = 0;
    int dpt = 0;                   // barrier of the next dP
    int done_row = -1;             // this thread's key (times heads) of a finished item
    int lo = 1, hi = 0, seg = 0;   // query positions that may see this key, and its segment
    // The step to come: its flags, this thread's key, and the columns that pair with it.  Looked up
    // while the step before waits for dP.
    int flags = 0, row = 0;
    const int rows = p.B * p.T * p.Hkv;
    uint32_t keep = 0u;
    auto look_up = [&]() -> bool {
      if (!wait_phase(&row_full[next_rs], rph, ab, kRoleSoftmax, kBarRowFull, -1)) return false;
      const int4 st = row_at(next_rs).what;
      flags = st.x;
      if (++next_rs == C::kRowSlots) { next_rs = 0; rph ^= 1; }
      if (flags & kEnd) return true;
      if (flags & kFirst) {
        row = (st.z + r) * p.Hkv + st.w;
        if (kSplit) row += (flags >> 16) * 2 * rows;  // below 4 x 152 x 2 x 128
      }
      if (flags & kSame) return true;
      const int mine = flags >> (q4 >> 1);  // this warp's 64 keys
      const bool in = (mine >> kIn) & 1, full = (mine >> kFull) & 1;
      Cols cols{};
      const int col = st.y + w * kCols;
      if (in && !full) cols = p.q_cols[col / 32];
      if (flags & kFirst) {
        // key k is seen from position q iff k <= q (causal), q - k <= left, k - q <= right
        const int key = st.z + r;
        in_view(p.kv_pos[key], p.causal ? 0 : p.window_right, p.window_left, lo, hi);
        seg = p.kv_seg[key];
        if (seg == p.pad_id) { lo = 1; hi = 0; }
      }
      keep = full ? 0xffffffffu : (in ? keep_bits(cols, p.q_pos + col, p.q_seg + col, lane, lo, hi, seg) : 0u);
      return true;
    };
    auto free_row = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&row_empty[rs]);
      if (++rs == C::kRowSlots) rs = 0;
    };
    const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
    auto finish = [&]() -> bool {
      if (!wait_phase(acc_full, accph, ab, kRoleSoftmax, kBarAccFull, row)) return false;
      accph ^= 1;
      tc_fence_after();
      const long long to = (long long)done_row * D + w * (D / 4), stride = (long long)p.Hkv * D;
      if constexpr (kSplit) {
        store_part<D / 4>(tmem + lane_off + C::kDvCol + w * (D / 4), p.parts + (long long)rows * D + to, stride, lane);
        store_part<D / 4>(tmem + lane_off + C::kDkCol + w * (D / 4), p.parts + to, stride, lane);
      } else {
        store_cols<D / 4>(tmem + lane_off + C::kDvCol + w * (D / 4), 1.f, p.dv + to, stride, lane);
        store_cols<D / 4>(tmem + lane_off + C::kDkCol + w * (D / 4), p.scale, p.dk + to, stride, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      done_row = -1;
      return true;
    };
    // P of a step, then the step behind it is looked up, then dS: look_up and finish are each written
    // once, as the loop's code has to share the instruction caches with the other warps' (two copies of
    // finish: dK / dV 350 -> 403 us at 8192 tokens).
    bool work = false;             // a step is in hand
    while (true) {
      float x[kCols];
      const bool last = work && (flags & kLast);
      const int this_row = row;
      if (work) {
        if (!wait_phase(s_full, sph, ab, kRoleSoftmax, kBarSFull, row)) break;
        sph ^= 1;
        tc_fence_after();
        tmem_ld_32x32b_x32(s_col, x);
        {
          const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(row_at(rs).nlse + w * kCols);
#pragma unroll
          for (int j = 0; j < kCols; j += 4) {
            const ulonglong2 l4 = nl[j / 4];
            float a0, a1, a2, a3;
            unpack_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), scale2, l4.x), a0, a1);
            unpack_f32x2(fma_f32x2(pack_f32x2(x[j + 2], x[j + 3]), scale2, l4.y), a2, a3);
            x[j] = ex2(a0); x[j + 1] = ex2(a1); x[j + 2] = ex2(a2); x[j + 3] = ex2(a3);
          }
        }
        if (__any_sync(0xffffffffu, keep != 0xffffffffu)) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) x[j] = (keep & (1u << j)) ? x[j] : 0.f;
        }
        {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
          tmem_st_32x32b_x16_u_nw(s_col, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (__builtin_expect(done_row >= 0, 0) && !finish()) break;
      if (flags & kEnd) break;
      if (!look_up()) break;
      if (work) {
        if (!wait_phase(&dp_full[dpt], dpph, ab, kRoleSoftmax, kBarDpFull, row)) break;
        if (++dpt == C::kDpBars) { dpt = 0; dpph ^= 1; }
        tc_fence_after();
        float y[kCols];
        tmem_ld_32x32b_x32(dp_col, y);
        {
          const ulonglong2* nd = reinterpret_cast<const ulonglong2*>(row_at(rs).ndelta + w * kCols);
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const int i = 2 * j;
            const ulonglong2 d4 = nd[i / 4];
            float a0, a1, a2, a3;
            unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(y[i], y[i + 1]), d4.x), pack_f32x2(x[i], x[i + 1])), a0, a1);
            unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(y[i + 2], y[i + 3]), d4.y), pack_f32x2(x[i + 2], x[i + 3])), a2, a3);
            pk[j] = pack_bf16(a0, a1);
            pk[j + 1] = pack_bf16(a2, a3);
          }
          tmem_st_32x32b_x16_u_nw(dp_col, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
        free_row();
      }
      if (last) done_row = this_row;
      work = !(flags & kEnd);
    }
  }
}

// ------------------------------------------------------------------ dQ
struct DqItem {
  int b, h, qblk, n_steps;  // n_steps -1: no more items
  Range r;
};

template <int D>
struct DqCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = kPanels * kPanel;
  static constexpr int kKStages = 3, kVStages = 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffDo = kTile;
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kKStages * kTile;
  static constexpr int kItemBytes = (static_cast<int>(sizeof(DqItem)) + 15) & ~15;
  static constexpr int kOffItems = kOffV + kVStages * kTile;
  static constexpr int kDataEnd = kOffItems + kItemSlots * kItemBytes;
  static constexpr int kNumBars = 2 * kItemSlots + 4 + kKStages + kVStages + 8;
  static constexpr int kSCol = 0, kDpCol = 128, kDqCol = 256, kQCol = 256 + D, kDoCol = kQCol + D / 2;
  static constexpr uint32_t kIdescS = make_idesc(128, kM, 1u, false, false);
  static constexpr uint32_t kIdescAcc = make_idesc(128, D, 1u, false, true);
  static_assert(kDoCol + D / 2 <= 512, "tensor memory budget");
};

template <int D>
struct DqBars {
  uint64_t *item_full, *item_empty, *q_full, *q_empty, *do_full, *do_empty, *k_full, *v_full, *s_full, *s_empty;
  uint64_t *dp_full, *ds_full, *dq_full, *dq_empty, *mma_done;  // dp_full by turns
  __device__ __forceinline__ explicit DqBars(uint64_t* bb) {
    using C = DqCfg<D>;
    item_full = bb;  bb += kItemSlots;
    item_empty = bb; bb += kItemSlots;
    q_full = bb;     bb += 1;
    q_empty = bb;    bb += 1;
    do_full = bb;    bb += 1;
    do_empty = bb;   bb += 1;
    k_full = bb;     bb += C::kKStages;
    v_full = bb;     bb += C::kVStages;
    s_full = bb;     bb += 1;
    s_empty = bb;    bb += 1;
    dp_full = bb;    bb += 2;
    ds_full = bb;    bb += 1;
    dq_full = bb;    bb += 1;
    dq_empty = bb;   bb += 1;
    mma_done = bb;
  }
  __device__ __forceinline__ void init() const {
    using C = DqCfg<D>;
    // an item slot is read by the MMA warp and the softmax warps
    for (int i = 0; i < kItemSlots; ++i) { mbar_init(&item_full[i], 1); mbar_init(&item_empty[i], 1 + kSoftWarps); }
    mbar_init(q_full, 1); mbar_init(q_empty, 1); mbar_init(do_full, 1); mbar_init(do_empty, 1);
    for (int i = 0; i < C::kKStages; ++i) mbar_init(&k_full[i], 1);
    for (int i = 0; i < C::kVStages; ++i) mbar_init(&v_full[i], 1);
    mbar_init(s_full, 1); mbar_init(s_empty, kSoftWarps); mbar_init(&dp_full[0], 1); mbar_init(&dp_full[1], 1);
    mbar_init(ds_full, kSoftWarps);
    mbar_init(dq_full, 1); mbar_init(dq_empty, kSoftWarps); mbar_init(mma_done, 1);
  }
};

// Items of dQ until there are none left.
template <int D>
__device__ __forceinline__ void dq_items(const Maps& maps, const Params& p, const Block& block, const DqBars<D>& bars) {
  using C = DqCfg<D>;
  uint64_t *const item_full = bars.item_full, *const item_empty = bars.item_empty, *const q_full = bars.q_full,
           *const q_empty = bars.q_empty, *const do_full = bars.do_full, *const do_empty = bars.do_empty,
           *const k_full = bars.k_full, *const v_full = bars.v_full, *const s_full = bars.s_full,
           *const s_empty = bars.s_empty, *const dp_full = bars.dp_full, *const ds_full = bars.ds_full,
           *const dq_full = bars.dq_full, *const dq_empty = bars.dq_empty, *const mma_done = bars.mma_done;
  uint8_t* const smem = block.smem;
  const uint32_t tmem = block.tmem, smem_base = smem_u32(smem);
  const Abort ab{block.abort_flag, &g_err_bsb, 6u, p.wait_limit};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto item_at = [&](int slot) -> DqItem& {
    return *reinterpret_cast<DqItem*>(smem + C::kOffItems + slot * C::kItemBytes);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ loader
    // dP(n - 2) read V(n - 2) and follows dQ(n - 3), which read K(n - 3): once it is there both stages
    // of step n are free.  dP(n), whose phase comes next on the same barrier, waits for V(n).
    static_assert(C::kVStages == 2 && C::kKStages == 3, "the order above");
    int islot = 0, ks = 0, vs = 0, n_loaded = 0;
    uint32_t iph = 0, qph = 0, kph = 0, vph = 0;
    uint32_t k_out = 0u, k_last = 0u, v_out = 0u, v_last = 0u;
    uint32_t q_last = 2u, do_last = 2u;  // phase of the last load, 2: none yet
    bool ok = true;
    while (ok) {
      // from the last query block down: under causal masking later ones have more keys
      int item = 0;
      if (lane == 0) item = atomicAdd(&p.next[1], 1);
      item = __shfl_sync(0xffffffffu, item, 0);
      if (!wait_phase(&item_empty[islot], iph ^ 1, ab, kRoleLoader, kBarItemEmpty, item)) break;
      if (item >= p.n_items_dq) {
        if (lane == 0) {
          item_at(islot).n_steps = -1;
          mbar_arrive(&item_full[islot]);
        }
        __syncwarp();
        break;
      }
      const int h = item % p.Hq, b = item / p.Hq % p.B, qblk = p.nb - 1 - item / p.Hq / p.B, hkv = h / p.G;
      const Range r = block_range(p, b, qblk);
      const int n = (r.up - r.lo + 1) / 2;
      if (lane == 0) {
        DqItem& it = item_at(islot);
        it.b = b; it.h = h; it.qblk = qblk; it.n_steps = n; it.r = r;
        mbar_arrive(&item_full[islot]);
      }
      __syncwarp();
      if (++islot == kItemSlots) { islot = 0; iph ^= 1; }
      if (n == 0) continue;
      const int tok0 = b * p.T + qblk * kM;
      for (int t = 0; t < n && ok; ++t) {
        const int key0 = b * p.T + (r.lo + 2 * t) * kSub;
        if (t == 0) {
          if (!wait_phase(q_empty, qph ^ 1, ab, kRoleLoader, kBarQEmpty, item)) { ok = false; break; }
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full, C::kTile);
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
              tma_load_3d(smem + C::kOffQ + pn * kPanel, &maps.q, q_full, pn * 64, h, tok0);
          }
          q_last = qph;
        }
        if (n_loaded >= 2 &&
            !wait_phase(&dp_full[n_loaded & 1], ((n_loaded >> 1) - 1) & 1, ab, kRoleLoader, kBarKEmpty, item)) {
          ok = false;
          break;
        }
        ++n_loaded;
        const int key1 = r.lo + 2 * t + 1 < r.up ? key0 + kSub : p.B * p.T;
        if (lane == 0) load_halves<C::kPanels>(smem + C::kOffK + ks * C::kTile, maps.k_half, &k_full[ks], hkv, key0, key1);
        k_out |= 1u << ks; k_last = (k_last & ~(1u << ks)) | (kph << ks);
        if (++ks == C::kKStages) { ks = 0; kph ^= 1; }
        if (t == 0) {
          if (!wait_phase(do_empty, qph ^ 1, ab, kRoleLoader, kBarDoEmpty, item)) { ok = false; break; }
          if (lane == 0) {
            mbar_arrive_expect_tx(do_full, C::kTile);
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
              tma_load_3d(smem + C::kOffDo + pn * kPanel, &maps.d_out, do_full, pn * 64, h, tok0);
          }
          do_last = qph; qph ^= 1;
        }
        if (lane == 0) load_halves<C::kPanels>(smem + C::kOffV + vs * C::kTile, maps.v_half, &v_full[vs], hkv, key0, key1);
        v_out |= 1u << vs; v_last = (v_last & ~(1u << vs)) | (vph << vs);
        if (++vs == C::kVStages) { vs = 0; vph ^= 1; }
      }
    }
    if (lane == 0) {
      for (int i = 0; i < C::kKStages; ++i)
        if ((k_out >> i) & 1u) drain_wait(&k_full[i], (k_last >> i) & 1u);
      for (int i = 0; i < C::kVStages; ++i)
        if ((v_out >> i) & 1u) drain_wait(&v_full[i], (v_last >> i) & 1u);
      if (q_last < 2u) drain_wait(q_full, q_last);
      if (do_last < 2u) drain_wait(do_full, do_last);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t leader = elect_one();
    const uint64_t q_desc = make_sdesc(smem_base + C::kOffQ, 16, 1024, kLayoutSW128);
    const uint64_t do_desc = make_sdesc(smem_base + C::kOffDo, 16, 1024, kLayoutSW128);
    const uint64_t k_desc = make_sdesc(smem_base + C::kOffK, 16, 1024, kLayoutSW128);
    const uint64_t kmn_desc = make_sdesc(smem_base + C::kOffK, kPanel, 1024, kLayoutSW128);
    const uint64_t v_desc = make_sdesc(smem_base + C::kOffV, 16, 1024, kLayoutSW128);
    auto off = [](int stage) { return static_cast<uint64_t>((stage * C::kTile) >> 4); };
    int islot = 0, ks = 0, vs = 0, left = 0;   // left: steps of the item not yet taken
    uint32_t iph = 0, qph = 0, doph = 0, kph = 0, vph = 0, seph = 0, dsph = 0, dqph = 0;
    // the next step's flags: kFirst, kLast, or kEnd
    auto next_step = [&](int& flags) -> bool {
      flags = 0;
      while (left == 0) {
        if (!wait_phase(&item_full[islot], iph, ab, kRoleMma, kBarItemFull, -1)) return false;
        left = item_at(islot).n_steps;
        __syncwarp();
        if (left < 0) { flags = kEnd; return true; }
        if (lane == 0) mbar_arrive(&item_empty[islot]);
        if (++islot == kItemSlots) { islot = 0; iph ^= 1; }
        flags = kFirst;
      }
      if (--left == 0) flags |= kLast;
      return true;
    };
    // S = Q K^T into its columns, which the softmax warps have read
    auto issue_s = [&](int flags) -> bool {
      if (flags & kFirst) {
        // Q of the item into tensor memory; the previous item's products that read it are done,
        // as the softmax warps have seen the last of them
        if (!wait_phase(q_full, qph, ab, kRoleMma, kBarQFull, -1)) return false;
        qph ^= 1;
      }
      if (!wait_phase(&k_full[ks], kph, ab, kRoleMma, kBarKFull, -1) ||
          !wait_phase(s_empty, seph ^ 1, ab, kRoleMma, kBarSEmpty, -1))
        return false;
      seph ^= 1;
      tc_fence_after();
      if (flags & kFirst) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) tmem_cp_128x256b_by(leader, tmem + C::kQCol + kk * 8, q_desc + kmajor(kk));
        mma_commit_by(leader, q_empty);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_f16_ts_by(leader, tmem + C::kSCol, tmem + C::kQCol + kk * 8, k_desc + off(ks) + kmajor(kk), C::kIdescS,
                      kk > 0 ? 1u : 0u);
      mma_commit_by(leader, s_full);
      if (++ks == C::kKStages) { ks = 0; kph ^= 1; }
      return true;
    };
    // dP = dO V^T over the dS that the product before it has read
    auto issue_dp = [&](int flags) -> bool {
      if (flags & kFirst) {
        if (!wait_phase(do_full, doph, ab, kRoleMma, kBarDoFull, -1)) return false;
        doph ^= 1;
      }
      if (!wait_phase(&v_full[vs], vph, ab, kRoleMma, kBarVFull, -1)) return false;
      tc_fence_after();
      if (flags & kFirst) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) tmem_cp_128x256b_by(leader, tmem + C::kDoCol + kk * 8, do_desc + kmajor(kk));
        mma_commit_by(leader, do_empty);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_f16_ts_by(leader, tmem + C::kDpCol, tmem + C::kDoCol + kk * 8, v_desc + off(vs) + kmajor(kk), C::kIdescS,
                      kk > 0 ? 1u : 0u);
      mma_commit_by(leader, &dp_full[vs]);
      if (++vs == C::kVStages) { vs = 0; vph ^= 1; }
      return true;
    };
    int cur = kEnd, next = kEnd, ck = 0;  // ck: stage of the current step's K
    bool ok = next_step(cur) && ((cur & kEnd) || (issue_s(cur) && issue_dp(cur)));
    while (ok && !(cur & kEnd)) {
      if (!next_step(next)) break;
      if (!(next & kEnd) && !issue_s(next)) break;
      // dQ += dS K
      if (!wait_phase(ds_full, dsph, ab, kRoleMma, kBarDsFull, -1)) break;
      dsph ^= 1;
      if (cur & kFirst) {
        if (!wait_phase(dq_empty, dqph ^ 1, ab, kRoleMma, kBarAccEmpty, -1)) break;
        dqph ^= 1;
      }
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kM / 16; ++kk)
        mma_f16_ts_by(leader, tmem + C::kDqCol, tmem + C::kDpCol + part_cols(kk), kmn_desc + off(ck) + mnmajor(kk),
                      C::kIdescAcc, ((cur & kFirst) && kk == 0) ? 0u : 1u);
      if (++ck == C::kKStages) ck = 0;
      if (cur & kLast) mma_commit_by(leader, dq_full);
      if (!(next & kEnd) && !issue_dp(next)) break;
      cur = next;
    }
    mma_commit_by(leader, mma_done);
    drain_wait(mma_done, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax / epilogue
    // Lane = query row.  Warpgroup w takes the step's keys 32 w .. 32 w + 31 (half of a 64-key tile
    // of the bounds), and of dQ the columns D / 4 w .. in the epilogue.
    const int w = (warp - 4) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t s_col = tmem + lane_off + C::kSCol + w * kCols, dp_col = tmem + lane_off + C::kDpCol + w * kCols;
    int islot = 0;
    uint32_t iph = 0, sph = 0, dpph = 0, dpt = 0, dqph = 0;
    int done_row = -1;             // this thread's row (token times heads) of a finished item
    const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
    auto finish = [&]() -> bool {
      if (!wait_phase(dq_full, dqph, ab, kRoleSoftmax, kBarAccFull, done_row)) return false;
      dqph ^= 1;
      tc_fence_after();
      store_cols<D / 4>(tmem + lane_off + C::kDqCol + w * (D / 4), p.scale,
                        p.dq + (long long)done_row * D + w * (D / 4), (long long)p.Hq * D, lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dq_empty);
      done_row = -1;
      return true;
    };
    // The item: steps left, this thread's row, the key positions that it sees and its segment, the
    // first key of the step's columns and the tiles of the bounds from there on.  The next one is
    // looked up within the last step, once that needs no more of these than ndelta.
    int left = 0, row = 0, lo = 0, hi = 0, seg = 0, col = 0;
    Range rg{};
    float nlse = 0.f, ndelta = 0.f, ndelta_next = 0.f;
    auto look_up = [&]() -> bool {
      while (true) {
        if (!wait_phase(&item_full[islot], iph, ab, kRoleSoftmax, kBarItemFull, -1)) return false;
        const DqItem& it = item_at(islot);
        left = it.n_steps;
        const int b = it.b, h = it.h, t0 = it.qblk * kM + r;
        rg = it.r;
        __syncwarp();
        if (left < 0) return true;
        if (lane == 0) mbar_arrive(&item_empty[islot]);
        if (++islot == kItemSlots) { islot = 0; iph ^= 1; }
        const int tok = b * p.T + t0;
        row = tok * p.Hq + h;
        if (left == 0) {
          // a query block without keys
#pragma unroll
          for (int j = 0; j < D / 4; j += 8)
            *reinterpret_cast<uint4*>(p.dq + (long long)row * D + w * (D / 4) + j) = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        const int o = (b * p.Hq + h) * p.T + t0;
        nlse = p.nlse[o];
        ndelta_next = p.ndelta[o];
        seg = p.q_seg[tok];
        in_view(p.q_pos[tok], p.window_left, p.causal ? 0 : p.window_right, lo, hi);
        if (seg == p.pad_id) { lo = 1; hi = 0; }
        rg.lo += w >> 1;  // this warp's 64-key tile of the step
        col = b * p.T + rg.lo * kSub + (w & 1) * kCols;
        return true;
      }
    };
    // as in dK / dV: P of a step, what comes next, dS
    bool work = false;
    while (true) {
      float x[kCols];
      if (work) {
        const bool in = rg.lo < rg.up, full = in && rg.lo >= rg.lof && rg.lo < rg.upf;
        Cols cols{};
        if (in && !full) cols = p.kv_cols[col / 32];
        if (!wait_phase(s_full, sph, ab, kRoleSoftmax, kBarSFull, row)) break;
        sph ^= 1;
        tc_fence_after();
        tmem_ld_32x32b_x32(s_col, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        {
          const uint64_t nl2 = pack_f32x2(nlse, nlse);
#pragma unroll
          for (int j = 0; j < kCols; j += 2) {
            float a0, a1;
            unpack_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), scale2, nl2), a0, a1);
            x[j] = ex2(a0);
            x[j + 1] = ex2(a1);
          }
        }
        if (!full) {
          const uint32_t keep = in ? keep_bits(cols, p.kv_pos + col, p.kv_seg + col, lane, lo, hi, seg) : 0u;
#pragma unroll
          for (int j = 0; j < kCols; ++j) x[j] = (keep & (1u << j)) ? x[j] : 0.f;
        }
      }
      if (__builtin_expect(done_row >= 0, 0) && !finish()) break;
      if (left < 0) break;
      const bool had = work, last = work && --left == 0;
      if (last) done_row = row;
      if (last || !work) {
        if (!look_up()) break;
        work = left > 0;
      } else {
        rg.lo += 2;
        col += kM;
      }
      if (had) {
        if (!wait_phase(&dp_full[dpt], dpph, ab, kRoleSoftmax, kBarDpFull, row)) break;
        dpph ^= dpt;
        dpt ^= 1;
        tc_fence_after();
        float y[kCols];
        tmem_ld_32x32b_x32(dp_col, y);
        {
          const uint64_t nd2 = pack_f32x2(ndelta, ndelta);
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int i = 2 * j;
            float a0, a1;
            unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(y[i], y[i + 1]), nd2), pack_f32x2(x[i], x[i + 1])), a0, a1);
            pk[j] = pack_bf16(a0, a1);
          }
          tmem_st_32x32b_x16_u_nw(dp_col, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (last || !had) ndelta = ndelta_next;
    }
  }
}

// ------------------------------------------------------------------ both
template <int D>
struct Cfg {
  using Kv = KvCfg<D>;
  using Dq = DqCfg<D>;
  static constexpr int kOffKvBars = Kv::kDataEnd > Dq::kDataEnd ? Kv::kDataEnd : Dq::kDataEnd;
  static constexpr int kOffDqBars = kOffKvBars + Kv::kNumBars * 8;
  static constexpr int kOffMisc = kOffDqBars + Dq::kNumBars * 8;  // tmem address, abort flag, step flags
  static constexpr int kUsed = kOffMisc + 8 + 4 * Kv::kQStages;
  // At least half of an SM's shared memory: one CTA an SM, as each holds all tensor memory.
  static constexpr int kSmemBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  // dK / dV's rows are read by the warps; copies of dQ do not go there, so that no proxy fence is due
  static_assert(Kv::kOffRows >= Dq::kOffItems, "rows behind the tiles of dQ");
};

// dK / dV and dQ are one kernel, set up while prep runs, so that every block waits for prep itself before
// it reads what prep left.  As two kernels, the second of them started ahead of the first one's end to fill
// its idle SMs, the second has no such wait that would not also be one for the end of the first.
template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
bsa_bwd_kernel(const __grid_constant__ Maps maps, const Params p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!swizzle_aligned(smem)) return;
  const KvBars<D> kv_bars(reinterpret_cast<uint64_t*>(smem + C::kOffKvBars));
  const DqBars<D> dq_bars(reinterpret_cast<uint64_t*>(smem + C::kOffDqBars));
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    kv_bars.init();
    dq_bars.init();
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.d_out);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.k_half);
    tma_prefetch_desc(&maps.v_half);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Block block{smem, *tmem_holder, abort_flag, reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8)};
  // prep's results (and all that ran before it) are there
  asm volatile("griddepcontrol.wait;" ::: "memory");
  dkdv_items<D, kSplit>(maps, p, block, kv_bars);
  // All copies have landed, all products are done and read: shared and tensor memory are dQ's, unless a
  // wait has run out.
  tc_fence_before();
  const int stop = __syncthreads_or(*abort_flag);
  tc_fence_after();
  if (stop == 0) dq_items<D>(maps, p, block, dq_bars);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(block.tmem, 512);
  }
}

// ------------------------------------------------------------------ 3. merge
// dK and dV of the parts added up in order: four elements a thread, each part read once.
__global__ void __launch_bounds__(256) bsa_bwd_merge_kernel(const float4* __restrict__ parts, int n_split, long long n4,
                                                            float scale, uint2* __restrict__ dk, uint2* __restrict__ dv) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < 2 * n4; i += gridDim.x * 256LL) {
    float4 s = parts[i];
    for (int k = 1; k < n_split; ++k) {
      const float4 t = parts[2 * n4 * k + i];
      s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
    }
    const bool keys = i < n4;
    const float f = keys ? scale : 1.f;
    (keys ? dk + i : dv + (i - n4))[0] = make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
  }
}

// ------------------------------------------------------------------ host
// Parts of a KV head's query heads.  An item is a key tile with all steps of its query heads; fewer
// items than SMs leave SMs without one while the longest run, so heads are divided until there are
// enough (one row of 8192, 16 heads over 1: 1454 -> 613 us; of 2048: 341 -> 68), at most into as many
// as four times the SMs, which bounds the sums' memory.  256 items divided in two as well only pay for
// the merge (16 heads over 4 at 8192: 606 -> 630 us), and so do items of at most 16 steps, which end
// soon (2 rows of 1024, 4 heads over 2: 22.5 -> 23.5; with 32 steps it pays: 53 -> 29).
int split_of(int B, int T, int Hq, int Hkv) {
  const int G = Hq / Hkv, nb = T / kM;
  const long long items = (long long)B * Hkv * nb;
  if ((long long)nb * G <= 16) return 1;
  int n = 1;
  for (int d = 2; d <= G && items * n < 152 && items * d <= 4 * 152; ++d)
    if (G % d == 0) n = d;
  return n;
}
struct Layout {
  size_t nlse, ndelta, reach, q_cols, kv_cols, next, parts, total;
  int n_split;
};
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
Layout layout(int B, int T, int Hq, int Hkv, int D) {
  Layout l{};
  const size_t rows = static_cast<size_t>(B) * T * Hq * 4;
  size_t o = 0;
  l.nlse = o;   o += round256(rows);
  l.ndelta = o; o += round256(rows);
  l.reach = o;  o += round256(static_cast<size_t>(B) * (T / kM) * sizeof(int4));
  const size_t cols = static_cast<size_t>(B) * (T / 32) * sizeof(int4);
  l.q_cols = o; o += round256(cols);
  l.kv_cols = o; o += round256(cols);
  l.next = o;   o += 256;
  l.n_split = split_of(B, T, Hq, Hkv);
  l.parts = o;
  if (l.n_split > 1) o += round256(static_cast<size_t>(l.n_split) * 2 * B * T * Hkv * D * 4);
  l.total = o;
  return l;
}

template <int D>
int launch_impl(const void* q, const void* k, const void* v, const void* d_out, const Params& p, cudaStream_t stream) {
  Maps maps;
  auto map = [&](CUtensorMap* m, const void* at, int heads, int rows) {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)p.B * p.T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(at), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
  };
  if (!map(&maps.q, q, p.Hq, kM) || !map(&maps.d_out, d_out, p.Hq, kM) || !map(&maps.k, k, p.Hkv, kM) ||
      !map(&maps.k_half, k, p.Hkv, kSub) || !map(&maps.v_half, v, p.Hkv, kSub))
    return set_error(SBA_ERR_CUDA, "blocksparse_attn_bwd: tensor map failed");
  const auto kernel = p.n_split > 1 ? bsa_bwd_kernel<D, true> : bsa_bwd_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
  if (e != cudaSuccess) return cuda_error(e, "blocksparse_attn_bwd: set smem attribute");
  const int tok_groups = p.T / kPrepTok, head_groups = (p.Hq + kPrepHeads - 1) / kPrepHeads;
  const int n_delta = p.B * tok_groups * head_groups, n_reach = (9 * p.B * p.nb + 7) / 8;  // 1 + 2 * 128 / 32 warps a block
  bsa_bwd_prep_kernel<D><<<n_delta + n_reach, 256, 0, stream>>>(p, n_delta, tok_groups, head_groups);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(p.n_items_kv + p.n_items_dq, num_sms()));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, maps, p);
  }
  if (e == cudaSuccess && p.n_split > 1) {
    const long long n4 = (long long)p.B * p.T * p.Hkv * D / 4;
    const int grid = static_cast<int>(std::min<long long>((2 * n4 + 255) / 256, 8LL * num_sms()));
    bsa_bwd_merge_kernel<<<grid, 256, 0, stream>>>(reinterpret_cast<const float4*>(p.parts), p.n_split, n4, p.scale,
                                                   reinterpret_cast<uint2*>(p.dk), reinterpret_cast<uint2*>(p.dv));
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_error(e, "blocksparse_attn_bwd launch");
  return SBA_OK;
}

}  // namespace

unsigned read_and_clear_error_blocksparse_bwd(cudaStream_t, std::string* where) {
  DevError w{0u, 0u, 0}, zero{0u, 0u, 0};
  cudaMemcpyFromSymbol(&w, g_err_bsb, sizeof(w));
  if (w.flags) {
    cudaMemcpyToSymbol(g_err_bsb, &zero, sizeof(zero));
    if (where && w.where) {
      char buf[96];
      snprintf(buf, sizeof(buf), " [blocksparse_attn_bwd %s role %u barrier %u item %d]",
               ((w.where >> 24) & 0xFFu) == 6u ? "dq" : "dkdv", (w.where >> 16) & 0xFFu, w.where & 0xFFFFu, w.item);
      *where += buf;
    }
  }
  return w.flags;
}

size_t blocksparse_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int D) { return layout(B, T, Hq, Hkv, D).total; }

int launch_blocksparse_attn_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse,
                                const void* d_out, const int32_t* q_pos, const int32_t* q_seg, const int32_t* kv_pos,
                                const int32_t* kv_seg, const int32_t* lower, const int32_t* upper,
                                const int32_t* lower_full, const int32_t* upper_full, int B, int T, int Hq, int Hkv,
                                int D, int kv_block, int causal, int window_left, int window_right, int pad_id,
                                float scale, void* dq, void* dk, void* dv, void* workspace, cudaStream_t stream) {
  const Layout l = layout(B, T, Hq, Hkv, D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Params p{};
  p.out = static_cast<const __nv_bfloat16*>(out);
  p.dout = static_cast<const __nv_bfloat16*>(d_out);
  p.lse = lse;
  p.q_pos = q_pos; p.q_seg = q_seg; p.kv_pos = kv_pos; p.kv_seg = kv_seg;
  p.lower = lower; p.upper = upper; p.lower_full = lower_full; p.upper_full = upper_full;
  p.nlse = reinterpret_cast<float*>(ws + l.nlse);
  p.ndelta = reinterpret_cast<float*>(ws + l.ndelta);
  p.reach = reinterpret_cast<int4*>(ws + l.reach);
  p.q_cols = reinterpret_cast<int4*>(ws + l.q_cols);
  p.kv_cols = reinterpret_cast<int4*>(ws + l.kv_cols);
  p.next = reinterpret_cast<int*>(ws + l.next);
  p.parts = l.n_split > 1 ? reinterpret_cast<float*>(ws + l.parts) : nullptr;
  p.n_split = l.n_split;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.B = B; p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.nb = T / kM;
  p.nbkv = T / kv_block;
  p.tpb = kv_block / kSub;
  p.causal = causal;
  p.window_left = window_left;
  p.window_right = window_right;
  p.pad_id = pad_id;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.n_items_dq = B * Hq * p.nb;
  p.n_items_kv = B * Hkv * p.nb * p.n_split;
  p.wait_limit = wait_timeout_cycles();
  return D == 128 ? launch_impl<128>(q, k, v, d_out, p, stream) : launch_impl<64>(q, k, v, d_out, p, stream);
}

}  // namespace sba
