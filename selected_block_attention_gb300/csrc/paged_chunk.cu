// Attention of many query tokens per row over a paged cache, on the tensor cores' own
// memory: paged_chunk_kernel (prompts and chunks of prompts; few tokens a row run in
// paged_attention.cu, which this file's definitions follow).
//
// An item is (batch row, KV head, group of 256 (query, head) rows); its two halves of 128
// rows read the same keys, walked in tiles of 64.  As in paged_attention.cu the items'
// tiles form one line cut into equal runs, here one for each of kCtas CTAs (one per SM),
// and a second kernel merges the items that were cut.  A CTA's warps:
//   warps 0..3   loaders: pairs take the tiles in turn, a warp half a tile.  e4m3: 16-byte
//                loads into registers (a pair's next tile is on its way while the other
//                pair's is stored), codes to fp16 (exact), stored in the 128-byte swizzle
//                that the MMA reads; bf16: cp.async straight into it.  The pages' scales
//                travel with the value tile.
//   warps 4, 5   MMA issuers, one for each half w: S_w = Q_w K^T into one of two buffers,
//                O_w += P_w V with P_w in tensor memory over the S it came from, in the
//                order S(0) S(1) | PV(t) S(t + 2) | ...
//   warp 6       scheduler: finds the run's items and publishes them; items whose queries
//                see no key it writes itself (warp 7 idle)
//   warps 8..15  softmax, four for each half, one thread per row: it brings its query row
//                in (e4m3: times a power of two into fp16, see paged_core.cuh), takes its
//                64 scores out of tensor memory, keeps (m, l, u) as described there,
//                writes P, and at the end of the item writes the row or its partial.
// Tensor memory: S_w,0 S_w,1 (64 columns each) for w = 0, 1, then O_0, O_1: 512 columns.
//
// What bounds it.  4 rows of 512 tokens over 512 to 16384 keys, 32 heads over 8, D = 128,
// e4m3: 300 GFLOP in 262.5 us, 1.14 PFLOP/s (bf16 250).  The tensor pipe is busy half of the time: per tile
// and half an S of N = 64 takes 8 x 50 cycles and a PV of N = 128 4 x 64 of about 1030; the
// rest is the chain of a row's softmax (its 64 scores out of tensor memory, maximum, P back),
// which the two halves hide for one another only in part, beside the conversion of a tile
// (2 x 8 loads, 128 conversions and 32 stores a thread).  Four stages of keys and of values
// keep the loaders ahead of an item's change (three of keys: 273 us where four took 264).
// Tiles of 128 keys would halve the S instructions' fixed part, but leave one S buffer a
// half and the softmax on the path of the MMAs: 333 us.
#include <climits>
#include <cstdio>
#include <string>

#include "paged_core.cuh"
#include "sync.cuh"

namespace sba {

static __device__ DevError g_err_chunk = {0u, 0u, 0};

namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kCtas = 152;    // one for each SM
constexpr int kM = 128;       // rows of a half
constexpr int kRows = 2 * kM;
constexpr int kKT = 64;       // keys of a tile
constexpr int kMinTiles = 4;  // tiles of a run, at least
constexpr int kItemCost = 12;  // tiles that an item's queries and output are worth
constexpr float kRaise = 8.f;
constexpr float kRaiseU = 6.f;
// e4m3: logit factors are not let below this.  A masked score is -inf before it is multiplied,
// and -inf * 0 is no number, but a small query's factor times the scale of a page of zeros is 0
// in fp32.  Scores are below 2^31, so what a larger factor makes of them is below 2^-94.
constexpr float kLeastFactor = 1.17549435e-38f;  // 2^-126

struct ChunkParams {
  PagedView c;
  const __nv_bfloat16* q;
  long long q_tok;
  __nv_bfloat16* out;
  float* lse;
  struct SplitChunk* split;  // [kCtas]
  float* part_ml;            // [2 kCtas][kRows][2]
  float* part_o;             // [2 kCtas][D][kRows]
  int Hq, G;
  float scale, cap;
  int window_left, window_right;
  long long wait_limit;
};

// The item that a CTA begins but does not end (n > 1 partials: slot 2 cta + 1, then
// 2 (cta + i)); n = 0: none.
struct SplitChunk {
  int n, rows, first, t0, h;
  int pad[3];
};

enum Role : unsigned { kRoleLoader = 1, kRoleMma = 2, kRoleSoftmax = 3, kRoleScheduler = 4 };
enum BarId : unsigned { kBarQ = 1, kBarKFull, kBarKEmpty, kBarVFull, kBarVEmpty, kBarS, kBarP, kBarPvTile, kBarPvLast, kBarO, kBarSegFull, kBarSegEmpty };

// Key tiles [ka, kb) that a group's queries see, and its place on the line: max(kb - ka,
// 1) tiles after kItemCost empty ones.
struct GroupTiles {
  int ka, kb, units;
};
__device__ __forceinline__ int win_lo(const ChunkParams& p, const PagedRow& r, int i) {
  return p.window_left < 0 ? 0 : (int)min(max((long long)r.len - r.n + i - p.window_left, 0LL), (long long)r.len);
}
__device__ __forceinline__ int win_end(const ChunkParams& p, const PagedRow& r, int i) {  // one past the last key
  return p.window_right < 0 ? r.len
                            : (int)min(max((long long)r.len - r.n + i + p.window_right + 1, 0LL), (long long)r.len);
}
__device__ __forceinline__ GroupTiles group_tiles(const ChunkParams& p, const PagedRow& r, int g) {
  const int rows = r.n * p.G, r0 = g * kRows, r1 = min(r0 + kRows, rows) - 1;
  const int lo = win_lo(p, r, r0 / p.G), hi = win_end(p, r, r1 / p.G);
  GroupTiles t;
  t.ka = lo / kKT;
  t.kb = hi > lo ? (hi + kKT - 1) / kKT : t.ka;
  t.units = kItemCost + max(t.kb - t.ka, 1);
  return t;
}
__device__ __forceinline__ int groups_of(const ChunkParams& p, const PagedRow& r) {
  return (int)(((long long)r.n * p.G + kRows - 1) / kRows);
}
__device__ __forceinline__ long long row_units(const ChunkParams& p, const PagedRow& r) {
  const int n = groups_of(p, r);
  long long s = 0;
  for (int g = 0; g < n; ++g) s += group_tiles(p, r, g).units;
  return s;  // of one KV head
}

// One item's part of the CTA's run, as the scheduler publishes it: one key tile at least (an
// item without any is whole, and the scheduler's own).
struct Segment {
  PagedRow r;
  int b, h, g, rows;   // rows of the group
  int t0, nt;          // key tiles [t0, t0 + nt)
  int lo;              // first key of the row that may be read
  int begins, whole;
  int n;               // CTAs of the item, when it begins here
  int end;             // no more items
};
constexpr int kMetas = 8;  // tiles whose scales are kept
// Slots; each is read by 4 loader, 2 MMA and 8 softmax warps.  A loader looks two tiles ahead
// of the one that it has not delivered yet, and that one keeps its segment's slot from coming
// round.  Every segment has a tile, so what it looks at is two slots ahead at most: three slots
// would do; with fewer, or with segments without tiles, it would wait for itself.
constexpr int kSegs = 4;
static_assert(kSegs >= 3, "a loader's look-ahead");
// Walks the run.
struct Walker {
  long long cur, end, per;
  int b, h, g, off, groups;
  PagedRow r;
  __device__ __forceinline__ void row(const ChunkParams& p) {
    bool bad;
    r = paged_row(p.c, b, &bad);
    groups = groups_of(p, r);
  }
  __device__ __forceinline__ bool next(const ChunkParams& p, int cta, Segment& s) {
    while (cur < end) {
      while (g >= groups) {  // also rows without tokens
        g = 0;
        if (groups == 0 || ++h == p.c.Hkv) {
          h = 0;
          if (++b >= p.c.B) {  // only if lengths change under the call
            cur = end;
            return false;
          }
          row(p);
        }
      }
      const GroupTiles t = group_tiles(p, r, g);
      const int x0 = off, x1 = (int)min((long long)t.units, x0 + (end - cur));
      const long long at = cur - x0;
      cur += x1 - x0;
      off = x1;
      s.g = g;
      if (x1 == t.units) {
        off = 0;
        ++g;
      }
      if (x1 <= kItemCost) continue;  // nothing but the empty tiles
      const int s0 = max(x0 - kItemCost, 0), s1 = x1 - kItemCost;
      s.r = r;
      s.b = b;
      s.h = h;
      s.rows = min(kRows, r.n * p.G - s.g * kRows);
      s.t0 = t.ka + s0;
      s.nt = max(min(t.ka + s1, t.kb) - s.t0, 0);
      s.begins = s0 == 0;
      s.whole = s.begins && x1 == t.units;
      s.n = (int)min((at + t.units - 1) / per, (long long)kCtas - 1) - cta + 1;
      s.lo = win_lo(p, r, 0);
      s.end = 0;
      return true;
    }
    return false;
  }
};

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kQPanel = kM * 128;
  static constexpr int kQBytes = kPanels * kQPanel;
  static constexpr int kTPanel = kKT * 128;
  static constexpr int kTBytes = kPanels * kTPanel;
  static constexpr int kStagesK = 4;
  static constexpr int kStages = 4;
  static constexpr int kOffK = 2 * kQBytes;
  static constexpr int kOffV = kOffK + kStagesK * kTBytes;
  static constexpr int kOffMeta = kOffV + kStages * kTBytes;  // per tile: 4 key, 4 value scales
  static constexpr int kOffSegs = kOffMeta + kMetas * 32;
  static constexpr int kOffBars = (kOffSegs + kSegs * (int)sizeof(Segment) + 7) & ~7;
  static constexpr int kNumBars = 2 * kSegs + 2 + 2 * kStagesK + 2 * kStages + 4 + 4 + 2 + 2 + 2 + 2;
  static constexpr int kOffMisc = (kOffBars + kNumBars * 8 + 15) & ~15;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static constexpr int kOCol = 4 * kKT;
  static constexpr int kTmemCols = 512;
  static_assert(kOCol + 2 * D <= kTmemCols, "tensor memory");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

__device__ __forceinline__ void mask_columns(float (&x)[kKT], int jlo, int jhi) {
  const uint32_t w0 = (jlo <= 31 && jhi >= 0)
      ? ((jhi >= 31 ? 0xffffffffu : ((2u << jhi) - 1u)) & (0xffffffffu << min(max(jlo, 0), 31))) : 0u;
  const uint32_t w1 = (jhi >= 32 && jlo <= 63)
      ? ((jhi >= 63 ? 0xffffffffu : ((2u << (jhi - 32)) - 1u)) & (0xffffffffu << max(jlo - 32, 0))) : 0u;
#pragma unroll
  for (int j = 0; j < 32; ++j) x[j] = (w0 & (1u << j)) ? x[j] : -INFINITY;
#pragma unroll
  for (int j = 0; j < 32; ++j) x[32 + j] = (w1 & (1u << j)) ? x[32 + j] : -INFINITY;
}

// kSub: groups of a tile's keys with one scale each: 1 for pages of 64 and more (and bf16),
// 4 for smaller ones.
template <bool kF8, int D, bool kCap, int kSub>
__global__ void __launch_bounds__(kThreads, 1)
paged_chunk_kernel(const ChunkParams p) {
  constexpr int kCols = kKT / kSub;
  using C = Cfg<D>;
  constexpr uint32_t kFmt = kF8 ? 0u : 1u;  // operands: fp16 or bf16
  constexpr uint32_t kIdescQK = make_idesc(128, kKT, kFmt, false, false);
  constexpr uint32_t kIdescPV = make_idesc(128, D, kFmt, false, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ long long s_sum[kThreads / 32], s_total;
  __shared__ int s_b, s_h, s_g, s_off;  // where the CTA's run begins
  uint64_t* bb = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  uint64_t* seg_full = bb;  bb += kSegs;
  uint64_t* seg_empty = bb; bb += kSegs;
  uint64_t* q_full = bb;   bb += 2;
  uint64_t* k_full = bb;   bb += C::kStagesK;
  uint64_t* k_empty = bb;  bb += C::kStagesK;
  uint64_t* v_full = bb;   bb += C::kStages;
  uint64_t* v_empty = bb;  bb += C::kStages;
  uint64_t* s_full = bb;   bb += 4;  // [2 w + buffer]
  uint64_t* p_full = bb;   bb += 4;
  uint64_t* pv_tile = bb;  bb += 2;
  uint64_t* pv_last = bb;  bb += 2;
  uint64_t* o_empty = bb;  bb += 2;
  uint64_t* mma_done = bb; bb += 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const Abort ab{abort_flag, &g_err_chunk, 5u, p.wait_limit};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  paged_wait_before();

  // ---- the CTA's run: each warp adds up a share of the rows, lanes over a row's groups
  // (few rows: they are long) or over rows
  {
    const bool by_row = p.c.B > 4 * (kThreads / 32);
    const int chunk = (p.c.B + kThreads / 32 - 1) / (kThreads / 32);
    const int b0 = min(warp * chunk, p.c.B), b1 = min(b0 + chunk, p.c.B);
    bool any_bad = false;
    // units of one KV head of row b, in every lane
    auto row_sum = [&](const PagedRow& r) {
      const int n = groups_of(p, r);
      long long x = 0;
      for (int g = lane; g < n; g += 32) x += group_tiles(p, r, g).units;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      return x;
    };
    auto units_of_lane = [&](int b) {  // of row b, all KV heads
      bool bad;
      const PagedRow r = paged_row(p.c, b, &bad);
      any_bad |= bad;
      return row_units(p, r) * p.c.Hkv;
    };
    long long sum = 0;
    if (by_row) {
      for (int b = b0 + lane; b < b1; b += 32) sum += units_of_lane(b);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    } else {
      for (int b = b0; b < b1; ++b) {
        bool bad;
        const PagedRow r = paged_row(p.c, b, &bad);
        any_bad |= bad;
        sum += row_sum(r) * p.c.Hkv;
      }
    }
    if (any_bad && cta == 0) atomicOr(&g_err_chunk.flags, (unsigned)kDevErrInput);
    if (lane == 0) s_sum[warp] = sum;
    if (tid == 0) s_b = s_h = s_g = s_off = 0;
    __syncthreads();
    long long total = 0, pre = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i == warp) pre = total;
      total += s_sum[i];
    }
    const long long t0 = (long long)cta * max((total + kCtas - 1) / kCtas, (long long)(kMinTiles + kItemCost));
    if (t0 >= pre && t0 < pre + sum) {
      long long off = t0 - pre;
      int b = b0;
      PagedRow r;
      long long one;
      for (;; ++b) {
        bool bad;
        r = paged_row(p.c, b, &bad);
        one = row_sum(r);
        if (off < one * p.c.Hkv || b + 1 >= b1) break;
        off -= one * p.c.Hkv;
      }
      const int h = one > 0 ? (int)min(off / one, (long long)p.c.Hkv - 1) : 0;
      off -= h * one;
      for (int g0 = 0; g0 < groups_of(p, r); g0 += 32) {  // the group: 32 at a time
        const int g = g0 + lane, u = g < groups_of(p, r) ? group_tiles(p, r, g).units : 0;
        int end = u;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, end, d);
          if (lane >= d) end += x;
        }
        const int all = __shfl_sync(0xffffffffu, end, 31);
        if (off >= all) {
          off -= all;
          continue;
        }
        if (off >= end - u && off < end) {
          s_b = b;
          s_h = h;
          s_g = g;
          s_off = (int)off - (end - u);
        }
        break;
      }
    }
    if (tid == 0) s_total = total;
  }
  if (tid == 0) {
    for (int i = 0; i < kSegs; ++i) { mbar_init(&seg_full[i], 1); mbar_init(&seg_empty[i], 14); }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&q_full[w], 4);
      mbar_init(&pv_tile[w], 1); mbar_init(&pv_last[w], 1);
      mbar_init(&o_empty[w], 4); mbar_init(&mma_done[w], 1);
    }
    // the MMA's completion, and the issuing warp itself: it has seen the tile's scales
    for (int i = 0; i < 4; ++i) { mbar_init(&s_full[i], 2); mbar_init(&p_full[i], 4); }
    // both loader warps fill a stage, both MMA warps release it
    for (int i = 0; i < C::kStagesK; ++i) { mbar_init(&k_full[i], 2); mbar_init(&k_empty[i], 2); }
    for (int i = 0; i < C::kStages; ++i) { mbar_init(&v_full[i], 2); mbar_init(&v_empty[i], 2); }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  paged_let_next();
  const uint32_t tmem = *tmem_holder;
  const uint32_t smem_base = smem_u32(smem);
  auto seg_at = [&](int slot) -> Segment& {
    return *reinterpret_cast<Segment*>(smem + C::kOffSegs + slot * (int)sizeof(Segment));
  };

  // registers of the four warpgroups: 128 + 64 + 160 + 160 = 4 x 128
  if (warp < 4) {
    // ------------------------------------------------------------------ loaders
    constexpr int kItem = kF8 ? 1 : 2;
    constexpr int kCpr = D * kItem / 16;  // 16-byte chunks of a row
    constexpr int kStep = 32 / kCpr;      // rows of a warp-wide access
    constexpr int kN = 32 / kStep;        // accesses for the warp's 32 keys
    const int pair = warp >> 1, half = warp & 1;
    // A lane's chunk and first row.  e4m3 at D = 128: eight lanes write chunks 0..3 (or 4..7)
    // of two rows, whose fp16 halves then lie in different banks.
    const int chunk = kF8 && D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane % kCpr;
    const int row0 = kF8 && D == 128 ? ((lane >> 2) & 1) + 2 * (lane >> 4) : lane / kCpr;
    const int pmask = (1 << p.c.p_shift) - 1;
    int ks = 0; uint32_t kphase = 0;
    int vs = 0; uint32_t vphase = 0;
    int ms = pair;  // the tile's place among the scales
    auto next_k = [&]() { if (++ks == C::kStagesK) { ks = 0; kphase ^= 1; } };
    auto next_v = [&]() { if (++vs == C::kStages) { vs = 0; vphase ^= 1; } };
    // ---- the run's tiles in order; this pair's are every second one
    int slot = -1; uint32_t sphase = 1;  // before slot 0 of phase 0
    int t = -1, nt = 0;
    bool have = true;
    auto step = [&]() {
      ++t;
      while (have && t >= nt) {
        if (slot >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&seg_empty[slot]);
        }
        if (slot < 0 || ++slot == kSegs) { slot = 0; sphase ^= 1; }
        have = warp_wait(&seg_full[slot], sphase, ab, kRoleLoader, kBarSegFull, cta) && !seg_at(slot).end;
        nt = have ? seg_at(slot).nt : 0;
        t = 0;
      }
    };
    // the tile that is fetched next: its keys (clamped to owned slots) and pages
    int key0 = 0, cl = 0, ch = 0, h = 0, pg[2] = {0, 0};
    auto look = [&]() {
      if (!have) return;
      const Segment& sg = seg_at(slot);
      key0 = (sg.t0 + t) * kKT + half * 32;
      cl = sg.lo;
      ch = sg.r.len - 1;
      h = sg.h;
      const int* table = p.c.table + (long long)sg.b * p.c.width;
#pragma unroll
      for (int i = 0; i < 2; ++i) pg[i] = __ldg(table + (min(max(key0 + 16 * i, cl), ch) >> p.c.p_shift));
    };
    auto page_at = [&](int i) -> int {
      if ((unsigned)pg[i] < (unsigned)p.c.num_pages) return pg[i];
      if (lane == 0) atomicOr(&g_err_chunk.flags, (unsigned)kDevErrInput);
      return 0;  // any page that exists: the row's result is undefined, the read is not
    };
    auto byte_of = [&](int page) -> long long {
      return page * p.c.page_bytes + (((long long)h << p.c.p_shift) * D) * kItem + chunk * 16;
    };
    // Byte offset in the page of access j of subtile x; inside the owned keys it steps by a
    // constant.
    constexpr int kHalf = kN / 2;  // accesses of a subtile
    auto row_off = [&](int x, int j, bool inside) -> int {
      const int first = key0 + 16 * x;
      if (inside) return ((first & pmask) + row0) * (D * kItem) + j * kStep * (D * kItem);
      return (min(max(first + row0 + j * kStep, cl), ch) & pmask) * (D * kItem);
    };
    if constexpr (kF8) {
      uint4 rk[kN], rv[kN];
      float kc[2], vc[2];
      auto load_scales = [&]() {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const long long at = (long long)page_at(x) * p.c.Hkv + h;
          kc[x] = __ldg(p.c.ks + at);
          vc[x] = __ldg(p.c.vs + at);
        }
      };
      auto load = [&](const uint8_t* pool, uint4 (&raw)[kN]) {
        const bool inside = key0 >= cl && key0 + 31 <= ch;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* src = pool + byte_of(page_at(x));
          auto rows = [&](bool in) {
#pragma unroll
            for (int j = 0; j < kHalf; ++j)
              raw[x * kHalf + j] = __ldg(reinterpret_cast<const uint4*>(src + row_off(x, j, in)));
          };
          if (inside) rows(true); else rows(false);
        }
      };
      // 16 codes as two 16-byte chunks of fp16
      const uint32_t s0 = (((chunk & 3) * 2) ^ (row0 & 7)) << 4;
      auto put = [&](uint32_t tile, const uint4 (&raw)[kN]) {
        const uint32_t dst = tile + (chunk >> 2) * C::kTPanel + (half * 32 + row0) * 128;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          // row & 7 is row0 (kStep = 8) or row0 + 4 (i & 1) with row0 < 4
          const uint32_t at = dst + i * (kStep * 128), x = kStep == 8 ? 0u : (i & 1) * 64u;
          uint4 a, c;
          e4m3x4_to_f16x2(raw[i].x, a.x, a.y);
          e4m3x4_to_f16x2(raw[i].y, a.z, a.w);
          e4m3x4_to_f16x2(raw[i].z, c.x, c.y);
          e4m3x4_to_f16x2(raw[i].w, c.z, c.w);
          paged_sts16(at + (s0 ^ x), a);
          paged_sts16(at + (s0 ^ x ^ 16u), c);
        }
      };
      step();
      if (pair == 1) {
        step();
        next_k();
        next_v();
      }
      look();
      if (have) {
        load_scales();
        load(p.c.k, rk);
        load(p.c.v, rv);
      }
      bool more = have;  // a tile is in registers
      step();
      step();
      look();
      // The next tile's keys are on their way while this one's values are stored, its
      // values while the next one's keys are.
      while (more) {
        if (!warp_wait(&k_empty[ks], kphase ^ 1, ab, kRoleLoader, kBarKEmpty, cta)) break;
        if (lane < 2) {
          float* meta = reinterpret_cast<float*>(smem + C::kOffMeta + ms * 32);
          meta[half * 2 + lane] = lane ? kc[1] : kc[0];
          meta[4 + half * 2 + lane] = lane ? vc[1] : vc[0];
        }
        put(smem_base + C::kOffK + ks * C::kTBytes, rk);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[ks]);
        more = have;
        if (have) {
          load_scales();
          load(p.c.k, rk);
        }
        if (!warp_wait(&v_empty[vs], vphase ^ 1, ab, kRoleLoader, kBarVEmpty, cta)) break;
        put(smem_base + C::kOffV + vs * C::kTBytes, rv);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[vs]);
        if (have) load(p.c.v, rv);
        ms = (ms + 2) % kMetas;
        next_k(); next_k();
        next_v(); next_v();
        step();
        step();
        look();
      }
    } else {
      auto copy = [&](uint8_t* tile, const uint8_t* pool) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* src = pool + byte_of(page_at(x));
          const bool inside = key0 >= cl && key0 + 31 <= ch;
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            const int row = half * 32 + row0 + (x * kHalf + j) * kStep;
            paged_cp16(smem_u32(tile + (chunk >> 3) * C::kTPanel + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)),
                       src + row_off(x, j, inside));
          }
        }
        paged_cp_commit();
      };
      step();
      if (pair == 1) {
        step();
        next_k();
        next_v();
      }
      look();
      while (have) {
        if (!warp_wait(&k_empty[ks], kphase ^ 1, ab, kRoleLoader, kBarKEmpty, cta)) break;
        copy(smem + C::kOffK + ks * C::kTBytes, p.c.k);
        if (!warp_wait(&v_empty[vs], vphase ^ 1, ab, kRoleLoader, kBarVEmpty, cta)) break;
        copy(smem + C::kOffV + vs * C::kTBytes, p.c.v);
        step();
        step();
        look();
        paged_cp_wait<1>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[ks]);
        paged_cp_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[vs]);
        next_k(); next_k();
        next_v(); next_v();
      }
      paged_cp_wait<0>();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ MMA issuer of half w
    setmaxnreg_dec<64>();
    if (warp < 6) {
      const int w = warp - 4;
      const uint32_t leader = elect_one();
      uint32_t qph = 0u, oph = 0u, pph = 0u;
      int ks = 0; uint32_t kphase = 0;
      int vs = 0; uint32_t vphase = 0;
      bool ok = true;
      const uint64_t q_desc = make_sdesc(smem_base + w * C::kQBytes, 16, 1024, kLayoutSW128);
      const uint64_t k_desc0 = make_sdesc(smem_base + C::kOffK, 16, 1024, kLayoutSW128);
      const uint64_t v_desc0 = make_sdesc(smem_base + C::kOffV, C::kTPanel, 1024, kLayoutSW128);
      const uint32_t o_tmem = tmem + C::kOCol + w * D;
      auto s_tmem = [&](int buf) { return tmem + (2 * w + buf) * kKT; };
      auto kstep = [](int kk, int panel) -> uint64_t {
        return static_cast<uint64_t>(((kk / 4) * panel + (kk % 4) * 32) >> 4);
      };
      auto next_k = [&]() { if (++ks == C::kStagesK) { ks = 0; kphase ^= 1; } };
      auto next_v = [&]() { if (++vs == C::kStages) { vs = 0; vphase ^= 1; } };
      auto issue_s = [&](int buf) -> bool {
        if (!warp_wait(&k_full[ks], kphase, ab, kRoleMma, kBarKFull, cta)) return false;
        tc_fence_after();
        const uint64_t kd = k_desc0 + static_cast<uint64_t>((ks * C::kTBytes) >> 4);
  #pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss_by(leader, s_tmem(buf), q_desc + kstep(kk, C::kQPanel), kd + kstep(kk, C::kTPanel), kIdescQK,
                        kk > 0 ? 1u : 0u);
        mma_commit_by(leader, &s_full[2 * w + buf]);
        if (lane == 0) mbar_arrive(&s_full[2 * w + buf]);
        mma_commit_by(leader, &k_empty[ks]);
        next_k();
        return true;
      };
      for (int slot = 0, phase = 0; ok; phase ^= ++slot == kSegs, slot %= kSegs) {
        if (!warp_wait(&seg_full[slot], phase, ab, kRoleMma, kBarSegFull, cta)) break;
        const int nt = seg_at(slot).nt, rows = seg_at(slot).rows, last = seg_at(slot).end;
        if (last) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[slot]);
        if (rows <= w * kM) {
          // no row in this half: release the stages so the rings stay in step
          for (int t = 0; t < nt && ok; ++t) {
            if (!warp_wait(&k_full[ks], kphase, ab, kRoleMma, kBarKFull, cta)) { ok = false; break; }
            if (lane == 0) mbar_arrive(&k_empty[ks]);
            next_k();
            if (!warp_wait(&v_full[vs], vphase, ab, kRoleMma, kBarVFull, cta)) { ok = false; break; }
            if (lane == 0) mbar_arrive(&v_empty[vs]);
            next_v();
          }
          continue;
        }
        if (!warp_wait(&q_full[w], qph, ab, kRoleMma, kBarQ, cta)) break;
        qph ^= 1;
        for (int t = 0; t < 2 && t < nt && ok; ++t)
          if (!issue_s(t)) ok = false;
        for (int t = 0; t < nt && ok; ++t) {
          const int buf = t & 1;
          if (!warp_wait(&v_full[vs], vphase, ab, kRoleMma, kBarVFull, cta)) { ok = false; break; }
          if (t == 0) {
            if (!warp_wait(&o_empty[w], oph ^ 1, ab, kRoleMma, kBarO, cta)) { ok = false; break; }
            oph ^= 1;
          }
          if (!warp_wait(&p_full[2 * w + buf], (pph >> buf) & 1u, ab, kRoleMma, kBarP, cta)) { ok = false; break; }
          pph ^= 1u << buf;
          tc_fence_after();
          const uint64_t vd = v_desc0 + static_cast<uint64_t>((vs * C::kTBytes) >> 4);
  #pragma unroll
          for (int kk = 0; kk < kKT / 16; ++kk)
            mma_f16_ts_by(leader, o_tmem, s_tmem(buf) + kk * 8, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4),
                          kIdescPV, (t == 0 && kk == 0) ? 0u : 1u);
          mma_commit_by(leader, &pv_tile[w]);
          if (t == nt - 1) mma_commit_by(leader, &pv_last[w]);
          mma_commit_by(leader, &v_empty[vs]);
          next_v();
          if (t + 2 < nt && !issue_s(buf)) { ok = false; break; }
        }
      }
      mma_commit_by(leader, &mma_done[w]);
      drain_wait(&mma_done[w], 0);
      __syncwarp();
    } else if (warp == 6) {
      // ---------------------------------------------------------------- scheduler
      const long long per = max((s_total + kCtas - 1) / kCtas, (long long)(kMinTiles + kItemCost));
      Walker walk;
      walk.per = per;
      walk.cur = (long long)cta * per;
      walk.end = min(walk.cur + per, s_total);
      if (lane == 0) p.split[cta].n = 0;
      if (walk.cur < walk.end) {
        walk.b = s_b;
        walk.h = s_h;
        walk.g = s_g;
        walk.off = s_off;
        walk.row(p);
      }
      // output 0 and LSE -inf of an item whose queries see no key
      auto write_empty = [&](const Segment& s) {
        constexpr int kCh = D / 8;
#pragma unroll 1  // unrolled it spills (64 registers)
        for (int x = lane; x < s.rows * kCh; x += 32) {
          const int row = x / kCh, rr = s.g * kRows + row, qi = rr / p.G;
          const long long orow = (long long)(s.r.t0 + qi) * p.Hq + s.h * p.G + (rr - qi * p.G);
          *reinterpret_cast<uint4*>(p.out + orow * D + x % kCh * 8) = make_uint4(0u, 0u, 0u, 0u);
          if (x % kCh == 0 && p.lse != nullptr) p.lse[orow] = -INFINITY;
        }
      };
      int slot = 0; uint32_t phase = 0;
      while (true) {
        Segment sg;
        sg.end = walk.next(p, cta, sg) ? 0 : 1;
        if (!sg.end && sg.nt == 0) {
          write_empty(sg);
          continue;
        }
        if (!warp_wait(&seg_empty[slot], phase ^ 1, ab, kRoleScheduler, kBarSegEmpty, cta)) break;
        if (lane == 0) {
          seg_at(slot) = sg;
          mbar_arrive(&seg_full[slot]);
        }
        __syncwarp();
        if (sg.end) break;
        if (++slot == kSegs) { slot = 0; phase ^= 1; }
      }
    }
  } else {
    setmaxnreg_inc<160>();
    // ------------------------------------------------------------------ softmax and output
    const int w = (warp - 8) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the half = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t o_col = tmem + lane_off + C::kOCol + w * D;
    uint8_t* my_q = smem + w * C::kQBytes + r * 128;
    int ms = 0;  // the tile's place among the scales
    uint32_t sph = 0u, pvt_ph = 0u, pvl_ph = 0u;
    for (int slot = 0, phase = 0;; phase ^= ++slot == kSegs, slot %= kSegs) {
      if (!warp_wait(&seg_full[slot], phase, ab, kRoleSoftmax, kBarSegFull, cta)) break;
      const Segment& sg = seg_at(slot);  // until this warp releases the slot
      if (sg.end) break;
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[slot]);
      };
      const int nt = sg.nt;
      const bool active = sg.rows > w * kM;
      const int rr = sg.g * kRows + w * kM + r;
      const bool row_ok = w * kM + r < sg.rows;
      const int qi = row_ok ? rr / p.G : 0, hq = sg.h * p.G + (row_ok ? rr - qi * p.G : 0);
      const int klo = win_lo(p, sg.r, qi), khi = row_ok ? win_end(p, sg.r, qi) - 1 : -1;  // the row's keys
      // every row of the group sees [full_lo, full_end)
      const int ia = sg.g * kRows / p.G, ib = (sg.g * kRows + sg.rows - 1) / p.G;
      const int full_lo = win_lo(p, sg.r, ib), full_end = win_end(p, sg.r, ia);
      float m = -INFINITY, l = 0.f, u = -INFINITY;
      bool ok = true;
      if (active) {
        // ---- the query row, into the swizzle that the MMA reads
        float f = kCap ? p.scale / p.cap : p.scale * kPagedLog2e;
        const __nv_bfloat16* src = p.q + (long long)(sg.r.t0 + qi) * p.q_tok + (long long)hq * D;
        uint4 raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          raw[i] = row_ok ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kF8) {
          uint32_t top = 0u;  // of bf16 magnitudes as integers
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            top = __vmaxu2(top, raw[i].x & 0x7FFF7FFFu); top = __vmaxu2(top, raw[i].y & 0x7FFF7FFFu);
            top = __vmaxu2(top, raw[i].z & 0x7FFF7FFFu); top = __vmaxu2(top, raw[i].w & 0x7FFF7FFFu);
          }
          const int ex = (int)(max(top & 0xFFFFu, top >> 16) >> 7);
          const int fe = (ex == 0 || ex == 255) ? 127 : min(127 + 14 - (ex - 127), 253);
          const float up = __uint_as_float((uint32_t)fe << 23);
          f *= __uint_as_float((uint32_t)(254 - fe) << 23);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            raw[i].x = pack_f16x2(bf16_lo(raw[i].x) * up, bf16_hi(raw[i].x) * up);
            raw[i].y = pack_f16x2(bf16_lo(raw[i].y) * up, bf16_hi(raw[i].y) * up);
            raw[i].z = pack_f16x2(bf16_lo(raw[i].z) * up, bf16_hi(raw[i].z) * up);
            raw[i].w = pack_f16x2(bf16_lo(raw[i].w) * up, bf16_hi(raw[i].w) * up);
          }
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<uint4*>(my_q + (i >> 3) * C::kQPanel + (((i & 7) ^ (r & 7)) << 4)) = raw[i];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[w]);

        for (int t = 0; t < nt; ++t) {
          const int buf = t & 1, key0 = (sg.t0 + t) * kKT;
          const uint32_t s_col = tmem + lane_off + (2 * w + buf) * kKT;
          if (!warp_wait(&s_full[2 * w + buf], (sph >> buf) & 1u, ab, kRoleSoftmax, kBarS, cta)) { ok = false; break; }
          sph ^= 1u << buf;
          float mult[kSub], lgv[kSub];  // logit factors, log2 of the value scales
          if constexpr (kF8) {
            const float* meta = reinterpret_cast<const float*>(smem + C::kOffMeta + ms * 32);
#pragma unroll
            for (int g = 0; g < kSub; ++g) {
              mult[g] = fmaxf(f * meta[g], kLeastFactor);
              asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lgv[g]) : "f"(meta[4 + g]));
            }
          } else {
            mult[0] = f;
          }
          ms = (ms + 1) % kMetas;
          float x[kKT];
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kKT / 32; ++c) tmem_ld_32x32b_x32_nw(s_col + c * 32, x + c * 32);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kKT; ++j) tmem_ld_ready(x[j]);
          if constexpr (kCap) {
            const float c1k = p.cap * kPagedLog2e;
#pragma unroll
            for (int j = 0; j < kKT; ++j) x[j] = paged_capped(x[j] * mult[j / kCols], c1k);
          }
          if (key0 < full_lo || key0 + kKT > full_end)
            mask_columns(x, min(max(klo - key0, 0), kKT), max(min(khi - key0, kKT - 1), -1));
          // maxima of the groups, in log2 units
          float tmax = -INFINITY, dmax = -INFINITY;
#pragma unroll
          for (int g = 0; g < kSub; ++g) {
            float a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = fmaxf(x[g * kCols + 2 * i], x[g * kCols + 2 * i + 1]);
#pragma unroll
            for (int j = 8; j < kCols; j += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) a[i] = fmax3f(a[i], x[g * kCols + j + 2 * i], x[g * kCols + j + 2 * i + 1]);
            float top = fmaxf(fmax3f(a[0], a[1], a[2]), a[3]);
            if constexpr (!kCap) top *= mult[g];
            tmax = fmaxf(tmax, top);
            if constexpr (kF8) dmax = fmaxf(dmax, top + lgv[g]);
          }
          const bool move = tmax > m + kRaise || (m == -INFINITY && tmax != -INFINITY);
          const float m_new = move ? tmax : m;
          l *= (move && m != -INFINITY) ? ex2(m - m_new) : 1.f;
          bool rescale;
          float alpha;
          if constexpr (kF8) {
            const bool mu = dmax > u + kRaiseU || (u == -INFINITY && dmax != -INFINITY);
            rescale = mu && u != -INFINITY;
            alpha = rescale ? ex2(u - dmax) : 1.f;
            if (mu) u = dmax;
          } else {
            rescale = move && m != -INFINITY;
            alpha = rescale ? ex2(m - m_new) : 1.f;
          }
          m = m_new;
          // P = 2^(x mult - m + lw): lw takes the probability to the reference u (e4m3).  Below
          // 2^-40 it is zero in fp16 whatever its size, so lw stops there and the sum of P
          // 2^-lw keeps every probability.
          float lw[kSub], tile_sum = 0.f;
#pragma unroll
          for (int g = 0; g < kSub; ++g)
            lw[g] = kF8 && m != -INFINITY ? fminf(fmaxf(lgv[g] + (m - u) + 8.f, -40.f), 100.f) : 0.f;
          const float mm = m == -INFINITY ? 0.f : m;
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < kSub; ++g) {
            uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
            const uint64_t base2 = pack_f32x2(lw[g] - mm, lw[g] - mm);
            const float ms = kCap ? 1.f : mult[g];
            const uint64_t m2 = pack_f32x2(ms, ms);
#pragma unroll
            for (int j = 0; j < kCols; j += 2) {
              const int col = g * kCols + j;
              float a0, a1;
              unpack_f32x2(fma_f32x2(pack_f32x2(x[col], x[col + 1]), m2, base2), a0, a1);
              a0 = ex2(a0);
              a1 = ex2(a1);
              sum2[(j >> 1) & 3] = add_f32x2(sum2[(j >> 1) & 3], pack_f32x2(a0, a1));
              pk[(col >> 1) & 15] = kF8 ? pack_f16x2(a0, a1) : pack_bf16x2(a0, a1);
              if ((col & 31) == 30) tmem_st_32x32b_x16_u_nw(s_col + (col >> 5) * 16, pk);
            }
            float lo, hi;
            unpack_f32x2(add_f32x2(add_f32x2(sum2[0], sum2[1]), add_f32x2(sum2[2], sum2[3])), lo, hi);
            tile_sum += kF8 ? (lo + hi) * ex2(-lw[g]) : lo + hi;
          }
          tmem_wait_st();
          l += tile_sum;
          if (t > 0) {
            // O_w holds PV(0 .. t - 2); a rescale also waits for PV(t - 1)
            if (__any_sync(0xffffffffu, rescale)) {
              if (!warp_wait(&pv_tile[w], pvt_ph, ab, kRoleSoftmax, kBarPvTile, cta)) { ok = false; break; }
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                float ov[32];
                tmem_ld_32x32b_x32(o_col + c * 32, ov);
#pragma unroll
                for (int j = 0; j < 32; ++j) ov[j] *= alpha;
                tmem_st_32x32b_x32(o_col + c * 32, ov);
              }
            }
            pvt_ph ^= 1u;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * w + buf]);
        }
        if (!ok) break;
        if (!warp_wait(&pv_last[w], pvl_ph, ab, kRoleSoftmax, kBarPvLast, cta)) break;
        pvl_ph ^= 1u;
        pvt_ph ^= 1u;
        tc_fence_after();
      } else {
        ms = (ms + nt) % kMetas;
      }

      // ---- the row's result, or its partial
      const float ref = kF8 ? u - 8.f : m;  // o stands for o 2^ref
      const bool some = active && l != 0.f;
      const int part = cta * 2 + (sg.begins ? 1 : 0);
      if (sg.begins && !sg.whole && warp == 8 && lane == 0) {
        SplitChunk s;
        s.n = sg.n;
        s.rows = sg.rows;
        s.first = sg.g * kRows;
        s.t0 = sg.r.t0;
        s.h = sg.h;
        p.split[cta] = s;
      }
      if (!active) {
        release();
        continue;
      }
      const long long orow = (long long)(sg.r.t0 + qi) * p.Hq + hq;
      // whole: o / l; partial: o relative to 2^m
      const float factor = !some ? 0.f : sg.whole ? ex2(ref - m) / l : ex2(ref - m);
      if (!sg.whole) {
        *reinterpret_cast<float2*>(p.part_ml + ((long long)part * kRows + w * kM + r) * 2) =
            make_float2(some ? m : -INFINITY, some ? l : 0.f);
      } else if (p.lse != nullptr && row_ok) {
        p.lse[orow] = some ? (m + log2f(l)) * kPagedLn2 : -INFINITY;
      }
      float* po = p.part_o + (long long)part * D * kRows + w * kM + r;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float ov[32];
        tmem_ld_32x32b_x32_nw(o_col + c * 32, ov);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) tmem_ld_ready(ov[j]);
        if (c == D / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[w]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) ov[j] = some ? ov[j] * factor : 0.f;
        if (!sg.whole) {
          // lanes are rows: one coalesced store a column
#pragma unroll
          for (int j = 0; j < 32; ++j) po[(long long)(c * 32 + j) * kRows] = ov[j];
        } else {
          // this row's part of the (consumed) query buffer
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4*>(my_q + (c >> 1) * C::kQPanel + ((((c & 1) * 4 + (j >> 3)) ^ (r & 7)) << 4)) =
                make_uint4(pack_bf16x2(ov[j], ov[j + 1]), pack_bf16x2(ov[j + 2], ov[j + 3]),
                           pack_bf16x2(ov[j + 4], ov[j + 5]), pack_bf16x2(ov[j + 6], ov[j + 7]));
        }
      }
      if (sg.whole) {
        __syncwarp();
        constexpr int kCh = D / 8;  // 16-byte chunks of an output row
        const long long mine = row_ok ? orow : -1;
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const int x = i * 32 + lane, row = x / kCh, ch = x % kCh;
          const long long to = __shfl_sync(0xffffffffu, mine, row);
          const int rq = q4 * 32 + row;
          const uint4 v = *reinterpret_cast<const uint4*>(smem + w * C::kQBytes + (ch >> 3) * C::kQPanel + rq * 128 +
                                                          (((ch & 7) ^ (rq & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(p.out + to * D + ch * 8) = v;
        }
      }
      release();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// 32 rows of an item that was cut: lanes are rows, a warp a quarter of the columns; the
// result goes out through shared memory in whole rows.
template <int D>
__global__ void __launch_bounds__(128)
paged_chunk_merge_kernel(const ChunkParams p) {
  constexpr int kCols = D / 4;
  __shared__ __align__(16) __nv_bfloat16 s_out[32][D + 8];
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  paged_wait_before();
  const SplitChunk it = p.split[cta];
  const int r0 = blockIdx.y * 32, r = r0 + lane;
  if (it.n == 0 || r0 >= it.rows) return;
  auto slot_of = [&](int i) -> long long { return i == 0 ? cta * 2 + 1 : (cta + i) * 2; };
  auto ml_of = [&](int i) { return *reinterpret_cast<const float2*>(p.part_ml + (slot_of(i) * kRows + r) * 2); };
  float M = -INFINITY, L = 0.f;
  for (int i = 0; i < it.n; ++i) M = fmaxf(M, ml_of(i).x);
  float o[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) o[j] = 0.f;
  for (int i = 0; i < it.n; ++i) {
    const float2 ml = ml_of(i);
    const float f = ml.y != 0.f ? ex2(ml.x - M) : 0.f;
    if (ml.y != 0.f) L = fmaf(f, ml.y, L);
    const float* src = p.part_o + (slot_of(i) * D + warp * kCols) * kRows + r;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const float v = src[(long long)j * kRows];
      if (f != 0.f) o[j] = fmaf(f, v, o[j]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int j = 0; j < kCols; j += 2)
    *reinterpret_cast<uint32_t*>(&s_out[lane][warp * kCols + j]) = pack_bf16x2(o[j] * inv, o[j + 1] * inv);
  auto row_at = [&](int x) -> long long {
    const int rr = it.first + x;
    return (long long)(it.t0 + rr / p.G) * p.Hq + it.h * p.G + rr % p.G;
  };
  if (warp == 0 && r < it.rows && p.lse != nullptr)
    p.lse[row_at(r)] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPagedLn2;
  __syncthreads();
  constexpr int kCh = D / 8;
  for (int x = threadIdx.x; x < 32 * kCh; x += 128) {
    const int row = x / kCh, ch = x % kCh;
    if (r0 + row < it.rows)
      *reinterpret_cast<uint4*>(p.out + row_at(r0 + row) * D + ch * 8) = *reinterpret_cast<const uint4*>(&s_out[row][ch * 8]);
  }
}

template <bool kF8, int D, bool kCap, int kSub>
cudaError_t launch(const ChunkParams& p, cudaStream_t st) {
  using C = Cfg<D>;
  auto* kernel = paged_chunk_kernel<kF8, D, kCap, kSub>;
  static thread_local unsigned long long devices = 0;
  cudaError_t e = paged_allow_smem(kernel, C::kSmemBytes, &devices);
  if (e == cudaSuccess) e = paged_launch(kernel, dim3(kCtas), kThreads, C::kSmemBytes, st, p);
  if (e == cudaSuccess) e = paged_launch(paged_chunk_merge_kernel<D>, dim3(kCtas, kRows / 32), 128, 0, st, p);
  return e;
}

template <int D>
cudaError_t launch_f8(const ChunkParams& p, cudaStream_t st) {
  const bool cap = p.cap > 0.f;
  if (p.c.p_shift >= 6) return cap ? launch<true, D, true, 1>(p, st) : launch<true, D, false, 1>(p, st);
  return cap ? launch<true, D, true, 4>(p, st) : launch<true, D, false, 4>(p, st);
}
template <int D>
cudaError_t launch_bf16(const ChunkParams& p, cudaStream_t st) {
  return p.cap > 0.f ? launch<false, D, true, 1>(p, st) : launch<false, D, false, 1>(p, st);
}

constexpr size_t kItemBytes = sizeof(SplitChunk) * kCtas;
constexpr size_t kMlBytes = sizeof(float) * 2 * 2 * kCtas * kRows;

}  // namespace

size_t paged_chunk_workspace_bytes(int D) {
  return kItemBytes + kMlBytes + sizeof(float) * 2 * kCtas * kRows * (size_t)D;
}

unsigned read_and_clear_error_chunk(cudaStream_t, std::string* where) {
  DevError w{0u, 0u, 0}, zero{0u, 0u, 0};
  cudaMemcpyFromSymbol(&w, g_err_chunk, sizeof(w));
  if (w.flags) {
    cudaMemcpyToSymbol(g_err_chunk, &zero, sizeof(zero));
    char buf[128];
    if (w.where)
      snprintf(buf, sizeof(buf), " [paged attention chunk role %u barrier %u CTA %d]", (w.where >> 16) & 0xFFu,
               w.where & 0xFFFFu, w.item);
    else
      snprintf(buf, sizeof(buf), " (paged attention: a length, a token offset or a page number out of range)");
    *where += buf;
  }
  return w.flags;
}

int launch_paged_chunk(const PagedView& c, int f8, int D, const void* q, long long q_tok, int Hq, float scale,
                       int window_left, int window_right, float cap, void* out, float* lse,
                       void* workspace, cudaStream_t stream) {
  ChunkParams p;
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_tok;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.split = reinterpret_cast<SplitChunk*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + kItemBytes);
  p.part_o = reinterpret_cast<float*>(ws + kItemBytes + kMlBytes);
  p.Hq = Hq;
  p.G = Hq / c.Hkv;
  p.scale = scale;
  p.cap = cap;
  p.window_left = window_left;
  p.window_right = window_right;
  p.wait_limit = wait_timeout_cycles();
  cudaError_t e;
  if (D == 128)
    e = f8 ? launch_f8<128>(p, stream) : launch_bf16<128>(p, stream);
  else
    e = f8 ? launch_f8<64>(p, stream) : launch_bf16<64>(p, stream);
  if (e != cudaSuccess) return cuda_error(e, "paged attention chunk launch");
  return SBA_OK;
}

}  // namespace sba
