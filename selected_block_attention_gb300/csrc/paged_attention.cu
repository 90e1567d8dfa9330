// Attention of one or several query tokens per row over a paged cache:
// paged_attention_kernel, paged_merge_kernel and, for few keys, paged_small_kernel.
//
// Row b's n_b query tokens are the last of its len_b tokens: query i sits at position
// p_i = len_b - n_b + i and sees key k < len_b iff p_i - window_left <= k <= p_i +
// window_right (a bound < 0 is open) or k < num_sinks.  Logit scale <q, k>, then cap
// tanh(. / cap), then + sink bias; the softmax is kept in fp32.
//
// Split.  An item is (batch row, KV head, 16 (query, head) rows); its keys are tiles of
// 4 KB of keys and 4 KB of values.  All items' tiles in order form one line that is cut
// into equal runs, one for each of kCtas CTAs (three per SM), so every CTA reads the same
// amount whatever the lengths are; each finds its place from the lengths on the device, and
// the grid does not depend on them.  An item's fixed cost (its queries, the merge of the
// CTA's warps) is kItemCost empty tiles ahead of its own, so that a run of many short items
// takes no longer than a run inside a long one.  A run that holds an item whole writes its
// output; else the item's partials (o, m, l) go to the workspace, two slots per CTA, and
// paged_merge_kernel, launched behind this one with its start overlapped, adds them up in
// the order of the line, so results do not depend on timing.
//
// What bounds it: the bytes of keys and values, with the work on a tile close behind.  One
// token for each of 4 rows, 64 heads over 4, D = 128, e4m3, 60000 to 131072 keys: 405 MB in
// 77.3 us (5.2 TB/s), of which 6 are the launch, the search for a run's place and the merge;
// the schedulers issue in 52 % of the cycles (three warps each) and the time that a warp
// waits for memory is an eighth of its own, so a warp's chain of conversions, MMAs and softmax
// steps is what is left.  64 rows with a window of 4096, cap and sinks: 503 MB in 96.0 us, the
// same with a tanh in the chain (93.4 without the cap).  Tried and left (against 78.2 then):
// tiles by TMA, one lane issuing (80.0), six warps a CTA, two CTAs an SM (77.2, but windows
// 98.0 against 93.7 and drafts 34.5 against 31.8); for D = 64 two groups of 16 rows sharing a
// warp's tiles (drafts 36.4 against 32.0).
#include <algorithm>
#include <string>

#include "paged_core.cuh"

namespace sba {

static __device__ unsigned g_err_paged = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtas = 456;    // three for each of 152 SMs
constexpr int kMinTiles = 4;  // tiles of a run, at least: one for each warp
constexpr int kItemCost = 12;  // tiles that an item's fixed cost is worth
// Tiles of a warp, at most, in paged_small_kernel, by the table's width (lengths are the
// device's).  Line and cluster, us, e4m3 D = 128, 8 KV heads, equal lengths and tables as wide:
// one row of 2000 keys 10.6 / 6.8, of 8000 17.6 / 12.9, of 16000 19.8 / 21.1; 16 rows of 2000
// 21.8 / 17.8, of 8000 51.4 / 50.2; 48 rows of 300 16.2 / 9.2.  Past 8 tiles a warp the two
// come level, and the cluster's fixed shares lose to the line once the rows' lengths differ.
// So one short row behind a wide table takes the line: 2011 keys, table of 131072: 10.8.
constexpr int kSmallTiles = 8;

struct PagedAttnParams {
  PagedView c;
  const __nv_bfloat16* q;  // [N, Hq, D], q_tok elements between tokens
  long long q_tok;
  const float* sink_bias;
  __nv_bfloat16* out;  // [N, Hq, D]
  float* lse;          // [N, Hq] or null
  struct SplitItem* split;  // [kCtas]
  float* part_ml;      // [2 kCtas][16][2]
  float* part_o;       // [2 kCtas][16][D]
  int Hq, G;
  float scale, cap;
  int window_left, window_right, num_sinks, sink_per_head;
  int cluster, groups;  // few keys: CTAs of an item and items of a KV head (else cluster = 0)
};

// The item that a CTA begins but does not end: its partials are slot 2 cta + 1 and the
// slots 2 (cta + i), 0 < i < n.  n = 0: there is none.
struct SplitItem {
  int n, n_rows, first, t0, h;  // rows first .. first + n_rows of the row's (query, head) rows
  int pad[3];
};

// The tiles of a row's items: all items of a row get the same number, that of the union
// of its queries' windows, and skip what their own queries do not see.
struct RowTiles {
  PagedRow r;
  int lo;      // first key of the first query's window
  int base;    // lo, down to a multiple of the tile
  int sink;    // 1: tile 0 is keys [0, kKeys) for the sinks, apart from the window's tiles
  int tiles;   // per item, at least 1
  int groups;  // 16-row groups
};
template <int kKeys>
__device__ __forceinline__ RowTiles row_tiles(const PagedAttnParams& p, int b, bool* bad) {
  RowTiles t;
  t.r = paged_row(p.c, b, bad);
  t.lo = 0;
  if (p.window_left >= 0) t.lo = (int)min(max((long long)t.r.len - t.r.n - p.window_left, 0LL), (long long)t.r.len);
  t.base = t.lo & ~(kKeys - 1);
  t.sink = p.num_sinks > 0 && t.base > 0;
  t.tiles = max(1, (t.r.len - t.base + kKeys - 1) / kKeys + t.sink);
  t.groups = (int)(((long long)t.r.n * p.G + 15) >> 4);
  return t;
}

// The 16 rows of an item, what they see, and the item's tiles of [s0, s1) that they need.
template <int kD>
struct Group {
  PagedMask mk;
  const __nv_bfloat16* q0;  // the thread's rows g and g + 8, or null
  const __nv_bfloat16* q1;
  int n_rows;
  int count, key_first;  // tile t < count is the keys from key_first + t kKeys on ...
  bool with_sink;        // ... but for tile 0, which is the sinks'
  int cl, ch;            // keys that may be read, besides sinks; of the sinks' tile, 0 .. sink_ch
  int sink_ch;
  template <int kKeys>
  __device__ __forceinline__ int key_of(int t) const {
    return with_sink && t == 0 ? 0 : key_first + t * kKeys;
  }
  __device__ __forceinline__ void limits(int t, int& lo, int& hi) const {
    const bool s = with_sink && t == 0;
    lo = s ? 0 : cl;
    hi = s ? sink_ch : ch;
  }
};
template <int kKeys, bool kHi, int kD>
__device__ __forceinline__ Group<kD> group_of(const PagedAttnParams& p, const RowTiles& rt, int h, int group, int s0,
                                              int s1) {
  Group<kD> gr;
  const int lane = threadIdx.x & 31, rows = rt.r.n * p.G;
  const int first_pos = rt.r.len - rt.r.n;  // position of query 0
  gr.n_rows = min(16, rows - group * 16);
  PagedMask& mk = gr.mk;
  mk.len = rt.r.len;
  mk.num_sinks = p.num_sinks;
  const int ra = group * 16 + (lane >> 2), rb = ra + 8;
  const bool ok0 = ra < rows, ok1 = kHi && rb < rows;
  const int i0 = ok0 ? ra / p.G : 0, i1 = ok1 ? rb / p.G : 0;
  const int h0 = h * p.G + (ok0 ? ra - i0 * p.G : 0), h1 = h * p.G + (ok1 ? rb - i1 * p.G : 0);
  auto win_lo = [&](int i) {
    return p.window_left < 0 ? 0 : (int)max((long long)first_pos + i - p.window_left, 0LL);
  };
  auto win_hi = [&](int i) {
    return p.window_right < 0 ? INT_MAX : (int)min((long long)first_pos + i + p.window_right, (long long)INT_MAX);
  };
  mk.wlo0 = win_lo(i0);
  mk.whi0 = ok0 ? win_hi(i0) : -1;
  mk.wlo1 = win_lo(i1);
  mk.whi1 = ok1 ? win_hi(i1) : -1;
  const int ia = group * 16 / p.G, ib = (group * 16 + gr.n_rows - 1) / p.G;  // queries of the group
  mk.all_lo = win_lo(ib);
  mk.all_hi = win_hi(ia);
  mk.bias0 = p.sink_bias + (p.sink_per_head ? (long long)h0 * p.num_sinks : 0);
  mk.bias_step = p.sink_per_head ? (h1 - h0) * p.num_sinks : 0;
  // tiles this group needs: [ka, kb) of the window's
  const bool sinks_at_base = p.num_sinks > 0 && !rt.sink;
  const int lo = sinks_at_base ? 0 : min(win_lo(ia), rt.r.len);
  int hi = (int)min((long long)max(win_hi(ib), -1) + 1, (long long)rt.r.len);
  if (sinks_at_base) hi = max(hi, min(p.num_sinks, rt.r.len));
  const int ka = (lo - rt.base) / kKeys;
  const int kb = hi > lo ? (hi - rt.base + kKeys - 1) / kKeys : ka;
  // of the segment [s0, s1): the sinks' tile, then the window's
  gr.with_sink = rt.sink && s0 == 0;
  const int wa = max(max(s0 - rt.sink, ka), 0), wb = min(s1 - rt.sink, kb);
  gr.count = rt.r.len > 0 ? (gr.with_sink ? 1 : 0) + max(wb - wa, 0) : 0;
  gr.key_first = rt.base + (wa - (gr.with_sink ? 1 : 0)) * kKeys;
  gr.cl = rt.lo;
  gr.ch = rt.r.len - 1;
  gr.sink_ch = min(p.num_sinks, rt.r.len) - 1;
  gr.q0 = ok0 ? p.q + (rt.r.t0 + i0) * p.q_tok + (long long)h0 * kD : nullptr;
  gr.q1 = ok1 ? p.q + (rt.r.t0 + i1) * p.q_tok + (long long)h1 * kD : nullptr;
  return gr;
}

template <bool kF8, int kD, bool kHi, bool kCap, bool kSinks>
__global__ void __launch_bounds__(kThreads, 3)
paged_attention_kernel(const PagedAttnParams p) {
  using W = PagedWarp<kF8, kD, 4096 / (kD * (kF8 ? 1 : 2)), kHi, kCap, kSinks>;
  constexpr int kKeys = W::kKeys;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kWarps];
  __shared__ long long s_total, s_off;
  __shared__ int s_row;
  // what the CTA needs again after an item's tiles; kept here to leave registers to them
  __shared__ struct {
    long long cur, off, item_at;
    int b, units, h, first, n_rows, t0, begins, whole;
  } s_it;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  paged_wait_before();

  // ---- this CTA's run [t0, t1) of the line, and the row it begins in
  {
    const int chunk = (p.c.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * chunk, p.c.B), b1 = min(b0 + chunk, p.c.B);
    long long sum = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      bool x;
      const RowTiles t = row_tiles<kKeys>(p, b, &x);
      bad |= x;
      sum += (long long)(t.tiles + kItemCost) * t.groups * p.c.Hkv;
    }
    if (bad && cta == 0) atomicOr(&g_err_paged, (unsigned)kDevErrInput);
    long long pre = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, pre, d);
      if (lane >= d) pre += x;
    }
    if (lane == 31) s_sum[warp] = pre;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) pre += total;
      total += s_sum[i];
    }
    pre -= sum;  // tiles before this thread's rows
    const long long per = max((total + kCtas - 1) / kCtas, (long long)kMinTiles);
    const long long t0 = (long long)cta * per;
    if (t0 >= pre && t0 < pre + sum) {
      long long off = t0 - pre;
      int b = b0;
      for (; b + 1 < b1; ++b) {  // (bounded, should the lengths change under the call)
        bool x;
        const RowTiles t = row_tiles<kKeys>(p, b, &x);
        const long long n = (long long)(t.tiles + kItemCost) * t.groups * p.c.Hkv;
        if (off < n) break;
        off -= n;
      }
      s_row = b;
      s_off = off;
    }
    if (tid == 0) s_total = total;
    __syncthreads();
  }
  auto run_length = [&]() { return max((s_total + kCtas - 1) / kCtas, (long long)kMinTiles); };
  long long cur = cta * run_length();
  int b = s_row;
  long long off = s_off;
  paged_let_next();
  if (tid == 0) p.split[cta].n = 0;

  const uint32_t ring = ptx::smem_u32(smem) + warp * W::kWarpBytes;
  float* so = reinterpret_cast<float*>(smem);          // [warps][16][kSmemRow]
  float* sm = so + kWarps * 16 * W::kSmemRow;     // [warps][16][3]
  float* sw = sm + kWarps * 16 * 3;               // [16][warps + 2]: weights, max, sum

  while (true) {
    const long long end = min((cta + 1) * run_length(), s_total);
    if (cur >= end) return;
    bool bad;
    const RowTiles rt = row_tiles<kKeys>(p, b, &bad);
    const int units = rt.tiles + kItemCost;
    const long long row_total = (long long)units * rt.groups * p.c.Hkv;
    if (off >= row_total) {
      off -= row_total;
      if (++b >= p.c.B) return;
      continue;
    }
    const int item = (int)(off / units);
    const int x0 = (int)(off - (long long)item * units);
    const int x1 = (int)min((long long)units, x0 + (end - cur));
    const long long item_at = cur - x0;  // the item's place on the line
    cur += x1 - x0;
    off += x1 - x0;
    if (x1 <= kItemCost) continue;  // nothing but the empty tiles
    const int s0 = max(x0 - kItemCost, 0), s1 = x1 - kItemCost;
    const int h = item / rt.groups, group = item - h * rt.groups;
    const Group<kD> gr = group_of<kKeys, kHi, kD>(p, rt, h, group, s0, s1);

    if (tid == 0) {
      s_it.cur = cur;
      s_it.off = off;
      s_it.item_at = item_at;
      s_it.b = b;
      s_it.units = units;
      s_it.h = h;
      s_it.first = group * 16;
      s_it.n_rows = gr.n_rows;
      s_it.t0 = rt.r.t0;
      s_it.begins = s0 == 0;
      s_it.whole = s0 == 0 && s1 == rt.tiles;
    }
    W w;
    w.init(p.c, b, h, ring, p.scale, p.cap, &g_err_paged);
    w.walk(
        warp, kWarps, gr.count, [&](int t) { return gr.template key_of<kKeys>(t); },
        [&](int t, int& lo, int& hi) { gr.limits(t, lo, hi); }, [&] { w.load_q(gr.q0, gr.q1); }, gr.mk);

    // ---- the CTA's warps become one partial
    __syncthreads();  // the rings become the merge buffer
    w.park(so, sm, warp);
    __syncthreads();
    const int rows = s_it.n_rows;
    if (tid < rows) paged_merge_row<kWarps>(sm, tid, sw + tid * (kWarps + 2));
    __syncthreads();
    const bool begins = s_it.begins, whole = s_it.whole;
    const int slot = cta * 2 + (begins ? 1 : 0);
    for (int x = tid; x < rows * (kD / 8); x += kThreads) {
      const int r = x / (kD / 8), d0 = x % (kD / 8) * 8;
      const float* wt = sw + r * (kWarps + 2);
      const float M = wt[kWarps], L = wt[kWarps + 1];
      float O[8];
      paged_merge_dims<W, kWarps>(so, wt, r, d0, O);
      if (whole) {
        const int rr = s_it.first + r;
        const long long row = (long long)(s_it.t0 + rr / p.G) * p.Hq + s_it.h * p.G + rr % p.G;
        paged_store_row(p.out + row * kD + d0, O, L == 0.f ? 0.f : 1.f / L);
        if (p.lse != nullptr && d0 == 0) p.lse[row] = paged_lse(M, L);
      } else {
        float4* to = reinterpret_cast<float4*>(p.part_o + ((long long)slot * 16 + r) * kD + d0);
        to[0] = make_float4(O[0], O[1], O[2], O[3]);
        to[1] = make_float4(O[4], O[5], O[6], O[7]);
        if (d0 == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * 16 + r) * 2) = make_float2(M, L);
      }
    }
    if (begins && !whole && tid == 0) {
      // the CTA that ends the item
      const int last = (int)min((s_it.item_at + s_it.units - 1) / run_length(), (long long)kCtas - 1);
      SplitItem it;
      it.n = last - cta + 1;
      it.n_rows = rows;
      it.first = s_it.first;
      it.t0 = s_it.t0;
      it.h = s_it.h;
      p.split[cta] = it;
    }
    cur = s_it.cur;
    off = s_it.off;
    b = s_it.b;
    __syncthreads();  // the merge buffer becomes the rings again
  }
}

// One warp for each row of an item that a CTA begins and others continue: the partials'
// common max, their weights, and the weighted sum, four (kD = 64: two) columns a lane.
template <int kD>
__global__ void __launch_bounds__(128)
paged_merge_kernel(const PagedAttnParams p) {
  constexpr int kCols = kD / 32;
  const int cta = blockIdx.x, r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  paged_wait_before();
  auto ml_of = [&](int i) {
    const int slot = i == 0 ? cta * 2 + 1 : (cta + i) * 2;
    return *reinterpret_cast<const float2*>(p.part_ml + (slot * 16 + r) * 2);
  };
  // the first 32 partials' (max, sum) are on their way before it is known how many there are
  const float2 first = cta + lane < kCtas ? ml_of(lane) : make_float2(0.f, 0.f);
  const SplitItem it = p.split[cta];
  if (it.n == 0 || r >= it.n_rows) return;
  float M = lane < it.n ? first.x : -INFINITY, L = 0.f;
  for (int i = 32 + lane; i < it.n; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float O[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) O[c] = 0.f;
  for (int base = 0; base < it.n; base += 32) {
    const float2 ml = base + lane < it.n ? (base == 0 ? first : ml_of(base + lane)) : make_float2(0.f, 0.f);
    const float f = ml.y != 0.f ? ptx::ex2(ml.x - M) : 0.f;
    if (ml.y != 0.f) L = fmaf(f, ml.y, L);
    const int n = min(32, it.n - base);
    // sixteen partials in flight (a few of the last group are read twice, with weight 0)
    for (int i0 = 0; i0 < n; i0 += 16) {
      float v[16][kCols];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int i = base + min(i0 + x, n - 1);
        const int slot = i == 0 ? cta * 2 + 1 : (cta + i) * 2;
        const float* src = p.part_o + ((long long)slot * 16 + r) * kD + lane * kCols;
        if constexpr (kCols == 4)
          *reinterpret_cast<float4*>(v[x]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(v[x]) = *reinterpret_cast<const float2*>(src);
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float fi = __shfl_sync(0xffffffffu, f, (i0 + x) & 31);
        if (i0 + x < n && fi != 0.f) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) O[c] = fmaf(fi, v[x][c], O[c]);
        }
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
  const int rr = it.first + r;
  const long long row = (long long)(it.t0 + rr / p.G) * p.Hq + it.h * p.G + rr % p.G;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* to = reinterpret_cast<uint32_t*>(p.out + row * kD + lane * kCols);
#pragma unroll
  for (int c = 0; c < kCols; c += 2) to[c / 2] = pack_bf16x2(O[c] * inv, O[c + 1] * inv);
  if (p.lse != nullptr && lane == 0) p.lse[row] = paged_lse(M, L);
}

// Few keys: an item's tiles are shared evenly by the `split` CTAs of one cluster, which merge
// through distributed shared memory, so there is neither a line to find a place on nor a
// second launch.
template <bool kF8, int kD, bool kHi, bool kCap, bool kSinks>
__global__ void __launch_bounds__(kThreads, 3)
paged_small_kernel(const PagedAttnParams p) {
  using W = PagedWarp<kF8, kD, 4096 / (kD * (kF8 ? 1 : 2)), kHi, kCap, kSinks>;
  constexpr int kKeys = W::kKeys;
  extern __shared__ __align__(128) uint8_t smem[];
  const int split = p.cluster, part = blockIdx.x % split, warp = threadIdx.x >> 5;
  const int item = blockIdx.x / split, groups = p.groups;
  const int group = item % groups, h = item / groups % p.c.Hkv, b = item / groups / p.c.Hkv;
  paged_wait_before();
  bool bad;
  const RowTiles rt = row_tiles<kKeys>(p, b, &bad);
  if (bad && threadIdx.x == 0) atomicOr(&g_err_paged, (unsigned)kDevErrInput);
  const Group<kD> gr = group_of<kKeys, kHi, kD>(p, rt, h, group, 0, rt.tiles);
  W w;
  w.init(p.c, b, h, ptx::smem_u32(smem) + warp * W::kWarpBytes, p.scale, p.cap, &g_err_paged);
  const int a = (int)((long long)gr.count * part / split), e = (int)((long long)gr.count * (part + 1) / split);
  w.walk(
      a + warp, kWarps, e, [&](int t) { return gr.template key_of<kKeys>(t); },
      [&](int t, int& lo, int& hi) { gr.limits(t, lo, hi); }, [&] { w.load_q(gr.q0, gr.q1); }, gr.mk);
  const int first = group * 16;
  paged_cluster_finish<W, kWarps, kD>(
      w, smem, split, part, gr.n_rows,
      [&](int r) -> long long {
        return (long long)(rt.r.t0 + (first + r) / p.G) * p.Hq + h * p.G + (first + r) % p.G;
      },
      [](int, float L) { return L == 0.f ? 0.f : 1.f / L; }, p.out, p.lse);
}

template <bool kF8, int kD, bool kHi, bool kCap, bool kSinks>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t st) {
  using W = PagedWarp<kF8, kD, 4096 / (kD * (kF8 ? 1 : 2)), kHi, kCap, kSinks>;
  constexpr int ring = kWarps * W::kWarpBytes;
  constexpr int merge = (kWarps * 16 * (W::kSmemRow + 3) + 16 * (kWarps + 2)) * 4;
  constexpr int bytes = ring > merge ? ring : merge;
  auto* kernel = paged_attention_kernel<kF8, kD, kHi, kCap, kSinks>;
  if (p.cluster > 0) {
    constexpr int finish = paged_finish_bytes<W, kWarps, kD>(), need = ring > finish ? ring : finish;
    static thread_local unsigned long long devices = 0;
    auto* small = paged_small_kernel<kF8, kD, kHi, kCap, kSinks>;
    const cudaError_t e = paged_allow_smem(small, need, &devices);
    if (e != cudaSuccess) return e;
    return paged_launch(small, dim3((unsigned)(p.c.B * p.c.Hkv * p.groups * p.cluster)), kThreads, need, st, p, p.cluster);
  }
  static thread_local unsigned long long devices = 0;
  cudaError_t e = paged_allow_smem(kernel, bytes, &devices);
  if (e == cudaSuccess) e = paged_launch(kernel, dim3(kCtas), kThreads, bytes, st, p);
  if (e == cudaSuccess) e = paged_launch(paged_merge_kernel<kD>, dim3(kCtas, kHi ? 4 : 2), 128, 0, st, p);
  return e;
}

template <bool kF8, int kD, bool kHi>
cudaError_t launch_hi(const PagedAttnParams& p, cudaStream_t st) {
  const bool sinks = p.num_sinks > 0;
  if (p.cap > 0.f) return sinks ? launch<kF8, kD, kHi, true, true>(p, st) : launch<kF8, kD, kHi, true, false>(p, st);
  return sinks ? launch<kF8, kD, kHi, false, true>(p, st) : launch<kF8, kD, kHi, false, false>(p, st);
}
template <bool kF8, int kD>
cudaError_t launch_d(const PagedAttnParams& p, bool hi, cudaStream_t st) {
  return hi ? launch_hi<kF8, kD, true>(p, st) : launch_hi<kF8, kD, false>(p, st);
}

constexpr size_t kItemBytes = sizeof(SplitItem) * kCtas;
constexpr size_t kMlBytes = sizeof(float) * 2 * 2 * kCtas * 16;

}  // namespace

// (query, head) rows of a batch row and KV head, on average, from which a call may go to the
// kernel with tensor-memory accumulators (paged_chunk.cu).
static bool may_have_many_rows(int B, int N, int Hq, int Hkv) { return (long long)N * (Hq / Hkv) > 16LL * B; }

// Whether it does.  This file's kernel reads the keys once for each 16 rows, the other one
// once for 256 at a higher price a tile.  32 rows of 7000 to 8000 keys, 8 KV heads, by
// (query, head) rows (us, here / there; there the rows up to 128 cost alike): e4m3 D = 128
// 16: 91 / 207, 32: 159 / 207, 40: 236 / 207; bf16 D = 128 16: 159 / 189, 24: 287 / 189; e4m3
// D = 64 48: 150 / 155, 64: 193 / 155; bf16 D = 64 32: 124 / 144, 40: 225 / 144.  Two such
// rows: e4m3 D = 128 40: 25 / 39, 96: 39 / 40: with few keys this file's finer runs win; the
// tables bound the keys, and the lines cross near half a million.
static bool many_rows(const PagedView& c, int f8, int D, int Hq) {
  const long long rows = (long long)c.N * (Hq / c.Hkv), keys = (long long)c.B * c.Hkv * c.width << c.p_shift;
  const int from = keys < (1 << 19) ? 96 : (f8 ? (D == 128 ? 32 : 48) : (D == 128 ? 16 : 32));
  return rows > (long long)from * c.B;
}

size_t paged_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D) {
  const size_t few = kItemBytes + kMlBytes + sizeof(float) * 2 * kCtas * 16 * (size_t)D;
  return may_have_many_rows(B, N, Hq, Hkv) ? std::max(few, paged_chunk_workspace_bytes(D)) : few;
}

unsigned read_and_clear_error_paged(cudaStream_t, std::string* where) {
  unsigned w = 0, zero = 0;
  cudaMemcpyFromSymbol(&w, g_err_paged, sizeof(w));
  if (w) {
    cudaMemcpyToSymbol(g_err_paged, &zero, sizeof(zero));
    *where += " (paged attention: a length, a token offset or a page number out of range)";
  }
  return w;
}

int launch_paged_attention(const PagedView& c, int f8, int D, const void* q, long long q_tok, int Hq,
                           float scale, int window_left, int window_right, float cap,
                           const float* sink_bias, int num_sinks, int sink_per_head, void* out,
                           float* lse, void* workspace, cudaStream_t stream) {
  // Sinks are this file's alone, whatever the rows: a sinks' tile and its bias are not in the
  // other kernel's pipeline.  512-token chunks with 4 sinks take 1484 us here, without sinks
  // 262 there.
  if (num_sinks == 0 && many_rows(c, f8, D, Hq))
    return launch_paged_chunk(c, f8, D, q, q_tok, Hq, scale, window_left, window_right, cap, out, lse, workspace,
                              stream);
  PagedAttnParams p;
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_tok;
  p.sink_bias = sink_bias;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.split = reinterpret_cast<SplitItem*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + kItemBytes);
  p.part_o = reinterpret_cast<float*>(ws + kItemBytes + kMlBytes);
  p.Hq = Hq;
  p.G = Hq / c.Hkv;
  p.scale = scale;
  p.cap = cap;
  p.window_left = window_left;
  p.window_right = window_right;
  p.num_sinks = num_sinks;
  p.sink_per_head = sink_per_head;
  p.cluster = 0;
  p.groups = 0;
  if (c.cu == nullptr) {
    // Every row has Qn tokens, so the items are known here; the tables bound their keys.
    const int tile = 4096 / (D * (f8 ? 1 : 2));
    long long keys = (long long)c.width << c.p_shift;
    if (window_left >= 0) keys = std::min(keys, (long long)window_left + c.Qn + 2 * tile + (num_sinks > 0 ? tile : 0));
    const long long tiles = (keys + tile - 1) / tile, groups = ((long long)c.Qn * p.G + 15) / 16;
    const long long items = (long long)c.B * c.Hkv * groups;
    int split = 1;
    while (split < kPagedMaxSplit && items * split * 2 <= kCtas && tiles > split * kWarps) split *= 2;
    if (items * split <= kCtas && tiles <= kSmallTiles * kWarps * split) {
      p.cluster = split;
      p.groups = (int)groups;
    }
  }
  // A group of 16 (query, head) rows uses rows 8..15 unless a row has at most 8 of them.
  const bool hi = c.cu != nullptr || (long long)c.Qn * p.G > 8;
  cudaError_t e;
  if (D == 128)
    e = f8 ? launch_d<true, 128>(p, hi, stream) : launch_d<false, 128>(p, hi, stream);
  else
    e = f8 ? launch_d<true, 64>(p, hi, stream) : launch_d<false, 64>(p, hi, stream);
  if (e != cudaSuccess) return cuda_error(e, "paged attention launch");
  return SBA_OK;
}

}  // namespace sba
