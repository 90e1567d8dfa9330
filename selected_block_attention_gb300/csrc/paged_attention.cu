// Attention of one or several query tokens per row over a paged cache:
// paged_attention_kernel.
//
// Row b's n_b query tokens are the last of its len_b tokens: query i sits at position
// p_i = len_b - n_b + i and sees key k < len_b iff p_i - window_left <= k <= p_i +
// window_right (a bound < 0 is open) or k < num_sinks.  Logit scale <q, k>, then cap
// tanh(. / cap), then + sink bias; the softmax is kept in fp32.
//
// Split.  An item is (batch row, KV head, 16 (query, head) rows); its keys are tiles of 32
// (e4m3) or 16 (bf16).  All items' tiles in order form one line that is cut into equal
// runs, one for each of kCtas CTAs (three per SM), so every CTA reads the same amount
// whatever the lengths are; each finds its place from the lengths on the device, and the
// grid does not depend on them.  A run that holds an item whole writes its output; else
// the item's partials (o, m, l) go to the workspace, two slots per CTA, and the CTA that
// counts the item complete merges them in the order of the line, so results do not
// depend on timing.  The counters are cleared by a small kernel that this one overlaps.
#include <string>

#include "paged_core.cuh"

namespace sba {

static __device__ unsigned g_err_paged = 0;

namespace {

constexpr int kThreads = kPagedWarps * 32;
constexpr int kCtas = 456;    // three for each of 152 SMs
constexpr int kMinTiles = 4;  // tiles of a run, at least: one for each warp

struct PagedAttnParams {
  PagedView c;
  const __nv_bfloat16* q;  // [N, Hq, D], q_tok elements between tokens
  long long q_tok;
  const float* sink_bias;
  __nv_bfloat16* out;  // [N, Hq, D]
  float* lse;          // [N, Hq] or null
  int* counters;       // [kCtas]
  float* part_ml;      // [2 kCtas][16][2]
  float* part_o;       // [2 kCtas][16][D]
  int Hq, G;
  float scale, cap;
  int window_left, window_right, num_sinks, sink_per_head;
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

template <bool kF8, int kD, bool kHi, bool kCap>
__global__ void __launch_bounds__(kThreads, 3)
paged_attention_kernel(const PagedAttnParams p) {
  using W = PagedWarp<kF8, kD, kHi, kCap>;
  constexpr int kKeys = W::kKeys;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kPagedWarps];
  __shared__ long long s_total, s_off;
  __shared__ int s_row, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

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
      sum += (long long)t.tiles * t.groups * p.c.Hkv;
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
    for (int i = 0; i < kPagedWarps; ++i) {
      if (i == warp) pre += total;
      total += s_sum[i];
    }
    pre -= sum;  // tiles before this thread's rows
    const long long per = max((total + kCtas - 1) / kCtas, (long long)kMinTiles);
    const long long t0 = (long long)cta * per;
    if (t0 >= pre && t0 < pre + sum) {
      long long off = t0 - pre;
      int b = b0;
      for (;; ++b) {
        bool x;
        const RowTiles t = row_tiles<kKeys>(p, b, &x);
        const long long n = (long long)t.tiles * t.groups * p.c.Hkv;
        if (off < n) break;
        off -= n;
      }
      s_row = b;
      s_off = off;
    }
    if (tid == 0) s_total = total;
    __syncthreads();
  }
  const long long total = s_total;
  const long long per = max((total + kCtas - 1) / kCtas, (long long)kMinTiles);
  long long cur = (long long)cta * per;
  const long long end = min(cur + per, total);
  int b = s_row;
  long long off = s_off;
  // The counters were cleared by the launch before this one, which may still be running.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (cur >= end) return;

  const uint32_t ring = ptx::smem_u32(smem) + warp * W::kWarpBytes;
  float* so = reinterpret_cast<float*>(smem);          // [warps][16][kSmemRow]
  float* sm = so + kPagedWarps * 16 * W::kSmemRow;     // [warps][16][3]
  float* sw = sm + kPagedWarps * 16 * 3;               // [16][warps + 2]: weights, max, sum

  while (cur < end) {
    bool bad;
    const RowTiles rt = row_tiles<kKeys>(p, b, &bad);
    const long long row_total = (long long)rt.tiles * rt.groups * p.c.Hkv;
    if (off >= row_total) {
      off -= row_total;
      ++b;
      continue;
    }
    const int item = (int)(off / rt.tiles);
    const int s0 = (int)(off - (long long)item * rt.tiles);
    const int s1 = (int)min((long long)rt.tiles, s0 + (end - cur));
    const int h = item / rt.groups, group = item - h * rt.groups;
    const int n_rows = min(16, rt.r.n * p.G - group * 16);
    const int first_pos = rt.r.len - rt.r.n;  // position of query 0

    PagedMask mk;
    mk.len = rt.r.len;
    mk.num_sinks = p.num_sinks;
    const int ra = group * 16 + (lane >> 2), rb = ra + 8;
    const bool ok0 = ra < rt.r.n * p.G, ok1 = kHi && rb < rt.r.n * p.G;
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
    const int ia = group * 16 / p.G, ib = (group * 16 + n_rows - 1) / p.G;  // queries of the group
    mk.all_lo = win_lo(ib);
    mk.all_hi = win_hi(ia);
    mk.bias0 = p.sink_bias + (p.sink_per_head ? (long long)h0 * p.num_sinks : 0);
    mk.bias1 = p.sink_bias + (p.sink_per_head ? (long long)h1 * p.num_sinks : 0);
    // tiles this group needs: [ka, kb) of the window's
    const bool sinks_at_base = p.num_sinks > 0 && !rt.sink;
    const int lo = sinks_at_base ? 0 : min(win_lo(ia), rt.r.len);
    int hi = (int)min((long long)max(win_hi(ib), -1) + 1, (long long)rt.r.len);
    if (sinks_at_base) hi = max(hi, min(p.num_sinks, rt.r.len));
    const int ka = (lo - rt.base) / kKeys;
    const int kb = hi > lo ? (hi - rt.base + kKeys - 1) / kKeys : ka;
    const int cl = sinks_at_base ? 0 : rt.lo;
    // tiles of the segment [s0, s1): the sinks' tile, then the window's
    const bool with_sink = rt.sink && s0 == 0;
    const int wa = max(s0 - rt.sink, ka), wb = min(s1 - rt.sink, kb);
    const int count = (with_sink ? 1 : 0) + max(wb - max(wa, 0), 0);
    const int w_first = max(wa, 0) - (with_sink ? 1 : 0);  // window tile of index t: w_first + t

    W w;
    w.init(p.c, b, h, ring, p.scale, p.cap, &g_err_paged);
    w.load_q(ok0 ? p.q + (rt.r.t0 + i0) * p.q_tok + (long long)h0 * kD : nullptr,
             ok1 ? p.q + (rt.r.t0 + i1) * p.q_tok + (long long)h1 * kD : nullptr);
    w.walk(
        warp, kPagedWarps, rt.r.len > 0 ? count : 0,
        [&](int t) { return (with_sink && t == 0) ? 0 : rt.base + (w_first + t) * kKeys; },
        [&](int t, int& c0, int& c1) {
          const bool s = with_sink && t == 0;
          c0 = s ? 0 : cl;
          c1 = s ? min(p.num_sinks, rt.r.len) - 1 : rt.r.len - 1;
        },
        mk);

    // ---- the CTA's warps become one partial
    __syncthreads();  // the rings become the merge buffer
    w.park(so, sm, warp);
    __syncthreads();
    if (tid < n_rows) {
      float M, L, wt[kPagedWarps];
      paged_merge_row(sm, tid, M, L, wt);
#pragma unroll
      for (int i = 0; i < kPagedWarps; ++i) sw[tid * (kPagedWarps + 2) + i] = wt[i];
      sw[tid * (kPagedWarps + 2) + kPagedWarps] = M;
      sw[tid * (kPagedWarps + 2) + kPagedWarps + 1] = L;
    }
    __syncthreads();
    const bool begins = s0 == 0, whole = begins && s1 == rt.tiles;
    auto out_row = [&](int r) -> long long {
      const int rr = group * 16 + r;
      return (long long)(rt.r.t0 + rr / p.G) * p.Hq + h * p.G + rr % p.G;
    };
    auto write = [&](int r, int pos, float O, float M, float L) {
      const long long row = out_row(r);
      p.out[row * kD + W::dim_of(pos)] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
      if (p.lse != nullptr && pos == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPagedLn2;
    };
    const int slot = cta * 2 + (begins ? 1 : 0);
    for (int x = tid; x < n_rows * kD; x += kThreads) {
      const int r = x / kD, pos = x % kD;
      const float* wt = sw + r * (kPagedWarps + 2);
      float O = 0.f;
#pragma unroll
      for (int i = 0; i < kPagedWarps; ++i)
        if (wt[i] != 0.f) O = fmaf(wt[i], so[(i * 16 + r) * W::kSmemRow + pos], O);
      const float M = wt[kPagedWarps], L = wt[kPagedWarps + 1];
      if (whole) {
        write(r, pos, O, M, L);
      } else {
        p.part_o[((long long)slot * 16 + r) * kD + pos] = O;
        if (pos == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * 16 + r) * 2) = make_float2(M, L);
      }
    }
    if (!whole) {
      // Partials visible before the count; the CTA that counts the last one merges.
      const long long g0 = cur - s0;  // the item's first tile
      const int ca = (int)(g0 / per), cb = (int)((g0 + rt.tiles - 1) / per);
      const int n = cb - ca + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(p.counters + ca, 1) == n - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        auto slot_of = [&](int i) { return i == 0 ? ca * 2 + 1 : (ca + i) * 2; };
        // eight lanes to a row: the common max and sum
        float* st = so;  // [16][2]
        {
          const int r = tid >> 3, k = tid & 7;
          float M = -INFINITY, L = 0.f;
          if (r < n_rows)
            for (int i = k; i < n; i += 8) M = fmaxf(M, __ldcg(p.part_ml + (slot_of(i) * 16 + r) * 2));
#pragma unroll
          for (int d = 1; d < 8; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
          if (r < n_rows)
            for (int i = k; i < n; i += 8) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (slot_of(i) * 16 + r) * 2));
              if (ml.y != 0.f) L = fmaf(ptx::ex2(ml.x - M), ml.y, L);
            }
#pragma unroll
          for (int d = 1; d < 8; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
          if (k == 0) {
            st[r * 2] = M;
            st[r * 2 + 1] = L;
          }
        }
        __syncthreads();
        for (int x = tid; x < n_rows * kD; x += kThreads) {
          const int r = x / kD, pos = x % kD;
          const float M = st[r * 2], L = st[r * 2 + 1];
          float O = 0.f;
#pragma unroll 4
          for (int i = 0; i < n; ++i) {
            const int s = slot_of(i);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (s * 16 + r) * 2));
            const float v = __ldcg(p.part_o + ((long long)s * 16 + r) * kD + pos);
            if (ml.y != 0.f) O = fmaf(ptx::ex2(ml.x - M), v, O);
          }
          write(r, pos, O, M, L);
        }
      }
    }
    __syncthreads();  // the merge buffer becomes the rings again
    cur += s1 - s0;
    off += s1 - s0;
  }
}

// Clears the counters; the attention kernel may start meanwhile (programmatic dependent
// launch) and waits for this one before it counts.
__global__ void paged_clear_kernel(int* counters) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < kCtas; i += blockDim.x) counters[i] = 0;
}

template <bool kF8, int kD, bool kHi, bool kCap>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t st) {
  using W = PagedWarp<kF8, kD, kHi, kCap>;
  constexpr int ring = kPagedWarps * W::kWarpBytes;
  constexpr int merge = (kPagedWarps * 16 * (W::kSmemRow + 3) + 16 * (kPagedWarps + 2)) * 4;
  constexpr int bytes = ring > merge ? ring : merge;
  auto* kernel = paged_attention_kernel<kF8, kD, kHi, kCap>;
  static thread_local unsigned long long set = 0;  // devices whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((set >> dev) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set |= 1ull << dev;
  }
  paged_clear_kernel<<<1, 512, 0, st>>>(p.counters);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool kF8, int kD>
cudaError_t launch_d(const PagedAttnParams& p, bool hi, cudaStream_t st) {
  const bool cap = p.cap > 0.f;
  if (hi) return cap ? launch<kF8, kD, true, true>(p, st) : launch<kF8, kD, true, false>(p, st);
  return cap ? launch<kF8, kD, false, true>(p, st) : launch<kF8, kD, false, false>(p, st);
}

constexpr size_t kCounterBytes = 2048;
static_assert(kCounterBytes >= kCtas * sizeof(int), "one counter per CTA");
constexpr size_t kMlBytes = sizeof(float) * 2 * 2 * kCtas * 16;

}  // namespace

size_t paged_attention_workspace_bytes(int D) {
  return kCounterBytes + kMlBytes + sizeof(float) * 2 * kCtas * 16 * (size_t)D;
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
  PagedAttnParams p;
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_tok;
  p.sink_bias = sink_bias;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counters = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + kCounterBytes);
  p.part_o = reinterpret_cast<float*>(ws + kCounterBytes + kMlBytes);
  p.Hq = Hq;
  p.G = Hq / c.Hkv;
  p.scale = scale;
  p.cap = cap;
  p.window_left = window_left;
  p.window_right = window_right;
  p.num_sinks = num_sinks;
  p.sink_per_head = sink_per_head;
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
