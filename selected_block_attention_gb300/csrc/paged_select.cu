// Selected-block attention of decode tokens over a paged cache: paged_select_kernel.
//
// The decode form of the NSA selection branch: query token i of row b sits at position
// p = len_b - Q + i and attends, for each KV head, to the keys of the blocks named in
// block_indices[b, i, h, :count] (block ids of the row's own sequence; ids < 0, past its
// end or, when causal, past the token's block are ignored, order does not matter,
// duplicates count once), up to key p when causal.
//
// One item is (row, token, KV head) with its Hq / Hkv <= 16 query heads.  Its key set is
// small (at most 32 blocks), so an item's tiles are shared evenly among the `split` CTAs of
// one cluster, which merge through distributed shared memory: one launch, no workspace.
//
// What bounds it: two rows, the chain of block ids, page table, keys and merge: 4.6 us.  64
// rows of 16 blocks of 64 keys, 4 KV heads, D = 128, e4m3: 67 MB in 19.0 us, the same chain
// and 13 us of reading.  The 256 items are one CTA each, all at once on 152 SMs: 104 SMs hold
// two and 48 one, and as every CTA begins with the chain nothing hides it.
#include <string>

#include "paged_core.cuh"

namespace sba {

static __device__ unsigned g_err_select = 0;

namespace {

constexpr int kMaxBlocks = 32;
constexpr int kWarps = 4;

struct PagedSelectParams {
  PagedView c;
  const __nv_bfloat16* q;  // [B, Q, Hq, D], q_tok elements between tokens
  long long q_tok;
  const int* idx;  // [B, Q, Hkv, S]
  const int* cnt;  // [B, Q, Hkv] or null
  int cnt_scalar, S, block_size, causal, split;
  const __nv_bfloat16* gate;  // [B, Q, Hq] or null
  __nv_bfloat16* out;
  float* lse;
  int Hq, G;
  float scale;
};

template <bool kF8, int kD, bool kHi>
__global__ void __launch_bounds__(kWarps * 32, 3)
paged_select_kernel(const PagedSelectParams p) {
  using W = PagedWarp<kF8, kD, kF8 || kD == 64 ? 32 : 16, kHi, false, false>;
  constexpr int kKeys = W::kKeys;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_key[kMaxBlocks * 128 / kKeys];  // first key of each tile
  __shared__ int s_tiles;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = p.split, part = blockIdx.x % split;  // a cluster is `split` blocks along x
  const int h = blockIdx.x / split % p.c.Hkv, token = blockIdx.x / split / p.c.Hkv;
  const int b = token / p.c.Qn, qi = token - b * p.c.Qn;

  paged_wait_before();
  bool bad;
  const PagedRow r = paged_row(p.c, b, &bad);
  if (bad && tid == 0) atomicOr(&g_err_select, (unsigned)kDevErrInput);
  const int pos = r.len - p.c.Qn + qi;
  const int limit = max(p.causal ? min(pos + 1, r.len) : r.len, 0);  // keys below it are visible

  // ---- tiles of the item's distinct blocks
  if (warp == 0) {
    const long long item = (long long)token * p.c.Hkv + h;
    const int count = min(p.cnt != nullptr ? p.cnt[item] : p.cnt_scalar, p.S);
    const int id = lane < count ? p.idx[item * p.S + lane] : -1;
    const bool valid = id >= 0 && (long long)id * p.block_size < limit;
    const unsigned same = __match_any_sync(0xffffffffu, valid ? id : -1 - lane);
    const bool first = valid && (same & ((1u << lane) - 1u)) == 0u;
    const int key0 = first ? id * p.block_size : 0;
    const int n = first ? (min(p.block_size, limit - key0) + kKeys - 1) / kKeys : 0;
    int pre = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, pre, d);
      if (lane >= d) pre += x;
    }
    for (int i = 0; i < n; ++i) s_key[pre - n + i] = key0 + i * kKeys;
    if (lane == 31) s_tiles = pre;
  }

  PagedMask mk;
  mk.len = limit;
  mk.num_sinks = 0;
  mk.wlo0 = mk.wlo1 = mk.all_lo = 0;
  mk.whi0 = mk.whi1 = mk.all_hi = INT_MAX;
  mk.bias0 = nullptr;
  mk.bias_step = 0;
  W w;
  w.init(p.c, b, h, ptx::smem_u32(smem) + warp * W::kWarpBytes, p.scale, 0.f, &g_err_select);
  {
    const int ra = lane >> 2, rb = ra + 8;
    const __nv_bfloat16* q = p.q + token * p.q_tok + (long long)h * p.G * kD;
    w.load_q(ra < p.G ? q + ra * kD : nullptr, rb < p.G ? q + rb * kD : nullptr);
  }
  __syncthreads();
  const int tiles = s_tiles;
  const int a = (int)((long long)tiles * part / split), e = (int)((long long)tiles * (part + 1) / split);
  w.walk(
      a + warp, kWarps, e, [&](int t) { return s_key[t]; },
      [&](int, int& cl, int& ch) {
        cl = 0;
        ch = limit - 1;
      },
      [] {}, mk);  // the queries came while the blocks were looked through

  const long long row0 = (long long)token * p.Hq + h * p.G;
  paged_cluster_finish<W, kWarps, kD>(
      w, smem, split, part, p.G, [&](int r) { return row0 + r; },
      [&](int r, float L) {
        return (L == 0.f ? 0.f : 1.f / L) * (p.gate != nullptr ? __bfloat162float(p.gate[row0 + r]) : 1.f);
      },
      p.out, p.lse);
}

template <bool kF8, int kD, bool kHi>
cudaError_t launch(const PagedSelectParams& p, cudaStream_t st) {
  using W = PagedWarp<kF8, kD, kF8 || kD == 64 ? 32 : 16, kHi, false, false>;
  constexpr int ring = kWarps * W::kWarpBytes;
  constexpr int merge = paged_finish_bytes<W, kWarps, kD>();
  constexpr int bytes = ring > merge ? ring : merge;
  auto* kernel = paged_select_kernel<kF8, kD, kHi>;
  static thread_local unsigned long long devices = 0;
  cudaError_t e = paged_allow_smem(kernel, bytes, &devices);
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.c.B * p.c.Qn * p.c.Hkv;
  return paged_launch(kernel, dim3((unsigned)(items * p.split)), kWarps * 32, bytes, st, p, p.split);
}
}  // namespace

unsigned read_and_clear_error_select(cudaStream_t, std::string* where) {
  unsigned w = 0, zero = 0;
  cudaMemcpyFromSymbol(&w, g_err_select, sizeof(w));
  if (w) {
    cudaMemcpyToSymbol(g_err_select, &zero, sizeof(zero));
    *where += " (paged selection: a length or a page number out of range)";
  }
  return w;
}

int launch_paged_select(const PagedView& c, int f8, int D, const void* q, long long q_tok, int Hq,
                        const int32_t* idx, const int32_t* cnt, int cnt_scalar, int S, int block_size,
                        int causal, float scale, const void* gate, void* out, float* lse,
                        cudaStream_t stream) {
  PagedSelectParams p;
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_tok;
  p.idx = idx;
  p.cnt = cnt;
  p.cnt_scalar = cnt_scalar;
  p.S = S;
  p.block_size = block_size;
  p.causal = causal;
  p.gate = static_cast<const __nv_bfloat16*>(gate);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.Hq = Hq;
  p.G = Hq / c.Hkv;
  p.scale = scale;
  // CTAs an item: the choice with the least (waves of resident CTAs, three on an SM) x (a
  // CTA's fixed time, worth about 2 tiles of a warp, + its warps' tiles).
  const long long items = (long long)c.B * c.Qn * c.Hkv;
  const int tiles = S * block_size / (f8 || D == 64 ? 32 : 16);
  int split = 1;
  long long best = LLONG_MAX;
  for (int s = 1; s <= kPagedMaxSplit; s *= 2) {
    const long long waves = (items * s + 455) / 456;
    const long long cost = waves * (2 + (tiles + s * kWarps - 1) / (s * kWarps));
    if (cost < best) {
      best = cost;
      split = s;
    }
  }
  p.split = split;
  const bool hi = p.G > 8;
  cudaError_t e;
  if (D == 128)
    e = f8 ? (hi ? launch<true, 128, true>(p, stream) : launch<true, 128, false>(p, stream))
           : (hi ? launch<false, 128, true>(p, stream) : launch<false, 128, false>(p, stream));
  else
    e = f8 ? (hi ? launch<true, 64, true>(p, stream) : launch<true, 64, false>(p, stream))
           : (hi ? launch<false, 64, true>(p, stream) : launch<false, 64, false>(p, stream));
  if (e != cudaSuccess) return cuda_error(e, "paged selection launch");
  return SBA_OK;
}

}  // namespace sba
