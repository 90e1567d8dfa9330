// Rotation of queries and keys by their positions, and the tables of its cosines and sines, for
// sm_103a.
//
// Pair i of a head's first rot_dim dimensions turns by position * f_i:
//   (x0, x1) -> (x0 c - x1 s, x1 c + x0 s),
// with s negated for the transpose (the gradient of the rotation).  The rotation only moves bytes, every
// element of q and k read and written once; the tables are written once and computed on the way.
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "common.cuh"
#include "rotary_turns.h"

namespace sba {

static __device__ unsigned g_err_rotary = 0u;

namespace {

// ------------------------------------------------------------------ tables
// The angle of a far position loses its fraction of a turn in 32 bits.  Here a pair's frequency
// is a 64-bit fixed-point number of turns a position (2^-64 steps), so position * frequency
// modulo 2^64 is the fraction of a turn itself, off by at most position * 2^-64 turns.  Its quarter turns
// are the two bits above the rest, which becomes a float, relative precision kept: r in [-1, 1) eighths of a turn.  There sin(pi/4 r) = r S(r^2) and
// cos(pi/4 r) = 1 + r^2 C(r^2) with cubic S and C, fitted here by exchange for the least maximal error on
// [0, 1]: 2.4e-9 and 1.9e-10, below a tenth of fp32's rounding.  Amplitude is in the coefficients.
// What bounds the kernel is instruction issue beside the writes: 131072 positions of 64 pairs take 14.8 us
// (67 MB are 10 at the rate of a fill); 18.4 with sincospif in place of the polynomials, or with one
// 64-bit conversion in place of two of 32 bits; 17.6 with those put together from the bits.
constexpr int kMaxPairs = 128;
constexpr double kSin[4] = {0.7853981609834035, -0.08074543483021554, 0.0024900071271047107, -3.595450778997901e-05};
constexpr double kCos[4] = {-0.3084251373439996, 0.015854338155325057, -0.0003259614016941051, 3.5419669590582045e-06};
struct TableParams {
  unsigned long long turn[kMaxPairs];
  float* cosp;
  float* sinp;
  int length, pairs;
  float amplitude, s[4], c[4];
};

// A thread keeps four pairs and walks over positions.
__global__ void __launch_bounds__(256) rotary_tables_kernel(const __grid_constant__ TableParams p) {
  const int cols = p.pairs / 4, rows = blockDim.x / cols;
  const int c = threadIdx.x % cols, r = threadIdx.x / cols;
  if (r >= rows) return;
  unsigned long long f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = p.turn[c * 4 + i];
  for (unsigned pos = blockIdx.x * rows + r; pos < static_cast<unsigned>(p.length); pos += gridDim.x * rows) {
    float co[4], si[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned long long t = f[i] * pos;
      const unsigned q = static_cast<unsigned>((t + (1ull << 61)) >> 62);  // the nearest quarter turn
      const long long rest = static_cast<long long>(t - (static_cast<unsigned long long>(q) << 62));
      const float r = fmaf(static_cast<float>(static_cast<int>(rest >> 30)), 0x1p-31f,
                           static_cast<float>(static_cast<unsigned>(rest) & 0x3fffffffu) * 0x1p-61f);
      const float u = r * r;
      const float a = r * fmaf(u, fmaf(u, fmaf(u, p.s[3], p.s[2]), p.s[1]), p.s[0]);
      const float b = fmaf(u, fmaf(u, fmaf(u, fmaf(u, p.c[3], p.c[2]), p.c[1]), p.c[0]), p.amplitude);
      const float y = (q & 1u) ? b : a, x = (q & 1u) ? a : b;
      si[i] = (q & 2u) ? -y : y;
      co[i] = ((q + 1u) & 2u) ? -x : x;
    }
    const long long o = (long long)pos * p.pairs + c * 4;
    *reinterpret_cast<float4*>(p.cosp + o) = make_float4(co[0], co[1], co[2], co[3]);
    *reinterpret_cast<float4*>(p.sinp + o) = make_float4(si[0], si[1], si[2], si[3]);
  }
}

// ------------------------------------------------------------------ rotation
struct EmbedParams {
  const uint8_t* q;
  const uint8_t* k;
  uint8_t* qo;
  uint8_t* ko;
  const int* positions;  // null: token % T
  const float* cosp;
  const float* sinp;
  long long q_tok, k_tok, qo_tok, ko_tok;  // bytes from token to token
  int N, T, Hq, heads, D, rot, max_pos, subs;
  float sign;            // -1: turned back
};

// Eight elements of a head in 32 bits.
template <typename E>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 raw;
  __device__ void load(const uint8_t* at) { raw = *reinterpret_cast<const uint4*>(at); }
  __device__ void store(uint8_t* at) const { *reinterpret_cast<uint4*>(at) = raw; }
  __device__ void get(float (&x)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ void set(const float (&x)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ void load(const uint8_t* at) {
    a = *reinterpret_cast<const float4*>(at);
    b = *reinterpret_cast<const float4*>(at + 16);
  }
  __device__ void store(uint8_t* at) const {
    *reinterpret_cast<float4*>(at) = a;
    *reinterpret_cast<float4*>(at + 16) = b;
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Bytes bound it from some MB on: 4 x 16384 tokens of 32 + 8 heads of 128 in bf16 196 us, 2 x 16384 in fp32 196.
// A thread takes two chunks of eight dimensions of kHeads heads of one token, so that the angles
// are read once for the heads and all loads of a thread are in flight at once.  The two chunks
// hold the two sides of eight pairs (half layout), or four pairs each (neighbouring pairs); chunks
// behind rot_dim, and tokens at negative positions, pass through as they are.
template <typename E, bool kPairs, int kHeads>
__global__ void __launch_bounds__(256) rotary_embed_kernel(const EmbedParams p) {
  const int units = p.D / 16;
  const int u = threadIdx.x % units;
  const int slot = blockIdx.x * (blockDim.x / units) + threadIdx.x / units;
  const int tok = slot / p.subs, h0 = (slot - tok * p.subs) * kHeads;
  if (tok >= p.N) return;
  int pos = p.positions ? p.positions[tok] : tok % p.T;
  if (pos >= p.max_pos) {
    atomicOr(&g_err_rotary, kDevErrInput);
    pos = -1;
  }
  int a, b;
  bool turn_a, turn_b;
  if (kPairs) {
    a = 8 * u;
    b = p.D / 2 + 8 * u;
    turn_a = pos >= 0 && a < p.rot;
    turn_b = pos >= 0 && b < p.rot;
  } else {
    const int turned = p.rot / 16;
    turn_a = turn_b = pos >= 0 && u < turned;
    a = u < turned ? 8 * u : 16 * u;
    b = u < turned ? p.rot / 2 + 8 * u : 16 * u + 8;
  }
  Chunk<E> x[kHeads], y[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h < p.heads) {
      const uint8_t* at = h < p.Hq ? p.q + tok * p.q_tok + (long long)h * p.D * sizeof(E)
                                   : p.k + tok * p.k_tok + (long long)(h - p.Hq) * p.D * sizeof(E);
      x[i].load(at + a * sizeof(E));
      y[i].load(at + b * sizeof(E));
    }
  }
  float c[8], s[8];
  if (turn_a) {  // the second chunk lies behind the first: it turns only if that does
    const long long row = (long long)pos * (p.rot / 2);
    // pairs of the first four and of the other four values
    const int i0 = kPairs ? a / 2 : a, i1 = kPairs ? (turn_b ? b / 2 : i0) : a + 4;
    *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(p.cosp + row + i0);
    *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(p.cosp + row + i1);
    *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(p.sinp + row + i0);
    *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(p.sinp + row + i1);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= p.sign;
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h >= p.heads) break;
    if (turn_a) {
      float v[8], w[8];
      x[i].get(v);
      y[i].get(w);
      if (kPairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v0 = v[2 * j], v1 = v[2 * j + 1], w0 = w[2 * j], w1 = w[2 * j + 1];
          v[2 * j] = v0 * c[j] - v1 * s[j];
          v[2 * j + 1] = v1 * c[j] + v0 * s[j];
          w[2 * j] = w0 * c[4 + j] - w1 * s[4 + j];
          w[2 * j + 1] = w1 * c[4 + j] + w0 * s[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v0 = v[j], w0 = w[j];
          v[j] = v0 * c[j] - w0 * s[j];
          w[j] = w0 * c[j] + v0 * s[j];
        }
      }
      x[i].set(v);
      if (turn_b) y[i].set(w);
    }
    uint8_t* to = h < p.Hq ? p.qo + tok * p.qo_tok + (long long)h * p.D * sizeof(E)
                           : p.ko + tok * p.ko_tok + (long long)(h - p.Hq) * p.D * sizeof(E);
    x[i].store(to + a * sizeof(E));
    y[i].store(to + b * sizeof(E));
  }
}

template <typename E, bool kPairs>
int launch_embed(EmbedParams p, cudaStream_t stream) {
  constexpr int kHeads = 4;
  const int units = p.D / 16, per_block = 256 / units;
  p.subs = (p.heads + kHeads - 1) / kHeads;
  const long long slots = (long long)p.N * p.subs;
  if (slots >= (1LL << 31) - 256) return set_error(SBA_ERR_UNSUPPORTED, "rotary_embed: too many heads in all");
  const int grid = static_cast<int>((slots + per_block - 1) / per_block);
  rotary_embed_kernel<E, kPairs, kHeads><<<grid, per_block * units, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SBA_OK : cuda_error(e, "rotary_embed launch");
}

}  // namespace

unsigned read_and_clear_error_rotary(cudaStream_t, std::string* where) {
  unsigned w = 0u, zero = 0u;
  cudaMemcpyFromSymbol(&w, g_err_rotary, sizeof(w));
  if (w) {
    cudaMemcpyToSymbol(g_err_rotary, &zero, sizeof(zero));
    if (where) *where += " [rotary_embed: a position outside the tables]";
  }
  return w;
}

int launch_rotary_tables(int length, int rot, double base, double factor, int original_length, double slow, double fast,
                         double amplitude, float* cosp, float* sinp, cudaStream_t stream) {
  TableParams p{};
  rotary_turns(rot, base, factor, original_length, slow, fast, p.turn);
  p.cosp = cosp;
  p.sinp = sinp;
  p.length = length;
  p.pairs = rot / 2;
  p.amplitude = static_cast<float>(amplitude);
  for (int i = 0; i < 4; ++i) {
    p.s[i] = static_cast<float>(amplitude * kSin[i]);
    p.c[i] = static_cast<float>(amplitude * kCos[i]);
  }
  const int rows = 256 / (p.pairs / 4);
  const int grid = static_cast<int>(std::min((length + rows - 1LL) / rows, 8LL * num_sms()));
  rotary_tables_kernel<<<grid, 256, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SBA_OK : cuda_error(e, "rotary_tables launch");
}

int launch_rotary_embed(const sba_rotary_embed_args& a, cudaStream_t stream) {
  const long long size = a.dtype == SBA_F32 ? 4 : 2;
  EmbedParams p{};
  p.q = static_cast<const uint8_t*>(a.q);
  p.k = static_cast<const uint8_t*>(a.k);
  p.qo = static_cast<uint8_t*>(a.q_out);
  p.ko = static_cast<uint8_t*>(a.k_out);
  p.positions = a.positions;
  p.cosp = a.cos;
  p.sinp = a.sin;
  p.q_tok = a.q_stride * size;
  p.k_tok = a.k_stride * size;
  p.qo_tok = a.q_out_stride * size;
  p.ko_tok = a.k_out_stride * size;
  p.N = a.B * a.T;
  p.T = a.T;
  p.Hq = a.Hq;
  p.heads = a.Hq + (a.k ? a.Hkv : 0);
  p.D = a.D;
  p.rot = a.rot_dim;
  p.max_pos = a.max_pos;
  p.sign = a.inverse ? -1.f : 1.f;
  if (a.dtype == SBA_F32) return a.interleaved ? launch_embed<float, true>(p, stream) : launch_embed<float, false>(p, stream);
  return a.interleaved ? launch_embed<__nv_bfloat16, true>(p, stream) : launch_embed<__nv_bfloat16, false>(p, stream);
}

}  // namespace sba
