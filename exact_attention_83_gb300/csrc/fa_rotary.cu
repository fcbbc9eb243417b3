// Rotation of query and key heads by their positions, with one or several
// axes, and the RMS norm of every head in the same pass; forward and gradient.
//
// Per row x of D elements (one head of one token), with n = 2 * sum(sections)
// rotated elements forming pairs (a_i, b_i):
//   angle_i = pos[axis(i)] * inv_freq[i]
//   norm (optional):  y = x * rstd * w,  rstd = (sum x^2 / D + eps)^(-1/2)
//   forward:          (a, b) -> (a cos - b sin, a sin + b cos) of y's pairs
//   gradient:         g = the incoming gradient rotated by -angle;
//                     dw = sum over rows of g o xhat,  xhat = x rstd,
//                     dx = rstd (g o w - xhat mean(g o w o xhat))
// Without the norm the gradient is the rotation by -angle alone, so the same
// kernel runs with the sine negated.
//
// Angles: a position far into a long context times a frequency near 1 loses
// its fraction of a turn in fp32 (at 10^6 the angle's ulp is 0.06 rad).  The
// fraction is formed exactly instead: inv_freq / 2 pi as a 64-bit binary
// fraction of a turn (from a 128-bit 1 / 2 pi), times the integer position
// modulo 2^64, whose top 32 bits are the angle in turns.  The error is below
// |pos| 2^-64 turns + 2^-25 half turns, for any position an int64 holds up to
// 2^36 in magnitude without loss.
//
// What bounds it: HBM.  Each row is read once and written once (the gradient
// of the norm reads two rows and writes one); the arithmetic is a few
// operations per element.  So each lane owns 16 elements of a row as two
// 16-byte units whose pairs it holds whole (units 8c and pairs + 8c for split
// halves, 32 contiguous bytes for neighbouring pairs): no exchange between
// lanes but the norm's sums.  A block takes a tile of tokens with all their
// heads, so that the cosines and sines of a token are computed once, into
// shared memory, for all its heads.

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTile = 8;     // tokens per tile, at most

struct RotArgs {
  const void* x[2];             // q, k (gradient: the incoming gradients)
  const void* in[2];            // gradient of the norm: the forward's q, k
  void* out[2];
  int64_t sx[2][3], sin[2][3], so[2][3];   // element strides (b, h, n)
  int64_t N;
  int heads[2];
  int h_fast[2];                // consecutive rows of a tile: heads of a token, or tokens of a head
  int tile, tiles;              // tokens per tile, tiles per batch entry
  int64_t items;                // B * tiles
  int pairs, interleaved, naxes;
  int sec_end[4];               // first pair past each axis
  const float* inv_freq;
  const void* pos;
  int pos64;
  int64_t ps[3];                // position strides (axis, b, n)
  const void* w[2];
  int w_f32;
  float eps, sign;              // sign: +1 forward, -1 gradient
  float* dw_part;               // [grid][2][D] partial weight gradients
};

// ------------------------------------------------------------------ row access
template <typename T> struct Unit;      // 8 consecutive elements
template <> struct Unit<float> {
  static __device__ __forceinline__ void load(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
};
template <typename T> struct Unit {
  static __device__ __forceinline__ void load(const T* p, float (&v)[8]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::to_f32(e[i]);
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[8]) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = Elem<T>::from_f32(v[i]);
    __stcs(reinterpret_cast<uint4*>(p), u);
  }
};

// ---------------------------------------------------------------------- angles
// frac(f / 2 pi) * 2^64 for a finite fp32 f: the 24-bit significand times the
// first 128 bits of 1 / 2 pi, shifted to where the binary point falls.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = static_cast<int>((bits >> 23) & 0xffu);
  const uint32_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  // 1 / 2 pi = 0.28BE60DB 9391054A 7F09D5F4 7D4D3770 (hexadecimal)
  const uint64_t p0 = static_cast<uint64_t>(m) * 0x7D4D3770u;
  const uint64_t p1 = static_cast<uint64_t>(m) * 0x7F09D5F4u + (p0 >> 32);
  const uint64_t p2 = static_cast<uint64_t>(m) * 0x9391054Au + (p1 >> 32);
  const uint64_t p3 = static_cast<uint64_t>(m) * 0x28BE60DBu + (p2 >> 32);
  const uint64_t lo = (p1 << 32) | (p0 & 0xffffffffu);          // bits 0 .. 63
  const uint64_t mid = (p3 << 32) | (p2 & 0xffffffffu);         // bits 64 .. 127
  const uint64_t hi = p3 >> 32;                                 // bits 128 .. 151
  // value = X * 2^(e - 128) turns with e = max(ex, 1) - 150; the wanted bits
  // are X >> (64 - e), of which the low 64 are kept
  const int sh = 64 - ((ex ? ex : 1) - 150);
  uint64_t r;
  if (sh >= 192) r = 0;
  else if (sh >= 128) r = hi >> (sh - 128);
  else if (sh > 64) r = (mid >> (sh - 64)) | (hi << (128 - sh));
  else if (sh == 64) r = mid;
  else if (sh > 0) r = (lo >> sh) | (mid << (64 - sh));
  else r = sh > -64 ? lo << -sh : 0;
  return (bits >> 31) ? 0 - r : r;
}

// Cosines and sines of a tile's tokens: cs[token][pair].
__device__ __forceinline__ void angle_table(const RotArgs& a, float2* cs, int64_t b, int64_t n0,
                                            int ntok) {
  const int total = ntok * a.pairs;
  for (int idx = threadIdx.x; idx < total; idx += kThreads) {
    const int tok = idx / a.pairs, i = idx - tok * a.pairs;
    int ax = 0;
#pragma unroll
    for (int s = 0; s < 3; ++s)
      if (s + 1 < a.naxes && i >= a.sec_end[s]) ax = s + 1;
    const int64_t at = ax * a.ps[0] + b * a.ps[1] + (n0 + tok) * a.ps[2];
    const int64_t p = a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + at)
                              : static_cast<int64_t>(__ldg(static_cast<const int*>(a.pos) + at));
    const uint64_t turn = static_cast<uint64_t>(p) * turns_per_position(__ldg(a.inv_freq + i));
    // top 32 bits as a signed fraction: half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half, &s, &c);
    cs[idx] = make_float2(c, a.sign * s);
  }
}

// Where a lane's two units of a row lie, and its first pair (or -1: elements
// past the rotated ones).
struct LaneUnits {
  int off_a, off_b, pair;
};
__device__ __forceinline__ LaneUnits lane_units(int c, int pairs, int interleaved) {
  LaneUnits u;
  const int rc = pairs / 8;                      // lanes that hold rotated pairs
  u.pair = c < rc ? 8 * c : -1;
  if (c >= rc || interleaved) {
    u.off_a = 16 * c;
    u.off_b = 16 * c + 8;
  } else {
    u.off_a = 8 * c;
    u.off_b = pairs + 8 * c;
  }
  return u;
}

// Rotates a lane's 16 elements in place by the tabled angles.
__device__ __forceinline__ void rotate(float (&va)[8], float (&vb)[8], const float2* cs,
                                       bool interleaved) {
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 t = *reinterpret_cast<const float4*>(cs + i);
    c[i] = t.x; s[i] = t.y; c[i + 1] = t.z; s[i + 1] = t.w;
  }
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = va[2 * i], y0 = va[2 * i + 1], x1 = vb[2 * i], y1 = vb[2 * i + 1];
      va[2 * i] = x0 * c[i] - y0 * s[i];
      va[2 * i + 1] = x0 * s[i] + y0 * c[i];
      vb[2 * i] = x1 * c[4 + i] - y1 * s[4 + i];
      vb[2 * i + 1] = x1 * s[4 + i] + y1 * c[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = va[i], y = vb[i];
      va[i] = x * c[i] - y * s[i];
      vb[i] = x * s[i] + y * c[i];
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row r of a tile's rows of tensor t (q or k): its token and head.
__device__ __forceinline__ void tile_row(const RotArgs& a, int t, int r, int ntok, int& tok, int& h) {
  if (a.h_fast[t]) {
    tok = r / a.heads[t];
    h = r - tok * a.heads[t];
  } else {
    h = r / ntok;
    tok = r - h * ntok;
  }
}

template <int D>
__device__ __forceinline__ void load_weights(const RotArgs& a, float* sw, bool half_type, bool bf16) {
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const void* w = a.w[i / D];
    const int d = i % D;
    float v;
    if (a.w_f32 || !half_type) v = static_cast<const float*>(w)[d];
    else if (bf16) v = __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d]);
    else v = __half2float(static_cast<const __half*>(w)[d]);
    sw[i] = v;
  }
}

template <typename T>
constexpr bool kHalf = sizeof(T) == 2;
template <typename T>
constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;

template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotArgs a) {
  constexpr int LPR = D / 16;            // lanes per row
  constexpr int RPW = 32 / LPR;          // rows per warp
  __shared__ __align__(16) float2 cs[kMaxTile * (D / 2)];
  __shared__ __align__(16) float sw[NORM ? 2 * D : 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LaneUnits u = lane_units(lane % LPR, a.pairs, a.interleaved);
  if constexpr (NORM) load_weights<D>(a, sw, kHalf<T>, kBf16<T>);
  const int64_t b = blockIdx.x / a.tiles, n0 = static_cast<int64_t>(blockIdx.x % a.tiles) * a.tile;
  const int ntok = static_cast<int>(a.N - n0 < a.tile ? a.N - n0 : a.tile);
  angle_table(a, cs, b, n0, ntok);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const T* x = static_cast<const T*>(a.x[t]) + b * a.sx[t][0] + n0 * a.sx[t][2];
    T* out = static_cast<T*>(a.out[t]) + b * a.so[t][0] + n0 * a.so[t][2];
    const int rows = ntok * a.heads[t];
    // whole warps stay in the loop: the norm's sums are exchanged
    for (int r0 = warp * RPW; r0 < rows; r0 += kWarps * RPW) {
      const int r = r0 + lane / LPR;
      const bool on = r < rows;
      int tok, h;
      tile_row(a, t, on ? r : 0, ntok, tok, h);
      float va[8], vb[8];
      const T* row = x + h * a.sx[t][1] + tok * a.sx[t][2];
      Unit<T>::load(row + u.off_a, va);
      Unit<T>::load(row + u.off_b, vb);
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(va[i], va[i], fmaf(vb[i], vb[i], ss));
        const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
        const float* w = sw + t * D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          va[i] *= rstd * w[u.off_a + i];
          vb[i] *= rstd * w[u.off_b + i];
        }
      }
      if (u.pair >= 0) rotate(va, vb, cs + tok * a.pairs + u.pair, a.interleaved);
      if (on) {
        T* dst = out + h * a.so[t][1] + tok * a.so[t][2];
        Unit<T>::store(dst + u.off_a, va);
        Unit<T>::store(dst + u.off_b, vb);
      }
    }
  }
}

// Gradient of the norm with the rotation.  A block walks tiles and keeps its
// lanes' sums of the weight gradients in registers (16 columns of each
// tensor's weight per lane), joins them once at the end and leaves one partial
// row per tensor; weight_grad_kernel adds the blocks' rows in a fixed order,
// so the result does not depend on the schedule.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const __grid_constant__ RotArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  __shared__ __align__(16) float2 cs[kMaxTile * (D / 2)];
  __shared__ __align__(16) float sw[2 * D];
  __shared__ float red[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LaneUnits u = lane_units(lane % LPR, a.pairs, a.interleaved);
  load_weights<D>(a, sw, kHalf<T>, kBf16<T>);
  float acc[2][16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;

  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int64_t b = item / a.tiles, n0 = (item - b * a.tiles) * a.tile;
    const int ntok = static_cast<int>(a.N - n0 < a.tile ? a.N - n0 : a.tile);
    __syncthreads();                      // the last tile's table is no longer read
    angle_table(a, cs, b, n0, ntok);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const T* g = static_cast<const T*>(a.x[t]) + b * a.sx[t][0] + n0 * a.sx[t][2];
      const T* x = static_cast<const T*>(a.in[t]) + b * a.sin[t][0] + n0 * a.sin[t][2];
      T* out = static_cast<T*>(a.out[t]) + b * a.so[t][0] + n0 * a.so[t][2];
      const int rows = ntok * a.heads[t];
      for (int r0 = warp * RPW; r0 < rows; r0 += kWarps * RPW) {
        const int r = r0 + lane / LPR;
        const bool on = r < rows;
        int tok, h;
        tile_row(a, t, on ? r : 0, ntok, tok, h);
        float ga[8], gb[8], xa[8], xb[8];
        const T* grow = g + h * a.sx[t][1] + tok * a.sx[t][2];
        const T* xrow = x + h * a.sin[t][1] + tok * a.sin[t][2];
        Unit<T>::load(grow + u.off_a, ga);
        Unit<T>::load(grow + u.off_b, gb);
        Unit<T>::load(xrow + u.off_a, xa);
        Unit<T>::load(xrow + u.off_b, xb);
        if (u.pair >= 0) rotate(ga, gb, cs + tok * a.pairs + u.pair, a.interleaved);
        const float* w = sw + t * D;
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
          sg = fmaf(ga[i] * w[u.off_a + i], xa[i], fmaf(gb[i] * w[u.off_b + i], xb[i], sg));
        }
        const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
        // xhat mean(g w xhat) = x rstd^2 (sum g w x) / D
        const float m = row_sum<LPR>(sg) * (1.f / D) * rstd * rstd;
        const float rs = on ? rstd : 0.f;      // lanes without a row add nothing
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[t][i] = fmaf(ga[i] * xa[i], rs, acc[t][i]);
          acc[t][8 + i] = fmaf(gb[i] * xb[i], rs, acc[t][8 + i]);
          ga[i] = rstd * (ga[i] * w[u.off_a + i] - xa[i] * m);
          gb[i] = rstd * (gb[i] * w[u.off_b + i] - xb[i] * m);
        }
        if (on) {
          T* dst = out + h * a.so[t][1] + tok * a.so[t][2];
          Unit<T>::store(dst + u.off_a, ga);
          Unit<T>::store(dst + u.off_b, gb);
        }
      }
    }
  }
  // lanes of a warp that hold the same columns, then the warps
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = acc[t][i];
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < LPR) red[warp][(i < 8 ? u.off_a : u.off_b) + (i & 7)] = v;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w][d];
      a.dw_part[(static_cast<int64_t>(blockIdx.x) * 2 + t) * D + d] = v;
    }
  }
}

// dq_weight | dk_weight: the blocks' partial rows added up, 32 columns per
// block, eight warps taking every eighth row.
__global__ void __launch_bounds__(kThreads) weight_grad_kernel(const float* part, int nparts, int D,
                                                               float* dqw, float* dkw) {
  __shared__ float red[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;          // of 2 * D (a multiple of 32)
  float v = 0.f;
  for (int p = warp; p < nparts; p += kWarps) v += __ldg(part + static_cast<int64_t>(p) * 2 * D + col);
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][lane];
    if (col < D) dqw[col] = v;
    else dkw[col - D] = v;
  }
}

// Tokens per tile: as many as keep the grid at four blocks per SM or more, so
// that short inputs spread over the SMs.
int pick_tile(int64_t B, int64_t N) {
  int tile = kMaxTile;
  while (tile > 1 && B * ((N + tile - 1) / tile) < 4 * static_cast<int64_t>(device_sm_count())) tile /= 2;
  return tile;
}

RotArgs make_args(const RotaryParams& p) {
  RotArgs a{};
  for (int t = 0; t < 2; ++t) {
    a.x[t] = p.x[t]; a.in[t] = p.in[t]; a.out[t] = p.out[t];
    for (int i = 0; i < 3; ++i) {
      a.sx[t][i] = p.sx[t][i]; a.sin[t][i] = p.sin[t][i]; a.so[t][i] = p.so[t][i];
    }
    a.heads[t] = static_cast<int>(t ? p.Hkv : p.Hq);
    a.h_fast[t] = p.sx[t][1] <= p.sx[t][2];
    a.w[t] = p.w[t];
  }
  a.N = p.N;
  a.tile = pick_tile(p.B, p.N);
  a.tiles = static_cast<int>((p.N + a.tile - 1) / a.tile);
  a.items = p.B * a.tiles;
  a.pairs = p.pairs; a.interleaved = p.interleaved; a.naxes = p.naxes;
  for (int i = 0; i < 4; ++i) a.sec_end[i] = p.sec_end[i];
  a.inv_freq = p.inv_freq; a.pos = p.pos; a.pos64 = p.pos64;
  for (int i = 0; i < 3; ++i) a.ps[i] = p.ps[i];
  a.w_f32 = p.w_f32; a.eps = p.eps;
  return a;
}

template <typename T, int D>
fa_status run_rotary(const RotaryParams& p, cudaStream_t s) {
  RotArgs a = make_args(p);
  if (a.items > 0x7fffffffLL) return FA_ERR_SHAPE;
  const bool norm = p.w[0] != nullptr;
  if (p.backward && norm) {
    a.sign = -1.f;
    a.dw_part = p.ws;
    const int64_t grid = a.items < kRotaryMaxParts ? a.items : kRotaryMaxParts;
    qk_norm_bwd_kernel<T, D><<<dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
    weight_grad_kernel<<<dim3(2 * D / 32), dim3(kThreads), 0, s>>>(
        p.ws, static_cast<int>(grid), D, p.dw[0], p.dw[1]);
  } else {
    a.sign = p.backward ? -1.f : 1.f;
    const dim3 grid(static_cast<unsigned>(a.items));
    if (norm) rotary_kernel<T, D, true><<<grid, dim3(kThreads), 0, s>>>(a);
    else rotary_kernel<T, D, false><<<grid, dim3(kThreads), 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

template <typename T>
fa_status run_rotary_d(const RotaryParams& p, cudaStream_t s) {
  switch (p.D) {
    case 16: return run_rotary<T, 16>(p, s);
    case 32: return run_rotary<T, 32>(p, s);
    case 64: return run_rotary<T, 64>(p, s);
    case 128: return run_rotary<T, 128>(p, s);
  }
  return FA_ERR_ARG;
}

}  // namespace

fa_status launch_rotary(const RotaryParams& p, cudaStream_t s) {
  switch (p.dtype) {
    case FA_F32: return run_rotary_d<float>(p, s);
    case FA_F16: return run_rotary_d<__half>(p, s);
    case FA_BF16: return run_rotary_d<__nv_bfloat16>(p, s);
  }
  return FA_ERR_ARG;
}

}  // namespace fa
