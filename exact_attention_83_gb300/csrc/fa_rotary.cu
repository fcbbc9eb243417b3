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
// 8-element units whose pairs it holds whole (elements 8c and pairs + 8c for
// split halves, 8c and D/2 + 8c for neighbouring pairs): no exchange between
// lanes but the norm's sums, and neighbouring lanes touch neighbouring units.
// A block takes a tile of tokens with all their heads, so that the cosines and
// sines of a token are computed once, into shared memory, for all its heads; a
// lane then keeps those of its pairs, and its weights, in registers while it
// walks the heads.  Arithmetic is on pairs of fp32, which halves its
// instructions, and rows are copied into shared memory steps ahead of the work
// (cp.async).  Cold L2, in us and TB/s (a copy reaches 6.8): 16384 tokens of
// 32 + 8 bf16 heads of 128 with norm: forward 53 (6.3), gradient 82 (6.1) and 2.5
// for joining the weight gradients; 4 x 4096 tokens of 16 + 16 fp16 heads of 64,
// two axes, rotation alone: 23 (5.7) either way.

#include "tc_common.cuh"

namespace fa {
namespace {

using tc::pack2;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Tokens per tile at most: the angles of a tile take 8 KB.
template <int D> constexpr int kMaxTile = 2048 / D;
constexpr int kMostTokens = 128;

// The tiles of a walk: tokens per tile, tiles per batch entry, tiles in all.
struct Tiles {
  int tok;
  int64_t per, items;
};

struct RotArgs {
  const void* x[2];             // q, k (gradient: the incoming gradients)
  const void* in[2];            // gradient of the norm: the forward's q, k
  void* out[2];
  int64_t sx[2][3], sin[2][3], so[2][3];   // element strides (b, h, n)
  int64_t N;
  int heads[2];
  Tiles tiles[2];               // forward: [0]; gradient of the norm: of q and of k
  int pairs, naxes;
  int sec_end[4];               // first pair past each axis
  const float* inv_freq;
  const void* pos;
  int pos64;
  int64_t ps[3];                // position strides (axis, b, n)
  const void* w[2];
  int w_f32;
  float eps, sign;              // sign: +1 forward, -1 gradient
  int split;                    // gradient of the norm: blocks that work on q
  float* dw_part;               // [grid][D] partial weight gradients
};

// ------------------------------------------------------------------ row access
// A lane's unit of a row is eight consecutive elements, taken as four pairs of
// fp32.  Units travel through a ring in shared memory (cp.async), a few rows
// ahead of the work and without registers; a thread copies and reads its own
// 16-byte pieces only, so the ring needs no barrier.
template <typename T> constexpr int kPieces = sizeof(T) == 2 ? 1 : 2;   // 16-byte pieces of a unit

template <typename T>
__device__ __forceinline__ void copy_unit(uint4* slot, const T* p) {
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(slot + i * kThreads)),
                 "l"(reinterpret_cast<const uint4*>(p) + i)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else
      x[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
}
__device__ __forceinline__ void unpack32(const uint4& u, const uint4& v, float2 (&x)[4]) {
  x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  x[2] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  x[3] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <typename T>
__device__ __forceinline__ void read_unit(const uint4* slot, float2 (&x)[4]) {
  if constexpr (sizeof(T) == 2) unpack16<T>(slot[0], x);
  else unpack32(slot[0], slot[kThreads], x);
}
template <typename T>
__device__ __forceinline__ void store_unit(T* p, const float2 (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[2].x, x[2].y, x[3].x, x[3].y));
  } else {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack2<T>(x[0].x, x[0].y), pack2<T>(x[1].x, x[1].y),
                                                   pack2<T>(x[2].x, x[2].y), pack2<T>(x[3].x, x[3].y)));
  }
}

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

// Per block: each pair's turns per position and its axis, and a tile's positions.
struct PairTable {
  uint64_t turns[64];
  int64_t pos[2][4][kMostTokens];   // of the tile at work and the next
  uint8_t axis[64];
};
__device__ __forceinline__ void pair_table(const RotArgs& a, PairTable& t) {
  for (int i = threadIdx.x; i < a.pairs; i += kThreads) {
    t.turns[i] = turns_per_position(__ldg(a.inv_freq + i));
    int ax = 0;
#pragma unroll
    for (int s = 0; s < 3; ++s)
      if (s + 1 < a.naxes && i >= a.sec_end[s]) ax = s + 1;
    t.axis[i] = static_cast<uint8_t>(ax);
  }
}
// The positions of tile `item` (nothing past the last one), into buffer `buf`.
__device__ __forceinline__ void tile_positions(const RotArgs& a, const Tiles& tl, PairTable& t,
                                               int64_t item, int buf) {
  if (item >= tl.items) return;
  const int64_t b = item / tl.per, n0 = (item - b * tl.per) * tl.tok;
  // from the last thread down: pair_table keeps the first ones busy
  for (int i = kThreads - 1 - static_cast<int>(threadIdx.x); i < a.naxes * tl.tok; i += kThreads) {
    const int ax = i / tl.tok, tok = i - ax * tl.tok;
    if (n0 + tok >= a.N) continue;
    const int64_t at = ax * a.ps[0] + b * a.ps[1] + (n0 + tok) * a.ps[2];
    t.pos[buf][ax][tok] = a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + at)
                                  : static_cast<int64_t>(__ldg(static_cast<const int*>(a.pos) + at));
  }
}

// Where the cosine of pair i of a token lies in its table of D floats (the sine
// 4 LPR floats on), so that the lanes of a row read 16-byte pieces that are
// neighbours: cosines of a lane's first four pairs, their sines, cosines of its
// last four, their sines, piece j of lane c at float 4 (j LPR + c).  Lane c's
// pairs are 8c .. 8c+7, or, with neighbouring pairs (IL), the four of unit c
// and the four of unit LPR + c.
template <int LPR, bool IL>
__device__ __forceinline__ int cos_at(int i) {
  const int unit = i >> 2;
  const int c = IL ? unit % LPR : unit >> 1, half = IL ? unit / LPR : unit & 1;
  return 4 * (2 * half * LPR + c) + (i & 3);
}

// Cosines and sines of a tile's tokens (cos_at), from the positions in buffer
// `buf`.  Tokens past the end get angles of whatever the buffer holds, which
// nobody uses.
template <int D, bool IL>
__device__ __forceinline__ void angle_table(const RotArgs& a, const PairTable& pt, float* cs, int tile,
                                            int buf) {
  constexpr int LPR = D / 16;
  const int total = tile * a.pairs;
  for (int idx = threadIdx.x; idx < total; idx += kThreads) {
    const int tok = idx / a.pairs, i = idx - tok * a.pairs;
    const uint64_t turn = static_cast<uint64_t>(pt.pos[buf][pt.axis[i]][tok]) * pt.turns[i];
    // top 32 bits as a signed fraction: half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half, &s, &c);
    float* dst = cs + tok * D + cos_at<LPR, IL>(i);
    dst[0] = c;
    dst[4 * LPR] = a.sign * s;
  }
}

// Where a lane's two units of a row lie, and whether their pairs are rotated.
struct LaneUnits {
  int off_a, off_b;
  bool rot_a, rot_b;
};
template <int LPR, bool IL>
__device__ __forceinline__ LaneUnits lane_units(int c, int pairs) {
  LaneUnits u;
  if constexpr (IL) {
    u.off_a = 8 * c;
    u.off_b = 8 * (LPR + c);
    u.rot_a = 4 * c < pairs;
    u.rot_b = 4 * (LPR + c) < pairs;
  } else {
    const int rc = pairs / 8;                    // lanes that hold rotated pairs
    u.rot_a = u.rot_b = c < rc;
    u.off_a = c < rc ? 8 * c : 2 * pairs + 8 * (c - rc);
    u.off_b = c < rc ? pairs + 8 * c : 2 * pairs + 8 * (LPR - rc + c - rc);
  }
  return u;
}

// A lane's eight cosines and sines (identity where nothing is rotated).
struct Angles {
  float2 c[4], s[4];
};
template <int LPR>
__device__ __forceinline__ void load_angles(const float* cs_tok, int c, const LaneUnits& u, Angles& g) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j ? u.rot_b : u.rot_a) {
      x = *reinterpret_cast<const float4*>(cs_tok + 4 * (2 * j * LPR + c));
      y = *reinterpret_cast<const float4*>(cs_tok + 4 * ((2 * j + 1) * LPR + c));
    }
    g.c[2 * j] = make_float2(x.x, x.y);
    g.c[2 * j + 1] = make_float2(x.z, x.w);
    g.s[2 * j] = make_float2(y.x, y.y);
    g.s[2 * j + 1] = make_float2(y.z, y.w);
  }
}

// The rotation of a lane's 16 elements as coefficients: a' = a ca + b sb,
// b' = a sa + b cb for each of the eight pairs.  A norm's weights are folded
// in: ca = w_a cos, sb = -w_b sin, sa = w_a sin, cb = w_b cos.  Split halves
// hold pairs 2i, 2i + 1 in element pair i of each unit; with neighbouring pairs
// (IL) element pair i of the first unit is pair i, of the second pair 4 + i.
struct Turn {
  float2 ca[4], sb[4], sa[4], cb[4];
};
__device__ __forceinline__ float2 neg(float2 x) { return make_float2(-x.x, -x.y); }
template <bool IL>
__device__ __forceinline__ void make_turn(const Angles& g, Turn& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.ca[i] = t.cb[i] = g.c[i];
    t.sa[i] = g.s[i];
    t.sb[i] = neg(g.s[i]);
  }
}
template <bool IL>
__device__ __forceinline__ void make_turn(const Angles& g, const float2 (&wa)[4], const float2 (&wb)[4],
                                          Turn& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 a, b;                         // weights of a's and b's of pairs 2i, 2i + 1
    if constexpr (IL) {
      const float2 e0 = i < 2 ? wa[2 * i] : wb[2 * i - 4], e1 = i < 2 ? wa[2 * i + 1] : wb[2 * i - 3];
      a = make_float2(e0.x, e1.x);
      b = make_float2(e0.y, e1.y);
    } else {
      a = wa[i];
      b = wb[i];
    }
    t.ca[i] = __fmul2_rn(a, g.c[i]);
    t.sa[i] = __fmul2_rn(a, g.s[i]);
    t.cb[i] = __fmul2_rn(b, g.c[i]);
    t.sb[i] = neg(__fmul2_rn(b, g.s[i]));
  }
}
template <bool IL>
__device__ __forceinline__ void turn(float2 (&va)[4], float2 (&vb)[4], const Turn& t) {
  if constexpr (IL) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2& v = i < 4 ? va[i & 3] : vb[i & 3];
      const float ca = i & 1 ? t.ca[i >> 1].y : t.ca[i >> 1].x, sb = i & 1 ? t.sb[i >> 1].y : t.sb[i >> 1].x;
      const float sa = i & 1 ? t.sa[i >> 1].y : t.sa[i >> 1].x, cb = i & 1 ? t.cb[i >> 1].y : t.cb[i >> 1].x;
      v = make_float2(fmaf(v.x, ca, v.y * sb), fmaf(v.x, sa, v.y * cb));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = va[i], y = vb[i];
      va[i] = __ffma2_rn(x, t.ca[i], __fmul2_rn(y, t.sb[i]));
      vb[i] = __ffma2_rn(x, t.sa[i], __fmul2_rn(y, t.cb[i]));
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float2 v2) {
  float v = v2.x + v2.y;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Which rows of a tile a warp takes.  A warp holds RPW rows at a time: `tpw`
// tokens (a power of two, as many as the tile has) with RPW / tpw heads each.
// The tile's token groups are dealt to the warps (a tile has at most kWarps of
// them); the warps left over share the heads of a group.  So a lane works on
// one token of a tile and walks its heads.
struct WarpRows {
  int tok;         // this lane's token within the tile
  int h0, step;    // its first head, and the distance to the next
  int first;       // the warp's first head
};
template <int RPW>
__device__ __forceinline__ WarpRows warp_rows(int tile, int warp, int sub) {
  const int tpw = RPW < tile ? RPW : tile, hpi = RPW / tpw, groups = tile / tpw;
  WarpRows r;
  r.tok = (warp % groups) * tpw + sub / hpi;
  r.first = (warp / groups) * hpi;
  r.h0 = r.first + sub % hpi;
  r.step = (kWarps / groups) * hpi;
  return r;
}
// Heads h0, h0 + step, ... below `heads`.
__device__ __forceinline__ int head_steps(int heads, int h0, int step) {
  return h0 < heads ? (heads - h0 + step - 1) / step : 0;
}

// A tensor's norm weights of a lane's 16 elements.
template <typename T>
__device__ __forceinline__ void load_weights(const RotArgs& a, int t, const LaneUnits& u,
                                             float2 (&wa)[4], float2 (&wb)[4]) {
  if (sizeof(T) == 4 || a.w_f32) {
    const float* w = static_cast<const float*>(a.w[t]);
    const uint4* pa = reinterpret_cast<const uint4*>(w + u.off_a);
    const uint4* pb = reinterpret_cast<const uint4*>(w + u.off_b);
    unpack32(__ldg(pa), __ldg(pa + 1), wa);
    unpack32(__ldg(pb), __ldg(pb + 1), wb);
  } else {
    if constexpr (sizeof(T) == 2) {
      const T* w = static_cast<const T*>(a.w[t]);
      unpack16<T>(__ldg(reinterpret_cast<const uint4*>(w + u.off_a)), wa);
      unpack16<T>(__ldg(reinterpret_cast<const uint4*>(w + u.off_b)), wb);
    }
  }
}

// Blocks per SM that the registers are kept to, and rows of the ring.
template <typename T>
constexpr int fwd_blocks(bool norm) { return !norm && sizeof(T) == 2 ? 3 : 2; }
constexpr int kBwdBlocks = 2;
template <typename T> constexpr int kFwdRing = sizeof(T) == 2 ? 5 : 3;
template <typename T> constexpr int kBwdRing = sizeof(T) == 2 ? 4 : 2;
template <typename T> constexpr int kFwdSmem = kFwdRing<T> * 2 * kPieces<T> * kThreads * 16;
template <typename T> constexpr int kBwdSmem = kBwdRing<T> * 4 * kPieces<T> * kThreads * 16;

// Both kernels walk tiles.  While a tile's rows are worked on, the rows of the
// steps to come (over the ends of tiles) are being copied, the next tile's
// angles are formed into the other half of the table and the positions of the
// tile after it are read: one barrier per tile, and no wait for memory at its
// start.
template <typename T, int D, bool NORM, bool IL>
__global__ void __launch_bounds__(kThreads, fwd_blocks<T>(NORM)) rotary_kernel(const __grid_constant__ RotArgs a) {
  constexpr int LPR = D / 16;            // lanes per row
  constexpr int RPW = 32 / LPR;          // rows per warp
  constexpr int S = kFwdRing<T>, U = kPieces<T> * kThreads;    // pieces of a unit of all threads
  extern __shared__ __align__(16) uint4 ring[];                 // [S][a | b][pieces][thread]
  __shared__ __align__(16) float cs[2][kMaxTile<D> * D];
  __shared__ PairTable pt;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPR;
  const LaneUnits u = lane_units<LPR, IL>(c, a.pairs);
  const int ab = u.off_b - u.off_a;
  const Tiles& tl = a.tiles[0];
  const WarpRows w = warp_rows<RPW>(tl.tok, warp, lane / LPR);
  // steps of the warp on a tile, and those of them in which this lane has a row
  const int it[2] = {head_steps(a.heads[0], w.first, w.step), head_steps(a.heads[1], w.first, w.step)};
  const int mine_q = head_steps(a.heads[0], w.h0, w.step), mine_k = head_steps(a.heads[1], w.h0, w.step);

  // The next step to copy: of q (p_t = 0) or k of tile p_item, p_seg steps left
  // for the warp, p_left for this lane, at p_row.
  int64_t p_item = static_cast<int64_t>(blockIdx.x) - gridDim.x;
  int p_t = 1, p_seg = 0, p_left = 0, p_slot = 0;
  int64_t p_n = 0, p_b = 0, p_step = 0;
  const T* p_row = nullptr;
  auto next_segment = [&]() {
    do {
      p_t ^= 1;
      if (p_t == 0) {
        p_item += gridDim.x;
        if (p_item >= tl.items) return;
        p_b = p_item / tl.per;
        p_n = (p_item - p_b * tl.per) * tl.tok + w.tok;
      }
      p_seg = p_t ? it[1] : it[0];
      p_left = p_n < a.N ? (p_t ? mine_k : mine_q) : 0;
      p_step = w.step * a.sx[p_t][1];
      p_row = static_cast<const T*>(a.x[p_t]) + p_b * a.sx[p_t][0] + p_n * a.sx[p_t][2] +
              w.h0 * a.sx[p_t][1] + u.off_a;
    } while (p_seg == 0);
  };
  uint4* mine = ring + threadIdx.x;
  auto issue = [&]() {
    if (p_seg > 0) {
      if (p_left > 0) {
        uint4* slot = mine + p_slot * 2 * U;
        copy_unit<T>(slot, p_row);
        copy_unit<T>(slot + U, p_row + ab);
      }
      p_slot = p_slot + 1 == S ? 0 : p_slot + 1;
      p_row += p_step;
      --p_left;
      if (--p_seg == 0) next_segment();
    }
    copy_commit();
  };
  if (it[0] + it[1] > 0) next_segment();   // a warp without heads copies nothing
  for (int i = 0; i < S - 1; ++i) issue();
  tile_positions(a, tl, pt, blockIdx.x, 0);
  tile_positions(a, tl, pt, static_cast<int64_t>(blockIdx.x) + gridDim.x, 1);
  pair_table(a, pt);
  __syncthreads();
  angle_table<D, IL>(a, pt, cs[0], tl.tok, 0);
  __syncthreads();
  int slot_i = 0, buf = 0;
  for (int64_t item = blockIdx.x; item < tl.items; item += gridDim.x, buf ^= 1) {
    const int64_t b = item / tl.per, n = (item - b * tl.per) * tl.tok + w.tok;
    Angles g;
    load_angles<LPR>(cs[buf] + w.tok * D, c, u, g);
    Turn tn;
    if constexpr (!NORM) make_turn<IL>(g, tn);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (NORM) {
        float2 wa[4], wb[4];
        load_weights<T>(a, t, u, wa, wb);
        make_turn<IL>(g, wa, wb, tn);
      }
      int left = n < a.N ? (t ? mine_k : mine_q) : 0;
      const int64_t step = w.step * a.so[t][1];
      T* out = static_cast<T*>(a.out[t]) + b * a.so[t][0] + n * a.so[t][2] + w.h0 * a.so[t][1] + u.off_a;
      // whole warps walk the steps: the norm's sums are exchanged
      for (int j = it[t]; j > 0; --j, --left, out += step) {
        float2 va[4], vb[4];
        copy_wait<S - 2>();
        const uint4* slot = mine + slot_i * 2 * U;
        read_unit<T>(slot, va);
        read_unit<T>(slot + U, vb);
        slot_i = slot_i + 1 == S ? 0 : slot_i + 1;
        issue();                         // into the slot that the last step read
        if constexpr (NORM) {
          float2 ss = __fmul2_rn(va[0], va[0]), st = __fmul2_rn(vb[0], vb[0]);
#pragma unroll
          for (int q = 1; q < 4; ++q) {
            ss = __ffma2_rn(va[q], va[q], ss);
            st = __ffma2_rn(vb[q], vb[q], st);
          }
          const float rstd = rsqrtf(row_sum<LPR>(__fadd2_rn(ss, st)) * (1.f / D) + a.eps);
          const float2 r2 = make_float2(rstd, rstd);
          turn<IL>(va, vb, tn);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            va[q] = __fmul2_rn(va[q], r2);
            vb[q] = __fmul2_rn(vb[q], r2);
          }
        } else {
          turn<IL>(va, vb, tn);
        }
        if (left > 0) {
          store_unit<T>(out, va);
          store_unit<T>(out + ab, vb);
        }
      }
    }
    if (item + gridDim.x < tl.items) {
      angle_table<D, IL>(a, pt, cs[buf ^ 1], tl.tok, buf ^ 1);
      tile_positions(a, tl, pt, item + 2 * static_cast<int64_t>(gridDim.x), buf);
      __syncthreads();
    }
  }
  copy_wait<0>();
}

// Gradient of the norm with the rotation.  A block works on one tensor
// (blocks below `split` on q, the others on k), walks that tensor's tiles and
// keeps its lanes' sums of the weight gradient in registers (16 columns per
// lane), joins them once at the end and leaves one partial row;
// weight_grad_kernel adds the blocks' rows in a fixed order, so the result does
// not depend on the schedule.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) qk_norm_bwd_kernel(const __grid_constant__ RotArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  constexpr int S = kBwdRing<T>, U = kPieces<T> * kThreads;
  extern __shared__ __align__(16) uint4 ring[];                 // [S][ga | gb | xa | xb][pieces][thread]
  __shared__ __align__(16) float cs[2][kMaxTile<D> * D];
  __shared__ PairTable pt;
  __shared__ float red[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPR;
  const LaneUnits u = lane_units<LPR, IL>(c, a.pairs);
  const int ab = u.off_b - u.off_a;
  const int t = static_cast<int>(blockIdx.x) >= a.split ? 1 : 0;
  const int blk = static_cast<int>(blockIdx.x) - (t ? a.split : 0);
  const int nblk = t ? static_cast<int>(gridDim.x) - a.split : a.split;
  const Tiles tl = a.tiles[t];
  const WarpRows w = warp_rows<RPW>(tl.tok, warp, lane / LPR);
  const int iters = head_steps(a.heads[t], w.first, w.step), mine_h = head_steps(a.heads[t], w.h0, w.step);
  const int64_t sg = w.step * a.sx[t][1], sx = w.step * a.sin[t][1], so = w.step * a.so[t][1];
  float2 wa[4], wb[4], acc_a[4], acc_b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc_a[i] = acc_b[i] = make_float2(0.f, 0.f);

  // the next step to copy: of tile p_item, p_seg steps left for the warp, p_left
  // for this lane, rows p_g and p_x
  int64_t p_item = static_cast<int64_t>(blk) - nblk;
  int p_seg = 0, p_left = 0, p_slot = 0;
  const T *p_g = nullptr, *p_x = nullptr;
  auto next_tile = [&]() {
    p_item += nblk;
    if (p_item >= tl.items) return;
    const int64_t b = p_item / tl.per, n = (p_item - b * tl.per) * tl.tok + w.tok;
    p_seg = iters;
    p_left = n < a.N ? mine_h : 0;
    p_g = static_cast<const T*>(a.x[t]) + b * a.sx[t][0] + n * a.sx[t][2] + w.h0 * a.sx[t][1] + u.off_a;
    p_x = static_cast<const T*>(a.in[t]) + b * a.sin[t][0] + n * a.sin[t][2] + w.h0 * a.sin[t][1] + u.off_a;
  };
  uint4* mine = ring + threadIdx.x;
  auto issue = [&]() {
    if (p_seg > 0) {
      if (p_left > 0) {
        uint4* slot = mine + p_slot * 4 * U;
        copy_unit<T>(slot, p_g);
        copy_unit<T>(slot + U, p_g + ab);
        copy_unit<T>(slot + 2 * U, p_x);
        copy_unit<T>(slot + 3 * U, p_x + ab);
      }
      p_slot = p_slot + 1 == S ? 0 : p_slot + 1;
      p_g += sg;
      p_x += sx;
      --p_left;
      if (--p_seg == 0) next_tile();
    }
    copy_commit();
  };
  next_tile();
  for (int i = 0; i < S - 1; ++i) issue();
  load_weights<T>(a, t, u, wa, wb);
  tile_positions(a, tl, pt, blk, 0);
  tile_positions(a, tl, pt, static_cast<int64_t>(blk) + nblk, 1);
  pair_table(a, pt);
  __syncthreads();
  angle_table<D, IL>(a, pt, cs[0], tl.tok, 0);
  __syncthreads();
  int slot_i = 0, buf = 0;
  for (int64_t item = blk; item < tl.items; item += nblk, buf ^= 1) {
    const int64_t b = item / tl.per, n = (item - b * tl.per) * tl.tok + w.tok;
    Angles ang;
    load_angles<LPR>(cs[buf] + w.tok * D, c, u, ang);
    Turn tn;
    make_turn<IL>(ang, tn);
    int left = n < a.N ? mine_h : 0;
    T* out = static_cast<T*>(a.out[t]) + b * a.so[t][0] + n * a.so[t][2] + w.h0 * a.so[t][1] + u.off_a;
    for (int j = iters; j > 0; --j, --left, out += so) {
      float2 ga[4], gb[4], xa[4], xb[4];
      copy_wait<S - 2>();
      const uint4* slot = mine + slot_i * 4 * U;
      read_unit<T>(slot, ga);
      read_unit<T>(slot + U, gb);
      read_unit<T>(slot + 2 * U, xa);
      read_unit<T>(slot + 3 * U, xb);
      slot_i = slot_i + 1 == S ? 0 : slot_i + 1;
      issue();                            // into the slot that the last step read
      turn<IL>(ga, gb, tn);
      // sums of x^2 and of g w x
      float2 ss = make_float2(0.f, 0.f), st = ss, sw = ss, sv = ss;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss = __ffma2_rn(xa[i], xa[i], ss);
        st = __ffma2_rn(xb[i], xb[i], st);
        sw = __ffma2_rn(__fmul2_rn(ga[i], wa[i]), xa[i], sw);
        sv = __ffma2_rn(__fmul2_rn(gb[i], wb[i]), xb[i], sv);
      }
      const float rstd = rsqrtf(row_sum<LPR>(__fadd2_rn(ss, st)) * (1.f / D) + a.eps);
      // xhat mean(g w xhat) = x rstd^2 (sum g w x) / D
      const float m = row_sum<LPR>(__fadd2_rn(sw, sv)) * (1.f / D) * rstd * rstd * rstd;
      const float2 r2 = make_float2(rstd, rstd), nm2 = make_float2(-m, -m);
      if (left > 0) {                     // other lanes hold an old row: they add nothing
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ga[i] = __fmul2_rn(ga[i], r2);
          gb[i] = __fmul2_rn(gb[i], r2);
          acc_a[i] = __ffma2_rn(ga[i], xa[i], acc_a[i]);
          acc_b[i] = __ffma2_rn(gb[i], xb[i], acc_b[i]);
          ga[i] = __ffma2_rn(ga[i], wa[i], __fmul2_rn(xa[i], nm2));
          gb[i] = __ffma2_rn(gb[i], wb[i], __fmul2_rn(xb[i], nm2));
        }
        store_unit<T>(out, ga);
        store_unit<T>(out + ab, gb);
      }
    }
    if (item + nblk < tl.items) {
      angle_table<D, IL>(a, pt, cs[buf ^ 1], tl.tok, buf ^ 1);
      tile_positions(a, tl, pt, item + 2 * static_cast<int64_t>(nblk), buf);
      __syncthreads();
    }
  }
  copy_wait<0>();
  // lanes of a warp that hold the same columns, then the warps
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v2 = i < 4 ? acc_a[i & 3] : acc_b[i & 3];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = e ? v2.y : v2.x;
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < LPR) red[warp][(i < 4 ? u.off_a : u.off_b) + 2 * (i & 3) + e] = v;
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += red[i][d];
    a.dw_part[static_cast<int64_t>(blockIdx.x) * D + d] = v;
  }
}

// dq_weight | dk_weight: the blocks' partial rows added up, 16 columns of one
// tensor per block, sixteen groups of threads taking every sixteenth row.
__global__ void __launch_bounds__(kThreads) weight_grad_kernel(const float* part, int split, int nparts,
                                                               int D, float* dqw, float* dkw) {
  __shared__ float red[16][16];
  const int grp = threadIdx.x >> 4, col = threadIdx.x & 15;
  const int t = static_cast<int>(blockIdx.x) * 16 >= D ? 1 : 0;
  const int d = static_cast<int>(blockIdx.x) * 16 - (t ? D : 0) + col;
  const int p0 = t ? split : 0, p1 = t ? nparts : split;
  float v = 0.f;
#pragma unroll 4
  for (int p = p0 + grp; p < p1; p += 16) v += __ldg(part + static_cast<int64_t>(p) * D + d);
  red[grp][col] = v;
  __syncthreads();
  if (grp == 0) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += red[w][col];
    (t ? dkw : dqw)[d] = v;
  }
}

// What a tile of `tok` tokens costs a block, in row steps of its warps: the
// steps of the heads, and the tile's own work (its angles, of which each thread
// forms tok * pairs / 256, its barrier and addresses).
double head_cost(int64_t heads, int64_t D, int tok) {
  const int64_t rpw = 512 / D, tpw = rpw < tok ? rpw : tok, groups = tok / tpw;
  const int64_t step = kWarps / groups * (rpw / tpw);      // heads per step of all warps of a group
  return static_cast<double>((heads + step - 1) / step);
}
double tile_cost(const RotaryParams& p, int tok) { return 0.7 + 0.35 * tok * p.pairs / kThreads; }

Tiles make_tiles(const RotaryParams& p, int tok) {
  Tiles t{};
  t.tok = tok;
  t.per = (p.N + tok - 1) / tok;
  t.items = p.B * t.per;
  return t;
}

// The tiles to choose from, with what each costs a block whose heads cost
// `heads(tok)`.
struct TileOptions {
  int n;
  Tiles t[8];
  double cost[8];
};
template <typename Cost>
TileOptions tile_options(const RotaryParams& p, Cost heads) {
  TileOptions o{};
  for (int tok = static_cast<int>(2048 / p.D); tok >= 1; tok /= 2, ++o.n) {
    o.t[o.n] = make_tiles(p, tok);
    o.cost[o.n] = heads(tok) + tile_cost(p, tok);
  }
  return o;
}
static_assert(kMostTokens == 1 << 7, "eight tile lengths");

// The tiles with which `slots` blocks end first.  Long tiles cost less in all,
// short ones spread short inputs over the SMs and leave less of the last round
// idle.
Tiles pick_tiles(const TileOptions& o, int64_t slots, double* time) {
  Tiles best{};
  *time = 0;
  for (int i = 0; i < o.n; ++i) {
    const int64_t rounds = o.t[i].items <= slots ? 1 : (o.t[i].items + slots - 1) / slots;
    const double ms = static_cast<double>(rounds) * o.cost[i];
    if (*time == 0 || ms < *time) {
      *time = ms;
      best = o.t[i];
    }
  }
  return best;
}

RotArgs make_args(const RotaryParams& p) {
  RotArgs a{};
  for (int t = 0; t < 2; ++t) {
    a.x[t] = p.x[t]; a.in[t] = p.in[t]; a.out[t] = p.out[t];
    for (int i = 0; i < 3; ++i) {
      a.sx[t][i] = p.sx[t][i]; a.sin[t][i] = p.sin[t][i]; a.so[t][i] = p.so[t][i];
    }
    a.heads[t] = static_cast<int>(t ? p.Hkv : p.Hq);
    a.w[t] = p.w[t];
  }
  a.N = p.N;
  a.pairs = p.pairs; a.naxes = p.naxes;
  for (int i = 0; i < 4; ++i) a.sec_end[i] = p.sec_end[i];
  a.inv_freq = p.inv_freq; a.pos = p.pos; a.pos64 = p.pos64;
  for (int i = 0; i < 3; ++i) a.ps[i] = p.ps[i];
  a.w_f32 = p.w_f32; a.eps = p.eps;
  return a;
}

template <typename T, int D, bool NORM, bool IL>
fa_status run_fwd(const RotaryParams& p, cudaStream_t s) {
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * fwd_blocks<T>(NORM);
  RotArgs a = make_args(p);
  double time;
  const auto heads = [&](int tok) { return head_cost(p.Hq, D, tok) + head_cost(p.Hkv, D, tok); };
  a.tiles[0] = pick_tiles(tile_options(p, heads), slots, &time);
  a.sign = p.backward ? -1.f : 1.f;      // without a norm the gradient is the rotation back
  const int64_t grid = a.tiles[0].items < slots ? a.tiles[0].items : slots;
  FA_CONFIGURE((rotary_kernel<T, D, NORM, IL>), kFwdSmem<T>);
  rotary_kernel<T, D, NORM, IL><<<dim3(static_cast<unsigned>(grid)), dim3(kThreads), kFwdSmem<T>, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

template <typename T, int D, bool IL>
fa_status run_bwd(const RotaryParams& p, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * kBwdBlocks;
  const int64_t slots = most < kRotaryMaxParts ? most : kRotaryMaxParts;
  RotArgs a = make_args(p);
  // The blocks dealt to q and k so that both end together: by their costs per
  // token, and the shares around that one.
  int64_t nq = 1, nk = 1;
  double best = 0;
  const int ref = static_cast<int>(1024 / D);
  const double cq = head_cost(p.Hq, D, ref) + tile_cost(p, ref), ck = head_cost(p.Hkv, D, ref) + tile_cost(p, ref);
  const int64_t mid = static_cast<int64_t>(static_cast<double>(slots) * cq / (cq + ck));
  const TileOptions oq = tile_options(p, [&](int tok) { return head_cost(p.Hq, D, tok); });
  const TileOptions ok = tile_options(p, [&](int tok) { return head_cost(p.Hkv, D, tok); });
  for (int64_t q = mid - 16; q <= mid + 16; q += 4) {
    if (q < 1 || q >= slots) continue;
    double tq, tk;
    const Tiles lq = pick_tiles(oq, q, &tq), lk = pick_tiles(ok, slots - q, &tk);
    const double t = tq > tk ? tq : tk;
    if (best == 0 || t < best) {
      best = t;
      a.tiles[0] = lq;
      a.tiles[1] = lk;
      nq = q < lq.items ? q : lq.items;
      nk = slots - q < lk.items ? slots - q : lk.items;
    }
  }
  a.sign = -1.f;
  a.dw_part = p.ws;
  a.split = static_cast<int>(nq);
  FA_CONFIGURE((qk_norm_bwd_kernel<T, D, IL>), kBwdSmem<T>);
  qk_norm_bwd_kernel<T, D, IL><<<dim3(static_cast<unsigned>(nq + nk)), dim3(kThreads), kBwdSmem<T>, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  weight_grad_kernel<<<dim3(2 * D / 16), dim3(kThreads), 0, s>>>(
      p.ws, a.split, static_cast<int>(nq + nk), D, p.dw[0], p.dw[1]);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

template <typename T, int D, bool IL>
fa_status run_layout(const RotaryParams& p, cudaStream_t s) {
  if (p.w[0] == nullptr) return run_fwd<T, D, false, IL>(p, s);
  return p.backward ? run_bwd<T, D, IL>(p, s) : run_fwd<T, D, true, IL>(p, s);
}

template <typename T, int D>
fa_status run_rotary(const RotaryParams& p, cudaStream_t s) {
  return p.interleaved ? run_layout<T, D, true>(p, s) : run_layout<T, D, false>(p, s);
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
