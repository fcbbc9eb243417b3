// FFMA (IEEE fp32) kernels of the prefix entry points: packed sequences behind
// one shared prefix, for fp32 inputs (whose products must not drop to TF32) and,
// when the FFMA path is selected, fp16 / bf16.
//
// The mathematics are those of fa_ffma.cu (online softmax in the log2 domain,
// P rebuilt from L in the gradient) with two sets of keys per query: the
// prefix's, all seen, then the sequence's own.  These problems are often small
// (a few short sequences), so the shape differs from that file's:
//  * a block has TM TY rows and 16 TY threads, each with TM x 4 of the scores,
//    and walks tiles of 64 rows of the other side, copied a tile ahead (cp.async
//    for fp32).  Operands are read from shared memory four at a time along the
//    contraction (rows padded to D + 4 floats: the eight rows that a quarter of a
//    warp reads cover all banks).  Small problems take 16 rows in four warps
//    (TM = 2, one warp per scheduler; two warps of TM = 4 issued half as fast);
//    where blocks of 64 rows (32 for the gradient at D = 128; TM = 4) come to two
//    per SM, those read the walked tiles a quarter as often;
//  * where even those leave SMs idle, a cluster of up to four blocks deals the
//    tiles of one walk out and joins its sums through distributed shared memory
//    (in the order of the blocks);
//  * every product is one fp32 FMA per term, in the order of the contraction;
//  * the gradient is one launch: blocks for dK / dV of the prefix (every packed
//    query row against it, the longest walks, first), for dK / dV of the own
//    keys and for dQ.  They share only inputs, and three launches in turn each
//    left most of the GPU idle.
// 3 sequences of up to 130 rows, 4 heads of 64, 200 prefix keys: forward 18 us,
// gradient 33 us (three launches of 64-row blocks with one operand per read:
// 65 and 282).  Bound by the instructions of one block's steps, four warps per
// SM; at large sizes by shared-memory reads, twice the FMAs' time.
//
// The gradient of small fp16 / bf16 problems takes these kernels too
// (prefix_ffma_pays): one launch instead of three, and no rounding of P and dS.

#include "tc_common.cuh"

#include <cmath>

namespace fa {
namespace {

constexpr int BC = 64;        // rows of a walked tile
constexpr int PLD = BC + 4;   // leading dimension of P and dS

struct Args {
  const void* q; const void* k; const void* v; const void* dout;
  void* o; float* lse; const float* lse_in; const float* delta;
  float* delta_out;           // few_keys_delta_kernel
  void* dq; void* dk; void* dv; void* dkp; void* dvp;
  Geo g, gp;                  // own keys; all query rows against the prefix
  Prefix pfx;
  int64_t sq[4], sk[4], sv[4], so[4], sdo[4], sdq[4], sdk[4], sdv[4], sdkp[4], sdvp[4];
  int causal;
  float scale;
  int64_t n_pre, n_own;       // gradient: blocks of the prefix's and the own keys' dK / dV
  int cl;                     // blocks (one cluster) that share a walk
  unsigned int* status;
};

// Copies rows [row0, row0 + ROWS) of a strided N x D matrix into fp32 rows of
// D + 4; rows at or past N are zero.  fp32 rows arrive asynchronously.
template <typename T, int D, int ROWS, int NT>
__device__ __forceinline__ void stage(float* dst, const T* base, int64_t sn, int64_t row0, int64_t N) {
  constexpr int VEC = 16 / sizeof(T), UN = D / VEC, LD = D + 4;
  for (int idx = threadIdx.x; idx < ROWS * UN; idx += NT) {
    const int r = idx / UN, u = idx % UN;
    const int64_t row = row0 + r;
    float* to = dst + r * LD + u * VEC;
    if constexpr (sizeof(T) == 4) {
      // the address of a row past N is not formed; the copy of 0 bytes fills zeros
      const T* from = row < N ? base + row * sn + u * VEC : base;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from),
                   "r"(row < N ? 16 : 0)
                   : "memory");
    } else {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (row < N) w = __ldg(reinterpret_cast<const uint4*>(base + row * sn + u * VEC));
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        *reinterpret_cast<float4*>(to + i) = make_float4(Elem<T>::to_f32(e[i]), Elem<T>::to_f32(e[i + 1]),
                                                         Elem<T>::to_f32(e[i + 2]), Elem<T>::to_f32(e[i + 3]));
    }
  }
}
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The columns of a D-wide accumulator row that thread tx owns: groups of VW
// neighbours, group e at e * 16 * VW + VW * tx.
template <int D>
struct Cols {
  static constexpr int E = D / 16, VW = E < 4 ? E : 4, GR = E / VW;
};
template <int D>
__device__ __forceinline__ void load_cols(const float* row, int tx, float (&x)[D / 16]) {
  using C = Cols<D>;
#pragma unroll
  for (int g = 0; g < C::GR; ++g) {
    const float* p = row + g * 16 * C::VW + C::VW * tx;
    if constexpr (C::VW == 4) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      x[4 * g] = t.x; x[4 * g + 1] = t.y; x[4 * g + 2] = t.z; x[4 * g + 3] = t.w;
    } else if constexpr (C::VW == 2) {
      const float2 t = *reinterpret_cast<const float2*>(p);
      x[0] = t.x; x[1] = t.y;
    } else {
      x[0] = *p;
    }
  }
}
template <typename T, int D>
__device__ __forceinline__ void store_cols(T* row, int tx, const float (&x)[D / 16], float mul) {
  using C = Cols<D>;
#pragma unroll
  for (int e = 0; e < C::E; ++e)
    row[(e / C::VW) * 16 * C::VW + C::VW * tx + e % C::VW] = Elem<T>::from_f32(x[e] * mul);
}

template <int D>
__device__ __forceinline__ void put_cols(float* row, int tx, const float (&x)[D / 16]) {
  using C = Cols<D>;
#pragma unroll
  for (int e = 0; e < C::E; ++e) row[(e / C::VW) * 16 * C::VW + C::VW * tx + e % C::VW] = x[e];
}

// Sums of a cluster's blocks: `part` (ROWS rows of D floats in every block's
// shared memory, published by a cluster barrier), times w(rank, row), in the
// order of the ranks; four elements at a time to put(row, column, sum).  Block
// `rank` takes every cl-th row.
template <int D, int ROWS, int NT, typename W, typename Put>
__device__ __forceinline__ void join_cluster(const float* part, int rank, int cl, W w, Put put) {
  for (int idx = threadIdx.x; idx < ROWS / cl * (D / 4); idx += NT) {
    const int row = (idx / (D / 4)) * cl + rank, col = 4 * (idx % (D / 4));
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < cl; ++r) {
      const float4 x = tc::ld_cluster_f4(tc::cluster_map(tc::smem_u32(part + row * D + col), static_cast<uint32_t>(r)));
      const float f = w(r, row);
      sum.x = fmaf(f, x.x, sum.x); sum.y = fmaf(f, x.y, sum.y);
      sum.z = fmaf(f, x.z, sum.z); sum.w = fmaf(f, x.w, sum.w);
    }
    put(row, col, sum);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& x, float mul) {
  p[0] = Elem<T>::from_f32(x.x * mul); p[1] = Elem<T>::from_f32(x.y * mul);
  p[2] = Elem<T>::from_f32(x.z * mul); p[3] = Elem<T>::from_f32(x.w * mul);
}
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];"
               : "=f"(v) : "r"(tc::cluster_map(tc::smem_u32(p), static_cast<uint32_t>(rank))) : "memory");
  return v;
}

__device__ __forceinline__ float at(const float4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// acc[i][j] += sum_d A[ty TM + i][d] B[tx + 16 j][d]
template <int D, int TM>
__device__ __forceinline__ void dots(const float* A, const float* B, int ty, int tx, float (&acc)[TM][4]) {
  constexpr int LD = D + 4;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 a[TM], b[4];
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty * TM + i) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(at(a[i], u), at(b[j], u), acc[i][j]);
  }
}

// acc[i][.] += sum_r W[ty TM + i][r] M[r][columns of tx]
template <int D, int TM>
__device__ __forceinline__ void sums(const float* W, const float* M, int ty, int tx,
                                     float (&acc)[TM][D / 16]) {
  constexpr int LD = D + 4;
#pragma unroll 2
  for (int r = 0; r < BC; r += 4) {
    float4 w[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) w[i] = *reinterpret_cast<const float4*>(W + (ty * TM + i) * PLD + r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float m[D / 16];
      load_cols<D>(M + (r + u) * LD, tx, m);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[i][e] = fmaf(at(w[i], u), m[e], acc[i][e]);
    }
  }
}

// The key tiles that a query tile walks: the prefix's, then the own ones.
template <typename T>
struct KeyWalk {
  const T *kp, *vp, *k, *v;
  int64_t P, nk, kend;        // prefix keys, own keys, own keys below kend are walked
  int64_t skp, svp, sk, sv;
  int np, n;                  // tiles of the prefix, of both
  __device__ __forceinline__ int64_t first(int t) const { return static_cast<int64_t>(t < np ? t : t - np) * BC; }
  __device__ __forceinline__ int64_t keys(int t) const { return t < np ? P : nk; }
};
template <typename T>
__device__ __forceinline__ KeyWalk<T> key_walk(const Args& a, const SeqView& s, int64_t hk, int64_t kend) {
  KeyWalk<T> w;
  w.kp = static_cast<const T*>(a.pfx.k) + hk * a.pfx.sk[1];
  w.vp = static_cast<const T*>(a.pfx.v) + hk * a.pfx.sv[1];
  w.k = static_cast<const T*>(a.k) + s.b * a.sk[0] + hk * a.sk[1] + s.k0 * a.sk[2];
  w.v = static_cast<const T*>(a.v) + s.b * a.sv[0] + hk * a.sv[1] + s.k0 * a.sv[2];
  w.P = a.pfx.P; w.nk = s.nk; w.kend = kend;
  w.skp = a.pfx.sk[2]; w.svp = a.pfx.sv[2]; w.sk = a.sk[2]; w.sv = a.sv[2];
  w.np = static_cast<int>((w.P + BC - 1) / BC);
  w.n = w.np + static_cast<int>((kend + BC - 1) / BC);
  return w;
}
template <typename T, int D, int NT>
__device__ __forceinline__ void stage_keys(const KeyWalk<T>& w, int t, float* ks, float* vs) {
  const bool pre = t < w.np;
  stage<T, D, BC, NT>(ks, pre ? w.kp : w.k, pre ? w.skp : w.sk, w.first(t), w.keys(t));
  stage<T, D, BC, NT>(vs, pre ? w.vp : w.v, pre ? w.svp : w.sv, w.first(t), w.keys(t));
}

// Block id -> (flat head of the query side, query tile), longest tiles first
// under a causal mask; false when the tile lies past its sequence.
__device__ __forceinline__ bool query_block(const Args& a, int64_t id, int rows, SeqView& s, int64_t& h,
                                            int64_t& q0) {
  const int64_t BH = a.g.B * a.g.Hq, nt = (a.g.Nq + rows - 1) / rows;
  const int64_t bh = id % BH, t = id / BH;
  h = bh % a.g.Hq;
  q0 = (a.causal ? nt - 1 - t : t) * rows;
  s = seq_view(a.g, bh / a.g.Hq);
  if (!s.ok) {
    if (threadIdx.x == 0) record_status(a.status, FA_ERR_SEQLENS);
    return false;
  }
  return q0 < s.nq;
}

template <typename T, int D, int TY, int TM>
__global__ void __launch_bounds__(16 * TY) fwd_prefix_ffma_kernel(const __grid_constant__ Args a) {
  constexpr int LD = D + 4, NT = 16 * TY, BR = TM * TY;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* KV = Qs + BR * LD;            // [2][K | V]
  float* Ps = KV + 4 * BC * LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  SeqView s;
  int64_t h, q0;
  const int cl = a.cl, rank = static_cast<int>(blockIdx.x % cl);
  if (!query_block(a, blockIdx.x / cl, BR, s, h, q0)) return;   // all blocks of a cluster alike
  const int64_t hk = h / a.g.G;
  const KeyWalk<T> w = key_walk<T>(a, s, hk, a.causal ? min(s.nk, q0 + BR) : s.nk);
  stage<T, D, BR, NT>(Qs, static_cast<const T*>(a.q) + s.b * a.sq[0] + h * a.sq[1] + s.q0 * a.sq[2], a.sq[2], q0,
                      s.nq);
  if (rank < w.n) stage_keys<T, D, NT>(w, rank, KV, KV + BC * LD);
  const float c = a.scale * kLog2e;
  float m[TM], l[TM], acc[TM][D / 16];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    m[i] = -INFINITY; l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) acc[i][e] = 0.f;
  }
  int buf = 0;
  for (int t = rank; t < w.n; t += cl, buf ^= 1) {
    const float* Ks = KV + buf * 2 * BC * LD;
    const float* Vs = Ks + BC * LD;
    stage_wait();
    __syncthreads();                   // this tile is here, the last one is no longer read
    if (t + cl < w.n)
      stage_keys<T, D, NT>(w, t + cl, KV + (buf ^ 1) * 2 * BC * LD, KV + ((buf ^ 1) * 2 + 1) * BC * LD);
    float sc[TM][4] = {};
    dots<D, TM>(Qs, Ks, ty, tx, sc);
    const int64_t k0 = w.first(t), nk = w.keys(t);
    const bool causal = a.causal && t >= w.np;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t qp = q0 + ty * TM + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t kp = k0 + tx + 16 * j;
        if (kp >= nk || (causal && kp > qp)) sc[i][j] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(sc[i][0], sc[i][1]), fmaxf(sc[i][2], sc[i][3]));
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(m[i], mx * c);
      // no key seen yet: exponents against 0, so that -inf stays a weight of 0
      const float ms = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m[i] - ms);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(fmaf(sc[i][j], c, -ms));
        Ps[(ty * TM + i) * PLD + tx + 16 * j] = p;
        sum += p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[i] = fmaf(l[i], alpha, sum);
      m[i] = m_new;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) acc[i][e] *= alpha;
    }
    __syncwarp();                      // a row of P is written and read by one half-warp
    sums<D, TM>(Ps, Vs, ty, tx, acc);
    __syncwarp();
  }
  stage_wait();
  if (cl > 1) {
    __syncthreads();
    float* part = KV;                  // [BR][D] sums, then [BR] maxima and [BR] sums of weights
    float* ml = KV + BR * D;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      put_cols<D>(part + (ty * TM + i) * D, tx, acc[i]);
      if (tx == 0) {
        ml[ty * TM + i] = m[i];
        ml[BR + ty * TM + i] = l[i];
      }
    }
    tc::cluster_sync_all();
    // weights of the blocks' sums of a row, over the sum of all weights
    if (threadIdx.x < BR) {
      const int row = threadIdx.x;
      float mx = -INFINITY, sum = 0.f;
      for (int r = 0; r < cl; ++r) mx = fmaxf(mx, ld_cluster(ml + row, r));
      const float ms = mx == -INFINITY ? 0.f : mx;
      for (int r = 0; r < cl; ++r) {
        const float f = exp2f(ld_cluster(ml + row, r) - ms);
        Ps[row * PLD + r] = f;
        sum = fmaf(ld_cluster(ml + BR + row, r), f, sum);
      }
      Ps[row * PLD + cl] = sum > 0.f ? 1.f / sum : 0.f;     // no key at all: O = 0
      if (rank == 0 && q0 + row < s.nq)
        a.lse[lse_index(a.g, s, h, q0 + row)] = sum > 0.f ? (ms + log2f(sum)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    T* o = static_cast<T*>(a.o) + s.b * a.so[0] + h * a.so[1] + (s.q0 + q0) * a.so[2];
    join_cluster<D, BR, NT>(part, rank, cl, [&](int r, int row) { return Ps[row * PLD + r]; },
                            [&](int row, int col, const float4& x) {
                              if (q0 + row < s.nq) store4<T>(o + row * a.so[2] + col, x, Ps[row * PLD + cl]);
                            });
    tc::cluster_sync_all();            // no block leaves while another reads its sums
    return;
  }
  T* o = static_cast<T*>(a.o) + s.b * a.so[0] + h * a.so[1] + s.q0 * a.so[2];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = q0 + ty * TM + i;
    if (row >= s.nq) continue;
    const bool any = l[i] > 0.f;       // no key at all: O = 0, L = -inf
    float x[D / 16];
#pragma unroll
    for (int e = 0; e < D / 16; ++e) x[e] = any ? acc[i][e] / l[i] : 0.f;
    store_cols<T, D>(o + row * a.so[2], tx, x, 1.f);
    if (tx == 0) a.lse[lse_index(a.g, s, h, row)] = any ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
  }
}

// dK / dV of TM TY keys: `g` and the key tensors are the sequences' own or the
// prefix's.
template <typename T, int D, int TY, int TM>
__device__ __forceinline__ void dkdv_block(const Args& a, const Geo& g, bool pre, int64_t id, int rank, float* sm) {
  constexpr int LD = D + 4, NT = 16 * TY, BR = TM * TY;
  float* Ks = sm;
  float* Vs = Ks + BR * LD;
  float* QG = Vs + BR * LD;            // [2][Q | dO]
  float* Ps = QG + 4 * BC * LD;
  float* dSs = Ps + BR * PLD;
  float* LDl = dSs + BR * PLD;         // [2][L * log2(e) | Delta]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t BH = g.B * g.Hkv;
  const int64_t bhk = id % BH, k0 = id / BH * BR;
  const int64_t hk = bhk % g.Hkv;
  const SeqView s = seq_view(g, bhk / g.Hkv);
  if (!s.ok) {
    if (threadIdx.x == 0) record_status(a.status, FA_ERR_SEQLENS);
    return;
  }
  if (k0 >= s.nk) return;
  const bool causal = a.causal && !pre;
  const int64_t* sk = pre ? a.pfx.sk : a.sk;
  const int64_t* sv = pre ? a.pfx.sv : a.sv;
  stage<T, D, BR, NT>(Ks, static_cast<const T*>(pre ? a.pfx.k : a.k) + hk * sk[1] + s.k0 * sk[2], sk[2], k0, s.nk);
  stage<T, D, BR, NT>(Vs, static_cast<const T*>(pre ? a.pfx.v : a.v) + hk * sv[1] + s.k0 * sv[2], sv[2], k0, s.nk);
  // the query tiles of every query head that reads these keys
  const int64_t first = causal ? k0 / BC : 0, tiles = (s.nq + BC - 1) / BC;
  const int64_t per = tiles > first ? tiles - first : 0, steps = per * g.G;
  auto load = [&](int64_t it, int buf) {
    const int64_t h = hk * g.G + it / per, q0 = (first + it % per) * BC;
    float* Qs = QG + buf * 2 * BC * LD;
    stage<T, D, BC, NT>(Qs, static_cast<const T*>(a.q) + h * a.sq[1] + s.q0 * a.sq[2], a.sq[2], q0, s.nq);
    stage<T, D, BC, NT>(Qs + BC * LD, static_cast<const T*>(a.dout) + h * a.sdo[1] + s.q0 * a.sdo[2], a.sdo[2], q0,
                        s.nq);
    static_assert(NT >= BC, "one L and Delta per thread");
    if (threadIdx.x < BC) {
      const int64_t row = q0 + threadIdx.x, li = lse_index(g, s, h, row);
      LDl[buf * 2 * BC + threadIdx.x] = row < s.nq ? a.lse_in[li] * kLog2e : 0.f;
      LDl[(buf * 2 + 1) * BC + threadIdx.x] = row < s.nq ? a.delta[li] : 0.f;
    }
  };
  const float c = a.scale * kLog2e;
  float dk[TM][D / 16] = {}, dv[TM][D / 16] = {};
  const int cl = a.cl;
  if (rank < steps) load(rank, 0);
  int buf = 0;
  for (int64_t it = rank; it < steps; it += cl, buf ^= 1) {
    const float* Qs = QG + buf * 2 * BC * LD;
    const float* Gs = Qs + BC * LD;
    const int64_t q0 = (first + it % per) * BC;
    stage_wait();
    __syncthreads();
    if (it + cl < steps) load(it + cl, buf ^ 1);
    // element (key ty TM + i, query tx + 16 j)
    float sc[TM][4] = {}, dp[TM][4] = {};
    dots<D, TM>(Ks, Qs, ty, tx, sc);
    dots<D, TM>(Vs, Gs, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ql = tx + 16 * j;
        const int64_t qp = q0 + ql, kp = k0 + ty * TM + i;
        const bool keep = qp < s.nq && (!causal || kp <= qp);
        const float p = keep ? exp2f(fmaf(sc[i][j], c, -LDl[buf * 2 * BC + ql])) : 0.f;
        Ps[(ty * TM + i) * PLD + ql] = p;
        dSs[(ty * TM + i) * PLD + ql] = p * (dp[i][j] - LDl[(buf * 2 + 1) * BC + ql]);
      }
    __syncwarp();
    sums<D, TM>(Ps, Gs, ty, tx, dv);
    sums<D, TM>(dSs, Qs, ty, tx, dk);
    __syncwarp();
  }
  stage_wait();
  const int64_t* sdk = pre ? a.sdkp : a.sdk;
  const int64_t* sdv = pre ? a.sdvp : a.sdv;
  T* dkp = static_cast<T*>(pre ? a.dkp : a.dk) + hk * sdk[1] + s.k0 * sdk[2];
  T* dvp = static_cast<T*>(pre ? a.dvp : a.dv) + hk * sdv[1] + s.k0 * sdv[2];
  if (cl > 1) {
    __syncthreads();
    float* part = QG;                  // [BR][D] of dK, then of dV
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      put_cols<D>(part + (ty * TM + i) * D, tx, dk[i]);
      put_cols<D>(part + (BR + ty * TM + i) * D, tx, dv[i]);
    }
    tc::cluster_sync_all();
    join_cluster<D, 2 * BR, NT>(part, rank, cl, [](int, int) { return 1.f; },
                                [&](int row, int col, const float4& x) {
                                  const int64_t key = k0 + row % BR;
                                  if (key >= s.nk) return;
                                  if (row < BR) store4<T>(dkp + key * sdk[2] + col, x, a.scale);
                                  else store4<T>(dvp + key * sdv[2] + col, x, 1.f);
                                });
    tc::cluster_sync_all();
    return;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = k0 + ty * TM + i;
    if (row >= s.nk) continue;
    store_cols<T, D>(dkp + row * sdk[2], tx, dk[i], a.scale);
    store_cols<T, D>(dvp + row * sdv[2], tx, dv[i], 1.f);
  }
}

template <typename T, int D, int TY, int TM>
__device__ __forceinline__ void dq_block(const Args& a, int64_t id, int rank, float* sm) {
  constexpr int LD = D + 4, NT = 16 * TY, BR = TM * TY;
  float* Qs = sm;
  float* Gs = Qs + BR * LD;
  float* KV = Gs + BR * LD;            // [2][K | V]
  float* dSs = KV + 4 * BC * LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  SeqView s;
  int64_t h, q0;
  if (!query_block(a, id, BR, s, h, q0)) return;
  const int64_t hk = h / a.g.G;
  const KeyWalk<T> w = key_walk<T>(a, s, hk, a.causal ? min(s.nk, q0 + BR) : s.nk);
  stage<T, D, BR, NT>(Qs, static_cast<const T*>(a.q) + h * a.sq[1] + s.q0 * a.sq[2], a.sq[2], q0, s.nq);
  stage<T, D, BR, NT>(Gs, static_cast<const T*>(a.dout) + h * a.sdo[1] + s.q0 * a.sdo[2], a.sdo[2], q0, s.nq);
  const int cl = a.cl;
  if (rank < w.n) stage_keys<T, D, NT>(w, rank, KV, KV + BC * LD);
  const float c = a.scale * kLog2e;
  float L2[TM], Dl[TM], dq[TM][D / 16] = {};
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = q0 + ty * TM + i, li = lse_index(a.g, s, h, row);
    L2[i] = row < s.nq ? a.lse_in[li] * kLog2e : 0.f;
    Dl[i] = row < s.nq ? a.delta[li] : 0.f;
  }
  int buf = 0;
  for (int t = rank; t < w.n; t += cl, buf ^= 1) {
    const float* Ks = KV + buf * 2 * BC * LD;
    const float* Vs = Ks + BC * LD;
    stage_wait();
    __syncthreads();
    if (t + cl < w.n)
      stage_keys<T, D, NT>(w, t + cl, KV + (buf ^ 1) * 2 * BC * LD, KV + ((buf ^ 1) * 2 + 1) * BC * LD);
    float sc[TM][4] = {}, dp[TM][4] = {};
    dots<D, TM>(Qs, Ks, ty, tx, sc);
    dots<D, TM>(Gs, Vs, ty, tx, dp);
    const int64_t k0 = w.first(t), nk = w.keys(t);
    const bool causal = a.causal && t >= w.np;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t kp = k0 + tx + 16 * j, qp = q0 + ty * TM + i;
        const bool keep = kp < nk && (!causal || kp <= qp);
        const float p = keep ? exp2f(fmaf(sc[i][j], c, -L2[i])) : 0.f;
        dSs[(ty * TM + i) * PLD + tx + 16 * j] = p * (dp[i][j] - Dl[i]);
      }
    __syncwarp();
    sums<D, TM>(dSs, Ks, ty, tx, dq);
    __syncwarp();
  }
  stage_wait();
  T* out = static_cast<T*>(a.dq) + h * a.sdq[1] + s.q0 * a.sdq[2];
  if (cl > 1) {
    __syncthreads();
    float* part = KV;                  // [BR][D]
#pragma unroll
    for (int i = 0; i < TM; ++i) put_cols<D>(part + (ty * TM + i) * D, tx, dq[i]);
    tc::cluster_sync_all();
    join_cluster<D, BR, NT>(part, rank, cl, [](int, int) { return 1.f; },
                            [&](int row, int col, const float4& x) {
                              if (q0 + row < s.nq) store4<T>(out + (q0 + row) * a.sdq[2] + col, x, a.scale);
                            });
    tc::cluster_sync_all();
    return;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = q0 + ty * TM + i;
    if (row < s.nq) store_cols<T, D>(out + row * a.sdq[2], tx, dq[i], a.scale);
  }
}

template <typename T, int D, int TY, int TM>
__global__ void __launch_bounds__(16 * TY) bwd_prefix_ffma_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) float sm[];
  const int64_t id = blockIdx.x / a.cl;
  const int rank = static_cast<int>(blockIdx.x % a.cl);
  if (id < a.n_pre) dkdv_block<T, D, TY, TM>(a, a.gp, true, id, rank, sm);
  else if (id < a.n_pre + a.n_own) dkdv_block<T, D, TY, TM>(a, a.g, false, id - a.n_pre, rank, sm);
  else dq_block<T, D, TY, TM>(a, id - a.n_pre - a.n_own, rank, sm);
}

// Delta of rows that see few keys.  Delta = sum_j P_j dP_j is the same number as
// rowsum(dO o O), but O has been rounded: with n keys that error is about 1 / sqrt(n)
// of the gradient's own rounding, and more where one key takes most of the weight
// (fp16, two keys per row: dQ was off by 3.2 times what rounding dQ alone costs,
// 1.4 with this).  A warp takes a row, a lane a key; above kFewKeys the
// error does not show and rowsum(dO o O) stays.  Launched for prefixes below kFewKeys
// only; a block per sequence and head, some microseconds.
template <typename T, int D>
__global__ void __launch_bounds__(256) few_keys_delta_kernel(const __grid_constant__ Args a) {
  constexpr int VEC = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t h = blockIdx.x % a.g.Hq, hk = h / a.g.G;
  const SeqView s = seq_view(a.g, blockIdx.x / a.g.Hq);
  if (!s.ok) {
    if (threadIdx.x == 0) record_status(a.status, FA_ERR_SEQLENS);
    return;
  }
  const int64_t P = a.pfx.P;
  // rows with at most kFewKeys keys: all, or the first under a causal mask
  const int64_t rows = P + s.nk <= kFewKeys ? s.nq : (a.causal ? min(s.nq, kFewKeys - P) : 0);
  const bool pre = lane < P;
  const int64_t key = pre ? lane : lane - P;
  const T* kr = pre ? static_cast<const T*>(a.pfx.k) + hk * a.pfx.sk[1] + key * a.pfx.sk[2]
                    : static_cast<const T*>(a.k) + hk * a.sk[1] + (s.k0 + key) * a.sk[2];
  const T* vr = pre ? static_cast<const T*>(a.pfx.v) + hk * a.pfx.sv[1] + key * a.pfx.sv[2]
                    : static_cast<const T*>(a.v) + hk * a.sv[1] + (s.k0 + key) * a.sv[2];
  for (int64_t row = warp; row < rows; row += 8) {
    const int64_t n = P + (a.causal ? min(row + 1, s.nk) : s.nk);
    const T* q = static_cast<const T*>(a.q) + h * a.sq[1] + (s.q0 + row) * a.sq[2];
    const T* g = static_cast<const T*>(a.dout) + h * a.sdo[1] + (s.q0 + row) * a.sdo[2];
    const int64_t li = lse_index(a.g, s, h, row);
    float sc = 0.f, dp = 0.f;
    if (lane < n) {
#pragma unroll 4
      for (int d = 0; d < D; d += VEC) {
        const uint4 w[4] = {__ldg(reinterpret_cast<const uint4*>(q + d)), __ldg(reinterpret_cast<const uint4*>(kr + d)),
                            __ldg(reinterpret_cast<const uint4*>(g + d)), __ldg(reinterpret_cast<const uint4*>(vr + d))};
        const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sc = fmaf(Elem<T>::to_f32(e[i]), Elem<T>::to_f32(e[VEC + i]), sc);
          dp = fmaf(Elem<T>::to_f32(e[2 * VEC + i]), Elem<T>::to_f32(e[3 * VEC + i]), dp);
        }
      }
    }
    float sum = lane < n ? exp2f(fmaf(sc, a.scale * kLog2e, -a.lse_in[li] * kLog2e)) * dp : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) a.delta_out[li] = sum;
  }
}

constexpr int fwd_smem(int D, int BR) { return 4 * ((BR + 4 * BC) * (D + 4) + BR * PLD); }
constexpr int bwd_smem(int D, int BR) {
  return 4 * ((2 * BR + 4 * BC) * (D + 4) + 2 * BR * PLD + 4 * BC);
}
// TY of the large blocks (TM = 4)
constexpr int fwd_big(int) { return 16; }
constexpr int bwd_big(int D) { return D == 128 ? 8 : 16; }
static_assert(bwd_smem(128, 4 * bwd_big(128)) <= 232448 && bwd_smem(64, 4 * bwd_big(64)) <= 232448 &&
                  fwd_smem(128, 4 * fwd_big(128)) <= 232448, "shared memory per block");

int64_t tiles(int64_t n, int rows) { return (n + rows - 1) / rows; }

int64_t fwd_blocks(const Args& a, int BR) { return a.g.B * a.g.Hq * tiles(a.g.Nq, BR); }

// Blocks that share a walk of `steps` tiles, with `per_sm` blocks per SM at
// most.  3 sequences of up to 130 rows behind 200 keys: forward 20.9 us with four
// blocks to a walk (two rounds of blocks), 17.8 with the two that stay resident;
// gradient 32.7 us at four per SM, 54 at the two that stay resident (its walks
// are longer and of unequal lengths).
int pick_cluster(int64_t blocks, int64_t steps, int64_t per_sm) {
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * per_sm;
  int cl = 1;
  while (cl < 4 && 2 * cl <= steps && blocks * 2 * cl <= slots) cl *= 2;
  return cl;
}

template <typename Kern>
fa_status launch(Kern kern, int64_t blocks, int threads, int smem, const Args& a, cudaStream_t s) {
  if (blocks * a.cl > 0x7fffffffLL) return FA_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * a.cl));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (a.cl > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.cl);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return FA_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

template <typename T, int D, int TY, int TM>
fa_status launch_fwd(Args a, cudaStream_t s) {
  const int64_t blocks = fwd_blocks(a, TM * TY);
  a.cl = pick_cluster(blocks, tiles(a.pfx.P, BC) + tiles(a.g.Nk, BC),
                      233472 / (fwd_smem(D, TM * TY) + 1024));
  FA_CONFIGURE((fwd_prefix_ffma_kernel<T, D, TY, TM>), fwd_smem(D, TM * TY));
  return launch(fwd_prefix_ffma_kernel<T, D, TY, TM>, blocks, 16 * TY, fwd_smem(D, TM * TY), a, s);
}

int64_t bwd_blocks(Args& a, int BR) {
  a.n_pre = a.pfx.P > 0 ? a.g.Hkv * tiles(a.pfx.P, BR) : 0;
  a.n_own = a.g.B * a.g.Hkv * tiles(a.g.Nk, BR);
  return a.n_pre + a.n_own + a.g.B * a.g.Hq * tiles(a.g.Nq, BR);
}

template <typename T, int D, int TY, int TM>
fa_status launch_bwd(Args a, cudaStream_t s) {
  const int64_t blocks = bwd_blocks(a, TM * TY);
  a.cl = pick_cluster(blocks, tiles(a.pfx.P, BC) + tiles(a.g.Nk, BC), 4);
  FA_CONFIGURE((bwd_prefix_ffma_kernel<T, D, TY, TM>), bwd_smem(D, TM * TY));
  return launch(bwd_prefix_ffma_kernel<T, D, TY, TM>, blocks, 16 * TY, bwd_smem(D, TM * TY), a, s);
}

template <typename T>
fa_status launch_few_keys(const Args& a, int64_t D, cudaStream_t s) {
  const int64_t blocks = a.g.B * a.g.Hq;
  if (blocks > 0x7fffffffLL) return FA_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>(blocks)), threads(256);
  switch (D) {
    case 16: few_keys_delta_kernel<T, 16><<<grid, threads, 0, s>>>(a); break;
    case 32: few_keys_delta_kernel<T, 32><<<grid, threads, 0, s>>>(a); break;
    case 64: few_keys_delta_kernel<T, 64><<<grid, threads, 0, s>>>(a); break;
    case 128: few_keys_delta_kernel<T, 128><<<grid, threads, 0, s>>>(a); break;
    default: return FA_ERR_ARG;
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// Large blocks where they come to two per SM.
template <typename T, int D>
fa_status run(const Args& a, bool bwd, cudaStream_t s) {
  const int64_t enough = 2 * static_cast<int64_t>(device_sm_count());
  if (!bwd)
    return fwd_blocks(a, 4 * fwd_big(D)) >= enough ? launch_fwd<T, D, fwd_big(D), 4>(a, s)
                                                   : launch_fwd<T, D, 8, 2>(a, s);
  Args t = a;
  return bwd_blocks(t, 4 * bwd_big(D)) >= enough ? launch_bwd<T, D, bwd_big(D), 4>(a, s)
                                                 : launch_bwd<T, D, 8, 2>(a, s);
}

template <typename T>
fa_status run_d(const Args& a, int64_t D, bool bwd, cudaStream_t s) {
  switch (D) {
    case 16: return run<T, 16>(a, bwd, s);
    case 32: return run<T, 32>(a, bwd, s);
    case 64: return run<T, 64>(a, bwd, s);
    case 128: return run<T, 128>(a, bwd, s);
  }
  return FA_ERR_ARG;
}
fa_status run_any(const Args& a, int64_t D, fa_dtype dt, bool bwd, cudaStream_t s) {
  switch (dt) {
    case FA_F32: return run_d<float>(a, D, bwd, s);
    case FA_F16: return run_d<__half>(a, D, bwd, s);
    case FA_BF16: return run_d<__nv_bfloat16>(a, D, bwd, s);
  }
  return FA_ERR_ARG;
}

void copy4(int64_t* dst, const int64_t* src) { for (int i = 0; i < 4; ++i) dst[i] = src[i]; }

}  // namespace

fa_status launch_fwd_prefix_ffma(const FwdParams& p, cudaStream_t s) {
  Args a{};
  a.q = p.q; a.k = p.k; a.v = p.v; a.o = p.o; a.lse = p.lse;
  a.g = p.g; a.pfx = p.pfx;
  copy4(a.sq, p.sq); copy4(a.sk, p.sk); copy4(a.sv, p.sv); copy4(a.so, p.so);
  a.causal = p.causal; a.scale = p.scale; a.status = p.status;
  return run_any(a, p.D, p.dtype, false, s);
}

// Small fp16 / bf16 gradients: the longest walk of a block (or of its share of a
// cluster's), times the rounds of blocks, against the three launches of the tensor
// cores' kernels (32 to 62 us).  A step takes 4, 6 and 11 us at D <= 32, 64 and 128.  4
// sequences of 30 rows, 8 heads of 64, 10 prefix keys: 21 us here, 39 there; 3 of 130 rows,
// 4 heads, 200 keys: 54 and 49.
bool prefix_ffma_pays(const BwdParams& p) {
  const Geo& g = p.g;
  Args a{};
  a.g = g; a.pfx = p.pfx;
  const int D = static_cast<int>(p.D);
  const int64_t blocks = bwd_blocks(a, 16), pre = p.pfx.P > 0 ? g.rows_q : 0;
  const int64_t keys = tiles(p.pfx.P, BC) + tiles(g.Nk, BC);
  const int64_t walk = g.G * tiles(pre > g.Nq ? pre : g.Nq, BC), cl = pick_cluster(blocks, keys, 4);
  const int64_t steps = ((walk > keys ? walk : keys) + cl - 1) / cl;
  const int64_t fit = 233472 / (bwd_smem(D, 16) + 1024), slots = device_sm_count() * (fit < 4 ? fit : 4);
  return steps * ((blocks * cl + slots - 1) / slots) <= (D <= 32 ? 6 : 4);
}

fa_status launch_few_keys_delta(const BwdParams& p, float* delta, cudaStream_t s) {
  Args a{};
  a.q = p.q; a.k = p.k; a.v = p.v; a.dout = p.dout; a.lse_in = p.lse; a.delta_out = delta;
  a.g = p.g; a.pfx = p.pfx;
  copy4(a.sq, p.sq); copy4(a.sk, p.sk); copy4(a.sv, p.sv); copy4(a.sdo, p.sdo);
  a.causal = p.causal; a.scale = p.scale; a.status = p.status;
  return p.dtype == FA_F16 ? launch_few_keys<__half>(a, p.D, s) : launch_few_keys<__nv_bfloat16>(a, p.D, s);
}

fa_status launch_bwd_prefix_ffma(const BwdParams& p, cudaStream_t s) {
  Args a{};
  a.q = p.q; a.k = p.k; a.v = p.v; a.dout = p.dout; a.lse_in = p.lse; a.delta = p.delta;
  a.dq = p.dq; a.dk = p.dk; a.dv = p.dv; a.dkp = p.dkp; a.dvp = p.dvp;
  a.g = p.g; a.pfx = p.pfx;
  if (p.pfx.P > 0) a.gp = prefix_geo(p.g, p.pfx.P);
  copy4(a.sq, p.sq); copy4(a.sk, p.sk); copy4(a.sv, p.sv); copy4(a.sdo, p.sdo);
  copy4(a.sdq, p.sdq); copy4(a.sdk, p.sdk); copy4(a.sdv, p.sdv); copy4(a.sdkp, p.sdkp); copy4(a.sdvp, p.sdvp);
  a.causal = p.causal; a.scale = p.scale; a.status = p.status;
  return run_any(a, p.D, p.dtype, true, s);
}

}  // namespace fa
