// Attention of a few new query tokens per request over a prefix that the whole
// batch shares, followed by each request's own cache rows (fp16 / bf16).
//
// Per request b, query head h and token t, with the keys of its key/value
// head: s_j = scale q k_j over all P prefix keys and over the own rows
// j < len_b (causal: j <= len_b - Nq + t), one softmax over both,
//   o = sum_j exp(s_j - L) v_j,   L = log sum_j exp(s_j).
// A softmax splits over sets of keys: each set leaves its normalised o_s and
// its L_s, and  L = log sum_s exp(L_s),  o = sum_s exp(L_s - L) o_s.
//
// Two kernels:
//  * prefix_kernel: the prefix is the same for every request, so the queries
//    of all requests that share a key/value head (B * G * Nq rows) form one
//    matrix and each prefix tile is read once for 128 or 256 of them:
//    S = Q K^T and O += P V on the tensor cores (tcgen05, accumulators in
//    tensor memory), K and V tiles by TMA through a ring.  The prefix is cut
//    into `ns` ranges of key tiles, so that few rows still fill the GPU; each
//    range leaves partial sums in the workspace (fp32).
//  * own_kernel: a request's own rows are read by its G * Nq query rows alone.
//    That is bound by HBM at any rate the matrix units run, so its warps stream K
//    and V through rings in shared memory into m16n8k16 products.  It also joins
//    all partial sums and writes o and L, unless requests with many rows are cut
//    into chunks or the own rows run beside a long prefix (plan_prefix): then
//    its blocks wait for nothing and join_kernel joins.
//
// Rows past a request's length are never read: what they hold does not matter.

#include "tc_common.cuh"

namespace fa {
namespace {

using namespace tc;

// ============================================================================
// The shared prefix
// ============================================================================
// 320 threads: warps 0-3 and 4-7 are two softmax groups, warp 8 the TMA
// producer and owner of the tensor memory, warp 9 issues the products.
//  * two = 1: the groups hold two row tiles (256 rows) and share every K and V
//    tile.  Ring order K_0, V_0, K_1, V_1, ...
//  * two = 0 (at most 128 rows): both groups work on the same rows, group 0 on
//    the even key tiles and group 1 on the odd ones, so that one group's
//    softmax overlaps the other's products; their sums are joined at the end.
//    Ring order K_0, K_1, V_0, K_2, V_1, ...
// Tensor memory: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D);
// P (rounded to the input type, as the forward does) over the first 64 columns
// of its S.
template <int D>
struct PreCfg {
  static constexpr int DC = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = DC * CHUNK;
  static constexpr int NS = 4;                      // ring tiles
  static constexpr int OFF_RING = 2 * TILE;
  // partial sums are staged over the ring: 2 x 128 rows x D fp32
  static constexpr int RING = NS * TILE > 2 * 128 * D * 4 ? NS * TILE : 2 * 128 * D * 4;
  static constexpr int OFF_ML = OFF_RING + RING;    // (m, l) of group 1's rows; at first the rows' places
  static constexpr int OFF_BAR = OFF_ML + 2048;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t COL_S0 = 0, COL_O0 = 256;
};

struct PreArgs {
  const void* q;
  int64_t sq[3];
  int R, GN, Nq, G, Hkv;      // rows per key/value head: R = B * GN, GN = G * Nq
  int dreal;
  int n;                      // key tiles of the prefix
  int lim_last;               // last valid key of the last tile
  int ns, two, groups;        // key ranges; two row tiles per block; row groups
  float c;                    // scale * log2(e)
  float* part_o;              // [Hkv][ns][R][dreal]
  float* part_l;              // [Hkv][ns][R], log2 units
  unsigned int* status;
  uint64_t timeout_ns;
};

template <typename T, int D>
__global__ void __launch_bounds__(320, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ PreArgs a) {
  using C = PreCfg<D>;
  static_assert(C::SMEM <= 232448, "shared memory per block");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::OFF_RING;
  float2* sML = reinterpret_cast<float2*>(smem + C::OFF_ML);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  Ctl* ctl = reinterpret_cast<Ctl*>(bars + 32);
  const uint32_t b_q = smem_u32(&bars[0]);
  const uint32_t b_full0 = smem_u32(&bars[1]);                  // + 8 * slot
  const uint32_t b_empty0 = smem_u32(&bars[1 + C::NS]);         // + 8 * slot
  const uint32_t b_sfull0 = smem_u32(&bars[1 + 2 * C::NS]);     // + 8 * g
  const uint32_t b_pready0 = smem_u32(&bars[3 + 2 * C::NS]);    // + 8 * g
  const uint32_t b_ofinal0 = smem_u32(&bars[5 + 2 * C::NS]);    // + 8 * g
  const uint32_t b_mmadone = smem_u32(&bars[7 + 2 * C::NS]);
  static_assert(8 + 2 * C::NS <= 32, "barriers below the control block");

  // the own rows' kernel may start as blocks of this one leave
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // blocks of one (head, key range) are neighbours: they read the same tiles
  const int rp = static_cast<int>(blockIdx.x % a.groups);
  const int rest = static_cast<int>(blockIdx.x / a.groups);
  const int sp = rest % a.ns, hk = rest / a.ns;
  const int t0 = static_cast<int>(static_cast<int64_t>(a.n) * sp / a.ns);
  const int n = static_cast<int>(static_cast<int64_t>(a.n) * (sp + 1) / a.ns) - t0;  // >= 1
  const bool two = a.two != 0;
  const int row0 = rp * (two ? 256 : 128);
  int nrows[2], steps[2];      // valid rows and key tiles of each group
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int left = a.R - (two ? row0 + 128 * g : row0);
    nrows[g] = left < 0 ? 0 : (left < 128 ? left : 128);
    steps[g] = nrows[g] == 0 ? 0 : (two ? n : (n + 1 - g) / 2);
  }
  const int nload = 2 * n;                     // tiles to load
  // load i of the ring order -> key tile (within the range) and K or V
  auto load_at = [&](int i, int& j, bool& v) {
    if (two) { j = i >> 1; v = i & 1; return; }
    if (i == 0) { j = 0; v = false; return; }
    // K_1, V_0, K_2, V_1, ..., K_{n-1}, V_{n-2}, V_{n-1}
    if (i == nload - 1) { j = n - 1; v = true; return; }
    v = !(i & 1);
    j = v ? i / 2 - 1 : (i + 1) / 2;
  };
  // and back: the ring position of K_j and V_j
  auto at_k = [&](int j) { return two ? 2 * j : (j == 0 ? 0 : 2 * j - 1); };
  auto at_v = [&](int j) { return two ? 2 * j + 1 : (j == n - 1 ? nload - 1 : 2 * j + 2); };
  auto load_tile = [&](int i) {
    int j;
    bool v;
    load_at(i, j, v);
    const int s = i % C::NS;
    mbar_arrive_expect_tx(b_full0 + 8 * s, C::TILE);
    for (int c = 0; c < C::DC; ++c)
      tma_load_4d(smem_u32(sRing + s * C::TILE + c * C::CHUNK), v ? &tmv : &tmk, b_full0 + 8 * s,
                  c * 64, (t0 + j) * 128, hk, 0);
  };
  const int early = nload < C::NS ? nload : C::NS;
  if (warp == 8) {
    if (lane == 0) {
      mbar_init(b_q, 256);
      for (int s = 0; s < C::NS; ++s) {
        mbar_init(b_full0 + 8 * s, 1);
        mbar_init(b_empty0 + 8 * s, 1);
      }
      for (int g = 0; g < 2; ++g) {
        mbar_init(b_sfull0 + 8 * g, 1);
        // only warps that hold valid rows take part in a group's steps
        const int warps = (nrows[g] + 31) / 32;
        mbar_init(b_pready0 + 8 * g, warps ? 32 * warps : 1);
        mbar_init(b_ofinal0 + 8 * g, 1);
      }
      mbar_init(b_mmadone, 1);
      ctl->abort = 0;
      mbar_fence_init();
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmv);
      for (int i = 0; i < early; ++i) load_tile(i);
    }
    __syncwarp();
    tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp < 8) {
    // Query rows gathered into the operand layout of a 128-byte-swizzled load,
    // while warp 8 sets up; columns past a narrow head dimension are zero, rows
    // past R hold whatever was there (their results are not used).  Each thread
    // finds the place of one row, then copies one 16-byte unit of every RPP-th
    // row with all its loads in flight (divisions and loads in turn took 5.7 us
    // for two tiles, a third of a short block).
    constexpr int UN = D / 8, RPP = 256 / UN;         // units per row, rows per pass
    constexpr int PASS = 256 / RPP;                   // passes over two row tiles
    const int nr = nrows[0] + (two ? nrows[1] : 0);
    int* sRow = reinterpret_cast<int*>(smem + C::OFF_ML);     // b and g, t of a row ((m, l) come later)
    if (static_cast<int>(threadIdx.x) < nr) {
      const int row = row0 + static_cast<int>(threadIdx.x), b = row / a.GN, rem = row - b * a.GN;
      const int hg = rem / a.Nq;
      sRow[2 * threadIdx.x] = b;
      sRow[2 * threadIdx.x + 1] = hg * 16 + (rem - hg * a.Nq);          // fewer than 16 tokens
    }
    bar_red_and(1, 256, true);
    const int un = threadIdx.x % UN, rt = threadIdx.x / UN;
    const bool col = 8 * un < a.dreal;
    const T* qh = static_cast<const T*>(a.q) + static_cast<int64_t>(hk) * a.G * a.sq[1] + 8 * un;
    uint4 x[PASS];
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int r = rt + i * RPP;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nr && col) {
        const int2 at = *reinterpret_cast<const int2*>(sRow + 2 * r);
        x[i] = __ldg(reinterpret_cast<const uint4*>(qh + at.x * a.sq[0] + (at.y >> 4) * a.sq[1] +
                                                    (at.y & 15) * a.sq[2]));
      }
    }
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int rr = rt + i * RPP, r = rr & 127;
      if (rr < nr)
        *reinterpret_cast<uint4*>(sQ + (rr >> 7) * C::TILE + (un >> 3) * C::CHUNK + r * 128 +
                                  (((un & 7) ^ (r & 7)) << 4)) = x[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int sent = early;
      for (int i = early; i < nload; ++i) {
        const int s = i % C::NS;
        if (!wait_bounded(b_empty0 + 8 * s, ((i / C::NS) - 1) & 1, ctl, a.status, a.timeout_ns)) break;
        load_tile(i);
        sent = i + 1;
      }
      // Drain: every copy issued has landed before the block may exit.
      for (int i = sent > C::NS ? sent - C::NS : 0; i < sent; ++i)
        wait_bounded(b_full0 + 8 * (i % C::NS), (i / C::NS) & 1, ctl, a.status, a.timeout_ns, false);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idS = idesc_f16<T>(128, 128, false, false);
    const uint32_t idO = idesc_f16<T>(128, D, false, true);
    const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dK0 = sdesc_sw128(smem_u32(sRing), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(smem_u32(sRing), C::CHUNK, 1024);
    auto wait_tile = [&](int i) {
      return wait_warp(b_full0 + 8 * (i % C::NS), (i / C::NS) & 1, ctl, a.status, a.timeout_ns);
    };
    auto free_tile = [&](int i) {
      if (leader) mma_commit(b_empty0 + 8 * (i % C::NS));
    };
    auto issue_S = [&](int g, int i) {       // S_g = Q K^T, K at ring position i
      const uint64_t qa = dQ0 + static_cast<uint64_t>(((two ? g : 0) * C::TILE) >> 4);
      const uint64_t kb = dK0 + static_cast<uint64_t>(((i % C::NS) * C::TILE) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4;
        if (leader) mma_ss(tmem + C::COL_S0 + 128 * g, qa + off, kb + off, idS, kk > 0 ? 1u : 0u);
      }
      if (leader) mma_commit(b_sfull0 + 8 * g);
    };
    auto issue_PV = [&](int g, int i, bool acc) {   // O_g += P V, V at ring position i
      const uint64_t vb = dV0 + static_cast<uint64_t>(((i % C::NS) * C::TILE) >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        if (leader)
          mma_ts(tmem + C::COL_O0 + D * g, tmem + C::COL_S0 + 128 * g + 8 * kk,
                 vb + static_cast<uint64_t>((kk * 2048) >> 4), idO, (acc || kk > 0) ? 1u : 0u);
    };
    bool ok = wait_warp(b_q, 0, ctl, a.status, a.timeout_ns) && wait_tile(0);
    if (ok) {
      tc_fence_after();
      issue_S(0, 0);
      if (two && steps[1] > 0) issue_S(1, 0);
      free_tile(0);
    }
    if (ok && !two && n > 1 && (ok = wait_tile(at_k(1)))) {
      tc_fence_after();
      issue_S(1, at_k(1));
      free_tile(at_k(1));
    }
    for (int j = 0; ok && j < n; ++j) {
      if (two) {
        if (!(ok = wait_tile(at_v(j)))) break;
        const bool next = j + 1 < n;
        if (next && !(ok = wait_tile(at_k(j + 1)))) break;
        for (int g = 0; ok && g < 2; ++g) {
          if (steps[g] == 0) continue;
          if (!(ok = wait_warp(b_pready0 + 8 * g, j & 1, ctl, a.status, a.timeout_ns))) break;
          tc_fence_after();
          issue_PV(g, at_v(j), j > 0);
          if (next) issue_S(g, at_k(j + 1));
          else if (leader) mma_commit(b_ofinal0 + 8 * g);
        }
        if (!ok) break;
        free_tile(at_v(j));
        if (next) free_tile(at_k(j + 1));
      } else {
        const int g = j & 1, jj = j >> 1;
        if (!(ok = wait_tile(at_v(j)))) break;
        if (!(ok = wait_warp(b_pready0 + 8 * g, jj & 1, ctl, a.status, a.timeout_ns))) break;
        tc_fence_after();
        issue_PV(g, at_v(j), jj > 0);
        free_tile(at_v(j));
        if (j + 2 < n) {
          if (!(ok = wait_tile(at_k(j + 2)))) break;
          tc_fence_after();
          issue_S(g, at_k(j + 2));
          free_tile(at_k(j + 2));
        } else if (leader) {
          mma_commit(b_ofinal0 + 8 * g);
        }
      }
    }
    // Drain: every product and commit of this thread is complete.
    if (leader) mma_commit(b_mmadone);
    wait_bounded(b_mmadone, 0, ctl, a.status, a.timeout_ns, false);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    // (the query rows were gathered before the sync)
    fence_async_smem();
    mbar_arrive(b_q);
    const int g = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tS = lane_base + C::COL_S0 + 128 * g;
    const uint32_t tO = lane_base + C::COL_O0 + D * g;
    const float c = a.c;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const bool active = quarter * 32 < nrows[g];      // whole warps
    const int ng = active ? steps[g] : 0;
    for (int j = 0; j < ng; ++j) {
      if (!(ok = wait_warp(b_sfull0 + 8 * g, j & 1, ctl, a.status, a.timeout_ns))) break;
      tc_fence_after();
      float s[128];
      {
        uint32_t r0[32], r1[32], r2[32], r3[32];
        tmem_ld32(tS + 0, r0);
        tmem_ld32(tS + 32, r1);
        tmem_ld32(tS + 64, r2);
        tmem_ld32(tS + 96, r3);
        tmem_wait_ld();
        reg_fence32(r0); reg_fence32(r1); reg_fence32(r2); reg_fence32(r3);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          s[i] = __uint_as_float(r0[i]);
          s[32 + i] = __uint_as_float(r1[i]);
          s[64 + i] = __uint_as_float(r2[i]);
          s[96 + i] = __uint_as_float(r3[i]);
        }
      }
      const int jt = t0 + (two ? j : 2 * j + g);
      if (jt == a.n - 1 && a.lim_last < 127) {         // keys past the prefix
#pragma unroll
        for (int kk = 0; kk < 128; ++kk)
          if (kk > a.lim_last) s[kk] = -INFINITY;
      }
      float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
      for (int kk = 0; kk < 128; kk += 8) {
        m0 = max3f(m0, s[kk], s[kk + 1]);
        m1 = max3f(m1, s[kk + 2], s[kk + 3]);
        m2 = max3f(m2, s[kk + 4], s[kk + 5]);
        m3 = max3f(m3, s[kk + 6], s[kk + 7]);
      }
      const float m_new = fmaxf(m, fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * c);
      // the running maximum moves only when it grows by more than 8 (2^8 in P)
      bool rescale = false;
      float alpha = 1.f;
      if (j == 0) {
        m = m_new;
      } else {
        const bool need = m_new > m + 8.f;
        rescale = __any_sync(0xffffffffu, need);
        if (need) {
          alpha = ex2(m - m_new);
          l *= alpha;
          m = m_new;
        }
      }
      // no finite score yet: exponents against 0, so that -inf stays a weight of 0
      const float ms = m == -INFINITY ? 0.f : m;
      const uint64_t cc = f32x2(c, c), nm = f32x2(-ms, -ms);
      uint64_t acc = f32x2(0.f, 0.f);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x0, x1;
          f32x2_split(fma_f32x2(f32x2(s[64 * hh + 2 * i], s[64 * hh + 2 * i + 1]), cc, nm), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          acc = add_f32x2(acc, f32x2(p0, p1));
          pk[i] = pack2<T>(p0, p1);
        }
        tmem_st32(tS + 32 * hh, pk);
        if (hh == 0 && rescale) {
          // the last P V of this group completed before its S did
#pragma unroll 1
          for (int c4 = 0; c4 < D / 16; ++c4) {
            uint32_t t[16];
            tmem_ld16(tO + 16 * c4, t);
            tmem_wait_ld();
            reg_fence16(t);
#pragma unroll
            for (int i = 0; i < 16; ++i) t[i] = __float_as_uint(__uint_as_float(t[i]) * alpha);
            tmem_st16(tO + 16 * c4, t);
          }
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(b_pready0 + 8 * g);
      float lo, hi;
      f32x2_split(acc, lo, hi);
      l += lo + hi;
    }
    // Every product of both groups is complete (and with them every copy): the
    // ring holds the staged sums now.
    if (steps[0] > 0 && ok) ok = wait_warp(b_ofinal0, 0, ctl, a.status, a.timeout_ns);
    if (steps[1] > 0 && ok) ok = wait_warp(b_ofinal0 + 8, 0, ctl, a.status, a.timeout_ns);
    tc_fence_after();
    // one staged row per thread, 16-byte chunk u of row r at chunk u ^ (r & 7)
    float* srow = reinterpret_cast<float*>(sRing) + (g * 128 + r) * D;
    auto stage = [&](float w0, float w1, const float* other) {
#pragma unroll 1
      for (int c4 = 0; c4 < D / 32; ++c4) {
        uint32_t t[32];
        tmem_ld32(tO + 32 * c4, t);
        tmem_wait_ld();
        reg_fence32(t);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int at = 4 * ((8 * c4 + u) ^ (r & 7));
          float4 x = make_float4(__uint_as_float(t[4 * u]) * w0, __uint_as_float(t[4 * u + 1]) * w0,
                                 __uint_as_float(t[4 * u + 2]) * w0, __uint_as_float(t[4 * u + 3]) * w0);
          if (other) {
            const float4 y = *reinterpret_cast<const float4*>(other + at);
            x.x = fmaf(y.x, w1, x.x); x.y = fmaf(y.y, w1, x.y);
            x.z = fmaf(y.z, w1, x.z); x.w = fmaf(y.w, w1, x.w);
          }
          *reinterpret_cast<float4*>(srow + at) = x;
        }
      }
    };
    const int64_t prow0 = (static_cast<int64_t>(hk) * a.ns + sp) * a.R;
    // group 1 of the same rows hands its sums over unscaled
    if (!two && g == 1) {
      if (ok && active && steps[1] > 0) {
        stage(1.f, 0.f, nullptr);
        sML[r] = make_float2(m, l);
      }
    }
    ok = bar_red_and(1, 256, ok);
    if (ok && active && (two ? steps[g] > 0 : g == 0)) {
      float w0 = 1.f, w1 = 0.f;
      const float* other = nullptr;
      if (!two && steps[1] > 0) {
        const float2 o = sML[r];
        const float mm = fmaxf(m, o.x);
        // a row whose scores are all -inf keeps its maximum at -inf
        w0 = m == -INFINITY ? 0.f : ex2(m - mm);
        w1 = o.x == -INFINITY ? 0.f : ex2(o.x - mm);
        l = l * w0 + o.y * w1;
        m = mm;
        other = reinterpret_cast<const float*>(sRing) + (128 + r) * D;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      stage(w0 * inv, w1 * inv, other);
      if (r < nrows[g])
        a.part_l[prow0 + row0 + (two ? 128 * g : 0) + r] = m + log2f(l);
    }
    if (bar_red_and(1, 256, ok)) {
      // dreal / 4 16-byte units of a partial row (a power of two), eight loads of
      // the staged rows before their stores
      const int sh = 31 - __clz(a.dreal / 4), total = nrows[0] + (two ? nrows[1] : 0);
      float4* dst = reinterpret_cast<float4*>(a.part_o + (prow0 + row0) * a.dreal);
      const int n16 = total << sh;                    // group 0's rows are full when both have some
      for (int i0 = threadIdx.x; i0 < n16; i0 += 8 * 256) {
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int idx = i0 + 256 * i, rr = idx >> sh, un = idx & ((1 << sh) - 1);
          if (idx < n16)
            x[i] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sRing) + rr * D +
                                                    4 * (un ^ (rr & 7)));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + 256 * i < n16) dst[i0 + 256 * i] = x[i];
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================
// Own rows
// ============================================================================
// A block of four warps takes 8 NT query rows of one (request, key/value head)
// and one chunk of the request's rows; warp w takes every fourth block of 16
// keys.  Scores are formed transposed, S^T = K Q^T, and so is the output,
// O^T = V^T P^T: the keys (then the columns of V) fill the 16 rows of the
// m16n8k16 products and the few query rows their 8 columns, so that no half of
// a product is padding for up to eight query rows and the sums take D / 4
// registers per lane and tile.
// Each warp copies its own blocks of keys into a ring in shared memory, ahead of
// its work (cp.async, 512 contiguous bytes per instruction, no barrier between
// warps): what has to be in flight to keep HBM busy, some 100 KB per SM, is more
// than registers hold (loads into the products' registers, half of them empty at
// any time, took 53.9 us where the rings take 45.8).  Blocks that walk several
// requests with their rings running ahead were no faster: the joins between them
// take longer than a ring covers.
// Lane 4 g + c holds, of an operand with rows g and g + 8, the elements in
// slots 2c, 2c+1, 2c+8, 2c+9 of 16.  The order of a contraction is free, so the
// slots of two products over K take the eight elements 8c .. 8c+7 of a
// 32-element piece: one 16-byte read.  Of V the lane holds keys 2c, 2c+1, 2c+8,
// 2c+9; product tile j takes as its rows g and g + 8 the elements 8g + 2j and
// 8g + 2j + 1 of a 64-element piece, so four tiles share one 16-byte read of
// each of the four keys.  P^T comes out of S^T with its halves the other way
// round; movmatrix turns them.  16-byte unit u of row r lies at unit
// u ^ 4 (r mod 2) of its row for K and u ^ 2 (r / 2 mod 4) for V, which spreads
// the eight reads of a quarter of a warp over all banks.
// The block joins its sums with the prefix's and writes o and L, or (apart) leaves
// its sums for join_kernel.
constexpr int kOwnThreads = 128;
constexpr int kOwnWarps = kOwnThreads / 32;
constexpr int kMaxRanges = 64;            // ranges of the prefix
constexpr int kMaxChunks = 64;            // chunks of a request's own rows
constexpr int kMaxSorted = 128;           // requests that a block ranks by length
constexpr int kDeepRows = 1024;           // rows per block above which deep rings pay (OwnCfg)

struct OwnArgs {
  const void* q; const void* k; const void* v;
  void* o;
  float* lse;
  int64_t sq[3], sk[3], sv[3], so[3];
  const int32_t* lens;
  int64_t S;
  int B, Hq, Hkv, G, Nq, GN, RT;     // RT: tiles of 8 NT of the GN rows
  int dreal, causal;
  float c;
  int longest_first;                 // blocks take the requests by falling length
  float len_scale;                   // 2^22 / (S + 1)
  int chunks, chunk;                 // chunks of `chunk` rows (a multiple of 64) per request
  int apart;                         // sums are left for join_kernel
  int ns, R;                         // prefix partial sums (ns = 0: none)
  const float* part_o;               // [Hkv][ns][R][dreal]
  const float* part_l;               // [Hkv][ns][R]
  float* own_o;                      // [Hkv][chunks][R][dreal]; apart
  float* own_l;                      // [Hkv][chunks][R]
  unsigned int* status;
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements, two neighbours of row lane / 4
// per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Sum or maximum over the eight lanes of one c.
__device__ __forceinline__ float max_g(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float sum_g(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// Shared memory of a block: per warp a ring of K | V blocks of 16 rows, over
// which its sums are laid at the end.
// Two shapes.  Deep rings (three blocks of rows, four at D = 64; two blocks of
// threads per SM, three) keep more in flight; shallow ones (one block of rows
// less, one block of threads more) hide more of the blocks' starts and joins.
// Own rows alone, D = 128, 8 heads: 128 requests of up to 1024 rows 56.0 us deep,
// 51.8 shallow; 64 of up to 2048 45.8 and 51.9 (5.9 TB/s of the 6.8 that a copy
// reaches); D = 64, 16 of up to 8192 in chunks 37.5 and 43.7.
template <int D, int NT, bool DEEP>
struct OwnCfg {
  static constexpr int STAGES = (D == 128 ? 3 : 4) - (DEEP ? 0 : 1);
  static constexpr int KV = 16 * D * 2;               // bytes of 16 rows of K or V
  static constexpr int RING = STAGES * 2 * KV;        // per warp
  static constexpr int SMEM = kOwnWarps * RING;
  static constexpr int BLOCKS = (D == 128 ? 3 : 4) - (DEEP || NT == 2 ? 1 : 0);     // per SM
  static_assert(8 * NT * D * 4 <= RING, "a warp's sums fit its ring");
};

template <typename T, int D, int NT, bool DEEP>
__global__ void __launch_bounds__(kOwnThreads, (OwnCfg<D, NT, DEEP>::BLOCKS))
    own_kernel(const __grid_constant__ OwnArgs a) {
  using C = OwnCfg<D, NT, DEEP>;
  constexpr int KP = D / 32;              // 32-element pieces of a K row
  constexpr int VP = D / 64;              // 64-element pieces of a V row
  constexpr int UN = D / 8;               // 16-byte units of a row
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t own_smem[];
  __shared__ float sL[kOwnWarps][ROWS];   // log2 of each warp's sum, -inf: no key
  __shared__ float sW[ROWS][kOwnWarps];
  __shared__ float sP[ROWS][kMaxRanges];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, c4 = lane & 3;
  int id = static_cast<int>(blockIdx.x);
  const int ck = id % a.chunks;
  id /= a.chunks;
  const int rt = id % a.RT;
  id /= a.RT;
  const int hk = id % a.Hkv;
  int b = id / a.Hkv;
  if (a.longest_first) {
    // Blocks start in the order of their index, and a long request that starts
    // last leaves the GPU idle around it.  So block b takes the request of rank b
    // by falling length, which the threads find by counting.  One key holds a
    // length (22 bits of it suffice) and, so that no two are alike, the request.
    __shared__ __align__(16) int sKey[kMaxSorted];
    __shared__ int sB;
    auto key_of = [&](int i) {
      const int n = __ldg(a.lens + i);
      const float f = static_cast<float>(n < 0 ? 0 : n) * a.len_scale;
      return static_cast<int>(f < 4194303.f ? f : 4194303.f) * kMaxSorted + (kMaxSorted - 1 - i);
    };
    static_assert(kMaxSorted == kOwnThreads, "one request per thread");
    const int i = static_cast<int>(threadIdx.x), mine = i < a.B ? key_of(i) : -1;
    sKey[i] = mine;
    __syncthreads();
    if (i < a.B) {
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < a.B; j += 4) {
        const int4 n = *reinterpret_cast<const int4*>(sKey + j);
        before += (n.x > mine) + (n.y > mine) + (n.z > mine) + (n.w > mine);
      }
      if (before == b) sB = i;
    }
    __syncthreads();
    b = sB;
  }
  const int len = a.lens ? __ldg(a.lens + b) : 0;
  const bool bad = len < 0 || len > a.S;
  if (bad && threadIdx.x == 0) record_status(a.status, FA_ERR_SEQLENS);
  const int key_from = ck * a.chunk;
  // Where join_kernel follows, only the last block waits for the prefix kernel, so
  // that the join finds both kernels' sums; the others leave as they end.
  const bool waits = !a.apart || blockIdx.x == gridDim.x - 1;
  if (a.apart) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (bad || (a.apart && key_from >= len)) {           // nothing to leave: join_kernel knows the length
    if (waits) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int key_to = len - key_from < a.chunk ? len : key_from + a.chunk;
  const int r0 = rt * ROWS;
  const int nr = a.GN - r0 < ROWS ? a.GN - r0 : ROWS;      // valid rows

  uint8_t* ring = own_smem + warp * C::RING;
  // This lane's units of a block: unit lane % UN of rows lane / UN, + 32 / UN, ...
  const int un = lane % UN, row_l = lane / UN;
  const bool col = 8 * un < a.dreal;
  const T* kbase = static_cast<const T*>(a.k) + b * a.sk[0] + hk * a.sk[1] + 8 * un;
  const T* vbase = static_cast<const T*>(a.v) + b * a.sv[0] + hk * a.sv[1] + 8 * un;
  const uint32_t ring_s = smem_u32(ring);
  constexpr int STRIDE = 16 * kOwnWarps;
  const int first = key_from + warp * 16;
  auto copy = [&](int key0, int stage) {
    if (key0 < key_to) {
#pragma unroll
      for (int i = 0; i < 16 * UN / 32; ++i) {
        const int r = row_l + i * (32 / UN), key = key0 + r;
        const bool on = col && key < key_to;
        // rows past the length are not read; the copy of 0 bytes fills zeros
        const T* ks = on ? kbase + key * a.sk[2] : kbase;
        const T* vs = on ? vbase + key * a.sv[2] : vbase;
        const uint32_t dst = ring_s + stage * 2 * C::KV + r * (D * 2);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + ((un ^ (4 * (r & 1))) << 4)),
                     "l"(ks), "r"(on ? 16 : 0)
                     : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + C::KV +
                                                                          ((un ^ (2 * ((r >> 1) & 3))) << 4)),
                     "l"(vs), "r"(on ? 16 : 0)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) copy(first + i * STRIDE, i);
  // Query rows as the second operand: row 8 nt + g, the same pieces as K's
  uint4 qr[NT][KP];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = 8 * nt + g8;
    const bool on = row < nr;
    const int gr = r0 + (on ? row : 0), hg = gr / a.Nq, tok = gr - hg * a.Nq;
    const T* q = static_cast<const T*>(a.q) + b * a.sq[0] + static_cast<int64_t>(hk * a.G + hg) * a.sq[1] +
                 tok * a.sq[2] + 8 * c4;
#pragma unroll
    for (int p = 0; p < KP; ++p)
      qr[nt][p] = on && 32 * p + 8 * c4 < a.dreal ? __ldg(reinterpret_cast<const uint4*>(q + 32 * p))
                                                  : make_uint4(0u, 0u, 0u, 0u);
  }
  int lim[NT][2];                          // last own key that query rows 8 nt + 2 c4 + e see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      lim[nt][e] = a.causal ? len - a.Nq + (r0 + 8 * nt + 2 * c4 + e) % a.Nq : len - 1;
  float o[4 * VP][NT][4];
#pragma unroll
  for (int i = 0; i < 4 * VP; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  int stage = 0;
  for (int key0 = first; key0 < key_to; key0 += STRIDE) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
    __syncwarp();                          // every lane's copies; the last block is no longer read
    copy(key0 + (C::STAGES - 1) * STRIDE, stage == 0 ? C::STAGES - 1 : stage - 1);
    const uint8_t* ks = ring + stage * 2 * C::KV;
    const uint8_t* vs = ks + C::KV;
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
    for (int p = 0; p < KP; ++p) {
      const int at = ((4 * p + c4) ^ (4 * (g8 & 1))) << 4;      // rows g and g + 8 swap alike
      const uint4 k0 = *reinterpret_cast<const uint4*>(ks + g8 * (D * 2) + at);
      const uint4 k1 = *reinterpret_cast<const uint4*>(ks + (g8 + 8) * (D * 2) + at);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16816<T>(s[nt], k0.x, k1.x, k0.y, k1.y, qr[nt][p].x, qr[nt][p].y);
        mma16816<T>(s[nt], k0.z, k1.z, k0.w, k1.w, qr[nt][p].z, qr[nt][p].w);
      }
    }
    uint32_t pb[NT][2];
    float alpha[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[2][2];                       // key g8 + 8 t, query row 2 c4 + e
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int key = key0 + 8 * t + g8;
          x[t] = key <= lim[nt][e] && key < key_to ? s[nt][2 * t + e] * a.c : -INFINITY;
        }
        const float mn = fmaxf(m[nt][e], max_g(fmaxf(x[0], x[1])));
        // no key seen yet: exponents against 0, so that -inf stays a weight of 0
        const float ms = mn == -INFINITY ? 0.f : mn;
        alpha[nt][e] = ex2(m[nt][e] - ms);
        moved |= mn != m[nt][e];
        m[nt][e] = mn;
        p[0][e] = ex2(x[0] - ms);
        p[1][e] = ex2(x[1] - ms);
        l[nt][e] = fmaf(l[nt][e], alpha[nt][e], p[0][e] + p[1][e]);
      }
      // P rounded to the input type for the product, as the forward does
      pb[nt][0] = transpose8x8(pack2<T>(p[0][0], p[0][1]));
      pb[nt][1] = transpose8x8(pack2<T>(p[1][0], p[1][1]));
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < 4 * VP; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[i][nt][0] *= alpha[nt][0];
          o[i][nt][1] *= alpha[nt][1];
          o[i][nt][2] *= alpha[nt][0];
          o[i][nt][3] *= alpha[nt][1];
        }
    }
#pragma unroll
    for (int p = 0; p < VP; ++p) {
      uint4 vr[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {        // keys 2 c4 + {0, 1} + {0, 8}: r / 2 mod 4 = c4
        const int r = 2 * c4 + (t & 1) + 8 * (t >> 1);
        vr[t] = *reinterpret_cast<const uint4*>(vs + r * (D * 2) + (((8 * p + g8) ^ (2 * c4)) << 4));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v0 = word(vr[0], j), v1 = word(vr[1], j), v2 = word(vr[2], j), v3 = word(vr[3], j);
        const uint32_t a0 = prmt(v0, v1, 0x5410u), a1 = prmt(v0, v1, 0x7632u),
                       a2 = prmt(v2, v3, 0x5410u), a3 = prmt(v2, v3, 0x7632u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816<T>(o[4 * p + j][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();                            // the ring is done with: the warp's sums go over it
  float* sO = reinterpret_cast<float*>(ring);             // [ROWS][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ls = sum_g(l[nt][e]);
      const int row = 8 * nt + 2 * c4 + e;
      const bool none = m[nt][e] == -INFINITY && ls == 0.f;      // no key seen
      const float inv = none ? 0.f : 1.f / ls;
      if (g8 == 0) sL[warp][row] = none ? -INFINITY : m[nt][e] + log2f(ls);
#pragma unroll
      for (int p = 0; p < VP; ++p) {
        float4* dst = reinterpret_cast<float4*>(sO + row * D + 64 * p + 8 * g8);
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          dst[j / 2] = make_float4(o[4 * p + j][nt][e] * inv, o[4 * p + j][nt][2 + e] * inv,
                                   o[4 * p + j + 1][nt][e] * inv, o[4 * p + j + 1][nt][2 + e] * inv);
      }
    }
  __syncthreads();
  // the prefix's partial sums are complete and visible from here on (unless apart)
  if (waits) asm volatile("griddepcontrol.wait;" ::: "memory");

  // Per row, the weights of the four warps' sums and, without a join to follow, of
  // the prefix's; warp w takes rows w, w + 4, ...
  const int ns = a.apart ? 0 : a.ns;
  const int64_t prow = static_cast<int64_t>(b) * a.GN + r0;    // row within the head's R rows
  const float* pl = a.part_l + static_cast<int64_t>(hk) * a.ns * a.R + prow;
  const int64_t orow = (static_cast<int64_t>(hk) * a.chunks + ck) * a.R + prow;
  for (int row = warp; row < nr; row += kOwnWarps) {
    const float own = lane < kOwnWarps ? sL[lane][row] : -INFINITY;
    float pre[kMaxRanges / 32];            // ranges lane, lane + 32 of the prefix
    float mx = own;
#pragma unroll
    for (int i = 0; i < kMaxRanges / 32; ++i) {
      const int rg = lane + 32 * i;
      pre[i] = rg < ns ? __ldg(pl + static_cast<int64_t>(rg) * a.R + row) : -INFINITY;
      mx = fmaxf(mx, pre[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float ms = mx == -INFINITY ? 0.f : mx;
    float sum = ex2(own - ms);
#pragma unroll
    for (int i = 0; i < kMaxRanges / 32; ++i) sum += ex2(pre[i] - ms);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float L2 = mx == -INFINITY ? -INFINITY : ms + log2f(sum);
    const float Lw = mx == -INFINITY ? 0.f : L2;
    if (lane < kOwnWarps) sW[row][lane] = ex2(own - Lw);
#pragma unroll
    for (int i = 0; i < kMaxRanges / 32; ++i)
      if (lane + 32 * i < ns) sP[row][lane + 32 * i] = ex2(pre[i] - Lw);
    if (lane == 0) {
      if (a.apart) {
        a.own_l[orow + row] = L2;
      } else {
        const int gr = r0 + row, hg = gr / a.Nq, tok = gr - hg * a.Nq;
        a.lse[(static_cast<int64_t>(b) * a.Hq + hk * a.G + hg) * a.Nq + tok] = L2 * kLn2;
      }
    }
  }
  __syncthreads();
  const int units = a.dreal / 4;
  for (int idx = threadIdx.x; idx < nr * units; idx += kOwnThreads) {
    const int row = idx / units, u4 = idx - row * units;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4& x) {
      acc.x = fmaf(w, x.x, acc.x); acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z); acc.w = fmaf(w, x.w, acc.w);
    };
    const float* po = a.part_o + (static_cast<int64_t>(hk) * a.ns * a.R + prow + row) * a.dreal + 4 * u4;
    const int64_t step = static_cast<int64_t>(a.R) * a.dreal;
    int i = 0;
    for (; i + 8 <= ns; i += 8) {            // eight loads in flight
      float4 x[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) x[t] = __ldg(reinterpret_cast<const float4*>(po + (i + t) * step));
#pragma unroll
      for (int t = 0; t < 8; ++t) add(sP[row][i + t], x[t]);
    }
    for (; i < ns; ++i) add(sP[row][i], __ldg(reinterpret_cast<const float4*>(po + i * step)));
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w)
      add(sW[row][w], *reinterpret_cast<const float4*>(own_smem + w * C::RING + (row * D + 4 * u4) * 4));
    if (a.apart) {
      *reinterpret_cast<float4*>(a.own_o + (orow + row) * a.dreal + 4 * u4) = acc;
    } else {
      const int gr = r0 + row, hg = gr / a.Nq, tok = gr - hg * a.Nq;
      T* dst = static_cast<T*>(a.o) + b * a.so[0] + static_cast<int64_t>(hk * a.G + hg) * a.so[1] +
               tok * a.so[2] + 4 * u4;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
    }
  }
}

// ============================================================================
// The join
// ============================================================================
// One warp per output row: the log-sum-exps of all its pieces (prefix ranges,
// then the chunks that the request's length reaches) give their weights, then
// the lanes add the pieces' sums, dreal / 4 lanes to a piece.
template <typename T>
__global__ void __launch_bounds__(kOwnThreads) join_kernel(const __grid_constant__ OwnArgs a) {
  constexpr int PIECES = kMaxRanges + kMaxChunks;
  __shared__ float sW[kOwnWarps][PIECES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kOwnWarps + warp;   // of Hkv * R
  if (row >= static_cast<int64_t>(a.Hkv) * a.R) return;
  const int hk = static_cast<int>(row / a.R), r = static_cast<int>(row - static_cast<int64_t>(hk) * a.R);
  const int b = r / a.GN, gr = r - b * a.GN, hg = gr / a.Nq, tok = gr - hg * a.Nq;
  const int len = __ldg(a.lens + b);
  if (len < 0 || len > a.S) return;          // reported by own_kernel
  const int nc = len / a.chunk + (len % a.chunk != 0), n = a.ns + nc;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the sums of both kernels
  auto piece_l = [&](int i) {
    return i < a.ns ? a.part_l[(static_cast<int64_t>(hk) * a.ns + i) * a.R + r]
                    : a.own_l[(static_cast<int64_t>(hk) * a.chunks + i - a.ns) * a.R + r];
  };
  float L[PIECES / 32], mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < PIECES / 32; ++i) {
    L[i] = lane + 32 * i < n ? piece_l(lane + 32 * i) : -INFINITY;
    mx = fmaxf(mx, L[i]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  const float ms = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < PIECES / 32; ++i) sum += ex2(L[i] - ms);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const float L2 = mx == -INFINITY ? -INFINITY : ms + log2f(sum), Lw = mx == -INFINITY ? 0.f : L2;
#pragma unroll
  for (int i = 0; i < PIECES / 32; ++i)
    if (lane + 32 * i < n) sW[warp][lane + 32 * i] = ex2(L[i] - Lw);
  __syncwarp();
  const int lpp = a.dreal / 4, grp = lane / lpp, col = lane % lpp, ngrp = 32 / lpp;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = grp; i < n; i += ngrp) {
    const float* src = i < a.ns ? a.part_o + ((static_cast<int64_t>(hk) * a.ns + i) * a.R + r) * a.dreal
                                : a.own_o + ((static_cast<int64_t>(hk) * a.chunks + i - a.ns) * a.R + r) * a.dreal;
    const float4 x = *reinterpret_cast<const float4*>(src + 4 * col);
    const float w = sW[warp][i];
    acc.x = fmaf(w, x.x, acc.x); acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z); acc.w = fmaf(w, x.w, acc.w);
  }
  for (int off = lpp; off < 32; off <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
  }
  const int64_t h = hk * a.G + hg;
  if (grp == 0) {
    T* dst = static_cast<T*>(a.o) + b * a.so[0] + h * a.so[1] + tok * a.so[2] + 4 * col;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
  }
  if (lane == 0) a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Nq + tok] = L2 * kLn2;
}

// ----------------------------------------------------------------- host side
// SMs the split of the prefix is planned for: every GB300 has 152, and the
// workspace's size must not depend on a device.
constexpr int kPlanSMs = 152;

// How the own rows are cut: into chunks of 512 rows at least, as long as that
// gives SMs without a block one, since several chunks cost a further kernel (4 us
// and more).  4 requests of up to 32768 rows, 8 heads: 65 us in chunks, 80 when a
// cluster of eight blocks joined its sums through distributed shared memory.
void plan_own(int64_t base, int64_t D, int64_t S, DecodePlan* pl) {
  const int64_t slots = static_cast<int64_t>(kPlanSMs) * (D == 128 ? 2 : 3);
  int64_t c = 1;
  while (c < kMaxChunks && base * c < slots && S / (2 * c) >= 512) c *= 2;
  pl->chunk = ((S + c - 1) / c + 63) / 64 * 64;
  if (pl->chunk < 64) pl->chunk = 64;
  pl->chunks = static_cast<int>(S > 0 ? (S + pl->chunk - 1) / pl->chunk : 1);
  pl->apart = pl->chunks > 1;
}

// How the prefix is cut, and whether the own rows run beside it.  A block costs
// a start and an end plus a time per key tile, its products' or that of reading
// the tiles of all blocks at once; the ranges' partial sums cost their way through
// the L2 cache in proportion to their number (microseconds; a trace of the blocks
// gave 10 to 12 beside their tiles).  Either
//  * the prefix takes all SMs, the own rows follow and join everything, or
//  * (apart) the prefix takes part of the SMs, and the own rows, which HBM bounds
//    and not the SMs, run on the others in the meantime; join_kernel follows (8
//    us with its launch, unless chunks need it anyway).
// The cheaper by that estimate, with requests half as long as S.  8 heads of 128,
// cold, in us: 128 requests of up to 1024 rows behind 16384 keys 92 and 81 apart,
// 64 requests 65 and 54, 128 behind 4096 keys 72 and 69; 32 requests of up to 512
// rows behind 8192 keys 29 and 38.
void plan_prefix(int64_t B, int64_t R, int64_t Hkv, int64_t D, int64_t P, int64_t S, DecodePlan* pl) {
  const int64_t n = (P + 127) / 128;
  pl->two = R > 128;
  pl->groups = pl->two ? (R + 255) / 256 : 1;
  const int64_t base = Hkv * pl->groups;
  const double products = (D > 64 ? 1.5 : 1.0) * (pl->two ? 1.0 : 0.53), fixed = 11.0, hbm = 6.2e6;
  const double join = static_cast<double>(R) * static_cast<double>(Hkv * D) * 8 / 10e6;  // per range
  const double own = static_cast<double>(B * Hkv) * static_cast<double>(S) / 2 * static_cast<double>(4 * D) / hbm;
  const bool chunked = pl->chunks > 1;
  double best = 0;
  const int64_t most = n < kMaxRanges ? n : kMaxRanges;
  for (int64_t ns = 1; ns <= most; ++ns) {
    const int64_t blocks = base * ns;
    const double waves = static_cast<double>((blocks + kPlanSMs - 1) / kPlanSMs);
    const double once = static_cast<double>(blocks < kPlanSMs ? blocks : kPlanSMs);
    const double reads = once / static_cast<double>(pl->groups) * static_cast<double>(128 * 4 * D) / hbm;
    const double tiles = static_cast<double>((n + ns - 1) / ns);
    const double pre = waves * (fixed + (reads > products ? reads : products) * tiles);
    const double joins = join * static_cast<double>(ns);
    double t = pre + own + joins;
    int apart = chunked;
    if (S > 0 && blocks < kPlanSMs) {
      // what the SMs left draw of HBM's rate, each a third more than its share at
      // most, and what the prefix leaves of it; at D <= 64 blocks of both kernels fit
      // one SM and slow each other
      const double mixed = D > 64 ? products : 2 * products, per_tile = reads > mixed ? reads : mixed;
      const double share = 1.3 * static_cast<double>(kPlanSMs - blocks) / kPlanSMs, rest = 1.0 - reads / per_tile;
      const double pre_b = fixed + per_tile * tiles;
      const double left = own - pre_b * (share < rest ? share : rest);
      const double beside = pre_b + (left > 0 ? left : 0.0) + joins + (chunked ? 0.0 : 8.0);
      if (chunked || beside < t) {
        t = beside;
        apart = 1;
      }
    }
    if (ns == 1 || t < best) {
      best = t;
      pl->ns = static_cast<int>(ns);
      pl->apart = apart;
    }
  }
}

// Query rows of a block of own_kernel: 8, or 16 where a request has more.
int own_rows(int64_t GN) { return GN <= 8 ? 8 : 16; }

template <typename T, int D>
fa_status run_decode(const DecodeParams& p, cudaStream_t stream) {
  const int64_t GN = p.G * p.Nq, R = p.B * GN;
  const DecodePlan& pl = p.plan;
  float* part_o = p.ws;
  float* part_l = part_o + static_cast<int64_t>(pl.ns) * p.Hkv * R * p.D;
  // the log-sum-exps take whole 16-byte units, so that the sums behind them stay aligned
  const int64_t nl = (static_cast<int64_t>(pl.ns) * p.Hkv * R + 3) / 4 * 4;
  float* own_o = part_l + nl;
  float* own_l = own_o + static_cast<int64_t>(pl.chunks) * p.Hkv * R * p.D;
  if (pl.ns > 0) {
    CUtensorMap mk, mv;
    if (!encode_tile_map(&mk, p.kp, p.dtype, 1, p.Hkv, p.P, p.D, p.skp, 128, 64) ||
        !encode_tile_map(&mv, p.vp, p.dtype, 1, p.Hkv, p.P, p.D, p.svp, 128, 64))
      return FA_ERR_LAUNCH;
    PreArgs a{};
    a.q = p.q;
    for (int i = 0; i < 3; ++i) a.sq[i] = p.sq[i];
    a.R = static_cast<int>(R); a.GN = static_cast<int>(GN); a.Nq = static_cast<int>(p.Nq);
    a.G = static_cast<int>(p.G); a.Hkv = static_cast<int>(p.Hkv);
    a.dreal = static_cast<int>(p.D);
    a.n = static_cast<int>((p.P + 127) / 128);
    a.lim_last = static_cast<int>((p.P - 1) % 128);
    a.ns = pl.ns; a.two = pl.two; a.groups = static_cast<int>(pl.groups);
    a.c = p.scale * kLog2e;
    a.part_o = part_o; a.part_l = part_l;
    a.status = p.status; a.timeout_ns = p.timeout_ns;
    auto kern = prefix_kernel<T, D>;
    FA_CONFIGURE((prefix_kernel<T, D>), PreCfg<D>::SMEM);
    const int64_t blocks = p.Hkv * pl.groups * pl.ns;
    if (blocks > 0x7fffffffLL) return FA_ERR_SHAPE;
    kern<<<dim3(static_cast<unsigned>(blocks)), dim3(320), PreCfg<D>::SMEM, stream>>>(mk, mv, a);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  }
  OwnArgs a{};
  a.q = p.q; a.k = p.k; a.v = p.v; a.o = p.o; a.lse = p.lse;
  for (int i = 0; i < 3; ++i) {
    a.sq[i] = p.sq[i]; a.sk[i] = p.sk[i]; a.sv[i] = p.sv[i]; a.so[i] = p.so[i];
  }
  a.lens = p.S > 0 ? p.lens : nullptr;
  a.S = p.S;
  a.B = static_cast<int>(p.B); a.Hq = static_cast<int>(p.Hkv * p.G); a.Hkv = static_cast<int>(p.Hkv);
  a.G = static_cast<int>(p.G); a.Nq = static_cast<int>(p.Nq); a.GN = static_cast<int>(GN);
  const int rows = own_rows(GN);
  a.RT = static_cast<int>((GN + rows - 1) / rows);
  a.dreal = static_cast<int>(p.D); a.causal = p.causal;
  a.c = p.scale * kLog2e;
  a.chunks = pl.chunks; a.chunk = static_cast<int>(pl.chunk); a.apart = pl.apart;
  a.ns = pl.ns; a.R = static_cast<int>(R);
  a.part_o = part_o; a.part_l = part_l; a.own_o = own_o; a.own_l = own_l;
  a.status = p.status;
  const int64_t base = p.B * p.Hkv * a.RT, blocks = base * pl.chunks;
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * OwnCfg<D, 1, true>::BLOCKS;
  a.len_scale = 4194304.f / static_cast<float>(p.S + 1);
  // Ranking costs every round of blocks a start, and gains the end of the last long
  // request: few rounds of long blocks.  8 heads of 128, ranked / not, in us: 64
  // requests of up to 2048 rows 47 / 54, 96 of 1024 39 / 44, 128 of 1024 52 / 55, 48 of
  // 700 25 / 27, 128 of 512 37 / 33, 256 of 1024 111 / 89; 16 heads of 64, 128 of 1024
  // 56 / 51.
  a.longest_first = p.B > 1 && p.B <= kMaxSorted && pl.chunks == 1 && base > slots &&
                    base * (256 * 128) <= slots * p.S * D;
  if (blocks > 0x7fffffffLL) return FA_ERR_SHAPE;
  // The own rows need nothing of the prefix kernel until their sums are joined,
  // where every block waits for it (griddepcontrol.wait): the blocks start on
  // SMs that the prefix kernel has left.  Without that kernel before it the
  // launch is an ordinary one.
  const auto launch = [&](auto kern, int64_t grid, int smem, bool overlap) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kOwnThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess && cudaGetLastError() == cudaSuccess;
  };
  bool ok;
#define FA_OWN(NT, DEEP)                                                                  \
  do {                                                                                    \
    FA_CONFIGURE((own_kernel<T, D, NT, DEEP>), (OwnCfg<D, NT, DEEP>::SMEM));              \
    ok = launch(own_kernel<T, D, NT, DEEP>, blocks, OwnCfg<D, NT, DEEP>::SMEM, pl.ns > 0); \
  } while (0)
  const bool deep = pl.chunk > kDeepRows || blocks <= slots;
  if (rows == 8) {
    if (deep) FA_OWN(1, true);
    else FA_OWN(1, false);
  } else {
    if (deep) FA_OWN(2, true);
    else FA_OWN(2, false);
  }
#undef FA_OWN
  if (ok && pl.apart) ok = launch(join_kernel<T>, (p.Hkv * R + kOwnWarps - 1) / kOwnWarps, 0, true);
  return ok ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace

DecodePlan decode_plan(int64_t B, int64_t Hkv, int64_t GN, int64_t D, int64_t P, int64_t S) {
  DecodePlan pl{};
  const int rows = own_rows(GN);
  plan_own(B * Hkv * ((GN + rows - 1) / rows), D, S, &pl);
  if (P > 0) plan_prefix(B, B * GN, Hkv, D, P, S, &pl);
  // per range, chunk and query row: D sums and a log-sum-exp
  const int64_t R = Hkv * B * GN, own = pl.apart ? pl.chunks * R * (D + 1) : 0;
  pl.floats = pl.ns * R * D + (pl.ns * R + 3) / 4 * 4 + own;
  return pl;
}

fa_status launch_decode(const DecodeParams& p, cudaStream_t s) {
  if (p.dtype == FA_BF16)
    return p.D == 128 ? run_decode<__nv_bfloat16, 128>(p, s) : run_decode<__nv_bfloat16, 64>(p, s);
  if (p.dtype == FA_F16)
    return p.D == 128 ? run_decode<__half, 128>(p, s) : run_decode<__half, 64>(p, s);
  return FA_ERR_DTYPE;
}

}  // namespace fa
