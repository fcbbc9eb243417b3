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
//    That is bound by HBM at any rate the matrix units run, so its warps load
//    K and V straight into the registers of m16n8k16 products, 16 bytes per
//    lane and whole 64- or 128-byte pieces per row, without shared memory, and
//    sixteen warps per SM keep the loads in flight.  A cluster of up to eight
//    blocks shares one request's rows when there are few requests.  The same
//    kernel then joins all partial sums and writes o and L.
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
  static constexpr int OFF_ML = OFF_RING + RING;    // (m, l) of group 1's rows
  static constexpr int OFF_BAR = OFF_ML + 1024;
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
    // past R hold whatever was there (their results are not used).  A thread
    // takes one 16-byte unit of every RPP-th row, all its loads at once (with a
    // division and a load per piece in turn the gather took 10 us of a block):
    // it finds the place of the rows by one division each, shared by the warp.
    constexpr int UN = D / 8, RPP = 256 / UN;         // units per row, rows per pass
    constexpr int PASS = 128 / RPP;                   // passes over one row tile
    const int nr = nrows[0] + (two ? nrows[1] : 0);
    const int un = threadIdx.x % UN, rt = threadIdx.x / UN;
    const bool col = 8 * un < a.dreal;
    const T* qh = static_cast<const T*>(a.q) + static_cast<int64_t>(hk) * a.G * a.sq[1] + 8 * un;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      if (tile == 1 && !two) break;
      uint4 x[PASS];
#pragma unroll
      for (int i = 0; i < PASS; ++i) {
        const int rr = 128 * tile + rt + i * RPP, row = row0 + rr;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (rr < nr && col) {
          const int b = row / a.GN, rem = row - b * a.GN, hg = rem / a.Nq, tok = rem - hg * a.Nq;
          x[i] = __ldg(reinterpret_cast<const uint4*>(qh + b * a.sq[0] + hg * a.sq[1] + tok * a.sq[2]));
        }
      }
#pragma unroll
      for (int i = 0; i < PASS; ++i) {
        const int r = rt + i * RPP;
        if (128 * tile + r < nr)
          *reinterpret_cast<uint4*>(sQ + tile * C::TILE + (un >> 3) * C::CHUNK + r * 128 +
                                    (((un & 7) ^ (r & 7)) << 4)) = x[i];
      }
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
      const uint64_t cc = f32x2(c, c), nm = f32x2(-m, -m);
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
      const float inv = 1.f / l;
      stage(w0 * inv, w1 * inv, other);
      if (r < nrows[g])
        a.part_l[prow0 + row0 + (two ? 128 * g : 0) + r] = m + log2f(l);
    }
    if (bar_red_and(1, 256, ok)) {
      const int units = a.dreal / 4;                  // 16-byte units of a partial row
      const int total = nrows[0] + (two ? nrows[1] : 0);   // group 0's rows are full when both have some
#pragma unroll 4
      for (int idx = threadIdx.x; idx < total * units; idx += 256) {
        const int rr = idx / units, un = idx - rr * units;
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sRing) +
                                                          rr * D + 4 * (un ^ (rr & 7)));
        *reinterpret_cast<float4*>(a.part_o + (prow0 + row0 + rr) * a.dreal + 4 * un) = x;
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
// Own rows, and the join
// ============================================================================
// A block of four warps takes 8 NT query rows of one (request, key/value
// head); warp w of block `rank` of the cluster takes every (4 * cluster)-th
// block of 16 keys.  Scores are formed transposed, S^T = K Q^T, and so is the
// output, O^T = V^T P^T: the keys (then the columns of V) fill the 16 rows of
// the m16n8k16 products and the few query rows their 8 columns, so that no
// half of a product is padding for up to eight query rows and the sums take
// D / 4 registers per lane and tile.
// Lane 4 g + c holds, of an operand with rows g and g + 8, the elements in
// slots 2c, 2c+1, 2c+8, 2c+9 of 16.  The order of a contraction is free, so the
// slots of two products over K take the eight elements 8c .. 8c+7 of a
// 32-element piece: one 16-byte load.  Of V the lane holds keys 2c, 2c+1, 2c+8,
// 2c+9; product tile j takes as its rows g and g + 8 the elements 8g + 2j and
// 8g + 2j + 1 of a 64-element piece, so four tiles share one 16-byte load of
// each of the four keys.  P^T comes out of S^T with its halves the other way
// round; movmatrix turns them.
constexpr int kOwnThreads = 128;
constexpr int kOwnWarps = kOwnThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxRanges = 64;            // ranges of the prefix
constexpr int kMaxSorted = 256;           // requests that a block ranks by length

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
  int cluster;
  int longest_first;                 // blocks take the requests by falling length
  int ns, R;                         // prefix partial sums (ns = 0: none)
  const float* part_o;
  const float* part_l;
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

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  return __ldcs(static_cast<const uint4*>(p));
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

// Blocks per SM that the registers are kept to.
constexpr int own_blocks(int D, int NT) {
  return D == 64 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 3 : 2);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kOwnThreads, own_blocks(D, NT))
    own_kernel(const __grid_constant__ OwnArgs a) {
  constexpr int KP = D / 32;              // 32-element pieces of a K row
  constexpr int VP = D / 64;              // 64-element pieces of a V row
  constexpr int ROWS = 8 * NT;
  __shared__ __align__(16) float sO[kOwnWarps][ROWS][D];
  __shared__ float sL[kOwnWarps][ROWS];   // log2 of each warp's sum, -inf: no key
  __shared__ float sW[ROWS][kOwnWarps * kMaxCluster];
  __shared__ float sP[ROWS][kMaxRanges];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, c4 = lane & 3;
  const int rank = static_cast<int>(blockIdx.x % a.cluster);
  int id = static_cast<int>(blockIdx.x / a.cluster);
  const int rt = id % a.RT;
  id /= a.RT;
  const int hk = id % a.Hkv;
  int b = id / a.Hkv;
  if (a.longest_first) {
    // Blocks start in the order of their index, and a long request that starts
    // last leaves the GPU idle around it (a fifth of the time at 128 requests of
    // 1 to 1024 rows).  So block b takes the request of rank b by falling
    // length, which the threads find by counting.
    __shared__ __align__(16) int sLen[kMaxSorted];
    __shared__ int sB;
    for (int i = threadIdx.x; i < kMaxSorted; i += kOwnThreads)
      sLen[i] = i < a.B ? __ldg(a.lens + i) : INT32_MIN;     // counts before nobody
    __syncthreads();
    for (int i = threadIdx.x; i < a.B; i += kOwnThreads) {
      const int mine = sLen[i];
      int before = 0;
#pragma unroll 4
      for (int j = 0; j < a.B; j += 4) {
        const int4 n = *reinterpret_cast<const int4*>(sLen + j);
        // of equal lengths the lower index comes first
        before += (n.x > mine || (n.x == mine && j < i)) + (n.y > mine || (n.y == mine && j + 1 < i)) +
                  (n.z > mine || (n.z == mine && j + 2 < i)) + (n.w > mine || (n.w == mine && j + 3 < i));
      }
      if (before == b) sB = i;
    }
    __syncthreads();
    b = sB;
  }
  const int len = a.lens ? __ldg(a.lens + b) : 0;
  if (len < 0 || len > a.S) {             // every block of the cluster takes this
    if (threadIdx.x == 0) record_status(a.status, FA_ERR_SEQLENS);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int r0 = rt * ROWS;
  const int nr = a.GN - r0 < ROWS ? a.GN - r0 : ROWS;      // valid rows

  const T* kbase = static_cast<const T*>(a.k) + b * a.sk[0] + hk * a.sk[1] + 8 * c4;
  const T* vbase = static_cast<const T*>(a.v) + b * a.sv[0] + hk * a.sv[1] + 8 * g8;
  const int stride = 16 * kOwnWarps * a.cluster;
  uint4 kr[2][KP], vr[4][VP];
  auto load_k = [&](int key0) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int key = key0 + 8 * t + g8;
      const T* row = kbase + key * a.sk[2];
#pragma unroll
      for (int p = 0; p < KP; ++p)
        kr[t][p] = key < len && 32 * p + 8 * c4 < a.dreal ? ld_stream(row + 32 * p)
                                                          : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto load_v = [&](int key0) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int key = key0 + 2 * c4 + (t & 1) + 8 * (t >> 1);
      const T* row = vbase + key * a.sv[2];
#pragma unroll
      for (int p = 0; p < VP; ++p)
        vr[t][p] = key < len && 64 * p + 8 * g8 < a.dreal ? ld_stream(row + 64 * p)
                                                          : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  const int first = (rank * kOwnWarps + warp) * 16;
  if (first < len) load_k(first);
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

  for (int key0 = first; key0 < len; key0 += stride) {
    load_v(key0);
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        mma16816<T>(s[nt], kr[0][p].x, kr[1][p].x, kr[0][p].y, kr[1][p].y, qr[nt][p].x, qr[nt][p].y);
        mma16816<T>(s[nt], kr[0][p].z, kr[1][p].z, kr[0][p].w, kr[1][p].w, qr[nt][p].z, qr[nt][p].w);
      }
    }
    if (key0 < len - stride) load_k(key0 + stride);
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
        for (int t = 0; t < 2; ++t)
          x[t] = key0 + 8 * t + g8 <= lim[nt][e] ? s[nt][2 * t + e] * a.c : -INFINITY;
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
    for (int p = 0; p < VP; ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v0 = word(vr[0][p], j), v1 = word(vr[1][p], j), v2 = word(vr[2][p], j),
                       v3 = word(vr[3][p], j);
        const uint32_t a0 = prmt(v0, v1, 0x5410u), a1 = prmt(v0, v1, 0x7632u),
                       a2 = prmt(v2, v3, 0x5410u), a3 = prmt(v2, v3, 0x7632u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816<T>(o[4 * p + j][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
  }
  // This warp's sums, normalised, with log2 of the sum of exponentials
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
        float4* dst = reinterpret_cast<float4*>(&sO[warp][row][64 * p + 8 * g8]);
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          dst[j / 2] = make_float4(o[4 * p + j][nt][e] * inv, o[4 * p + j][nt][2 + e] * inv,
                                   o[4 * p + j + 1][nt][e] * inv, o[4 * p + j + 1][nt][2 + e] * inv);
      }
    }
  if (a.cluster > 1) cluster_sync_all();
  else __syncthreads();
  // the prefix's partial sums are complete and visible from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // Join: per row, the weights of every piece; warp w takes rows w, w + 4, ...
  const int pieces = kOwnWarps * a.cluster;
  const int64_t prow = static_cast<int64_t>(b) * a.GN + r0;    // row within the head's R rows
  const float* pl = a.part_l + static_cast<int64_t>(hk) * a.ns * a.R + prow;
  for (int row = warp; row < nr; row += kOwnWarps) {
    float own = -INFINITY;                 // piece `lane` of the own rows (at most 32)
    if (lane < pieces) {
      const uint32_t at = smem_u32(&sL[lane % kOwnWarps][row]);
      if (a.cluster > 1)
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(own) : "r"(cluster_map(at, static_cast<uint32_t>(lane / kOwnWarps))) : "memory");
      else
        own = sL[lane][row];
    }
    float pre[kMaxRanges / 32];            // ranges lane, lane + 32 of the prefix
    float mx = own;
#pragma unroll
    for (int i = 0; i < kMaxRanges / 32; ++i) {
      const int rg = lane + 32 * i;
      pre[i] = rg < a.ns ? __ldg(pl + static_cast<int64_t>(rg) * a.R + row) : -INFINITY;
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
    if (lane < pieces) sW[row][lane] = ex2(own - Lw);
#pragma unroll
    for (int i = 0; i < kMaxRanges / 32; ++i)
      if (lane + 32 * i < a.ns) sP[row][lane + 32 * i] = ex2(pre[i] - Lw);
    if (lane == 0 && rank == 0) {
      const int gr = r0 + row, hg = gr / a.Nq, tok = gr - hg * a.Nq;
      a.lse[(static_cast<int64_t>(b) * a.Hq + hk * a.G + hg) * a.Nq + tok] = L2 * kLn2;
    }
  }
  __syncthreads();
  const int units = a.dreal / 4;
  for (int idx = threadIdx.x + kOwnThreads * rank; idx < nr * units; idx += kOwnThreads * a.cluster) {
    const int row = idx / units, un = idx - row * units;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4& x) {
      acc.x = fmaf(w, x.x, acc.x); acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z); acc.w = fmaf(w, x.w, acc.w);
    };
    const float* po = a.part_o + (static_cast<int64_t>(hk) * a.ns * a.R + prow + row) * a.dreal + 4 * un;
    const int64_t step = static_cast<int64_t>(a.R) * a.dreal;
    int i = 0;
    for (; i + 8 <= a.ns; i += 8) {          // eight loads in flight
      float4 x[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) x[t] = __ldg(reinterpret_cast<const float4*>(po + (i + t) * step));
#pragma unroll
      for (int t = 0; t < 8; ++t) add(sP[row][i + t], x[t]);
    }
    for (; i < a.ns; ++i) add(sP[row][i], __ldg(reinterpret_cast<const float4*>(po + i * step)));
    for (int rk = 0; rk < a.cluster; ++rk)
#pragma unroll
      for (int w = 0; w < kOwnWarps; ++w) {
        const float4 x = a.cluster > 1
                             ? ld_cluster_f4(cluster_map(smem_u32(&sO[w][row][4 * un]), static_cast<uint32_t>(rk)))
                             : *reinterpret_cast<const float4*>(&sO[w][row][4 * un]);
        add(sW[row][rk * kOwnWarps + w], x);
      }
    const int gr = r0 + row, hg = gr / a.Nq, tok = gr - hg * a.Nq;
    T* dst = static_cast<T*>(a.o) + b * a.so[0] + static_cast<int64_t>(hk * a.G + hg) * a.so[1] +
             tok * a.so[2] + 4 * un;
    uint2 w2;
    w2.x = pack2<T>(acc.x, acc.y);
    w2.y = pack2<T>(acc.z, acc.w);
    *reinterpret_cast<uint2*>(dst) = w2;
  }
  // no block leaves while another still reads its shared memory
  if (a.cluster > 1) cluster_sync_all();
}

// ----------------------------------------------------------------- host side
// SMs the split of the prefix is planned for: every GB300 has 152, and the
// workspace's size must not depend on a device.
constexpr int kPlanSMs = 152;

// How the prefix is cut.  A block costs a start and an end plus a time per key
// tile; the ranges' partial sums cost their way through the L2 cache in
// proportion to their number.  The cheapest number of ranges by that estimate.
PrefixPlan make_plan(int64_t B, int64_t Hkv, int64_t GN, int64_t D, int64_t P) {
  PrefixPlan pl{};
  if (P < 1) return pl;
  const int64_t R = B * GN, n = (P + 127) / 128;
  pl.two = R > 128;
  pl.groups = pl.two ? (R + 255) / 256 : 1;
  const int64_t base = Hkv * pl.groups;
  const double per_tile = D > 64 ? 1.5 : 0.8, fixed = 5.0;      // microseconds
  const double join = static_cast<double>(R) * Hkv * D * 8 / 10e6;  // per range
  double best = 0;
  const int64_t most = n < kMaxRanges ? n : kMaxRanges;
  for (int64_t ns = 1; ns <= most; ++ns) {
    const double waves = static_cast<double>((base * ns + kPlanSMs - 1) / kPlanSMs);
    const double t = waves * (fixed + per_tile * static_cast<double>((n + ns - 1) / ns)) + join * ns;
    if (ns == 1 || t < best) {
      best = t;
      pl.ns = static_cast<int>(ns);
    }
  }
  return pl;
}

template <typename T, int D>
fa_status run_decode(const DecodeParams& p, cudaStream_t stream) {
  const int64_t GN = p.G * p.Nq, R = p.B * GN;
  const PrefixPlan pl = make_plan(p.B, p.Hkv, GN, p.D, p.P);
  float* part_o = p.ws;
  float* part_l = p.ws + static_cast<int64_t>(pl.ns) * p.Hkv * R * p.D;
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
  const int NT = GN <= 8 ? 1 : 2;
  a.RT = static_cast<int>((GN + 8 * NT - 1) / (8 * NT));
  a.dreal = static_cast<int>(p.D); a.causal = p.causal;
  a.c = p.scale * kLog2e;
  a.ns = pl.ns; a.R = static_cast<int>(R);
  a.part_o = part_o; a.part_l = part_l;
  a.status = p.status;
  const int64_t base = p.B * p.Hkv * a.RT;
  // blocks of a cluster: as many as stay resident together, while each warp
  // keeps at least two blocks of 16 keys of the longest request allowed
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * own_blocks(D, NT);
  int cl = 1;
  while (cl < kMaxCluster && 2 * base * cl <= slots && p.S >= 2 * 16 * kOwnWarps * 2 * cl) cl *= 2;
  a.cluster = cl;
  a.longest_first = p.S > 0 && base * cl > slots && p.B > 1 && p.B <= kMaxSorted;
  const int64_t blocks = base * cl;
  if (blocks > 0x7fffffffLL) return FA_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kOwnThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (cl > 1) {
    cudaLaunchAttribute& at = attr[cfg.numAttrs++];
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(cl);
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
  }
  if (pl.ns > 0) {
    // The own rows need nothing of the prefix kernel until the join, where
    // every block waits for it (griddepcontrol.wait): its blocks start on SMs
    // that the prefix kernel has left.  Without that kernel before it the
    // launch is an ordinary one.
    cudaLaunchAttribute& at = attr[cfg.numAttrs++];
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
  }
  auto kern = NT == 1 ? own_kernel<T, D, 1> : own_kernel<T, D, 2>;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return FA_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace

PrefixPlan decode_plan(int64_t B, int64_t Hkv, int64_t GN, int64_t D, int64_t P) {
  return make_plan(B, Hkv, GN, D, P);
}

fa_status launch_decode(const DecodeParams& p, cudaStream_t s) {
  if (p.dtype == FA_BF16)
    return p.D == 128 ? run_decode<__nv_bfloat16, 128>(p, s) : run_decode<__nv_bfloat16, 64>(p, s);
  if (p.dtype == FA_F16)
    return p.D == 128 ? run_decode<__half, 128>(p, s) : run_decode<__half, 64>(p, s);
  return FA_ERR_DTYPE;
}

}  // namespace fa
