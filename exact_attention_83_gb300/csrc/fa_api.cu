// The C ABI of libfa: argument validation, per-device set-up and dispatch.
//
// Nothing here computes attention; every step of the path runs in the kernels
// of the other translation units.  Validation happens before any launch, so an
// invalid call returns its fa_status without touching the device.

#include "fa_internal.h"

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

// Device status word of the current context.  A kernel whose bounded wait
// runs out stores FA_ERR_TIMEOUT here (first writer wins);
// fa_get_device_status reads and clears it.  A file-scope device variable, so
// the library allocates no device memory.
__device__ unsigned int fa_device_status_word;

namespace fa {
namespace {

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;

std::atomic<int> g_path{FA_PATH_AUTO};
std::atomic<uint64_t> g_timeout_ns{kDefaultTimeoutNs};
std::mutex g_mu;
cudaEvent_t g_prof_events[3];
std::atomic<bool> g_prof_on{false};
std::atomic<int> g_withhold_next{0};   // one-shot test switch (fa_test_withhold_next_arrival)
std::atomic<int64_t> g_l2_override{0};  // test switch (fa_test_set_l2_bytes)
struct DeviceInfo {
  int state = 0;              // 0: not set up, 1: ready, -1: not sm_103
  int sm_count = 0;
  int64_t l2_bytes = 0;
  unsigned int* status = nullptr;
};
DeviceInfo g_dev[kMaxDevices];

// Once per device, with that device current: check the architecture, cache
// the SM count and the device address of the status word.
fa_status device_setup(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_LAUNCH;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (d.state == 0) {
    int major = 0, minor = 0, sms = 0, l2 = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev) != cudaSuccess)
      return FA_ERR_LAUNCH;
    if (major != 10 || minor != 3) {
      d.state = -1;
    } else {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, fa_device_status_word) != cudaSuccess) return FA_ERR_LAUNCH;
      d.status = static_cast<unsigned int*>(p);
      d.sm_count = sms;
      d.l2_bytes = l2;
      d.state = 1;
    }
  }
  if (d.state < 0) return FA_ERR_ARCH;
  *out = &d;
  return FA_OK;
}

#define FA_TRY(expr)                   \
  do {                                 \
    const fa_status st_ = (expr);      \
    if (st_ != FA_OK) return st_;      \
  } while (0)

int64_t elem_size(fa_dtype dt) { return dt == FA_F32 ? 4 : 2; }

bool mul_ok(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }

fa_status check_shape(int64_t B, int64_t H, int64_t N, int64_t D, fa_dtype dt) {
  if (dt != FA_F32 && dt != FA_F16 && dt != FA_BF16) return FA_ERR_DTYPE;
  if (B < 1 || H < 1 || N < 1) return FA_ERR_SHAPE;
  if (D != 16 && D != 32 && D != 64 && D != 128) return FA_ERR_HEADDIM;
  int64_t bh, bhn, bhnd;
  if (!mul_ok(B, H, &bh) || !mul_ok(bh, N, &bhn) || !mul_ok(bhn, D * 8, &bhnd)) return FA_ERR_SHAPE;
  if (bh > (int64_t)INT32_MAX || N > (int64_t)INT32_MAX) return FA_ERR_SHAPE;
  return FA_OK;
}

// Checks one [B,H,N,D] tensor and copies its strides into dst.  The stride of
// a dimension of extent 1 is never used; it is replaced by 0.
fa_status check_tensor(const void* p, const int64_t* s, int64_t B, int64_t H, int64_t N,
                       fa_dtype dt, int64_t* dst) {
  if (!p || !s) return FA_ERR_NULL;
  if (s[3] != 1) return FA_ERR_STRIDE;
  const int64_t ext[3] = {B, H, N};
  const int64_t es = elem_size(dt);
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return FA_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) { dst[i] = 0; continue; }
    if (s[i] < 0) return FA_ERR_STRIDE;
    int64_t bytes;
    if (!mul_ok(s[i], es, &bytes)) return FA_ERR_SHAPE;
    if (bytes % 16 != 0) return FA_ERR_ALIGN;
    dst[i] = s[i];
  }
  dst[3] = 1;
  return FA_OK;
}

fa_status check_f32_vec(const void* p) {
  if (!p) return FA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return FA_ERR_ALIGN;
  return FA_OK;
}

// check_tensor for the entry points that also refuse a stride of 0 (a
// broadcast dimension): a tensor map cannot carry one, and rows of an output
// would fall on one another.
fa_status check_dense(const void* p, const int64_t* s, int64_t B, int64_t H, int64_t N,
                      fa_dtype dt, int64_t* dst) {
  FA_TRY(check_tensor(p, s, B, H, N, dt, dst));
  const int64_t ext[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (ext[i] > 1 && s[i] == 0) return FA_ERR_STRIDE;
  return FA_OK;
}

fa_status check_scale(float scale) {
  return (std::isfinite(scale) && scale > 0.f) ? FA_OK : FA_ERR_SCALE;
}

bool use_tc(fa_dtype dt) { return g_path.load() == FA_PATH_AUTO && dt != FA_F32; }

// A validated fa_problem.
struct Problem {
  Geo g;
  int64_t D;
  int causal;
  float scale;
  fa_dtype dtype;
  Dropout drop;
};

fa_status check_problem(const fa_problem* pr, Problem* out) {
  if (!pr) return FA_ERR_NULL;
  const fa_dtype dt = pr->dtype;
  if (dt != FA_F32 && dt != FA_F16 && dt != FA_BF16) return FA_ERR_DTYPE;
  if (pr->B < 1 || pr->Hq < 1 || pr->Hkv < 1 || pr->Nq < 1 || pr->Nk < 1) return FA_ERR_SHAPE;
  if (pr->Hq % pr->Hkv != 0) return FA_ERR_SHAPE;
  const int64_t D = pr->D;
  if (D != 16 && D != 32 && D != 64 && D != 128) return FA_ERR_HEADDIM;
  const bool packed = pr->cu_seqlens_q != nullptr;
  if (packed != (pr->cu_seqlens_k != nullptr)) return FA_ERR_SHAPE;
  if (packed && (pr->total_q < 1 || pr->total_k < 1)) return FA_ERR_SHAPE;
  if (packed && (reinterpret_cast<uintptr_t>(pr->cu_seqlens_q) % 4 != 0 ||
                 reinterpret_cast<uintptr_t>(pr->cu_seqlens_k) % 4 != 0))
    return FA_ERR_ALIGN;
  Geo g{};
  g.B = pr->B; g.Hq = pr->Hq; g.Hkv = pr->Hkv; g.G = pr->Hq / pr->Hkv;
  g.Nq = pr->Nq; g.Nk = pr->Nk;
  g.cu_q = pr->cu_seqlens_q; g.cu_k = pr->cu_seqlens_k;
  g.rows_q = packed ? pr->total_q : pr->Nq;
  g.rows_k = packed ? pr->total_k : pr->Nk;
  g.Bt = packed ? 1 : pr->B;
  // Every element count, and the int32 quantities the kernels use (flat head
  // index, row positions, grid sizes), must fit.
  int64_t t;
  const int64_t heads[2] = {g.Hq, g.Hkv}, rows[2] = {g.rows_q, g.rows_k};
  for (int i = 0; i < 2; ++i)
    if (!mul_ok(g.Bt, heads[i], &t) || !mul_ok(t, rows[i], &t) || !mul_ok(t, D * 8, &t))
      return FA_ERR_SHAPE;
  if (!mul_ok(g.B, g.Hq, &t) || t > (int64_t)INT32_MAX) return FA_ERR_SHAPE;
  // TMA row coordinates are int32 and run up to one tile past the last row.
  const int64_t row_max = (int64_t)INT32_MAX - 1024;
  if (g.rows_q > row_max || g.rows_k > row_max || g.Nq > row_max || g.Nk > row_max)
    return FA_ERR_SHAPE;
  FA_TRY(check_scale(pr->scale));
  const float p = pr->dropout_p;
  if (!(p >= 0.f && p < 1.f)) return FA_ERR_ARG;
  Dropout d{};
  if (p > 0.f) {
    d.on = 1;
    const double thr = std::floor(static_cast<double>(p) * 65536.0);
    d.thr = static_cast<uint32_t>(thr < 65535.0 ? thr : 65535.0);
    d.rscale = static_cast<float>(1.0 / (1.0 - static_cast<double>(p)));
    d.key0 = static_cast<uint32_t>(pr->seed & 0xffffffffu);
    d.key1 = static_cast<uint32_t>(pr->seed >> 32);
    d.offset = pr->offset;
    for (int r = 0; r < 10; ++r) {   // Philox4x32 key schedule (Weyl increments)
      d.rk0[r] = d.key0 + static_cast<uint32_t>(r) * 0x9E3779B9u;
      d.rk1[r] = d.key1 + static_cast<uint32_t>(r) * 0xBB67AE85u;
    }
    if (pr->dropout_mask) {
      if (reinterpret_cast<uintptr_t>(pr->dropout_mask) % 16 != 0) return FA_ERR_ALIGN;
      if (dropout_mask_bytes(g) == 0) return FA_ERR_SHAPE;
      d.mask = pr->dropout_mask;
      d.mask_kt = (g.Nk + 127) / 128;
    }
  }
  out->g = g; out->D = D; out->causal = pr->causal ? 1 : 0; out->scale = pr->scale;
  out->dtype = dt; out->drop = d;
  return FA_OK;
}

fa_status run_fwd(const Problem& pb, const void* q, const int64_t* sq, const void* k,
                  const int64_t* sk, const void* v, const int64_t* sv, void* o,
                  const int64_t* so, float* lse, cudaStream_t stream, const Prefix* pfx = nullptr) {
  FwdParams p{};
  const Geo& g = pb.g;
  if (pfx) p.pfx = *pfx;
  FA_TRY(check_tensor(q, sq, g.Bt, g.Hq, g.rows_q, pb.dtype, p.sq));
  FA_TRY(check_tensor(k, sk, g.Bt, g.Hkv, g.rows_k, pb.dtype, p.sk));
  FA_TRY(check_tensor(v, sv, g.Bt, g.Hkv, g.rows_k, pb.dtype, p.sv));
  FA_TRY(check_tensor(o, so, g.Bt, g.Hq, g.rows_q, pb.dtype, p.so));
  FA_TRY(check_f32_vec(lse));
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
  p.g = g; p.D = pb.D;
  p.causal = pb.causal; p.scale = pb.scale; p.dtype = pb.dtype; p.drop = pb.drop;
  p.status = dev->status; p.timeout_ns = g_timeout_ns.load();
  if (use_tc(pb.dtype) && have_fwd_tc(pb.D, pb.dtype)) {
    p.withhold_arrival = g_withhold_next.exchange(0);
    return launch_fwd_tc(p, stream);   // stores the keep mask as it draws it
  }
  if (p.pfx.on) return launch_fwd_prefix_ffma(p, stream);
  FA_TRY(launch_fwd_ffma(p, stream));
  // the FFMA forward draws inline and stores nothing: fill the caller's keep
  // mask for the backward
  if (p.drop.on && p.drop.mask != nullptr)
    return launch_dropout_mask(g, pb.causal, p.drop, p.drop.mask, p.status, stream);
  return FA_OK;
}

// Validates the backward's tensors and fills p (everything but the path).
fa_status prepare_bwd(const Problem& pb, const void* q, const int64_t* sq, const void* k,
                      const int64_t* sk, const void* v, const int64_t* sv, const void* dout,
                      const int64_t* sdo, const float* lse, const float* delta, void* dq,
                      const int64_t* sdq, void* dk, const int64_t* sdk, void* dv,
                      const int64_t* sdv, BwdParams* out) {
  BwdParams& p = *out;
  p = BwdParams{};
  const Geo& g = pb.g;
  FA_TRY(check_tensor(q, sq, g.Bt, g.Hq, g.rows_q, pb.dtype, p.sq));
  FA_TRY(check_tensor(k, sk, g.Bt, g.Hkv, g.rows_k, pb.dtype, p.sk));
  FA_TRY(check_tensor(v, sv, g.Bt, g.Hkv, g.rows_k, pb.dtype, p.sv));
  FA_TRY(check_tensor(dout, sdo, g.Bt, g.Hq, g.rows_q, pb.dtype, p.sdo));
  FA_TRY(check_tensor(dq, sdq, g.Bt, g.Hq, g.rows_q, pb.dtype, p.sdq));
  FA_TRY(check_tensor(dk, sdk, g.Bt, g.Hkv, g.rows_k, pb.dtype, p.sdk));
  FA_TRY(check_tensor(dv, sdv, g.Bt, g.Hkv, g.rows_k, pb.dtype, p.sdv));
  FA_TRY(check_f32_vec(lse));
  FA_TRY(check_f32_vec(delta));
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.q = q; p.k = k; p.v = v; p.dout = dout; p.lse = lse; p.delta = delta;
  p.dq = dq; p.dk = dk; p.dv = dv;
  p.g = g; p.D = pb.D;
  p.causal = pb.causal; p.scale = pb.scale; p.dtype = pb.dtype; p.drop = pb.drop;
  p.status = dev->status; p.timeout_ns = g_timeout_ns.load();
  p.prof = g_prof_on.load() ? g_prof_events : nullptr;
  return FA_OK;
}

fa_status run_bwd(const Problem& pb, const void* q, const int64_t* sq, const void* k,
                  const int64_t* sk, const void* v, const int64_t* sv, const void* dout,
                  const int64_t* sdo, const float* lse, const float* delta, void* dq,
                  const int64_t* sdq, void* dk, const int64_t* sdk, void* dv,
                  const int64_t* sdv, cudaStream_t stream, bool allow_side = true) {
  BwdParams p{};
  FA_TRY(prepare_bwd(pb, q, sq, k, sk, v, sv, dout, sdo, lse, delta, dq, sdq, dk, sdk, dv, sdv,
                     &p));
  p.allow_side = allow_side;
  if (use_tc(pb.dtype) && have_bwd_tc(pb.D, pb.dtype)) return launch_bwd_tc(p, stream);
  return launch_bwd_ffma(p, stream);
}

// fa_problem of the square, equal-heads, fixed-length, no-dropout entry points.
fa_problem square_problem(int64_t B, int64_t H, int64_t N, int64_t D, int causal, float scale,
                          fa_dtype dtype) {
  fa_problem pr{};
  pr.B = B; pr.Hq = H; pr.Hkv = H; pr.Nq = N; pr.Nk = N; pr.D = D;
  pr.causal = causal; pr.scale = scale; pr.dtype = dtype;
  return pr;
}

}  // namespace

fa_status validate_square_bwd(const void* q, const void* k, const void* v, const void* o,
                              const void* dout, const float* lse, const void* dq,
                              const void* dk, const void* dv, int64_t B, int64_t H, int64_t N,
                              int64_t D, const int64_t* sq, const int64_t* sk,
                              const int64_t* sv, const int64_t* so, const int64_t* sdo,
                              const int64_t* sdq, const int64_t* sdk, const int64_t* sdv,
                              int causal, float scale, fa_dtype dtype) {
  FA_TRY(check_shape(B, H, N, D, dtype));
  const fa_problem pr = square_problem(B, H, N, D, causal, scale, dtype);
  Problem pb{};
  FA_TRY(check_problem(&pr, &pb));
  int64_t st[4];
  const void* tensors[8] = {q, k, v, o, dout, dq, dk, dv};
  const int64_t* strides[8] = {sq, sk, sv, so, sdo, sdq, sdk, sdv};
  for (int i = 0; i < 8; ++i) FA_TRY(check_tensor(tensors[i], strides[i], B, H, N, dtype, st));
  return check_f32_vec(lse);
}

int device_sm_count() {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < kMaxDevices && g_dev[dev].state == 1) return g_dev[dev].sm_count;
  int sms = 0;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

bool configure_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  const uint64_t bit = 1ull << dev;
  if (done->load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return false;
  done->fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Side stream of each device, for a kernel that may overlap the caller's
// stream (the backward's dQ kernel beside its dK/dV kernel).  One fork/join
// at a time per device: the lock is held from side_begin to side_end, so two
// host threads never interleave the records of the shared events.
struct SideStream {
  std::mutex mu;
  cudaStream_t s = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};
SideStream g_side[kMaxDevices];

fa_status side_begin(cudaStream_t caller, cudaStream_t* side) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_LAUNCH;
  SideStream& ss = g_side[dev];
  ss.mu.lock();
  if (ss.s == nullptr) {
    cudaStream_t st = nullptr;
    cudaEvent_t f = nullptr, j = nullptr;
    if (cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&f, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&j, cudaEventDisableTiming) != cudaSuccess) {
      if (j) cudaEventDestroy(j);
      if (f) cudaEventDestroy(f);
      if (st) cudaStreamDestroy(st);
      ss.mu.unlock();
      return FA_ERR_LAUNCH;
    }
    ss.s = st; ss.fork = f; ss.join = j;
  }
  if (cudaEventRecord(ss.fork, caller) != cudaSuccess ||
      cudaStreamWaitEvent(ss.s, ss.fork, 0) != cudaSuccess) {
    ss.mu.unlock();
    return FA_ERR_LAUNCH;
  }
  *side = ss.s;
  return FA_OK;
}

fa_status side_end(cudaStream_t caller) {
  int dev = 0;
  cudaGetDevice(&dev);
  SideStream& ss = g_side[dev];
  const bool ok = cudaEventRecord(ss.join, ss.s) == cudaSuccess &&
                  cudaStreamWaitEvent(caller, ss.join, 0) == cudaSuccess;
  ss.mu.unlock();
  return ok ? FA_OK : FA_ERR_LAUNCH;
}

bool stream_capturing(cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {
    cudaGetLastError();          // clear the error; treat as capturing
    return true;
  }
  return cs != cudaStreamCaptureStatusNone;
}

int64_t head_group(int64_t BH, int64_t per_head_bytes) {
  int dev = 0;
  cudaGetDevice(&dev);
  int64_t l2 = 0;
  if (dev >= 0 && dev < kMaxDevices && g_dev[dev].state == 1) {
    l2 = g_dev[dev].l2_bytes;
  } else {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrL2CacheSize, dev);
    l2 = v;
  }
  const int64_t forced = g_l2_override.load();
  if (forced > 0) l2 = forced;
  // All heads at once when their operands fit in L2 together (the order is
  // then the plain longest-first one); otherwise groups of 3/8 of L2.
  if (per_head_bytes <= 0 || BH * per_head_bytes <= l2 * 3 / 4) return BH;
  const int64_t g = l2 * 3 / 8 / per_head_bytes;
  return g < 1 ? 1 : (g > BH ? BH : g);
}

fa_status bwd_square(const void* q, const void* k, const void* v, const void* dout,
                     const float* lse, const float* delta, void* dq, void* dk, void* dv,
                     int64_t B, int64_t H, int64_t N, int64_t D, const int64_t* sq,
                     const int64_t* sk, const int64_t* sv, const int64_t* sdo,
                     const int64_t* sdq, const int64_t* sdk, const int64_t* sdv, int causal,
                     float scale, fa_dtype dtype, cudaStream_t stream, bool allow_side) {
  FA_TRY(check_shape(B, H, N, D, dtype));
  const fa_problem pr = square_problem(B, H, N, D, causal, scale, dtype);
  Problem pb{};
  FA_TRY(check_problem(&pr, &pb));
  return run_bwd(pb, q, sq, k, sk, v, sv, dout, sdo, lse, delta, dq, sdq, dk, sdk, dv, sdv,
                 stream, allow_side);
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int64_t B, int64_t H, int64_t N, int64_t D,
                 const int64_t* sq, const int64_t* sk, const int64_t* sv,
                 const int64_t* so, int causal, float scale, fa_dtype dtype,
                 cudaStream_t stream) {
  FA_TRY(check_shape(B, H, N, D, dtype));
  const fa_problem pr = square_problem(B, H, N, D, causal, scale, dtype);
  Problem pb{};
  FA_TRY(check_problem(&pr, &pb));
  return run_fwd(pb, q, sq, k, sk, v, sv, o, so, lse, stream);
}

fa_status fa_fwd_ex(const fa_problem* prob, const void* q, const int64_t* sq, const void* k,
                    const int64_t* sk, const void* v, const int64_t* sv, void* o,
                    const int64_t* so, float* lse, cudaStream_t stream) {
  Problem pb{};
  FA_TRY(check_problem(prob, &pb));
  return run_fwd(pb, q, sq, k, sk, v, sv, o, so, lse, stream);
}

fa_status fa_bwd_preprocess(const void* o, const void* dout, float* delta,
                            int64_t B, int64_t H, int64_t N, int64_t D,
                            const int64_t* so, const int64_t* sdo, fa_dtype dtype,
                            cudaStream_t stream) {
  PreParams p{};
  FA_TRY(check_shape(B, H, N, D, dtype));
  FA_TRY(check_tensor(o, so, B, H, N, dtype, p.so));
  FA_TRY(check_tensor(dout, sdo, B, H, N, dtype, p.sdo));
  FA_TRY(check_f32_vec(delta));
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.o = o; p.dout = dout; p.delta = delta;
  p.B = B; p.H = H; p.N = N; p.D = D; p.dtype = dtype;
  return launch_preprocess(p, stream);
}


fa_status fa_bwd(const void* q, const void* k, const void* v, const void* dout,
                 const float* lse, const float* delta, void* dq, void* dk, void* dv,
                 int64_t B, int64_t H, int64_t N, int64_t D,
                 const int64_t* sq, const int64_t* sk, const int64_t* sv,
                 const int64_t* sdo, const int64_t* sdq, const int64_t* sdk,
                 const int64_t* sdv, int causal, float scale, fa_dtype dtype,
                 cudaStream_t stream) {
  return bwd_square(q, k, v, dout, lse, delta, dq, dk, dv, B, H, N, D, sq, sk, sv, sdo, sdq,
                    sdk, sdv, causal, scale, dtype, stream, true);
}

fa_status fa_bwd_ex(const fa_problem* prob, const void* q, const int64_t* sq, const void* k,
                    const int64_t* sk, const void* v, const int64_t* sv, const void* dout,
                    const int64_t* sdo, const float* lse, const float* delta, void* dq,
                    const int64_t* sdq, void* dk, const int64_t* sdk, void* dv,
                    const int64_t* sdv, cudaStream_t stream) {
  Problem pb{};
  FA_TRY(check_problem(prob, &pb));
  return run_bwd(pb, q, sq, k, sk, v, sv, dout, sdo, lse, delta, dq, sdq, dk, sdk, dv, sdv,
                 stream);
}

// The problem and the prefix of a prefix entry point.
static fa_status check_prefix(const fa_problem* prob, int64_t P, const void* kp, const int64_t* skp,
                              const void* vp, const int64_t* svp, Problem* pb, Prefix* pfx) {
  FA_TRY(check_problem(prob, pb));
  if (!pb->g.cu_q) return FA_ERR_SHAPE;             // packed sequences only
  if (pb->drop.on) return FA_ERR_ARG;
  const int64_t row_max = (int64_t)INT32_MAX - 1024;
  int64_t t;
  if (P < 0 || P > row_max || !mul_ok(pb->g.Hkv, P, &t) || !mul_ok(t, pb->D * 8, &t))
    return FA_ERR_SHAPE;
  // tiles of both key sets are counted in one int, rows in int32
  if (P + pb->g.Nk > row_max) return FA_ERR_SHAPE;
  *pfx = Prefix{};
  pfx->on = true;
  pfx->P = P;
  if (P > 0) {
    pfx->k = kp; pfx->v = vp;
    FA_TRY(check_dense(kp, skp, 1, pb->g.Hkv, P, pb->dtype, pfx->sk));
    FA_TRY(check_dense(vp, svp, 1, pb->g.Hkv, P, pb->dtype, pfx->sv));
  }
  return FA_OK;
}

fa_status fa_fwd_prefix(const fa_problem* prob, int64_t P, const void* q, const int64_t* sq,
                        const void* k_prefix, const int64_t* skp, const void* v_prefix,
                        const int64_t* svp, const void* k, const int64_t* sk, const void* v,
                        const int64_t* sv, void* o, const int64_t* so, float* lse,
                        cudaStream_t stream) {
  Problem pb{};
  Prefix pfx{};
  FA_TRY(check_prefix(prob, P, k_prefix, skp, v_prefix, svp, &pb, &pfx));
  int64_t st[4];
  const Geo& g = pb.g;
  FA_TRY(check_dense(q, sq, 1, g.Hq, g.rows_q, pb.dtype, st));
  FA_TRY(check_dense(k, sk, 1, g.Hkv, g.rows_k, pb.dtype, st));
  FA_TRY(check_dense(v, sv, 1, g.Hkv, g.rows_k, pb.dtype, st));
  FA_TRY(check_dense(o, so, 1, g.Hq, g.rows_q, pb.dtype, st));
  return run_fwd(pb, q, sq, k, sk, v, sv, o, so, lse, stream, &pfx);
}

fa_status fa_bwd_prefix(const fa_problem* prob, int64_t P, const void* q, const int64_t* sq,
                        const void* k_prefix, const int64_t* skp, const void* v_prefix,
                        const int64_t* svp, const void* k, const int64_t* sk, const void* v,
                        const int64_t* sv, const void* dout, const int64_t* sdo, const float* lse,
                        const float* delta, void* dq, const int64_t* sdq, void* dk_prefix,
                        const int64_t* sdkp, void* dv_prefix, const int64_t* sdvp, void* dk,
                        const int64_t* sdk, void* dv, const int64_t* sdv, cudaStream_t stream) {
  Problem pb{};
  BwdParams p{};
  Prefix pfx{};
  FA_TRY(check_prefix(prob, P, k_prefix, skp, v_prefix, svp, &pb, &pfx));
  const Geo& g = pb.g;
  int64_t st[4];
  FA_TRY(check_dense(q, sq, 1, g.Hq, g.rows_q, pb.dtype, st));
  FA_TRY(check_dense(dout, sdo, 1, g.Hq, g.rows_q, pb.dtype, st));
  FA_TRY(check_dense(dq, sdq, 1, g.Hq, g.rows_q, pb.dtype, st));
  const void* own[4] = {k, v, dk, dv};
  const int64_t* sown[4] = {sk, sv, sdk, sdv};
  for (int i = 0; i < 4; ++i) FA_TRY(check_dense(own[i], sown[i], 1, g.Hkv, g.rows_k, pb.dtype, st));
  int64_t sdkp4[4] = {}, sdvp4[4] = {};
  if (P > 0) {
    FA_TRY(check_dense(dk_prefix, sdkp, 1, g.Hkv, P, pb.dtype, sdkp4));
    FA_TRY(check_dense(dv_prefix, sdvp, 1, g.Hkv, P, pb.dtype, sdvp4));
  }
  FA_TRY(prepare_bwd(pb, q, sq, k, sk, v, sv, dout, sdo, lse, delta, dq, sdq, dk, sdk, dv, sdv, &p));
  p.pfx = pfx;
  p.dkp = dk_prefix; p.dvp = dv_prefix;
  for (int i = 0; i < 4; ++i) { p.sdkp[i] = sdkp4[i]; p.sdvp[i] = sdvp4[i]; }
  p.prof = nullptr;
  if (use_tc(pb.dtype) && have_bwd_tc(pb.D, pb.dtype) && !prefix_ffma_pays(p)) return launch_bwd_tc(p, stream);
  return launch_bwd_prefix_ffma(p, stream);
}

fa_status fa_bwd_prefix_delta(const fa_problem* prob, int64_t P, const void* q, const int64_t* sq,
                              const void* k_prefix, const int64_t* skp, const void* v_prefix,
                              const int64_t* svp, const void* k, const int64_t* sk, const void* v,
                              const int64_t* sv, const void* o, const int64_t* so, const void* dout,
                              const int64_t* sdo, const float* lse, float* delta,
                              cudaStream_t stream) {
  Problem pb{};
  BwdParams p{};
  FA_TRY(check_prefix(prob, P, k_prefix, skp, v_prefix, svp, &pb, &p.pfx));
  const Geo& g = pb.g;
  FA_TRY(check_dense(q, sq, 1, g.Hq, g.rows_q, pb.dtype, p.sq));
  FA_TRY(check_dense(k, sk, 1, g.Hkv, g.rows_k, pb.dtype, p.sk));
  FA_TRY(check_dense(v, sv, 1, g.Hkv, g.rows_k, pb.dtype, p.sv));
  int64_t t[4];
  FA_TRY(check_dense(o, so, 1, g.Hq, g.rows_q, pb.dtype, t));
  FA_TRY(check_dense(dout, sdo, 1, g.Hq, g.rows_q, pb.dtype, p.sdo));
  FA_TRY(check_f32_vec(lse));
  FA_TRY(fa_bwd_preprocess(o, dout, delta, 1, g.Hq, g.rows_q, pb.D, so, sdo, pb.dtype, stream));
  if (pb.dtype == FA_F32 || P >= kFewKeys) return FA_OK;
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.q = q; p.k = k; p.v = v; p.dout = dout; p.lse = lse;
  p.g = g; p.D = pb.D; p.causal = pb.causal; p.scale = pb.scale; p.dtype = pb.dtype;
  p.status = dev->status;
  return launch_few_keys_delta(p, delta, stream);
}

size_t fa_dropout_mask_bytes(const fa_problem* prob) {
  Problem pb{};
  if (check_problem(prob, &pb) != FA_OK || !pb.drop.on) return 0;
  return dropout_mask_bytes(pb.g);
}

fa_status fa_dropout_mask(const fa_problem* prob, uint8_t* mask, size_t bytes,
                          cudaStream_t stream) {
  if (!prob) return FA_ERR_NULL;
  fa_problem pr = *prob;
  pr.dropout_mask = nullptr;           // the buffer being filled is not an input
  Problem pb{};
  FA_TRY(check_problem(&pr, &pb));
  if (!pb.drop.on) return FA_ERR_ARG;
  if (!mask) return FA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(mask) % 16 != 0) return FA_ERR_ALIGN;
  const size_t need = dropout_mask_bytes(pb.g);
  if (need == 0) return FA_ERR_SHAPE;
  if (bytes < need) return FA_ERR_SCRATCH;
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  return launch_dropout_mask(pb.g, pb.causal, pb.drop, mask, dev->status, stream);
}

size_t fa_bwd_fused_workspace_bytes(const fa_problem* prob) {
  Problem pb{};
  if (check_problem(prob, &pb) != FA_OK) return 0;
  return bwd_fused_workspace_floats(pb.g, pb.D) * sizeof(float);
}

fa_status fa_bwd_fused(const fa_problem* prob, const void* q, const int64_t* sq, const void* k,
                       const int64_t* sk, const void* v, const int64_t* sv, const void* dout,
                       const int64_t* sdo, const float* lse, const float* delta, void* dq,
                       const int64_t* sdq, void* dk, const int64_t* sdk, void* dv,
                       const int64_t* sdv, float* dq_accum, size_t workspace_bytes,
                       cudaStream_t stream) {
  Problem pb{};
  FA_TRY(check_problem(prob, &pb));
  if (pb.dtype == FA_F32) return FA_ERR_DTYPE;
  if (!dq_accum) return FA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(dq_accum) % 16 != 0) return FA_ERR_ALIGN;
  if (workspace_bytes < bwd_fused_workspace_floats(pb.g, pb.D) * sizeof(float))
    return FA_ERR_SCRATCH;
  BwdParams p{};
  FA_TRY(prepare_bwd(pb, q, sq, k, sk, v, sv, dout, sdo, lse, delta, dq, sdq, dk, sdk, dv, sdv,
                     &p));
  p.withhold_arrival = g_withhold_next.exchange(0);
  return launch_bwd_fused(p, dq_accum, stream);
}

static fa_status check_rotary(const fa_rotary* r, RotaryParams* out) {
  if (!r) return FA_ERR_NULL;
  FA_TRY(check_shape(r->B, r->Hq, r->N, r->D, r->dtype));
  FA_TRY(check_shape(r->B, r->Hkv, r->N, r->D, r->dtype));
  // rows of a tile of tokens are counted in 32 bits
  if (r->Hq > (1 << 20) || r->Hkv > (1 << 20)) return FA_ERR_SHAPE;
  RotaryParams p{};
  if (r->n_axes < 1 || r->n_axes > 4) return FA_ERR_ARG;
  int64_t pairs = 0;
  for (int64_t i = 0; i < r->n_axes; ++i) {
    if (r->sections[i] < 1 || r->sections[i] > r->D) return FA_ERR_ARG;
    pairs += r->sections[i];
    p.sec_end[i] = static_cast<int>(pairs);
  }
  if (pairs % 8 != 0 || 2 * pairs > r->D) return FA_ERR_ARG;
  if (!r->inv_freq || !r->positions) return FA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(r->inv_freq) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(r->positions) % (r->positions_64 ? 8 : 4) != 0)
    return FA_ERR_ALIGN;
  for (int i = 0; i < 3; ++i)
    if (r->pos_stride[i] < 0) return FA_ERR_STRIDE;
  if ((r->q_weight != nullptr) != (r->k_weight != nullptr)) return FA_ERR_NULL;
  if (r->q_weight) {
    if (reinterpret_cast<uintptr_t>(r->q_weight) % 16 != 0 ||
        reinterpret_cast<uintptr_t>(r->k_weight) % 16 != 0)
      return FA_ERR_ALIGN;
    if (!(std::isfinite(r->eps) && r->eps >= 0.f)) return FA_ERR_ARG;
  }
  p.B = r->B; p.N = r->N; p.Hq = r->Hq; p.Hkv = r->Hkv; p.D = r->D; p.dtype = r->dtype;
  p.pairs = static_cast<int>(pairs);
  p.interleaved = r->interleaved ? 1 : 0;
  p.naxes = static_cast<int>(r->n_axes);
  p.inv_freq = r->inv_freq; p.pos = r->positions; p.pos64 = r->positions_64 ? 1 : 0;
  for (int i = 0; i < 3; ++i) p.ps[i] = r->pos_stride[i];
  p.w[0] = r->q_weight; p.w[1] = r->k_weight;
  p.w_f32 = r->weight_f32 ? 1 : 0;
  p.eps = r->eps;
  *out = p;
  return FA_OK;
}

static fa_status rotary_tensor(const RotaryParams& p, int t, const void* x, const int64_t* s,
                               int64_t* dst) {
  return check_dense(x, s, p.B, t ? p.Hkv : p.Hq, p.N, p.dtype, dst);
}

fa_status fa_rotary_fwd(const fa_rotary* rot, const void* q, const int64_t* sq, const void* k,
                        const int64_t* sk, void* qo, const int64_t* sqo, void* ko,
                        const int64_t* sko, cudaStream_t stream) {
  RotaryParams p{};
  FA_TRY(check_rotary(rot, &p));
  FA_TRY(rotary_tensor(p, 0, q, sq, p.sx[0]));
  FA_TRY(rotary_tensor(p, 1, k, sk, p.sx[1]));
  FA_TRY(rotary_tensor(p, 0, qo, sqo, p.so[0]));
  FA_TRY(rotary_tensor(p, 1, ko, sko, p.so[1]));
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.x[0] = q; p.x[1] = k; p.out[0] = qo; p.out[1] = ko;
  return launch_rotary(p, stream);
}

size_t fa_rotary_bwd_workspace_bytes(const fa_rotary* rot) {
  RotaryParams p{};
  if (check_rotary(rot, &p) != FA_OK || !p.w[0]) return 0;
  return static_cast<size_t>(kRotaryMaxParts) * static_cast<size_t>(p.D) * sizeof(float);
}

fa_status fa_rotary_bwd(const fa_rotary* rot, const void* q, const int64_t* sq, const void* k,
                        const int64_t* sk, const void* dqo, const int64_t* sdqo, const void* dko,
                        const int64_t* sdko, void* dq, const int64_t* sdq, void* dk,
                        const int64_t* sdk, float* dq_weight, float* dk_weight, float* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  RotaryParams p{};
  FA_TRY(check_rotary(rot, &p));
  p.backward = 1;
  if (p.w[0]) {
    FA_TRY(rotary_tensor(p, 0, q, sq, p.sin[0]));
    FA_TRY(rotary_tensor(p, 1, k, sk, p.sin[1]));
    FA_TRY(check_f32_vec(dq_weight));
    FA_TRY(check_f32_vec(dk_weight));
    FA_TRY(check_f32_vec(workspace));
    if (workspace_bytes < fa_rotary_bwd_workspace_bytes(rot)) return FA_ERR_SCRATCH;
  }
  FA_TRY(rotary_tensor(p, 0, dqo, sdqo, p.sx[0]));
  FA_TRY(rotary_tensor(p, 1, dko, sdko, p.sx[1]));
  FA_TRY(rotary_tensor(p, 0, dq, sdq, p.so[0]));
  FA_TRY(rotary_tensor(p, 1, dk, sdk, p.so[1]));
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.in[0] = q; p.in[1] = k; p.x[0] = dqo; p.x[1] = dko; p.out[0] = dq; p.out[1] = dk;
  p.dw[0] = dq_weight; p.dw[1] = dk_weight; p.ws = workspace;
  return launch_rotary(p, stream);
}

// Everything of a decode problem but its tensors.
static fa_status check_decode(const fa_decode_problem* pr, DecodeParams* out) {
  if (!pr) return FA_ERR_NULL;
  if (pr->dtype != FA_F16 && pr->dtype != FA_BF16) return FA_ERR_DTYPE;
  if (pr->B < 1 || pr->Hq < 1 || pr->Hkv < 1 || pr->Hq % pr->Hkv != 0) return FA_ERR_SHAPE;
  if (pr->Nq < 1 || pr->Nq > FA_DECODE_MAX_TOKENS) return FA_ERR_SHAPE;
  if (pr->P < 0 || pr->S < 0) return FA_ERR_SHAPE;
  const int64_t D = pr->D;
  if (D != 16 && D != 32 && D != 64 && D != 128) return FA_ERR_HEADDIM;
  // rows and blocks are counted in 32 bits; TMA rows run up to a tile past P
  const int64_t row_max = (int64_t)INT32_MAX - 1024;
  int64_t t, u;
  if (!mul_ok(pr->B, pr->Hq, &t) || !mul_ok(t, pr->Nq, &t) || t > row_max) return FA_ERR_SHAPE;
  if (pr->P > row_max || pr->S > row_max) return FA_ERR_SHAPE;
  if (!mul_ok(pr->B, pr->Hkv, &u) || !mul_ok(u, pr->S, &u) || !mul_ok(u, D * 8, &u))
    return FA_ERR_SHAPE;
  if (!mul_ok(pr->Hkv, pr->P, &u) || !mul_ok(u, D * 8, &u)) return FA_ERR_SHAPE;
  FA_TRY(check_scale(pr->scale));
  if (pr->S > 0) {
    if (!pr->seq_lens) return FA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pr->seq_lens) % 4 != 0) return FA_ERR_ALIGN;
  }
  DecodeParams p{};
  p.B = pr->B; p.Hkv = pr->Hkv; p.G = pr->Hq / pr->Hkv; p.Nq = pr->Nq; p.D = D;
  p.P = pr->P; p.S = pr->S; p.lens = pr->seq_lens;
  p.causal = pr->causal ? 1 : 0; p.scale = pr->scale; p.dtype = pr->dtype;
  *out = p;
  return FA_OK;
}

size_t fa_decode_workspace_bytes(const fa_decode_problem* prob) {
  DecodeParams p{};
  if (check_decode(prob, &p) != FA_OK) return 0;
  return static_cast<size_t>(decode_plan(p.B, p.Hkv, p.G * p.Nq, p.D, p.P, p.S).floats) * sizeof(float);
}

fa_status fa_decode(const fa_decode_problem* prob, const void* q, const int64_t* sq,
                    const void* k_prefix, const int64_t* skp, const void* v_prefix,
                    const int64_t* svp, const void* k, const int64_t* sk, const void* v,
                    const int64_t* sv, void* o, const int64_t* so, float* lse, float* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  DecodeParams p{};
  FA_TRY(check_decode(prob, &p));
  const int64_t Hq = p.Hkv * p.G;
  FA_TRY(check_dense(q, sq, p.B, Hq, p.Nq, p.dtype, p.sq));
  if (p.P > 0) {
    FA_TRY(check_dense(k_prefix, skp, 1, p.Hkv, p.P, p.dtype, p.skp));
    FA_TRY(check_dense(v_prefix, svp, 1, p.Hkv, p.P, p.dtype, p.svp));
  }
  if (p.S > 0) {
    FA_TRY(check_dense(k, sk, p.B, p.Hkv, p.S, p.dtype, p.sk));
    FA_TRY(check_dense(v, sv, p.B, p.Hkv, p.S, p.dtype, p.sv));
  }
  FA_TRY(check_dense(o, so, p.B, Hq, p.Nq, p.dtype, p.so));
  FA_TRY(check_f32_vec(lse));
  p.plan = decode_plan(p.B, p.Hkv, p.G * p.Nq, p.D, p.P, p.S);
  const size_t need = static_cast<size_t>(p.plan.floats) * sizeof(float);
  if (need > 0) {
    FA_TRY(check_f32_vec(workspace));
    if (workspace_bytes < need) return FA_ERR_SCRATCH;
  }
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  p.q = q; p.kp = k_prefix; p.vp = v_prefix; p.k = k; p.v = v; p.o = o; p.lse = lse;
  p.ws = workspace;
  p.status = dev->status; p.timeout_ns = g_timeout_ns.load();
  return launch_decode(p, stream);
}

fa_status fa_get_device_status(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return FA_ERR_LAUNCH;
  DeviceInfo* dev = nullptr;
  FA_TRY(device_setup(&dev));
  unsigned int word = 0;
  if (cudaMemcpyFromSymbol(&word, fa_device_status_word, sizeof(word)) != cudaSuccess)
    return FA_ERR_LAUNCH;
  if (word != 0) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(fa_device_status_word, &zero, sizeof(zero)) != cudaSuccess)
      return FA_ERR_LAUNCH;
  }
  return static_cast<fa_status>(word);
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_NULL: return "FA_ERR_NULL: a required pointer is NULL";
    case FA_ERR_SHAPE: return "FA_ERR_SHAPE: B, H or N < 1, or sizes overflow";
    case FA_ERR_HEADDIM: return "FA_ERR_HEADDIM: D must be 16, 32, 64 or 128";
    case FA_ERR_DTYPE: return "FA_ERR_DTYPE: unknown dtype";
    case FA_ERR_STRIDE: return "FA_ERR_STRIDE: d-stride must be 1 and strides non-negative";
    case FA_ERR_ALIGN: return "FA_ERR_ALIGN: bases and strides must be 16-byte multiples";
    case FA_ERR_LAUNCH: return "FA_ERR_LAUNCH: CUDA error configuring or launching a kernel";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a device-side bounded wait ran out";
    case FA_ERR_ARCH: return "FA_ERR_ARCH: the current device is not sm_103";
    case FA_ERR_SCALE: return "FA_ERR_SCALE: scale must be finite and > 0";
    case FA_ERR_ARG: return "FA_ERR_ARG: invalid argument";
    case FA_ERR_SCRATCH:
      return "FA_ERR_SCRATCH: B*H*N exceeds FA_NOALLOC_MAX_ROWS, or the workspace is too small";
    case FA_ERR_SEQLENS: return "FA_ERR_SEQLENS: packed sequence offsets are inconsistent";
  }
  return "unknown fa_status";
}

fa_status fa_set_path(fa_path path) {
  if (path != FA_PATH_AUTO && path != FA_PATH_FFMA) return FA_ERR_ARG;
  g_path.store(path);
  return FA_OK;
}

void fa_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns ? ns : kDefaultTimeoutNs); }

void fa_set_profile_events(const cudaEvent_t* events) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (events) {
    for (int i = 0; i < 3; ++i) g_prof_events[i] = events[i];
    g_prof_on.store(true);
  } else {
    g_prof_on.store(false);
  }
}

void fa_test_withhold_next_arrival(void) { g_withhold_next.store(1); }

void fa_test_set_l2_bytes(int64_t bytes) { g_l2_override.store(bytes > 0 ? bytes : 0); }

int fa_version(void) { return 0x000400; }

}  // extern "C"
